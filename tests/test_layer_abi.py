"""CPU tests of the refusals of a decoder layer's calls: bad arguments are rejected on the
host, by status, before any device work; and a rule of their sources."""
import os
import re

import pytest

OK, INVALID, WORKSPACE = 0, 1, 4
A = 1 << 20          # an aligned address that is never read
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_gemm_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import moe_gemm_gb300 as w8
    return w8.lib()


def call(f, order, base, **change):
    args = dict(base, **change)
    return f(*[args[n] for n in order])


APPEND = ("q qt qh Hq k kt kh v vt vh positions slots inv_freq rot interleaved amplitude T Hkv d P "
          "page out ot oh kc ks vc vs stream").split()
APPEND_OK = dict(q=A, qt=8192, qh=128, Hq=64, k=A, kt=1024, kh=128, v=A, vt=1024, vh=128,
                 positions=A, slots=A, inv_freq=A, rot=128, interleaved=0, amplitude=1.0, T=0,
                 Hkv=8, d=128, P=10, page=64, out=A, ot=8192, oh=128, kc=A, ks=A, vc=A, vs=A,
                 stream=None)


def test_append(lib):
    f = lib.w8a8_paged_kv_append
    assert call(f, APPEND, APPEND_OK) == OK                      # no tokens
    assert call(f, APPEND, APPEND_OK, ks=None, vs=None, q=None, out=None, Hq=0) == OK
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hq=65536), dict(Hkv=0), dict(Hkv=65536), dict(d=64),
                dict(P=0), dict(page=0), dict(P=1 << 26), dict(T=1 << 30), dict(rot=0),
                dict(rot=8), dict(rot=24), dict(rot=144), dict(amplitude=float("inf")),
                dict(qt=4), dict(qh=-8), dict(kt=1028), dict(vh=4), dict(ot=12), dict(oh=-8),
                dict(ks=None), dict(vs=None), dict(T=1, q=None), dict(T=1, out=None),
                dict(T=1, q=A + 8), dict(T=1, out=A + 8), dict(T=1, k=None), dict(T=1, v=A + 8),
                dict(T=1, positions=None), dict(T=1, positions=A + 2), dict(T=1, slots=None),
                dict(T=1, inv_freq=None), dict(T=1, inv_freq=A + 1), dict(T=1, kc=A + 4),
                dict(T=1, vc=None), dict(T=1, ks=A + 2)):
        assert call(f, APPEND, APPEND_OK, **bad) == INVALID, bad


def test_append_outputs_apart(lib):
    f = lib.w8a8_paged_kv_append
    for bad in (dict(T=2, ot=0), dict(T=2, ot=120), dict(oh=0), dict(oh=64)):
        assert call(f, APPEND, APPEND_OK, **bad) == INVALID, bad
    for good in (dict(Hq=1, oh=0), dict(ot=0), dict(Hq=0, q=None, out=None, ot=0, oh=0)):
        assert call(f, APPEND, APPEND_OK, **good) == OK, good


# A projection's rows: 64 query, 8 key and 8 value heads of 128 side by side, in bytes from A.
QKV = dict(APPEND_OK, T=3, qt=10240, kt=10240, vt=10240, ot=10240, k=A + 64 * 256, v=A + 72 * 256)
AWAY = A + (1 << 24)


def written_rows_are_refused(lib, **change):
    """Whether the call is refused for its operands; without a GPU, one that is not is for that."""
    return call(lib.w8a8_paged_kv_append, APPEND, QKV, **change) == INVALID


def brute_force(T, a, b, same):
    """Whether two rows of 128 share memory; a, b: (address, token stride, head stride, heads)."""
    def rows(x):
        return [x[0] // 2 + t * x[1] + h * x[2] for t in range(T) for h in range(x[3])]
    p, q = rows(a), rows(b)
    return any(abs(x - y) < 128 and not (same and i == j)
               for i, x in enumerate(p) for j, y in enumerate(q))


def test_append_rows_that_share_memory(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that are not refused would run on addresses that are none")
    for bad in (dict(out=AWAY, Hq=2, T=2, ot=128, oh=128), dict(out=AWAY, Hq=3, T=2, ot=256, oh=128),
                dict(out=AWAY, Hq=2, T=4, ot=128, oh=384),          # rows of q_out
                dict(out=A + 256), dict(out=A - 256), dict(out=A + 240), dict(ot=10368), dict(oh=256),
                dict(ot=8192), dict(out=A + 10240 * 2), dict(qh=256),   # q_out and q
                dict(out=A + 70 * 256, Hq=2), dict(q=AWAY, k=A), dict(q=AWAY, v=A + 63 * 256),
                dict(q=AWAY, k=A + 200 * 256)):                     # q_out and k or v
        assert written_rows_are_refused(lib, **bad), bad
    for good in (dict(), dict(T=1), dict(T=1, ot=0), dict(out=AWAY), dict(out=AWAY, ot=8192),
                 dict(out=AWAY, ot=128, oh=384), dict(out=AWAY, Hq=2, T=4, ot=256, oh=128),
                 dict(out=AWAY, Hq=2, T=3, ot=128, oh=384), dict(Hq=0, q=None, out=None),
                 dict(Hq=1, oh=0, qh=128), dict(q=AWAY), dict(q=AWAY, out=A + 3 * 20480 - 16, k=AWAY, v=AWAY)):
        assert not written_rows_are_refused(lib, **good), good


def test_append_rows_against_every_pair(lib):
    # where strides agree, the answer is that of a comparison of every two rows
    import random

    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that are not refused would run on addresses that are none")
    rng = random.Random(7)
    seen = set()
    for _ in range(3000):
        T, Hq, Hkv = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 3)
        ts, hs = 8 * rng.randint(16, 160), 8 * rng.randint(16, 90)
        kh = rng.choice([hs, 8 * rng.randint(0, 90)])
        out = A + 16 * rng.randint(-200, 200)
        q, k = A + 16 * rng.randint(-500, 500), A + 16 * rng.randint(-500, 500)
        if rng.random() < 0.2:
            q = out
        if rng.random() < 0.5:
            q = AWAY
        got = written_rows_are_refused(lib, T=T, Hq=Hq, Hkv=Hkv, q=q, k=k, v=AWAY * 2, out=out, qt=ts,
                                       kt=ts, vt=ts, ot=ts, qh=hs, oh=hs, kh=kh, vh=kh)
        o = (out, ts, hs, Hq)
        want = (brute_force(T, o, o, True) or brute_force(T, o, (q, ts, hs, Hq), q == out)
                or brute_force(T, o, (k, ts, kh, Hkv), False))
        assert got == want, (T, Hq, Hkv, ts, hs, kh, out, q, k)
        seen.add((got, q == out))
    assert len(seen) == 4


LAYER = ("x ldx logits ldt ld T k H I E score bias n_group topk_group renorm scale qu su qd sd ids "
         "w y ydt ws wsb stream").split()
LAYER_OK = dict(x=A, ldx=1024, logits=A, ldt=1, ld=64, T=0, k=8, H=1024, I=512, E=64, score=0,
                bias=None, n_group=1, topk_group=1, renorm=1, scale=1.0, qu=A, su=A, qd=A, sd=A,
                ids=A, w=A, y=A, ydt=0, ws=A, wsb=1 << 40, stream=None)


def test_layer(lib):
    f = lib.w8a8_moe_layer
    assert call(f, LAYER, LAYER_OK) == OK
    for bad in (dict(T=-1), dict(k=0), dict(k=65), dict(H=1000), dict(I=0), dict(I=100),
                dict(I=8320), dict(E=0), dict(E=1025), dict(E=4), dict(ld=63), dict(ldt=2),
                dict(ydt=2), dict(score=3), dict(n_group=7), dict(topk_group=2),
                dict(scale=float("nan")), dict(ldx=1023), dict(T=1, x=None), dict(T=1, x=A + 1),
                dict(T=1, logits=None), dict(T=1, qu=A + 8), dict(T=1, qd=None), dict(T=1, su=A + 2),
                dict(T=1, sd=None), dict(T=1, ids=None), dict(T=1, w=A + 2), dict(T=1, y=A + 8),
                dict(T=1, bias=A + 1)):
        assert call(f, LAYER, LAYER_OK, **bad) == INVALID, bad
    for T in (1, 32, 33):
        need = lib.w8a8_moe_layer_workspace_size(T, 8, 1024, 512, 64)
        assert need > 0 and need % 256 == 0
        for bad in (dict(ws=None), dict(ws=A + 128), dict(wsb=need - 1)):
            assert call(f, LAYER, dict(LAYER_OK, T=T), **bad) == WORKSPACE, bad
    assert lib.w8a8_moe_layer_workspace_size(0, 8, 1024, 512, 64) == 0
    assert lib.w8a8_moe_layer_workspace_size(4, 8, 1000, 512, 64) == 0


@pytest.mark.parametrize("name", ["paged_append.cu", "moe_layer.cu", "quant_fp8.cu", "gemm_fp8.cu"])
def test_no_read_only_loads(name):
    # They start while the kernel before may still write what they read.
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"__ldg|ld\.global(?:\.\w+)*\.nc|__restrict__", code) == []


def test_binding_refuses_host_tensors(lib):
    import torch

    import moe_gemm_gb300 as w8
    i = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w8.paged_kv_append(k, k, k, i, i, torch.zeros(64), c, c)
    x = torch.zeros(1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w8.moe_layer(x, torch.zeros(1, 4), 1, torch.zeros(4, 256, 128, dtype=torch.int8),
                     torch.zeros(4, 256, 1), torch.zeros(4, 128, 128, dtype=torch.int8),
                     torch.zeros(4, 128, 1))


GEMM8 = "qa sa qw sw y dtype M N K stream".split()
GEMM8_OK = dict(qa=A, sa=A, qw=A, sw=A, y=A, dtype=0, M=0, N=1000, K=512, stream=None)
LINEAR8 = "a lda mode qw sw y dtype M N K ws wsb stream".split()
LINEAR8_OK = dict(a=A, lda=512, mode=0, qw=A, sw=A, y=A, dtype=0, M=0, N=1000, K=512, ws=A,
                  wsb=1 << 40, stream=None)


def test_fp8(lib):
    f = lib.w8a8_gemm_fp8
    assert call(f, GEMM8, GEMM8_OK) == OK
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=500), dict(dtype=2), dict(M=1 << 23),
                dict(N=1 << 22), dict(M=1 << 21, K=128, N=1 << 10), dict(M=1, qa=None),
                dict(M=1, qa=A + 8), dict(M=1, sa=None), dict(M=1, sa=A + 2), dict(M=1, qw=A + 4),
                dict(M=1, sw=None), dict(M=1, y=None), dict(M=1, y=A + 1),
                dict(M=1, y=A + 2, dtype=1)):
        assert call(f, GEMM8, GEMM8_OK, **bad) == INVALID, bad
    f = lib.w8a8_linear_fp8
    assert call(f, LINEAR8, LINEAR8_OK) == OK
    for bad in (dict(mode=2), dict(lda=511), dict(K=64), dict(M=1, a=None), dict(M=1, a=A + 1),
                dict(M=-1), dict(M=1 << 20, lda=1 << 20)):
        assert call(f, LINEAR8, LINEAR8_OK, **bad) == INVALID, bad
    need = lib.w8a8_linear_fp8_workspace_size(3, 1000, 512)
    assert need == 3 * 512 + 256
    for bad in (dict(ws=None), dict(ws=A + 64), dict(wsb=need - 1)):
        assert call(f, LINEAR8, dict(LINEAR8_OK, M=3), **bad) == WORKSPACE, bad
    f = lib.w8a8_quant_act_fp8
    order = "a M K lda qa sa mode stream".split()
    ok = dict(a=A, M=0, K=256, lda=256, qa=A, sa=A, mode=0, stream=None)
    assert call(f, order, ok) == OK
    for bad in (dict(M=-1), dict(K=200), dict(lda=255), dict(mode=3), dict(M=1, qa=A + 8),
                dict(M=1, a=None), dict(M=1, sa=A + 2)):
        assert call(f, order, ok, **bad) == INVALID, bad
    f = lib.w8a8_quant_weight_fp8
    order = "w N K mode qw sw stream".split()
    ok = dict(w=A, N=0, K=256, mode=0, qw=A, sw=A, stream=None)
    assert call(f, order, ok) == OK
    for bad in (dict(N=-1), dict(K=200), dict(mode=3), dict(N=1, w=A + 8), dict(N=1, qw=None),
                dict(N=65535 * 128 + 1, K=128)):
        assert call(f, order, ok, **bad) == INVALID, bad
