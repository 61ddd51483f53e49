"""CPU tests of the serving calls' refusals: bad arguments are rejected on the
host, by status, before any device work (no GPU is needed or touched)."""
import ctypes

import pytest

OK, INVALID, WORKSPACE = 0, 1, 4
A = 1 << 20          # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import moe_gemm_gb300 as w8
    return w8.lib()


def call(f, order, base, **change):
    args = dict(base, **change)
    return f(*[args[n] for n in order])


GATE = "logits dtype ld T E k score bias n_group topk_group renorm scale ids w stream".split()
GATE_OK = dict(logits=A, dtype=1, ld=64, T=0, E=64, k=8, score=0, bias=None, n_group=8,
               topk_group=4, renorm=1, scale=1.0, ids=A, w=A, stream=None)


def test_gate(lib):
    f = lib.w8a8_moe_gate
    assert call(f, GATE, GATE_OK) == OK                      # no tokens
    assert call(f, GATE, GATE_OK, logits=None, ids=None) == OK
    for bad in (dict(dtype=2), dict(ld=63), dict(T=-1), dict(E=0), dict(E=1025, ld=2048, n_group=1),
                dict(k=0), dict(k=65), dict(k=33, E=64, topk_group=4), dict(score=2),
                dict(n_group=0), dict(n_group=7), dict(n_group=128), dict(topk_group=0),
                dict(topk_group=9), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(T=1 << 31), dict(T=1, logits=None), dict(T=1, logits=A + 2), dict(T=1, ids=None),
                dict(T=1, w=A + 1), dict(T=1, bias=A + 2)):
        assert call(f, GATE, GATE_OK, **bad) == INVALID, bad


PLAN = ("table lens target free n_free B W P page n_tokens cu kv slots positions stream").split()
PLAN_OK = dict(table=A, lens=A, target=A, free=A, n_free=A, B=4, W=8, P=64, page=16, n_tokens=10,
               cu=A, kv=A, slots=A, positions=A, stream=None)


def test_plan(lib):
    f = lib.w8a8_paged_kv_plan
    for bad in (dict(B=-1), dict(B=4097), dict(W=0), dict(P=0), dict(page=0), dict(n_tokens=-1),
                dict(n_tokens=1 << 31), dict(W=1 << 27), dict(P=1 << 27), dict(table=None),
                dict(lens=None), dict(target=None), dict(free=None), dict(n_free=None),
                dict(cu=None), dict(kv=None), dict(slots=None), dict(positions=None),
                dict(table=A + 2), dict(slots=A + 1), dict(n_free=A + 3)):
        assert call(f, PLAN, PLAN_OK, **bad) == INVALID, bad


WRITE = ("k kt kh v vt vh slots T Hkv d P page kc ks vc vs stream").split()
WRITE_OK = dict(k=A, kt=1024, kh=128, v=A, vt=1024, vh=128, slots=A, T=0, Hkv=8, d=128, P=10,
                page=64, kc=A, ks=A, vc=A, vs=A, stream=None)


def test_write(lib):
    f = lib.w8a8_paged_kv_write
    assert call(f, WRITE, WRITE_OK) == OK
    assert call(f, WRITE, WRITE_OK, ks=None, vs=None) == OK
    for bad in (dict(T=-1), dict(Hkv=0), dict(Hkv=65536), dict(d=64), dict(P=0), dict(page=0),
                dict(P=1 << 26), dict(T=1 << 30), dict(kt=1028), dict(vh=4), dict(vt=-8),
                dict(ks=None), dict(vs=None), dict(T=1, k=None), dict(T=1, v=A + 8),
                dict(T=1, slots=None), dict(T=1, kc=A + 4), dict(T=1, vc=None),
                dict(T=1, ks=A + 2), dict(T=1, slots=A + 2)):
        assert call(f, WRITE, WRITE_OK, **bad) == INVALID, bad


ATT = ("q qt qh kc ks vc vs table kv cu T B W Hq Hkv d P page scale window out dtype ws wsb "
       "stream").split()
ATT_OK = dict(q=A, qt=8192, qh=128, kc=A, ks=A, vc=A, vs=A, table=A, kv=A, cu=A, T=0, B=2, W=8,
              Hq=64, Hkv=8, d=128, P=32, page=64, scale=0.1, window=0, out=A, dtype=0, ws=A,
              wsb=1 << 40, stream=None)


def test_attention(lib):
    f = lib.w8a8_attention_paged
    assert call(f, ATT, ATT_OK) == OK
    for bad in (dict(T=-1), dict(B=0), dict(B=65536), dict(W=0), dict(Hq=0), dict(Hkv=0),
                dict(Hq=60), dict(Hq=17 * 8), dict(d=64), dict(P=0), dict(page=0), dict(page=12),
                dict(page=4), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(window=-1), dict(dtype=2), dict(qt=4), dict(qh=-8),
                dict(ks=None), dict(vs=None), dict(W=1 << 26), dict(P=1 << 24), dict(T=1 << 26),
                dict(T=1, q=None), dict(T=1, q=A + 8), dict(T=1, kc=A + 4), dict(T=1, ks=A + 4),
                dict(T=1, out=None), dict(T=1, out=A + 4), dict(T=1, table=None),
                dict(T=1, kv=A + 2), dict(T=1, cu=None), dict(window=1 << 31)):
        assert call(f, ATT, ATT_OK, **bad) == INVALID, bad
    need = lib.w8a8_attention_paged_workspace_size(1, 2, 64, 8)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=A + 8), dict(wsb=need - 1)):
        assert call(f, ATT, dict(ATT_OK, T=1), **bad) == WORKSPACE, bad


def test_workspace_size(lib):
    f = lib.w8a8_attention_paged_workspace_size
    assert f(0, 2, 64, 8) == 0 and f(1, 0, 64, 8) == 0 and f(1, 2, 60, 8) == 0
    assert f(1, 1, 64, 8) % 16 == 0
    # it depends on the grid and the tile, not on lengths or requests
    assert f(1, 1, 64, 8) == f(1, 1000, 64, 8)


def test_binding_refuses_host_tensors(lib):
    import torch

    import moe_gemm_gb300 as w8
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        w8.moe_gate(x, 8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        w8.paged_kv_plan(torch.zeros(2, 4, dtype=torch.int32), i, i, i, i, 16, 1)
    k = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w8.paged_kv_write(k, k, i[:1], c, c)
    with pytest.raises(ValueError):
        w8.attention_paged(k, c, c, torch.zeros(1, 4, dtype=torch.int32), i[:1], i, 0.1)
