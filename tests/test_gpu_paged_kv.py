"""GPU tests of the paged KV cache: the plan (block tables, free pages, slots)
against a sequential restatement of its rules, whole numbers equal; the write
against the definition (codes and scales bit for bit; the contiguous cache's
quantizer on the same vectors).

Source: "Deploying Hunyuan 770B in INT8 on domestic accelerators" §3.4.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import moe_gemm_gb300 as w8  # noqa: E402

DEV = torch.device("cuda:0")
D = 128


def plan_rules(table, lens, target, free, n_free, page, n_tokens):
    """The plan, one request after the other (numpy / python integers)."""
    table, free, lens = table.copy(), free.copy(), list(lens)
    B, W = table.shape
    P = len(free)
    n_free = min(max(n_free, 0), P)
    pages = lambda n: -(-n // page)  # noqa: E731
    bad = [lens[b] < 0 or target[b] < 0 or pages(lens[b]) > W for b in range(B)]
    kv = [0 if bad[b] else target[b] for b in range(B)]
    held = list(lens)
    for b in range(B):
        if not bad[b] and target[b] < held[b]:
            for j in range(pages(target[b]), pages(held[b])):
                if n_free < P:
                    free[n_free] = table[b, j]
                    n_free += 1
                table[b, j] = -1
            lens[b] = target[b]
    cu, slots, positions, need, top = [0], [], [], 0, n_free
    for b in range(B):
        n = max(0, target[b] - held[b]) if held[b] >= 0 else 0
        cu.append(cu[-1] + n)
        if n == 0:
            continue
        ok = not bad[b] and pages(target[b]) <= W and cu[-1] <= n_tokens
        if ok:
            more = pages(target[b]) - pages(held[b])
            need += more
            ok = more == 0 or need <= top
        if not ok:
            kv[b] = 0
            slots += [-1] * n
            positions += [-1] * n
            continue
        for j in range(pages(held[b]), pages(target[b])):
            n_free -= 1
            table[b, j] = free[n_free]
        lens[b] = target[b]
        for p in range(held[b], target[b]):
            slots.append(int(table[b, p // page]) * page + p % page)
            positions.append(p)
    slots = (slots + [-1] * n_tokens)[:n_tokens]
    positions = (positions + [-1] * n_tokens)[:n_tokens]
    return table, lens, free, n_free, cu, kv, slots, positions


def make(B, W, P, page, lens, n_free, seed=0):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((B, W), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        n = -(-max(lens[b], 0) // page)
        if n <= W:
            table[b, :n] = ids[at:at + n]
            at += n
    free = np.full(P, -5, dtype=np.int32)
    free[:n_free] = ids[at:at + n_free]
    return table, free


def run_plan(table, lens, target, free, n_free, page, n_tokens, **kw):
    dev = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)  # noqa: E731
    t, l, g, f, nf = dev(table), dev(lens), dev(target), dev(free), dev([n_free])
    cu, kv, slots, pos = w8.paged_kv_plan(t, l, g, f, nf, page, n_tokens, **kw)
    torch.cuda.synchronize()
    return (t.cpu().numpy(), l.cpu().tolist(), f.cpu().numpy(), int(nf.item()),
            cu.cpu().tolist(), kv.cpu().tolist(), slots.cpu().tolist(), pos.cpu().tolist())


def check_plan(table, lens, target, free, n_free, page, n_tokens):
    got = run_plan(table, lens, target, free, n_free, page, n_tokens)
    want = plan_rules(table, lens, target, free, n_free, page, n_tokens)
    for name, a, b in zip("table lens free n_free cu kv slots positions".split(), got, want):
        assert np.array_equal(np.asarray(a), np.asarray(b)), name
    return got


@pytest.mark.parametrize("B,page,seed", [(1, 16, 0), (7, 8, 1), (32, 64, 2), (300, 16, 3),
                                         (1024, 32, 4), (2049, 1, 5), (4096, 16, 6)])
def test_plan_mixed(B, page, seed):
    rng = np.random.default_rng(seed)
    W = 12
    lens = rng.integers(0, W * page + 1, B)
    target = np.clip(lens + rng.integers(-3 * page, 3 * page + 2, B), 0, W * page + 2)
    target[rng.random(B) < 0.2] = 0
    used = int((-(-lens // page)).sum())
    n_free = 2 * B
    table, free = make(B, W, used + n_free + 3, page, lens, n_free, seed)
    n_tokens = int(np.maximum(target - lens, 0).sum())
    check_plan(table, lens.tolist(), target.tolist(), free, n_free, page, n_tokens)


@pytest.mark.parametrize("n_free", [0, 1, 2, 3, 5])
def test_plan_tight_pool(n_free):
    lens, target = [15, 16, 0, 31, 16], [16, 33, 17, 32, 5]
    table, free = make(5, 4, 20, 16, lens, n_free)
    got = check_plan(table, lens, target, free, n_free, 16, 1 + 17 + 17 + 1)
    if n_free == 0:
        # nothing free and nothing given back (16 -> 5 keeps its page): those
        # that need pages are refused, those that do not are served
        assert got[5] == [16, 0, 0, 32, 5]


def test_plan_uses_pages_given_back_in_the_same_call():
    lens, target = [40, 0], [0, 48]
    table, free = make(2, 4, 3, 16, lens, 0)
    got = check_plan(table, lens, target, free, 0, 16, 48)
    assert got[5] == [0, 48] and got[3] == 0


def test_plan_impossible_lengths():
    # negative, past the row, and a target past the row
    lens, target = [-1, 3, 200, 10, 10, 16], [5, -2, 210, 65, 11, 16]
    table, free = make(6, 4, 40, 16, lens, 9)
    check_plan(table, lens, target, free, 9, 16, 200)


@pytest.mark.parametrize("n_tokens", [0, 1, 19, 20, 30])
def test_plan_tokens_past_the_buffer(n_tokens):
    lens, target = [3, 0, 5], [13, 10, 15]
    table, free = make(3, 2, 9, 16, lens, 5)
    check_plan(table, lens, target, free, 5, 16, n_tokens)


def test_plan_no_requests_and_repeat():
    cu, kv, slots, pos = w8.paged_kv_plan(
        torch.empty((0, 4), dtype=torch.int32, device=DEV),
        *(torch.empty(0, dtype=torch.int32, device=DEV) for _ in range(2)),
        torch.arange(4, dtype=torch.int32, device=DEV),
        torch.tensor([4], dtype=torch.int32, device=DEV), 16, 3)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and pos.tolist() == [-1] * 3
    # the same call twice gives the same answer
    lens, target = list(range(0, 640, 2)), list(range(1, 960, 3))
    table, free = make(320, 70, 20000, 16, lens, 9000)
    a = run_plan(table, lens, target, free, 9000, 16, 5000)
    b = run_plan(table, lens, target, free, 9000, 16, 5000)
    assert all(np.array_equal(np.asarray(x), np.asarray(y)) for x, y in zip(a, b))


def _definition(x):
    """INT8 codes and scales of BF16 vectors, binary32 arithmetic."""
    x = x.float().cpu().numpy()
    s = np.abs(x).max(-1, keepdims=True) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.rint(x / s), 0)
    return np.clip(c, -127, 127).astype(np.int8), s[..., 0]


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("T,Hkv,page", [(1, 1, 16), (3, 8, 64), (17, 2, 8), (130, 5, 24), (64, 1, 3)])
def test_write(T, Hkv, page, int8):
    g = torch.Generator().manual_seed(T)
    qkv = torch.randn(T, 3 * Hkv + 1, D, generator=g) * 3
    qkv[0, Hkv] = 0
    qkv[-1, -1] *= 1e-38                                   # subnormal scale
    qkv = qkv.to(torch.bfloat16).to(DEV)
    k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv + 1:]       # parts of one projection
    P = T // page + 5
    slots = torch.randperm(P * page, generator=g)[:T].to(torch.int32)
    if T > 2:
        slots[1] = -1
        slots[2] = P * page
    dt = torch.int8 if int8 else torch.bfloat16
    kc = torch.full((P, Hkv, page, D), 7, dtype=dt, device=DEV)
    vc = torch.full_like(kc, 9)
    ks = torch.full((P, Hkv, page), -1.0, device=DEV) if int8 else None
    vs = torch.full((P, Hkv, page), -2.0, device=DEV) if int8 else None
    w8.paged_kv_write(k, v, slots.to(DEV), kc, vc, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for x, cache, scales, fill, sfill in ((k, kc, ks, 7, -1.0), (v, vc, vs, 9, -2.0)):
        got = cache.cpu().transpose(1, 2).reshape(P * page, Hkv, D)
        want = torch.full_like(got, fill)
        idx = [t for t in range(T) if 0 <= int(slots[t]) < P * page]
        at = slots[idx].long()
        if int8:
            codes, s = _definition(x)
            want[at] = torch.from_numpy(codes[idx])
            sg = scales.cpu().transpose(1, 2).reshape(P * page, Hkv)
            sw = torch.full_like(sg, sfill)
            sw[at] = torch.from_numpy(s[idx])
            assert torch.equal(sg, sw)
            assert torch.equal(got, want)
        else:
            want[at] = x.cpu()[idx]
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_write_matches_the_contiguous_cache():
    g = torch.Generator().manual_seed(5)
    T, Hkv, page, P = 40, 2, 16, 6
    k = (torch.randn(T, Hkv, D, generator=g) * 2).to(torch.bfloat16).to(DEV)
    slots = torch.randperm(P * page, generator=g)[:T].to(torch.int32).to(DEV)
    kc = torch.zeros(P, Hkv, page, D, dtype=torch.int8, device=DEV)
    vc, ks = torch.zeros_like(kc), torch.zeros(P, Hkv, page, device=DEV)
    vs = torch.zeros_like(ks)
    w8.paged_kv_write(k, k, slots, kc, vc, k_scale=ks, v_scale=vs)
    kc2, ks2 = torch.zeros_like(kc), torch.zeros_like(ks)
    rows = ((slots // page)[:, None] * Hkv + torch.arange(Hkv, device=DEV)) * page \
        + (slots % page)[:, None]
    w8.kv_quant(k.view(-1, D), kc2, ks2, dst_rows=rows.to(torch.int32).flatten())
    torch.cuda.synchronize()
    assert torch.equal(kc, kc2) and torch.equal(ks, ks2) and torch.equal(vc, kc2)


def test_write_past_32_bit_offsets():
    # 40960 pages of 8 heads x 64 positions: the last page's bytes lie past 2^31
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    P, Hkv, page = 40960, 8, 64
    kc = torch.empty(P, Hkv, page, D, dtype=torch.int8, device=DEV)
    vc = torch.empty_like(kc)
    ks = torch.empty(P, Hkv, page, device=DEV)
    vs = torch.empty_like(ks)
    k = torch.randn(2, Hkv, D, device=DEV).to(torch.bfloat16)
    slots = torch.tensor([P * page - 1, 5], dtype=torch.int32, device=DEV)
    w8.paged_kv_write(k, k, slots, kc, vc, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    codes, s = _definition(k)
    for t, (p, off) in enumerate([(P - 1, page - 1), (0, 5)]):
        assert np.array_equal(vc[p, :, off].cpu().numpy(), codes[t])
        assert np.array_equal(ks[p, :, off].cpu().numpy(), s[t])


def test_plan_then_write_in_a_graph():
    page, P, B = 16, 32, 3
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    table = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(P, dtype=torch.int32, device=DEV)
    n_free = torch.tensor([P], dtype=torch.int32, device=DEV)
    step = torch.tensor([5, 1, 20], dtype=torch.int32, device=DEV)
    k = torch.randn(26, 2, D, device=DEV).to(torch.bfloat16)
    kc = torch.zeros(P, 2, page, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    target = torch.empty_like(lens)

    def one():
        torch.add(lens, step, out=target)
        cu, kv, slots, pos = w8.paged_kv_plan(table, lens, target, free, n_free, page, 26)
        w8.paged_kv_write(k, k, slots, kc, vc)
        return slots

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slots = one()
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [5 * (i + 1), i + 1, 20 * (i + 1)]
        s = slots.tolist()
        assert len(set(s)) == 26 and min(s) >= 0
        flat = kc.transpose(1, 2).reshape(P * page, 2, D)
        assert torch.equal(flat[slots.long()], k)
    held = sorted(t for t in table.flatten().tolist() if t >= 0)
    assert sorted(held + free[:int(n_free)].tolist()) == list(range(P))


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("T,Hkv,page", [(8192, 5, 16), (16385, 2, 24), (32768, 1, 64), (4096, 8, 128),
                                        (5000, 7, 8)])
def test_write_of_long_prompts(T, Hkv, page, int8):
    # several heads per warp, their last ones fewer; some tokens without a slot
    g = torch.Generator(device=DEV).manual_seed(T + Hkv)
    qkv = (torch.randn(T, 2 * Hkv + 3, D, generator=g, device=DEV) * 3).to(torch.bfloat16)
    qkv[5] = 0
    qkv[6] *= 1e-38
    k, v = qkv[:, 1:1 + Hkv], qkv[:, 2 + Hkv:2 + 2 * Hkv]
    P = T // page + 5
    slots = torch.randperm(P * page, generator=g, device=DEV)[:T].to(torch.int32)
    slots[3::97] = -1
    slots[4::89] = P * page
    dt = torch.int8 if int8 else torch.bfloat16
    kc = torch.full((P, Hkv, page, D), 7, dtype=dt, device=DEV)
    vc = torch.full_like(kc, 9)
    ks = torch.full((P, Hkv, page), -1.0, device=DEV) if int8 else None
    vs = torch.full((P, Hkv, page), -2.0, device=DEV) if int8 else None
    w8.paged_kv_write(k, v, slots, kc, vc, k_scale=ks, v_scale=vs)
    has = (slots >= 0) & (slots < P * page)
    at = slots[has].long()
    for x, cache, scales, fill, sfill in ((k, kc, ks, 7, -1.0), (v, vc, vs, 9, -2.0)):
        got = cache.transpose(1, 2).reshape(P * page, Hkv, D)
        want = torch.full_like(got, fill)
        if int8:
            codes, s = _definition(x[has])
            want[at] = torch.from_numpy(codes).to(DEV)
            sw = torch.full((P * page, Hkv), sfill, device=DEV)
            sw[at] = torch.from_numpy(s).to(DEV)
            assert torch.equal(scales.transpose(1, 2).reshape(P * page, Hkv), sw)
            assert torch.equal(got, want)
        else:
            want[at] = x[has]
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_plan_with_room_for_the_most_tokens():
    n = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table, lens = torch.full((1, 4), -1, dtype=torch.int32, device=DEV), one(0)
    cu, kv, slots, pos = w8.paged_kv_plan(table, lens, one(20), one(2, 0, 1), one(3), 16, n)
    assert cu.tolist() == [0, 20] and kv.tolist() == [20] and table.tolist() == [[1, 0, -1, -1]]
    assert slots[:20].tolist() == [16 + i for i in range(16)] + [0, 1, 2, 3]
    assert pos[:20].tolist() == list(range(20))
    assert slots.shape == pos.shape == (n,)
    assert int(slots[20:].max()) == int(slots[20:].min()) == -1
    assert int(pos[20:].max()) == int(pos[20:].min()) == -1
