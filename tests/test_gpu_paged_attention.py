"""GPU tests of attention over the paged KV cache against the definition in 64
bits, per output:

  |out - out*| <= (2 A (D + 2) 2^-24 + 2 A E + (S + 64) 2^-24 + 16 * 2^-22
                   + R) T + U S V + H |out*|

with A the largest sum_d |scale q_d k_jd| of the row's visible keys (a score is
a 128-term FP32 sum of exact products, scaled; a score's error moves the
weights by at most twice itself), E = 2^-22 (an exponential's argument, up to
2 A log2(e), is rounded in units of its last place), T = sum_j p_j |v_jd| and S
the positions. R is what a probability loses when it is rounded for the output
product: 2^-8 (BF16 pages, half a step of BF16), 2^-11 (INT8 pages, half a step
of fp16); and for calls of one row per item, which split the probabilities into
two or three parts, 2^-20. U is what a weight loses below its type's normal
range, of each of S weights, in units of V, the largest |v| of the request:
2^-25 (fp16, weights scaled to at most 1 or more), 2^-38 when they are split
(scaled to 2^14), 2^-125 (BF16 pages: binary32's own). H is half a step of the
output type.

Source: "Deploying Hunyuan 770B in INT8 on domestic accelerators" §3.4.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import moe_gemm_gb300 as w8  # noqa: E402

DEV = torch.device("cuda:0")
D = 128
SCALE = 1 / math.sqrt(D)


class Batch:
    """Requests with n_new new tokens on top of ctx cached positions, their
    pages shuffled through a pool whose unused part holds no numbers."""

    def __init__(self, n_new, ctx, Hq, Hkv, page, int8, seed=0, spread=1.0, spare=3, extra_w=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.n_new, self.ctx, self.Hq, self.Hkv, self.page = n_new, ctx, Hq, Hkv, page
        self.kv = [c + n for c, n in zip(ctx, n_new)]
        have = [-(-n // page) for n in self.kv]
        self.P = sum(have) + spare
        W = max(max(have), 1) + extra_w
        ids = torch.randperm(self.P, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((len(ctx), W), -1, dtype=torch.int32, device=DEV)
        self.cu = [0]
        at = 0
        for b, n in enumerate(have):
            self.table[b, :n] = ids[at:at + n]
            at += n
            self.cu.append(self.cu[-1] + n_new[b])
        T = self.cu[-1]
        self.q = (torch.randn(T, Hq, D, generator=g, device=DEV) * spread).to(torch.bfloat16)
        shape = (self.P, Hkv, page, D)
        k = torch.randn(shape, generator=g, device=DEV)
        k[..., ::51] *= 4
        v = torch.randn(shape, generator=g, device=DEV)
        self.ks = self.vs = None
        if int8:
            self.ks, self.vs = (x.abs().amax(-1) / 127 for x in (k, v))
            self.kc, self.vc = (torch.round(x / s[..., None]).to(torch.int8)
                                for x, s in ((k, self.ks), (v, self.vs)))
        else:
            self.kc, self.vc = k.to(torch.bfloat16), v.to(torch.bfloat16)
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32, device=DEV)
        self.cu_new = torch.tensor(self.cu, dtype=torch.int32, device=DEV)
        # positions past a request's length, and free pages, hold anything
        used = torch.zeros(self.P, page, dtype=torch.bool, device=DEV)
        for b, L in enumerate(self.kv):
            for j in range(have[b]):
                used[int(self.table[b, j]), :max(0, min(page, L - j * page))] = True
        self.poison(~used)

    def poison(self, where):
        w = where[:, None, :].expand(-1, self.Hkv, -1)
        if self.ks is not None:
            self.ks[w] = math.nan
            self.vs[w] = math.inf
        else:
            self.kc[w] = math.inf
            self.vc[w] = math.nan

    def run(self, **kw):
        kw.setdefault("out_dtype", torch.float32)
        out = w8.attention_paged(self.q, self.kc, self.vc, self.table, self.kv_lens, self.cu_new,
                                 SCALE, k_scale=self.ks, v_scale=self.vs, **kw)
        torch.cuda.synchronize()
        return out

    def rows(self, b, cache, scales):
        L = self.kv[b]
        pos = torch.arange(L, device=DEV)
        p, off = self.table[b].long()[pos // self.page], pos % self.page
        x = cache[p, :, off].double()                        # [L, Hkv, D]
        return x if scales is None else x * scales[p, :, off].double()[..., None]

    def check(self, out, window=0, split=False, half=2.0 ** -24, dead=None):
        """dead(b, positions) -> True where the position is masked for everyone."""
        G = self.Hq // self.Hkv
        worst = 0.0
        if self.ks is not None:
            R, U = (2.0 ** -20, 2.0 ** -38) if split else (2.0 ** -11, 2.0 ** -25)
        else:
            R, U = 2.0 ** -20 if split else 2.0 ** -8, 2.0 ** -125
        for b, n in enumerate(self.n_new):
            if n == 0:
                continue
            L, t0 = self.kv[b], self.cu[b]
            got = out[t0:t0 + n].double()
            k, v = self.rows(b, self.kc, self.ks), self.rows(b, self.vc, self.vs)
            pos = L - n + torch.arange(n, device=DEV)[:, None]
            j = torch.arange(L, device=DEV)
            seen = j <= pos
            if window:
                seen &= j > pos - window
            if dead is not None:
                m = dead(b, j)
                seen &= ~m
                v = torch.where(m[:, None, None], 0.0, v)
                k = torch.where(m[:, None, None], 0.0, k)
            for h in range(self.Hq):
                q = self.q[t0:t0 + n, h].double()
                kh, vh = k[:, h // G], v[:, h // G]
                s = torch.where(seen, (q @ kh.T) * SCALE, -math.inf)
                top = s.amax(-1, keepdim=True) if L else torch.zeros(n, 1, device=DEV)
                p = torch.where(seen, (s - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
                den = p.sum(-1, keepdim=True)
                p = torch.where(den > 0, p / den, 0.0)
                want, T = p @ vh, p @ vh.abs()
                A = torch.where(seen, (q.abs() @ kh.abs().T) * SCALE, 0.0)
                A = A.amax(-1, keepdim=True) if L else torch.zeros(n, 1, device=DEV)
                rel = 2 * A * (D + 2) * 2.0 ** -24 + 2 * A * 2.0 ** -22 + (L + 64) * 2.0 ** -24 \
                    + 16 * 2.0 ** -22 + R
                lost = U * L * vh.abs().amax() if L else 0.0
                bound = rel * T + lost + half * want.abs()
                err = (got[:, h] - want).abs()
                assert bool((err <= bound).all()), \
                    (b, h, float((err / bound.clamp_min(1e-30)).max()))
                if L:
                    worst = max(worst, float((err / bound.clamp_min(1e-30)).max()))
        return worst


KINDS = [True, False]


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("page", [8, 16, 24, 64, 128, 256])
def test_single_tokens(page, int8):
    b = Batch([1] * 6, [0, 1, 127, 128, 300, 777], 16, 2, page, int8)
    b.check(b.run(), split=True)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (14, 2), (8, 8), (32, 2), (26, 2)])
def test_head_groups(Hq, Hkv, int8):
    b = Batch([1, 1, 1], [5, 200, 1000], Hq, Hkv, 32, int8, seed=1)
    b.check(b.run(), split=True)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 1), (10, 2), (48, 3)])
def test_mixed_chunks(Hq, Hkv, int8):
    b = Batch([1, 37, 0, 4, 300, 1, 129], [700, 0, 40, 127, 65, 0, 256], Hq, Hkv, 16, int8, seed=2)
    b.check(b.run())


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("n", [1, 2, 3, 31, 64, 127, 128, 129, 255, 257, 513])
def test_whole_prompts(n, int8):
    b = Batch([n], [0], 8, 2, 64, int8, seed=n)
    b.check(b.run())


@pytest.mark.parametrize("int8", KINDS)
def test_long_context_is_divided(int8):
    b = Batch([1, 1], [9000, 33], 8, 1, 64, int8, seed=3)
    b.check(b.run(), split=True)
    b = Batch([70], [6000], 8, 1, 64, int8, seed=4)
    b.check(b.run())


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("window", [1, 7, 100, 128, 129, 1000, 100000])
def test_windows(window, int8):
    b = Batch([1, 1, 200, 5, 400], [0, 900, 0, 300, 650], 8, 2, 16, int8, seed=5)
    if window < 300:
        # what lies before every new token's window is not read: pages there
        # may be gone, and hold anything
        for r in range(5):
            first = max(0, b.ctx[r] - window + 1) // b.page
            gone = b.table[r, :first].clone()
            if first:
                b.kc[gone.long()] = 99
                b.vc[gone.long()] = 99
                where = torch.zeros(b.P, b.page, dtype=torch.bool, device=DEV)
                where[gone.long()] = True
                # (the reference must not read it either)
                lo = max(0, b.ctx[r] - window + 1)
                assert first * b.page <= lo
    b.check(b.run(window=window), window=window)


@pytest.mark.parametrize("int8", KINDS)
def test_pages_before_the_window_may_be_gone(int8):
    b = Batch([1, 130], [1000, 1000], 8, 2, 16, int8, seed=6)
    whole = b.run(window=100)
    before = [(1000 - 100 + 1) // 16] * 2
    for r in range(2):
        where = torch.zeros(b.P, b.page, dtype=torch.bool, device=DEV)
        where[b.table[r, :before[r]].long()] = True
        b.poison(where)
        b.table[r, :before[r]] = -1
    again = b.run(window=100)
    assert torch.equal(whole, again)
    assert w8.device_error() == 0


@pytest.mark.parametrize("int8", KINDS)
def test_rows_that_see_nothing(int8):
    # more new tokens than positions: the first ones stand before position 0
    b = Batch([4, 300, 1, 2], [0, 0, 0, 50], 8, 2, 16, int8, seed=7)
    b.kv = [2, 100, 0, 52]
    b.kv_lens = torch.tensor(b.kv, dtype=torch.int32, device=DEV)
    out = torch.full((sum(b.n_new), 8, D), math.nan, device=DEV)
    b.run(out=out)
    assert bool((out[0:2] == 0).all()) and bool((out[4:204] == 0).all())
    assert bool((out[304] == 0).all())
    b.check(out)


@pytest.mark.parametrize("int8", KINDS)
def test_rows_of_no_request(int8):
    b = Batch([1, 20], [10, 10], 4, 2, 16, int8, seed=8)
    b.q = torch.cat([b.q, b.q[:5]])
    out = torch.full((26, 4, D), math.nan, device=DEV)
    b.run(out=out)
    assert bool((out[21:] == 0).all())
    b.check(out)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("n", [1, 60])
def test_absent_pages_are_masked_and_told(int8, n):
    b = Batch([n, 1], [300, 40], 8, 2, 16, int8, seed=9)
    b.table[0, 3] = -1
    b.table[0, 5] = b.P
    w8.device_error()
    out = b.run()
    assert w8.device_error() != 0 and w8.device_error() == 0
    b.table[0, 3] = b.table[0, 5] = 0                       # (for the reference's gather)
    b.check(out, dead=lambda r, j: ((j // 16 == 3) | (j // 16 == 5)) if r == 0 else j < 0)


@pytest.mark.parametrize("int8", KINDS)
def test_lengths_past_the_table_are_cut(int8):
    b = Batch([1], [63], 4, 2, 16, int8, seed=10)
    want = b.run()
    b.kv_lens = torch.tensor([1000], dtype=torch.int32, device=DEV)
    assert torch.equal(b.run(), want)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("n_new", [[1, 1, 1], [1, 150, 9]])
def test_bf16_output_strides_stream_and_graph(int8, n_new):
    b = Batch(n_new, [300, 20, 129], 8, 2, 32, int8, seed=11, extra_w=3)
    want = b.run(out_dtype=torch.bfloat16)
    b.check(want, half=2.0 ** -8)
    # q as a part of a fused projection's rows
    T = b.q.shape[0]
    rows = torch.zeros(T, 14, D, dtype=torch.bfloat16, device=DEV)
    rows[:, 3:11] = b.q
    b.q = rows[:, 3:11]
    assert torch.equal(b.run(out_dtype=torch.bfloat16), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(b.run(out_dtype=torch.bfloat16, stream=side), want)
    out = torch.empty_like(want)
    ws = torch.empty(w8.attention_paged_workspace_size(T, 3, 8, 2), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w8.attention_paged(b.q, b.kc, b.vc, b.table, b.kv_lens, b.cu_new, SCALE, k_scale=b.ks,
                           v_scale=b.vs, out=out, workspace=ws)
    for _ in range(2):
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("spread", [0.01, 8.0, 40.0])
def test_flat_and_peaked_scores(int8, spread):
    b = Batch([1, 90], [500, 700], 8, 2, 64, int8, seed=12, spread=spread)
    b.check(b.run())


@pytest.mark.parametrize("n", [1, 100])
def test_scales_of_very_different_size(n):
    b = Batch([n], [400], 8, 2, 32, True, seed=13)
    g = torch.Generator(device=DEV).manual_seed(1)
    b.vs *= torch.exp2(torch.randint(-30, 10, b.vs.shape, generator=g, device=DEV).float())
    b.kc[1], b.ks[1], b.vs[2] = 0, 0.0, 0.0                 # vectors of zeros
    b.vc[2] = 0
    b.poison(torch.zeros(b.P, 32, dtype=torch.bool, device=DEV))
    b.check(b.run())


def test_same_numbers_as_the_contiguous_cache():
    # pages in order are the contiguous layout of one sequence
    b = Batch([1], [512 - 1], 8, 2, 512, True, seed=14, spare=0)
    out = b.run()
    lens = torch.tensor([512], dtype=torch.int32, device=DEV)
    ref = w8.attention_decode(b.q, b.kc, b.vc, lens, SCALE, k_scale=b.ks, v_scale=b.vs,
                              out_dtype=torch.float32)
    assert bool(((out - ref).abs() <= 1e-5).all())


@pytest.mark.parametrize("int8", KINDS)
def test_many_requests(int8):
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 4, (600,), generator=g).tolist()
    c = torch.randint(0, 90, (600,), generator=g).tolist()
    b = Batch(n, c, 4, 2, 16, int8, seed=15)
    b.check(b.run())


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("n_new,Hq", [([2, 2, 1, 3], 8), ([4, 0, 7, 1], 4), ([1, 0, 0, 3], 16),
                                      ([2, 2, 2, 2], 10)])
def test_few_tokens_per_request(n_new, Hq, int8):
    b = Batch(n_new, [130, 5, 700, 0], Hq, 2, 16, int8, seed=12)
    b.check(b.run(), split=True)


@pytest.mark.parametrize("int8", KINDS)
def test_every_sm_busy_gives_the_same_numbers(int8):
    b = Batch([2048, 1500, 1, 700], [0, 2500, 4000, 65], 32, 8, 64, int8, seed=13)
    w8.device_error()
    out = b.run()
    for _ in range(4):
        assert torch.equal(b.run(), out)
    assert w8.device_error() == 0
    b.check(out)


@pytest.mark.parametrize("int8", KINDS)
def test_pool_past_32_bit_offsets(int8):
    # the pool's bytes (and, BF16, elements) pass 2^31; the request's pages lie at its end
    Hkv, page = 8, 64
    P = (1 << 31) // (Hkv * page * D) + 8
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    b = Batch([1, 40], [100, 60], 16, Hkv, page, int8, seed=16)
    big = lambda x: torch.zeros((P,) + tuple(x.shape[1:]), dtype=x.dtype, device=DEV)  # noqa: E731
    kc, vc = big(b.kc), big(b.vc)
    kc[P - b.P:], vc[P - b.P:] = b.kc, b.vc
    if int8:
        ks, vs = big(b.ks), big(b.vs)
        ks[P - b.P:], vs[P - b.P:] = b.ks, b.vs
    else:
        ks = vs = None
    want = b.run()
    table = torch.where(b.table >= 0, b.table + (P - b.P), -1)
    out = w8.attention_paged(b.q, kc, vc, table, b.kv_lens, b.cu_new, SCALE, k_scale=ks,
                             v_scale=vs, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("value", [math.nan, math.inf, -3e38, 1e30])
@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("n_new,spare", [([1, 1, 1], 2), ([2, 1, 3], 5), ([20, 33, 5], 37),
                                         ([1, 200, 70], 64)])
def test_rows_of_q_that_are_not_a_requests_own(n_new, spare, int8, value):
    # rows past the last request's (a padded step's) hold anything; so may a neighbour's
    b = Batch(n_new, [40, 300, 129], 8, 2, 16, int8, seed=21)
    T = b.q.shape[0]
    b.q = torch.cat([b.q, b.q[:1].expand(spare, -1, -1)])
    clean = b.run()
    b.check(clean[:T], split=(T + spare) * 4 <= 16 * 3)
    b.q[T:] = value
    assert torch.equal(b.run(), clean)
    for r in range(3):
        q = b.q.clone()
        b.q[b.cu[r]:b.cu[r + 1]] = value
        out, b.q = b.run(), q
        out[b.cu[r]:b.cu[r + 1]] = clean[b.cu[r]:b.cu[r + 1]]
        assert torch.equal(out, clean)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("n_new", [[1, 1], [3, 1], [70, 9]])
def test_a_row_that_is_no_number_is_so_alone(n_new, int8, value):
    # one head of one token: the other heads and tokens of the request keep their answers
    b = Batch(n_new, [200, 90], 8, 2, 16, int8, seed=23)
    q = b.q.clone()
    at = (n_new[0] - 1, 5)
    b.q[at][7] = value
    out, b.q = b.run(), q
    if math.isnan(value):
        assert bool(torch.isnan(out[at]).all())
    out[at] = b.run()[at]
    b.check(out, split=sum(n_new) * 4 <= 16 * 2)


def check_by_tile(b, out):
    """One request, INT8 pages, the many-rows kernel: Batch.check with the absolute
    term of each weight taken of its own tile of 128 positions. A weight times its v scale
    is held as fp16 in units of 2^e, 2^e <= 2^3 s with s the tile's largest v scale: it
    loses 2^-25 2^e <= 2^-22 s at most, and no more than itself; the sum of weights that
    it is divided by is 1 at least (2^-10 for what that sum is off)."""
    G, L, n = b.Hq // b.Hkv, b.kv[0], b.n_new[0]
    pos = torch.arange(L, device=DEV)
    pg, off = b.table[0].long()[pos // b.page], pos % b.page
    seen = pos <= L - n + torch.arange(n, device=DEV)[:, None]
    for h in range(b.Hq):
        codes, vs = b.vc[pg, h // G, off].double(), b.vs[pg, h // G, off].double()
        k = b.kc[pg, h // G, off].double() * b.ks[pg, h // G, off].double()[:, None]
        v, q = codes * vs[:, None], b.q[:, h].double()
        s = torch.where(seen, (q @ k.T) * SCALE, -math.inf)
        p = torch.softmax(s, -1)
        tiles = torch.nn.functional.pad(vs, (0, -L % 128)).view(-1, 128)
        tile = tiles.amax(-1).repeat_interleave(128)[:L]
        lost = torch.minimum(2.0 ** -22 * tile, p * vs) @ codes.abs() * (1 + 2.0 ** -10)
        want, bound = p @ v, lost
        # (the error of a score moves its own weight: keys of next to no weight by themselves)
        for part in (p >= 2.0 ** -40, p < 2.0 ** -40):
            A = torch.where(part & seen, (q.abs() @ k.abs().T) * SCALE, 0.0).amax(-1, keepdim=True)
            rel = 2 * A * (D + 2) * 2.0 ** -24 + 2 * A * 2.0 ** -22 + (L + 64) * 2.0 ** -24 \
                + 16 * 2.0 ** -22 + 2.0 ** -11
            bound = bound + rel * (torch.where(part, p, 0.0) @ v.abs())
        bound = bound + 2.0 ** -24 * want.abs()
        err = (out[:, h].double() - want).abs()
        assert bool((err <= bound).all()), (h, float((err / bound).max()))


@pytest.mark.parametrize("power", [12, 20, 30])
@pytest.mark.parametrize("every", [1000, 2, 3])
@pytest.mark.parametrize("n,ctx", [(70, 900), (300, 128), (513, 1000)])
def test_large_value_vectors_cost_their_own_tiles(n, ctx, every, power):
    # tiles whose vectors are 2^power larger, and that no query gives weight (their keys point
    # away from what the queries share), take no bits from the others
    b = Batch([n], [ctx], 8, 2, 32, True, seed=22)
    pos = torch.arange(ctx // 128 * 128, device=DEV)
    pos = pos[pos // 128 % every == 0]
    pg, off = b.table[0].long()[pos // 32], pos % 32
    b.vs[pg, :, off] *= 2.0 ** power
    b.q[..., 1] = 256.0
    b.kc[..., 1] = 0
    b.kc[pg, :, off, 1] = -127
    check_by_tile(b, b.run())


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("shape,strides", [((1, 8, D), (3, D, 1)), ((5, 1, D), (D, 1, 1)),
                                           ((1, 1, D), (1, 2, 1)), ((40, 1, D), (2 * D, 7, 1))])
def test_dimensions_of_one_have_no_stride(shape, strides, int8):
    T, H = shape[:2]
    b = Batch([T], [100], H, H, 16, int8, seed=24)
    want = b.run()
    rows = torch.zeros(T, 2 * H, D, dtype=torch.bfloat16, device=DEV)
    rows = rows.view(-1)
    view = rows.as_strided(shape, strides)
    view.copy_(b.q)
    b.q = view
    assert b.q.stride() == strides and torch.equal(b.run(), want)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    for k in (view, view.contiguous()):
        kc = torch.zeros(T, H, 16, D, dtype=torch.bfloat16, device=DEV)
        vc = torch.zeros_like(kc)
        w8.paged_kv_write(k, k, slots, kc, vc)
        assert torch.equal(kc.transpose(1, 2).reshape(-1, H, D)[:T], view) and torch.equal(kc, vc)


@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("first", [0, 1])
def test_scales_at_both_ends_of_binary32(first, n):
    # (tiles in turn; the weights' unit changes by 2^130 between them)
    b = Batch([n], [900], 4, 1, 32, True, seed=25)
    pos = torch.arange(b.kv[0], device=DEV)
    pg, off = b.table[0].long()[pos // 32], pos % 32
    far = torch.where(pos // 128 % 2 == first, 50.0, -100.0)
    b.vs[pg, :, off] *= torch.exp2(far)[:, None]
    b.check(b.run(), split=n == 1)


def test_scales_at_both_ends_in_the_contiguous_cache():
    b = Batch([1], [900], 4, 1, 1024, True, seed=25, spare=0)
    far = torch.where(torch.arange(1024, device=DEV) // 128 % 2 == 0, 50.0, -100.0)
    b.vs *= torch.exp2(far)
    lens = torch.tensor([901], dtype=torch.int32, device=DEV)
    out = w8.attention_decode(b.q, b.kc, b.vc, lens, SCALE, k_scale=b.ks, v_scale=b.vs,
                              out_dtype=torch.float32)
    b.check(out, split=True)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("window", [1, 31, 100, 128, 129, 1000])
@pytest.mark.parametrize("n_new", [[1, 1, 1, 1], [2, 1, 3, 4]])
def test_few_rows_with_a_window(n_new, window, int8):
    b = Batch(n_new, [0, 130, 900, 2000], 8, 2, 16, int8, seed=26)
    whole = b.run(window=window)
    b.check(whole, window=window, split=True)
    # pages before every new token's window may be gone, and hold anything
    for r, (c, n) in enumerate(zip(b.ctx, n_new)):
        first = max(0, c - window + 1) // 16
        where = torch.zeros(b.P, 16, dtype=torch.bool, device=DEV)
        where[b.table[r, :first].long()] = True
        b.poison(where)
        b.table[r, :first] = -1
    w8.device_error()
    assert torch.equal(b.run(window=window), whole) and w8.device_error() == 0


@pytest.mark.parametrize("int8", KINDS)
def test_few_rows_that_see_nothing(int8):
    # refused requests (no positions) and tokens before position 0 in a decode step
    b = Batch([1, 1, 3, 1, 2], [50, 0, 0, 700, 0], 8, 2, 16, int8, seed=27)
    b.kv = [51, 0, 0, 701, 1]
    b.kv_lens = torch.tensor(b.kv, dtype=torch.int32, device=DEV)
    b.q = torch.cat([b.q, b.q[:1]])
    out = torch.full((9, 8, D), math.nan, device=DEV)
    b.run(out=out)
    assert bool((out[1:5] == 0).all()) and bool((out[6] == 0).all()) and bool((out[8] == 0).all())
    b.check(out, split=True)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("qt,qh", [(80, 8), (8, 128), (1024, 64), (0, 128)])
def test_rows_of_q_that_overlap(qt, qh, int8):
    # strides below a row's length take the few-rows kernel at any number of rows
    b = Batch([90, 1, 40], [10, 300, 0], 8, 2, 16, int8, seed=28)
    T = b.q.shape[0]
    g = torch.Generator(device=DEV).manual_seed(5)
    store = torch.randn(T * 1024 + 2048, generator=g, device=DEV).to(torch.bfloat16)
    b.q = store.as_strided((T, 8, D), (qt, qh, 1))
    b.check(b.run(), split=True)


def test_few_rows_with_scales_of_very_different_size():
    b = Batch([1], [400], 8, 2, 32, True, seed=13)
    g = torch.Generator(device=DEV).manual_seed(1)
    b.vs *= torch.exp2(torch.randint(-30, 10, b.vs.shape, generator=g, device=DEV).float())
    b.poison(torch.zeros(b.P, 32, dtype=torch.bool, device=DEV))
    b.check(b.run(), split=True)


@pytest.mark.parametrize("int8", KINDS)
def test_many_requests_keep_all_bits(int8):
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 4, (600,), generator=g).tolist()
    c = torch.randint(0, 90, (600,), generator=g).tolist()
    b = Batch(n, c, 4, 2, 16, int8, seed=15)
    b.check(b.run(), split=True)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("page", [8, 24, 48, 128, 256])
@pytest.mark.parametrize("window", [0, 100])
def test_many_rows_over_pages_of_other_sizes(window, page, int8):
    b = Batch([70, 1, 150], [500, 130, 0], 14, 2, page, int8, seed=29)
    b.check(b.run(window=window), window=window)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("n_new,Hq,Hkv,page", [([1] * 30, 16, 2, 128), ([1] * 14, 8, 8, 64),
                                               ([2] * 20 + [1] * 4, 16, 2, 16), ([7, 8, 5, 1] * 4, 4, 2, 32)])
def test_few_rows_repeat_themselves(n_new, Hq, Hkv, page, int8):
    # a cache in L2, so that copies are as fast as they get: none may overtake a read
    g = torch.Generator().manual_seed(9)
    ctx = torch.randint(300, 4000, (len(n_new),), generator=g).tolist()
    b = Batch(n_new, ctx, Hq, Hkv, page, int8, seed=30)
    b.q = torch.cat([b.q, b.q[:2]])                     # (16 rows per item)
    out = b.run()
    b.check(out[:-2], split=True)
    for _ in range(100):
        assert torch.equal(b.run(), out)


@pytest.mark.parametrize("int8", KINDS)
@pytest.mark.parametrize("page", [8, 16, 24, 128])
def test_many_tiles_of_one_request_per_block(page, int8):
    # more tiles than a warp looks up in the block table at once
    b = Batch([1] * 32, [8000 - 13 * i for i in range(32)], 8, 8, page, int8, seed=31)
    w8.device_error()
    b.check(b.run(), split=True)
    assert w8.device_error() == 0
