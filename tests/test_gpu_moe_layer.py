"""GPU tests of the whole MoE layer: the numbers of moe_gate followed by moe_ffn, bit
for bit, and against the definition in 64 bits.

Sources: "Deploying Hunyuan 770B in INT8 on domestic accelerators" §1.3, §4.1, §4.4.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import moe_gemm_gb300 as w8  # noqa: E402

DEV = torch.device("cuda:0")
GROUP = 128


def make(T, E, H, I, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5

    def weights(n, k):
        qw, sw = w8.quant_weight(torch.randn(E * n, k, generator=g, device=DEV) * 0.02)
        return qw.view(E, n, k), sw.view(E, n, k // GROUP)

    return x, logits, [*weights(2 * I, H), *weights(H, I)]


def same(x, logits, k, w, **how):
    y, ids, ww = w8.moe_layer(x, logits, k, *w, **how)
    out = {n: how.pop(n) for n in ("out_dtype", "out", "stream") if n in how}
    ids2, ww2 = w8.moe_gate(logits, k, **how)
    want = w8.moe_ffn(x, ids2, ww2, *w, out_dtype=out.get("out_dtype", torch.bfloat16))
    assert torch.equal(ids, ids2) and torch.equal(ww, ww2)
    assert torch.equal(y, want)
    assert w8.device_error() == 0
    return y, ids, ww


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 8, 2, 256, 128), (1, 64, 8, 1024, 384), (2, 1, 1, 128, 128), (3, 7, 7, 384, 256),
    (5, 256, 8, 512, 128), (8, 16, 4, 2048, 512), (16, 64, 8, 1024, 640), (17, 33, 5, 640, 256),
    (31, 12, 3, 1280, 896), (32, 64, 16, 512, 256), (32, 4, 4, 256, 384), (32, 9, 1, 128, 1152),
    (1, 1000, 64, 256, 128), (9, 40, 6, 7168, 256), (33, 64, 8, 512, 256), (32, 64, 17, 256, 128),
    (100, 16, 4, 512, 256), (32, 16, 16, 4992, 128), (32, 16, 16, 4864, 128), (4, 6, 5, 128, 8192)])
def test_same_as_gate_and_ffn(T, E, k, H, I):
    x, logits, w = make(T, E, H, I, seed=T + E)
    same(x, logits, k, w)
    same(x, logits, k, w, out_dtype=torch.float32, scoring="sigmoid", scale=2.5)


def test_gates_of_all_kinds():
    x, logits, w = make(16, 64, 512, 256)
    bias = torch.randn(64, device=DEV) * 0.1
    same(x, logits, 6, w, scoring="sigmoid", bias=bias, n_group=8, topk_group=4)
    same(x, logits.to(torch.bfloat16), 6, w, bias=bias, renormalize=False)
    wide = torch.randn(16, 100, device=DEV)
    same(x, wide[:, 20:84], 6, w)


def test_token_counts_of_an_expert():
    # all tokens to one expert, and every number of tokens from 1 to 32 at some expert
    x, logits, w = make(32, 8, 512, 256)
    logits[:, 3] = 100.0
    same(x, logits, 1, w)
    x, logits, w = make(32, 32, 256, 128)
    logits[:] = 0.0
    for e in range(32):
        logits[:e + 1, e] = 10.0 + e
    same(x, logits, 16, w)


def test_tokens_without_experts():
    x, logits, w = make(6, 16, 512, 256)
    logits[1] = float("nan")
    logits[4] = float("-inf")
    logits[2, 3:] = float("-inf")          # three experts left of the five asked for
    y, ids, _ = same(x, logits, 5, w)
    assert torch.all(y[[1, 4]] == 0) and torch.all(ids[2, 3:] == -1)
    logits[:] = float("nan")
    y, ids, _ = same(x, logits, 5, w)
    assert torch.all(y == 0) and torch.all(ids == -1)


@pytest.mark.parametrize("T", [1, 9])
def test_weights_of_zero(T):
    # an expert that counts 0 times still gives NaN where its output is not finite
    x, logits, (qu, su, qd, sd) = make(T, 6, 256, 128)
    sd[2, ::3] = 3e38
    sd[4, 1::3] = 3e38
    for how in (dict(scale=0.0), dict(scoring="softmax", renormalize=False)):
        logits[:, 2] = logits[:, 4] = -200.0       # (the softmax of -200 is 0 in FP32)
        y, ids, ww = w8.moe_layer(x, logits, 6, qu, su, qd, sd, **how)
        want = w8.moe_ffn(x, *w8.moe_gate(logits, 6, **how), qu, su, qd, sd)
        assert torch.all((ww == 0) == (((ids == 2) | (ids == 4)) | ("scale" in how)))
        assert torch.any(torch.isnan(want)) and not torch.all(torch.isnan(want))
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_zero_and_unaligned_rows():
    x, logits, w = make(7, 16, 512, 256)
    x[3] = 0
    y, _, _ = same(x, logits, 4, w)
    assert torch.all(y[3] == 0)
    wide = torch.randn(7, 521, device=DEV).to(torch.bfloat16)
    same(wide[:, 9:], logits, 4, w)        # rows at odd addresses, an odd stride
    assert w8.moe_layer(x[:0], logits[:0], 4, *w)[0].shape == (0, 512)


@pytest.mark.parametrize("T", [1, 12])
def test_against_64_bits(T):
    """Codes of h may differ where FP32 and 64 bits round h / scale to different
    integers, which moves d by one code: a scale times a weight. Tokens' codes are the
    same (decided in FP32 by definition). So |y - y*| is at most half a BF16 step, 2^-8
    |y*|, FP32's error, below 2^-20 of the magnitudes summed, and for such codes (h is
    off by 2^-20 relative at most, so a share of 127 * 2^-20 * 2 of them at most, 2^-12;
    none to two of a row's 384) the codes' worth: 2 max_n |W| scale."""
    H, I, E, k = 512, 384, 8, 3
    x, logits, (qu, su, qd, sd) = make(T, E, H, I, seed=5)
    y, ids, ww = w8.moe_layer(x, logits, k, qu, su, qd, sd, out_dtype=torch.float32)
    xf = x.float()
    m = xf.abs().amax(1, keepdim=True) / torch.tensor(127.0, device=DEV)
    xq = torch.round(xf / m).double() * m.double()
    up = qu.double() * su.double().repeat_interleave(GROUP, 2)
    down = qd.double() * sd.double().repeat_interleave(GROUP, 2)
    for t in range(T):
        want = torch.zeros(H, dtype=torch.float64, device=DEV)
        mag, flip = torch.zeros_like(want), torch.zeros_like(want)
        for j in range(k):
            e = int(ids[t, j])
            u = up[e] @ xq[t]
            h = u[:I] * torch.sigmoid(u[:I]) * u[I:]
            s = h.abs().max() / 127
            hq = torch.round(h / s) * s
            p = float(ww[t, j])
            want += p * (down[e] @ hq)
            mag += p * (down[e].abs() @ hq.abs())
            flip += p * 2 * s * down[e].abs().amax(1)
        assert torch.all((y[t].double() - want).abs() <= 2.0 ** -20 * mag + flip)


def test_streams_graphs_and_repeats():
    x, logits, w = make(8, 32, 1024, 512)
    want, ids, _ = same(x, logits, 4, w)
    for _ in range(20):
        assert torch.equal(w8.moe_layer(x, logits, 4, *w)[0], want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = w8.moe_layer(x, logits, 4, *w, stream=s)[0]
    s.synchronize()
    assert torch.equal(y, want)
    # a workspace full of anything
    ws = torch.full((w8.moe_layer_workspace_size(8, 4, 1024, 512, 32),), 255, dtype=torch.uint8,
                    device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, ids, _ = w8.moe_layer(x, logits, 4, *w, workspace=ws)
    x2, logits2, _ = make(8, 32, 1024, 512, seed=9)
    x.copy_(x2)
    logits.copy_(logits2)
    ws.fill_(171)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    same(x, logits, 4, w)
    assert torch.equal(y, w8.moe_layer(x, logits, 4, *w)[0])


def test_two_at_once():
    # two calls on two streams, each with its own workspace (one waits for the other's SMs)
    a, b = make(16, 64, 1024, 512, seed=1), make(4, 64, 1024, 512, seed=2)
    want = [w8.moe_layer(x, lg, 8, *w)[0] for x, lg, w in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s, (x, lg, w) in zip(streams, (a, b)):
            got.append(w8.moe_layer(x, lg, 8, *w, stream=s)[0])
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    assert w8.device_error() == 0


def test_refusals():
    x, logits, w = make(4, 8, 256, 128)
    for bad in (lambda: w8.moe_layer(x, logits[:3], 2, *w), lambda: w8.moe_layer(x, logits, 9, *w),
                lambda: w8.moe_layer(x, logits.half(), 2, *w),
                lambda: w8.moe_layer(x[:, :128], logits, 2, *w),
                lambda: w8.moe_layer(x, logits, 2, w[0], w[1], w[2][:, :128], w[3]),
                lambda: w8.moe_layer(x, logits, 2, *w, scoring="relu"),
                lambda: w8.moe_layer(x, logits, 2, *w, workspace=torch.empty(64, dtype=torch.uint8,
                                                                             device=DEV)),
                lambda: w8.moe_layer(x.float(), logits, 2, *w),
                lambda: w8.moe_layer(x, logits, 2, *w, bias=torch.zeros(7, device=DEV))):
        with pytest.raises((ValueError, w8.W8A8Error)):
            bad()
