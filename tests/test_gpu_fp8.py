"""GPU tests of the FP8 linear layer with a scale per block of 128: quantizers bit for
bit against their definition, the product against 64 bits.

Tolerance of the product: a group's 128 products are exact, and summed in FP32 by the tensor
cores, whose additions may truncate: 128 of them, 2^-23 of a partial sum each, which
is at most T: 2^-16 T. The scales' product and the additions of G groups round to
nearest, 2^-24 each. BF16 outputs add half a step, 2^-8 of the value.

Source: "Running DeepSeek-V4-Flash-Vision on 4xA800" §一 (FP8 weights in [128, 128]
blocks, power-of-two scales).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import moe_gemm_gb300 as w8  # noqa: E402

DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn


def scale_rule(m, mode):
    """The scales, on the CPU: binary32 division, or powers of two by exact comparison."""
    m = m.float().cpu()
    if mode == w8.SCALE_AMAX:
        return m / torch.tensor(448.0)
    s = torch.full_like(m, 2.0 ** -127)
    for e in range(-126, 128):
        s = torch.where(448.0 * s.double() >= m.double(), s, torch.tensor(2.0 ** e))
    return s


def code_rule(x, s):
    """x, s on the CPU, same shape: quotients in binary32 and their e4m3 bytes."""
    q = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)
    return q.to(E4M3).view(torch.uint8)


def check_act(a, mode):
    M, K = a.shape
    qa, sa = w8.quant_act_fp8(a, scale_mode=mode)
    x = a.float().cpu().view(M, K // 128, 128)
    s = scale_rule(x.abs().amax(-1), mode)
    assert torch.equal(sa.cpu().view(torch.int32), s.view(torch.int32))
    want = code_rule(x, s[..., None].expand_as(x)).view(M, K)
    got = qa.cpu().view(torch.uint8)
    assert torch.equal(got, want)


@pytest.mark.parametrize("mode", [w8.SCALE_AMAX, w8.SCALE_POW2])
@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (17, 1152), (333, 2048), (1024, 4096)])
def test_quant_act(M, K, mode):
    g = torch.Generator(device=DEV).manual_seed(M)
    a = torch.randn(M, K, generator=g, device=DEV)
    a[:, ::37] *= 50
    a *= torch.exp2(torch.randint(-30, 30, (M, 1), generator=g, device=DEV).float())
    check_act(a.to(torch.bfloat16), mode)


@pytest.mark.parametrize("mode", [w8.SCALE_AMAX, w8.SCALE_POW2])
def test_quant_act_borders(mode):
    a = torch.zeros(10, 256, dtype=torch.bfloat16, device=DEV)
    a[1, :128] = 3e38
    a[2, :128] = 1e-38
    a[2, 3] = -1e-40
    a[3] = torch.arange(256, device=DEV) - 128.0
    a[4, 128:] = 448.0                                  # a scale of one
    a[4, 129:140] = torch.tensor([0.5, 1.0625, 17.0, -19.0, 2.0 ** -10, 3 * 2.0 ** -10,
                                  2.0 ** -9, 432.0, 416.0, -17.0, 0.0], device=DEV)   # ties
    a[5, 7] = 2.0 ** -130
    a[6] = 449.0
    a[7] = 2.0 ** 127
    a[8, ::2] = 1.0
    check_act(a, mode)


def test_quant_act_rows_anywhere():
    a = torch.randn(9, 700, device=DEV).to(torch.bfloat16)
    check_act(a[:, 64:64 + 512], w8.SCALE_AMAX)          # aligned start, stride 700
    check_act(a[:, 5:5 + 512], w8.SCALE_POW2)            # odd start
    assert w8.quant_act_fp8(a[:0, :256])[0].shape == (0, 256)


@pytest.mark.parametrize("mode", [w8.SCALE_AMAX, w8.SCALE_POW2])
@pytest.mark.parametrize("M,K", [(4097, 1152), (4095, 1152), (32771, 128), (2341, 1920)])
def test_quant_act_units_left_over(M, K, mode):
    # four units per thread, and an odd number of units that ends inside them
    assert M * (K // 128) % 2 == 1 and M * (K // 128) >= 1 << 15
    g = torch.Generator(device=DEV).manual_seed(M)
    a = torch.randn(M, K + 3, generator=g, device=DEV).to(torch.bfloat16)
    check_act(a[:, 3:], mode)                            # rows at odd addresses
    check_act(a[:, :K].contiguous(), mode)
    # nothing behind the last unit
    qa = torch.full((M + 1, K), 0x11, dtype=torch.uint8, device=DEV)
    sa = torch.full((M + 1, K // 128), 7.0, device=DEV)
    w8.quant_act_fp8(a[:, 3:], qa[:M].view(E4M3), sa[:M], scale_mode=mode)
    assert torch.all(qa[M] == 0x11) and torch.all(sa[M] == 7)


@pytest.mark.parametrize("mode", [w8.SCALE_AMAX, w8.SCALE_POW2])
@pytest.mark.parametrize("N,K", [(1, 128), (128, 128), (200, 384), (515, 1024)])
def test_quant_weight(N, K, mode):
    w = torch.randn(N, K, device=DEV) * 0.02
    w[-1, :128] = 0
    qw, sw = w8.quant_weight_fp8(w, scale_mode=mode)
    rows = -(-N // 128)
    x = torch.zeros(rows * 128, K)
    x[:N] = w.cpu()
    x = x.view(rows, 128, K // 128, 128)
    s = scale_rule(x.abs().amax((1, 3)), mode)
    assert torch.equal(sw.cpu().view(torch.int32), s.view(torch.int32))
    want = code_rule(x, s[:, None, :, None].expand_as(x)).reshape(rows * 128, K)[:N]
    assert torch.equal(qw.cpu().view(torch.uint8), want)


def test_quant_weight_smallest():
    # scales of a few 2^-149: amax / 448 rounds to 1 of them for 225 to 672, to 2 up to 1120
    step = 2.0 ** -149
    k = torch.zeros(256, 384, dtype=torch.int32)
    k[:128, :128] = torch.arange(128 * 128).view(128, 128) % 668
    k[:128, 128:256] = torch.arange(128)[None] % 225
    k[:128, 256:] = torch.arange(128 * 128).view(128, 128) % 226
    k[128:, :128] = torch.arange(128 * 128).view(128, 128) % 1001
    k[::3] *= -1
    w = torch.where(k < 0, (-k) | (-1 << 31), k).to(torch.int32).view(torch.float32)
    assert torch.equal(w.double(), k.double() * step)
    qw, sw = w8.quant_weight_fp8(w.to(DEV))
    s = torch.tensor([[1, 0, 1], [2, 0, 0]]).double()
    assert torch.equal(sw.double().cpu(), s * step)
    s = s.repeat_interleave(128, 0).repeat_interleave(128, 1)
    x = torch.where(s > 0, k / torch.where(s > 0, s, 1.0), 0.0).clamp(-448, 448)
    assert torch.equal(qw.cpu().view(torch.uint8) & 0x7F, x.abs().float().to(E4M3).view(torch.uint8))
    assert torch.equal(qw.float().cpu().sign(), x.float().to(E4M3).float().sign())
    qw, sw = w8.quant_weight_fp8(w.to(DEV), scale_mode=w8.SCALE_POW2)
    assert torch.all(sw == 2.0 ** -127) and torch.all(qw.float() == 0)


@pytest.mark.parametrize("M", [3, 20, 40, 300, 1200])
def test_smallest_scales(M):
    """Scale products from 2^-160 to 2^-120. Below 2^-126 they are rounded to multiples of
    2^-149 (off by 2^-150, times the group's sum of |qa qw|), below 2^-150 to 0; and each addition
    of a group is off by 2^-150 where its result is below 2^-126. BF16: half a step there, 2^-134."""
    N, K = 520, 1152
    g = torch.Generator(device=DEV).manual_seed(M)
    qa = torch.randint(-8, 9, (M, K), generator=g, device=DEV).float().to(E4M3)
    qw = torch.randint(-8, 9, (N, K), generator=g, device=DEV).float().to(E4M3)

    def scales(rows):
        e = torch.randint(-80, -59, (rows, K // 128), generator=g, device=DEV).float()
        return torch.exp2(e) * (1 + torch.rand(rows, K // 128, generator=g, device=DEV))

    sa, sw = scales(M), scales(-(-N // 128))
    want, T = exact(qa, sa, qw, sw)
    f = sa.double()[:, None] * sw.double()[None]                         # [M, blocks, G]
    small = torch.where(f < 2.0 ** -126, 1.0, 0.0).repeat_interleave(128, 1)[:, :N]
    U = (torch.einsum("mgk,ngk->mng", qa.double().abs().view(M, -1, 128),
                      qw.double().abs().view(N, -1, 128)) * small).sum(-1) + K // 128
    assert 0 < small.mean() < 1
    lim = (2.0 ** -16 + (K // 128 + 1) * 2.0 ** -24) * T + 2.0 ** -149 * U
    y = w8.gemm_fp8(qa, sa, qw, sw, out_dtype=torch.float32)
    assert torch.all((y.double() - want).abs() <= lim)
    y = w8.gemm_fp8(qa, sa, qw, sw)
    assert torch.all((y.double() - want).abs() <= lim * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -134)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_scale_products_that_vanish(M):
    # products of 2^-160 are 0 and of 1.5 * 2^-149 are 2^-148: a bound relative to T alone would not hold
    qa = torch.full((M, 128), 448.0, device=DEV).to(E4M3)
    qw = torch.full((256, 128), 448.0, device=DEV).to(E4M3)
    sa = torch.full((M, 1), 2.0 ** -80, device=DEV)
    sw = torch.tensor([[2.0 ** -80], [1.5 * 2.0 ** -69]], device=DEV)
    y = w8.gemm_fp8(qa, sa, qw, sw, out_dtype=torch.float32).double()
    want, T = exact(qa, sa, qw, sw)
    assert torch.all(y[:, :128] == 0) and torch.all(T[:, :128] > 2.0 ** -136)
    assert torch.all(y[:, 128:] == 128 * 448.0 ** 2 * 2.0 ** -148)
    assert torch.all((y - want).abs() <= 2.0 ** -16 * T + 2.0 ** -149 * (1 + 128 * 448.0 ** 2))


def operands(M, N, K, seed=0, mode=w8.SCALE_AMAX):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.randn(M, K, generator=g, device=DEV)
    a[:, ::101] *= 30
    return (*w8.quant_act_fp8(a.to(torch.bfloat16), scale_mode=mode),
            *w8.quant_weight_fp8(torch.randn(N, K, generator=g, device=DEV) * 0.02,
                                 scale_mode=mode))


def exact(qa, sa, qw, sw, rows=None):
    """(y, T) in 64 bits, of some rows."""
    N, K = qw.shape
    if rows is not None:
        qa, sa = qa.view(torch.uint8)[rows].view(E4M3), sa[rows]
    x = qa.double() * sa.double().repeat_interleave(128, 1)
    w = qw.double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    return x @ w.T, x.abs() @ w.abs().T


def check(y, qa, sa, qw, sw, rows=None):
    want, T = exact(qa, sa, qw, sw, rows)
    got = (y if rows is None else y[rows]).double()
    lim = (2.0 ** -16 + (qa.shape[1] // 128 + 1) * 2.0 ** -24) * T
    if y.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * want.abs() + 2.0 ** -8 * lim
    assert torch.all((got - want).abs() <= lim)


SHAPES = [(1, 1, 128), (1, 8, 128), (1, 1000, 256), (2, 129, 384), (5, 4104, 1024), (8, 28672, 512),
          (16, 1024, 1024), (16, 7, 2048), (17, 130, 128), (31, 2050, 640), (32, 10240, 256),
          (33, 333, 1152), (64, 5000, 512), (65, 255, 256), (100, 1536, 1408), (127, 640, 384),
          (128, 4096, 512), (129, 4097, 256), (200, 264, 2048), (333, 1000, 640),
          (777, 4200, 2048), (1000, 72, 384), (1024, 2048, 128), (2049, 1280, 512),
          (4096, 512, 1024), (300, 16384, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    q = operands(M, N, K, seed=M + N)
    for dt in (torch.float32, torch.bfloat16):
        check(w8.gemm_fp8(*q, out_dtype=dt), *q)
    assert w8.device_error() == 0


@pytest.mark.parametrize("M,N,K", [(1, 256, 128), (24, 1000, 512), (130, 392, 1024),
                                   (513, 2064, 256)])
def test_exact_where_sums_are(M, N, K):
    # integers up to 8 and powers of two as scales: every sum is exact in FP32
    g = torch.Generator(device=DEV).manual_seed(3)
    qa = torch.randint(-8, 9, (M, K), generator=g, device=DEV).float().to(E4M3)
    qw = torch.randint(-8, 9, (N, K), generator=g, device=DEV).float().to(E4M3)
    sa = torch.exp2(torch.randint(-2, 2, (M, K // 128), generator=g, device=DEV).float())
    sw = torch.exp2(torch.randint(-2, 2, (-(-N // 128), K // 128), generator=g, device=DEV).float())
    y = w8.gemm_fp8(qa, sa, qw, sw, out_dtype=torch.float32)
    assert torch.equal(y.double(), exact(qa, sa, qw, sw)[0])


@pytest.mark.parametrize("M,N,K", [(4096, 8192, 8192), (8191, 8200, 1024)])
def test_product_large(M, N, K):
    q = operands(M, N, K)
    y = w8.gemm_fp8(*q)
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 1000, 2047, 2048, M - 130, M - 1], device=DEV)
    check(y, *q, rows=rows)
    # every row, by a product in 32 bits (its own error: K additions of 2^-24 of T at most)
    z = w8.gemm_fp8(*q, out_dtype=torch.float32)
    x = q[0].float() * q[1].repeat_interleave(128, 1)
    w = q[2].float() * q[3].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    lim = (2.0 ** -16 + (K // 128 + 1 + K) * 2.0 ** -24) * (x.abs() @ w.abs().T)
    assert torch.all((z - x @ w.T).abs() <= lim)
    assert torch.equal(z.to(torch.bfloat16), y)
    # and each row is what it is by itself, in whatever tile
    for r in (0, 200, M - 1):
        one = w8.gemm_fp8(q[0][r:r + 1], q[1][r:r + 1], q[2], q[3], out_dtype=torch.float32)
        assert torch.equal(one[0], z[r])


@pytest.mark.parametrize("M", [3, 40, 300])
def test_rows_stand_alone(M):
    # a row of NaN codes and one of infinite scales leave the others as they are
    N, K = 392, 640
    qa, sa, qw, sw = operands(M, N, K)
    want = w8.gemm_fp8(qa, sa, qw, sw, out_dtype=torch.float32)
    qa.view(torch.uint8)[1, 5] = 0x7F
    sa[2, 3] = float("inf")
    y = w8.gemm_fp8(qa, sa, qw, sw, out_dtype=torch.float32)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[1:3] = False
    assert torch.equal(y[keep], want[keep])
    assert torch.all(torch.isnan(y[1])) and not torch.any(torch.isfinite(y[2]))
    # and a row's result is that of the row by itself, whatever tile it lands in
    one = w8.gemm_fp8(qa[:1], sa[:1], qw, sw, out_dtype=torch.float32)
    assert torch.equal(one[0], want[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(1, 128), (127, 640), (129, 1152), (392, 4736), (20000, 384),
                                 (40001, 896)])
def test_few_tokens_as_in_many(N, K, dtype):
    # up to 32 tokens the weights' rows are the lanes, else the tokens: the sums are the same
    qa, sa, qw, sw = operands(40, N, K, seed=N)
    want = w8.gemm_fp8(qa, sa, qw, sw, out_dtype=dtype)
    for m in (1, 2, 15, 16, 17, 31, 32):
        y = torch.full((m + 2, N), 7.0, dtype=dtype, device=DEV)
        for r in (0, 40 - m):
            w8.gemm_fp8(qa[r:r + m], sa[r:r + m], qw, sw, out_dtype=dtype, out=y[1:m + 1])
            assert torch.equal(y[1:m + 1], want[r:r + m])
        assert torch.all(y[0] == 7) and torch.all(y[m + 1] == 7)
    assert w8.device_error() == 0


def test_outputs_anywhere():
    q = operands(50, 264, 256)
    want = w8.gemm_fp8(*q)
    buf = torch.zeros(50 * 264 + 16, dtype=torch.bfloat16, device=DEV)
    for off in (0, 1, 8):
        out = buf[off:off + 50 * 264].view(50, 264)
        assert w8.gemm_fp8(*q, out=out) is out
        assert torch.equal(out, want)
    assert torch.all(buf[8 + 50 * 264:] == 0)


@pytest.mark.parametrize("mode", [w8.SCALE_AMAX, w8.SCALE_POW2])
@pytest.mark.parametrize("M,N,K", [(1, 10240, 512), (7, 300, 256), (64, 1024, 1024),
                                   (600, 2000, 384)])
def test_linear_is_both_calls(M, N, K, mode):
    g = torch.Generator(device=DEV).manual_seed(M)
    a = torch.randn(M, K + 24, generator=g, device=DEV).to(torch.bfloat16)[:, 8:8 + K]
    qw, sw = w8.quant_weight_fp8(torch.randn(N, K, generator=g, device=DEV) * 0.02)
    for dt in (torch.float32, torch.bfloat16):
        y = w8.linear_fp8(a, qw, sw, out_dtype=dt, act_scale_mode=mode)
        qa, sa = w8.quant_act_fp8(a, scale_mode=mode)
        assert torch.equal(y, w8.gemm_fp8(qa, sa, qw, sw, out_dtype=dt))


def test_streams_graphs_and_no_tokens():
    g = torch.Generator(device=DEV).manual_seed(0)
    a = torch.randn(20, 512, generator=g, device=DEV).to(torch.bfloat16)
    qw, sw = w8.quant_weight_fp8(torch.randn(1000, 512, generator=g, device=DEV) * 0.02)
    want = w8.linear_fp8(a, qw, sw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = w8.linear_fp8(a, qw, sw, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w8.linear_fp8(a, qw, sw)
        y2 = w8.linear_fp8(y[:, :512], qw, sw)
    a.neg_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, -want)
    assert torch.equal(y2, w8.linear_fp8(y[:, :512], qw, sw))
    assert w8.linear_fp8(a[:0], qw, sw).shape == (0, 1000)


def test_refusals():
    qa, sa, qw, sw = operands(4, 200, 256)
    a = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: w8.gemm_fp8(qa.float(), sa, qw, sw),
                lambda: w8.gemm_fp8(qa, sa[:3], qw, sw),
                lambda: w8.gemm_fp8(qa, sa, qw[:, :128], sw),
                lambda: w8.gemm_fp8(qa, sa, qw, sw[:1]),
                lambda: w8.gemm_fp8(qa, sa, qw, sw, out_dtype=torch.float16),
                lambda: w8.gemm_fp8(qa, sa, qw, sw, out=torch.empty(4, 199, device=DEV)),
                lambda: w8.linear_fp8(a.float(), qw, sw),
                lambda: w8.linear_fp8(a, qw, sw, act_scale_mode=2),
                lambda: w8.linear_fp8(a, qw, sw, workspace=torch.empty(8, dtype=torch.uint8,
                                                                       device=DEV)),
                lambda: w8.quant_act_fp8(a[:, :100]),
                lambda: w8.quant_act_fp8(a, scale_mode=7),
                lambda: w8.quant_weight_fp8(a.float()[:, :64].contiguous())):
        with pytest.raises((ValueError, w8.W8A8Error)):
            bad()
