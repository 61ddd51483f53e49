"""GPU tests that a product reads its weights after the kernels that write them, however early
the kernels of a stream may start.

Most kernels of the library let the next one start before they are done, and wait for the one
before them by themselves. So a writer of weights, started early and still waiting for a long
kernel, may have another call's kernels behind it on the GPU already. The weights here are written
by paged_kv_append at position 0, which copies its queries' bytes (cos 1, sin 0), behind a
quantizer that one CTA works at for some hundred microseconds.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import moe_gemm_gb300 as w8  # noqa: E402

DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn
N, K = 128, 1024


class Late:
    """Writes `value` into `into` (a multiple of 4096 bytes) behind a long kernel, without a wait."""

    def __init__(self, value, into):
        def rows(t):
            return t.view(torch.uint8).view(-1).view(torch.bfloat16).view(-1, 16, 128)

        self.q, self.out = rows(value), rows(into)
        T = self.q.shape[0]
        self.kv = torch.zeros(T, 1, 128, dtype=torch.bfloat16, device=DEV)
        self.pages = [torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        self.pos = torch.zeros(T, dtype=torch.int32, device=DEV)
        self.slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        self.freq = torch.zeros(8, device=DEV)
        self.long = torch.ones(1, 1 << 24, dtype=torch.bfloat16, device=DEV)
        self.codes = torch.empty(1, 1 << 24, dtype=torch.int8, device=DEV)
        self.scale = torch.empty(1, device=DEV)

    def write(self):
        w8.quant_act(self.long, qa=self.codes, sa=self.scale)
        w8.paged_kv_append(self.q, self.kv, self.kv, self.pos, self.slots, self.freq, *self.pages,
                           q_out=self.out)


def check(value, call):
    """call(weights, out) with weights still to be written gives what it gives with them there."""
    want = call(value, None)
    into = torch.zeros_like(value)
    late = Late(value, into)
    got = torch.zeros_like(want)
    late.write()
    torch.cuda.synchronize()
    assert torch.equal(into.view(torch.uint8), value.view(torch.uint8))
    for _ in range(3):
        into.view(torch.uint8).zero_()
        got.zero_()
        torch.cuda.synchronize()
        late.write()
        call(into, got)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert w8.device_error() == 0


def fp8_weights():
    g = torch.Generator(device=DEV).manual_seed(1)
    sign = torch.randint(0, 2, (N, K), generator=g, device=DEV) * 2 - 1
    qw = (torch.randint(1, 9, (N, K), generator=g, device=DEV) * sign).float().to(E4M3)
    return qw, torch.full((1, K // 128), 0.01, device=DEV)


def tokens(M):
    return torch.randn(M, K, generator=torch.Generator(device=DEV).manual_seed(M), device=DEV).to(
        torch.bfloat16)


@pytest.mark.parametrize("M", [1, 24, 40, 300])
def test_fp8_product(M):
    qw, sw = fp8_weights()
    qa, sa = w8.quant_act_fp8(tokens(M))
    check(qw, lambda w, out: w8.gemm_fp8(qa, sa, w, sw, out=out))


@pytest.mark.parametrize("M", [1, 24, 40, 300])
def test_fp8_linear(M):
    qw, sw = fp8_weights()
    a = tokens(M)
    ws = torch.empty(w8.linear_fp8_workspace_size(M, N, K), dtype=torch.uint8, device=DEV)
    check(qw, lambda w, out: w8.linear_fp8(a, w, sw, out=out, workspace=ws))


def int8_weights():
    # (positive codes: no pair of bytes is a BF16 number that is not finite)
    g = torch.Generator(device=DEV).manual_seed(2)
    qw = torch.randint(1, 101, (N, K), generator=g, device=DEV).to(torch.int8)
    return qw, torch.full((N, K // 128), 0.01, device=DEV)


@pytest.mark.parametrize("M", [1, 4, 16, 100, 300])
def test_int8_product(M):
    qw, sw = int8_weights()
    qa, sa = w8.quant_act(tokens(M))
    ws = torch.empty(w8.gemm_workspace_size(M, N, K), dtype=torch.uint8, device=DEV)
    check(qw, lambda w, out: w8.gemm(qa, sa, w, sw, torch.bfloat16, out=out, workspace=ws))


@pytest.mark.parametrize("M", [1, 4, 16, 100, 300])
def test_int8_linear(M):
    qw, sw = int8_weights()
    a = tokens(M)
    ws = torch.empty(w8.linear_workspace_size(M, N, K), dtype=torch.uint8, device=DEV)
    check(qw, lambda w, out: w8.linear(a, w, sw, out=out, workspace=ws))


@pytest.mark.parametrize("M", [1, 16, 300])
def test_int8_weights_alone(M):
    qw, sw = int8_weights()
    a = tokens(M)
    check(qw, lambda w, out: w8.w8a16_gemm(a, w, sw, out=out))


@pytest.mark.parametrize("M", [1, 16, 300])
def test_int8_scales(M):
    qw, _ = int8_weights()
    g = torch.Generator(device=DEV).manual_seed(3)
    sw = torch.exp2(torch.randint(-6, 3, (N, K // 128), generator=g, device=DEV).float())
    qa, sa = w8.quant_act(tokens(M))
    check(sw, lambda s, out: w8.gemm(qa, sa, qw, s, torch.bfloat16, out=out))


def test_experts_weights():
    # (one expert; the gate_up weights, then the down weights, written late)
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(12, 512, generator=g, device=DEV).to(torch.bfloat16)
    up = torch.randint(1, 101, (1, 256, 512), generator=g, device=DEV).to(torch.int8)
    down = torch.randint(1, 101, (1, 512, 128), generator=g, device=DEV).to(torch.int8)
    s_up, s_down = (torch.full(s, 0.01, device=DEV) for s in ((1, 256, 4), (1, 512, 1)))
    ids = torch.zeros(12, 1, dtype=torch.int32, device=DEV)
    w = torch.ones(12, 1, device=DEV)
    ws = torch.empty(w8.moe_ffn_workspace_size(12, 1, 512, 128, 1), dtype=torch.uint8, device=DEV)
    check(up, lambda q, out: w8.moe_ffn(x, ids, w, q, s_up, down, s_down, out=out, workspace=ws))
    check(down, lambda q, out: w8.moe_ffn(x, ids, w, up, s_up, q, s_down, out=out, workspace=ws))


def test_int8_offsets():
    # (where the experts' rows end; the rest of the 4096 bytes is not read)
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randn(40, 256, generator=g, device=DEV).to(torch.bfloat16)
    qw = torch.randint(-127, 128, (4, 128, 256), generator=g, device=DEV).to(torch.int8)
    sw = torch.full((4, 128, 2), 0.01, device=DEV)
    ends = torch.zeros(1024, dtype=torch.int32, device=DEV)
    ends[:5] = torch.tensor([0, 7, 7, 23, 40], device=DEV)
    ws = torch.empty(w8.grouped_linear_workspace_size(40, 4, 128, 256), dtype=torch.uint8, device=DEV)
    check(ends, lambda o, out: w8.grouped_linear(a, o[:5], qw, sw, out=out, workspace=ws))
    check(ends, lambda o, out: w8.w8a16_grouped_gemm(a, o[:5], qw, sw, out=out))
