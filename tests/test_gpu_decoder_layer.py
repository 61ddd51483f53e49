"""A decoder layer's calls together: the serving example with rotated positions and FP8
projections, requests served together against each alone, and a decode step captured
into a graph against the same calls made one by one.
"""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

import moe_gemm_gb300 as w8  # noqa: E402
import paged_serving  # noqa: E402


@pytest.mark.parametrize("args", [["--rotate"], ["--fp8"], ["--rotate", "--fp8"]])
def test_together_as_alone(args):
    # As for the example without these (five BF16 results, 2^-8 each, and INT8 codes that
    # step by one, 2^-6). FP8: where two runs differ by a BF16 step, 2^-8, a code of the output
    # projection's input rounds the other way in a share of 2^-8 / 2^-3 of the places, by 2^-3 of
    # the value at most: sqrt(2^-5) 2^-3 < 2^-5 of the row.
    worst = paged_serving.main(args)
    assert worst < 5 * 2.0 ** -8 + 2.0 ** -6 + (2.0 ** -5 if "--fp8" in args else 0.0)


def test_decode_steps_in_a_graph():
    layer = paged_serving.Layer(rotate=True, fp8=True, seed=5)
    g = torch.Generator(device="cuda").manual_seed(3)
    B = 6
    prompt = torch.randn(B * 20, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
    steps = [torch.randn(B, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
             for _ in range(4)]

    def run(captured):
        cache = paged_serving.Cache(layer, B, pages=64)
        layer(prompt, cache, cache.plan([20] * B, B * 20))
        target = torch.full((B,), 20, dtype=torch.int32, device="cuda")
        x = torch.empty_like(steps[0])

        def step():
            target.add_(1)
            plan = w8.paged_kv_plan(cache.table, cache.lens, target, cache.free, cache.n_free,
                                    cache.page, B)
            return layer(x, cache, plan)

        outs = []
        if captured:
            # (the captured work does not run at capture)
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                y = step()
            torch.cuda.current_stream().wait_stream(stream)
        for s in steps:
            x.copy_(s)
            if captured:
                graph.replay()
            else:
                y = step()
            outs.append(y.clone())
        torch.cuda.synchronize()
        return torch.stack(outs), cache

    eager, c0 = run(False)
    replayed, c1 = run(True)
    assert torch.equal(eager, replayed)
    assert torch.equal(c0.lens, c1.lens) and c0.lens.tolist() == [24] * B
    assert math.isfinite(float(eager.float().abs().max()))
    assert w8.device_error() == 0


def test_rotation_is_relative():
    """Attention over rotated keys depends on distances alone: a request whose positions all
    move by the same number gives the same answer, up to the roundings of q and k
    (BF16, 2^-9 RMS each at most, three times over through the softmax) and of the output."""
    hq, hkv, n, page = 8, 2, 50, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn(n, hq, 128, generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn(n, hkv, 128, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(n, hkv, 128, generator=g, device="cuda").to(torch.bfloat16)
    f = (1e4 ** -(torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    slots = torch.arange(n, **i32)
    table = torch.arange(4, **i32).view(1, 4)
    outs = []
    for shift in (0, 123456):
        kc = torch.zeros(4, hkv, page, 128, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        turned = w8.paged_kv_append(q, k, v, slots + shift, slots, f, kc, vc)
        outs.append(w8.attention_paged(turned, kc, vc, table, torch.tensor([n], **i32),
                                       torch.tensor([0, n], **i32), 1 / math.sqrt(128)).double())
    err = (outs[0] - outs[1]).norm() / outs[0].norm()
    assert err < 2 ** -6
