"""The serving example: requests served together, prompts in pieces over the
paged cache, give what serving each alone in one piece gives, up to rounding."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

import paged_serving  # noqa: E402


def test_together_as_alone():
    # Between the two runs only the grouping of FP32 sums and the kernels'
    # roundings of a weight (2^-11 and less) differ. A BF16 output of a step may
    # then round the other way (2^-8 of it), in five BF16 results that follow one another;
    # an INT8 code of a later layer input may step by one (1 / 254 of a row's
    # largest value, some 2^-6 of a typical one), in few places.
    worst = paged_serving.main([])
    assert worst < 5 * 2.0 ** -8 + 2.0 ** -6


def test_a_tight_pool_serves_all_in_the_end():
    layer = paged_serving.Layer(seed=3)
    g = torch.Generator(device="cuda").manual_seed(2)
    streams = [torch.randn(n, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
               for n in (60, 45, 70)]
    prompts = [50, 40, 64]
    # 9 pages of 16, where the three requests come to need 12: some are refused
    # until others leave
    outs = paged_serving.serve(layer, streams, prompts, chunk=32, pages=9, steps=400)
    assert [None if o is None else len(o) for o in outs] == [60, 45, 70]
    for s, p, o in zip(streams, prompts, outs):
        alone = paged_serving.serve(layer, [s], [p], chunk=len(s))[0]
        assert float((o.float() - alone.float()).norm() / alone.float().norm()) < \
            5 * 2.0 ** -8 + 2.0 ** -6
