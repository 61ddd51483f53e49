"""GPU tests of the router's gate against a plain implementation in 64 bits:
the chosen experts exactly, in order, and the weights.

Weights: with FP32 inputs every weight is a quotient of at most 64 + 1 rounded
terms. An exponential of an argument rounded once, |arg| <= 30 in these tests,
is off by 30 * 2^-24 + 2 ulp (2^-22) relative; a sigmoid's term adds two roundings and
a division; the sum of k terms k roundings; the quotient and the factor two:
(30 + 4 + 4 + 64 + 4) * 2 * 2^-24 < 2^-16 relative.

Source: "Deploying Hunyuan 770B in INT8 on domestic accelerators" §1.3.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import moe_gemm_gb300 as w8  # noqa: E402

DEV = torch.device("cuda:0")
TOL = 2.0 ** -16


def reference(x, k, scoring="softmax", bias=None, n_group=1, topk_group=1, renormalize=True,
              scale=1.0):
    x = x.double().cpu()
    T, E = x.shape
    x = torch.where(torch.isnan(x), torch.tensor(-math.inf, dtype=torch.double), x)
    x = x.clamp_max(torch.finfo(torch.float32).max)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.double)
    size = E // n_group
    for t in range(T):
        row = x[t]
        able = row > -math.inf
        if not able.any():
            continue
        if scoring == "softmax":
            e = (row - row.max()).exp()
            s = e / e.sum()
        else:
            s = torch.where(row >= 0, 1 / (1 + (-row).exp()), row.exp() / (1 + row.exp()))
        # without a bias the order of the scores is that of the logits
        key = row.tolist() if bias is None else (s + bias.double().cpu()).tolist()
        groups = []
        for g in range(n_group):
            ks = sorted((key[e] for e in range(g * size, (g + 1) * size) if able[e]), reverse=True)
            if not ks:
                groups.append(-math.inf)
            else:
                groups.append(ks[0] if bias is None or len(ks) == 1 else ks[0] + ks[1])
        kept = sorted(range(n_group), key=lambda g: (-groups[g], g))[:topk_group]
        cand = [e for e in range(E) if able[e] and e // size in kept]
        cand = sorted(cand, key=lambda e: (-key[e], e))[:k]
        if scoring == "sigmoid" and renormalize:      # without underflow of the sum
            r = min(0.0, max(float(row[e]) for e in cand))
            num = [math.exp(min(float(row[e]), 0.0) - r) / (1 + math.exp(-abs(float(row[e]))))
                   for e in cand]
        elif renormalize:
            r = max(float(row[e]) for e in cand)
            num = [math.exp(float(row[e]) - r) for e in cand]
        else:
            num = [float(s[e]) for e in cand]
        den = sum(num) if renormalize else 1.0
        for j, e in enumerate(cand):
            ids[t, j] = e
            w[t, j] = num[j] / den * scale
    return ids, w


def check(x, k, **kw):
    ids, w = w8.moe_gate(x, k, **kw)
    torch.cuda.synchronize()
    rid, rw = reference(x, k, **kw)
    assert torch.equal(ids.cpu(), rid)
    err = (w.cpu().double() - rw).abs()
    assert bool((err <= TOL * rw.abs() + 1e-37).all()), float((err / rw.abs().clamp_min(1e-30)).max())
    return ids, w


def logits(T, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(dtype).to(DEV)


def bias_of(E, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(E, generator=g) * 0.05).to(DEV)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 64, 8), (3, 1, 1), (7, 33, 5), (4, 100, 8),
                                   (130, 256, 8), (2, 511, 16), (3, 1024, 64), (6, 48, 48)])
def test_sizes(T, E, k, dtype, scoring):
    check(logits(T, E, T + E, dtype), k, scoring=scoring)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,n_group,topk_group,k", [(256, 8, 4, 8), (64, 4, 1, 8), (60, 5, 2, 7),
                                                    (64, 64, 9, 5), (192, 8, 3, 6), (160, 10, 10, 6),
                                                    (1024, 16, 2, 8), (48, 48, 48, 3)])
def test_groups(E, n_group, topk_group, k, with_bias, scoring):
    check(logits(37, E, E + n_group), k, scoring=scoring,
          bias=bias_of(E, 7) if with_bias else None, n_group=n_group, topk_group=topk_group,
          scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_without_renormalising(scoring):
    check(logits(21, 64, 3), 6, scoring=scoring, renormalize=False, scale=0.5)
    check(logits(21, 64, 3), 6, scoring=scoring, renormalize=False, bias=bias_of(64, 9))


@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lower_expert(with_bias):
    x = torch.zeros(9, 64, device=DEV)
    x[1] = 1.0
    x[2, ::2] = -0.0
    x[3, 5:9] = 2.0
    bias = torch.zeros(64, device=DEV) if with_bias else None
    ids, w = check(x, 8, bias=bias)
    assert ids[0].tolist() == list(range(8))
    assert ids[3].tolist()[:4] == [5, 6, 7, 8]
    check(x, 8, scoring="sigmoid", bias=bias, n_group=8, topk_group=3)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_keys_closer_than_32_bits_resolve(scoring):
    # scores + bias that agree to far below 2^-24: experts e and e + 1 differ by
    # one unit of the logit's last place, against a bias that cancels it nearly
    g = torch.Generator().manual_seed(11)
    T, E = 64, 64
    x = torch.randn(T, E, generator=g)
    x[:, 1::2] = x[:, ::2]
    bits = x.view(torch.int32)
    bits[:, 1::2] += torch.randint(-2, 3, (T, E // 2), generator=g, dtype=torch.int32)
    bias = torch.zeros(E)
    check(x.to(DEV), 8, scoring=scoring, bias=bias.to(DEV))
    bias[1::2] = 1e-9
    check(x.to(DEV), 8, scoring=scoring, bias=bias.to(DEV), n_group=4, topk_group=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(scoring, with_bias):
    x = logits(8, 64, 5)
    x[0] = -math.inf                       # nothing to pick
    x[1, 3:] = -math.inf                   # fewer than k
    x[2, ::3] = math.nan
    x[3] = math.nan
    x[4, 10] = math.inf
    x[5, :32] = -math.inf                  # whole groups
    x[6, 1:] = -math.inf
    bias = bias_of(64, 2) if with_bias else None
    ids, w = check(x, 8, scoring=scoring, bias=bias)
    assert bool((ids[0] == -1).all()) and bool((w[0] == 0).all())
    check(x, 8, scoring=scoring, bias=bias, n_group=4, topk_group=2)


@pytest.mark.parametrize("E,n_group,topk_group", [(64, 1, 1), (256, 8, 4), (60, 5, 2), (512, 4, 2)])
def test_biases_that_mark_experts(E, n_group, topk_group):
    x, b = logits(41, E, 31), bias_of(E, 32)
    never = torch.arange(0, E, 3, device=DEV)
    b[never] = torch.where(never % 2 == 0, math.nan, -math.inf)
    kw = dict(n_group=n_group, topk_group=topk_group)
    ids, w = w8.moe_gate(x, 8, scoring="sigmoid", bias=b, **kw)
    masked = x.clone()
    masked[:, never] = -math.inf
    rid, rw = reference(masked, 8, scoring="sigmoid", bias=b.nan_to_num(0.0, neginf=0.0), **kw)
    assert torch.equal(ids.cpu(), rid)
    assert bool(((w.cpu().double() - rw).abs() <= TOL * rw).all())
    ids, w = w8.moe_gate(x, 8, scoring="softmax", bias=b, **kw)
    assert not bool(torch.isin(ids, never.int()).any()) and bool(torch.isfinite(w).all())


def clustered(T, E, seed):
    """Logits in few narrow clusters, and biases of two values:
    keys and group scores that 32 bits cannot tell apart are common (and 1e-11
    apart or more, which 64 bits do tell)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-3, 4, (T, E), generator=g) * 0.5 + torch.randn(T, E, generator=g) * 1e-4
    b = torch.randint(0, 2, (E,), generator=g) * 0.05
    return x.float().to(DEV), b.float().to(DEV)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,k", [(24, 4, 2, 4), (64, 8, 3, 6), (60, 5, 2, 3),
                                                    (256, 8, 4, 8), (256, 32, 5, 8)])
def test_close_groups_resolve(E, n_group, topk_group, k, scoring):
    x, b = clustered(64, E, E + n_group)
    check(x, k, scoring=scoring, bias=b, n_group=n_group, topk_group=topk_group)


def test_far_logits():
    x = logits(6, 64, 8) * 40
    x[1] -= 300
    x[2] += 300
    for scoring in ("softmax", "sigmoid"):
        ids, w = w8.moe_gate(x, 8, scoring=scoring)
        rid, rw = reference(x, 8, scoring=scoring)
        assert torch.equal(ids.cpu(), rid)
        # the argument of an exponential is rounded once: 2^-24 of |x| <= 640
        assert bool(((w.cpu().double() - rw).abs() <= (TOL + 640 * 2.0 ** -23) * rw + 1e-37).all())
        assert bool((w.sum(-1) - 1).abs().max() < 1e-4)


def test_strided_logits_and_outputs():
    full = logits(17, 96, 12, torch.bfloat16)
    x = full[:, 16:80]
    ids = torch.full((17, 4), -7, dtype=torch.int32, device=DEV)
    w = torch.full((17, 4), -7.0, device=DEV)
    a, b = w8.moe_gate(x, 4, topk_ids=ids, topk_w=w)
    assert a is ids and b is w
    rid, rw = reference(x, 4)
    assert torch.equal(ids.cpu(), rid)
    assert bool(((w.cpu().double() - rw).abs() <= TOL * rw).all())


def test_stream_and_graph():
    x = logits(33, 64, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, w = w8.moe_gate(x, 8, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    with torch.cuda.graph(g):
        w8.moe_gate(x, 8, topk_ids=ids2, topk_w=w2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_feeds_the_expert_ffn():
    T, H, I, E, k = 9, 256, 128, 8, 2
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    up = (torch.randn(E, 2 * I, H, generator=g) * 0.02).to(DEV)
    down = (torch.randn(E, H, I, generator=g) * 0.02).to(DEV)
    qu, su = zip(*(w8.quant_weight(up[e]) for e in range(E)))
    qd, sd = zip(*(w8.quant_weight(down[e]) for e in range(E)))
    args = [torch.stack(z) for z in (qu, su, qd, sd)]
    lg = logits(T, E, 6)
    ids, w = w8.moe_gate(lg, k)
    y = w8.moe_ffn(x, ids, w, *args, out_dtype=torch.float32)
    rid, rw = reference(lg, k)
    y2 = w8.moe_ffn(x, rid.to(DEV), rw.float().to(DEV), *args, out_dtype=torch.float32)
    assert bool(((y - y2).abs() <= 2 * TOL * y2.abs().max()).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,k", [(24, 4, 2, 4), (64, 8, 3, 6), (60, 5, 2, 3),
                                                    (256, 8, 4, 8), (256, 32, 5, 8), (64, 1, 1, 8)])
def test_nan_biases_among_close_groups(E, n_group, topk_group, k, scoring):
    # (for the reference: keys far below all others, never among a group's two largest here)
    x, b = clustered(64, E, 2 * E + n_group)
    never = torch.arange(1, E, 3, device=DEV)
    low = b.clone()
    b[never], low[never] = math.nan, -1e30
    kw = dict(scoring=scoring, n_group=n_group, topk_group=topk_group)
    ids, w = w8.moe_gate(x, k, bias=b, **kw)
    rid, rw = reference(x, k, bias=low, **kw)
    assert torch.equal(ids.cpu(), rid)
    assert bool(((w.cpu().double() - rw).abs() <= TOL * rw).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group", [(64, 8, 4), (256, 32, 9), (256, 8, 3), (96, 8, 4),
                                                  (1024, 32, 8)])
@pytest.mark.parametrize("size", [100.0, 300.0, 1000.0])
def test_group_sums_of_large_opposite_keys(size, E, n_group, topk_group, scoring):
    # a group's two largest keys nearly cancel: its score is small, its 32-bit error that of the keys.
    # (No two groups' keys are close, so the picks themselves are clear.)
    g = torch.Generator().manual_seed(int(size) + E)
    T, per = 96, E // n_group
    x = torch.randn(T, n_group, per, generator=g) * 1e-4
    b = torch.full((n_group, per), -4 * size)
    up = size + 7 * torch.arange(n_group)
    b[:, per // 2], b[:, 1] = up, 0.25 - up
    x, b = x.view(T, E).to(DEV), b.view(E).to(DEV)
    check(x, 2 * topk_group, scoring=scoring, bias=b, n_group=n_group, topk_group=topk_group)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_token_has_no_row_stride(dtype):
    x = logits(64, 1, 3, dtype).t()
    assert x.shape == (1, 64) and x.stride() == (1, 1)
    check(x, 8)
    check(logits(64, 1, 3, dtype).t()[:, :40], 8, scoring="sigmoid", bias=bias_of(40, 1))


def test_one_expert_has_no_column_stride():
    x = logits(2, 7, 3).t()[:, 1:]
    assert x.shape == (7, 1) and x.stride() == (1, 7)
    check(x, 1, scoring="sigmoid")
