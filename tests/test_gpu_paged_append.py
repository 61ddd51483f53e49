"""GPU tests of the append to the paged cache with the position rotation, against
the rotation in 64 bits.

Tolerances. cos and sin come from an angle of at most pi / 4 rounded to binary32, and a
sine and cosine good to 2 ulp: each is off by less than 2^-22. A turned value
a cos - b sin is then off by less than 2^-22 (|a| + |b|) and two roundings, together below
2^-21 (|a| + |b|). Its phase is off by 2^-55 turns per position as well. Then
one rounding: BF16 half a step, 2^-8 of the value; INT8 half a scale.

Source: "Deploying Hunyuan 770B in INT8 on domestic accelerators" §3.4 (the cache's format).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import moe_gemm_gb300 as w8  # noqa: E402

DEV = torch.device("cuda:0")
D = 128


def freqs(rot, base=1e4):
    half = rot // 2
    return torch.pow(torch.tensor(base, dtype=torch.float64),
                     -torch.arange(half, dtype=torch.float64) / half).float().to(DEV)


def make(T, Hq, Hkv, page, int8, far, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    qkv[:, Hq:Hq + Hkv, ::51] *= 8
    P = -(-T // page) * 2 + 1
    slots = torch.randperm(P * page, generator=g, device=DEV)[:T].to(torch.int32)
    pos = torch.randint(0, far, (T,), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots, pos, pages(P, Hkv, page, int8)


def pages(P, Hkv, page, int8):
    if not int8:
        c = [torch.full((P, Hkv, page, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        return dict(k_cache=c[0], v_cache=c[1])
    c = [torch.full((P, Hkv, page, D), 77, dtype=torch.int8, device=DEV) for _ in range(2)]
    s = [torch.full((P, Hkv, page), 7.0, device=DEV) for _ in range(2)]
    return dict(k_cache=c[0], v_cache=c[1], k_scale=s[0], v_scale=s[1])


def turned(x, pos, inv_freq, interleaved, amplitude=1.0):
    """(exact values, bound on what FP32 may be off), float64 numpy."""
    x = x.double().cpu().numpy()
    f = inv_freq.double().cpu().numpy()
    half = len(f)
    p = pos.cpu().numpy().astype(np.float64)
    ang = (p[:, None] * f)[:, None]
    c, s = np.cos(ang) * amplitude, np.sin(ang) * amplitude
    at = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    a, b = x[..., at[0]], x[..., at[1]]
    y, off = x.copy(), np.zeros_like(x)
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    # numpy's own product p f in binary64 is off by 2^-53 of it
    per = (2.0 ** -21 + np.abs(p)[:, None, None] * (2 * math.pi * 2.0 ** -55 + 2.0 ** -53 * f)) * \
        abs(amplitude)
    off[..., at[0]] = off[..., at[1]] = per * (np.abs(a) + np.abs(b))
    return y, off


def slot_rows(cache, slots, page):
    p, o = (slots // page).long(), (slots % page).long()
    return cache[p, :, o]


def check(q, k, v, slots, pos, cache, inv_freq, interleaved, amplitude=1.0, got=None):
    page = cache["k_cache"].shape[2]
    live = (pos >= 0).cpu().numpy()
    held = ((slots >= 0) & (pos >= 0)).cpu().numpy()
    if q is not None:
        y, off = turned(q, pos, inv_freq, interleaved, amplitude)
        err = np.abs(got.double().cpu().numpy() - y)
        assert np.all((err <= 2.0 ** -8 * np.abs(y) + off)[live])
    y, off = turned(k, pos, inv_freq, interleaved, amplitude)
    y, off = y[held], off[held]
    at = slots[torch.from_numpy(held).to(DEV)]
    kc = slot_rows(cache["k_cache"], at, page).double().cpu().numpy()
    if "k_scale" in cache:
        s = slot_rows(cache["k_scale"], at, page).double().cpu().numpy()
        want = np.abs(y).max(-1) / 127
        assert np.all(np.abs(s - want) <= off.max(-1) / 127 + 2.0 ** -23 * want)
        assert np.all(np.abs(kc).max(-1)[want > 0] == 127)
        # half a scale, FP32's error of the value, and that of the quotient's rounding
        lim = 0.5 * s[..., None] + off + 2.0 ** -22 * np.abs(y)
        assert np.all(np.abs(kc * s[..., None] - y) <= lim)
    else:
        assert np.all(np.abs(kc - y) <= 2.0 ** -8 * np.abs(y) + off)
    # v: what paged_kv_write writes, bit for bit, and nothing outside the slots
    ref = pages(cache["k_cache"].shape[0], k.shape[1], page, "k_scale" in cache)
    w8.paged_kv_write(k, v, torch.where(pos >= 0, slots, -1), **ref)
    assert torch.equal(ref["v_cache"], cache["v_cache"])
    if "k_scale" in cache:
        assert torch.equal(ref["v_scale"], cache["v_scale"])
    other = torch.ones(cache["k_cache"].shape[0], page, dtype=torch.bool, device=DEV)
    other[(at // page).long(), (at % page).long()] = False
    for name in cache:
        assert torch.equal(cache[name].transpose(1, 2)[other], ref[name].transpose(1, 2)[other])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,page,rot,far", [
    (1, 64, 8, 64, 128, 131072), (1, 1, 1, 8, 16, 10), (32, 64, 8, 64, 128, 131072),
    (33, 5, 1, 16, 96, 1 << 20), (257, 28, 4, 32, 64, 4096), (700, 3, 3, 1, 48, 1 << 24),
    (3, 40, 8, 128, 112, 1 << 30), (400, 16, 16, 24, 32, 2)])
def test_append(T, Hq, Hkv, page, rot, far, int8, interleaved):
    q, k, v, slots, pos, cache = make(T, Hq, Hkv, page, int8, far, seed=T)
    f = freqs(rot)
    got = w8.paged_kv_append(q, k, v, pos, slots, f, **cache, interleaved=interleaved)
    check(q, k, v, slots, pos, cache, f, interleaved, got=got)


@pytest.mark.parametrize("int8", [False, True])
def test_tokens_without_slot_or_position(int8):
    q, k, v, slots, pos, cache = make(40, 12, 4, 16, int8, 5000)
    pos[3], pos[4], pos[39] = -1, -(1 << 31), -1
    slots[3], slots[7], slots[8], slots[39] = -1, -1, cache["k_cache"].shape[0] * 16, -1
    out = torch.full((40, 12, D), 3.0, dtype=torch.bfloat16, device=DEV)
    got = w8.paged_kv_append(q, k, v, pos, slots, freqs(128), **cache, q_out=out)
    assert got is out
    slots[8] = -1                                   # (outside the pool: as no slot)
    check(q, k, v, slots, pos, cache, freqs(128), False, got=got)
    assert torch.all(out[[3, 4, 39]] == 3.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_of_all_sizes(interleaved):
    q, k, v, slots, pos, cache = make(64, 8, 2, 16, True, 100)
    pos[:] = torch.tensor([(1 << i) - j for i in range(32) for j in (1, 0 if i < 31 else 2)],
                          dtype=torch.int64).clamp(0, 2 ** 31 - 1).to(torch.int32)
    f = freqs(128, 1e7)
    got = w8.paged_kv_append(q, k, v, pos, slots, f, **cache, interleaved=interleaved)
    check(q, k, v, slots, pos, cache, f, interleaved, got=got)


def test_given_frequencies_and_amplitude():
    q, k, v, slots, pos, cache = make(50, 8, 2, 16, True, 3000)
    f = torch.tensor([0.0, 1.0, -0.3, 6.2831855, 2.5, 1e-30, -1.0, 0.5], device=DEV)
    got = w8.paged_kv_append(q, k, v, pos, slots, f, **cache, amplitude=1.25)
    check(q, k, v, slots, pos, cache, f, False, 1.25, got=got)


@pytest.mark.parametrize("T", [5, 2000])
def test_in_place_and_keys_only(T):
    q, k, v, slots, pos, cache = make(T, 24, 8, 16, True, 9000)
    q0, f = q.clone(), freqs(128)
    want = w8.paged_kv_append(q0, k, v, pos, slots, f, **cache)
    first = {n: t.clone() for n, t in cache.items()}
    assert w8.paged_kv_append(q, k, v, pos, slots, f, **cache, q_out=q) is q
    assert torch.equal(q, want)
    assert w8.paged_kv_append(None, k, v, pos, slots, f, **cache) is None
    for n in cache:
        assert torch.equal(first[n], cache[n])


def test_zero_vectors_and_no_tokens():
    q, k, v, slots, pos, cache = make(9, 4, 2, 16, True, 100)
    k[2] = 0
    v[5] = 0
    got = w8.paged_kv_append(q, k, v, pos, slots, freqs(128), **cache)
    check(q, k, v, slots, pos, cache, freqs(128), False, got=got)
    before = {n: t.clone() for n, t in cache.items()}
    out = w8.paged_kv_append(q[:0], k[:0], v[:0], pos[:0], slots[:0], freqs(128), **cache)
    assert out.shape == (0, 4, D)
    assert all(torch.equal(before[n], cache[n]) for n in cache)


def test_stream_and_graph():
    q, k, v, slots, pos, cache = make(100, 16, 4, 16, True, 100000)
    f = freqs(128)
    want = w8.paged_kv_append(q, k, v, pos, slots, f, **cache)
    k_want = cache["k_cache"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w8.paged_kv_append(q, k, v, pos, slots, f, **cache, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = w8.paged_kv_append(q, k, v, pos, slots, f, **cache)
    pos.add_(1)
    g.replay()
    torch.cuda.synchronize()
    check(q, k, v, slots, pos, cache, f, False, got=got)
    pos.sub_(1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(cache["k_cache"], k_want)


def test_refusals():
    q, k, v, slots, pos, cache = make(4, 8, 2, 16, True, 100)
    f = freqs(128)
    ok = dict(q=q, k=k, v=v, positions=pos, slots=slots, inv_freq=f, **cache)

    def refused(**change):
        with pytest.raises((ValueError, w8.W8A8Error)):
            w8.paged_kv_append(**dict(ok, **change))

    refused(positions=pos[:3])
    refused(positions=pos.long())
    refused(slots=slots.cpu())
    refused(inv_freq=f.double())
    refused(inv_freq=f[:4])
    refused(inv_freq=torch.zeros(72, device=DEV))
    refused(inv_freq=torch.zeros(0, device=DEV))
    refused(q=q[:2])
    refused(q=q.float())
    refused(q_out=torch.empty(4, 4, D, dtype=torch.bfloat16, device=DEV))
    refused(q=None, q_out=q)
    refused(v=v[:, :1])
    refused(k=k[:, :1], v=v[:, :1])
    refused(amplitude=float("nan"))
    refused(k_scale=None)


@pytest.mark.parametrize("T", [1, 3, 600])
def test_outputs_beside_or_refused(T):
    q, k, v, slots, pos, cache = make(T, 6, 2, 16, True, 9000)
    f = freqs(128)
    want = w8.paged_kv_append(q, k, v, pos, slots, f, **cache)
    rows = torch.zeros(T, 16, D, dtype=torch.bfloat16, device=DEV)     # q k v and room for q_out
    rows[:, :6], rows[:, 6:8], rows[:, 8:10] = q, k, v
    parts = dict(q=rows[:, :6], k=rows[:, 6:8], v=rows[:, 8:10], positions=pos, slots=slots,
                 inv_freq=f, **cache)
    before = rows.clone()
    got = w8.paged_kv_append(**parts, q_out=rows[:, 10:])
    assert torch.equal(got, want) and torch.equal(rows[:, :10], before[:, :10])
    for out in (rows[:, 1:7], rows[:, 9:15], rows.view(-1)[64:64 + T * 768].view(T, 6, D)):
        with pytest.raises(w8.W8A8Error):
            w8.paged_kv_append(**parts, q_out=out)
    assert torch.equal(rows[:, :10], before[:, :10])
