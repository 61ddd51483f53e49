"""Cases of the serving operators: expert gating, the paged KV cache and the
attention over it.

Each case is a dict of plain values. prepare() makes what a serving program
has in hand before a step, run() makes one pass through the operator, and
exact() computes the same outputs from the definition in 64 bits. With
own = False, run() uses elementary torch operations in 32 bits (64 where a
comparison decides a whole number); with own = True it makes the calls that
a user makes of the package.

Operators:
  gate   scores of the experts, group-limited top-k, weights (what moe_ffn takes)
  plan   block tables, slot map and positions from request lengths
  write  new K and V vectors into the pages, INT8 with one scale per vector, or BF16
  attend attention of each request's new tokens over its pages
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension


# ------------------------------------------------------------------ the cases
def listed():
    """The listed cases; each comment says what it stands for. Lengths of several
    requests are a text: one number for each request."""
    return [
        # the router of one decode step: few tokens, softmax over 64 experts, top-8
        {"name": "gate_decode", "op": "gate", "T": 16, "E": 64, "k": 8, "dtype": "float32",
         "scoring": "softmax", "bias": False, "n_group": 1, "topk_group": 1},
        # the router of a chunk of prompt tokens over 64 experts, BF16 logits
        {"name": "gate_prompt", "op": "gate", "T": 8191, "E": 64, "k": 8, "dtype": "bfloat16",
         "scoring": "softmax", "bias": False, "n_group": 1, "topk_group": 1},
        # a balanced sigmoid router with expert groups over a large prompt batch
        {"name": "gate_groups", "op": "gate", "T": 16384, "E": 256, "k": 8, "dtype": "float32",
         "scoring": "sigmoid", "bias": True, "n_group": 8, "topk_group": 4},
        # one decode step of 32 requests: one new position each, now and then a new page
        {"name": "plan_decode", "op": "plan", "B": 32, "page": 64, "ctx": 4096, "new": 1,
         "growing": 32, "leaving": 0},
        # a continuous batch: decodes, prompts of up to 1024 tokens, and requests that leave
        {"name": "plan_mixed", "op": "plan", "B": 1021, "page": 16, "ctx": 8192, "new": 1024,
         "growing": 900, "leaving": 61},
        # K and V of one decode step of 32 requests into the INT8 pages
        {"name": "write_decode", "op": "write", "T": 32, "Hkv": 8, "page": 64, "int8": True},
        # K and V of a chunk of prompt tokens into the INT8 pages
        {"name": "write_prompt", "op": "write", "T": 8192, "Hkv": 8, "page": 64, "int8": True},
        # a single request decoding early in its answer: the latency of one small call
        {"name": "attend_one", "op": "attend", "n_new": "1", "ctx": "777", "Hq": 64,
         "Hkv": 8, "page": 64, "int8": True, "window": 0},
        # a decode step of 32 requests of up to 4096 positions, INT8 pages
        {"name": "attend_decode", "op": "attend", "n_new": _text([1] * 32),
         "ctx": _text(4096 - 61 * i for i in range(32)), "Hq": 64, "Hkv": 8, "page": 64,
         "int8": True, "window": 0},
        # four requests decoding far into long contexts, BF16 pages
        {"name": "attend_decode_long", "op": "attend", "n_new": "1 1 1 1",
         "ctx": "131071 65537 98304 33333", "Hq": 64, "Hkv": 8, "page": 128,
         "int8": False, "window": 0},
        # a continuous batch: a chunk of a long prompt over what is cached of it, with decodes
        {"name": "attend_chunk", "op": "attend", "n_new": "2048 1 1 1 1 1 1 1 1",
         "ctx": "30001 512 4097 8192 1500 2999 100 16000 1", "Hq": 64, "Hkv": 8,
         "page": 64, "int8": True, "window": 0},
        # whole prompts of different lengths packed into one call, BF16 pages
        {"name": "attend_prompts", "op": "attend",
         "n_new": "8192 1 333 4096 1777 1000 129 64", "ctx": "0 0 0 0 0 0 0 0",
         "Hq": 64, "Hkv": 8, "page": 32, "int8": False, "window": 0},
    ]


def _text(lengths):
    return " ".join(str(n) for n in lengths)


def _lengths(case):
    """(new tokens, cached positions) of each request."""
    return [int(n) for n in case["n_new"].split()], [int(n) for n in case["ctx"].split()]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["gate", "plan", "write", "attend", "attend", "attend"])
    if op == "gate":
        n_group = rng.choice([1, 1, 4, 8])
        E = n_group * rng.randint(max(2, 16 // n_group), 256 // n_group)
        topk_group = rng.randint(max(1, n_group // 2), n_group)
        k = rng.randint(1, min(8, topk_group * (E // n_group)))
        return {"op": "gate", "T": _log_int(rng, 1, 16384), "E": E, "k": k,
                "dtype": rng.choice(["float32", "bfloat16"]),
                "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "n_group": n_group, "topk_group": topk_group}
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        growing = rng.randint((B + 1) // 2, B)
        return {"op": "plan", "B": B, "page": rng.choice([16, 32, 64, 128]),
                "ctx": _log_int(rng, 64, 8192), "new": _log_int(rng, 1, 1024),
                "growing": growing, "leaving": rng.randint(0, B - growing)}
    if op == "write":
        return {"op": "write", "T": _log_int(rng, 1, 8192), "Hkv": rng.choice([1, 2, 4, 8]),
                "page": rng.choice([16, 32, 64, 128]), "int8": rng.random() < 0.7}
    Hkv = rng.choice([1, 2, 4, 8])
    G = min(rng.choice([1, 2, 4, 5, 7, 8, 16]), 64 // Hkv)
    kind = rng.choice(["decode", "decode", "few", "chunk", "prompts", "mixed"])
    if kind == "decode":
        B = _log_int(rng, 1, 48)
        top = _log_int(rng, 64, min(131072, 262144 // B))
        n_new = [1] * B
        ctx = [rng.randint(0, top) for _ in range(B)]
    elif kind == "few":
        # several guessed tokens of each request are checked in one step
        B = _log_int(rng, 1, 32)
        top = _log_int(rng, 64, 8192)
        n_new = [rng.randint(1, 8) for _ in range(B)]
        ctx = [rng.randint(0, top) for _ in range(B)]
    elif kind == "chunk":
        B = rng.randint(1, 2)
        n_new = [_log_int(rng, 16, 1024) for _ in range(B)]
        ctx = [_log_int(rng, 1, 24000) for _ in range(B)]
    elif kind == "prompts":
        B = _log_int(rng, 1, 16)
        n_new = [_log_int(rng, 1, 2048) for _ in range(B)]
        ctx = [0] * B
    else:
        B = rng.randint(2, 24)
        n_new = [_log_int(rng, 1, 1024) if rng.random() < 0.2 else 1 for _ in range(B)]
        ctx = [_log_int(rng, 1, 8192) for _ in range(B)]
    return {"op": "attend", "n_new": _text(n_new), "ctx": _text(ctx), "Hq": Hkv * G,
            "Hkv": Hkv, "page": rng.choice([16, 32, 64, 128]), "int8": rng.random() < 0.6,
            "window": rng.choice([0, 0, 0, _log_int(rng, 32, 4096)])}


# ------------------------------------------------------------------- the data
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _pages(n, page):
    return (n + page - 1) // page


def _plan_state(case, seed):
    rng = np.random.default_rng(seed)
    B, page = case["B"], case["page"]
    held = rng.integers(0, case["ctx"] + 1, B)
    target = held.copy()
    order = rng.permutation(B)
    grow = order[:case["growing"]]
    # most requests that grow decode one position; one in 64 brings a prompt, whose
    # lengths are spread evenly up to the longest
    step = np.ones(len(grow), dtype=np.int64)
    prompts = len(grow) // 64
    if prompts:
        step[:prompts] = np.maximum(case["new"] * np.arange(1, prompts + 1) // prompts, 1)
    target[grow] += step
    target[order[case["growing"]:case["growing"] + case["leaving"]]] = 0
    have, want = _pages(held, page), _pages(target, page)
    W = _pages(case["ctx"] + case["new"], page)
    # the pool is shared: what these requests neither hold nor find free is others'.
    # One call in three finds it tight: the last requests that need pages get none
    P = B * W + 16
    used = int(have.sum())
    lack = int((want - have).sum())
    n_free = max(0, lack - 1) if rng.random() < 1 / 3 else max(lack, 0) + 8
    n_free = min(n_free, P - used)
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((B, W), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.full(P, -1, dtype=np.int32)
    free[:n_free] = ids[used:used + n_free]
    state = {"case": case, "tokens": int(step.sum()), "target": _ints(target.tolist()),
             "table0": torch.from_numpy(table).cuda(), "lens0": _ints(held.tolist()),
             "free0": torch.from_numpy(free).cuda(), "n_free0": _ints([n_free])}
    for name in ("table", "lens", "free", "n_free"):
        state[name] = state[name + "0"].clone()
    return state


def _write_state(case, g):
    T, Hkv, page = case["T"], case["Hkv"], case["page"]
    P = _pages(T, page) * 2 + 1
    # K and V are parts of one fused projection's rows, behind 8 Hkv query heads
    qkv = torch.randn(T, 10 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, 8 * Hkv:9 * Hkv], qkv[:, 9 * Hkv:]
    k[..., ::51] *= 8                                 # channels that stand out in K
    slots = torch.randperm(P * page, generator=g, device="cuda")[:T].to(torch.int32)
    dt = torch.int8 if case["int8"] else torch.bfloat16
    state = {"case": case, "k": k, "v": v, "slots": slots, "ks": None, "vs": None,
             "kc": torch.zeros(P, Hkv, page, D, dtype=dt, device="cuda"),
             "vc": torch.zeros(P, Hkv, page, D, dtype=dt, device="cuda")}
    if case["int8"]:
        state["ks"] = torch.zeros(P, Hkv, page, device="cuda")
        state["vs"] = torch.zeros(P, Hkv, page, device="cuda")
    return state


def _attend_state(case, g):
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    n_new, ctx = _lengths(case)
    B = len(n_new)
    kv = [c + n for c, n in zip(ctx, n_new)]
    have = [_pages(n, page) for n in kv]
    P, W = sum(have) + 3, max(have)
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    cu, at = [0], 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
        cu.append(cu[-1] + n_new[b])
    q = torch.randn(cu[-1], Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    kc = torch.empty(P, Hkv, page, D, dtype=torch.int8 if case["int8"] else torch.bfloat16,
                     device="cuda")
    vc = torch.empty_like(kc)
    ks = vs = None
    if case["int8"]:
        ks = torch.empty(P, Hkv, page, device="cuda")
        vs = torch.empty(P, Hkv, page, device="cuda")
    step = max(1, (1 << 28) // (Hkv * page * D))      # a part of the pool at a time
    for i in range(0, P, step):
        for c, s in ((kc, ks), (vc, vs)):
            x = torch.randn(c[i:i + step].shape, generator=g, device="cuda")
            if c is kc:
                x[..., ::51] *= 8                     # channels that stand out in K
            if case["int8"]:
                m = x.abs().amax(-1) / 127
                s[i:i + step] = m
                c[i:i + step] = torch.round(x / m[..., None]).to(torch.int8)
            else:
                c[i:i + step] = x.to(torch.bfloat16)
    return {"case": case, "q": q, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "table": table,
            "kv_lens": _ints(kv), "cu_new": _ints(cu), "cu": cu, "kv": kv, "n_new": n_new,
            "scale": 1.0 / math.sqrt(D)}


def prepare(case, seed):
    op = case["op"]
    if op == "plan":
        return _plan_state(case, seed)
    g = _gen(seed)
    if op == "write":
        return _write_state(case, g)
    if op == "attend":
        return _attend_state(case, g)
    x = torch.randn(case["T"], case["E"], generator=g, device="cuda") * 1.5
    bias = None
    if case["bias"]:
        bias = torch.randn(case["E"], generator=g, device="cuda") * 0.05
    return {"case": case, "x": x.to(getattr(torch, case["dtype"])), "bias": bias}


# ------------------------------------------------------------- the plain forms
def _plain_gate(s):
    c = s["case"]
    E, k, n_group = c["E"], c["k"], c["n_group"]
    x = s["x"].double()          # a selection is decided next to borders
    if c["scoring"] == "softmax":
        x = x - x.amax(-1, keepdim=True)
        score = x.exp() / x.exp().sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + (-x).exp())
    key = score if s["bias"] is None else score + s["bias"].double()
    if n_group > 1:
        by = key.view(-1, n_group, E // n_group).sort(dim=-1, descending=True).values
        gs = by[..., 0] if s["bias"] is None or E == n_group else by[..., 0] + by[..., 1]
        order = gs.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(keep.repeat_interleave(E // n_group, 1), key, -math.inf)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": w.float()}


def _plain_plan(s):
    page, n_tokens = s["case"]["page"], s["tokens"]
    table, lens, free = s["table0"], s["lens0"].long(), s["free0"]
    target = s["target"].long()
    B, W = table.shape
    P = free.shape[0]
    have, want = _pages(lens, page), _pages(target, page)
    col = torch.arange(W, device="cuda")
    # pages given back, in request order
    back = torch.where(target < lens, have - want, 0)
    first = s["n_free0"].long() + back.cumsum(0) - back
    gone = (col >= want[:, None]) & (col < have[:, None]) & (target < lens)[:, None]
    at = torch.where(gone, first[:, None] + col - want[:, None], P)
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, at.flatten(), table.flatten())[:P]
    have_free = s["n_free0"].long() + back.sum()
    # pages taken, in request order, as long as they last
    asked = (target - lens).clamp_min(0)
    cu = asked.cumsum(0)
    fits = (target > lens) & (want <= W) & (cu <= n_tokens)
    need = torch.where(fits, want - have, 0)
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= have_free))
    taken = torch.where(served, need, 0)
    new = (col >= have[:, None]) & (col < want[:, None]) & served[:, None]
    src = have_free - 1 - ((upto - need)[:, None] + col - have[:, None])
    out = torch.where(gone, -1, table)
    out = torch.where(new, stack[src.clamp(0, P - 1)], out)
    # the new tokens' positions and slots
    t = torch.arange(n_tokens, device="cuda")
    b = torch.searchsorted(cu, t, right=True).clamp_max(B - 1)
    pos = lens[b] + t - (cu - asked)[b]
    ok = served[b] & (t < cu[-1])
    slot = out[b, (pos // page).clamp(0, W - 1)].long() * page + pos % page
    refused = (target > lens) & ~served
    return {"table": out, "lens": torch.where(refused, lens, target).int(), "free": stack,
            "n_free": (have_free - taken.sum()).int().view(1),
            "cu_new": torch.cat([cu.new_zeros(1), cu]).int(),
            "kv_lens": torch.where(refused, 0, target).int(),
            "slots": torch.where(ok, slot, -1).int(),
            "positions": torch.where(ok, pos, -1).int()}


def _written(s):
    """The vectors that the slots hold, as the values they stand for."""
    page = s["case"]["page"]
    p, off = (s["slots"] // page).long(), (s["slots"] % page).long()
    if s["ks"] is None:
        return {"k": s["kc"][p, :, off], "v": s["vc"][p, :, off]}
    return {"k": s["kc"][p, :, off] * s["ks"][p, :, off, None],
            "v": s["vc"][p, :, off] * s["vs"][p, :, off, None]}


def _plain_write(s):
    page = s["case"]["page"]
    p, off = (s["slots"] // page).long(), (s["slots"] % page).long()
    for x, cache, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        if scales is None:
            cache[p, :, off] = x
            continue
        x = x.float()
        top = x.abs().amax(-1)
        m = top / torch.full_like(top, 127)      # one rounding, as the format defines it
        scales[p, :, off] = m
        cache[p, :, off] = torch.round(x / torch.where(m > 0, m, 1.0)[..., None]).to(torch.int8)
    return _written(s)


def _plain_attend(s):
    c = s["case"]
    Hq, Hkv, page, window = c["Hq"], c["Hkv"], c["page"], c["window"]
    G = Hq // Hkv
    out = torch.zeros_like(s["q"])
    for b, n in enumerate(s["n_new"]):
        L = s["kv"][b]
        p = s["table"][b, :_pages(L, page)].long()

        def rows(cache, scales):
            x = cache[p].float()
            if scales is not None:
                x = x * scales[p][..., None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :L]

        k, v = rows(s["kc"], s["ks"]), rows(s["vc"], s["vs"])
        q = s["q"][s["cu"][b]:s["cu"][b + 1]].float().view(n, Hkv, G, D).transpose(0, 1)
        step = max(1, (1 << 28) // (Hq * L))          # rows of scores at a time
        j = torch.arange(L, device="cuda")
        for i in range(0, n, step):
            qi = q[:, i:i + step].reshape(Hkv, -1, D)
            pos = L - n + torch.arange(i, min(n, i + step), device="cuda")
            seen = j <= pos[:, None]
            if window > 0:
                seen &= j > pos[:, None] - window
            seen = seen.repeat_interleave(G, 0)
            w = torch.matmul(qi, k.transpose(1, 2)) * s["scale"]
            w = torch.where(seen, w, -math.inf)
            w = (w - w.amax(-1, keepdim=True)).exp()
            o = torch.matmul(w, v) / w.sum(-1, keepdim=True)
            out[s["cu"][b] + i:s["cu"][b] + i + len(pos)] = \
                o.view(Hkv, -1, G, D).transpose(0, 1).reshape(-1, Hq, D).to(out.dtype)
    return out


# ------------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if op == "plan":
        for name in ("table", "lens", "free", "n_free"):     # the call updates them in place
            s[name].copy_(s[name + "0"])
    if not own:
        return {"gate": _plain_gate, "plan": _plain_plan, "write": _plain_write,
                "attend": _plain_attend}[op](s)
    import moe_gemm_gb300 as w8
    if op == "gate":
        ids, w = w8.moe_gate(s["x"], c["k"], scoring=c["scoring"], bias=s["bias"],
                             n_group=c["n_group"], topk_group=c["topk_group"])
        return {"ids": ids, "w": w}
    if op == "plan":
        cu_new, kv_lens, slots, positions = w8.paged_kv_plan(
            s["table"], s["lens"], s["target"], s["free"], s["n_free"], c["page"], s["tokens"])
        return {"table": s["table"], "lens": s["lens"], "free": s["free"],
                "n_free": s["n_free"], "cu_new": cu_new, "kv_lens": kv_lens, "slots": slots,
                "positions": positions}
    if op == "write":
        w8.paged_kv_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"], k_scale=s["ks"],
                          v_scale=s["vs"])
        return _written(s)
    return w8.attention_paged(s["q"], s["kc"], s["vc"], s["table"], s["kv_lens"], s["cu_new"],
                              s["scale"], k_scale=s["ks"], v_scale=s["vs"], window=c["window"])


def _pairs(case):
    """(query, key) pairs that the masks leave, and the positions that some query sees."""
    pairs = seen = 0
    for n, ctx in zip(*_lengths(case)):
        w = case["window"]
        if w == 0:
            pairs += n * ctx + n * (n + 1) // 2
            seen += ctx + n
        else:
            full = max(0, min(n, w - ctx))            # queries that see fewer than w keys
            pairs += full * ctx + full * (full + 1) // 2 + (n - full) * w
            seen += min(ctx + n, w + n - 1)
    return pairs, seen


def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * E * size + T * k * 8 + (4 * E if case["bias"] else 0),
                "flops": T * E * 4}
    if op == "plan":
        B, page = case["B"], case["page"]
        prompts = case["growing"] // 64
        tokens = case["growing"] + sum(max(case["new"] * i // prompts, 1) - 1
                                       for i in range(1, prompts + 1))
        pages = tokens // page + case["leaving"] * case["ctx"] // (2 * page)
        # lengths in and out, a free page read and a table entry written for each new
        # page, and of each token its slot and position
        return {"bytes": B * 5 * 4 + pages * 8 + tokens * 8, "flops": 0}
    if op == "write":
        n = case["T"] * case["Hkv"] * 2
        return {"bytes": n * (2 * D + (D + 4 if case["int8"] else 2 * D)) + case["T"] * 4,
                "flops": n * D * 2}
    pairs, seen = _pairs(case)
    row = D + 4 if case["int8"] else 2 * D
    n_new, ctx = _lengths(case)
    pages = sum(_pages(c + n, case["page"]) for c, n in zip(ctx, n_new))
    return {"bytes": 2 * seen * case["Hkv"] * row + sum(n_new) * case["Hq"] * D * 4 +
            pages * 4 + 8 * len(n_new), "flops": 4 * D * case["Hq"] * pairs}


# --------------------------------------------------------- definitions, 64 bits
def _exact_gate(s):
    c = s["case"]
    E, k, n_group = c["E"], c["k"], c["n_group"]
    x = s["x"].double().cpu().numpy()
    if c["scoring"] == "softmax":
        score = np.exp(x - np.logaddexp.reduce(x, axis=1)[:, None])
    else:
        score = np.where(x >= 0, 1.0, np.exp(-np.abs(x))) / (1 + np.exp(-np.abs(x)))
    key = score.copy()
    if s["bias"] is not None:
        key += s["bias"].double().cpu().numpy()
    if n_group > 1:
        size = E // n_group
        top = np.sort(key.reshape(-1, n_group, size), axis=2)
        gs = top[:, :, -1]
        if s["bias"] is not None and size > 1:
            gs = gs + top[:, :, -2]
        rank = np.argsort(np.argsort(-gs, axis=1, kind="stable"), axis=1, kind="stable")
        key[np.repeat(rank >= c["topk_group"], size, axis=1)] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(score, ids, axis=1)
    w /= w.sum(axis=1, keepdims=True)
    return {"ids": torch.from_numpy(ids.astype(np.int32)).cuda(), "w": torch.from_numpy(w).cuda()}


def _exact_plan(s):
    page = s["case"]["page"]
    table = s["table0"].cpu().numpy().copy()
    held, target = s["lens0"].cpu().tolist(), s["target"].cpu().tolist()
    free = s["free0"].cpu().numpy().copy()
    n_free = int(s["n_free0"].item())
    B, W = table.shape
    lens, kv = list(held), list(held)
    for b in range(B):                                 # pages given back first
        if target[b] < held[b]:
            for j in range(-(-target[b] // page), -(-held[b] // page)):
                free[n_free] = table[b, j]
                table[b, j] = -1
                n_free += 1
            lens[b] = kv[b] = target[b]
    cu, slots, positions, asked_pages, top = [0], [], [], 0, n_free
    for b in range(B):
        n = max(0, target[b] - held[b])
        cu.append(cu[-1] + n)
        if n == 0:
            continue
        have, want = -(-held[b] // page), -(-target[b] // page)
        ok = want <= W and cu[-1] <= s["tokens"]
        if ok:
            asked_pages += want - have
            ok = want == have or asked_pages <= top
        if not ok:
            kv[b] = 0
            slots += [-1] * n
            positions += [-1] * n
            continue
        for j in range(have, want):
            n_free -= 1
            table[b, j] = free[n_free]
        lens[b] = kv[b] = target[b]
        for pos in range(held[b], target[b]):
            slots.append(int(table[b, pos // page]) * page + pos % page)
            positions.append(pos)
    return {"table": torch.from_numpy(table).cuda(), "lens": _ints(lens),
            "free": torch.from_numpy(free).cuda(), "n_free": _ints([n_free]),
            "cu_new": _ints(cu), "kv_lens": _ints(kv), "slots": _ints(slots),
            "positions": _ints(positions)}


def _exact_write(s):
    out = {}
    for name, x in (("k", s["k"]), ("v", s["v"])):
        if s["ks"] is None:
            out[name] = x.clone()
            continue
        x = x.float().cpu().numpy()
        # the scale is a binary32 number and the code is decided by binary32 division
        m = np.max(np.abs(x), axis=-1, keepdims=True) / np.float32(127)
        code = np.rint(np.divide(x, m, out=np.zeros_like(x), where=m > 0))
        out[name] = torch.from_numpy(code.astype(np.float64) * m.astype(np.float64)).cuda()
    return out


def _exact_attend(s):
    c = s["case"]
    Hq, Hkv, page = c["Hq"], c["Hkv"], c["page"]
    G = Hq // Hkv
    if _pairs(c)[0] * Hq * D * 4 > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["n_new"]):
        L, t0 = s["kv"][b], s["cu"][b]
        where = torch.arange(L, device="cuda")
        pid, off = s["table"][b].long()[where // page], where % page
        for h in range(Hkv):
            k, v = s["kc"][pid, h, off].double(), s["vc"][pid, h, off].double()
            if s["ks"] is not None:
                k *= s["ks"][pid, h, off].double()[:, None]
                v *= s["vs"][pid, h, off].double()[:, None]
            for head in range(h * G, (h + 1) * G):
                for i in range(0, n, 1024):
                    rows = torch.arange(i, min(n, i + 1024), device="cuda")
                    at = (L - n + rows)[:, None]
                    logit = (s["q"][t0 + rows, head].double() @ k.T).mul_(s["scale"])
                    logit.masked_fill_(where[None] > at, -math.inf)
                    if c["window"] > 0:
                        logit.masked_fill_(where[None] <= at - c["window"], -math.inf)
                    out[t0 + rows, head] = torch.softmax(logit, dim=1) @ v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "plan": _exact_plan, "write": _exact_write,
            "attend": _exact_attend}[case["op"]](s)
