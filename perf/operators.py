"""The 8-bit paged KV cache's operators as they are used: what is called, on what, and what it cannot do without.

Three operators share one cache: ``append`` (rotate and quantise new keys and values into pages, rotate the queries),
``attend`` (one query token a sequence over every cached position) and ``hybrid`` (the hybrid-head step: retrieval heads
over every position, handing on the set of their largest logits, sparse heads over the sets they were handed).

``run`` computes them with elementary torch operations, or (``own``) by the framework's calls.  Sizes are the ones of
this repository's workloads (32 query heads on 8 KV heads of 128 or 64 dimensions, contexts up to 131072, budgets of 30 %)
and of ordinary serving: batches of ragged lengths, prompts, odd sizes.

The cache: codes [pages, Hkv, page, d] (e4m3 or int8) and a power-of-two fp32 scale [pages, Hkv] for keys and for values;
position j of sequence b is slot j % page of page block_table[b, j // page].  e4m3 codes are returned as the float8 values
they are, beside their scales; int8 codes as whole numbers, because the arithmetic that makes them is fixed operation by
operation (fp32 products and sums, each rounded once).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LARGEST = {"e4m3": 448.0, "int8": 127.0}
SCALE_EXP = (-60, 60)     # exponents a block's scale may take
SPARE = 3                 # pages of the cache that no sequence owns


# ---- the cases ---------------------------------------------------------------------------------------------------

def _append(name, B, new, ctx, Hq, Hkv, d, rot, page, dtype, codes, interleaved=False):
    """new, ctx: (least, most) new tokens and cached tokens a sequence, spread evenly over the batch."""
    return {"name": name, "op": "append", "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "page": page, "dtype": dtype, "codes": codes,
            "interleaved": interleaved}


def _attend(name, B, n, Hq, Hkv, d, page, dtype, codes):
    return {"name": name, "op": "attend", "B": B, "n_lo": n[0], "n_hi": n[1], "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "dtype": dtype, "codes": codes}


def _hybrid(name, B, n, share, retrieval, Hq, Hkv, d, page, dtype, codes):
    """share: the sets' size as a part of the length; retrieval: retrieval heads, each in another KV group."""
    return {"name": name, "op": "hybrid", "B": B, "n_lo": n[0], "n_hi": n[1], "share": share, "retrieval": retrieval,
            "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype, "codes": codes}


def listed():
    return [
        # a single conversation's next token, far into its context: latency is all there is
        _append("append 1 token", 1, (1, 1), (32767, 32767), 32, 8, 128, 128, 64, "bf16", "e4m3"),
        # a serving batch's next tokens, ragged contexts, small pages, half the dimensions rotated in adjacent pairs
        _append("append batch int8", 64, (1, 1), (0, 8190), 32, 8, 128, 64, 16, "bf16", "int8", True),
        # prompts of several requests arriving together
        _append("append prompts", 5, (61, 3500), (0, 0), 32, 8, 128, 128, 64, "bf16", "e4m3"),
        # chunks of prompts that continue inside a page, fp32, as many query heads as KV heads
        _append("append chunks fp32", 3, (37, 777), (13, 1000), 8, 8, 64, 64, 32, "fp32", "int8"),
        # the start of a conversation
        _attend("attend short", 1, (499, 499), 32, 8, 128, 64, "bf16", "e4m3"),
        # one long conversation
        _attend("attend 128K", 1, (131072, 131072), 32, 8, 128, 64, "bf16", "e4m3"),
        # a serving batch of ragged lengths, one of them a single token
        _attend("attend batch int8", 64, (1, 8191), 32, 8, 128, 16, "bf16", "int8"),
        # many short conversations
        _attend("attend many short", 256, (1, 600), 32, 8, 128, 32, "bf16", "e4m3"),
        # fp32 queries, eight heads a group, 64 dimensions
        _attend("attend fp32 d64", 4, (777, 20001), 16, 2, 64, 128, "fp32", "int8"),
        # the repository's small layer: roles R S R S, 30 % of 1024 positions
        _hybrid("hybrid small fp32", 1, (1024, 1024), 0.3, 2, 4, 2, 64, 32, "fp32", "int8"),
        # its 128K layer with four retrieval heads
        _hybrid("hybrid 128K", 1, (131072, 131072), 0.3, 4, 32, 8, 128, 64, "bf16", "e4m3"),
        # its ragged batch of four, 32K to 128K, as a middle layer has it: a single retrieval head
        _hybrid("hybrid ragged", 4, (32768, 131071), 0.3, 1, 32, 8, 128, 64, "bf16", "int8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "hybrid"])
    d, G, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 4, 8]), rng.choice([1, 2, 3, 4, 8, 8])
    page, dtype, codes = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["e4m3", "int8"])
    Hq = G * Hkv
    if op == "append":
        B = _log(rng, 1, 128)
        most = _log(rng, 1, max(1, 8000 // B)) if rng.random() < 0.6 else 1
        ctx = _log(rng, 1, 32768) - 1
        c = _append("", B, (rng.randint(1, most), most), (rng.randint(0, ctx), ctx), Hq, Hkv, d, rng.choice([d, d, d // 2]),
                    page, dtype, codes, rng.random() < 0.3)
    elif op == "attend":
        B = _log(rng, 1, 128)
        n = _log(rng, 1, min(131072, 300000 // B))
        c = _attend("", B, (rng.randint(1, n), n), Hq, Hkv, d, page, dtype, codes)
    else:
        B = _log(rng, 1, 8)
        n = _log(rng, 64, min(131072, 200000 // B))
        c = _hybrid("", B, (rng.randint(64, n), n), rng.choice([0.05, 0.1, 0.3, 0.45]), rng.randint(0, Hkv), Hq, Hkv, d,
                    page, dtype, codes)
    del c["name"]
    return c


def _spread(lo, hi, B):
    """B whole numbers from lo to hi, evenly spread (hi alone for one)."""
    return [hi] if B == 1 else [lo + (hi - lo) * i // (B - 1) for i in range(B)]


def work(c):
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        new = _spread(c["new_lo"], c["new_hi"], B)
        T = sum(new)
        blocks = sum((m + page - 1) // page for m in new)
        rows = T * (2 * Hq + 2 * Hkv) * d * es + T * 2 * Hkv * d       # q in and out, k and v in; codes out
        return {"bytes": rows + T * c["rot"] * 4 + blocks * Hkv * 2 * 4, "flops": T * (3 * c["rot"] * (Hq + Hkv) + 4 * Hkv * d)}
    lens = _spread(c["n_lo"], c["n_hi"], B)
    N = sum(lens)
    ends = 2 * B * Hq * d * es                                          # q and out
    scales = sum((n + page - 1) // page for n in lens) * Hkv * 2 * 4
    if c["op"] == "attend":
        return {"bytes": N * 2 * Hkv * d + scales + ends, "flops": 4 * Hq * d * N}
    G, R = Hq // Hkv, c["retrieval"]
    union = 1.0 - (1.0 - c["share"]) ** G                               # of a group whose heads' sets are independent
    rows = N * (R + (Hkv - R) * union)
    sets = N * c["share"]
    used = N * R + sets * (Hq - R)
    return {"bytes": int(rows * 2 * d + scales + ends + sets * 4 * (Hq - R) + sets * 4 * Hq), "flops": int(4 * d * used)}


# ---- the inputs --------------------------------------------------------------------------------------------------

def _scale_of(amax, codes):
    """The smallest power of two that brings amax within the codes' range, its exponent kept within SCALE_EXP."""
    frac, exp = torch.frexp(amax)                      # amax = frac * 2^exp, 0.5 <= frac < 1
    frac_max, exp_max = math.frexp(LARGEST[codes])
    e = exp - exp_max + (frac > frac_max).to(exp.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_EXP[0])).clamp(*SCALE_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _quantise(y, codes):
    """Values already divided by their scale -> codes, to nearest with ties to even, saturated; as bytes."""
    y = y.clamp(-LARGEST[codes], LARGEST[codes])
    return (y if codes == "e4m3" else torch.round(y)).to(CODES[codes]).view(torch.int8)


def _values(bytes_, codes, dtype=torch.float32):
    return bytes_.view(CODES[codes]).to(dtype)


def _pages(c, lens, gen, dev):
    """A block table of pages in random order, -1 behind each sequence's last page; the number of pages."""
    page, B = c["page"], c["B"]
    need = [(n + page - 1) // page for n in lens]
    P = sum(need) + SPARE
    order = torch.randperm(P, generator=gen, device=dev)[:sum(need)]
    table = torch.full((B, max(max(need), 1)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]].int()
        at += need[b]
    return table, P


def _cache(c, P, gen, dev, plant=None):
    """Keys and values ~ N(0, 1), each head with a size of its own; plant(k) may change the keys before they are quantised."""
    shape = (P, c["Hkv"], c["page"], c["d"])
    out = []
    for which in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=dev)
        if which == "k" and plant is not None:
            plant(x)
        elif which == "v":
            x *= 0.25 + 1.5 * torch.rand((1, c["Hkv"], 1, 1), generator=gen, device=dev)
        s = _scale_of(x.abs().amax((2, 3)), c["codes"])
        out += [_quantise(x / s[:, :, None, None], c["codes"]).view(CODES[c["codes"]]), s]
    return out[0], out[2], out[1], out[3]


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, d, page, dt = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], DTYPES[c["dtype"]]
    mix = torch.randperm(B, generator=gen, device=dev).tolist()
    state = {"case": c}
    if c["op"] == "append":
        new = [_spread(c["new_lo"], c["new_hi"], B)[i] for i in mix]
        ctx = [_spread(c["ctx_lo"], c["ctx_hi"], B)[i] for i in reversed(mix)]
        lens, T = [m + n for m, n in zip(new, ctx)], sum(new)
        table, P = _pages(c, lens, gen, dev)
        # the projections' output: q, k and v of a token side by side
        qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=gen, device=dev).to(dt)
        k, v, ks, vs = _cache(c, P, gen, dev)
        inv = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        angle = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * inv
        cu = torch.tensor([0] + new, device=dev).cumsum(0).int()
        state |= {"q": qkv[:, :Hq], "k_new": qkv[:, Hq:Hq + Hkv], "v_new": qkv[:, Hq + Hkv:], "cu_new": cu,
                  "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float()}
    else:
        lens = [_spread(c["n_lo"], c["n_hi"], B)[i] for i in mix]
        table, P = _pages(c, lens, gen, dev)
        state["q"] = torch.randn((B, Hq, d), generator=gen, device=dev).to(dt)
        plant = None
        if c["op"] == "hybrid":
            G, R = Hq // Hkv, c["retrieval"]
            # retrieval heads in different KV groups, then each one's set: its group's keys there point along its query
            groups = torch.randperm(Hkv, generator=gen, device=dev)[:R].tolist()
            heads = [g * G + int(torch.randint(G, (1,), generator=gen, device=dev)) for g in groups]
            budget = [max(1, int(n * c["share"])) for n in lens]
            k = max(budget)
            idx = torch.full((B, Hq, k), -1, dtype=torch.int32, device=dev)
            for b in range(B):
                at = torch.rand((Hq, lens[b]), generator=gen, device=dev).topk(budget[b], dim=1).indices
                idx[b, :, :budget[b]] = at.sort(dim=1).values.int()

            def plant(x):
                for b in range(B):
                    for h in heads:
                        at = idx[b, h, :budget[b]].long()
                        along = state["q"][b, h].float()
                        x[table[b, at // page].long(), h // G, at % page] += 16.0 * along / along.norm()

            role = torch.zeros(Hq, dtype=torch.uint8)
            role[heads] = 1
            state |= {"role": role, "idx_in": idx, "k": k,
                      "k_per_seq": torch.tensor(budget, dtype=torch.int32, device=dev)}
        k_codes, v_codes, ks, vs = _cache(c, P, gen, dev, plant)
        if c["op"] == "hybrid":
            state["idx_in"] = state["idx_in"].clone()
            state["idx_in"][:, heads] = -1                     # a retrieval head is handed nothing it reads
        k, v = k_codes, v_codes
    state |= {"cache": (k, v, ks, vs), "block_table": table, "seqlens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    return state


# ---- the operators -----------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "hybrid": _own_hybrid}[op](s)
    return {"append": _plain_append, "attend": _plain_attend, "hybrid": _plain_hybrid}[op](s)


def _own_append(s):
    from hybrid_head_sparse_decode_b200 import ops
    cache = ops.Q8Cache(*s["cache"])
    q = ops.append_rope_q8(s["k_new"], s["v_new"], cache, s["block_table"], s["seqlens"], s["cos_sin"], q=s["q"],
                           cu_new=s["cu_new"] if s["case"]["new_hi"] > 1 else None, interleaved=s["case"]["interleaved"])
    return {"q": q, "k": cache.k, "v": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}


def _own_attend(s):
    from hybrid_head_sparse_decode_b200 import ops
    return {"out": ops.decode_attn_q8(s["q"], ops.Q8Cache(*s["cache"]), s["block_table"], s["seqlens"])}


def _own_hybrid(s):
    from hybrid_head_sparse_decode_b200 import ops
    out, idx = ops.hybrid_decode_attn_q8(s["q"], ops.Q8Cache(*s["cache"]), s["block_table"], s["seqlens"], s["role"],
                                         s["idx_in"], s["k"], k_per_seq=s["k_per_seq"])
    return {"out": out, "idx": idx}


def _rotate(x, cs, interleaved):
    """x [T, heads, d] in fp32, cs [T, rot] (cosines, then sines): the first rot dimensions turned pair by pair."""
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    head, rest = x[..., :rot], x[..., rot:]
    x1, x2 = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :rot // 2], head[..., rot // 2:])
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    y = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
    return torch.cat([y, rest], -1)


def _plain_append(s):
    c, (k, v, ks, vs) = s["case"], s["cache"]
    page, codes, B = c["page"], c["codes"], c["B"]
    T, dev = s["q"].shape[0], s["q"].device
    table, lens, cu = s["block_table"].long(), s["seqlens"].long(), s["cu_new"].long()
    seq = torch.repeat_interleave(torch.arange(B, device=dev), cu[1:] - cu[:-1], output_size=T)
    pos = lens[seq] - cu[seq + 1] + torch.arange(T, device=dev)
    pid, slot = table[seq, pos // page], pos % page
    cs = s["cos_sin"][pos]
    first = lens - (cu[1:] - cu[:-1])                          # where each sequence's new rows begin
    inside = torch.nonzero(first % page > 0)[:, 0]             # the sequences that go on inside a page
    old_page, old_rows = table[inside, first[inside] // page], first[inside] % page
    old = torch.arange(page, device=dev)[None, :] < old_rows[:, None]
    for new, store, scale, turned in ((s["k_new"], k, ks, True), (s["v_new"], v, vs, False)):
        x = new.float()
        x = _rotate(x, cs, c["interleaved"]) if turned else x
        amax = torch.zeros_like(scale).index_reduce_(0, pid, x.abs().amax(-1), "amax")
        fresh = _scale_of(amax, codes)
        before, after = scale[old_page], torch.maximum(scale[old_page], fresh[old_page])
        raw = store.view(torch.int8)
        was = raw[old_page]
        grown = _quantise(_values(was, codes) * (before / after)[:, :, None, None], codes)
        raw[old_page] = torch.where(old[:, None, :, None], grown, was)
        scale[pid] = fresh[pid]
        scale[old_page] = after
        raw[pid, :, slot] = _quantise(x / scale[pid][:, :, None], codes)
    q = _rotate(s["q"].float(), cs, c["interleaved"]).to(s["q"].dtype)
    return {"q": q, "k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _rows(s):
    """Every sequence's keys and values [B, Hkv, n, d] in fp32, zero past its length, and which positions are its own."""
    c, (k, v, ks, vs) = s["case"], s["cache"]
    table = s["block_table"].long()
    n = table.shape[1] * c["page"]
    live = torch.arange(n, device=table.device)[None, :] < s["seqlens"].long()[:, None]
    pid = table.clamp(min=0)
    out = []
    for store, scale in ((k, ks), (v, vs)):
        x = _values(store.view(torch.int8)[pid], c["codes"]) * scale[pid][..., None, None]       # [B, pages, Hkv, page, d]
        x = x.transpose(1, 2).flatten(2, 3)
        out.append(torch.where(live[:, None, :, None], x, x.new_zeros(())))
    return out[0], out[1], live


def _softmax_rows(score, may, v):
    """softmax over the permitted positions, times v; zeros where nothing is permitted.  score, may [B, Hkv, G, n]."""
    score = torch.where(may, score, score.new_full((), -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return out


def _plain_attend(s):
    c = s["case"]
    k, v, live = _rows(s)
    q = s["q"].float().view(c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"])
    score = (q @ k.transpose(2, 3)) / math.sqrt(c["d"])
    out = _softmax_rows(score, live[:, None, None, :].expand_as(score), v)
    return {"out": out.view(c["B"], c["Hq"], c["d"]).to(s["q"].dtype)}


def _plain_hybrid(s):
    c = s["case"]
    B, Hq, Hkv, G = c["B"], c["Hq"], c["Hkv"], c["Hq"] // c["Hkv"]
    k, v, live = _rows(s)
    n, cap = live.shape[1], s["k"]
    q = s["q"].double().view(B, Hkv, G, c["d"])
    raw = (q @ k.double().transpose(2, 3)).view(B, Hq, n)            # in 64 bits: the sets are cut between neighbours
    idx = s["idx_in"].long()
    member = torch.zeros((B, Hq, n + 1), dtype=torch.bool, device=idx.device)
    member.scatter_(2, torch.where(idx >= 0, idx, n), True)
    retrieval = (s["role"].to(idx.device) == 1)[None, :, None]
    may = torch.where(retrieval, live[:, None, :], member[:, :, :n])
    out = _softmax_rows((raw / math.sqrt(c["d"])).float().view(B, Hkv, G, n), may.view(B, Hkv, G, n), v)
    # the largest k_b logits of each head, lower positions first among equals, then by position
    ranked = torch.where(live[:, None, :], raw, raw.new_full((), -math.inf)).sort(dim=-1, descending=True, stable=True).indices
    taken = torch.arange(cap, device=idx.device)[None, None, :] < s["k_per_seq"].long()[:, None, None]
    best = torch.where(taken, ranked[:, :, :cap], n).sort(dim=-1).values
    best = torch.where(best < n, best, -1)
    return {"out": out.view(B, Hq, c["d"]).to(s["q"].dtype), "idx": torch.where(retrieval, best, idx).int()}


# ---- the same from the definitions, in 64 bits --------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "attend": _exact_heads, "hybrid": _exact_heads}[c["op"]](c, s)


def _exact_append(c, s):
    k, v, ks, vs = s["cache"]
    page, rot, top = c["page"], c["rot"], LARGEST[c["codes"]]
    cu, lens, table = s["cu_new"].tolist(), s["seqlens"].tolist(), s["block_table"].tolist()
    cs = s["cos_sin"].double()

    def turn(x, pos):                                           # as a product of complex numbers
        z = torch.complex(cs[pos, :rot // 2], cs[pos, rot // 2:])[:, None]
        x, y = x.double(), x.double().clone()
        if c["interleaved"]:
            w = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * z
            y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
        else:
            w = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
            y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
        return y

    def grid(x):                                                # to the codes' values, nearest, ties to even
        x = x.clamp(-top, top)
        if c["codes"] == "int8":
            return torch.round(x)
        e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(e - 3)
        return torch.round(x / step) * step

    kk, vv = _values(k.view(torch.int8), c["codes"], torch.float64), _values(v.view(torch.int8), c["codes"], torch.float64)
    ksc, vsc = ks.double(), vs.double()
    q = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(c["B"]):
        t0, t1 = cu[b], cu[b + 1]
        start = lens[b] - (t1 - t0)
        pos = torch.arange(start, lens[b], device=q.device)
        q[t0:t1] = turn(s["q"][t0:t1], pos)
        for x, store, scale in ((turn(s["k_new"][t0:t1], pos), kk, ksc), (s["v_new"][t0:t1].double(), vv, vsc)):
            for j in range(start // page, (lens[b] - 1) // page + 1):
                lo, hi = max(start, j * page), min(lens[b], (j + 1) * page)
                rows, p = x[lo - start:hi - start], table[b][j]
                e = torch.ceil(torch.log2(rows.abs().amax((0, 2)) / top)).clamp(*SCALE_EXP)
                now = torch.exp2(e)
                if lo > j * page:
                    was = scale[p].clone()
                    now = torch.maximum(now, was)
                    store[p, :, :lo - j * page] = grid(store[p, :, :lo - j * page] * (was / now)[:, None, None])
                scale[p] = now
                store[p, :, lo - j * page:hi - j * page] = grid(rows.transpose(0, 1) / now[:, None, None])
    whole = c["codes"] == "int8"
    return {"q": q, "k": None if whole else kk, "v": None if whole else vv, "k_scale": ksc, "v_scale": vsc}


def _exact_heads(c, s):
    k, v, ks, vs = s["cache"]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G, lens = Hq // Hkv, s["seqlens"].tolist()
    out = torch.zeros((B, Hq, d), dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        n = lens[b]
        own_pages = s["block_table"][b, :(n + page - 1) // page].long()
        K, V = ((_values(x.view(torch.int8)[own_pages], c["codes"], torch.float64) * y[own_pages].double()[:, :, None, None])
                .permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n] for x, y in ((k, ks), (v, vs)))
        for h in range(Hq):
            score = (K[h // G] @ s["q"][b, h].double()) / math.sqrt(d)
            if c["op"] == "hybrid" and int(s["role"][h]) == 0:
                mine = s["idx_in"][b, h]
                mine = mine[mine >= 0].long()
                out[b, h] = torch.softmax(score[mine], 0) @ V[h // G][mine]
            else:
                out[b, h] = torch.softmax(score, 0) @ V[h // G]
    return {"out": out} if c["op"] == "attend" else {"out": out, "idx": None}
