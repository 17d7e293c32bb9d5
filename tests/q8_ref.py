"""The 8-bit paged cache's operators written out on the CPU: the append operation by operation in
fp32 (its codes are fixed that way), attention in fp64, and the error bounds of the kernels."""
import math

import torch

LARGEST = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def values(codes, dtype=torch.float64):
    return codes.to(torch.float32).to(dtype)


def quantise(y, code):
    y = torch.nan_to_num(y, nan=0.0, posinf=math.inf, neginf=-math.inf).clamp(-LARGEST[code], LARGEST[code])
    return (y if code == torch.float8_e4m3fn else torch.round(y)).to(code)


def block_scale(rows, code):
    """2^ceil(log2(amax / largest)) within 2^-60 .. 2^60, by search (no logarithm)."""
    mag = rows.abs()
    amax = float(torch.where(torch.isfinite(mag), mag, torch.zeros_like(mag)).max())
    e = -60
    while e < 60 and amax > LARGEST[code] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, cs, interleaved):
    """x [heads, d] fp32, cs [rot]: each product and sum rounded to fp32."""
    rot = cs.numel()
    c, s = cs[:rot // 2], cs[rot // 2:]
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    x1, x2 = x[:, a], x[:, b]
    y[:, a] = x1 * c - x2 * s
    y[:, b] = x2 * c + x1 * s
    return y


def append(k_new, v_new, q, k, v, ks, vs, table, seqlens, cu, cos_sin, interleaved, q_out):
    """In place on the CPU tensors k, v, ks, vs and q_out."""
    page, code = k.shape[2], k.dtype
    for b in range(table.shape[0]):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        first = int(seqlens[b]) - (t1 - t0)
        if t1 == t0:
            continue
        rk, rv = k_new[t0:t1].float(), v_new[t0:t1].float()
        if cos_sin is not None:
            rk = torch.stack([rotate(rk[i], cos_sin[first + i], interleaved) for i in range(t1 - t0)])
        if q is not None:
            for i in range(t1 - t0):
                x = q[t0 + i].float()
                q_out[t0 + i] = (x if cos_sin is None else rotate(x, cos_sin[first + i], interleaved)).to(q.dtype)
        for j in range(first // page, (first + t1 - t0 - 1) // page + 1):
            lo, hi = max(first, j * page), min(first + t1 - t0, (j + 1) * page)
            p = int(table[b, j])
            for store, scale, rows in ((k, ks, rk), (v, vs, rv)):
                for h in range(k.shape[1]):
                    new = rows[lo - first:hi - first, h]
                    now = block_scale(new, code)
                    if lo > j * page:
                        was = float(scale[p, h])
                        now = max(now, was)
                        old = store[p, h, :lo - j * page].float()
                        store[p, h, :lo - j * page] = quantise(old * (was / now), code)
                    scale[p, h] = now
                    store[p, h, lo - j * page:hi - j * page] = quantise(new / now, code)


def rows_of(store, scale, table_row, n):
    """One sequence's rows [Hkv, n, d] in fp64."""
    page = store.shape[2]
    ids = table_row[:(n + page - 1) // page].long()
    x = values(store[ids]) * scale[ids].double()[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(store.shape[1], -1, store.shape[3])[:, :n]


def scale_rows(scale, table_row, n, page):
    """One sequence's scales, row by row [Hkv, n], in fp64."""
    ids = table_row[:(n + page - 1) // page].long()
    return scale[ids].double().T.repeat_interleave(page, 1)[:, :n]


def attend(q, cache, table, seqlens, sets=None):
    """fp64 attention.  q [B, Hq, d]; sets: None, or sets[b][h] = None (every position) or a list.
    Returns out, the bound of the kernels' error, raw logits[b] [Hq, n], their error's bound[b] [Hq]."""
    k, v, ks, vs = cache
    B, Hq, d = q.shape
    G, page = Hq // k.shape[1], k.shape[2]
    out = torch.zeros(B, Hq, d, dtype=torch.float64)
    tol = torch.zeros(B, Hq, d, dtype=torch.float64)
    raws, raw_tols = [], []
    for b in range(B):
        n = int(seqlens[b])
        K, V = rows_of(k, ks, table[b], n), rows_of(v, vs, table[b], n)
        qb = q[b].double()
        raw = torch.stack([K[h // G] @ qb[h] for h in range(Hq)]) if n else torch.zeros(Hq, 0)
        mag = torch.stack([K[h // G].abs() @ qb[h].abs() for h in range(Hq)]) if n else torch.zeros(Hq, 0)
        # raw dot products: q in two 11-bit parts when fp32 (2^-22 |q|), at most d + 8 fp32 sums and
        # scalings that may truncate (2^-23 each)
        rt = (2.0 ** -22 + (d + 8) * 2.0 ** -23) * (mag.amax(1) if n else torch.zeros(Hq).double())
        raws.append(raw)
        raw_tols.append(rt)
        for h in range(Hq):
            at = torch.arange(n) if sets is None or sets[b][h] is None else torch.as_tensor(sets[b][h], dtype=torch.long)
            if at.numel() == 0:
                continue
            p = torch.softmax(raw[h, at] / math.sqrt(d), 0)
            Vh = V[h // G][at]
            out[b, h] = p @ Vh
            spread = p @ Vh.abs() + out[b, h].abs()
            # a weight's relative error: its score's (times two: the maximum's and its own), the
            # exponential (2^-21), its rounding to 11 bits (bf16; 22 bits in two parts for fp32);
            # sums of one rounding per 16 rows and per merged state (2^-23 each)
            w = 2 * float(rt[h]) / math.sqrt(d) + 2.0 ** -21 + (2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22)
            tol[b, h] = (w + (at.numel() / 16 + 64) * 2.0 ** -23) * spread + UNIT[q.dtype] * out[b, h].abs()
            # a weight p sv multiplies codes as a half (or two) whose smallest step is 2^-24, the
            # largest weight being 2^6 or more: each is off by at most 2^-25 2^-6 of the largest
            sv = scale_rows(vs, table[b], n, page)[h // G][at]
            tol[b, h] += 2.0 ** -31 * float((p * sv).max()) * (Vh.abs() / sv[:, None]).sum(0)
    return out, tol, raws, raw_tols


def check_topk(picked, raw, budget, tol):
    """`picked` is a top-`budget` set of logits known within tol."""
    assert picked.numel() == budget and bool((picked[1:] > picked[:-1]).all())
    best = raw.sort(descending=True).values
    kth = float(best[budget - 1])
    assert float(raw[picked].min()) >= kth - 2 * tol
    rest = torch.ones_like(raw, dtype=torch.bool)
    rest[picked] = False
    if bool(rest.any()):
        assert float(raw[rest].max()) <= float(raw[picked].min()) + 2 * tol


def make_cache(gen, P, Hkv, page, d, code, scale_spread=0, stale=True):
    """Random codes over the whole range; scales 2^(-6 +- scale_spread)."""
    if code == torch.int8:
        k, v = (torch.randint(-127, 128, (P, Hkv, page, d), generator=gen, dtype=torch.int64).to(code) for _ in range(2))
        base = -5
    else:
        k, v = ((torch.randn(P, Hkv, page, d, generator=gen) * 64).clamp(-448, 448).to(code) for _ in range(2))
        base = -6
    def sc():
        e = torch.randint(base - scale_spread, base + scale_spread + 1, (P, Hkv), generator=gen)
        return torch.ldexp(torch.ones(P, Hkv), e)
    return [k, v, sc(), sc()]


def make_table(gen, seqlens, page, spare=2):
    need = [(int(n) + page - 1) // page for n in seqlens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=gen)
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m].int()
        at += m
    return table, P
