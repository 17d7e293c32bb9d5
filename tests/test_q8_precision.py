"""How much precision the 8-bit cache's attention keeps, in the mean rather than at worst: bounds that a kernel with
softmax weights or fp32 queries of 11 bits does not meet.  The bounds are first held against such a loss, planted in the
reference on the CPU; then the kernels are held against them.

bf16: with a relative error e before its last rounding an output lands on a neighbouring bf16 (spacing 2^-8 to 2^-7 of
the value) with probability up to 2^8 |e|, about five times that over outputs of both signs, many of them small against
the terms of their sum.  fp32 sums give e about 2^-21, so 2^-11 of the outputs; weights of 11 bits (2^-12.3 in the mean) give
2^-2.5.  FLIPS lies between them, a factor of 16 from the first.
fp32: errors of q in two parts (2^-23 in the mean) and of sums of 128 and of n terms in fp32 make about 2^-21 of the outputs'
mean magnitude; one part alone makes 2^-12.  RMS lies between them, a factor of 8 from the first."""
import math

import pytest
import torch

import q8_ref as R
from hybrid_head_sparse_decode_b200 import ops

DEV = "cuda"
E4, I8 = torch.float8_e4m3fn, torch.int8
BF, F32 = torch.bfloat16, torch.float32
FLIPS, RMS = 2.0 ** -7, 2.0 ** -18
CASES = [([900], 32, 8, 128, 64), ([9001, 1500, 20000], 8, 2, 128, 64), ([30011], 4, 4, 64, 16), ([700, 5000], 16, 2, 64, 32),
         ([3000], 8, 1, 128, 16), ([2100, 600], 4, 2, 128, 128)]


def keeps(out, ref):
    """Whether outputs (of either type) meet the bound against the fp64 values."""
    if out.dtype == BF:
        return float((out != ref.to(BF)).double().mean()) <= FLIPS
    return float((out.double() - ref).square().mean().sqrt() / ref.square().mean().sqrt()) <= RMS


def inputs(lens, Hq, Hkv, d, page, dtype, code, seed=41):
    g = torch.Generator().manual_seed(seed)
    table, P = R.make_table(g, lens, page)
    cache = R.make_cache(g, P, Hkv, page, d, code)
    if code == I8:
        for s in cache[2:]:
            s.mul_(0.25)             # scores of a few units: many rows count
    q = torch.randn(len(lens), Hq, d, generator=g).to(dtype)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32)


def to_11_bits(x):
    """fp64 values rounded to 11 significant bits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2048) / 2048, e)


def attend(q, cache, table, seq, weights=lambda p: p, queries=lambda x: x):
    """fp64 attention with functions put around the queries and the weights."""
    k, v, ks, vs = cache
    out = torch.zeros(q.shape, dtype=torch.float64)
    G = q.shape[1] // k.shape[1]
    for b, n in enumerate(seq.tolist()):
        K, V = R.rows_of(k, ks, table[b], n), R.rows_of(v, vs, table[b], n)
        for h in range(q.shape[1]):
            s = K[h // G] @ queries(q[b, h].double()) / math.sqrt(q.shape[2])
            w = torch.exp(s - s.max())
            out[b, h] = weights(w) @ V[h // G] / w.sum()
    return out


@pytest.mark.parametrize("code", [E4, I8])
@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[5]], ids=str)
def test_the_bounds_see_a_lost_half(case, code):
    q, cache, table, seq = inputs(*case, F32, code)
    ref = attend(q, cache, table, seq)
    short_w = attend(q, cache, table, seq, weights=to_11_bits)
    short_q = attend(q, cache, table, seq, queries=to_11_bits)
    assert keeps(ref.float(), ref) and not keeps(short_w.float(), ref) and not keeps(short_q.float(), ref)
    qb = q.to(BF)
    ref = attend(qb, cache, table, seq)
    assert keeps(ref.to(BF), ref)
    assert not keeps(attend(qb, cache, table, seq, weights=to_11_bits).to(BF), ref)
    assert torch.allclose(ref, R.attend(qb, cache, table, seq)[0], rtol=1e-12, atol=1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code", [(BF, E4), (BF, I8), (F32, E4), (F32, I8)])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention_keeps_its_bits(case, dtype, code):
    q, cache, table, seq = inputs(*case, dtype, code)
    ref = attend(q, cache, table, seq)
    out = ops.decode_attn_q8(q.to(DEV), ops.Q8Cache(*(t.to(DEV) for t in cache)), table.to(DEV), seq.to(DEV))
    torch.cuda.synchronize()
    assert keeps(out.cpu(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code", [(BF, E4), (F32, I8)])
@pytest.mark.parametrize("case", CASES[3:], ids=str)
def test_hybrid_layers_keep_them(case, dtype, code):
    """The hybrid layer's ways of reading rows: consecutive ones for retrieval heads, with bits for sparse heads beside them,
    listed ones for sparse heads alone.  (Sets of every position: the values of the attention over all.)"""
    q, cache, table, seq = inputs(*case, dtype, code)
    ref = attend(q, cache, table, seq)
    B, Hq, n = q.shape[0], q.shape[1], int(seq.max())
    idx = torch.full((B, Hq, n), -1, dtype=torch.int32)
    for b, m in enumerate(seq.tolist()):
        idx[b, :, :m] = torch.arange(m, dtype=torch.int32)
    dev = ops.Q8Cache(*(t.to(DEV) for t in cache))
    for roles in ([1] * Hq, [0] * Hq, [1] + [0] * (Hq - 1)):
        out, _ = ops.hybrid_decode_attn_q8(q.to(DEV), dev, table.to(DEV), seq.to(DEV), roles, idx.to(DEV), n)
        torch.cuda.synchronize()
        assert keeps(out.cpu(), ref)
