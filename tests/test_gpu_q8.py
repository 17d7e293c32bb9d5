"""The 8-bit paged cache's operators on the GPU against their definitions (q8_ref.py): the append
bit for bit, attention and the hybrid layer in fp64 within derived bounds."""
import pytest
import torch

import q8_ref as R
from hybrid_head_sparse_decode_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4, I8 = torch.float8_e4m3fn, torch.int8
BF, F32 = torch.bfloat16, torch.float32


def to_dev(cache):
    return ops.Q8Cache(*(t.to(DEV) for t in cache))


def same(a, b):
    """Equal bit for bit (NaN codes included)."""
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def cos_sin(n_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def no_flags(err):
    assert int(err.item()) == 0


# ---- the append ------------------------------------------------------------------------------

def run_append(new, ctx, Hq, Hkv, d, page, dtype, code, rot, interleaved, extra=0, ragged=True, grow=False,
               seed=1, big=None):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(new, ctx)]
    table, P = R.make_table(g, lens, page)
    cache = R.make_cache(g, P, Hkv, page, d, code)
    T = sum(new) + extra
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g)
    if grow:
        qkv *= 64.0        # above what the cache's scales reach: old rows are requantised
    if big is not None:
        for i, x in enumerate(big):
            qkv[i % T, Hq + (i % (2 * Hkv)), (5 * i) % d] = x
    qkv = qkv.to(dtype)
    q, kn, vn = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = torch.tensor([0] + new).cumsum(0).int()
    seq = torch.tensor(lens, dtype=torch.int32)
    cs = cos_sin(max(max(lens), 1), rot) if rot else None
    gpu, qkvd = to_dev(cache), qkv.to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full((T, Hq, d), 7.0, dtype=dtype)
    q_gpu = q_out.to(DEV)
    R.append(kn, vn, q, *cache, table, seq, cu, cs, interleaved, q_out)
    got = ops.append_rope_q8(qkvd[:, Hq:Hq + Hkv], qkvd[:, Hq + Hkv:], gpu, table.to(DEV), seq.to(DEV),
                             None if cs is None else cs.to(DEV), q=qkvd[:, :Hq],
                             cu_new=cu.to(DEV) if ragged else None, interleaved=interleaved, q_out=q_gpu,
                             device_error=err)
    torch.cuda.synchronize()
    assert got is q_gpu
    for name, a, b in zip(("k", "v", "k_scale", "v_scale"), gpu, cache):
        assert same(a, b), name
    assert same(q_gpu, q_out)
    return int(err.item())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,code,d,rot,page", [(BF, E4, 128, 128, 64), (BF, I8, 128, 64, 16), (F32, I8, 64, 64, 32),
                                                   (F32, E4, 64, 8, 128), (F32, E4, 128, 40, 128), (BF, E4, 64, 0, 16)])
def test_append_ragged(dtype, code, d, rot, page, interleaved):
    assert run_append([37, 0, 1, 130, 16, 5], [13, 40, 0, 77, 48, page - 2], 8, 2, d, page, dtype, code, rot, interleaved,
                      extra=3) == 0


@pytest.mark.parametrize("dtype,code", [(BF, E4), (BF, I8), (F32, E4), (F32, I8)])
def test_append_requantises_old_rows(dtype, code):
    assert run_append([3, 20, 1, 64], [5, 30, 31, 1], 6, 3, 128, 32, dtype, code, 128, False, grow=True) == 0


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_append_single_tokens(d, page):
    """One token a sequence: the first of all, the last of a page, the first of the next."""
    ctx = [0, page - 1, page, 3 * page + 5, 1]
    assert run_append([1] * 5, ctx, 16, 2, d, page, BF, E4, d, False, ragged=False) == 0
    assert run_append([1] * 5, ctx, 16, 2, d, page, BF, I8, d, True, ragged=False, grow=True) == 0


def test_append_extremes():
    """Zeros, the codes' borders, subnormal and huge magnitudes."""
    vals = [0.0, 448.0, 449.0, 127.0, 128.0, 1e-38, 3e38, -3e38, 2.0 ** -60, 464.0, 2.0 ** -126, 1.9 * 2.0 ** 60]
    for code in (E4, I8):
        assert run_append([9, 6], [0, 3], 2, 2, 64, 16, F32, code, 0, False, big=vals) == 0
        assert run_append([9, 6], [0, 3], 2, 2, 64, 16, F32, code, 0, False, big=[0.0], grow=False) == 0
    # an infinity is stored as the largest code and a NaN as 0; both are flagged
    assert run_append([9, 6], [0, 3], 2, 2, 64, 16, F32, E4, 0, False, big=[float("inf"), float("nan"), -float("inf")]) == 16
    assert run_append([9, 6], [0, 3], 2, 2, 64, 16, F32, I8, 0, False, big=[float("inf"), float("nan"), -float("inf")]) == 16


def test_append_many_sequences():
    """More sequences than a CTA has threads: blocks are found across rounds of the prefix sum."""
    new = [(i * 7) % 5 for i in range(700)]
    ctx = [(i * 13) % 40 for i in range(700)]
    assert run_append(new, ctx, 1, 1, 64, 16, BF, I8, 64, False) == 0


def test_append_skips_and_flags_what_does_not_fit():
    g = torch.Generator().manual_seed(3)
    page, Hkv, d = 16, 2, 64
    cache = R.make_cache(g, 8, Hkv, page, d, I8)
    table = torch.tensor([[0, 1], [2, 9], [4, -1], [5, 6], [7, 3]], dtype=torch.int32)
    #            fits, page 9 of 8, page -1, more rows than max_pages, beyond cos_sin
    seq = torch.tensor([20, 20, 20, 33, 32], dtype=torch.int32)
    cs = cos_sin(31, d)
    kn = torch.randn(5, Hkv, d, generator=g).to(BF)
    gpu = to_dev(cache)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.append_rope_q8(kn.to(DEV), kn.to(DEV), gpu, table.to(DEV), seq.to(DEV), cs.to(DEV), device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 3
    cu = torch.tensor([0, 1, 1, 1, 1, 1])
    R.append(kn, kn, None, *cache, table, seq, cu, cs, False, None)
    for a, b in zip(gpu, cache):
        assert same(a, b)
    # the numbers of cu_new: descending, and more new rows than the length
    err.zero_()
    for bad in ([0, 3, 1, 5, 5, 5], [0, 1, 1, 1, 1, 6]):
        ops.append_rope_q8(kn.to(DEV), kn.to(DEV), to_dev(cache), table[:, :1].contiguous().to(DEV),
                           torch.tensor([1, 0, 0, 0, 3], dtype=torch.int32, device=DEV),
                           cu_new=torch.tensor(bad, dtype=torch.int32, device=DEV), device_error=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 2
        err.zero_()


# ---- attention over every position --------------------------------------------------------------

def run_attend(lens, Hq, Hkv, d, page, dtype, code, seed=5, spread=0, q_size=1.0, change=None):
    g = torch.Generator().manual_seed(seed)
    table, P = R.make_table(g, lens, page)
    cache = R.make_cache(g, P, Hkv, page, d, code, scale_spread=spread)
    # what no sequence reads: NaN codes and scales in rows past the ends and in spare pages
    used = torch.zeros(P, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range((n + page - 1) // page):
            used[int(table[b, j]), :max(0, min(page, n - j * page))] = True
    if code == E4:
        for t in cache[:2]:
            raw = t.view(torch.uint8)
            raw[(~used)[:, None, :].expand(P, Hkv, page)] = 0x7f
    for t in cache[2:]:
        t[~used.any(1)] = float("nan")
    q = (torch.randn(len(lens), Hq, d, generator=g) * q_size).to(dtype)
    if change is not None:
        change(q, cache, table)
    seq = torch.tensor(lens, dtype=torch.int32)
    ref, tol, _, _ = R.attend(q, cache, table, seq)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ops.decode_attn_q8(q.to(DEV), to_dev(cache), table.to(DEV), seq.to(DEV), device_error=err)
    torch.cuda.synchronize()
    no_flags(err)
    off = (out.cpu().double() - ref).abs()
    assert bool((off <= tol + 1e-30).all()), float((off / (tol + 1e-30)).max())
    return out


@pytest.mark.parametrize("dtype,code", [(BF, E4), (BF, I8), (F32, E4), (F32, I8)])
@pytest.mark.parametrize("Hq,Hkv,d,page", [(32, 8, 128, 64), (3, 3, 64, 16), (4, 2, 128, 32), (16, 2, 64, 128), (8, 1, 128, 16),
                                           (5, 5, 128, 128), (6, 3, 64, 64)])
def test_attend_lengths(Hq, Hkv, d, page, dtype, code):
    run_attend([0, 1, 15, 16, 17, 63, 64, 65, 127, 499, 1023], Hq, Hkv, d, page, dtype, code)


@pytest.mark.parametrize("dtype,code", [(BF, E4), (F32, I8)])
def test_attend_long(dtype, code):
    run_attend([9001, 1, 20000], 8, 2, 128, 64, dtype, code)
    run_attend([30011], 4, 4, 64, 16, dtype, code)


@pytest.mark.parametrize("lens", [[1], [16], [300], [0], [0, 0, 0]])
def test_attend_alone(lens):
    run_attend(lens, 32, 8, 128, 64, BF, E4)
    run_attend(lens, 8, 1, 64, 16, F32, I8)


def test_attend_many_sequences():
    run_attend([(i * 37) % 71 for i in range(700)], 2, 1, 64, 16, BF, I8)
    run_attend([1] * 300, 8, 8, 128, 16, BF, E4)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_scales_far_apart(dtype):
    """Blocks whose scales differ by 2^+-20: small values beside large ones, and one-sided softmaxes."""
    run_attend([700, 65], 8, 2, 128, 32, dtype, E4, spread=20, q_size=1e-6)
    run_attend([700, 65], 8, 2, 64, 32, dtype, I8, spread=8)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_large_and_small_queries(dtype):
    for size in (1e-20, 1e18):
        def tame(q, cache, table):
            cache[2].fill_(2.0 ** (-60 if size > 1 else 60))
        run_attend([100, 37], 4, 2, 64, 16, dtype, E4, q_size=size, change=tame)
    def zero(q, cache, table):
        q.zero_()
        q[0, 1, 3] = 2.0 ** -100
    run_attend([100, 37], 4, 2, 64, 16, dtype, I8, change=zero)


def test_attend_first_or_last_row_takes_all():
    """A single dominating row, at the beginning, at the end and in the middle."""
    for at in (0, 499, 250):
        def lift(q, cache, table):
            for h in range(2):
                p = int(table[0, at // 16])
                cache[0][p, h] = 0
                cache[0][p, h, at % 16] = torch.sign(q[0, 4 * h].float()).mul(127).to(I8)
                cache[2][p, h] = 1.0
        run_attend([499 if at < 499 else 500], 8, 2, 64, 16, BF, I8, change=lift)


def test_attend_shared_pages_and_bad_entries():
    """Two sequences on one prefix; a bad page number is flagged and its rows are skipped, a length
    past the table is cut."""
    g = torch.Generator().manual_seed(8)
    cache = R.make_cache(g, 6, 2, 16, 64, E4)
    q = torch.randn(3, 8, 64, generator=g).to(BF)
    table = torch.tensor([[0, 1, 2], [0, 1, 3], [4, 5, 0]], dtype=torch.int32)
    seq = torch.tensor([40, 47, 48], dtype=torch.int32)
    ref, tol, _, _ = R.attend(q, cache, table, seq)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ops.decode_attn_q8(q.to(DEV), to_dev(cache), table.to(DEV), seq.to(DEV), device_error=err)
    torch.cuda.synchronize()
    no_flags(err)
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
    bad = table.clone()
    bad[0, 1], bad[1, 2] = 6, -1
    long = torch.tensor([40, 47, 49], dtype=torch.int32)
    out = ops.decode_attn_q8(q.to(DEV), to_dev(cache), bad.to(DEV), long.to(DEV), device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 3
    keep = [[list(range(16)) + list(range(32, 40))] * 8, [list(range(32))] * 8, [None] * 8]
    fix = bad.clone()
    fix[0, 1], fix[1, 2] = 0, 0
    ref, tol, _, _ = R.attend(q, cache, fix, seq, keep)
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
    err.zero_()
    out = ops.decode_attn_q8(q.to(DEV), to_dev(cache), table.to(DEV), torch.tensor([-3, 47, 48], dtype=torch.int32, device=DEV),
                             device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 2 and not bool(out[0].any())


# ---- the hybrid layer ---------------------------------------------------------------------------

def run_hybrid(lens, Hq, Hkv, d, page, dtype, code, roles, density, seed=11, block=0, budgets=None, k=None, spread=0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    table, P = R.make_table(g, lens, page)
    cache = R.make_cache(g, P, Hkv, page, d, code, scale_spread=spread)
    q = torch.randn(B, Hq, d, generator=g).to(dtype)
    seq = torch.tensor(lens, dtype=torch.int32)
    n_max = table.shape[1] * page
    sets = [[None if roles[h] else torch.nonzero(torch.rand(lens[b], generator=g) < density[(b + h) % len(density)])[:, 0].tolist()
             for h in range(Hq)] for b in range(B)]
    k = k or min(n_max, max([len(s) for row in sets for s in row if s is not None] + [budgets and max(budgets) or 1, block, 1]))
    idx = torch.full((B, Hq, k), -1, dtype=torch.int32)
    for b in range(B):
        for h in range(Hq):
            if sets[b][h] is not None:
                sets[b][h] = sets[b][h][:k]
                idx[b, h, :len(sets[b][h])] = torch.tensor(sets[b][h], dtype=torch.int32)
    kps = None if budgets is None else torch.tensor(budgets, dtype=torch.int32, device=DEV)
    ref, tol, raws, raw_tols = R.attend(q, cache, table, seq, sets)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, nxt = ops.hybrid_decode_attn_q8(q.to(DEV), to_dev(cache), table.to(DEV), seq.to(DEV), roles, idx.to(DEV), k,
                                         k_per_seq=kps, device_error=err, block=block)
    torch.cuda.synchronize()
    no_flags(err)
    off = (out.cpu().double() - ref).abs()
    assert bool((off <= tol + 1e-30).all()), float((off / (tol + 1e-30)).max())
    nxt = nxt.cpu()
    for b in range(B):
        for h in range(Hq):
            row = nxt[b, h]
            if not roles[h]:
                assert torch.equal(row, idx[b, h])
                continue
            m = int((row >= 0).sum())
            assert bool((row[m:] == -1).all())
            kb = min(k if budgets is None else budgets[b], k, lens[b])
            got, raw, rt = row[:m].long(), raws[b][h], float(raw_tols[b][h])
            if lens[b] == 0:
                assert m == 0
            elif block > 1:
                nblk = (lens[b] + block - 1) // block
                score = torch.stack([raw[i * block:(i + 1) * block].max() for i in range(nblk)])
                picked = torch.unique(got // block)
                whole = torch.cat([torch.arange(int(i) * block, min(lens[b], (int(i) + 1) * block)) for i in picked])
                assert torch.equal(got, whole[:k])
                R.check_topk(picked, score, min(max(1, kb // block), nblk), rt)
            else:
                R.check_topk(got, raw, kb, rt)
    return out, nxt


MIX = {1: [1, 0, 0, 1, 0], 2: [1, 0, 0, 0, 1, 1], 4: [0, 1, 0, 0, 0, 0, 0, 0, 1, 1, 1, 1], 8: [0] * 8 + [0, 0, 0, 1, 0, 0, 1, 0]}


@pytest.mark.parametrize("dtype,code", [(BF, E4), (BF, I8), (F32, E4), (F32, I8)])
@pytest.mark.parametrize("G,d,page", [(1, 64, 16), (2, 128, 32), (4, 128, 64), (8, 64, 128), (4, 64, 16), (8, 128, 16)])
def test_hybrid_lengths(G, d, page, dtype, code):
    roles = MIX[G]
    run_hybrid([0, 1, 16, 33, 64, 300, 1100], len(roles), len(roles) // G, d, page, dtype, code, roles,
               [0.3, 0.02, 0.0, 1.0, 0.6], budgets=[1, 1, 5, 10, 19, 90, 330])


@pytest.mark.parametrize("roles", [[1] * 8, [0] * 8])
def test_hybrid_one_kind_of_head(roles):
    run_hybrid([513, 40], 8, 2, 128, 64, BF, E4, roles, [0.25], budgets=[150, 12])


def test_hybrid_long_and_sparse():
    run_hybrid([20011, 7000], 8, 2, 128, 64, BF, E4, [1, 0, 0, 0, 0, 0, 0, 0], [0.05, 0.3], budgets=[6000, 2100])
    run_hybrid([33000], 4, 1, 64, 16, F32, I8, [0, 0, 0, 0], [0.001, 0.0])
    run_hybrid([40000], 4, 4, 64, 128, BF, I8, [0, 1, 0, 1], [0.4, 0.002], budgets=[12000])


def test_hybrid_many_tiles():
    """More tiles than the attention's CTAs have threads: ranges are found in rounds."""
    lens = [16384] + [50 + i for i in range(24)]
    run_hybrid(lens, 4, 4, 64, 64, BF, I8, [0, 1, 0, 0], [0.1, 0.0, 0.5], budgets=[100] + [20] * 24, k=2000)
    run_hybrid([0] * 5 + lens[::-1], 8, 4, 64, 64, BF, E4, [0, 0, 0, 0, 0, 1, 0, 0], [0.002, 0.3], budgets=[1] * 5 + [20] * 24 + [100],
               k=5000)


def test_hybrid_in_place():
    """idx_out may be idx_in: sets of sparse heads stay, retrieval heads' are replaced."""
    g = torch.Generator().manual_seed(5)
    table, P = R.make_table(g, [3000], 32)
    cache = to_dev(R.make_cache(g, P, 2, 32, 64, I8))
    q = torch.randn(1, 8, 64, generator=g).to(BF).to(DEV)
    seq = torch.tensor([3000], dtype=torch.int32, device=DEV)
    idx = torch.rand(1, 8, 3000, generator=g).topk(700, dim=2).indices.sort(dim=2).values.int().to(DEV)
    roles = [1, 0, 0, 0, 0, 0, 0, 0]
    out, nxt = ops.hybrid_decode_attn_q8(q, cache, table.to(DEV), seq, roles, idx, 700)
    same_buffer = idx.clone()
    out2, nxt2 = ops.hybrid_decode_attn_q8(q, cache, table.to(DEV), seq, roles, same_buffer, 700, idx_out=same_buffer)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(nxt, nxt2) and nxt2 is same_buffer


def test_hybrid_blocks():
    run_hybrid([700, 64, 1, 0, 95], 8, 2, 64, 32, BF, E4, [1, 0, 0, 0, 1, 1, 0, 0], [0.3], block=64,
               budgets=[256, 64, 64, 64, 64], k=256)


def test_hybrid_without_budgets_and_full_rows():
    """k equal to the table's capacity: rows hold every position."""
    run_hybrid([128, 100], 4, 2, 64, 16, F32, E4, [1, 0, 0, 1], [1.0], k=128)


def test_hybrid_scales_far_apart():
    run_hybrid([700, 90], 8, 2, 64, 32, F32, I8, [1, 0, 0, 0, 0, 0, 0, 0], [0.3], spread=6, budgets=[200, 30])


def test_hybrid_flags_bad_indices():
    g = torch.Generator().manual_seed(4)
    cache = R.make_cache(g, 4, 1, 16, 64, I8)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    q = torch.randn(2, 2, 64, generator=g).to(BF)
    seq = torch.tensor([20, 32], dtype=torch.int32)
    for row in ([3, 3], [5, 4], [0, 20], [1 << 30, -1], [-7, 1], [-1, 2]):
        idx = torch.full((2, 2, 2), -1, dtype=torch.int32)
        idx[0, 1] = torch.tensor(row, dtype=torch.int32)
        idx[1, 1, 0] = 9
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, nxt = ops.hybrid_decode_attn_q8(q.to(DEV), to_dev(cache), table.to(DEV), seq.to(DEV), [1, 0], idx.to(DEV), 2,
                                             device_error=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 1, row
        assert torch.equal(nxt[:, 1].cpu(), idx[:, 1])
        # the other heads and sequences are untouched by it
        ref, tol, _, _ = R.attend(q, cache, table, seq, [[None, []], [None, [9]]])
        off = (out.cpu().double() - ref).abs()
        assert bool((off <= tol + 1e-30)[[0, 1, 1], [0, 0, 1]].all())


# ---- streams, graphs, together ---------------------------------------------------------------------

def test_streams_and_repeatability():
    """The same bits on another stream, with dirty workspaces, and again."""
    g = torch.Generator().manual_seed(9)
    lens = [3001, 17, 900, 0]
    table, P = R.make_table(g, lens, 32)
    cache = to_dev(R.make_cache(g, P, 2, 32, 128, E4))
    q = torch.randn(4, 8, 128, generator=g).to(BF).to(DEV)
    table, seq = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    idx = torch.full((4, 8, 500), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(lens):
        m = min(n, 500)
        idx[b, :, :m] = torch.arange(m, dtype=torch.int32, device=DEV)
    roles = [1, 0, 0, 0, 0, 0, 0, 0]
    first = ops.decode_attn_q8(q, cache, table, seq)
    hyb = ops.hybrid_decode_attn_q8(q, cache, table, seq, roles, idx, 500)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n0 = ops.q8_workspace_size(4, 8, 2, 128, 32, P, table.shape[1], BF, E4)
    n1 = ops.q8_workspace_size(4, 8, 2, 128, 32, P, table.shape[1], BF, E4, 500)
    for fill in (0, 255, 77):
        w0 = torch.full((n0,), fill, dtype=torch.uint8, device=DEV)
        w1 = torch.full((n1,), fill, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        again = ops.decode_attn_q8(q, cache, table, seq, workspace=w0, stream=side)
        hyb2 = ops.hybrid_decode_attn_q8(q, cache, table, seq, roles, idx, 500, workspace=w1, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(first, again)
        assert torch.equal(hyb[0], hyb2[0]) and torch.equal(hyb[1], hyb2[1])


def test_rotated_queries_in_place():
    """q_out may be q itself."""
    g = torch.Generator().manual_seed(31)
    seq = torch.tensor([9, 40], dtype=torch.int32)
    cache = to_dev(R.make_cache(g, 8, 2, 16, 128, E4))
    table = torch.arange(8, dtype=torch.int32).view(2, 4)
    q, kn = torch.randn(2, 8, 128, generator=g).to(BF).to(DEV), torch.randn(2, 2, 128, generator=g).to(BF).to(DEV)
    cs = cos_sin(64, 96).to(DEV)
    apart = ops.append_rope_q8(kn, kn, cache, table.to(DEV), seq.to(DEV), cs, q=q)
    same_place = q.clone()
    assert ops.append_rope_q8(kn, kn, cache, table.to(DEV), seq.to(DEV), cs, q=same_place, q_out=same_place) is same_place
    torch.cuda.synchronize()
    assert same(apart, same_place)


def test_calls_back_to_back_in_one_workspace():
    """Calls of different shapes queued one behind another in one workspace, the launches overlapping
    as they may, give what each gives alone."""
    jobs = []
    for seed, lens, roles, share in ((1, [9000], [1] + [0] * 7, 0.3), (2, [4000, 800, 3], [0] * 8, 0.1),
                                     (3, [2500, 2500], [1] * 8, 0.2), (4, [70 + i for i in range(40)], [1, 0, 0, 0, 0, 0, 0, 1], 0.3),
                                     (5, [600], [0, 0, 1, 0, 0, 0, 0, 0], 0.3)):
        g = torch.Generator().manual_seed(seed)
        table, P = R.make_table(g, lens, 64)
        cache = to_dev(R.make_cache(g, P, 2, 64, 128, E4))
        k = max(1, int(max(lens) * share))
        idx = torch.full((len(lens), 8, k), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            m = max(1, int(n * share))
            idx[b, :, :m] = torch.rand(8, n, generator=g).topk(m, dim=1).indices.sort(dim=1).values.int()
        rows = torch.randn(len(lens), 2, 128, generator=g).to(BF).to(DEV)
        jobs.append((torch.randn(len(lens), 8, 128, generator=g).to(BF).to(DEV), cache, table.to(DEV),
                     torch.tensor(lens, dtype=torch.int32, device=DEV), roles, idx.to(DEV), k, rows, P))
    n = max(ops.q8_workspace_size(q.shape[0], 8, 2, 128, 64, P, t.shape[1], BF, E4, k) for q, _, t, _, _, _, k, _, P in jobs)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def run(job):
        q, cache, table, seq, roles, idx, k, rows, _ = job
        ops.append_rope_q8(rows, rows, cache, table, seq)     # (the same rows again: nothing changes)
        kps = (seq.float() * 0.3).int().clamp(min=1)
        return (ops.decode_attn_q8(q, cache, table, seq, workspace=ws),
                *ops.hybrid_decode_attn_q8(q, cache, table, seq, roles, idx, k, k_per_seq=kps, workspace=ws))

    for job in jobs:
        run(job)
    alone = []
    for job in jobs:
        torch.cuda.synchronize()
        alone.append([x.clone() for x in run(job)])
    torch.cuda.synchronize()
    for _ in range(10):
        order = [0, 3, 1, 4, 2, 0, 2, 4, 1, 3]
        outs = [run(jobs[i]) for i in order]
        torch.cuda.synchronize()
        for i, got in zip(order, outs):
            assert all(torch.equal(a, b) for a, b in zip(got, alone[i]))


def test_a_decode_step_captured_and_replayed():
    """A prompt, then tokens one by one, as a serving loop runs them: the step (append with rotation,
    attention, hybrid layer) is captured once and replayed with lengths and rows changed in place;
    every result against the fp64 definition on the cache the append made."""
    g = torch.Generator().manual_seed(21)
    B, Hq, Hkv, d, page, k = 3, 8, 2, 128, 16, 40
    cap, prompt = 8, [50, 1, 33]
    code, dt = E4, BF
    table = torch.randperm(B * cap, generator=g).int().view(B, cap)
    cache = ops.alloc_q8_cache(B * cap, Hkv, page, d, code, DEV)
    cs = cos_sin(cap * page, d)
    tab, csd = table.to(DEV), cs.to(DEV)
    host = [t.cpu().clone() for t in cache]
    qkv = torch.randn(sum(prompt), Hq + 2 * Hkv, d, generator=g).to(dt)
    cu = torch.tensor([0] + prompt).cumsum(0).int()
    seq = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    x = qkv.to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.append_rope_q8(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, tab, seq, csd, cu_new=cu.to(DEV), device_error=err)
    R.append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], None, *host, table, prompt, cu, cs, False, None)
    tok = torch.zeros(B, Hq + 2 * Hkv, d, dtype=dt, device=DEV)
    roles = [1, 0, 0, 0, 0, 1, 0, 0]
    idx = torch.full((B, Hq, k), -1, dtype=torch.int32, device=DEV)
    idx[:, :, 0] = 0
    shape = (B, Hq, Hkv, d, page, B * cap, cap, dt, code)
    wa, wh = ops.alloc_q8_workspace(*shape), ops.alloc_q8_workspace(*shape, k)
    qr, o1, o2 = (torch.empty(B, Hq, d, dtype=dt, device=DEV) for _ in range(3))
    nxt = torch.empty_like(idx)

    def step():
        ops.append_rope_q8(tok[:, Hq:Hq + Hkv], tok[:, Hq + Hkv:], cache, tab, seq, csd, q=tok[:, :Hq], q_out=qr,
                           device_error=err)
        ops.decode_attn_q8(qr, cache, tab, seq, out=o1, workspace=wa, device_error=err)
        ops.hybrid_decode_attn_q8(qr, cache, tab, seq, roles, idx, k, out=o2, idx_out=nxt, workspace=wh, device_error=err)

    side = torch.cuda.Stream()
    graph = None
    for i in range(20):
        t = torch.randn(B, Hq + 2 * Hkv, d, generator=g).to(dt)
        tok.copy_(t)
        seq += 1
        torch.cuda.synchronize()
        if graph is None:
            with torch.cuda.stream(side):
                step()
            torch.cuda.synchronize()
            # once captured, nothing of the step has run a second time yet
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        lens = seq.cpu()
        qh = torch.empty(B, Hq, d, dtype=dt)
        R.append(t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], t[:, :Hq], *host, table, lens, torch.arange(B + 1), cs, False, qh)
        for a, b in zip(cache, host):
            for r in range(B):
                for j in range((int(lens[r]) + page - 1) // page):
                    p, m = int(table[r, j]), min(page, int(lens[r]) - j * page)
                    assert same(a[p] if a.dim() == 2 else a[p, :, :m], b[p] if b.dim() == 2 else b[p, :, :m])
        assert same(qr, qh)
        for out, sets in ((o1, None), (o2, [[None if r else idx[b, h][idx[b, h] >= 0].tolist()
                                             for h, r in enumerate(roles)] for b in range(B)])):
            ref, tol, raws, rts = R.attend(qh, host, table, lens, sets)
            assert bool(((out.cpu().double() - ref).abs() <= tol + 1e-30).all())
        for b in range(B):
            for h, r in enumerate(roles):
                if r:
                    row = nxt[b, h].cpu()
                    R.check_topk(row[row >= 0].long(), raws[b][h], min(k, int(lens[b])), float(rts[b][h]))
        # the retrieval heads' sets go to the next step's sparse heads
        for h, r in enumerate(roles):
            idx[:, h] = nxt[:, 0 if h < 4 else 5]
    no_flags(err)
