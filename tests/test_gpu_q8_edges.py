"""The 8-bit cache's calls at the edges of what their documentation allows: bad pages, queries and scores that are not
ordinary numbers, workspaces that held something else."""
import pytest
import torch

import q8_ref as R
from hybrid_head_sparse_decode_b200 import _native as N
from hybrid_head_sparse_decode_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4, I8 = torch.float8_e4m3fn, torch.int8
BF, F32 = torch.bfloat16, torch.float32


def to_dev(cache):
    return ops.Q8Cache(*(t.to(DEV) for t in cache))


# ---- pages that are none --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,code,page,n,block", [(BF, E4, 64, 1500, 0), (F32, I8, 16, 300, 0), (BF, I8, 32, 9000, 64),
                                                     (BF, E4, 16, 1030, 32)])
def test_positions_on_bad_pages_rank_last(dtype, code, page, n, block):
    """A retrieval head's set holds no position whose page is none while there are others, whatever the workspace held; and
    no head attends to one."""
    g = torch.Generator().manual_seed(17)
    lens, Hq, Hkv, d = [n, 90], 16, 4, 64
    roles = [1, 0, 0, 0] + [1, 1, 1, 1] + [0, 0, 0, 0] + [0, 0, 1, 1]
    table, P = R.make_table(g, lens, page)
    cache = R.make_cache(g, P, Hkv, page, d, code)
    q = torch.randn(2, Hq, d, generator=g).to(dtype)
    bad = table.clone()
    last = (n + page - 1) // page - 1
    for j, x in ((0, -1), (last // 2, P), (last // 2 + 1, 1 << 30), (last, -7)):
        bad[0, j] = x
    here = [torch.tensor([0 <= int(bad[b, i // page]) < P for i in range(m)]) for b, m in enumerate(lens)]
    k = 256
    sets = [[None if roles[h] else torch.nonzero(torch.rand(lens[b], generator=g) < 0.1)[:k, 0] for h in range(Hq)] for b in range(2)]
    idx = torch.full((2, Hq, k), -1, dtype=torch.int32)
    for b in range(2):
        for h in range(Hq):
            if sets[b][h] is not None:
                idx[b, h, :len(sets[b][h])] = sets[b][h].int()
    keep = [[(torch.nonzero(here[b])[:, 0] if s is None else s[here[b][s]]) for s in sets[b]] for b in range(2)]
    seq = torch.tensor(lens, dtype=torch.int32)
    ref, tol, raws, rts = R.attend(q, cache, torch.where((bad < 0) | (bad >= P), 0, bad), seq, keep)
    size = ops.q8_workspace_size(2, Hq, Hkv, d, page, P, table.shape[1], dtype, code, k)
    seen = []
    for fill in (0, 0x7f, 0xff):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, nxt = ops.hybrid_decode_attn_q8(q.to(DEV), to_dev(cache), bad.to(DEV), seq.to(DEV), roles, idx.to(DEV), k,
                                             workspace=ws, device_error=err, block=block)
        torch.cuda.synchronize()
        assert int(err.item()) == 1
        off = (out.cpu().double() - ref).abs()
        assert bool((off <= tol + 1e-30).all())
        nxt = nxt.cpu()
        seen.append(nxt)
        for b in range(2):
            for h in range(Hq):
                if not roles[h]:
                    assert torch.equal(nxt[b, h], idx[b, h])
                    continue
                got = nxt[b, h][nxt[b, h] >= 0].long()
                raw = torch.where(here[b], raws[b][h], -torch.inf)
                if block:
                    nblk = (lens[b] + block - 1) // block
                    score = torch.stack([raw[i * block:(i + 1) * block].max() for i in range(nblk)])
                    R.check_topk(torch.unique(got // block), score, min(max(1, min(k, lens[b]) // block), nblk), float(rts[b][h]))
                else:
                    R.check_topk(got, raw, min(k, lens[b]), float(rts[b][h]))
                    # (the rest of a set larger than what is there: the lowest positions)
                    lost = got[~here[b][got]]
                    assert torch.equal(lost, torch.nonzero(~here[b])[:len(lost), 0])
    assert torch.equal(seen[0], seen[1]) and torch.equal(seen[0], seen[2])


# ---- queries and scores that are not ordinary numbers ---------------------------------------------

@pytest.mark.parametrize("n", [1, 300, 1030, 20000])
@pytest.mark.parametrize("dtype,Hq", [(BF, 8), (F32, 8), (BF, 16), (F32, 2)])
def test_queries_that_are_no_numbers(dtype, Hq, n):
    """A NaN or an infinity in a query makes its head's output NaN, however the work is split; the other heads' are as
    without it.  A head whose set is empty gives zeros all the same."""
    g = torch.Generator().manual_seed(23)
    Hkv, d, page = 2, 128, 64
    table, P = R.make_table(g, [n], page)
    cache = to_dev(R.make_cache(g, P, Hkv, page, d, E4))
    table, seq = table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    q = torch.randn(1, Hq, d, generator=g).to(dtype).to(DEV)
    bad = q.clone()
    bad[0, 0, 77] = float("nan")
    bad[0, Hq - 1, 0] = -float("inf")
    hit = torch.zeros(Hq, dtype=torch.bool, device=DEV)
    hit[0] = hit[Hq - 1] = True
    out, want = ops.decode_attn_q8(bad, cache, table, seq), ops.decode_attn_q8(q, cache, table, seq)
    assert bool(out[0, hit].isnan().all()) and torch.equal(out[0, ~hit], want[0, ~hit])
    k = min(n, 50)
    idx = torch.arange(k, dtype=torch.int32, device=DEV).expand(1, Hq, k).contiguous()
    for roles in ([1] * Hq, [0] * Hq, [1] + [0] * (Hq - 1)):
        got, sets = ops.hybrid_decode_attn_q8(bad, cache, table, seq, roles, idx, k)
        want, _ = ops.hybrid_decode_attn_q8(q, cache, table, seq, roles, idx, k)
        assert bool(got[0, hit].isnan().all()) and torch.equal(got[0, ~hit], want[0, ~hit])
        assert bool((sets[0, :, 1:] > sets[0, :, :-1]).all()) and int(sets.min()) >= 0 and int(sets.max()) < n
    none = torch.full_like(idx, -1)
    got, _ = ops.hybrid_decode_attn_q8(bad, cache, table, seq, [0] * Hq, none, k)
    assert not bool(got.any())


@pytest.mark.parametrize("n", [40, 5000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_near_the_end_of_fp32(dtype, n):
    """Scores of -1e34, all equal or with one above the rest, and huge queries on rows of zeros: softmaxes like any other."""
    g = torch.Generator().manual_seed(29)
    Hq, Hkv, d, page = 8, 2, 128, 32
    table, P = R.make_table(g, [n], page)
    cache = R.make_cache(g, P, Hkv, page, d, I8)
    seq = torch.tensor([n], dtype=torch.int32)
    cache[2].fill_(1.0)
    cache[0].fill_(-1)
    q = torch.full((1, Hq, d), 2.0 ** 106, dtype=dtype)
    idx = torch.arange(n, dtype=torch.int32).expand(1, Hq, n).contiguous()

    def check():
        ref, tol, _, _ = R.attend(q, cache, table, seq)
        args = q.to(DEV), to_dev(cache), table.to(DEV), seq.to(DEV)
        for out in (ops.decode_attn_q8(*args), ops.hybrid_decode_attn_q8(*args, [0] * Hq, idx.to(DEV), n)[0]):
            off = (out.cpu().double() - ref).abs()
            # (the scores are powers of two or zeros, exact in every step: nothing is lost in them)
            V = R.rows_of(cache[1], cache[3], table[0], n)
            assert bool((off <= 2.0 ** -8 * ref.abs() + 2.0 ** -16 * V.abs().max()).all()), float(off.max())

    check()                                         # the mean of the values
    at = n // 3
    cache[0][int(table[0, at // page]), :, at % page] = -127
    cache[0][int(table[0, 0]), :, 1] = 0            # one row's scores are 0, above all others
    check()
    cache[0].fill_(0)                               # scores of 0 with the largest query and scale
    cache[2].fill_(2.0 ** 60)
    q.fill_(2.0 ** 127)
    check()


# ---- errors without an error word of the caller's --------------------------------------------------

def test_flags_go_to_the_workspace():
    """Without device_error the bits are OR-ed into the workspace's first word, stay there over calls, and
    check_device_error reads and clears them; with it the workspace keeps none."""
    g = torch.Generator().manual_seed(37)
    lens, Hq, Hkv, d, page, k = [2000, 70], 8, 2, 64, 16, 30
    table, P = R.make_table(g, lens, page)
    cache = to_dev(R.make_cache(g, P, Hkv, page, d, I8))
    bad = table.clone()
    bad[0, 3] = P
    table, bad, seq = table.to(DEV), bad.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn(2, Hq, d, generator=g).to(BF).to(DEV)
    idx = torch.arange(k, dtype=torch.int32, device=DEV).expand(2, Hq, k).contiguous()
    wrong = idx.clone()
    wrong[1, 7, 5] = 4
    roles = [1] + [0] * 7
    shape = (2, Hq, Hkv, d, page, P, table.shape[1], BF, I8)
    ws, wh = ops.alloc_q8_workspace(*shape), ops.alloc_q8_workspace(*shape, k)

    def dense(table, **kw):
        return ops.decode_attn_q8(q, cache, table, seq, workspace=ws, **kw)

    def hybrid(table, sets, **kw):
        return ops.hybrid_decode_attn_q8(q, cache, table, seq, roles, sets, k, workspace=wh, **kw)

    clean, layer = dense(table), hybrid(table, idx)
    assert ops.check_device_error(ws) == (N.OK, 0) and ops.check_device_error(wh) == (N.OK, 0)
    dense(bad)
    dense(table)
    hybrid(table, wrong)
    hybrid(table, idx, k_per_seq=torch.zeros(2, dtype=torch.int32, device=DEV))
    assert ops.check_device_error(ws) == (N.ERR_BAD_INDEX, 1) and ops.check_device_error(wh) == (N.ERR_BAD_INDEX, 5)
    assert ops.check_device_error(ws) == (N.OK, 0) and ops.check_device_error(wh) == (N.OK, 0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dense(bad, device_error=err)
    hybrid(table, wrong, device_error=err)
    assert int(err.item()) == 1
    assert ops.check_device_error(ws) == (N.OK, 0) and ops.check_device_error(wh) == (N.OK, 0)
    # reading and clearing the word changes no call's results
    again = hybrid(table, idx)
    assert torch.equal(dense(table), clean) and torch.equal(again[0], layer[0]) and torch.equal(again[1], layer[1])


@pytest.mark.parametrize("dtype,Hq,d,interleaved", [(BF, 8, 128, False), (F32, 16, 64, True), (BF, 2, 64, True)])
def test_queries_of_skipped_sequences(dtype, Hq, d, interleaved):
    """Rotated queries of a sequence whose numbers do not fit are NaN, not what the buffer held; rows of tokens that no
    sequence owns, and of empty places, stay as they were."""
    g = torch.Generator().manual_seed(43)
    Hkv, page, new = 2, 16, [3, 5, 0, 40, 2, 1]
    T = sum(new) + 2
    table = torch.arange(12, dtype=torch.int32).view(6, 2)
    #                  fits, beyond max_pages, none, beyond cos_sin, shorter than its new tokens, fits
    seq = torch.tensor([20, 33, 99, 32, 1, 31], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0] + new).cumsum(0).int()
    a = torch.rand(31, d // 2, generator=g)
    cs = torch.cat([a.cos(), a.sin()], 1).to(DEV)
    q, kn = torch.randn(T, Hq, d, generator=g).to(dtype).to(DEV), torch.randn(T, Hkv, d, generator=g).to(dtype).to(DEV)
    cache = to_dev(R.make_cache(g, 12, Hkv, page, d, I8))
    before = [t.clone() for t in cache]
    out = torch.full_like(q, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.append_rope_q8(kn, kn, cache, table.to(DEV), seq, cs, q=q, q_out=out, cu_new=cu.to(DEV), interleaved=interleaved,
                       device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 2
    lost = torch.zeros(T, dtype=torch.bool, device=DEV)
    lost[cu[1]:cu[2]] = lost[cu[3]:cu[4]] = lost[cu[4]:cu[5]] = True
    assert bool(out[lost].isnan().all()) and not bool(out[~lost].isnan().any())
    assert bool((out[T - 2:] == 7.0).all()) and not bool((out[:T - 2][~lost[:T - 2]] == 7.0).any())
    for t, was in zip(cache, before):
        assert torch.equal(t.view(torch.uint8)[2:4], was.view(torch.uint8)[2:4])
        assert torch.equal(t.view(torch.uint8)[4:10], was.view(torch.uint8)[4:10])
    # a token each: an empty place, a length that does not fit, below zero
    for n, is_nan in ((0, False), (32, True), (-4, True)):
        out = torch.full_like(q[:2], 7.0)
        ops.append_rope_q8(kn[:2], kn[:2], cache, table[:2].contiguous().to(DEV), torch.tensor([n, 9], dtype=torch.int32, device=DEV),
                           cs, q=q[:2], q_out=out, interleaved=interleaved)
        torch.cuda.synchronize()
        assert bool(out[0].isnan().all()) if is_nan else bool((out[0] == 7.0).all())
        assert not bool(out[1].isnan().any())
