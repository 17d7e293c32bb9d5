"""Tables far wider than the sequences they hold, up to the capacity that a hybrid layer's selection can take."""
import ctypes

import pytest
import torch

import q8_ref as R
from hybrid_head_sparse_decode_b200 import _native as N
from hybrid_head_sparse_decode_b200 import ops
from test_q8_host import FAKE, cache, lib, shape  # noqa: F401  (lib: the fixture)

DEV = "cuda"
E4, I8 = torch.float8_e4m3fn, torch.int8
BF, F32 = torch.bfloat16, torch.float32


def test_capacities_beyond_the_selection(lib):  # noqa: F811
    """Refused before anything is launched; with sparse heads only, or with blocks, they are taken (and the calls end at
    the next thing that is wrong, the workspace)."""
    c, some, none = cache(), (ctypes.c_uint8 * 8)(1), (ctypes.c_uint8 * 8)()

    def call(pages, roles, B=2, block=0):
        return lib.lychee_hybrid_decode_attn_q8(shape(page=128, max_pages=pages, B=B), 64, block, FAKE + (1 << 24), c, FAKE, None,
                                                roles, FAKE, FAKE + (1 << 25), FAKE + (1 << 26), None, 0, None, None)

    assert call(39800, some) == N.ERR_WORKSPACE            # 5 094 400 positions
    assert call(39801, some, B=100) == N.ERR_UNSUPPORTED
    assert call(63217, some) == N.ERR_UNSUPPORTED          # 8 091 776
    assert call(1 << 17, some) == N.ERR_UNSUPPORTED
    assert call(1 << 17, none) == N.ERR_WORKSPACE
    assert call(8192, some, block=32) == N.ERR_WORKSPACE   # 32768 blocks


def run(lens, pages, page, Hq, Hkv, d, dtype, code, roles, k, seed=53):
    """One hybrid layer and the attention over every position, the table `pages` wide; the narrow table gives the same bits
    where the split is the same, and the definition bounds both."""
    g = torch.Generator().manual_seed(seed)
    table, P = R.make_table(g, lens, page)
    cache_ = R.make_cache(g, P, Hkv, page, d, code)
    q = torch.randn(len(lens), Hq, d, generator=g).to(dtype)
    seq = torch.tensor(lens, dtype=torch.int32)
    idx = torch.full((len(lens), Hq, k), -1, dtype=torch.int32)
    sets = [[None] * Hq for _ in lens]
    for b, n in enumerate(lens):
        for h in range(Hq):
            if not roles[h]:
                s = torch.randperm(n, generator=g)[:k].sort().values
                sets[b][h], idx[b, h, :len(s)] = s.tolist(), s.int()
    wide = torch.full((len(lens), pages), -5, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    dev = ops.Q8Cache(*(t.to(DEV) for t in cache_))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, nxt = ops.hybrid_decode_attn_q8(q.to(DEV), dev, wide.to(DEV), seq.to(DEV), roles, idx.to(DEV), k, device_error=err)
    full = ops.decode_attn_q8(q.to(DEV), dev, wide.to(DEV), seq.to(DEV), device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for got, which in ((out, sets), (full, None)):
        ref, tol, raws, rts = R.attend(q, cache_, table, seq, which)
        assert bool(((got.cpu().double() - ref).abs() <= tol + 1e-30).all())
    nxt = nxt.cpu()
    for b, n in enumerate(lens):
        for h in range(Hq):
            if roles[h]:
                R.check_topk(nxt[b, h][nxt[b, h] >= 0].long(), raws[b][h], min(k, n), float(rts[b][h]))
            else:
                assert torch.equal(nxt[b, h], idx[b, h])


@pytest.mark.gpu
@pytest.mark.parametrize("pages,page", [(2048, 64), (39800, 128), (39801, 128), (63216, 128)])
def test_wide_tables(pages, page):
    run([3000, 70, 1], pages, page, 2, 1, 64, BF, E4, [1, 0], 200)


@pytest.mark.gpu
def test_the_widest_table_of_sparse_heads():
    run([3000, 5], 1 << 17, 128, 2, 1, 64, F32, I8, [0, 0], 100)


@pytest.mark.gpu
@pytest.mark.parametrize("roles", [[1] * 8, [1, 1, 0, 0, 1, 1, 1, 1], [0, 1, 1, 1, 0, 0, 0, 0]])
def test_long_rows_with_several_retrieval_heads_a_group(roles):
    run([60000, 33333], 1100, 64, 8, 2, 128, BF, E4, roles, 18000)


@pytest.mark.gpu
def test_refused_capacities_launch_nothing():
    g = torch.Generator().manual_seed(3)
    for pages, B in ((39801, 100), (63217, 1)):
        table = torch.zeros(B, pages, dtype=torch.int32, device=DEV)
        c = ops.Q8Cache(*(t.to(DEV) for t in R.make_cache(g, 2, 1, 128, 64, E4)))
        q = torch.randn(B, 2, 64, generator=g).to(BF).to(DEV)
        idx = torch.zeros(B, 2, 4, dtype=torch.int32, device=DEV)
        out, nxt = torch.full_like(q, 3.0), torch.full_like(idx, 9)
        with pytest.raises(N.LycheeError, match="unsupported"):
            ops.hybrid_decode_attn_q8(q, c, table, torch.ones(B, dtype=torch.int32, device=DEV), [1, 0], idx, 4, out=out, idx_out=nxt,
                                      workspace=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        assert bool((out == 3.0).all()) and bool((nxt == 9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("page,code", [(128, E4), (16, I8)])
def test_a_cache_of_more_than_4_gib(page, code):
    """Codes beyond 2^32 bytes: the same bits as from a small cache, appended, attended to and selected from."""
    g = torch.Generator().manual_seed(61)
    Hq, Hkv, d, lens, k = 8, 2, 128, [3001, 500], 300
    P = (4500 << 20) // (Hkv * page * d)
    table, small_pages = R.make_table(g, lens, page)
    small = ops.Q8Cache(*(t.to(DEV) for t in R.make_cache(g, small_pages, Hkv, page, d, code)))
    big = ops.alloc_q8_cache(P, Hkv, page, d, code, DEV)
    # page i of the small cache lies near the big one's end, or (every third) where it is
    at = torch.arange(small_pages)
    at = torch.where(at % 3 == 0, at, P - 1 - at)
    assert big.k.numel() > 1 << 32 and int(at.max()) * Hkv * page * d > 1 << 32
    for a, b in zip(big, small):
        a.view(torch.uint8)[at.to(DEV)] = b.view(torch.uint8)
    far = torch.where(table >= 0, at[table.clamp(min=0).long()].int(), -1).int()
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q, rows = torch.randn(2, Hq, d, generator=g).to(BF).to(DEV), torch.randn(40, Hkv, d, generator=g).to(BF).to(DEV)
    idx = torch.stack([torch.stack([torch.randperm(n, generator=g)[:k].sort().values for _ in range(Hq)]) for n in lens]).int().to(DEV)
    cu = torch.tensor([0, 17, 40], dtype=torch.int32, device=DEV)
    got = []
    for c, t in ((small, table.to(DEV)), (big, far.to(DEV))):
        ops.append_rope_q8(rows, rows, c, t, seq, cu_new=cu)
        got.append([ops.decode_attn_q8(q, c, t, seq), *ops.hybrid_decode_attn_q8(q, c, t, seq, [1] + [0] * 7, idx, k)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    for a, b in zip(big, small):
        assert torch.equal(a.view(torch.uint8)[at.to(DEV)], b.view(torch.uint8))
