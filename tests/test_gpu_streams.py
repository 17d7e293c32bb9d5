"""Calls given a stream of their own allocate there: what they make is neither memory that another stream is still using
nor memory that another stream gets while their kernels run."""
import pytest
import torch

import q8_ref as R
from hybrid_head_sparse_decode_b200 import inputs, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F64 = torch.bfloat16, torch.float64


def q8_job(seed, n=5000, B=2):
    """Calls on a cache of their own, as functions of the stream."""
    g = torch.Generator().manual_seed(seed)
    table, P = R.make_table(g, [n] * B, 64)
    cache = ops.Q8Cache(*(t.to(DEV) for t in R.make_cache(g, P, 2, 64, 128, torch.float8_e4m3fn)))
    table, seq = table.to(DEV), torch.full((B,), n, dtype=torch.int32, device=DEV)
    q = torch.randn(B, 8, 128, generator=g).to(BF).to(DEV)
    rows = torch.randn(B, 2, 128, generator=g).to(BF).to(DEV)
    k = 700
    idx = torch.rand(B, 8, n, generator=g).topk(k, dim=2).indices.sort(dim=2).values.int().to(DEV)
    other = ops.Q8Cache(*(t.clone() for t in cache))
    return [lambda s: (ops.decode_attn_q8(q, cache, table, seq, stream=s),),
            lambda s: ops.hybrid_decode_attn_q8(q, cache, table, seq, [1] + [0] * 7, idx, k, stream=s),
            lambda s: (ops.append_rope_q8(rows, rows, other, table, seq, q=q, stream=s),)]


def bf16_job(seed):
    p = inputs.make_layer(1, 8, 2, 128, 4096, roles=[1, 0, 0, 0, 0, 0, 0, 1], seed=seed, k_frac=0.3, device=torch.device(DEV))
    st = inputs.make_stack(3, 1, 8, 2, 128, 2048, seed=seed, k_frac=0.3, n_extra_retrieval=2)
    qs, ks, vs, sl, kps = (st.q.to(DEV), [t.to(DEV) for t in st.k_caches], [t.to(DEV) for t in st.v_caches], st.seqlens.to(DEV),
                           st.k_per_seq.to(DEV))
    ab = torch.rand(3, 8, dtype=F64, device=DEV) + 0.5
    return [lambda s: ops.hybrid_decode_attn(p.q, p.k_cache, p.v_cache, p.seqlens, p.role, p.idx_in, p.k, k_per_seq=p.k_per_seq,
                                             stream=s),
            lambda s: ops.hybrid_decode_attn_noalloc(p.q, p.k_cache, p.v_cache, p.seqlens, p.role, p.idx_in, p.k,
                                                     k_per_seq=p.k_per_seq, stream=s),
            lambda s: ops.decode_stack(qs, ks, vs, sl, st.roles, st.k, k_per_seq=kps, want_layers=True, stream=s),
            lambda s: ops.hardkuma_roles(ab, ab, stream=s)]


def stream_of(t):
    """The stream whose pool holds t's memory."""
    at = t.data_ptr()
    return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]


@pytest.mark.parametrize("make", [q8_job, bf16_job])
def test_what_a_call_allocates_belongs_to_its_stream(make, monkeypatch):
    calls = make(3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made = []
    plain = torch.empty

    def spy(*a, **kw):
        t = plain(*a, **kw)
        if t.is_cuda:
            made.append(stream_of(t))      # the temporary workspace among them
        return t

    monkeypatch.setattr(torch, "empty", spy)
    for call in calls:
        made.clear()
        outs = [t for t in call(side) if t is not None]
        assert made and all(m == [side.cuda_stream] for m in made), made
        assert all(stream_of(t) == [side.cuda_stream] for t in outs)
        made.clear()
        call(None)
        assert made and all(m == [torch.cuda.current_stream().cuda_stream] for m in made), made
    torch.cuda.synchronize()


def test_a_forked_stream_in_a_capture():
    """A call on a stream that a capture was forked to, making its own workspace and outputs: replays give its results."""
    calls = q8_job(7)[:2]
    want = [[t.clone() for t in call(None)] for call in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for call in calls:
            call(side)                            # (dropped at once)
        got = [call(side) for call in calls]
        torch.cuda.current_stream().wait_stream(side)
        kept = [[t.clone() for t in outs] for outs in got]
    del got
    for _ in range(3):
        for outs in kept:
            for t in outs:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for outs, ref in zip(kept, want) for a, b in zip(outs, ref))


def test_two_streams_without_workspaces():
    """Calls side by side on two streams, each with a workspace of its own making, other work on the current stream taking
    memory meanwhile: the results of the calls alone."""
    jobs = [q8_job(1)[:2], q8_job(2, 9000, 1)[:2]]
    alone = []
    for job in jobs:
        alone.append([[t.clone() for t in call(None)] for call in job])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i, job in enumerate(jobs):
            got.append([(i, c, call(streams[i])) for c, call in enumerate(job)])
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (1 << 20, 5 << 20, 1 << 24)]
        del junk
    torch.cuda.synchronize()
    for rows in got:
        for i, c, outs in rows:
            assert all(torch.equal(a, b) for a, b in zip(outs, alone[i][c]))
