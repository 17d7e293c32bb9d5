"""The failure path of the 8-bit cache's bounded waits, on the GPU without a fault: in a child process whose environment
shortens the limit to 200 ms and makes every warp's first stage expect an arrival that never comes
(LYCHEE_TEST_WAIT_LIMIT_MS, LYCHEE_TEST_WITHHOLD_ITEM, read once per process by the library), the waits run out, the
slabs on their way still land in the ring, every kernel returns, the error word reports it (bit 8) and the context is
still usable.  The parent process sets neither variable."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import sys, time, torch
    sys.path[:0] = [{root!r}, {root!r} + "/tests"]
    import q8_ref as R
    from hybrid_head_sparse_decode_b200 import ops
    for n, page, dtype, code in ((300, 16, torch.float32, torch.int8), (9001, 64, torch.bfloat16, torch.float8_e4m3fn)):
        g = torch.Generator().manual_seed(1)
        table, P = R.make_table(g, [n], page)
        cache = ops.Q8Cache(*(t.cuda() for t in R.make_cache(g, P, 2, page, 64, code)))
        table, seq = table.cuda(), torch.tensor([n], dtype=torch.int32).cuda()
        q = torch.randn(1, 8, 64, generator=g).to(dtype).cuda()
        idx = torch.arange(100, dtype=torch.int32).expand(1, 8, 100).contiguous().cuda()
        shape = (1, 8, 2, 64, page, P, table.shape[1], dtype, code)
        ws, wh = ops.alloc_q8_workspace(*shape), ops.alloc_q8_workspace(*shape, 100)
        t0 = time.time()
        ops.decode_attn_q8(q, cache, table, seq, workspace=ws)
        a = ops.check_device_error(ws)
        ops.hybrid_decode_attn_q8(q, cache, table, seq, [1, 1, 0, 0, 0, 0, 0, 0], idx, 100, workspace=wh)
        b = ops.check_device_error(wh)
        ok = float(torch.ones(1000, device="cuda").sum().item()) == 1000.0
        print("RESULT", *a, *b, ok, round(time.time() - t0, 2))
""")


def test_waits_run_out_and_report_timeout():
    env = dict(os.environ, LYCHEE_TEST_WAIT_LIMIT_MS="200", LYCHEE_TEST_WITHHOLD_ITEM="1")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [x.split()[1:] for x in r.stdout.splitlines() if x.startswith("RESULT")]
    assert len(lines) == 2
    for st_a, bits_a, st_b, bits_b, ok, secs in lines:
        assert st_a == st_b == "6" and int(bits_a) & 8 and int(bits_b) & 8      # LYCHEE_ERR_TIMEOUT
        assert ok == "True" and float(secs) < 20
