"""The first call of a process may be a captured one: nothing that a call looks up or sets once disturbs
the capture, and the replayed results are the eager ones."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SCRIPT = r"""
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import numpy as np, torch
from eagle_speculative_decoding_03_gb300 import binding as eb
from kv_util import cu, dev, make_cache
which, kind, rows = sys.argv[2], sys.argv[3], int(sys.argv[4])
rng = np.random.default_rng(0)
lens = [5000, 300]
cache, _ = make_cache(rng, kind, 64, 64, 16, lens)
own, _ = make_cache(rng, "bf16", 64, 64, 16, [40 + rows, 9 + rows])
q = torch.randn(2 * rows, 32, 64, device="cuda").to(torch.bfloat16)
at, n, ctx, groups = dev(cu([rows, rows])), dev(np.array(lens, np.int32)), dev(np.array([40, 9], np.int32)), dev(np.array([0, 1, 2], np.int32))
out = torch.zeros_like(q)
calls = {
    "own": lambda o: eb.kv_attention(cache, q, at, n - rows, max_rows=rows, max_len=5000, out=o),
    "cross": lambda o: eb.kv_cross_attention(cache, q, at, n, max_rows=rows, max_len=5000, out=o),
    "shared": lambda o: eb.kv_shared_attention(cache, groups, n, own, q, at, ctx, max_group_rows=rows, max_prefix=5000, max_rows=rows, max_len=40 + rows, out=o),
}
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls[which](out)
g.replay()
torch.cuda.synchronize()
want = torch.zeros_like(q)
calls[which](want)
assert torch.equal(out, want) and torch.isfinite(want.float()).all() and want.abs().max() > 0
assert cache.check() == 0 and own.check() == 0
"""


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("kind", ["bf16", "f4"])
@pytest.mark.parametrize("which", ["own", "cross", "shared"])
def test_first_call_is_captured(which, kind, rows):
    from eagle_speculative_decoding_03_gb300 import build
    build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT, root, which, kind, str(rows)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
