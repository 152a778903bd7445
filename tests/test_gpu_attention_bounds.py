"""Bounds far above the lengths, as a captured step has that is bounded by its cache's capacity: the ranges are
shared out over the keys that there are, so that results stay right and the call takes no multiple of its time."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb
from kv_util import cu, dev, make_cache
from test_gpu_cross_attention import run as run_cross
from test_gpu_kv_attention import lib  # noqa: F401
from test_gpu_kv_attention import run as run_own


@pytest.mark.parametrize("kind", ["bf16", "f4"])
@pytest.mark.parametrize("hd,ps,Hkv,G,lens,rows", [
    (128, 64, 2, 4, [3000], [1]), (64, 32, 3, 5, [700, 0, 5000], [2, 1, 3]), (128, 128, 8, 4, [1000 + 99 * i for i in range(12)], [1] * 12),
    (128, 64, 1, 8, [4000, 129], [30, 7]), (64, 64, 2, 4, [900, 2500], [90, 64]),
])
@pytest.mark.parametrize("bound", [20_000, 300_000, 1 << 24])
def test_results_under_loose_bounds(kind, hd, ps, Hkv, G, lens, rows, bound):
    run_cross(np.random.default_rng(sum(lens)), kind, hd, ps, Hkv, G, lens, rows, pad=1, max_len=bound)
    run_own(np.random.default_rng(sum(lens)), kind, hd, ps, Hkv, G, lens, rows, pad=1, max_len=bound)


def elapsed(f):
    for _ in range(3):
        f()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    times = []
    for _ in range(15):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        g.replay()
        e[1].record()
        torch.cuda.synchronize()
        times.append(e[0].elapsed_time(e[1]))
    return float(np.median(times))


@pytest.mark.parametrize("G,rows", [(4, 1), (4, 8)])
def test_a_loose_bound_takes_no_multiple_of_the_time(G, rows):
    """One request of 32,000 keys under a bound 16 times as high: eight CTAs did all of the work, 7 times as long."""
    n, H = 32000, 8
    table = torch.randperm(500, device="cuda").int()[None].contiguous()
    cache = eb.KVCache.empty(500, 64, H, 128, table)
    cache.k.normal_()
    cache.v.normal_()
    q = torch.randn(rows, H * G, 128, device="cuda").to(torch.bfloat16)
    c, lens = dev(cu([rows])), dev(np.array([n - rows], np.int32))
    for call in (eb.kv_cross_attention, eb.kv_attention):
        tight, loose = (elapsed(lambda: call(cache, q, c, lens, max_rows=rows, max_len=m)) for m in (n, 16 * n))
        assert loose < 1.6 * tight, (call.__name__, tight, loose)
    assert cache.check() == 0
