"""GPU parity of eagle_kv_cross_attention (bf16 and 4-bit pages) against the float64 oracle, on
pools whose every unused row holds NaN.  The bound is test_gpu_kv_attention's: the same products,
softmax and roundings."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb
from oracle import kv_oracle as K
from kv_util import cu, dev, make_cache
from test_gpu_kv_attention import check, lib  # noqa: F401

KINDS = ["bf16", "f4"]


def reference(q, held, rows, hd, scale=0.0):
    """(out, lse, magnitudes ...) of all rows: request b's see all of held[b]."""
    parts, at = [], 0
    for (k, v), r in zip(held, rows):
        parts.append(K.attention(q[at:at + r], k, v, np.ones((r, k.shape[0]), bool), scale or hd ** -0.5))
        at += r
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(5))


def run(rng, kind, hd, ps, Hkv, G, lens, rows, pad=0, max_len=None, max_rows=None, scale=0.0, **kw):
    cache, held = make_cache(rng, kind, hd, ps, Hkv, lens)
    N = sum(rows) + pad
    q = K.bf16(rng.standard_normal((N, Hkv * G, hd)))
    out = torch.full((N, Hkv * G, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hkv * G), 7.0, device="cuda")
    eb.kv_cross_attention(cache, dev(q, torch.bfloat16), dev(cu(rows)), dev(np.array(lens, np.int32)),
                          max_rows=max_rows or max(max(rows), 1), max_len=max_len or max(max(lens), 1), scale=scale, out=out, lse=lse, **kw)
    assert cache.check() == 0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = sum(rows)
    check(o[:n], l[:n], reference(q, held, rows, hd, scale), hd)
    empty = np.repeat(np.array(lens) == 0, rows)
    assert (o[:n][empty] == 0).all() and (l[:n][empty] == -np.inf).all()
    assert (o[n:] == 7.0).all() and (l[n:] == 7.0).all()   # rows of no request
    return cache, held, q, out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hd,ps,Hkv,G,lens,rows", [
    (128, 64, 2, 4, [1], [1]),
    (128, 64, 2, 4, [0], [1]),                       # nothing to see
    (64, 16, 1, 1, [0, 1, 15, 16, 17], [1, 1, 1, 1, 1]),
    (128, 64, 2, 4, [127, 128, 129, 0, 255, 256], [1, 1, 1, 1, 1, 1]),
    (64, 32, 16, 1, [300, 1500], [1, 1]),            # a KV head for each query head
    (64, 32, 3, 5, [40, 300, 63], [1, 1, 1]),        # odd group, odd head count
    (128, 128, 1, 8, [1000, 37], [1, 1]),
    (64, 128, 2, 64, [200], [1]),                    # the largest group
    (128, 32, 2, 7, [5000, 3, 0], [1, 1, 0]),        # several key ranges; a request without rows
    (128, 64, 1, 4, [20000], [2]),                   # more ranges than a cluster takes
    (128, 64, 1, 2, [20001, 0, 140], [1, 2, 4]),
    (64, 64, 1, 20, [20001, 140], [1, 1]),
    (128, 64, 8, 2, [1500, 0, 130, 1], [4, 4, 4, 4]),  # ranges of a cluster, some of them empty
    (64, 16, 16, 1, [100 * i for i in range(25)], [1] * 25),
    (128, 128, 4, 8, [64 * i + 1 for i in range(30)], [1] * 30),
    (128, 32, 1, 1, [40000, 63, 64, 65], [7, 8, 0, 5]),
])
def test_few_rows(kind, hd, ps, Hkv, G, lens, rows):
    run(np.random.default_rng(hd + ps + G), kind, hd, ps, Hkv, G, lens, rows, pad=1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hd,ps,Hkv,G,lens,rows", [
    (128, 64, 1, 4, [333], [61]),                    # two query tiles
    (128, 64, 2, 4, [100, 0, 64, 1], [70, 33, 12, 64]),
    (128, 16, 1, 1, [129, 700], [257, 128]),         # blocks with one live tile, with one live vector
    (64, 32, 2, 3, [31, 97, 4000], [64, 33, 90]),
    (64, 16, 1, 8, [513], [300]),
    (128, 128, 2, 8, [900, 128, 127], [77, 0, 40]),
    (128, 32, 1, 8, [6000], [40]),                   # key ranges that meet in a second kernel
    (128, 64, 1, 64, [1, 2, 129], [5, 3, 7]),
])
def test_many_rows(kind, hd, ps, Hkv, G, lens, rows):
    run(np.random.default_rng(hd + sum(rows)), kind, hd, ps, Hkv, G, lens, rows, pad=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [[1, 1], [40, 33]])
def test_bounds_above_the_sizes_and_a_scale(kind, rows):
    """max_rows and max_len are bounds: looser ones leave results within the same tolerance."""
    run(np.random.default_rng(3), kind, 128, 32, 2, 4, [150, 60], rows, max_len=9000, max_rows=130, scale=0.3)


@pytest.mark.parametrize("hd,G,rows,n", [(128, 4, 2, 100), (64, 1, 1, 1500), (128, 5, 3, 30000), (128, 8, 40, 700), (64, 16, 20, 260)])
def test_non_finite_values_in_cached_keys(hd, G, rows, n):
    """An infinity or a NaN among the cached values reaches its own dim of every row and nothing
    else; one in another sequence's keys or behind the last key reaches nothing."""
    rng = np.random.default_rng(21)
    ps = 32
    cache, held = make_cache(rng, "bf16", hd, ps, 1, [n, 50])
    tab = cache.page_table.cpu().numpy()
    kk, vv = held[0]
    for key, dim, val in ((3, 5, np.inf), (n // 2, 17, -np.inf), (n - 1, 30, np.nan), (1, 63, np.inf), (2, 63, -np.inf)):
        cache.v[tab[0, key // ps], 0, key % ps, dim] = float(val)
        vv[key, 0, dim] = 0.0                        # (the other dims' reference)
    q = K.bf16(rng.standard_normal((2 * rows, G, hd)))
    out, lse = eb.kv_cross_attention(cache, dev(q, torch.bfloat16), dev(cu([rows, rows])), dev(np.array([n, 50], np.int32)),
                                     max_rows=rows, max_len=n, lse=True)
    assert cache.check() == 0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (o[:rows, :, 5] == np.inf).all() and (o[:rows, :, 17] == -np.inf).all() and np.isnan(o[:rows][..., [30, 63]]).all()
    ref = reference(q, held, [rows, rows], hd)
    rest = np.delete(np.arange(hd), [5, 17, 30, 63])
    check(o[..., rest], l, (ref[0][..., rest], ref[1], ref[2][..., rest], ref[3], ref[4][..., rest]), hd)
    check(o[rows:], l[rows:], tuple(x[rows:] for x in ref), hd)


@pytest.mark.parametrize("rows", [1, 40])
def test_scores_that_are_not_finite(rows):
    """A key of -infinity scores has no weight; a row that sees nothing else gets zeros and -inf; a
    NaN query makes its own row NaN."""
    rng = np.random.default_rng(5)
    n, G, hd = 200, 4, 128
    cache, held = make_cache(rng, "bf16", hd, 64, 1, [n])
    tab = cache.page_table.cpu().numpy()
    q = K.bf16(np.abs(K.bf16(rng.standard_normal((rows, G, hd)))) + 0.5)      # positive: -inf in a key gives -inf
    cache.k[tab[0, 1], 0, 7, 11] = -float("inf")
    kk, vv = held[0]
    args = (dev(cu([rows])), dev(np.array([n], np.int32)))
    out, lse = eb.kv_cross_attention(cache, dev(q, torch.bfloat16), *args, max_rows=rows, max_len=n, lse=True)
    keep = np.delete(np.arange(n), 64 + 7)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), reference(q, [(kk[keep], vv[keep])], [rows], hd), hd)
    cache.k[torch.from_numpy(tab[0]).long().cuda(), :, :, 11] = -float("inf")
    out, lse = eb.kv_cross_attention(cache, dev(q, torch.bfloat16), *args, max_rows=rows, max_len=n, lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    cache2, _ = make_cache(rng, "bf16", hd, 64, 1, [n])
    good = eb.kv_cross_attention(cache2, dev(q, torch.bfloat16), *args, max_rows=rows, max_len=n)
    q[0, 1, 3] = np.nan
    bad = eb.kv_cross_attention(cache2, dev(q, torch.bfloat16), *args, max_rows=rows, max_len=n)
    assert torch.isnan(bad[0, 1]).all()
    flat, want = bad.reshape(rows * G, hd), good.reshape(rows * G, hd)
    keep = torch.arange(rows * G, device="cuda") != 1
    assert torch.equal(flat[keep], want[keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [[5, 3], [90, 61]])
def test_strided_rows_graph_and_streams(kind, rows):
    """q and out as slices of one buffer of wider rows; replayed from a CUDA graph after the lengths
    changed, on another stream, and two calls at once with a workspace each: bit-equal results."""
    rng = np.random.default_rng(9)
    lens, H, G = [1000, 400], 2, 4
    cache, held = make_cache(rng, kind, 128, 64, H, lens)
    N, w = sum(rows), H * G * 128
    wide = torch.randn(N, 2 * w + 64, device="cuda").to(torch.bfloat16)
    before = wide.clone()
    q, out = wide[:, :w].unflatten(1, (H * G, 128)), wide[:, w + 64:].unflatten(1, (H * G, 128))
    c, n = dev(cu(rows)), dev(np.array(lens, np.int32))
    need = eb.kv_cross_attention_workspace(cache, H * G, N, 2, max(rows), 1000)
    ws = [torch.empty(max(need, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]
    call = lambda **kw: eb.kv_cross_attention(cache, q, c, n, max_rows=max(rows), max_len=1000, **{"workspace": ws[0], **kw})  # noqa: E731
    plain, lse = call(lse=True)
    check(plain.double().cpu().numpy(), lse.double().cpu().numpy(), reference(q.double().cpu().numpy(), held, rows, 128), 128)
    call(out=out)
    assert torch.equal(out, plain) and torch.equal(wide[:, :w + 64], before[:, :w + 64])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = call(stream=side, workspace=ws[1]), call()
    torch.cuda.synchronize()
    assert torch.equal(a, plain) and torch.equal(b, plain)
    gout = torch.zeros_like(plain)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=gout)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, plain)
    n -= 37
    want = call().clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, want) and not torch.equal(want, plain)
    assert cache.check() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 2, 3, 40, 70])
def test_many_short_sequences_repeat(kind, rows):
    """Sequences of one tile, two, none and a few in turn, so that every CTA has items with and without
    a tile for each of its halves, and cuts fall anywhere: right, and the same bits every time."""
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.choice([0, 1, 100, 128, 129, 250, 256, 384, 400, 1000], 60)]
    G = 4
    cache, held, q, out, lse = run(rng, kind, 64, 32, 2, G, lens, [rows] * 60)
    args = (cache, dev(q, torch.bfloat16), dev(cu([rows] * 60)), dev(np.array(lens, np.int32)))
    for _ in range(20):
        o, l = eb.kv_cross_attention(*args, max_rows=rows, max_len=max(lens), lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert cache.check() == 0


def test_bad_pages_rows_and_lengths_are_reported():
    rng = np.random.default_rng(10)
    for rows in ([1, 1], [40, 40]):
        cache, _ = make_cache(rng, "bf16", 128, 16, 1, [40, 40])
        q = torch.randn(sum(rows), 4, 128, device="cuda").to(torch.bfloat16)
        good = cache.page_table.clone()
        R = rows[0]

        def call(c, n, max_rows=R, out=None):
            return eb.kv_cross_attention(cache, q, dev(np.array(c, np.int32)), dev(np.array(n, np.int32)), max_rows=max_rows, max_len=40, out=out)

        def flagged(bits):
            with pytest.raises(eb.EagleError) as e:
                cache.check()
            assert e.value.status == eb.EAGLE_ERR_DEVICE and bits in str(e.value)
        want = call([0, R, 2 * R], [40, 40])
        assert cache.check() == 0
        cache.page_table[0, 1] = cache.k.shape[0]
        got = call([0, R, 2 * R], [40, 40])
        flagged("0x10")
        assert torch.equal(got[R:], want[R:])        # the other request is whole
        cache.page_table.copy_(good)
        for n in ([40, 41], [40, -1]):
            call([0, R, 2 * R], n)
            flagged("0x2")
        for c in ([0, R, 2 * R + 1], [0, R, R - 1], [-1, R, 2 * R]):
            call(c, [40, 40])
            flagged("0x2")
        if R > 1:
            out = torch.full_like(want, 7.0)
            call([0, R, 2 * R], [40, 40], max_rows=R - 1, out=out)
            flagged("0x2")
            assert (out[R - 1] == 7.0).all() and torch.isfinite(out.float()).all()
        assert cache.check() == 0


def test_refusals_of_the_binding():
    cache, _ = make_cache(np.random.default_rng(0), "bf16", 64, 16, 2, [30, 20])
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    c, n = dev(cu([1, 1])), dev(np.array([30, 20], np.int32))
    ok = dict(max_rows=1, max_len=30)
    eb.kv_cross_attention(cache, q, c, n, **ok)
    for bad in (lambda: eb.kv_cross_attention(cache, q.float(), c, n, **ok), lambda: eb.kv_cross_attention(cache, q.cpu(), c, n, **ok),
                lambda: eb.kv_cross_attention(cache, q[:, :, :32], c, n, **ok), lambda: eb.kv_cross_attention(cache, q[:, :3], c, n, **ok),
                lambda: eb.kv_cross_attention(cache, q, c[:2], n, **ok), lambda: eb.kv_cross_attention(cache, q, c.long(), n, **ok),
                lambda: eb.kv_cross_attention(cache, q, c, n, max_rows=0, max_len=30),
                lambda: eb.kv_cross_attention(cache, q, c, n, out=q, **ok),
                lambda: eb.kv_cross_attention(cache, q, c, n, lse=torch.zeros(2, 3, device="cuda"), **ok),
                lambda: eb.kv_cross_attention(cache, q, dev(cu([1, 1, 0])), dev(np.array([1, 1, 1], np.int32)), **ok)):
        with pytest.raises(eb.EagleError) as e:
            bad()
        assert e.value.status == eb.EAGLE_ERR_INVALID_ARG
    empty = eb.kv_cross_attention(cache, q[:0], c * 0, n, **ok)
    assert empty.shape == (0, 4, 64)
    assert cache.check() == 0


def test_pool_of_more_than_2_31_elements():
    """Pages whose offsets pass 32 bits."""
    ps, hd, H = 64, 128, 2
    P = 2 ** 31 // (ps * hd * H) + 600
    rng = np.random.default_rng(11)
    small, held = make_cache(rng, "bf16", hd, ps, H, [500])
    k = torch.zeros(P, H, ps, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    n = small.k.shape[0]
    k[P - n:], v[P - n:] = small.k, small.v
    cache = eb.KVCache(k, v, (small.page_table + (P - n)).contiguous())
    for R in (1, 40):
        q = torch.randn(R, 8, hd, device="cuda").to(torch.bfloat16)
        args = (q, dev(cu([R])), dev(np.array([500], np.int32)))
        assert torch.equal(eb.kv_cross_attention(cache, *args, max_rows=R, max_len=500),
                           eb.kv_cross_attention(small, *args, max_rows=R, max_len=500))
    assert cache.check() == 0
