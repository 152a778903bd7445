"""GPU parity of eagle_kv_attention (bf16 and 4-bit pages; tree masks and causal rows) against
the float64 oracle, on pools whose every unused row holds NaN.

Bound, per output: the products are exact in fp32 up to the accumulation, so a score is off by
at most eps_s = (hd + 4) 2^-24 qk (qk the largest sum |q k| scale) plus the exponent's own rounding
(2^-22 relative in 2^x, and its argument's 2^-23 |s| twice); p keeps 8 significant bits at least in
the second product (relative 2^-8), sums add (hd + 128) 2^-24 relative.  So out is off by at most
(2^-8 + 2 (eps_s + eps_e)) sum p |v| / sum p, and its bf16 rounding 2^-8 |out| on top.  With a
4-bit cache p is an fp16 number held times 2^7 or more where it is largest: below fp16's normal
range its rounding is absolute, half a step of 2^-24, which is 2^-32 of the largest p per key, or
2^-32 sum |v| of the output (a key that takes all and whose value is a zero code leaves no
relative bound).  The
log-sum-exp is off by eps_s + eps_e + 2^-23 |lse|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb
from oracle import kv_oracle as K
from kv_util import cu, dev, make_cache, see_matrix, tree_masks


@pytest.fixture(scope="module", autouse=True)
def lib():
    from eagle_speculative_decoding_03_gb300 import build
    build.build()
    return eb.load()


def check(out, lse, ref, hd):
    o, l, mag, qk, vsum = ref
    eps_s = (hd + 4) * 2.0 ** -24 * qk
    eps_e = 2.0 ** -21 + 2.0 ** -21 * qk
    tol = (2.0 ** -8 + 2 * (eps_s + eps_e)[..., None] + (hd + 128) * 2.0 ** -24) * mag + 2.0 ** -8 * np.abs(o) + 2.0 ** -32 * vsum + 1e-30
    bad = ~(np.abs(out - o) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], float(np.nanmax(np.abs(out - o) / tol)))
    some = np.isfinite(l)
    assert (lse[~some] == -np.inf).all()
    dl = np.abs(lse[some] - l[some])
    tl = (eps_s + eps_e)[some] + 2.0 ** -21 * (1 + np.abs(l[some]))
    assert (dl <= tl).all(), float((dl / tl).max())


def run(rng, kind, hd, ps, Hkv, G, ctx, rows, tree=False, S=None, scale=0.0, mask=None, pad=0, max_len=None, qscale=1.0):
    keys = [c + r for c, r in zip(ctx, rows)]
    cache, held = make_cache(rng, kind, hd, ps, Hkv, keys)
    N = sum(rows) + pad
    q = K.bf16(qscale * rng.standard_normal((N, Hkv * G, hd)))
    if tree and mask is None:
        mask = tree_masks(rng, len(ctx), S or max(max(rows), 1), rows)
    out = torch.full((N, Hkv * G, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hkv * G), 7.0, device="cuda")
    eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu(rows)), dev(np.array(ctx, np.int32)), max_rows=max(max(rows), 1),
                    max_len=max_len or max(max(keys), 1), mask=None if mask is None else dev(mask), scale=scale, out=out, lse=lse)
    assert cache.check() == 0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    at = 0
    for b, (c, r) in enumerate(zip(ctx, rows)):
        if r:
            ref = K.attention(q[at:at + r], held[b][0], held[b][1], see_matrix(c, r, None if mask is None else mask[b]),
                              scale or hd ** -0.5)
            check(o[at:at + r], l[at:at + r], ref, hd)
        at += r
    assert (o[at:] == 7.0).all() and (l[at:] == 7.0).all()   # rows of no request
    return cache, out


KINDS = ["bf16", "f4"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hd,ps,Hkv,G,ctx,rows", [
    (128, 64, 2, 4, [0], [1]),                       # the first token
    (128, 16, 1, 1, [1, 0, 15, 16, 17], [1, 1, 1, 1, 1]),
    (128, 64, 2, 4, [127, 128, 129, 0, 255], [1, 1, 1, 1, 1]),
    (64, 32, 3, 5, [40, 300, 63], [1, 1, 1]),        # odd group, odd head count
    (128, 128, 1, 8, [1000, 37], [1, 1]),            # a page larger than what is left of it
    (64, 128, 2, 64, [200], [1]),                    # the largest group
    (128, 32, 2, 7, [5000, 3, 0], [1, 1, 0]),        # several key ranges; a request without rows
    (128, 64, 1, 4, [20000], [2]),                   # more ranges than a cluster takes
    (64, 64, 1, 20, [20001, 140], [1, 1]),           # the same, the second request in the first range
    (128, 64, 8, 2, [1500, 130, 1], [4, 4, 4]),      # ranges of a cluster, some of them empty
])
def test_single_tokens(kind, hd, ps, Hkv, G, ctx, rows):
    run(np.random.default_rng(hd + ps + G), kind, hd, ps, Hkv, G, ctx, rows)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hd,ps,Hkv,G,ctx,rows,S", [
    (128, 64, 2, 4, [100, 0, 64], [7, 1, 12], 12),
    (128, 16, 1, 4, [333], [61], 64),                # 244 vectors: two query tiles
    (128, 128, 2, 8, [120, 127], [61, 13], 61),      # the tree crosses a tile; two blocks of vectors
    (64, 32, 2, 3, [31, 97], [64, 33], 64),
    (128, 64, 1, 1, [2000], [40], 40),
])
def test_tree_rows(kind, hd, ps, Hkv, G, ctx, rows, S):
    run(np.random.default_rng(S + ps), kind, hd, ps, Hkv, G, ctx, rows, tree=True, S=S, pad=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hd,ps,Hkv,G,ctx,rows", [
    (128, 64, 2, 4, [0], [130]),                     # a prompt on its own
    (128, 16, 1, 3, [70, 0, 5], [200, 17, 90]),
    (64, 32, 1, 2, [129, 257], [150, 64]),
    (128, 128, 1, 8, [900], [77]),
])
def test_causal_chunks(kind, hd, ps, Hkv, G, ctx, rows):
    run(np.random.default_rng(ctx[0] + 7), kind, hd, ps, Hkv, G, ctx, rows)


@pytest.mark.parametrize("kind", KINDS)
def test_ranges_behind_what_a_causal_block_sees(kind):
    """A prompt cut into key ranges: its first blocks of rows see none of the last ranges' keys, and
    those ranges contribute nothing to them."""
    rng = np.random.default_rng(17)
    cache, _ = run(rng, kind, 128, 64, 1, 8, [0], [1000], pad=2)
    assert eb.kv_attention_workspace(cache, 8, 1002, 1, 1000, 1000) > 0      # (several ranges, not joined)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ctx", [0, 50])
def test_rows_that_see_nothing(kind, ctx):
    """Mask rows of zeros: without a context zeros and -inf, with one the context alone."""
    rng = np.random.default_rng(3)
    mask = np.zeros((1, 9, 9), np.uint8)
    mask[0, 4, :3] = 1
    run(rng, kind, 128, 16, 2, 4, [ctx], [9], mask=mask)


@pytest.mark.parametrize("kind", KINDS)
def test_sharp_and_scaled_scores(kind):
    """Scores of hundreds (one key takes all), a given scale, a bound larger than the lengths."""
    run(np.random.default_rng(4), kind, 128, 32, 2, 4, [700, 10], [3, 2], qscale=40.0, max_len=4096)
    run(np.random.default_rng(5), kind, 64, 32, 2, 4, [700, 10], [3, 2], scale=0.01)
    run(np.random.default_rng(6), kind, 128, 32, 1, 4, [300], [2], qscale=1e-18)


@pytest.mark.parametrize("vg", [1e30, 1e-30])
@pytest.mark.parametrize("G,rows,ctx", [(4, 1, 60000), (20, 1, 20000), (4, 61, 12000), (4, 1, 300)])
def test_extreme_global_factors_of_the_values(vg, G, rows, ctx):
    """Values of 2688 (code 6, scale 448) times the largest and smallest factor: the same finite
    answer however the keys are cut into ranges."""
    rng = np.random.default_rng(18)
    cache, held = make_cache(rng, "f4", 128, 64, 1, [ctx + rows], k_global=1.0, v_global=vg)
    vg32 = float(np.float32(vg))
    sign = np.where(rng.random((1, 1, 128)) < 0.2, -1.0, 1.0)
    code = np.broadcast_to(np.where(sign > 0, 7, 15), (ctx + rows, 1, 128)).astype(np.uint8)
    t = np.arange(ctx + rows)
    pg, r = cache.page_table.cpu().numpy()[0, t // 64], t % 64
    v, vs = cache.v.cpu().numpy(), cache.v_scale.cpu().numpy()
    v[pg, :, r], vs[pg, :, r] = code[..., 0::2] | (code[..., 1::2] << 4), 0x7E          # 0x7e: 448
    cache.v.copy_(dev(v)), cache.v_scale.copy_(dev(vs))
    V = np.broadcast_to(sign * 2688 * vg32, (ctx + rows, 1, 128))
    q = K.bf16(rng.standard_normal((rows, G, 128)))
    out, lse = eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu([rows])), dev(np.array([ctx], np.int32)), max_rows=rows,
                               max_len=ctx + rows, lse=True)
    assert cache.check() == 0
    ref = K.attention(q, held[0][0], V, see_matrix(ctx, rows), 128 ** -0.5)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, 128)


@pytest.mark.parametrize("kg,size", [(1e-30, 0.0), (1e-12, 0.0), (1e30, 1e15)])
@pytest.mark.parametrize("G,rows", [(4, 1), (4, 2), (20, 3), (8, 40)])
def test_score_factors_that_leave_fp32(kg, size, G, rows):
    """A zero query over a small factor of the keys, a large query over zero codes and a large factor:
    every score is 0, and the keys a row does not see stay out of it."""
    rng = np.random.default_rng(19)
    ctx = 150
    cache, held = make_cache(rng, "f4", 64, 16, 1, [ctx + rows], k_global=kg)
    if size:
        cache.k.zero_()
    q = K.bf16(np.full((rows, G, 64), size))
    out, lse = eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu([rows])), dev(np.array([ctx], np.int32)), max_rows=rows,
                               max_len=ctx + rows, lse=True)
    assert cache.check() == 0
    ref = K.attention(q * 0, held[0][0] * 0, held[0][1], see_matrix(ctx, rows), 0.125)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, 64)


def test_largest_scale():
    """A scale whose product with log2(e) passes fp32, over zero queries: equal weights."""
    rng = np.random.default_rng(20)
    cache, held = make_cache(rng, "bf16", 64, 16, 1, [70])
    q = np.zeros((3, 4, 64))
    out, lse = eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu([3])), dev(np.array([67], np.int32)), max_rows=3, max_len=70,
                               scale=3e38, lse=True)
    ref = K.attention(q, held[0][0] * 0, held[0][1], see_matrix(67, 3), 1.0)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, 64)


@pytest.mark.parametrize("kind,hd,G,ctx,rows,p_step", [
    ("bf16", 128, 4, 900, 3, 2.0 ** -16), ("bf16", 64, 16, 3000, 8, 2.0 ** -16),    # one query tile: hi + lo
    ("bf16", 128, 8, 900, 40, 2.0 ** -8),                                           # two: 8 bits
    ("f4", 128, 4, 900, 3, 2.0 ** -11), ("f4", 128, 2, 900, 2, 2.0 ** -11), ("f4", 64, 8, 700, 40, 2.0 ** -11)])
def test_bits_of_the_probabilities(kind, hd, G, ctx, rows, p_step):
    """The second product's probabilities have the bits that the header states: hi + lo parts of 8 are
    off by 2^-8 of the lower part, 2^-16 of p; fp16 by 2^-11 (and 2^-32 of the largest where it is
    subnormal); one bf16 by 2^-8.  The rest of the bound is the file's."""
    rng = np.random.default_rng(23)
    cache, held = make_cache(rng, kind, hd, 32, 2, [ctx + rows])
    q = K.bf16(rng.standard_normal((rows, 2 * G, hd)))
    out = eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu([rows])), dev(np.array([ctx], np.int32)), max_rows=rows,
                          max_len=ctx + rows).double().cpu().numpy()
    o, _, mag, qk, vsum = K.attention(q, held[0][0], held[0][1], see_matrix(ctx, rows), hd ** -0.5)
    eps = 2 * ((hd + 4) * 2.0 ** -24 * qk + 2.0 ** -21 * (1 + qk))[..., None] + (hd + 128) * 2.0 ** -24
    tol = (p_step + eps) * mag + 2.0 ** -8 * np.abs(o) + 2.0 ** -32 * vsum + 1e-30
    assert (np.abs(out - o) <= tol).all(), float((np.abs(out - o) / tol).max())


def test_non_finite_values_in_masked_keys():
    """Infinite and NaN keys and values of rows that a row's mask hides do not reach it; a row
    that sees them gets what the sums give."""
    rng = np.random.default_rng(8)
    ctx, R, S = 70, 6, 6
    cache, held = make_cache(rng, "bf16", 128, 16, 1, [ctx + R])
    mask = np.eye(S, dtype=np.uint8)[None]
    k, v = (x.clone() for x in (cache.k, cache.v))
    tab = cache.page_table.cpu().numpy()
    def put(t, i, val):
        pg, r = int(tab[0, (ctx + i) // 16]), (ctx + i) % 16
        t[pg, 0, r, 5] = val
    put(cache.v, 1, float("nan"))
    put(cache.v, 2, float("inf"))
    put(cache.k, 3, float("nan"))
    q = K.bf16(rng.standard_normal((R, 4, 128)))
    out, lse = eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu([R])), dev(np.array([ctx], np.int32)), max_rows=R,
                               max_len=ctx + R, mask=dev(mask), lse=True)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref = K.attention(q, held[0][0], held[0][1], see_matrix(ctx, R, mask[0]), 128 ** -0.5)
    for i in (0, 4, 5):
        check(o[i:i + 1], l[i:i + 1], tuple(x[i:i + 1] for x in ref), 128)
    assert np.isnan(o[1, :, 5]).all() and np.isfinite(np.delete(o[1], 5, 1)).all()
    assert np.isinf(o[2, :, 5]).all() and np.isfinite(np.delete(o[2], 5, 1)).all()
    assert np.isnan(o[3]).all() and np.isnan(l[3]).all()
    # a NaN query: its own row only
    cache.k.copy_(k)
    cache.v.copy_(v)
    qn = q.copy()
    qn[2, 1, 7] = np.nan
    out = eb.kv_attention(cache, dev(qn, torch.bfloat16), dev(cu([R])), dev(np.array([ctx], np.int32)), max_rows=R,
                          max_len=ctx + R, mask=dev(mask)).double().cpu().numpy()
    assert np.isnan(out[2, 1]).all() and np.isfinite(np.delete(out.reshape(R * 4, 128), 2 * 4 + 1, 0)).all()


@pytest.mark.parametrize("hd,G,rows,ctx,pages", [
    (128, 4, 1, 100, 16),                    # one range
    (64, 4, 1, 1500, 64),                    # ranges of a cluster
    (128, 5, 3, 30000, 64),                  # ranges that the combine kernel joins
    (128, 8, 40, 700, 32), (64, 16, 20, 260, 128)])   # two query tiles
def test_visible_non_finite_values_in_cached_keys(hd, G, rows, ctx, pages):
    """An infinity or a NaN among the cached values reaches its own dim of every row, as the sum has
    it, and nothing else."""
    rng = np.random.default_rng(21)
    cache, held = make_cache(rng, "bf16", hd, pages, 1, [ctx + rows])
    tab = cache.page_table.cpu().numpy()
    kk, vv = held[0]
    for key, dim, val in ((3, 5, np.inf), (ctx // 2, 17, -np.inf), (ctx - 1, 30, np.nan), (1, 63, np.inf), (2, 63, -np.inf)):
        cache.v[tab[0, key // pages], 0, key % pages, dim] = float(val)
        vv[key, 0, dim] = 0.0                                      # (the other dims' reference)
    q = K.bf16(rng.standard_normal((rows, G, hd)))
    mask = np.tril(np.ones((rows, rows), np.uint8))[None]
    for m in (None, dev(mask)):
        out, lse = eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu([rows])), dev(np.array([ctx], np.int32)), max_rows=rows,
                                   max_len=ctx + rows, mask=m, lse=True)
        assert cache.check() == 0
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (o[..., 5] == np.inf).all() and (o[..., 17] == -np.inf).all() and np.isnan(o[..., [30, 63]]).all()
        ref = K.attention(q, kk, vv, see_matrix(ctx, rows), hd ** -0.5)
        rest = np.delete(np.arange(hd), [5, 17, 30, 63])
        check(o[..., rest], l, (ref[0][..., rest], ref[1], ref[2][..., rest], ref[3], ref[4][..., rest]), hd)


def test_a_nan_query_costs_no_second_pass():
    """NaN queries give NaN rows, in about the time of any others: their sums are not formed again
    (a walk of one thread over 20,000 keys would take some hundred times the call)."""
    rng = np.random.default_rng(22)
    ctx, R, G = 20000, 61, 8
    cache, _ = make_cache(rng, "bf16", 128, 64, 1, [ctx + R], poison=False)
    q = torch.randn(R, G, 128, device="cuda").to(torch.bfloat16)
    bad = q.clone()
    bad[::7, 3, 9] = float("nan")
    args = (dev(cu([R])), dev(np.array([ctx], np.int32)))
    def timed(x):
        best = float("inf")
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            o = eb.kv_attention(cache, x, *args, max_rows=R, max_len=ctx + R)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best, o
    t0, good = timed(q)
    t1, o = timed(bad)
    assert torch.isnan(o[::7, 3]).all()
    keep = torch.ones(R, G, dtype=torch.bool, device="cuda")
    keep[::7, 3] = False
    assert torch.equal(o[keep], good[keep])
    assert t1 < 5 * t0 + 0.2, (t0, t1)


@pytest.mark.parametrize("kind", KINDS)
def test_strided_rows_graph_and_streams(kind):
    """q and out as slices of wider rows; the same call replayed from a CUDA graph after the cache
    and the lengths changed, and run on another stream: bit-equal results."""
    rng = np.random.default_rng(9)
    ctx, rows, H, G = [400, 90], [5, 3], 2, 4
    cache, held = make_cache(rng, kind, 128, 64, H, [c + r for c, r in zip(ctx, rows)], room=[1000, 1000])
    wide = torch.randn(8, H * G * 128 + 256, device="cuda").to(torch.bfloat16)
    q = wide[:, 128:128 + H * G * 128].unflatten(1, (H * G, 128))
    outw = torch.zeros(8, H * G * 128 + 64, dtype=torch.bfloat16, device="cuda")
    out = outw[:, :H * G * 128].unflatten(1, (H * G, 128))
    c, n = dev(cu(rows)), dev(np.array(ctx, np.int32))
    need = eb.kv_attention_workspace(cache, H * G, 8, 2, 5, 1000)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    call = lambda **kw: eb.kv_attention(cache, q, c, n, max_rows=5, max_len=1000, workspace=ws, **kw)  # noqa: E731
    plain = call().clone()
    call(out=out)
    assert torch.equal(out, plain) and (outw[:, H * G * 128:] == 0).all()
    at = 0
    qd = q.double().cpu().numpy()
    lse = call(lse=True)[1].double().cpu().numpy()
    for b, r in enumerate(rows):
        ref = K.attention(qd[at:at + r], held[b][0], held[b][1], see_matrix(ctx[b], r), 128 ** -0.5)
        check(plain[at:at + r].double().cpu().numpy(), lse[at:at + r], ref, 128)
        at += r
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, plain)
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert torch.equal(got, plain)
    gout = torch.zeros_like(plain)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=gout)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, plain)
    n -= 37                                    # the graph reads the lengths of the day
    want = call().clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, want) and not torch.equal(want, plain)
    assert cache.check() == 0


def test_bad_pages_and_lengths_are_reported():
    rng = np.random.default_rng(10)
    cache, _ = make_cache(rng, "bf16", 128, 16, 1, [40, 40])
    q = torch.randn(2, 4, 128, device="cuda").to(torch.bfloat16)
    good = cache.page_table.clone()
    args = (dev(cu([1, 1])), dev(np.array([39, 39], np.int32)))
    want = eb.kv_attention(cache, q, *args, max_rows=1, max_len=40)
    assert cache.check() == 0
    cache.page_table[0, 1] = cache.k.shape[0]
    got = eb.kv_attention(cache, q, *args, max_rows=1, max_len=40)
    with pytest.raises(eb.EagleError) as e:
        cache.check()
    assert e.value.status == eb.EAGLE_ERR_DEVICE and "0x10" in str(e.value)
    assert torch.equal(got[1], want[1])        # the other request is whole
    cache.page_table.copy_(good)
    eb.kv_attention(cache, q, args[0], dev(np.array([39, 80], np.int32)), max_rows=1, max_len=40)
    with pytest.raises(eb.EagleError) as e:
        cache.check()
    assert "0x2" in str(e.value)
    assert cache.check() == 0


def test_pool_of_more_than_2_31_elements():
    """Pages whose offsets pass 32 bits."""
    ps, hd, H = 64, 128, 2
    P = 2 ** 31 // (ps * hd * H) + 600
    rng = np.random.default_rng(11)
    for kind in KINDS:
        w, dt = (hd, torch.bfloat16) if kind == "bf16" else (hd // 2, torch.uint8)
        PP = P if kind == "bf16" else 2 * P
        k = torch.zeros(PP, H, ps, w, dtype=dt, device="cuda")
        v = torch.zeros_like(k)
        small, held = make_cache(rng, kind, hd, ps, H, [500])
        n = small.k.shape[0]
        table = small.page_table + (PP - n)
        k[PP - n:], v[PP - n:] = small.k, small.v
        sc = []
        if kind == "f4":
            for s in (small.k_scale, small.v_scale):
                t = torch.zeros(PP, H, ps, hd // 16, dtype=torch.uint8, device="cuda")
                t[PP - n:] = s
                sc.append(t)
        cache = eb.KVCache(k, v, table.contiguous(), *sc, **({} if kind == "bf16" else {"k_global": 1.0, "v_global": 0.5}))
        q = torch.randn(1, 8, hd, device="cuda").to(torch.bfloat16)
        args = (q, dev(cu([1])), dev(np.array([499], np.int32)))
        assert torch.equal(eb.kv_attention(cache, *args, max_rows=1, max_len=500),
                           eb.kv_attention(small, *args, max_rows=1, max_len=500))
        assert cache.check() == 0
        del k, v, sc, cache
