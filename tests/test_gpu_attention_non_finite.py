"""Values that are not finite, in keys whose weight is far below the row's largest (e^-200 and less: 0
in 32 bits).  Dim 0 of every key is +16 or -16 and of every query +8 or -8, the scale is 1, so that a
row's keys lie 256 apart in the exponent, and half of the rows have the low keys on top.  e^-256 is
not 0 in 64 bits, so numpy's sums are the formula's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb
from oracle import kv_oracle as K
from kv_util import cu, dev, make_cache, see_matrix
from test_gpu_kv_attention import check, lib  # noqa: F401

INF, NAN = np.inf, np.nan
# dims of non-finite values: of a key on the +16 side, of one on the -16 side
ODD = [(5, INF, 0.0), (9, 0.0, -INF), (17, -INF, 0.0), (30, 0.0, NAN), (33, NAN, 0.0), (40, INF, -INF), (47, -INF, -INF), (63, 0.0, INF)]


def steep(rng, cache, held, sides):
    """Sets dim 0 of every held key to 16 times its side (per request, [n] of +1 / -1) and small other dims."""
    ps = cache.k.shape[2]
    tab = cache.page_table.cpu().numpy()
    for b, ((kk, vv), side) in enumerate(zip(held, sides)):
        n = len(side)
        if not n:
            continue
        kk *= 2.0 ** -4
        kk[:, :, 0] = 16.0 * np.asarray(side)[:, None]
        t = np.arange(n)
        cache.k[torch.from_numpy(tab[b, t // ps]).long().cuda(), :, torch.from_numpy(t % ps).long().cuda()] = dev(kk, torch.bfloat16)


def put(cache, held, b, key, dim, val):
    if val == 0.0:
        return
    ps = cache.k.shape[2]
    cache.v[int(cache.page_table[b, key // ps]), :, key % ps, dim] = float(val)
    held[b][1][key, :, dim] = val


def odd_values(cache, held, b, high, low):
    for dim, h, lo in ODD:
        put(cache, held, b, high, dim, h)
        put(cache, held, b, low, dim, lo)


def queries(rng, N, Hq, hd):
    q = K.bf16(rng.standard_normal((N, Hq, hd)))
    q[..., 0] = 8.0 * np.where((np.arange(N)[:, None] + np.arange(Hq)) % 2, 1.0, -1.0)
    return q


def compare(out, lse, q, keys, see, hd, exact=True):
    """Rows q [r, Hq, hd] over keys (k, v) [n, Hkv, hd]: what is finite within the bound of finite inputs,
    the rest not finite (with `exact`: the infinity or NaN of the sum)."""
    k, v = keys
    finite = np.where(np.isfinite(v), v, 0.0)
    ref = K.attention(q, k, finite, see, 1.0)
    G = q.shape[1] // k.shape[1]
    with np.errstate(invalid="ignore"):
        odd = np.zeros(ref[0].shape)
        for j in np.unique(np.argwhere(~np.isfinite(v))[:, 0]):
            w = np.where(np.isfinite(v[j]), 0.0, v[j])
            odd += np.where(see[:, j][:, None, None], np.repeat(w, G, 0)[None], 0.0)   # (its weight is above 0)
    some = odd == 0.0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    check(np.where(some, o, 0.0), l, (np.where(some, ref[0], 0.0), *ref[1:]), hd)
    if exact:
        assert np.array_equal(o[~some], odd[~some], equal_nan=True), (o[~some][:8], odd[~some][:8])
    else:
        assert not np.isfinite(o[~some]).any()


CROSS = [
    # hd, ps, Hkv, G, lens, rows: little to read by ranges (joined in a cluster, in a second kernel), ...
    (128, 64, 1, 4, [1500], [2]), (64, 32, 2, 1, [700], [3]), (128, 64, 1, 4, [60000], [2]),
    # ... dealt out in line, few query vectors
    (128, 64, 8, 4, [700 + 31 * i for i in range(20)], [1] * 20), (64, 32, 16, 1, [9000, 300, 2000], [1, 2, 1]),
    # ... and many: one block or several, both groups on the same vectors or not, one CTA and several
    (128, 64, 1, 4, [300], [20]), (128, 64, 1, 5, [5000, 129], [13, 30]), (64, 128, 1, 8, [9000], [40]), (128, 16, 2, 2, [2000, 500], [150, 90]),
    (128, 64, 1, 8, [130, 257], [70, 33]),
]


def cross_case(hd, ps, Hkv, G, lens, rows, first):
    """first: the side of the first keys (the other side's are the last); 0: of either side in turn."""
    rng = np.random.default_rng(hd + sum(lens))
    cache, held = make_cache(rng, "bf16", hd, ps, Hkv, lens)
    sides = [np.where(np.arange(n) < n // 2, first, -first) if first else np.where(rng.random(n) < 0.5, 1, -1) for n in lens]
    steep(rng, cache, held, sides)
    for b, n in enumerate(lens):
        at = [n // 9, n - 1 - n // 7]
        if first == 0:
            at = [int(rng.choice(np.flatnonzero(sides[b] == s))) for s in (1, -1)]
        odd_values(cache, held, b, *(at if first >= 0 else at[::-1]))
    q = queries(rng, sum(rows), Hkv * G, hd)
    out, lse = eb.kv_cross_attention(cache, dev(q, torch.bfloat16), dev(cu(rows)), dev(np.array(lens, np.int32)), max_rows=max(rows),
                                     max_len=max(lens), scale=1.0, lse=True)
    assert cache.check() == 0
    c = cu(rows)
    for b, (n, r) in enumerate(zip(lens, rows)):
        s = slice(c[b], c[b + 1])
        yield out[s], lse[s], q[s], held[b], np.ones((r, n), bool)


@pytest.mark.parametrize("first", [1, -1])
@pytest.mark.parametrize("hd,ps,Hkv,G,lens,rows", CROSS)
def test_far_values_reach_every_row(hd, ps, Hkv, G, lens, rows, first):
    for out, lse, q, keys, see in cross_case(hd, ps, Hkv, G, lens, rows, first):
        compare(out, lse, q, keys, see, hd, exact=False)


@pytest.mark.parametrize("first", [1, -1, 0])
@pytest.mark.parametrize("hd,ps,Hkv,G,lens,rows", CROSS)
def test_far_infinities_are_the_formulas(hd, ps, Hkv, G, lens, rows, first):
    """The sum's infinity, or NaN where it meets the other or a NaN: also where p is 0 in 32 bits."""
    for out, lse, q, keys, see in cross_case(hd, ps, Hkv, G, lens, rows, first):
        compare(out, lse, q, keys, see, hd)


def shared_case(hd, Hkv, G, plens, groups, ctx, rows, side):
    """side: of the prefix's keys (the own keys have the other)."""
    rng = np.random.default_rng(sum(rows) + hd)
    prefix, pre = make_cache(rng, "bf16", hd, 64, Hkv, plens)
    cache, own = make_cache(rng, "bf16", hd, 32, Hkv, [c + r for c, r in zip(ctx, rows)])
    steep(rng, prefix, pre, [np.full(n, side) for n in plens])
    steep(rng, cache, own, [np.full(c + r, -side) for c, r in zip(ctx, rows)])
    owner = [next(g for g in range(len(plens)) if groups[g] <= b < groups[g + 1]) for b in range(len(rows))]
    for g, n in enumerate(plens):
        for dim, h, lo in ODD:
            put(prefix, pre, g, n // 3, dim, h if side > 0 else lo)
    for b, c in enumerate(ctx):
        for dim, h, lo in ODD:
            put(cache, own, b, c // 2, dim, lo if side > 0 else h)
    q = queries(rng, sum(rows), Hkv * G, hd)
    c = cu(rows)
    ints = lambda x: dev(np.array(x, np.int32))  # noqa: E731
    out, lse = eb.kv_shared_attention(prefix, ints(groups), ints(plens), cache, dev(q, torch.bfloat16), dev(c), ints(ctx),
                                      max_group_rows=max(c[b] - c[a] for a, b in zip(groups[:-1], groups[1:])), max_prefix=max(plens),
                                      max_rows=max(rows), max_len=max(x + r for x, r in zip(ctx, rows)), scale=1.0, lse=True)
    assert cache.check() == 0 and prefix.check() == 0
    for b, r in enumerate(rows):
        keys = tuple(np.concatenate([x, y]) for x, y in zip(pre[owner[b]], own[b]))
        see = np.ones((r, len(keys[0])), bool)
        see[:, plens[owner[b]]:] = see_matrix(ctx[b], r)
        yield out[c[b]:c[b + 1]], lse[c[b]:c[b + 1]], q[c[b]:c[b + 1]], keys, see


SHARED = [
    (128, 2, 4, [500], [0, 2], [30, 9], [1, 1]),                       # ranges and their join
    (64, 2, 2, [4000, 300], [0, 6, 9], [40 + i for i in range(9)], [1] * 9),
    (128, 8, 4, [3000], [0, 40], [300 + i for i in range(40)], [1] * 40),   # own keys in line, prefix wide
    (128, 8, 4, [700] * 40, list(range(41)), [300 + i for i in range(40)], [1] * 40),   # both in line
    (128, 2, 4, [9000], [0, 3], [70, 200, 5], [30, 40, 7]),            # prefix wide and cut
    (64, 1, 8, [200, 300], [0, 1, 3], [10, 300, 64], [50, 90, 20]),
]


@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("hd,Hkv,G,plens,groups,ctx,rows", SHARED)
def test_far_values_of_prefix_or_own_keys_reach_every_row(hd, Hkv, G, plens, groups, ctx, rows, side):
    for out, lse, q, keys, see in shared_case(hd, Hkv, G, plens, groups, ctx, rows, side):
        compare(out, lse, q, keys, see, hd, exact=False)


@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("hd,Hkv,G,plens,groups,ctx,rows", SHARED)
def test_far_infinities_of_prefix_or_own_keys_are_the_formulas(hd, Hkv, G, plens, groups, ctx, rows, side):
    for out, lse, q, keys, see in shared_case(hd, Hkv, G, plens, groups, ctx, rows, side):
        compare(out, lse, q, keys, see, hd)


@pytest.mark.parametrize("first", [1, -1, 0])
@pytest.mark.parametrize("hd,G,ctx,rows", [(128, 4, [900, 130], [1, 2]), (64, 2, [40000], [1]), (128, 8, [700, 60], [30, 64]), (64, 4, [0, 3000], [200, 10])])
def test_the_steps_own_attention_too(hd, G, ctx, rows, first):
    """eagle_kv_attention, whose rows are keys of the sequence: an infinity in keys that a row does not see
    leaves nothing, in the others the sum's."""
    rng = np.random.default_rng(hd + G)
    lens = [c + r for c, r in zip(ctx, rows)]
    cache, held = make_cache(rng, "bf16", hd, 64, 1, lens)
    sides = [np.where(np.arange(n) < n // 2, first, -first) if first else np.where(rng.random(n) < 0.5, 1, -1) for n in lens]
    steep(rng, cache, held, sides)
    for b, n in enumerate(lens):
        for key in (n // 3, n - 1):                  # (the last: the last row's alone)
            for dim, h, lo in ODD:
                put(cache, held, b, key, dim, h if sides[b][key] > 0 else lo)
    q = queries(rng, sum(rows), G, hd)
    out, lse = eb.kv_attention(cache, dev(q, torch.bfloat16), dev(cu(rows)), dev(np.array(ctx, np.int32)), max_rows=max(rows), max_len=max(lens),
                               scale=1.0, lse=True)
    assert cache.check() == 0
    at = cu(rows)
    for b, r in enumerate(rows):
        s = slice(at[b], at[b + 1])
        compare(out[s], lse[s], q[s], held[b], see_matrix(ctx[b], r), hd)


@pytest.mark.parametrize("rows", [[1] * 20, [40] * 20])
def test_an_infinity_at_a_key_of_no_weight(rows):
    """A key of score -infinity has a weight of 0, and 0 times an infinite value is NaN; the other dims
    are as without that key."""
    rng = np.random.default_rng(4)
    lens, hd, Hkv, G = [300 + 41 * i for i in range(len(rows))], 128, 8, 1
    cache, held = make_cache(rng, "bf16", hd, 64, Hkv, lens)
    q = K.bf16(np.abs(K.bf16(rng.standard_normal((sum(rows), Hkv * G, hd)))) + 0.5)
    for b in range(len(lens)):
        cache.k[int(cache.page_table[b, 1]), :, 7, 11] = -INF
        cache.v[int(cache.page_table[b, 1]), :, 7, 20] = INF
    out, lse = eb.kv_cross_attention(cache, dev(q, torch.bfloat16), dev(cu(rows)), dev(np.array(lens, np.int32)), max_rows=max(rows),
                                     max_len=max(lens), lse=True)
    o, l, at = out.double().cpu().numpy(), lse.double().cpu().numpy(), cu(rows)
    assert np.isnan(o[..., 20]).all()
    for b, r in enumerate(rows):
        s, keep = slice(at[b], at[b + 1]), np.delete(np.arange(lens[b]), 64 + 7)
        ref = K.attention(q[s], held[b][0][keep], held[b][1][keep], np.ones((r, len(keep)), bool), hd ** -0.5)
        rest = np.delete(np.arange(hd), 20)
        check(o[s][..., rest], l[s], (ref[0][..., rest], ref[1], ref[2][..., rest], ref[3], ref[4][..., rest]), hd)


def test_a_nan_key_reaches_every_row_from_any_part():
    """Its score is NaN, however far the other keys of its part lie below: out and lse are NaN."""
    for Hkv, G, lens, rows in ((1, 4, [60000], [2]), (8, 4, [700 + 31 * i for i in range(20)], [1] * 20), (1, 4, [9000], [40]), (2, 2, [2000], [150])):
        rng = np.random.default_rng(3)
        for first in (1, -1):
            cache, held = make_cache(rng, "bf16", 128, 64, Hkv, lens)
            steep(rng, cache, held, [np.where(np.arange(n) < n // 2, first, -first) for n in lens])
            for key in (lens[0] // 9, lens[0] - 1):
                page = int(cache.page_table[0, key // 64])
                keep = cache.k[page, :, key % 64, 11].clone()
                cache.k[page, :, key % 64, 11] = NAN
                q = queries(rng, sum(rows), Hkv * G, 128)
                out, lse = eb.kv_cross_attention(cache, dev(q, torch.bfloat16), dev(cu(rows)), dev(np.array(lens, np.int32)), max_rows=max(rows),
                                                 max_len=max(lens), scale=1.0, lse=True)
                assert torch.isnan(out[:rows[0]]).all() and torch.isnan(lse[:rows[0]]).all()
                assert torch.isfinite(out[rows[0]:]).all()
                cache.k[page, :, key % 64, 11] = keep


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_merge_of_far_parts(dt):
    """What is not finite in a part reaches the result from any lse but -infinity."""
    o = [torch.ones(1, 2, 16, dtype=dt, device="cuda") for _ in range(3)]
    for i, x in enumerate((float("inf"), -float("inf"), float("nan"))):
        o[1][..., i] = x
    o[2][..., 3], o[0][..., 4], o[1][..., 4] = float("inf"), float("inf"), -float("inf")
    for far in (-90.0, -104.0, -110.0, -1e6):
        l = [torch.full((1, 2), x, device="cuda") for x in (3.0, far, -float("inf"))]
        got, lse = eb.attention_merge(o, l, lse=True)
        x = got.double().cpu().numpy()[0, 0]
        assert x[0] == INF and x[1] == -INF and np.isnan(x[2]) and np.isnan(x[4]), far
        assert (np.delete(x, [0, 1, 2, 4]) == 1.0).all() and (lse == 3.0).all()   # (the part of lse -inf adds nothing)
    l = [torch.full((1, 2), x, device="cuda") for x in (float("inf"), 3.0, -float("inf"))]
    x = eb.attention_merge(o, l).double().cpu().numpy()[0, 0]
    assert x[0] == INF and x[1] == -INF and np.isnan(x[2]) and np.isnan(x[4]) and x[3] == 1.0
