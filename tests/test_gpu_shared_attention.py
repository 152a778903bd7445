"""GPU parity of eagle_kv_shared_attention and eagle_attention_merge against float64: shared
attention is one softmax over the prefix's keys and the request's own, in test_gpu_kv_attention's
bound (the join's factors and sums add a few 2^-22 to its eps_e)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb
from oracle import kv_oracle as K
from kv_util import cu, dev, make_cache, pages, see_matrix, tree_masks
from test_gpu_kv_attention import check, lib  # noqa: F401


def reference(q, pre, groups, own, ctx, rows, mask, hd, scale=0.0):
    parts, at = [], 0
    for b, r in enumerate(rows):
        g = next(i for i in range(len(groups) - 1) if groups[i] <= b < groups[i + 1])
        k, v = (np.concatenate([x, y]) for x, y in zip(pre[g], own[b]))
        see = np.ones((r, k.shape[0]), bool)
        see[:, pre[g][0].shape[0]:] = see_matrix(ctx[b], r, None if mask is None else mask[b])
        parts.append(K.attention(q[at:at + r], k, v, see, scale or hd ** -0.5))
        at += r
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(5))


def run(rng, kinds, hd, ps, Hkv, G, plens, groups, ctx, rows, tree=False, S=None, mask=None, pad=0, scale=0.0, loose=False, **kw):
    prefix, pre = make_cache(rng, kinds[0], hd, ps[0], Hkv, plens)
    held = [c + r for c, r in zip(ctx, rows)]
    cache, own = make_cache(rng, kinds[1], hd, ps[1], Hkv, held, v_global=0.25)
    N = sum(rows) + pad
    q = K.bf16(rng.standard_normal((N, Hkv * G, hd)))
    if tree and mask is None:
        mask = tree_masks(rng, len(ctx), S or max(max(rows), 1), rows)
    grows = [sum(rows[a:b]) for a, b in zip(groups[:-1], groups[1:])]
    more = 3 if loose else 1
    out = torch.full((N, Hkv * G, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hkv * G), 7.0, device="cuda")
    args = (prefix, dev(np.array(groups, np.int32)), dev(np.array(plens, np.int32)), cache, dev(q, torch.bfloat16), dev(cu(rows)),
            dev(np.array(ctx, np.int32)))
    sizes = dict(max_group_rows=more * max(max(grows), 1), max_prefix=more * max(max(plens), 1), max_rows=more * max(max(rows), 1) if mask is None else max(rows),
                 max_len=more * max(max(held), 1), mask=None if mask is None else dev(mask), scale=scale)
    eb.kv_shared_attention(*args, **sizes, out=out, lse=lse, **kw)
    assert cache.check() == 0 and prefix.check() == 0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = sum(rows)
    check(o[:n], l[:n], reference(q, pre, groups, own, ctx, rows, mask, hd, scale), hd)
    assert (o[n:] == 7.0).all() and (l[n:] == 7.0).all()   # rows of no request
    return args, sizes, out, lse


KINDS = [("bf16", "bf16"), ("f4", "bf16"), ("bf16", "f4"), ("f4", "f4")]


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("hd,ps,Hkv,G,plens,groups,ctx,rows", [
    (128, (64, 64), 2, 4, [1], [0, 1], [0], [1]),
    (128, (64, 16), 2, 4, [0], [0, 2], [0, 5], [1, 1]),             # no prefix
    (64, (16, 32), 1, 1, [17, 300], [0, 3, 5], [0, 1, 40, 15, 16], [1, 1, 1, 1, 1]),
    (128, (64, 64), 2, 4, [700], [0, 2], [30, 4], [1, 1]),
    (128, (32, 128), 2, 5, [129, 0, 1000], [0, 1, 3, 4], [70, 0, 128, 600], [1, 1, 1, 1]),
    (64, (64, 64), 4, 2, [2000], [0, 6], [3, 5, 0, 100, 1, 64], [1, 1, 0, 1, 1, 1]),   # a request without rows
    (128, (64, 64), 1, 8, [9000], [0, 3], [20, 4000, 1], [1, 1, 1]),        # ranges of both
    (128, (64, 64), 8, 4, [4100, 257], [0, 20, 40], list(range(40)), [1] * 40),
    (64, (128, 16), 1, 64, [130], [0, 2], [0, 9], [1, 1]),
    (128, (64, 64), 2, 2, [300, 40, 60], [0, 0, 2, 2], [9, 8], [1, 1]),     # groups without requests
    (128, (128, 128), 1, 3, [500], [0, 5], [9, 800, 0, 127, 128], [1] * 5),  # odd numbers of rows and heads
    (64, (32, 64), 3, 5, [70, 4000], [0, 1, 3], [63, 64, 900], [1, 1, 1]),
    (128, (16, 16), 2, 8, [64, 65], [0, 30, 60], [(37 * i) % 700 for i in range(60)], [1] * 60),
])
def test_single_tokens(kinds, hd, ps, Hkv, G, plens, groups, ctx, rows):
    run(np.random.default_rng(hd + G + sum(plens)), kinds, hd, ps, Hkv, G, plens, groups, ctx, rows, pad=2)


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("hd,ps,Hkv,G,plens,groups,ctx,rows,tree", [
    (128, (64, 64), 2, 4, [500], [0, 3], [40, 0, 64], [61, 7, 33], True),
    (128, (16, 64), 1, 4, [333, 128], [0, 2, 4], [0, 100, 31, 5], [13, 64, 1, 20], True),
    (64, (32, 32), 2, 3, [97], [0, 2], [31, 129], [64, 33], True),
    (128, (64, 128), 1, 8, [260], [0, 2], [0, 0], [150, 77], False),
    (64, (128, 64), 1, 2, [1, 0], [0, 1, 2], [300, 70], [257, 90], False),
    (128, (64, 64), 1, 4, [6000], [0, 4], [10, 20, 30, 1000], [40, 40, 1, 40], False),   # prefix ranges
])
def test_trees_and_chunks(kinds, hd, ps, Hkv, G, plens, groups, ctx, rows, tree):
    run(np.random.default_rng(hd + sum(rows)), kinds, hd, ps, Hkv, G, plens, groups, ctx, rows, tree=tree, S=64 if tree else None, pad=1)


@pytest.mark.parametrize("kinds", KINDS)
def test_masks_that_leave_the_own_part_empty(kinds):
    """Rows that see none of the step's rows and have no own keys: the prefix alone; without one too,
    zeros and -inf."""
    rng = np.random.default_rng(8)
    rows, ctx = [5, 4], [0, 0]
    mask = tree_masks(rng, 2, 8, rows)
    mask[0, 2, :] = 0
    mask[1, 1, :] = 0
    _, _, out, lse = run(rng, kinds, 128, (64, 64), 2, 4, [200, 0], [0, 1, 2], ctx, rows, mask=mask)
    assert (out[6] == 0).all() and (lse[6] == -float("inf")).all()
    assert torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("rows", [[1, 1, 1], [30, 1, 44]])
def test_loose_bounds_and_scale(rows):
    run(np.random.default_rng(2), ("bf16", "bf16"), 128, (64, 64), 2, 4, [400, 90], [0, 2, 3], [9, 100, 0], rows, scale=0.2, loose=True)


def test_equals_one_cache_of_all_keys():
    """A step over a shared prefix is the same step over caches that hold prefix and own keys in
    one sequence each (kv_attention), whose pages share the prefix."""
    rng = np.random.default_rng(12)
    hd, ps, Hkv, G, P, ctx, rows = 128, 64, 2, 4, 320, [64, 10, 130], [3, 1, 2]
    args, sizes, out, lse = run(rng, ("bf16", "bf16"), hd, (ps, ps), Hkv, G, [P], [0, 3], ctx, rows)
    prefix, cache = args[0], args[3]
    k, v = torch.cat([prefix.k, cache.k]), torch.cat([prefix.v, cache.v])
    own = torch.where(cache.page_table >= 0, cache.page_table + prefix.k.shape[0], -1)
    table = torch.cat([prefix.page_table[0, :P // ps].expand(3, -1), own], 1).int().contiguous()
    whole = eb.KVCache(k, v, table)
    o2, l2 = eb.kv_attention(whole, args[4], args[5], args[6] + P, max_rows=3, max_len=P + max(c + r for c, r in zip(ctx, rows)), lse=True)
    assert whole.check() == 0
    # two roundings to bf16 and each side's own bound on p: 2^-8 sum p |v| / sum p at most
    assert float((out.float() - o2.float()).abs().max()) <= 2 * (2 ** -8 * 4 + 2 ** -8 * float(o2.float().abs().max()))
    assert float((lse - l2).abs().max()) < 1e-4


def test_shared_is_cross_and_own_merged():
    """The three operators together: shared attention = merge(cross over the prefix, kv_attention over
    the own keys), up to the merge's bf16 parts."""
    rng = np.random.default_rng(13)
    args, sizes, out, lse = run(rng, ("f4", "bf16"), 128, (64, 32), 2, 4, [500, 70], [0, 2, 3], [40, 9, 200], [7, 1, 12])
    prefix, cg, pl, cache, q, c, ctx = args
    po, pl_ = eb.kv_cross_attention(prefix, q, c[cg.long()].contiguous(), pl, max_rows=12, max_len=500, lse=True)
    oo, ol = eb.kv_attention(cache, q, c, ctx, max_rows=12, max_len=300, lse=True)
    m, ml = eb.attention_merge([po, oo], [pl_, ol], lse=True)
    scale = float(torch.stack([po, oo]).float().abs().max())
    assert float((m.float() - out.float()).abs().max()) <= 4 * 2 ** -8 * scale
    assert float((ml - lse).abs().max()) < 1e-4


@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("f4", "f4")])
@pytest.mark.parametrize("rows", [[1, 1, 1], [40, 33, 61]])
def test_graph_streams_and_repeats(kinds, rows):
    """Replayed from a CUDA graph after lengths changed, on another stream at once with its own
    workspace, and again: bit-equal results."""
    rng = np.random.default_rng(9)
    args, sizes, out, lse = run(rng, kinds, 128, (64, 64), 2, 4, [1500, 300], [0, 2, 3], [100, 40, 300], rows)
    need = eb.kv_shared_attention_workspace(args[0], args[3], 8, sum(rows), 2, 3, sizes["max_group_rows"], sizes["max_prefix"], sizes["max_rows"], sizes["max_len"])
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    call = lambda **kw: eb.kv_shared_attention(*args, **sizes, **{"workspace": ws[0], **kw})  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a, b = call(stream=side, workspace=ws[1]), call()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, out)
    gout = torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=gout)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, out)
    args[2].sub_(29)                           # prefix lengths
    args[6].sub_(7)                            # own lengths
    want = call().clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, want) and not torch.equal(want, out)
    assert args[3].check() == 0


def test_a_round_of_samples_behind_one_prompt():
    """As a program uses it: a prompt appended once, three samples' tokens appended to their own
    pages at positions behind it, a step of all of them; then the accepted path of their trees is
    kept and the next step reads it.  Every step equals attention over one whole sequence."""
    rng = np.random.default_rng(14)
    hd, Hkv, G, P, B, ps = 64, 2, 4, 150, 3, 32
    rope = eb.Rope(hd)
    bf = torch.bfloat16

    def rows(n):
        return [torch.randn(n, h, hd, device="cuda").to(bf) for h in (Hkv * G, Hkv, Hkv)]
    ints = lambda x: dev(np.array(x, np.int32))  # noqa: E731
    tab_p, np_ = pages(rng, [P], ps)
    tab_o, no_ = pages(rng, [40] * B, ps)
    prefix, cache = eb.KVCache.empty(np_, ps, Hkv, hd, dev(tab_p)), eb.KVCache.empty(no_, ps, Hkv, hd, dev(tab_o))
    _, pk, pv = rows(P)
    eb.kv_append(prefix, pk, pv, ints([0, P]), ints([0]), positions=torch.arange(P, device="cuda", dtype=torch.int32), rope=rope)
    seq = [[(pk, pv, torch.arange(P, device="cuda", dtype=torch.int32))] for _ in range(B)]
    lens = ints([0] * B)
    groups, plen = ints([0, B]), ints([P])

    def step(R, mask=None, pos=None):
        N = B * R
        q, k, v = rows(N)
        positions = (lens[:, None] + P + (torch.arange(R, device="cuda") if pos is None else pos)).int().reshape(-1).contiguous()
        c = ints([R * b for b in range(B + 1)])
        qr = eb.kv_append(cache, k, v, c, lens, positions=positions, rope=rope, q=q)
        out = eb.kv_shared_attention(prefix, groups, plen, cache, qr, c, lens, max_group_rows=N, max_prefix=P, max_rows=R, max_len=40, mask=mask)
        for b in range(B):
            s = slice(b * R, (b + 1) * R)
            ks = torch.cat([x[0] for x in seq[b]] + [k[s]])
            vs = torch.cat([x[1] for x in seq[b]] + [v[s]]).double().cpu().numpy()
            at = torch.cat([x[2] for x in seq[b]] + [positions[s]])
            kr = eb.rotary(ks, at, rope).double().cpu().numpy()
            see = see_matrix(len(vs) - R, R, None if mask is None else mask[b].cpu().numpy())
            o, _, mag, qk, _ = K.attention(qr[s].double().cpu().numpy(), kr, vs, see, hd ** -0.5)
            tol = (2.0 ** -8 + 2.0 ** -14 * (1 + qk)[..., None]) * mag + 2.0 ** -8 * np.abs(o) + 1e-6
            assert (np.abs(out[s].double().cpu().numpy() - o) <= tol).all()
        return k, v, positions
    for R in (1, 1):
        k, v, p = step(R)
        for b in range(B):
            seq[b].append((k[b:b + 1], v[b:b + 1], p[b:b + 1]))
        lens = lens + 1
    parents = [-1, 0, 0, 1, 2]
    m = np.zeros((5, 5), np.uint8)
    for i, x in enumerate(parents):
        m[i] = m[x] if x >= 0 else 0
        m[i, i] = 1
    depth = torch.tensor([0, 1, 1, 2, 2], device="cuda")
    k, v, p = step(5, mask=dev(np.stack([m] * B)), pos=depth)
    paths = [[1, 3], [2], []]
    slots = np.full((B, 5), -1, np.int32)
    for b, x in enumerate(paths):
        slots[b, :len(x)] = x
        for s in [0] + x:
            seq[b].append((k[5 * b + s:5 * b + s + 1], v[5 * b + s:5 * b + s + 1], p[5 * b + s:5 * b + s + 1]))
    lens = eb.kv_accept(cache, lens, ints([len(x) for x in paths]), dev(slots))
    step(1)
    assert cache.check() == 0 and prefix.check() == 0


def test_bad_groups_are_reported():
    rng = np.random.default_rng(10)
    for rows in ([1, 1, 1], [40, 20, 30]):
        args, sizes, out, lse = run(rng, ("bf16", "bf16"), 128, (16, 16), 1, 4, [100, 60], [0, 2, 3], [9, 4, 0], rows)
        prefix, cg, pl, cache, q, c, ctx = args

        def call(groups=cg, plens=pl, **kw):
            o = torch.full_like(out, 7.0)
            eb.kv_shared_attention(prefix, groups, plens, cache, q, c, ctx, **{**sizes, "out": o, **kw})
            return o

        def flagged(bits):
            with pytest.raises(eb.EagleError) as e:
                cache.check()
            assert e.value.status == eb.EAGLE_ERR_DEVICE and bits in str(e.value)
        ints = lambda x: dev(np.array(x, np.int32))  # noqa: E731
        last = sum(rows[:2])
        o = call(ints([0, 2, 2]))                    # a request left out
        flagged("0x2")
        assert torch.equal(o[:last], out[:last]) and (o[last:] == 7.0).all()
        o = call(ints([1, 2, 3]))
        flagged("0x2")
        assert (o[:rows[0]] == 7.0).all() and torch.equal(o[last:], out[last:])
        for g in ([0, 2, 4], [0, 4, 3], [0, 2, 1], [-1, 2, 3]):
            o = call(ints(g))
            flagged("0x2")
        for n in ([101, 60], [100, -1]):
            o = call(plens=ints(n))
            flagged("0x2")
        o = call(max_group_rows=rows[0])             # rows past the bound: left as they were
        flagged("0x2")
        assert (o[rows[0]:last] == 7.0).all() and torch.isfinite(o.float()).all()
        good = prefix.page_table.clone()
        prefix.page_table[1, 2] = prefix.k.shape[0]
        o = call()
        flagged("0x10")
        assert torch.equal(o[:last], out[:last])
        prefix.page_table.copy_(good)
        assert torch.equal(call(), out) and cache.check() == 0


def test_refusals_of_the_binding():
    rng = np.random.default_rng(0)
    args, sizes, out, _ = run(rng, ("bf16", "bf16"), 64, (16, 16), 2, 2, [30], [0, 2], [3, 4], [1, 1])
    prefix, cg, pl, cache, q, c, ctx = args
    four, _ = make_cache(rng, "bf16", 64, 16, 4, [30])
    for a, kw in (((prefix, cg[:1], pl, cache, q, c, ctx), {}), ((prefix, cg.long(), pl, cache, q, c, ctx), {}),
                  ((prefix, dev(cu([1, 1])), dev(np.array([3, 3], np.int32)), cache, q, c, ctx), {}),
                  ((prefix, cg, pl, cache, q.float(), c, ctx), {}), ((four, cg, pl, cache, q, c, ctx), {}),
                  (args, dict(max_prefix=0)), (args, dict(max_group_rows=0)), (args, dict(out=q)),
                  (args, dict(mask=torch.zeros(2, 3, 3, device="cuda"))), (args, dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(eb.EagleError) as e:
            eb.kv_shared_attention(*a, **{**sizes, **kw})
        assert e.value.status == eb.EAGLE_ERR_INVALID_ARG
    assert eb.kv_shared_attention(prefix, cg, pl, cache, q[:0], c * 0, ctx, **sizes).shape == (0, 4, 64)


# ------------------------------------------------------------------------------ merge
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def merge_reference(outs, lses):
    """float64 (out, lse, sum w |o| / sum w); a part of lse -inf has no weight whatever it holds."""
    l = np.stack([x.double().cpu().numpy() for x in lses])
    o = np.stack([x.double().cpu().numpy() for x in outs])
    o = np.where((l == -np.inf)[..., None], 0.0, o)
    with np.errstate(divide="ignore", invalid="ignore"):
        top = l.max(0)
        w = np.exp(l - np.where(top == -np.inf, 0.0, top))
        z = w.sum(0)
        den = np.where(z > 0, z, 1.0)[..., None]
        return (w[..., None] * o).sum(0) / den, top + np.log(z), (w[..., None] * np.abs(o)).sum(0) / den


def merge_check(out, lse, ref, n):
    """exp is off by 2^-22 and its argument by 2^-24 |l - M| (times e^-|l - M|: below 2^-24), sums add
    (n + 2) 2^-24, the quotient 2^-22, and the output's rounding half a step."""
    o, l, mag = ref
    half = torch.finfo(out.dtype).eps / 2
    got = out.double().cpu().numpy()
    tol = (n + 10) * 2.0 ** -23 * mag + half * np.abs(o) * (1 + 2.0 ** -10) + 1e-38
    assert (np.abs(got - o) <= tol).all()
    if lse is not None:
        g = lse.double().cpu().numpy()
        some = np.isfinite(l)
        assert (g[~some] == l[~some]).all()
        assert (np.abs(g - l)[some] <= (n + 8) * 2.0 ** -23 * (1 + np.abs(l[some]))).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("n,N,H,hd", [(1, 1, 1, 8), (2, 8, 32, 128), (3, 33, 5, 64), (16, 7, 3, 80), (4, 1000, 8, 256), (5, 257, 1, 24)])
def test_merge(dt, odt, n, N, H, hd):
    torch.manual_seed(n + N)
    outs = [torch.randn(N, H, hd, device="cuda").to(DT[dt]) for _ in range(n)]
    lses = [3 * torch.randn(N, H, device="cuda") + 5 for _ in range(n)]
    gone = torch.rand(n, N, H, device="cuda") < 0.3
    for i in range(n):                               # parts without a key: whatever they hold
        lses[i][gone[i]] = -float("inf")
        outs[i][gone[i]] = float("nan")
    out, lse = eb.attention_merge(outs, lses, dtype=DT[odt], lse=True)
    assert out.dtype == DT[odt]
    merge_check(out, lse, merge_reference(outs, lses), n)
    assert torch.equal(eb.attention_merge(outs, lses, dtype=DT[odt]), out)


def test_merge_strides_in_place_graph_and_streams():
    torch.manual_seed(0)
    N, H, hd = 50, 4, 128
    wide = [torch.randn(N, H * hd + 64 * (i + 1), device="cuda").to(torch.bfloat16) for i in range(3)]
    outs = [w[:, 32:32 + H * hd].unflatten(1, (H, hd)) for w in wide]
    lses = [torch.randn(N, H, device="cuda") for _ in range(3)]
    want, wl = eb.attention_merge(outs, lses, lse=True)
    merge_check(want, wl, merge_reference(outs, lses), 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = eb.attention_merge(outs, lses, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g, gout = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(g):
        eb.attention_merge(outs, lses, out=gout)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gout, want)
    keep = wide[1].clone()
    eb.attention_merge(outs, lses, out=outs[1])      # in place of a part
    assert torch.equal(outs[1], want)
    wide[1][:, 32:32 + H * hd] = keep[:, 32:32 + H * hd]
    assert torch.equal(wide[1], keep)                # nothing beside its rows


def test_merge_of_infinite_and_nan_lse():
    o = [torch.full((1, 1, 8), float(i), device="cuda") for i in range(3)]
    l = lambda *x: [torch.full((1, 1), v, device="cuda") for v in x]  # noqa: E731
    inf, nan = float("inf"), float("nan")
    out, lse = eb.attention_merge(o, l(inf, 3.0, inf), lse=True)
    assert (out == 1.0).all() and lse.item() == inf
    out, lse = eb.attention_merge(o, l(0.0, nan, -inf), lse=True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    out, lse = eb.attention_merge(o, l(-inf, -inf, -inf), lse=True)
    assert (out == 0).all() and lse.item() == -inf


def test_merge_refusals_of_the_binding():
    o = torch.zeros(3, 2, 64, device="cuda")
    l = torch.zeros(3, 2, device="cuda")
    eb.attention_merge([o], [l])
    for args, kw in ((([], []), {}), (([o] * 17, [l] * 17), {}), (([o, o], [l]), {}), (([o, o.to(torch.bfloat16)], [l, l]), {}),
                     (([o, o[:2]], [l, l]), {}), (([o], [l.double()]), {}), (([o.half()], [l]), {}), (([o], [l]), dict(dtype=torch.float16)),
                     (([o], [l]), dict(out=o[:2])), (([o], [l]), dict(lse=l)), (([o.transpose(0, 1).contiguous().transpose(0, 1)], [l]), {}),
                     (([o], [l]), dict(out=o.to(torch.bfloat16), dtype=torch.float32))):
        with pytest.raises(eb.EagleError):
            eb.attention_merge(*args, **kw)
    assert eb.attention_merge([o[:0]], [l[:0]]).shape == (0, 2, 64)


@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("f4", "f4")])
@pytest.mark.parametrize("rows,plen,clen", [([1] * 32, 4096, 500), ([300, 150, 260, 390], 2000, 0), ([9, 60, 33, 1, 64, 20], 700, 130)])
def test_calls_behind_each_other_repeat(kinds, rows, plen, clen):
    """Many calls in flight, each beginning while the one before ends, so that copies take their time
    and land in any order: the same bits as the first call that ran alone."""
    rng = np.random.default_rng(17)
    B, hd, Hkv, G = len(rows), 128, 4, 4
    ctx = [(97 * i) % (clen + 1) for i in range(B)]
    prefix, _ = make_cache(rng, kinds[0], hd, 64, Hkv, [plen])
    cache, _ = make_cache(rng, kinds[1], hd, 128, Hkv, [c + r for c, r in zip(ctx, rows)])
    args = (prefix, dev(np.array([0, B], np.int32)), dev(np.array([plen], np.int32)), cache)
    lens, at = dev(np.array(ctx, np.int32)), dev(cu(rows))
    sizes = dict(max_group_rows=sum(rows), max_prefix=plen, max_rows=max(rows), max_len=max(c + r for c, r in zip(ctx, rows)), lse=True)
    qs = [torch.randn(sum(rows), Hkv * G, hd, device="cuda").to(torch.bfloat16) for _ in range(2)]
    first = []
    for q in qs:
        first.append(eb.kv_shared_attention(*args, q, at, lens, **sizes))
        torch.cuda.synchronize()
    for _ in range(40):
        outs = [eb.kv_shared_attention(*args, qs[i & 1], at, lens, **sizes) for i in range(10)]
        for i, (o, l) in enumerate(outs):
            assert torch.equal(o, first[i & 1][0]) and torch.equal(l, first[i & 1][1])
    assert cache.check() == 0 and prefix.check() == 0
