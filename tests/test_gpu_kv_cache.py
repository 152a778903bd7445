"""GPU parity of the paged cache's calls (eagle_rotary, eagle_kv_append, eagle_kv_gather,
eagle_kv_accept) against the float64 oracle, and a run of all of them around a drafted tree.

Rotation bound: with u = 2^-24, an angle is off by at most pi u (the fraction of a half turn rounded
to fp32), cos and sin by 2 u more, their product with the amplitude by u; y = x c + z s then rounds
twice.  Together less than 8 u (|x| + |z|) amplitude, and half a step of the output's type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb, configs, synth
from oracle import kv_oracle as K
from kv_util import cu, dev, make_cache, pack_codes, pages, see_matrix

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    from eagle_speculative_decoding_03_gb300 import build
    build.build()
    return eb.load()


def partner(x, rot, inter):
    z = np.zeros_like(x)
    i = np.arange(rot)
    j = i ^ 1 if inter else (i + rot // 2) % rot
    z[..., i] = x[..., j]
    return np.abs(z)


def check_rotation(y, x, pos, w, inter, amp, half_step):
    ref = K.rotary(x, pos, w, inter, amp)
    tol = 8 * U * (np.abs(x) + partner(x, 2 * len(w), inter)) * max(abs(amp), 1) + half_step * np.abs(ref) + 1e-37
    assert (np.abs(y - ref) <= tol).all(), float((np.abs(y - ref) / tol).max())
    assert (y[..., 2 * len(w):] == x[..., 2 * len(w):]).all()     # the rest of the head is copied


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,hd,rot,inter,far", [
    (1, 1, 128, 128, False, 5), (3, 5, 64, 32, True, 4000), (7, 3, 96, 48, False, 10 ** 6), (2, 40, 128, 16, True, 2 ** 31 - 1),
    (700, 9, 128, 128, True, 10 ** 5), (2500, 2, 256, 112, False, 100), (333, 4, 80, 80, False, 32000), (5, 2, 16, 16, False, 9),
    (1301, 6, 40, 32, True, 50000)])
def test_rotary(dtype, N, H, hd, rot, inter, far):
    rng = np.random.default_rng(N + hd)
    x = K.bf16(rng.standard_normal((N, H, hd))) if dtype == "bf16" else rng.standard_normal((N, H, hd)).astype(np.float32).astype(np.float64)
    pos = rng.integers(0, far, N, endpoint=True)
    pos[0] = far
    t = dev(x, torch.bfloat16 if dtype == "bf16" else torch.float32)
    rope = eb.Rope(rot, theta=5e5, interleaved=inter)
    w = 5e5 ** (-np.arange(0, rot, 2) / rot)
    y = eb.rotary(t, dev(pos.astype(np.int32)), rope)
    check_rotation(y.double().cpu().numpy(), x, pos, w, inter, 1.0, 2.0 ** -8 if dtype == "bf16" else U)
    eb.rotary(t, dev(pos.astype(np.int32)), rope, out=t)          # in place: the same
    assert torch.equal(t, y)


def test_rotary_scaled_frequencies_amplitude_and_strides():
    rng = np.random.default_rng(1)
    w = eb.rope_frequencies(64, 1e4, banded=(8.0, 1.0, 4.0, 8192))
    wide = torch.randn(50, 700, device="cuda")
    x = wide[:, 60:60 + 5 * 128].unflatten(1, (5, 128))
    pos = rng.integers(-100, 200000, 50)                           # a negative position turns back
    rope = eb.Rope(64, inv_freq=w, amplitude=1.25)
    outw = torch.zeros(50, 1280, device="cuda")
    y = eb.rotary(x, dev(pos.astype(np.int32)), rope, out=outw[:, 640:].unflatten(1, (5, 128)))
    check_rotation(y.double().cpu().numpy(), x.double().cpu().numpy(), pos, np.array(w), False, 1.25, U)
    assert (outw[:, :640] == 0).all()
    assert eb.rotary(x[:0], dev(pos[:0].astype(np.int32)), rope).shape == (0, 5, 128)


def turn_fractions(pos, w):
    """pos * w / (2 pi) as (nearest quarter turn mod 4, signed rest in turns), to 40 digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    q, r = np.zeros((len(pos), len(w)), int), np.zeros((len(pos), len(w)))
    for i, p in enumerate(pos):
        for j, f in enumerate(w):
            t = Decimal(int(p)) * Decimal(float(f)) / turn * 4
            k = t.to_integral_value()
            q[i, j], r[i, j] = int(k) % 4, float(t - k) / 4
    return q, r


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("theta,far", [(1e4, 5000), (5e5, 10 ** 6), (5e5, 2 ** 31 - 1)])
def test_angles_keep_their_precision_at_any_position(inter, theta, far):
    """The cosine and sine themselves (rows of ones and zeros), relative to their own size.  An angle is
    rounded once, as a distance t of at most an eighth of a turn from a quarter: 2^-24 t, which is at
    most 2^-24 of the sine (t <= tan t) and of the cosine; sincospif is off by an ulp, 2^-23.  With a
    rounding to spare 2^-22 relative, and |position| 2^-65 turns from the fixed point."""
    rng = np.random.default_rng(70)
    w = eb.rope_frequencies(32, theta)
    pos = np.concatenate([rng.integers(far // 2, far, 250, endpoint=True), -rng.integers(far // 2, far, 50), [0, 1, far]])
    x = torch.zeros(len(pos), 1, 32, device="cuda")
    i = np.arange(16)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + 16)
    x[:, 0, a] = 1.0
    y = eb.rotary(x, dev(pos.astype(np.int32)), eb.Rope(32, theta=theta, interleaved=inter)).double().cpu().numpy()[:, 0]
    q, r = turn_fractions(pos, w)
    c, s = np.cos(2 * np.pi * r), np.sin(2 * np.pi * r)
    cos, sin = np.choose(q, [c, -s, -c, s]), np.choose(q, [s, c, -s, -c])
    slack = 2 * np.pi * np.abs(pos)[:, None] * 2.0 ** -64 + 1e-37
    for got, ref in ((y[:, a], cos), (y[:, b], sin)):
        tol = 2.0 ** -22 * np.abs(ref) + slack
        assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


def test_rotary_of_the_longest_row():
    """2^31 - 128 elements in one row: its first and last heads are what they are alone."""
    H = (1 << 24) - 1
    x = torch.zeros(1, H, 128, dtype=torch.bfloat16, device="cuda")
    ends = torch.randn(1, 6, 128, device="cuda").to(torch.bfloat16)
    x[:, :3], x[:, -3:] = ends[:, :3], ends[:, 3:]
    pos = dev(np.array([77], np.int32))
    y, want = eb.rotary(x, pos, eb.Rope(128)), eb.rotary(ends, pos, eb.Rope(128))
    assert torch.equal(y[:, :3], want[:, :3]) and torch.equal(y[:, -3:], want[:, 3:]) and (y[:, 3:-3] == 0).all()


def held_rows(cache, table, b, n, ps):
    """Request b's first n rows of every pool tensor, on the host."""
    t = np.arange(n)
    pg, r = table[b, t // ps], t % ps
    out = []
    for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        out.append(None if x is None else x.float().cpu().numpy()[pg, :, r] if x.dtype == torch.bfloat16 else x.cpu().numpy()[pg, :, r])
    return out


@pytest.mark.parametrize("kind", ["bf16", "f4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,ps,Hkv,Hq,lens,rows,rot,inter", [
    (128, 16, 2, 8, [0], [1], 128, False), (128, 64, 3, 9, [15, 0, 63, 64], [2, 1, 0, 70], 64, True),
    (64, 32, 8, 8, [31, 5, 100] * 12, [1] * 36, 64, False), (64, 128, 1, 5, [200, 0], [300, 129], 48, False),
    (128, 16, 4, 0, [7, 8, 9], [61, 61, 61], 128, False)])
def test_append(kind, dtype, hd, ps, Hkv, Hq, lens, rows, rot, inter):
    """Rotated keys and values land in their pages, queries come back rotated, nothing else of
    the pool or of the rows behind the last request changes."""
    rng = np.random.default_rng(ps + hd + len(lens))
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    N, pad = sum(rows), 3
    room = [a + r for a, r in zip(lens, rows)]
    table, P = pages(rng, room, ps)
    f4 = kind == "f4"
    cache = eb.KVCache.empty(P, ps, Hkv, hd, dev(table), four_bit=f4, k_global=1.0, v_global=0.25)
    for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if x is not None:
            x.fill_(3)
    qkv = torch.randn(N + pad, (Hq + 2 * Hkv) * hd, device="cuda").to(tt)
    if f4:
        qkv[0, -hd:-hd + 16] = 0                                   # a group of zeros
        qkv[0, -16:] = 1e5                                         # one past the largest value
    q, k, v = (x.unflatten(1, (-1, hd)) for x in (qkv[:, :Hq * hd] if Hq else qkv[:, :hd], qkv[:, Hq * hd:(Hq + Hkv) * hd],
                                                  qkv[:, (Hq + Hkv) * hd:]))
    pos = dev(np.concatenate([np.arange(a, a + r) for a, r in zip(lens, rows)] + [np.zeros(pad)]).astype(np.int32))
    rope = eb.Rope(rot, theta=1e4, interleaved=inter)
    q_out = torch.full((N + pad, max(Hq, 1), hd), 7.0, dtype=tt, device="cuda")
    eb.kv_append(cache, k, v, dev(cu(rows)), dev(np.array(lens, np.int32)), positions=pos, rope=rope, q=q if Hq else None,
                 q_out=q_out if Hq else None)
    assert cache.check() == 0
    if Hq:
        want = eb.rotary(q, pos, rope)
        assert torch.equal(q_out[:N], want[:N]) and (q_out[N:] == 7.0).all()
        check_rotation(want.double().cpu().numpy(), q.double().cpu().numpy(), pos.cpu().numpy(), 1e4 ** (-np.arange(0, rot, 2) / rot),
                       inter, 1.0, 2.0 ** -8 if dtype == "bf16" else U)
    # the stored keys: the rotation (checked above on its own) rounded to bf16
    rk = eb.rotary(k, pos, rope).to(torch.bfloat16).double().cpu().numpy()
    rv = v.to(torch.bfloat16).double().cpu().numpy()
    at = 0
    untouched = np.ones((P, ps), bool)
    for b, (a, r) in enumerate(zip(lens, rows)):
        got = held_rows(cache, table, b, a + r, ps)
        for i, x in ((0, rk[at:at + r]), (1, rv[at:at + r])):
            if not f4:
                assert (got[i][a:] == x).all()
            else:
                code, sc, _ = K.quantise(x, 1.0 if i == 0 else 0.25)
                assert (got[i][a:] == pack_codes(code)).all() and (got[2 + i][a:] == sc).all()
        t = np.arange(a, a + r)
        untouched[table[b, t // ps], t % ps] = False
        at += r
    for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if x is not None:
            assert (x.float().cpu().numpy().transpose(0, 2, 1, 3)[untouched] == 3).all()


def test_append_without_rope_and_with_special_values():
    rng = np.random.default_rng(5)
    table, P = pages(rng, [40], 16)
    x = torch.randn(40, 2, 128, device="cuda")
    cache = eb.KVCache.empty(P, 16, 2, 128, dev(table))
    x[3, 0, 4], x[3, 1, 5], x[4, 0, 6] = float("nan"), float("inf"), -float("inf")
    args = (dev(cu([40])), dev(np.array([0], np.int32)))
    assert eb.kv_append(cache, x, x, *args) is None
    got = held_rows(cache, table, 0, 40, 16)
    assert np.array_equal(got[0], x.to(torch.bfloat16).float().cpu().numpy(), equal_nan=True) and np.array_equal(got[0], got[1], equal_nan=True)
    c4 = eb.KVCache.empty(P, 16, 2, 128, dev(table), four_bit=True)
    eb.kv_append(c4, x, x, *args)
    k, v = eb.kv_gather(c4, dev(cu([40])), 40)
    assert torch.equal(k, v) and torch.isfinite(k).all()
    assert k[3, 0, 4] == 0 and k[3, 1, 5] == 2688 and k[4, 0, 6] == -2688    # NaN -> 0, infinities saturate


def test_append_reports_places_outside_the_table():
    rng = np.random.default_rng(6)
    table, P = pages(rng, [32, 32], 16)
    cache = eb.KVCache.empty(P, 16, 1, 64, dev(table))
    x = torch.randn(4, 1, 64, device="cuda").to(torch.bfloat16)
    eb.kv_append(cache, x, x, dev(cu([2, 2])), dev(np.array([31, 3], np.int32)))   # key 32 has no page
    with pytest.raises(eb.EagleError) as e:
        cache.check()
    assert "0x10" in str(e.value) and cache.check() == 0
    assert (held_rows(cache, table, 0, 32, 16)[0][31] == x[0].float().cpu().numpy()).all()
    assert (held_rows(cache, table, 1, 5, 16)[0][3:] == x[2:].float().cpu().numpy()).all()


@pytest.mark.parametrize("kind", ["bf16", "f4"])
@pytest.mark.parametrize("hd,ps,Hkv,keys", [(128, 16, 2, [1]), (64, 32, 3, [0, 33, 64, 7, 0]), (128, 64, 8, [300, 1, 129]),
                                           (64, 128, 1, [127, 128, 129])])
def test_gather(kind, hd, ps, Hkv, keys):
    rng = np.random.default_rng(hd + ps)
    cache, held = make_cache(rng, kind, hd, ps, Hkv, keys)
    total = sum(keys)
    k = torch.full((total + 5, Hkv, hd), 9.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    eb.kv_gather(cache, dev(cu(keys)), total + 5, k_out=k, v_out=v)
    assert cache.check() == 0
    for got, i in ((k, 0), (v, 1)):
        got = got.double().cpu().numpy()
        assert (got[:total] == np.concatenate([h[i] for h in held])).all() and (got[total:] == 9.0).all()


@pytest.mark.parametrize("kind", ["bf16", "f4"])
@pytest.mark.parametrize("hd,ps,Hkv,layers", [(128, 16, 2, 1), (64, 32, 3, 5), (128, 64, 1, 64)])
def test_accept(kind, hd, ps, Hkv, layers):
    rng = np.random.default_rng(layers)
    S, lens = 24, [0, 30, 61, 5, 17, 40]
    B = len(lens)
    acc = np.array([0, 1, S - 1, 9, 5, 20], np.int32)
    slots = np.full((B, S), -1, np.int32)
    for b in range(B):
        slots[b, :acc[b]] = np.sort(rng.choice(np.arange(1, S), acc[b], replace=False))
    slots[4, :5] = [1, 2, 3, 4, 5]                                  # nothing to move
    slots[5, :20] = np.arange(20)                                   # each move's source is the next one's place
    room = [n + S for n in lens]
    made = [make_cache(np.random.default_rng(7), kind, hd, ps, Hkv, room) for _ in range(layers)]
    table = made[0][0].page_table                                   # (one shape, one table)
    caches = []
    for i, (c, _) in enumerate(made):
        sc = () if kind == "bf16" else (c.k_scale, c.v_scale, 1.0, 0.5)
        caches.append(eb.KVCache(c.k, c.v.roll(i, 0).contiguous() if i else c.v, table, *sc))
    before = [eb.kv_gather(c, dev(cu(room)), sum(room)) for c in caches]
    lens_t = dev(np.array(lens, np.int32))
    new = eb.kv_accept(caches, lens_t, dev(acc), dev(slots))
    for c in caches:
        assert c.check() == 0
    assert new.cpu().tolist() == [n + 1 + a for n, a in zip(lens, acc)]
    at = cu(room)
    for c, old in zip(caches, before):
        got = eb.kv_gather(c, dev(cu(room)), sum(room))
        for x, y in zip(got, old):
            x, y = x.view(torch.int16).cpu().numpy(), y.view(torch.int16).cpu().numpy()   # bits: poisoned rows are NaN
            for b in range(B):
                o = at[b]
                want = y[o:at[b + 1]].copy()
                want[lens[b] + 1:lens[b] + 1 + acc[b]] = y[o + lens[b] + slots[b, :acc[b]]]
                assert (x[o:at[b + 1]] == want).all()
    same = eb.kv_accept(caches, lens_t, dev(np.zeros(B, np.int32)), dev(slots), new_lens=lens_t)   # in place
    assert same is lens_t and lens_t.cpu().tolist() == [n + 1 for n in lens]


def test_accept_cuts_paths_of_more_than_the_tree_without_its_root():
    """S slots, the root's among them, and a tree of its root alone: S - 1 are kept, and reported."""
    for S in (1, 4):
        cache, held = make_cache(np.random.default_rng(63), "bf16", 64, 16, 1, [30])
        new = eb.kv_accept(cache, dev(np.array([20], np.int32)), dev(np.array([S], np.int32)), dev(np.arange(S, dtype=np.int32)[None]))
        with pytest.raises(eb.EagleError) as e:
            cache.check()
        assert "0x4" in str(e.value) and new.tolist() == [20 + S]
        k, _ = eb.kv_gather(cache, dev(cu([30])), 30)
        want = held[0][0].copy()
        want[21:20 + S] = held[0][0][20:19 + S]
        assert (k.double().cpu().numpy() == want).all()


def test_accept_refuses_paths_that_do_not_ascend():
    rng = np.random.default_rng(8)
    cache, held = make_cache(rng, "bf16", 64, 16, 1, [30, 30, 30])
    slots = np.full((3, 8), -1, np.int32)
    slots[0, :3] = [2, 5, 5]
    slots[1, :3] = [1, 9, 3]
    slots[2, :2] = [3, 6]
    new = eb.kv_accept([cache], dev(np.array([20, 20, 20], np.int32)), dev(np.array([3, 3, 2], np.int32)), dev(slots))
    with pytest.raises(eb.EagleError) as e:
        cache.check()
    assert "0x4" in str(e.value)
    assert new.cpu().tolist() == [23, 22, 23]                        # each path ends before the bad slot
    k, _ = eb.kv_gather(cache, dev(cu([30] * 3)), 90)
    k = k.double().cpu().numpy()
    assert (k[21] == held[0][0][22]).all() and (k[22] == held[0][0][25]).all() and (k[60 + 22] == held[2][0][26]).all()


@pytest.mark.parametrize("kind", ["bf16", "f4"])
def test_a_round_of_drafting_and_verification(kind):
    """A prefix appended to pages, gathered for the draft; its tree appended layer by layer and
    attended with the tree's mask; the accepted path kept in every layer; the next prefix gathered.
    The whole round runs on one stream without reading anything back."""
    cfg = configs.get("small_dyn")
    W, I = synth.make_weights(cfg), synth.make_inputs(cfg)
    B, H, hd, ps = cfg.B, cfg.n_kv_heads, cfg.head_dim, 32
    n = np.diff(I["cu_seqlens"])
    S = cfg.kept_per_request() + 1
    rng = np.random.default_rng(11)
    table, P = pages(rng, [int(x) + S for x in n], ps)
    shared = dev(table)                                              # the layers' one page table
    layers = [eb.KVCache.empty(P, ps, H, hd, shared, four_bit=kind == "f4") for _ in range(2)]
    dI = eb.device_inputs(I)
    cus, zero = dI["cu_seqlens"], torch.zeros(B, dtype=torch.int32, device="cuda")
    kk, vv = (dI[x].view(torch.bfloat16).view(-1, H, hd) for x in ("k_cache", "v_cache"))
    for c in layers:
        eb.kv_append(c, kk, vv, cus, zero)                            # (already rotated)
    k, v = eb.kv_gather(layers[0], cus, int(n.sum()))
    if kind == "bf16":
        assert torch.equal(k, kk) and torch.equal(v, vv)
    dI["k_cache"], dI["v_cache"] = k.view(torch.int16), v.view(torch.int16)
    d = eb.EagleDraft(cfg, eb.device_weights(W))
    tree = d.tree(dI)
    lens = (cus[1:] - cus[:-1]).contiguous()
    cr = torch.arange(B + 1, dtype=torch.int32, device="cuda") * S
    rope = eb.Rope(hd, theta=cfg.rope_theta)
    pos = tree["positions"].reshape(-1)
    qkv = [torch.randn(B * S, (cfg.n_heads + 2 * H) * hd, device="cuda").to(torch.bfloat16) for _ in layers]
    outs = []
    for c, x in zip(layers, qkv):
        q, k1, v1 = (y.unflatten(1, (-1, hd)) for y in x.split([cfg.n_heads * hd, H * hd, H * hd], 1))
        qr = eb.kv_append(c, k1, v1, cr, lens, positions=pos, rope=rope, q=q)
        outs.append((qr, eb.kv_attention(c, qr, cr, lens, max_rows=S, max_len=int(n.max()) + S, mask=tree["mask"])))
    # a path of the tree: the greedy walk down the first children
    acc, slots = torch.zeros(B, dtype=torch.int32), torch.full((B, S), -1, dtype=torch.int32)
    par = tree["parents"].cpu()
    for b in range(B):
        u = 0
        while True:
            kids = [i for i in range(1, S) if par[b, i] == u]
            if not kids:
                break
            u = kids[-1]
            slots[b, acc[b]] = u
            acc[b] += 1
    assert int(acc.min()) >= 1
    before = [eb.kv_gather(c, dev(cu([int(x) + S for x in n])), int(n.sum()) + B * S) for c in layers]
    new = eb.kv_accept(layers, lens, acc.cuda(), slots.cuda())
    for c in layers:
        assert c.check() == 0
    d.check()
    nl = new.cpu().numpy()
    assert (nl == n + 1 + acc.numpy()).all()
    at = cu([int(x) + S for x in n])
    for c, (bk, bv), (qr, o) in zip(layers, before, outs):
        k, v = eb.kv_gather(c, dev(cu(nl)), int(nl.sum()))
        to = cu(nl)
        for b in range(B):
            path = [0] + slots[b, :acc[b]].tolist()
            idx = at[b] + np.concatenate([np.arange(n[b]), n[b] + np.array(path)])
            assert torch.equal(k[to[b]:to[b + 1]], bk[idx]) and torch.equal(v[to[b]:to[b + 1]], bv[idx])
            K64, V64 = (x[at[b]:at[b] + n[b] + S].double().cpu().numpy() for x in (bk, bv))
            m = tree["mask"][b].cpu().numpy()
            ref, _, mag, qk, vs = K.attention(qr[b * S:(b + 1) * S].double().cpu().numpy(), K64, V64, see_matrix(int(n[b]), S, m), hd ** -0.5)
            got = o[b * S:(b + 1) * S].double().cpu().numpy()
            # (the attention's own test derives this bound)
            tol = (2.0 ** -8 + 2 * ((hd + 4) * U * qk + 2.0 ** -21 * (1 + qk))[..., None] + (hd + 128) * U) * mag + 2.0 ** -8 * np.abs(ref) \
                + 2.0 ** -32 * vs + 1e-30
            assert (np.abs(got - ref) <= tol).all()
    d.close()


def test_bindings_refuse_what_the_kernels_cannot_take():
    rng = np.random.default_rng(12)
    cache, _ = make_cache(rng, "bf16", 128, 16, 2, [20])
    x = torch.randn(1, 2, 128, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 4, 128, device="cuda").to(torch.bfloat16)
    c1, n1 = dev(cu([1])), dev(np.array([19], np.int32))
    bad = [lambda: eb.kv_append(cache, x.half(), x.half(), c1, n1), lambda: eb.kv_append(cache, x, x.float(), c1, n1),
           lambda: eb.kv_append(cache, x[:, :1], x, c1, n1), lambda: eb.kv_append(cache, x, x, c1.long(), n1),
           lambda: eb.kv_append(cache, x.transpose(0, 1), x, c1, n1), lambda: eb.kv_append(cache, x, x, c1, n1, q=q),
           lambda: eb.kv_append(cache, x, x, c1, n1, rope=eb.Rope(128)), lambda: eb.kv_append(cache, x.cpu(), x, c1, n1),
           lambda: eb.kv_append(cache, x[..., ::2], x, c1, n1),
           lambda: eb.kv_append(cache, x, x, dev(cu([1, 0])), dev(np.array([1, 1], np.int32))),
           lambda: eb.kv_attention(cache, q.float(), c1, n1, 1, 20), lambda: eb.kv_attention(cache, q[:, :3], c1, n1, 1, 20),
           lambda: eb.kv_attention(cache, q, c1, n1, 1, 20, mask=torch.ones(1, 1, 1, device="cuda")),
           lambda: eb.kv_attention(cache, q, c1, n1, 0, 20), lambda: eb.kv_attention(cache, q, c1, n1, 1, 20, out=q.float()),
           lambda: eb.kv_attention(cache, q, c1, n1, 1, 500000, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: eb.kv_gather(cache, dev(cu([1, 1, 1])), 3), lambda: eb.kv_gather(cache, c1, -1),
           lambda: eb.kv_gather(cache, c1, 1, k_out=torch.empty(2, 2, 128, dtype=torch.bfloat16, device="cuda")),
           lambda: eb.kv_accept([], n1, n1, n1[None]), lambda: eb.kv_accept(cache, n1, n1.long(), n1[None]),
           lambda: eb.rotary(q.half(), n1, eb.Rope(128)), lambda: eb.rotary(q, n1.cpu(), eb.Rope(128)),
           lambda: eb.rotary(q, dev(np.zeros(2, np.int32)), eb.Rope(128)), lambda: eb.Rope(128, inv_freq=[1.0]),
           lambda: eb.KVCache(cache.k, cache.v, cache.page_table.long()), lambda: eb.KVCache(cache.k, cache.v[:1], cache.page_table),
           lambda: eb.KVCache(cache.k, cache.v, cache.page_table, k_scale=cache.k), lambda: eb.KVCache(cache.k.cpu(), cache.v, cache.page_table)]
    for i, f in enumerate(bad):
        with pytest.raises(eb.EagleError):
            f()
            raise AssertionError(f"case {i} was taken")
    assert cache.check() == 0


@pytest.mark.parametrize("kind", ["bf16", "f4"])
def test_a_captured_step_replays_on_the_lengths_of_the_day(kind):
    """append -> attention -> accept with the lengths updated in place, captured once: three
    replays equal three eager steps on a copy of the state, bit for bit."""
    rng = np.random.default_rng(20)
    B, S, H, G, hd, ps = 3, 5, 2, 4, 128, 16
    lens0 = [0, 30, 129]
    def state():
        c, _ = make_cache(np.random.default_rng(21), kind, hd, ps, H, lens0, room=[n + 40 for n in lens0])
        return c, dev(np.array(lens0, np.int32))
    mask = np.tril(np.ones((S, S), np.uint8))[None].repeat(B, 0)
    mask[:, 3, 2] = 0                                                # slot 3 branches off slot 1
    slots = np.full((B, S), -1, np.int32)
    slots[:, :2] = [1, 3]
    acc, slots, mask = dev(np.array([2, 0, 2], np.int32)), dev(slots), dev(mask)
    cr, rope = dev(cu([S] * B)), eb.Rope(64, theta=1e4, interleaved=True)
    qkv = torch.randn(B * S, (H * G + 2 * H) * hd, device="cuda").to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, hd)) for x in qkv.split([H * G * hd, H * hd, H * hd], 1))
    off = torch.arange(S, dtype=torch.int32, device="cuda").repeat(B)
    def step(c, lens, out):
        pos = lens.repeat_interleave(S, output_size=B * S) + off
        qr = eb.kv_append(c, k, v, cr, lens, positions=pos, rope=rope, q=q)
        eb.kv_attention(c, qr, cr, lens, max_rows=S, max_len=200, mask=mask, out=out)
        eb.kv_accept(c, lens, acc, slots, new_lens=lens)
    c1, l1 = state()
    want, outs = torch.zeros(B * S, H * G, hd, dtype=torch.bfloat16, device="cuda"), []
    for _ in range(3):
        step(c1, l1, want)
        outs.append(want.clone())
    c2, l2 = state()
    got = torch.zeros_like(want)
    warm, lw = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm, lw, got.clone())
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c2, l2, got)
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, outs[i]), i
    assert l1.tolist() == l2.tolist() == [9, 33, 138] and c1.check() == 0 and c2.check() == 0
    for x, y in ((c1.k, c2.k), (c1.v, c2.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_streams_at_once():
    """Caches of their own on two streams: what each gives alone."""
    made = []
    for i, kind in enumerate(("bf16", "f4")):
        c, _ = make_cache(np.random.default_rng(30 + i), kind, 128, 64, 4, [3000, 700])
        q = torch.randn(2, 16, 128, device="cuda").to(torch.bfloat16)
        made.append((c, q, dev(cu([1, 1])), dev(np.array([2999, 699], np.int32)), dev(cu([3000, 700]))))
    def work(m, stream=None):
        c, q, cr, n, cs = m
        return (eb.kv_attention(c, q, cr, n, 1, 3000, stream=stream),) + eb.kv_gather(c, cs, 3700, stream=stream)
    want = [work(m) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[work(m, s) for _ in range(20)] for m, s in zip(made, streams)]
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for x in gs:
            assert all(torch.equal(a, b) for a, b in zip(w, x))


def test_many_requests_and_rows():
    """More requests than a warp, rows of one request spread over many CTAs, an empty call."""
    rng = np.random.default_rng(40)
    rows = rng.integers(0, 9, 300).tolist()
    table, P = pages(rng, rows, 16)
    cache = eb.KVCache.empty(P, 16, 1, 64, dev(table))
    N = sum(rows)
    x = torch.randn(N, 1, 64, device="cuda").to(torch.bfloat16)
    zero = torch.zeros(300, dtype=torch.int32, device="cuda")
    eb.kv_append(cache, x, x, dev(cu(rows)), zero)
    k, v = eb.kv_gather(cache, dev(cu(rows)), N)
    assert cache.check() == 0 and torch.equal(k, x) and torch.equal(v, x)
    q = torch.randn(N, 2, 64, device="cuda").to(torch.bfloat16)
    o = eb.kv_attention(cache, q, dev(cu(rows)), zero, max_rows=8, max_len=8)
    at = cu(rows)
    for b in (0, 150, 299):
        if rows[b]:
            s = slice(at[b], at[b + 1])
            ref = K.attention(q[s].double().cpu().numpy(), x[s].double().cpu().numpy(), x[s].double().cpu().numpy(),
                              see_matrix(0, rows[b]), 64 ** -0.5)
            # (p rounded to 8 bits at least, the output to bf16; |out| <= sum p |v| / sum p)
            assert (np.abs(o[s].double().cpu().numpy() - ref[0]) <= (2.0 ** -7 + 2.0 ** -14) * ref[2]).all()
    none = x[:0]
    assert eb.kv_append(cache, none, none, dev(cu([0])), zero[:1]) is None
    assert eb.kv_attention(cache, q[:0], dev(cu([0])), zero[:1], 1, 1).shape == (0, 2, 64)
    assert eb.kv_gather(cache, dev(cu([0])), 0)[0].shape == (0, 1, 64)


@pytest.mark.parametrize("kg,vg", [(0.37, 3.1), (1e-3, 700.0), (2.0 ** -20, 2.0 ** 20)])
def test_four_bit_store_with_any_global_factor(kg, vg):
    """Scales and codes equal the definition's but where a quotient lies within the kernel's own
    rounding of a border: the scale's quotient is rounded to 18 bits (2^-18 relative with the
    product's error), a code's to multiples of 2^-18 (off by less than 2^-17 in all)."""
    rng = np.random.default_rng(50)
    n, H, hd = 400, 4, 128
    kg32, vg32 = float(np.float32(kg)), float(np.float32(vg))
    table, P = pages(rng, [n], 32)
    cache = eb.KVCache.empty(P, 32, H, hd, dev(table), four_bit=True, k_global=kg, v_global=vg)
    x = K.bf16(rng.standard_normal((n, H, hd)) * np.exp2(rng.integers(-6, 7, (n, H, 1))))
    k, v = K.bf16(x * kg32), K.bf16(x * vg32)
    eb.kv_append(cache, dev(k, torch.bfloat16), dev(v, torch.bfloat16), dev(cu([n])), dev(np.array([0], np.int32)))
    assert cache.check() == 0
    got = held_rows(cache, table, 0, n, 32)
    for i, (src, g) in enumerate(((k, kg32), (v, vg32))):
        code, sc, _ = K.quantise(src, g)
        gsc, gc = got[2 + i], got[i]
        ratio = np.abs(src.reshape(n, H, -1, 16)).max(-1) / (6 * g)
        off = gsc != sc
        mid = (K.E4M3[1:] + K.E4M3[:-1]) / 2
        near = np.abs(ratio[..., None] / mid - 1).min(-1) < 2.0 ** -17
        assert (near | ~off).all() and off.mean() < 1e-2
        gcode = np.stack([gc & 15, gc >> 4], -1).reshape(n, H, hd)
        unit = (K.E4M3[gsc] * g)[..., None]
        mag = np.abs(src.reshape(n, H, -1, 16)) / np.where(unit > 0, unit, 1)
        border = (K.E2M1[1:] + K.E2M1[:-1]) / 2
        near = (np.abs(mag[..., None] - border).min(-1) < 2.0 ** -17).reshape(n, H, hd) | off.repeat(16, -1)
        assert (near | (gcode == code)).all()


def reported(cache, word):
    with pytest.raises(eb.EagleError) as e:
        cache.check()
    assert str(e.value).endswith(f"0x{word:x}") and cache.check() == 0


@pytest.mark.parametrize("kind", ["bf16", "f4"])
def test_gather_reports_ranges_past_its_bounds(kind):
    """Packed rows that the outputs have no room for, or that descend, are reported; the rows
    inside are right."""
    rng = np.random.default_rng(60)
    cache, held = make_cache(rng, kind, 128, 16, 2, [20, 30])
    k, v = eb.kv_gather(cache, dev(cu([20, 30])), 45)                # five rows short
    reported(cache, eb.DEVERR_PREFIX)
    for got, i in ((k, 0), (v, 1)):
        assert (got.double().cpu().numpy() == np.concatenate([h[i] for h in held])[:45]).all()
    for ranges in ([-2, 18, 40], [0, 20, 10]):
        eb.kv_gather(cache, dev(np.array(ranges, np.int32)), 40)
        reported(cache, eb.DEVERR_PREFIX)
    eb.kv_gather(cache, dev(np.array([3, 20, 40], np.int32)), 41)    # rows of no request at both ends
    assert cache.check() == 0


@pytest.mark.parametrize("kind", ["bf16", "f4"])
def test_append_reports_ranges_past_its_bounds(kind):
    rng = np.random.default_rng(61)
    table, P = pages(rng, [32, 32], 16)
    x = torch.randn(6, 2, 64, device="cuda").to(torch.bfloat16)
    def fresh():
        return eb.KVCache.empty(P, 16, 2, 64, dev(table), four_bit=kind == "f4")
    def call(ranges, lens):
        c = fresh()
        eb.kv_append(c, x, x, dev(np.array(ranges, np.int32)), dev(np.array(lens, np.int32)))
        return c
    want = call([0, 2, 6], [5, 7])
    assert want.check() == 0
    c = call([0, 2, 9], [5, 7])                                      # rows 6 to 8 are not there
    reported(c, eb.DEVERR_PREFIX)
    assert torch.equal(c.k.view(torch.uint8), want.k.view(torch.uint8)) and torch.equal(c.v.view(torch.uint8), want.v.view(torch.uint8))
    reported(call([0, 4, 3], [5, 7]), eb.DEVERR_PREFIX)
    reported(call([-1, 2, 6], [5, 7]), eb.DEVERR_PREFIX)
    c = call([0, 2, 6], [-1, 7])                                     # a negative length: that request is skipped
    reported(c, eb.DEVERR_PREFIX)
    w = fresh()
    eb.kv_append(w, x, x, dev(np.array([2, 2, 6], np.int32)), dev(np.array([0, 7], np.int32)))
    assert w.check() == 0 and torch.equal(c.k.view(torch.uint8), w.k.view(torch.uint8))
    reported(call([0, 2, 6], [2 ** 31 - 1, 7]), eb.DEVERR_PAGE)      # past every page


def test_accept_reports_negative_lengths():
    rng = np.random.default_rng(62)
    cache, held = make_cache(rng, "bf16", 64, 16, 1, [30, 30])
    slots = dev(np.array([[2, 5, -1, -1, -1, -1], [2, 5, -1, -1, -1, -1]], np.int32))
    acc, lens = dev(np.array([2, 2], np.int32)), dev(np.array([-2, 20], np.int32))
    new = eb.kv_accept(cache, lens, acc, slots)
    reported(cache, eb.DEVERR_PREFIX)
    assert new.tolist() == [-2, 23]
    k, _ = eb.kv_gather(cache, dev(cu([30, 30])), 60)
    want = np.concatenate([held[0][0], held[1][0]])
    want[30 + 21], want[30 + 22] = held[1][0][22], held[1][0][25]
    assert (k.double().cpu().numpy() == want).all()
    eb.kv_accept(cache, lens, acc, slots, new_lens=lens)             # in place
    reported(cache, eb.DEVERR_PREFIX)
    assert lens.tolist() == [-2, 23]


def test_four_bit_groups_of_scale_zero_are_zeros():
    """Values whose scale rounds to 0, of either sign: codes and scales are 0."""
    cache = eb.KVCache.empty(2, 16, 1, 64, dev(np.zeros((1, 1), np.int32)), four_bit=True, k_global=64.0, v_global=50.1)
    x = torch.full((4, 1, 64), -0.01, device="cuda").to(torch.bfloat16)
    eb.kv_append(cache, x, x, dev(cu([4])), dev(np.array([0], np.int32)))
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        assert (t == 0).all()


def test_four_bit_store_next_to_the_borders():
    """Global factors that put a scale's or a code's quotient within fp32's last places of a border
    between two codes, on either side and on it: scales and codes are the definition's."""
    rng = np.random.default_rng(64)
    n, H, hd = 32, 1, 64
    table, P = pages(rng, [n], 32)
    mids = (K.E4M3[1:] + K.E4M3[:-1]) / 2
    halves = (K.E2M1[1:] + K.E2M1[:-1]) / 2
    for trial in range(120):
        top = float(K.bf16(np.exp2(rng.uniform(-3, 3, 1)))[0])
        if trial % 2:      # a scale's quotient, top / (6 g), beside the middle of two scales
            g = np.float32(top / (6.0 * rng.choice(mids[mids > 2.0 ** -7])))
        else:              # a value's, x / (scale g), beside the middle of two codes
            g = np.float32(top / (rng.choice(halves) * rng.choice(K.E4M3[8:])))
        for step in (-1, 0, 1):
            glob = float(np.nextafter(g, np.float32(step * np.inf))) if step else float(g)
            x = rng.standard_normal((n, H, hd)) * top / 4
            x[:, :, 0] = top
            x[::2, :, 16:32] *= 2.0 ** -3
            if trial % 2 == 0:                                  # groups whose largest is another: the scale varies
                x[:, 0, 1] = top * np.exp2(rng.uniform(0, 4, n))
            x = K.bf16(x)
            cache = eb.KVCache.empty(P, 32, H, hd, dev(table), four_bit=True, k_global=glob, v_global=glob)
            t = dev(x, torch.bfloat16)
            eb.kv_append(cache, t, t, dev(cu([n])), dev(np.array([0], np.int32)))
            got = held_rows(cache, table, 0, n, 32)
            code, sc, _ = K.quantise(x, glob)
            for i in (0, 1):
                assert (got[2 + i] == sc).all(), (trial, glob, np.argwhere(got[2 + i] != sc)[:4])
                assert (got[i] == pack_codes(code)).all(), (trial, glob, np.argwhere(got[i] != pack_codes(code))[:4])
