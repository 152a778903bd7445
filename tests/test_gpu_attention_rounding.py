"""Calls of few query vectors over bf16 pages keep 16 bits of the probabilities, however the keys are cut.

Keys of three scores, 0, c1 and c2, whose e^c is about as far from its 8-bit rounding as it gets; in
each dim the values of two of them cancel, so that the output is near 0 and a rounding of p stands
out against the sum of magnitudes: 2^-9 of it with 8 bits.  With p in two parts of 8 bits each is off by
at most 2^-16, the rest as in test_gpu_kv_attention's bound."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb
from oracle import kv_oracle as K
from kv_util import cu, dev, make_cache
from test_gpu_kv_attention import lib  # noqa: F401


def far_scores():
    c = K.bf16(-np.arange(20, 700) / 256.0)
    p = np.exp(c)
    off = np.abs(K.bf16(p) / p - 1)
    return c[np.argsort(-off)[:2]]


def fill(rng, cache, held):
    """Gives every held key one of the three scores against a query of 1 in dim 0 (scale 1)."""
    c = np.array([0.0, *far_scores()])
    hd, ps = cache.k.shape[-1], cache.k.shape[2]
    tab = cache.page_table.cpu().numpy()
    pairs = [(0, 1), (0, 2), (1, 2)]
    v3 = np.zeros((3, hd))
    for d in range(hd):
        i, j = pairs[d % 3]
        v3[i, d] = 1.0 + d / 64.0
        v3[j, d] = -v3[i, d] * np.exp(c[i] - c[j])
    v3 = K.bf16(v3)
    for b, (kk, vv) in enumerate(held):
        n = len(kk)
        if not n:
            continue
        cls = rng.integers(0, 3, n)
        kk[:] = 0.0
        kk[:, :, 0] = c[cls][:, None]
        vv[:] = v3[cls][:, None]
        t = np.arange(n)
        at = (torch.from_numpy(tab[b, t // ps]).long().cuda(), slice(None), torch.from_numpy(t % ps).long().cuda())
        cache.k[at], cache.v[at] = dev(kk, torch.bfloat16), dev(vv, torch.bfloat16)


def close(out, keys, Hq, hd, rows):
    """16 bits of p: see above."""
    q = np.zeros((rows, Hq, hd))
    q[..., 0] = 1.0
    o, _, mag, qk, _ = K.attention(q, keys[0], keys[1], np.ones((rows, len(keys[0])), bool), 1.0)
    eps = (hd + 4) * 2.0 ** -24 * qk + 2.0 ** -21 * (1 + qk)
    tol = (2.0 ** -16 + 2 * eps[..., None] + (hd + 128) * 2.0 ** -24) * mag + 2.0 ** -8 * np.abs(o)
    got = out.double().cpu().numpy()
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) / tol).max())
    # What the test is worth: p of 8 bits is off by 2^-9.5 or more for one of a dim's two scores, half of the
    # magnitudes, so 2^-10.5 mag; the output's own rounding hides that where |o| is 2^-3 mag and more (the three
    # scores' counts differ by chance, so it is looked at where there are many keys).
    assert len(keys[0]) < 700 or (np.abs(o) < 2.0 ** -3 * mag).all()


@pytest.mark.parametrize("bound", [0, 1 << 20])      # (by a bound so far above the lengths the keys are dealt out in line)
@pytest.mark.parametrize("hd,ps,Hkv,G,lens,rows", [
    (128, 64, 2, 4, [1500], 1), (64, 32, 1, 1, [20000], 1),
    (128, 64, 8, 4, [1000 + 37 * i for i in range(16)], 2), (64, 16, 16, 1, [700] * 16, 1),
    (128, 128, 8, 1, [9000, 5, 1200], 8),
])
def test_cross_attention_of_few_vectors(hd, ps, Hkv, G, lens, rows, bound):
    rng = np.random.default_rng(1)
    cache, held = make_cache(rng, "bf16", hd, ps, Hkv, lens)
    fill(rng, cache, held)
    B = len(lens)
    q = torch.zeros(B * rows, Hkv * G, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    out = eb.kv_cross_attention(cache, q, dev(cu([rows] * B)), dev(np.array(lens, np.int32)), max_rows=rows,
                                max_len=max(max(lens), bound), scale=1.0)
    assert cache.check() == 0
    for b in range(B):
        close(out[b * rows:(b + 1) * rows], held[b], Hkv * G, hd, rows)


@pytest.mark.parametrize("bound", [0, 1 << 20])
@pytest.mark.parametrize("hd,Hkv,G,plens,ctx", [(128, 8, 4, [700] * 40, [300 + i for i in range(40)]), (64, 2, 4, [500, 90], [30, 9]),
                                                (64, 8, 8, [0] * 30, [400 + 9 * i for i in range(30)])])
def test_steps_behind_a_prefix_each(hd, Hkv, G, plens, ctx, bound):
    """One request a group: prefix and own keys both as few vectors."""
    rng = np.random.default_rng(2)
    B = len(ctx)
    prefix, pre = make_cache(rng, "bf16", hd, 64, Hkv, plens)
    cache, own = make_cache(rng, "bf16", hd, 32, Hkv, [c + 1 for c in ctx])
    fill(rng, prefix, pre)
    fill(rng, cache, own)
    q = torch.zeros(B, Hkv * G, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    ints = lambda x: dev(np.array(x, np.int32))  # noqa: E731
    out = eb.kv_shared_attention(prefix, ints(list(range(B + 1))), ints(plens), cache, q, ints(list(range(B + 1))), ints(ctx), max_group_rows=1,
                                 max_prefix=max(max(plens), 1), max_rows=1, max_len=max(max(ctx) + 1, bound), scale=1.0)
    assert cache.check() == 0 and prefix.check() == 0
    for b in range(B):
        close(out[b:b + 1], tuple(np.concatenate(x) for x in zip(pre[b], own[b])), Hkv * G, hd, 1)


@pytest.mark.parametrize("hd,Hkv,G,plens,groups,ctx", [(128, 8, 4, [3000], [0, 32], [200 + i for i in range(32)]), (64, 2, 8, [900, 1200], [0, 7, 15], [9 * i for i in range(15)]),
                                                       (128, 1, 16, [1500], [0, 8], [90] * 8)])
def test_steps_of_up_to_128_vectors_behind_a_prefix(hd, Hkv, G, plens, groups, ctx):
    rng = np.random.default_rng(3)
    B = len(ctx)
    prefix, pre = make_cache(rng, "bf16", hd, 64, Hkv, plens)
    cache, own = make_cache(rng, "bf16", hd, 32, Hkv, [c + 1 for c in ctx])
    fill(rng, prefix, pre)
    fill(rng, cache, own)
    q = torch.zeros(B, Hkv * G, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    ints = lambda x: dev(np.array(x, np.int32))  # noqa: E731
    out = eb.kv_shared_attention(prefix, ints(groups), ints(plens), cache, q, ints(list(range(B + 1))), ints(ctx),
                                 max_group_rows=max(np.diff(groups)), max_prefix=max(plens), max_rows=1, max_len=max(ctx) + 1, scale=1.0)
    assert cache.check() == 0 and prefix.check() == 0
    for b in range(B):
        g = next(i for i in range(len(plens)) if groups[i] <= b < groups[i + 1])
        close(out[b:b + 1], tuple(np.concatenate(x) for x in zip(pre[g], own[b])), Hkv * G, hd, 1)
