"""Paged caches for the tests: pools with shuffled pages, rows behind the keys poisoned."""
import numpy as np
import torch

from eagle_speculative_decoding_03_gb300 import binding as eb
from oracle import kv_oracle as K


def cu(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def pages(rng, room, ps, spare=2):
    """page_table [B, width] (unused places -1) and the pool's page count for `room` tokens each."""
    need = [(n + ps - 1) // ps for n in room]
    total = sum(need) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(room), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def pack_codes(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def make_cache(rng, kind, hd, ps, Hkv, keys, room=None, k_global=1.0, v_global=0.5, poison=True):
    """A cache holding keys[b] random tokens per request.  Returns (KVCache, list of per-request
    float64 K, V [n, Hkv, hd] as stored).  Every other row of the pool is NaN (bf16) or NaN scales."""
    room = keys if room is None else room
    table, P = pages(rng, room, ps)
    held = []
    if kind == "bf16":
        fill = np.float32(np.nan if poison else 0.0)
        k = np.full((P, Hkv, ps, hd), fill, np.float32)
        v = np.full((P, Hkv, ps, hd), fill, np.float32)
    else:
        k = np.full((P, Hkv, ps, hd // 2), 0x77, np.uint8)
        v = k.copy()
        ks = np.full((P, Hkv, ps, hd // 16), 0x7F if poison else 0, np.uint8)
        vs = ks.copy()
    for b, n in enumerate(keys):
        kk = K.bf16(rng.standard_normal((n, Hkv, hd)) * np.exp(0.4 * rng.standard_normal((1, Hkv, hd))))
        vv = K.bf16(rng.standard_normal((n, Hkv, hd)))
        t = np.arange(n)
        pg, r = table[b, t // ps], t % ps
        if kind == "bf16":
            k[pg, :, r], v[pg, :, r] = kk, vv
            held.append((kk, vv))
        else:
            kc, ksc, kval = K.quantise(kk, k_global)
            vc, vsc, vval = K.quantise(vv, v_global)
            k[pg, :, r], v[pg, :, r] = pack_codes(kc), pack_codes(vc)
            ks[pg, :, r], vs[pg, :, r] = ksc, vsc
            held.append((kval, vval))
    if kind == "bf16":
        c = eb.KVCache(dev(k, torch.bfloat16), dev(v, torch.bfloat16), dev(table))
    else:
        c = eb.KVCache(dev(k), dev(v), dev(table), dev(ks), dev(vs), k_global, v_global)
    return c, held


def tree_masks(rng, B, S, rows):
    """Ancestor-or-self masks [B, S, S] of random trees (uint8); only the first rows[b] rows used."""
    m = np.zeros((B, S, S), np.uint8)
    for b in range(B):
        for i in range(S):
            if i:
                m[b, i] |= m[b, rng.integers(0, i)]
            m[b, i, i] = 1
        m[b, rows[b]:] = 1                    # rows and columns past the request's own must not matter
        m[b, :, rows[b]:] = 1
    return m


def see_matrix(ctx, R, mask=None):
    see = np.ones((R, ctx + R), bool)
    see[:, ctx:] = np.tril(np.ones((R, R), bool)) if mask is None else mask[:R, :R] != 0
    return see
