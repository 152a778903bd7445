"""Workspace sizes of shared attention: what kv_shared_attention_workspace gives is enough for the
call, with a mask and without."""
import ctypes as C
from types import SimpleNamespace

import pytest

from eagle_speculative_decoding_03_gb300 import binding as eb
from test_kv_abi_cpu import P, cache, lib  # noqa: F401


@pytest.mark.parametrize("kind", [eb.CACHE_BF16, eb.CACHE_F4])
@pytest.mark.parametrize("hd,Hkv,G", [(64, 1, 8), (64, 8, 4), (128, 2, 1), (128, 8, 8), (128, 4, 16)])
@pytest.mark.parametrize("max_rows", [1, 2, 64, 300])
def test_helper_covers_the_call(lib, kind, hd, Hkv, G, max_rows):  # noqa: F811
    scales = {} if kind == eb.CACHE_F4 else dict(k_scale=None, v_scale=None)
    c = cache(kind=kind, head_dim=hd, n_kv_heads=Hkv, **scales)
    handle = SimpleNamespace(c=c)
    for B in (1, 16, 64, 256):
        for max_len in (64, 1000, 4096, 32768):
            N, Hq = B * max_rows, Hkv * G
            if N * Hq * max_len > 1 << 32:
                continue
            sizes = dict(n_groups=2, max_group_rows=(N + 1) // 2, max_prefix=2048, max_rows=max_rows, max_len=max_len)
            have = eb.kv_shared_attention_workspace(handle, handle, Hq, N, B=B, **sizes)
            g = eb.KVGroups(n_groups=2, max_rows=sizes["max_group_rows"], max_len=2048)
            for S in (0, max_rows, 64):
                if S and S < max_rows or S > 64:
                    continue
                a = eb.KVAttention(B=B, N=N, n_heads=Hq, max_rows=max_rows, max_len=max_len, mask=P if S else None, mask_slots=S)
                need = lib.eagle_kv_shared_attention_workspace(C.byref(c), C.byref(g), C.byref(c), C.byref(a))
                assert 0 < need <= have, (B, max_len, S)
