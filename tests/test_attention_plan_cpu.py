"""How attention calls are cut, told from the workspace that they ask for (sizes of a GB300, without a device)."""
import ctypes as C

import pytest

from eagle_speculative_decoding_03_gb300 import binding as eb
from test_kv_abi_cpu import cache, lib  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="plans for the device that is there")


def bf16(**kw):
    return cache(kind=eb.CACHE_BF16, k_scale=None, v_scale=None, **kw)


def attention(lib, c, Hq, B=1, rows=1, max_len=1000):  # noqa: F811
    return lib.eagle_kv_attention_workspace(C.byref(c), C.byref(eb.KVAttention(B=B, N=B * rows, n_heads=Hq, max_rows=rows, max_len=max_len)))


def test_ranges_join_in_clusters_only_where_all_run_at_once(lib):  # noqa: F811
    """15 clusters of 8 CTAs run at once: with 16 of them, 9 ranges of 14 tiles that leave their results in
    a workspace take less than two waves of 8 ranges of 16."""
    for H in (1, 8, 15):
        assert attention(lib, bf16(n_kv_heads=H, head_dim=64), H, max_len=16000 * H // 15) == 0
    assert attention(lib, bf16(n_kv_heads=16, head_dim=64), 16, max_len=16000) == 9 * 16 * (4 * 64 + 8)
