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


def wide(hd):
    return 152 * (32 + 8 * 256 * (hd + 2))


def few(hd):
    return 152 * (32 + 8 * 8 * (hd + 2))


def cross(lib, c, Hq, B, rows, max_len):  # noqa: F811
    return lib.eagle_kv_cross_attention_workspace(C.byref(c), C.byref(eb.KVCross(B=B, N=B * rows, n_heads=Hq, max_rows=rows, max_len=max_len)))


# kind, Hkv, hd, G, B, rows, max_len: the faster side of a measurement each (us by ranges, in line)
MEASURED = [
    ("bf16", 8, 128, 4, 1, 3, 8000, "ranges"),       # 17.8, 31.2
    ("bf16", 8, 128, 4, 32, 16, 870, "ranges"),      # 26.0, 65.5
    ("bf16", 8, 128, 4, 1, 32, 80000, "ranges"),     # 63.9, 87.4
    ("bf16", 8, 128, 4, 32, 128, 870, "ranges"),     # 63.3, 117.1
    ("bf16", 8, 128, 4, 4, 128, 10500, "wide"),      # 81.4, 64.2
    ("bf16", 8, 128, 4, 2, 2047, 4099, "wide"),      # 229, 219
    ("f4", 8, 128, 4, 1, 16, 32000, "ranges"),       # 32.9, 52.5
    ("f4", 8, 128, 4, 4, 4, 35000, "ranges"),        # 73.9, 74.5
    ("f4", 8, 128, 4, 4, 64, 35000, "wide"),         # 119.4, 90.3
    ("bf16", 8, 128, 4, 4, 32, 35000, "ranges"),     # 81.1, 83.2
    ("bf16", 8, 128, 4, 4, 64, 35000, "wide"),       # 97.6, 86.2
    ("f4", 8, 128, 4, 1, 256, 16000, "wide"),        # 84.5, 74.4
    ("f4", 8, 128, 4, 32, 64, 870, "ranges"),        # 46.4, 66.1
    ("bf16", 16, 64, 1, 32, 1, 3000, "few"),         # 86.5, 56.7
    ("bf16", 8, 128, 4, 32, 1, 3500, "few"),         # 59.4, 48.5
    ("bf16", 8, 128, 8, 32, 1, 1200, "ranges"),      # 29.5, 36.9
    ("bf16", 8, 128, 4, 1, 1, 20000, "ranges"),      # 23.2, 28.7
]


@pytest.mark.parametrize("kind,Hkv,hd,G,B,rows,max_len,by", MEASURED)
def test_cross_attention_is_cut_the_faster_way(lib, kind, Hkv, hd, G, B, rows, max_len, by):  # noqa: F811
    c = bf16(n_kv_heads=Hkv, head_dim=hd) if kind == "bf16" else cache(n_kv_heads=Hkv, head_dim=hd)
    need = cross(lib, c, Hkv * G, B, rows, max_len)
    assert (need == wide(hd)) == (by == "wide") and (need == few(hd)) == (by == "few")


@pytest.mark.parametrize("B,max_len", [(1, 700), (4, 35000), (32, 3000), (128, 600), (2, 30000)])
@pytest.mark.parametrize("rows", [3, 8, 32])
def test_up_to_128_vectors_over_bf16_pages_never_lose_bits(lib, B, max_len, rows):  # noqa: F811
    """The wide kernel keeps 8 bits of p over bf16 pages, the ranges 16: which it is goes by the vectors alone."""
    for hd, Hkv in ((128, 8), (64, 16)):
        assert cross(lib, bf16(n_kv_heads=Hkv, head_dim=hd), Hkv * 4, B, rows, max_len) != wide(hd)


def test_calls_of_more_blocks_than_a_launch_has_are_taken(lib):  # noqa: F811
    assert cross(lib, bf16(n_kv_heads=1, head_dim=128), 16, 70000, 1, 100) == wide(128)
    for G in (1, 16):                                # a prefix for each of 70,000 requests
        c = bf16(n_kv_heads=1, head_dim=128)
        g = eb.KVGroups(n_groups=70000, max_rows=1, max_len=100)
        a = eb.KVAttention(B=70000, N=70000, n_heads=G, max_rows=1, max_len=100)
        if G == 1:                                   # (their own keys are cut by ranges with 16 heads, which refuses them)
            assert lib.eagle_kv_shared_attention_workspace(C.byref(c), C.byref(g), C.byref(c), C.byref(a)) > wide(128)
        a = eb.KVAttention(B=60000, N=60000, n_heads=G, max_rows=1, max_len=100)
        assert lib.eagle_kv_shared_attention_workspace(C.byref(c), C.byref(g), C.byref(c), C.byref(a)) > wide(128)


@pytest.mark.parametrize("kind", ["bf16", "f4"])
def test_bounds_far_above_the_rows_do_not_launch_empty_blocks(lib, kind):  # noqa: F811
    """A prompt among single tokens: 64 requests of up to 4,096 rows, 4,159 in all."""
    c = bf16() if kind == "bf16" else cache()

    def need(N, rows):
        return lib.eagle_kv_cross_attention_workspace(C.byref(c), C.byref(eb.KVCross(B=64, N=N, n_heads=32, max_rows=rows, max_len=1000)))
    assert need(4159, 4096) == wide(128)               # 285 us by ranges, 143 in line (bf16)
    assert need(64 * 128, 128) != wide(128)
    g = eb.KVGroups(n_groups=64, max_rows=4096, max_len=1000)
    a = eb.KVAttention(B=64, N=4159, n_heads=32, max_rows=1, max_len=40)
    few_rows = eb.KVAttention(B=64, N=64, n_heads=32, max_rows=1, max_len=40)
    for w in (a, few_rows):
        assert lib.eagle_kv_shared_attention_workspace(C.byref(c), C.byref(g), C.byref(c), C.byref(w)) > wide(128)
