"""The tests of cross and shared attention once more through each kernel that the sizes could choose: the
choice goes by the call's bounds (max_rows, max_len ...), which may be larger than the sizes, so that
the wide kernel and the one for few vectors see small, odd and ragged calls too."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from eagle_speculative_decoding_03_gb300 import binding as eb
from kv_util import cu, dev, make_cache
from test_gpu_attention_non_finite import (test_a_nan_key_reaches_every_row_from_any_part, test_far_infinities_are_the_formulas,  # noqa: F401
                                           test_far_infinities_of_prefix_or_own_keys_are_the_formulas)
from test_gpu_cross_attention import (test_few_rows, test_many_rows, test_many_short_sequences_repeat,  # noqa: F401
                                      test_non_finite_values_in_cached_keys, test_scores_that_are_not_finite, test_strided_rows_graph_and_streams)
from test_gpu_kv_attention import lib  # noqa: F401
from test_gpu_shared_attention import (test_calls_behind_each_other_repeat, test_graph_streams_and_repeats,  # noqa: F401
                                       test_masks_that_leave_the_own_part_empty, test_single_tokens, test_trees_and_chunks)

CROSS, CROSS_WS, SHARED, SHARED_WS = eb.kv_cross_attention, eb.kv_cross_attention_workspace, eb.kv_shared_attention, eb.kv_shared_attention_workspace


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def wide_bounds(Hkv, G, B, max_rows, max_len):
    """More than 128 vectors, and 100 tiles of 128 keys for every SM."""
    max_rows = max(max_rows, 128 // G + 1)
    items = B * Hkv * ((max_rows * G + 255) // 256)
    return max_rows, max(max_len, 128 * max(20, -(-101 * sms() // items)))


def few_bounds(Hkv, B, max_len, least):
    return max(max_len, 64 * -(-least * sms() // (B * Hkv)) + 64)


def wide_bytes(hd):
    return sms() * (32 + 8 * 256 * (hd + 2))


def few_bytes(hd):
    return sms() * (32 + 8 * 8 * (hd + 2))


def cross_bounds(kernel, cache, Hq, N, B, max_rows, max_len):
    G = Hq // cache.k.shape[1]
    if kernel == "wide":
        max_rows, max_len = wide_bounds(cache.k.shape[1], G, B, max_rows, max_len)
        assert CROSS_WS(cache, Hq, N, B, max_rows, max_len) == wide_bytes(cache.head_dim)
    elif cache.k_scale is None and max_rows * G <= 8:
        max_len = few_bounds(cache.k.shape[1], B, max_len, 91)
        assert CROSS_WS(cache, Hq, N, B, max_rows, max_len) == few_bytes(cache.head_dim)
    return max_rows, max_len


def shared_bounds(kernel, prefix, cache, Hq, n_groups, B, mg, mp, mr, ml, mask):
    Hkv = cache.k.shape[1]
    if kernel == "wide":
        mg, mp = wide_bounds(Hkv, Hq // Hkv, n_groups, mg, mp)
    elif cache.k_scale is None and mr == 1 and mask is None and Hq // Hkv <= 8:
        ml = few_bounds(Hkv, B, ml, 81)
    return mg, mp, mr, ml


@pytest.fixture(autouse=True, params=["wide", "few"])
def kernel(request, monkeypatch):
    name = request.param

    def cross(cache, q, cu_rows, lens, max_rows, max_len, **kw):
        r, n = cross_bounds(name, cache, q.shape[1], q.shape[0], lens.shape[0], max_rows, max_len)
        return CROSS(cache, q, cu_rows, lens, r, n, **kw)

    def cross_ws(cache, n_heads, N, B, max_rows, max_len):
        return CROSS_WS(cache, n_heads, N, B, *cross_bounds(name, cache, n_heads, N, B, max_rows, max_len))

    def shared(prefix, cu_groups, prefix_lens, cache, q, cu_rows, lens, max_group_rows, max_prefix, max_rows, max_len, mask=None, **kw):
        b = shared_bounds(name, prefix, cache, q.shape[1], prefix_lens.shape[0], lens.shape[0], max_group_rows, max_prefix, max_rows, max_len, mask)
        return SHARED(prefix, cu_groups, prefix_lens, cache, q, cu_rows, lens, *b, mask=mask, **kw)

    def shared_ws(prefix, cache, n_heads, N, n_groups, B, mg, mp, mr, ml):
        return SHARED_WS(prefix, cache, n_heads, N, n_groups, B, *shared_bounds(name, prefix, cache, n_heads, n_groups, B, mg, mp, mr, ml, None))
    monkeypatch.setattr(eb, "kv_cross_attention", cross)
    monkeypatch.setattr(eb, "kv_cross_attention_workspace", cross_ws)
    monkeypatch.setattr(eb, "kv_shared_attention", shared)
    monkeypatch.setattr(eb, "kv_shared_attention_workspace", shared_ws)
    return name


@pytest.mark.parametrize("rows", [1, 2, 40])
def test_bad_pages_and_rows_are_reported(kernel, rows):
    rng = np.random.default_rng(10)
    cache, _ = make_cache(rng, "bf16", 128, 16, 1, [40, 40])
    q = torch.randn(2 * rows, 4, 128, device="cuda").to(torch.bfloat16)
    good = cache.page_table.clone()

    def call(c, n, max_rows=rows, out=None):
        return eb.kv_cross_attention(cache, q, dev(np.array(c, np.int32)), dev(np.array(n, np.int32)), max_rows, 40, out=out)

    def flagged(bits):
        with pytest.raises(eb.EagleError) as e:
            cache.check()
        assert e.value.status == eb.EAGLE_ERR_DEVICE and bits in str(e.value)
    want = call([0, rows, 2 * rows], [40, 40])
    assert cache.check() == 0
    cache.page_table[0, 1] = cache.k.shape[0]
    got = call([0, rows, 2 * rows], [40, 40])
    flagged("0x10")
    assert torch.equal(got[rows:], want[rows:])          # the other request is whole
    cache.page_table.copy_(good)
    call([0, rows, 2 * rows], [40, -1])
    flagged("0x2")
    if kernel == "wide" or rows <= 2:                    # (where the bound is above 65) behind the table's last page
        call([0, rows, 2 * rows], [40, 65])
        flagged("0x10")
    for c in ([0, rows, 2 * rows + 1], [0, rows, rows - 1], [-1, rows, 2 * rows]):
        call(c, [40, 40])
        flagged("0x2")
    assert torch.equal(call([0, rows, 2 * rows], [40, 40]), want) and cache.check() == 0


def test_groups_of_one_and_two_behind_prefixes_of_any_length(kernel):
    """Forty groups, prefixes of 0 to 4,000 keys, 8 heads; own keys on both sides of the choice."""
    import test_gpu_shared_attention as T
    plens = [(97 * i * i) % 4001 if i % 7 else 0 for i in range(40)]
    groups = [0]
    for i in range(40):
        groups.append(groups[-1] + 1 + i % 2)
    ctx = [(53 * i) % 300 for i in range(groups[-1])]
    for kinds, G in ((("bf16", "bf16"), 1), (("f4", "bf16"), 4), (("bf16", "f4"), 8), (("bf16", "bf16"), 4)):
        rng = np.random.default_rng(G)
        args, sizes, out, lse = T.run(rng, kinds, 64, (32, 64), 8, G, plens, groups, ctx, [1] * groups[-1], pad=1)
        for _ in range(3):
            o = eb.kv_shared_attention(*args, **sizes)
            assert torch.equal(o[:groups[-1]], out[:groups[-1]])
