"""What cross and shared attention write is their own: lse and the workspace that overlap another buffer of the call
are refused before any GPU work (pointers are never dereferenced)."""
import ctypes as C

import pytest

from eagle_speculative_decoding_03_gb300 import binding as eb
from test_cross_abi_cpu import cross, groups, own
from test_kv_abi_cpu import P, cache, lib  # noqa: F401

M = 1 << 20


def overlap_error(lib):  # noqa: F811
    return b"overlap" in lib.eagle_draft_last_error()


# two rows of 16 heads of 128: q at M, out at 2 M (8,192 bytes each), lse 128 bytes
@pytest.mark.parametrize("lse", [M, M + 8188, 2 * M, 2 * M + 4096, M - 124, 2 * M - 4])
def test_lse_in_q_or_out(lib, lse):  # noqa: F811
    c = C.byref(cache())
    assert lib.eagle_kv_cross_attention(c, C.byref(cross(q=M, out=2 * M, lse=lse, workspace=16 * M, workspace_bytes=1 << 40)), P, None) == 1
    assert overlap_error(lib)
    a = own(q=M, out=2 * M, lse=lse, workspace=16 * M)
    assert lib.eagle_kv_shared_attention(c, C.byref(groups()), c, C.byref(a), P, None) == 1
    assert overlap_error(lib)


@pytest.mark.parametrize("at", [0, 1, 2])
def test_workspace_in_q_out_or_lse(lib, at):  # noqa: F811
    c = C.byref(cache())
    buffers = dict(q=M, out=2 * M, lse=3 * M)
    name = ("q", "out", "lse")[at]
    many = dict(B=1, N=2, max_rows=2, max_len=1 << 20)           # ranges that need a workspace
    need = lib.eagle_kv_cross_attention_workspace(c, C.byref(cross(**many)))
    assert need > 0
    for ws in (buffers[name], buffers[name] - 16):
        w = dict(buffers, workspace=ws, workspace_bytes=1 << 40)
        w[name] = 64 * M if ws < 0 else buffers[name]
        assert lib.eagle_kv_cross_attention(c, C.byref(cross(**many, **w)), P, None) == 1
        assert overlap_error(lib)
        assert lib.eagle_kv_shared_attention(c, C.byref(groups()), c, C.byref(own(**{k: v for k, v in w.items() if k != "workspace_bytes"})), P, None) == 1
        assert overlap_error(lib)
