"""CPU checks of cross attention, shared attention and the merge: struct layouts, and that every
bad argument is refused before any GPU work (pointers are never dereferenced)."""
import ctypes as C

import pytest

from eagle_speculative_decoding_03_gb300 import binding as eb
from test_kv_abi_cpu import BAD_CACHE, HEADER, P, cache, lib  # noqa: F401


def test_struct_layout_matches_header(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    pairs = [("eagle_kv_cross_t", "KVCross"), ("eagle_kv_groups_t", "KVGroups"), ("eagle_attention_parts_t", "AttentionParts")]
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void) {"]
    for cname, pyname in pairs:
        lines.append(f'  printf("{pyname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{pyname} {f[0]} %zu\\n", offsetof({cname}, {f[0]}));' for f in getattr(eb, pyname)._fields_]
    lines.append('  printf("MAX_PARTS size %d\\n", EAGLE_MAX_PARTS);')
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0; }"]))
    subprocess.run([cc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout
    for line in out.split("\n")[:-1]:
        n, f, v = line.split()
        cls = getattr(eb, n)
        assert int(v) == (cls if n == "MAX_PARTS" else C.sizeof(cls) if f == "size" else getattr(cls, f).offset), line


def cross(**kw):
    d = dict(B=1, N=2, n_heads=16, max_rows=1, max_len=10, cu_rows=P, lens=P, q=P, q_stride=2048, out=4 * P, out_stride=2048)
    d.update(kw)
    return eb.KVCross(**d)


def own(**kw):
    d = dict(B=2, N=2, n_heads=16, max_rows=1, max_len=10, cu_rows=P, lens=P, q=P, q_stride=2048, out=4 * P, out_stride=2048,
             workspace=P, workspace_bytes=1 << 40)
    d.update(kw)
    return eb.KVAttention(**d)


def groups(**kw):
    d = dict(n_groups=1, cu_groups=P, lens=P, max_rows=2, max_len=10)
    d.update(kw)
    return eb.KVGroups(**d)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches_are_refused(lib, kw, status):  # noqa: F811
    good, bad = C.byref(cache()), C.byref(cache(**kw))
    assert lib.eagle_kv_cross_attention(bad, C.byref(cross()), P, None) == status
    assert lib.eagle_kv_cross_attention_workspace(bad, C.byref(cross())) == -1
    for a, b in ((good, bad), (bad, good)):
        assert lib.eagle_kv_shared_attention(a, C.byref(groups()), b, C.byref(own()), P, None) in (status, 1)
        assert lib.eagle_kv_shared_attention_workspace(a, C.byref(groups()), b, C.byref(own())) == -1
    assert lib.eagle_draft_last_error()


BAD_ROWS = [(dict(B=0), 1), (dict(N=-1), 1), (dict(max_rows=0), 1), (dict(max_len=0), 1), (dict(max_len=(1 << 30) + 1), 2),
            (dict(n_heads=0), 1), (dict(n_heads=12), 1), (dict(n_heads=8 * 65), 1), (dict(scale=-1.0), 1),
            (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(cu_rows=None), 1), (dict(lens=None), 1),
            (dict(q=None), 1), (dict(out=None), 1), (dict(q=P + 8), 1), (dict(q_stride=2040), 1), (dict(q_stride=2052), 1),
            (dict(out_stride=2047), 1), (dict(out=P), 1), (dict(out=P + 4096), 1), (dict(N=1 << 28), 2)]


@pytest.mark.parametrize("kw,status", BAD_ROWS)
def test_bad_rows_are_refused(lib, kw, status):  # noqa: F811
    c = C.byref(cache())
    assert lib.eagle_kv_cross_attention(c, C.byref(cross(**kw)), P, None) == status
    assert lib.eagle_kv_shared_attention(c, C.byref(groups()), c, C.byref(own(**kw)), P, None) == status


def test_other_refusals(lib):  # noqa: F811
    c = C.byref(cache())
    assert lib.eagle_kv_cross_attention(c, C.byref(cross()), None, None) == 1
    assert lib.eagle_kv_cross_attention(c, None, P, None) == 1
    assert lib.eagle_kv_cross_attention(None, C.byref(cross()), P, None) == 1
    assert lib.eagle_kv_cross_attention(c, C.byref(cross(N=0)), P, None) == 0
    many = dict(B=1, N=64, max_len=1 << 20, out=1 << 20)                           # ranges that need a workspace
    need = lib.eagle_kv_cross_attention_workspace(c, C.byref(cross(**many)))
    assert need > 0
    for ws in (dict(), dict(workspace=P, workspace_bytes=need - 1), dict(workspace=P + 8, workspace_bytes=need)):
        assert lib.eagle_kv_cross_attention(c, C.byref(cross(**many, **ws)), P, None) == 1
    assert lib.eagle_kv_cross_attention(c, C.byref(cross(B=70000)), P, None) == 2
    # q and out as slices of one buffer: rows that interleave are taken, rows that meet refused
    wide = dict(q_stride=8192, out_stride=8192, N=0)
    assert lib.eagle_kv_cross_attention(c, C.byref(cross(out=P + 4096, **wide)), P, None) == 0
    for out in (P + 4080, P + 16384 - 4080):
        assert lib.eagle_kv_cross_attention(c, C.byref(cross(out=out, **dict(wide, N=3))), P, None) == 1

    def sh(a=c, g=None, b=c, w=None, err=P):
        return lib.eagle_kv_shared_attention(a, C.byref(groups() if g is None else g), b, C.byref(own() if w is None else w), err, None)
    for g, status in ((dict(n_groups=0), 1), (dict(n_groups=-1), 1), (dict(cu_groups=None), 1), (dict(lens=None), 1),
                      (dict(max_rows=0), 1), (dict(max_len=0), 1), (dict(max_len=(1 << 30) + 1), 2)):
        assert sh(g=groups(**g)) == status, g
    for w in (dict(mask=P, mask_slots=0), dict(mask=P, mask_slots=65), dict(mask=P, mask_slots=2, max_rows=3),
              dict(workspace=None), dict(workspace_bytes=16), dict(workspace=P + 4)):
        assert sh(w=own(**w)) == 1, w
    assert sh(a=C.byref(cache(n_kv_heads=4))) == 1
    assert sh(b=C.byref(cache(head_dim=64))) == 1
    assert sh(err=None) == 1
    assert sh(w=own(N=0)) == 0
    assert lib.eagle_kv_shared_attention(c, None, c, C.byref(own()), P, None) == 1
    assert lib.eagle_kv_shared_attention(c, C.byref(groups()), c, None, P, None) == 1
    # a prefix and own keys of different kinds and page sizes belong together
    bf = C.byref(cache(kind=eb.CACHE_BF16, k_scale=None, v_scale=None, page_size=16))
    for a, b in ((bf, c), (c, bf)):
        assert lib.eagle_kv_shared_attention_workspace(a, C.byref(groups()), b, C.byref(own())) > 0


def test_merge_refusals(lib):  # noqa: F811
    F = 1 << 20

    def call(outs=(F, 2 * F), lses=(3 * F, 4 * F), strides=None, **kw):
        d = dict(parts=len(outs), N=3, H=2, head_dim=64, dtype=1, out_dtype=1, out=5 * F, out_stride=128, lse=6 * F)
        d.update(kw)
        d["outs"] = (C.c_void_p * len(outs))(*outs)
        d["lses"] = (C.c_void_p * len(lses))(*lses)
        if strides:
            d["strides"] = (C.c_int64 * len(strides))(*strides)
        return lib.eagle_attention_merge(C.byref(eb.AttentionParts(**d)), None)
    assert call(N=0) == 0
    assert lib.eagle_attention_merge(None, None) == 1
    for kw in (dict(parts=0), dict(parts=17), dict(N=-1), dict(H=0), dict(dtype=2), dict(out_dtype=7), dict(out=None), dict(out=5 * F + 8),
               dict(out_stride=120), dict(out_stride=132), dict(outs=(F, None)), dict(lses=(None, F)), dict(outs=(F, 2 * F + 8)),
               dict(lses=(3 * F, 4 * F + 2)), dict(strides=(128, 120)), dict(strides=(128, 132)),
               dict(outs=(F, 5 * F + 16)), dict(outs=(F, 5 * F), out_dtype=0, out_stride=128), dict(outs=(5 * F, 2 * F), strides=(256, 128)),
               dict(lse=5 * F), dict(lse=5 * F + 760), dict(lse=3 * F), dict(lse=4 * F + 20), dict(lse=F + 16), dict(lses=(3 * F, 5 * F + 4))):
        assert call(**kw) == 1, kw
    for kw in (dict(head_dim=60), dict(head_dim=264), dict(head_dim=0), dict(N=1 << 30, H=2), dict(H=1 << 28)):
        kw = dict(dict(out_stride=1 << 40), **kw)
        assert call(**kw) == 2, kw
