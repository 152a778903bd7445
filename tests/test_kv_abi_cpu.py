"""CPU checks of the paged-cache entry points: struct layouts, and that every bad argument is
refused before any GPU work (pointers are never dereferenced)."""
import ctypes as C
import os

import pytest

from eagle_speculative_decoding_03_gb300 import binding as eb

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "eagle_draft.h")
P = 4096   # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    from eagle_speculative_decoding_03_gb300 import build
    build.build()
    return eb.load()


def test_struct_layout_matches_header(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    pairs = [("eagle_kv_cache_t", "KVCacheC"), ("eagle_rope_t", "RopeC"), ("eagle_kv_rows_t", "KVRows"),
             ("eagle_kv_attention_t", "KVAttention")]
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void) {"]
    for cname, pyname in pairs:
        lines.append(f'  printf("{pyname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{pyname} {f[0]} %zu\\n", offsetof({cname}, {f[0]}));' for f in getattr(eb, pyname)._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0; }"]))
    subprocess.run([cc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout
    for line in out.split("\n")[:-1]:
        n, f, v = line.split()
        cls = getattr(eb, n)
        assert int(v) == (C.sizeof(cls) if f == "size" else getattr(cls, f).offset), line


def cache(**kw):
    d = dict(kind=eb.CACHE_F4, n_kv_heads=8, head_dim=128, page_size=64, num_pages=100, max_pages=10, k=P, v=P, k_scale=P,
             v_scale=P, k_global=1.0, v_global=1.0, page_table=P)
    d.update(kw)
    return eb.KVCacheC(**d)


def rope(**kw):
    d = dict(rot_dim=128, interleaved=0, theta=1e4, amplitude=1.0)
    freq = kw.pop("freq", None)
    d.update(kw)
    r = eb.RopeC(**d)
    if freq is not None:
        r._keep = (C.c_double * len(freq))(*freq)
        r.inv_freq = r._keep
    return r


BAD_CACHE = [(dict(kind=7), 1), (dict(head_dim=96), 2), (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(n_kv_heads=0), 1),
             (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(num_pages=1 << 22), 2), (dict(k=None), 1), (dict(v=None), 1),
             (dict(k_scale=None), 1), (dict(page_table=None), 1), (dict(k=P + 8), 1), (dict(v_scale=P + 4), 1),
             (dict(k_global=0.0), 1), (dict(v_global=float("nan")), 1), (dict(v_global=float("inf")), 1)]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches_are_refused_everywhere(lib, kw, status):
    c = cache(**kw)
    w = eb.KVRows(B=1, N=1, cu_rows=P, lens=P, positions=P, dtype=1, k=P, v=P, k_stride=1024, v_stride=1024)
    assert lib.eagle_kv_append(C.byref(c), C.byref(w), C.byref(rope()), P, None) == status
    assert lib.eagle_kv_gather(C.byref(c), 1, P, 8, P, P, P, None) == status
    assert lib.eagle_kv_accept(C.byref(c), 1, 1, 4, P, P, P, P, P, None) == status
    a = eb.KVAttention(B=1, N=1, n_heads=8, max_rows=1, max_len=10, cu_rows=P, lens=P, q=P, q_stride=1024, out=2 * P, out_stride=1024)
    assert lib.eagle_kv_attention(C.byref(c), C.byref(a), P, None) == status
    assert lib.eagle_kv_attention_workspace(C.byref(c), C.byref(a)) == -1
    assert lib.eagle_draft_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), 2), (dict(rot_dim=24), 2), (dict(rot_dim=144), 2), (dict(interleaved=2), 1), (dict(theta=0.0), 1),
    (dict(theta=float("inf")), 1), (dict(amplitude=float("nan")), 1), (dict(freq=[-1.0] * 64), 1),
    (dict(freq=[float("nan")] * 64), 1), (dict(freq=[1e7] * 64), 1)])
def test_bad_ropes_are_refused(lib, kw, status):
    r = rope(**kw)
    assert lib.eagle_rotary(1, P, 1024, 1, 8, 128, P, C.byref(r), P, 1024, None) == status
    w = eb.KVRows(B=1, N=1, cu_rows=P, lens=P, positions=P, dtype=1, k=P, v=P, k_stride=1024, v_stride=1024)
    assert lib.eagle_kv_append(C.byref(cache()), C.byref(w), C.byref(r), P, None) == status


def test_rotary_arguments(lib):
    r = C.byref(rope())
    def call(dtype=1, x=P, xs=1024, N=1, H=8, hd=128, pos=P, rp=r, out=P, os_=1024):
        return lib.eagle_rotary(dtype, x, xs, N, H, hd, pos, rp, out, os_, None)
    for kw in (dict(x=None), dict(pos=None), dict(rp=None), dict(out=None), dict(dtype=9), dict(N=-1), dict(H=0), dict(x=P + 2),
               dict(xs=1000), dict(xs=1025), dict(os_=512), dict(os_=2048)):
        assert call(**kw) == 1, kw
    for hd in (8, 132, 264):
        assert call(hd=hd) == 2
    assert call(N=0) == 0          # nothing to do


def test_append_arguments(lib):
    c, r = cache(), rope()
    def call(rp=r, err=P, **kw):
        d = dict(B=1, N=1, cu_rows=P, lens=P, positions=P, dtype=1, n_heads=16, k=P, v=P, q=P, q_out=P, k_stride=1024,
                 v_stride=1024, q_stride=2048, q_out_stride=2048)
        d.update(kw)
        return lib.eagle_kv_append(C.byref(c), C.byref(eb.KVRows(**d)), None if rp is None else C.byref(rp), err, None)
    for kw in (dict(B=0), dict(N=-1), dict(cu_rows=None), dict(lens=None), dict(positions=None), dict(dtype=3), dict(n_heads=0),
               dict(k=None), dict(v=None), dict(q_out=None), dict(k=P + 8), dict(k_stride=1000), dict(v_stride=1020),
               dict(q_stride=1024), dict(q_out_stride=4096), dict(err=None), dict(rp=None)):
        assert call(**kw) == 1, kw
    assert call(N=0) == 0
    assert lib.eagle_kv_append(C.byref(c), None, None, P, None) == 1


def test_gather_and_accept_arguments(lib):
    c = cache()
    def ga(B=1, cu=P, total=8, k=P, v=P, err=P):
        return lib.eagle_kv_gather(C.byref(c), B, cu, total, k, v, err, None)
    for kw in (dict(B=0), dict(total=-1), dict(cu=None), dict(k=None), dict(v=None), dict(err=None), dict(k=P + 8)):
        assert ga(**kw) == 1, kw
    assert ga(total=0) == 0
    def ac(n=1, B=1, S=4, a=P, b=P, d=P, e=P, err=P, cs=None):
        return lib.eagle_kv_accept(C.byref(c) if cs is None else cs, n, B, S, a, b, d, e, err, None)
    for kw in (dict(n=0), dict(n=65), dict(B=0), dict(S=0), dict(S=65), dict(a=None), dict(b=None), dict(d=None), dict(e=None),
               dict(err=None)):
        assert ac(**kw) == 1, kw
    assert lib.eagle_kv_accept(None, 1, 1, 4, P, P, P, P, P, None) == 1
    for kw in (dict(n_kv_heads=4), dict(page_size=32), dict(max_pages=9), dict(page_table=P + 64), dict(num_pages=99), dict(kind=1)):
        assert ac(n=2, cs=(eb.KVCacheC * 2)(cache(), cache(k=2 * P, v=3 * P, **kw))) == 1, kw
    for kw in (dict(), dict(k=2 * P), dict(v=2 * P), dict(k=2 * P, v=P)):       # two caches over one pool
        assert ac(n=2, cs=(eb.KVCacheC * 2)(cache(k=P, v=4 * P), cache(**{**dict(k=P, v=4 * P), **kw}))) == 1, kw


def test_attention_arguments(lib):
    c = cache()
    def call(err=P, **kw):
        d = dict(B=1, N=1, n_heads=8, max_rows=1, max_len=10, cu_rows=P, lens=P, q=P, q_stride=1024, out=2 * P, out_stride=1024)
        d.update(kw)
        return lib.eagle_kv_attention(C.byref(c), C.byref(eb.KVAttention(**d)), err, None)
    for kw in (dict(B=0), dict(N=-1), dict(n_heads=0), dict(n_heads=12), dict(n_heads=8 * 65), dict(max_rows=0), dict(max_len=0),
               dict(cu_rows=None), dict(lens=None), dict(q=None), dict(out=None), dict(err=None), dict(out=P), dict(q=P + 8), dict(q_stride=1000),
               dict(q_stride=1028), dict(out_stride=512), dict(scale=-1.0), dict(scale=float("nan")),
               dict(mask=P, mask_slots=0), dict(mask=P, mask_slots=65), dict(mask=P, mask_slots=4, max_rows=5),
               dict(max_len=100000)):      # (ranges need a workspace)
        assert call(**kw) == 1, kw
    assert call(N=0) == 0
    assert lib.eagle_kv_attention(C.byref(c), None, P, None) == 1
    a = eb.KVAttention(B=2, N=2, n_heads=32, max_rows=1, max_len=100000)
    need = lib.eagle_kv_attention_workspace(C.byref(c), C.byref(a))
    assert need > 0
    a.cu_rows = a.lens = a.q = a.workspace = P
    a.out = 2 * P
    a.q_stride = a.out_stride = 4096
    a.workspace_bytes = need - 1
    assert lib.eagle_kv_attention(C.byref(c), C.byref(a), P, None) == 1
    a.workspace_bytes, a.workspace = need, P + 8
    assert lib.eagle_kv_attention(C.byref(c), C.byref(a), P, None) == 1


def test_rows_past_32_bit_arithmetic_are_refused(lib):
    """The kernels index a row's elements and the rows in 32 bits: larger calls are refused before
    any launch."""
    big = 1 << 24                                     # heads: 2^31 elements a row at 128
    for H, hd, N in ((big, 128, 1), (1 << 30, 16, 1), (1, 128, 2 ** 31 - 1), (1, 128, 2 ** 31 - 8)):
        rp = C.byref(rope(rot_dim=16))
        assert lib.eagle_rotary(1, P, H * hd, N, H, hd, P, rp, P, H * hd, None) == 2, (H, hd, N)
    def append(c, **kw):
        d = dict(B=1, N=1, cu_rows=P, lens=P, positions=P, dtype=1, n_heads=16, k=P, v=P, q=P, q_out=P, k_stride=1 << 40,
                 v_stride=1 << 40, q_stride=1 << 40, q_out_stride=1 << 40)
        d.update(kw)
        return lib.eagle_kv_append(C.byref(c), C.byref(eb.KVRows(**d)), C.byref(rope()), P, None)
    assert append(cache(), n_heads=big) == 2
    assert append(cache(), N=2 ** 31 - 1) == 2
    assert append(cache(n_kv_heads=1 << 24, num_pages=1, page_size=16)) == 2
    assert lib.eagle_kv_gather(C.byref(cache()), 1, P, 2 ** 31 - 1, P, 2 * P, P, None) == 2


def test_buffers_that_calls_write_are_not_shared(lib):
    """Keys and values of one launch are written by CTAs in no order: one buffer for both, scales
    in common, or new lengths over the path that other CTAs still read are refused."""
    own = dict(k=P, v=2 * P, k_scale=3 * P, v_scale=4 * P)
    w = eb.KVRows(B=1, N=1, cu_rows=P, lens=P, positions=P, dtype=1, k=P, v=P, k_stride=1024, v_stride=1024)
    for kw in (dict(v=P), dict(v_scale=3 * P)):
        c = cache(**{**own, **kw})
        assert lib.eagle_kv_append(C.byref(c), C.byref(w), None, P, None) == 1, kw
        assert lib.eagle_kv_accept(C.byref(c), 1, 1, 4, P, 2 * P, 3 * P, 4 * P, P, None) == 1, kw
    two = dict(k=5 * P, v=6 * P, k_scale=7 * P, v_scale=8 * P)
    for kw in (dict(k_scale=3 * P), dict(v_scale=4 * P), dict(k_scale=4 * P), dict(v_scale=3 * P)):
        cs = (eb.KVCacheC * 2)(cache(**own), cache(**{**two, **kw}))
        assert lib.eagle_kv_accept(cs, 2, 1, 4, P, 2 * P, 3 * P, 4 * P, P, None) == 1, kw
    c = cache(**own)
    assert lib.eagle_kv_gather(C.byref(c), 1, P, 8, 5 * P, 5 * P, P, None) == 1
    for new in (2 * P, 3 * P):
        assert lib.eagle_kv_accept(C.byref(c), 1, 1, 4, P, 2 * P, 3 * P, new, P, None) == 1


def test_caches_and_streams_of_another_device_are_refused(monkeypatch):
    """Tensors of the current device beside a cache (or on a stream) of another: refused before the
    library is reached.  Devices are played here by numbers: CPU tensors are on device -1."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    at = [-1]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    def reached():
        raise AssertionError("the library was reached")
    monkeypatch.setattr(eb, "load", reached)
    def pool():
        return torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, one = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x, cu = pool()[:1, :, 0].contiguous(), torch.tensor([0, 1], dtype=torch.int32)
    here, there = eb.KVCache(pool(), pool(), table), eb.KVCache(pool(), pool(), table)
    there.device_index = 1                            # (its own tensors are only looked at when it is made)
    calls = [lambda c, s: eb.kv_append(c, x, x, cu, one, stream=s), lambda c, s: eb.kv_gather(c, cu, 1, stream=s),
             lambda c, s: eb.kv_attention(c, x, cu, one, 1, 8, stream=s), lambda c, s: eb.kv_accept(c, one, one, one[None], stream=s),
             lambda c, s: eb.kv_accept([here, c], one, one, one[None], stream=s)]
    for f in calls:
        with pytest.raises(AssertionError, match="library was reached"):
            f(here, None)
        with pytest.raises(eb.EagleError, match="cache must be on the current"):
            f(there, None)
        with pytest.raises(eb.EagleError, match="stream must be of the current"):
            f(here, SimpleNamespace(cuda_stream=0, device_index=0))
    with pytest.raises(eb.EagleError, match="stream must be of the current"):
        eb.rotary(x, one, eb.Rope(64), stream=SimpleNamespace(cuda_stream=0, device_index=0))
