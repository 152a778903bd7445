"""ctypes binding of libeagle_draft.so (include/eagle_draft.h).

Argument marshalling only: every step of the draft tree runs in the library's CUDA
kernels.  torch is used for device memory and streams; tensors are passed as raw
pointers.  ``load()`` raises if the library has not been built.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

from .configs import DraftConfig

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libeagle_draft.so")

EAGLE_OK, EAGLE_ERR_INVALID_ARG, EAGLE_ERR_UNSUPPORTED, EAGLE_ERR_OOM, EAGLE_ERR_CUDA, EAGLE_ERR_DEVICE = range(6)
DTYPE_F32, DTYPE_BF16 = 0, 1
TREE_STATIC, TREE_DYNAMIC = 1, 2
FEAT_F, FEAT_FUSED = 1, 3
FLAG_NO_GRAPH, FLAG_NO_PDL, FLAG_GEMM_TWO_CTA = 1, 2, 4
MAX_DEPTH = 16
KERNEL_KINDS = 14
DEVERR_TIMEOUT, DEVERR_PREFIX, DEVERR_TOKEN, DEVERR_SELECT, DEVERR_PAGE = 1, 2, 4, 8, 16
CACHE_BF16, CACHE_F4 = 1, 2


class Config(C.Structure):
    _fields_ = [("d", C.c_int32), ("n_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("d_ff", C.c_int32), ("vocab", C.c_int32),
                ("rms_eps", C.c_float), ("rope_theta", C.c_float), ("dtype", C.c_int32),
                ("tree_kind", C.c_int32), ("feat_kind", C.c_int32), ("depth", C.c_int32),
                ("k", C.c_int32), ("m", C.c_int32), ("branching", C.c_int32 * MAX_DEPTH),
                ("max_batch", C.c_int32), ("max_prefix", C.c_int32), ("flags", C.c_int32)]


class Weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("embed", "w_fc", "w_fc3", "attn_norm", "w_qkv", "w_o",
                                         "mlp_norm", "w_gate", "w_up", "w_down", "w_lm")]


class Inputs(C.Structure):
    _fields_ = [("B", C.c_int32), ("root_feat", C.c_void_p), ("root_tok", C.c_void_p),
                ("k_cache", C.c_void_p), ("v_cache", C.c_void_p), ("cu_seqlens", C.c_void_p),
                ("seeds", C.c_void_p)]


class Outputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("tokens", "parents", "positions", "logv", "mask")]


TRACE_FIELDS = ("h", "q", "attn", "y", "a", "lse", "children", "child_logp", "frontier",
                "final_nodes", "tree_k", "tree_v")


class Trace(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in TRACE_FIELDS]


class Info(C.Structure):
    _fields_ = [("slots", C.c_int32), ("generated", C.c_int32), ("rows", C.c_int32),
                ("n_max", C.c_int32), ("k_max", C.c_int32), ("f_max", C.c_int32),
                ("launches_per_tree", C.c_int32), ("tensor_core_gemm", C.c_int32),
                ("workspace_bytes", C.c_int64)]


class VerifyConfig(C.Structure):
    _fields_ = [("d", C.c_int32), ("n_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("d_ff", C.c_int32), ("vocab", C.c_int32),
                ("rms_eps", C.c_float), ("rope_theta", C.c_float), ("dtype", C.c_int32),
                ("max_batch", C.c_int32), ("max_slots", C.c_int32), ("max_prefix", C.c_int32),
                ("flags", C.c_int32)]


class VerifyWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("embed", "attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gate",
                                         "w_up", "w_down", "final_norm", "w_lm")]


class VerifyInputs(C.Structure):
    _fields_ = [("B", C.c_int32), ("S", C.c_int32)] + \
        [(n, C.c_void_p) for n in ("tokens", "positions", "mask", "parents", "k_cache", "v_cache", "cu_seqlens")]


VERIFY_OUTPUTS = ("top_id", "top_logp", "lse", "hidden", "logits", "accept_len", "accept_slots", "correction")


class VerifyOutputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in VERIFY_OUTPUTS]


class DFlashConfigC(C.Structure):
    _fields_ = [("d", C.c_int32), ("n_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("d_ff", C.c_int32), ("vocab", C.c_int32),
                ("rms_eps", C.c_float), ("rope_theta", C.c_float), ("dtype", C.c_int32),
                ("n_layers", C.c_int32), ("gamma", C.c_int32), ("k", C.c_int32), ("mask_token", C.c_int32),
                ("max_batch", C.c_int32), ("max_prefix", C.c_int32), ("flags", C.c_int32)]


class DFlashWeights(C.Structure):
    _fields_ = [("embed", C.c_void_p), ("w_lm", C.c_void_p), ("final_norm", C.c_void_p)] + \
        [(n, C.POINTER(C.c_void_p)) for n in ("attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gate", "w_up", "w_down")]


class DFlashInputs(C.Structure):
    _fields_ = [("B", C.c_int32), ("anchor", C.c_void_p), ("ctx_k", C.POINTER(C.c_void_p)),
                ("ctx_v", C.POINTER(C.c_void_p)), ("cu_seqlens", C.c_void_p)]


class DFlashOutputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("tokens", "logp", "lse", "hidden")]


class KVCacheC(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("kind", "n_kv_heads", "head_dim", "page_size", "num_pages", "max_pages")] + \
        [(n, C.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
        [("k_global", C.c_float), ("v_global", C.c_float), ("page_table", C.c_void_p)]


class RopeC(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("interleaved", C.c_int32), ("theta", C.c_double),
                ("inv_freq", C.POINTER(C.c_double)), ("amplitude", C.c_float)]


class KVRows(C.Structure):
    _fields_ = [("B", C.c_int32), ("N", C.c_int32), ("cu_rows", C.c_void_p), ("lens", C.c_void_p),
                ("positions", C.c_void_p), ("dtype", C.c_int32), ("n_heads", C.c_int32)] + \
        [(n, C.c_void_p) for n in ("k", "v", "q", "q_out")] + \
        [(n, C.c_int64) for n in ("k_stride", "v_stride", "q_stride", "q_out_stride")]


class KVAttention(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("B", "N", "n_heads", "max_rows", "max_len", "mask_slots")] + \
        [("cu_rows", C.c_void_p), ("lens", C.c_void_p), ("q", C.c_void_p), ("q_stride", C.c_int64),
         ("mask", C.c_void_p), ("scale", C.c_float), ("out", C.c_void_p), ("out_stride", C.c_int64),
         ("lse", C.c_void_p), ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64)]


class KVCross(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("B", "N", "n_heads", "max_rows", "max_len")] + \
        [("cu_rows", C.c_void_p), ("lens", C.c_void_p), ("q", C.c_void_p), ("q_stride", C.c_int64),
         ("scale", C.c_float), ("out", C.c_void_p), ("out_stride", C.c_int64), ("lse", C.c_void_p),
         ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64)]


class KVGroups(C.Structure):
    _fields_ = [("n_groups", C.c_int32), ("cu_groups", C.c_void_p), ("lens", C.c_void_p), ("max_rows", C.c_int32),
                ("max_len", C.c_int32)]


MAX_PARTS = 16


class AttentionParts(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("parts", "N", "H", "head_dim", "dtype", "out_dtype")] + \
        [("outs", C.POINTER(C.c_void_p)), ("strides", C.POINTER(C.c_int64)), ("lses", C.POINTER(C.c_void_p)),
         ("out", C.c_void_p), ("out_stride", C.c_int64), ("lse", C.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Load the library (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (python -m "
                           "eagle_speculative_decoding_03_gb300.build)")
    lib = C.CDLL(path)
    P = C.c_void_p
    lib.eagle_draft_create.argtypes = [C.POINTER(Config), C.POINTER(Weights), C.POINTER(P)]
    lib.eagle_draft_create.restype = C.c_int
    lib.eagle_draft_tree.argtypes = [P, C.POINTER(Inputs), C.POINTER(Outputs), C.POINTER(Trace), P]
    lib.eagle_draft_tree.restype = C.c_int
    lib.eagle_draft_lm_head_topk.argtypes = [P, P, C.c_int32, C.c_int32, P, P, P, P]
    lib.eagle_draft_lm_head_topk.restype = C.c_int
    lib.eagle_draft_query.argtypes = [P, C.POINTER(Info)]
    lib.eagle_draft_query.restype = C.c_int
    lib.eagle_draft_check.argtypes = [P, C.POINTER(C.c_uint32)]
    lib.eagle_draft_check.restype = C.c_int
    lib.eagle_draft_set_wait_limit.argtypes = [P, C.c_int64]
    lib.eagle_draft_set_wait_limit.restype = C.c_int
    lib.eagle_draft_destroy.argtypes = [P]
    lib.eagle_draft_destroy.restype = None
    lib.eagle_draft_profile.argtypes = [P, C.c_int32]
    lib.eagle_draft_profile.restype = C.c_int
    lib.eagle_draft_profile_read.argtypes = [P, C.POINTER(C.c_float), C.POINTER(C.c_int32)]
    lib.eagle_draft_profile_read.restype = C.c_int
    lib.eagle_draft_kernel_name.argtypes = [C.c_int32]
    lib.eagle_draft_kernel_name.restype = C.c_char_p
    lib.eagle_lm_head_topk_noalloc.argtypes = [P, C.c_int32, C.c_int32, P, C.c_int32, C.c_int32, P, P, P, P]
    lib.eagle_lm_head_topk_noalloc.restype = C.c_int
    lib.eagle_verify_create.argtypes = [C.POINTER(VerifyConfig), C.POINTER(VerifyWeights), C.POINTER(P)]
    lib.eagle_verify_create.restype = C.c_int
    lib.eagle_verify_tree.argtypes = [P, C.POINTER(VerifyInputs), C.POINTER(VerifyOutputs), P]
    lib.eagle_verify_tree.restype = C.c_int
    lib.eagle_verify_check.argtypes = [P, C.POINTER(C.c_uint32)]
    lib.eagle_verify_check.restype = C.c_int
    lib.eagle_verify_destroy.argtypes = [P]
    lib.eagle_verify_destroy.restype = None
    lib.eagle_dflash_create.argtypes = [C.POINTER(DFlashConfigC), C.POINTER(DFlashWeights), C.POINTER(P)]
    lib.eagle_dflash_create.restype = C.c_int
    lib.eagle_dflash_draft.argtypes = [P, C.POINTER(DFlashInputs), C.POINTER(DFlashOutputs), P]
    lib.eagle_dflash_draft.restype = C.c_int
    lib.eagle_dflash_check.argtypes = [P, C.POINTER(C.c_uint32)]
    lib.eagle_dflash_check.restype = C.c_int
    lib.eagle_dflash_destroy.argtypes = [P]
    lib.eagle_dflash_destroy.restype = None
    lib.eagle_speculative_accept.argtypes = [C.c_int32, C.c_int32, C.c_int32, P, P, P, P, P, P, P, P, P, P]
    lib.eagle_speculative_accept.restype = C.c_int
    lib.eagle_rotary.argtypes = [C.c_int32, P, C.c_int64, C.c_int32, C.c_int32, C.c_int32, P, C.POINTER(RopeC), P,
                                 C.c_int64, P]
    lib.eagle_rotary.restype = C.c_int
    lib.eagle_kv_append.argtypes = [C.POINTER(KVCacheC), C.POINTER(KVRows), C.POINTER(RopeC), P, P]
    lib.eagle_kv_append.restype = C.c_int
    lib.eagle_kv_gather.argtypes = [C.POINTER(KVCacheC), C.c_int32, P, C.c_int32, P, P, P, P]
    lib.eagle_kv_gather.restype = C.c_int
    lib.eagle_kv_accept.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, P, P, P, P, P, P]
    lib.eagle_kv_accept.restype = C.c_int
    lib.eagle_kv_attention_workspace.argtypes = [C.POINTER(KVCacheC), C.POINTER(KVAttention)]
    lib.eagle_kv_attention_workspace.restype = C.c_int64
    lib.eagle_kv_attention.argtypes = [C.POINTER(KVCacheC), C.POINTER(KVAttention), P, P]
    lib.eagle_kv_attention.restype = C.c_int
    lib.eagle_kv_cross_attention_workspace.argtypes = [C.POINTER(KVCacheC), C.POINTER(KVCross)]
    lib.eagle_kv_cross_attention_workspace.restype = C.c_int64
    lib.eagle_kv_cross_attention.argtypes = [C.POINTER(KVCacheC), C.POINTER(KVCross), P, P]
    lib.eagle_kv_cross_attention.restype = C.c_int
    lib.eagle_kv_shared_attention_workspace.argtypes = [C.POINTER(KVCacheC), C.POINTER(KVGroups), C.POINTER(KVCacheC),
                                                        C.POINTER(KVAttention)]
    lib.eagle_kv_shared_attention_workspace.restype = C.c_int64
    lib.eagle_kv_shared_attention.argtypes = [C.POINTER(KVCacheC), C.POINTER(KVGroups), C.POINTER(KVCacheC),
                                              C.POINTER(KVAttention), P, P]
    lib.eagle_kv_shared_attention.restype = C.c_int
    lib.eagle_attention_merge.argtypes = [C.POINTER(AttentionParts), P]
    lib.eagle_attention_merge.restype = C.c_int
    lib.eagle_draft_last_error.argtypes = []
    lib.eagle_draft_last_error.restype = C.c_char_p
    _lib = lib
    return lib


class EagleError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"eagle status {status}: {msg}")
        self.status = status


def _check(status: int):
    if status != EAGLE_OK:
        raise EagleError(status, load().eagle_draft_last_error().decode())


def make_config(cfg: DraftConfig, max_batch: int | None = None, max_prefix: int | None = None,
                flags: int = 0) -> Config:
    c = Config()
    c.d, c.n_heads, c.n_kv_heads, c.head_dim = cfg.d, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim
    c.d_ff, c.vocab, c.rms_eps, c.rope_theta = cfg.d_ff, cfg.vocab, cfg.rms_eps, cfg.rope_theta
    c.dtype = DTYPE_BF16 if cfg.dtype == "bf16" else DTYPE_F32
    c.tree_kind = TREE_STATIC if cfg.tree == "static" else TREE_DYNAMIC
    c.feat_kind = FEAT_FUSED if cfg.feat == "fused" else FEAT_F
    c.depth, c.k, c.m = cfg.depth, cfg.k, cfg.m
    for i, b in enumerate(cfg.branching):
        c.branching[i] = b
    c.max_batch = cfg.B if max_batch is None else max_batch
    c.max_prefix = cfg.prefix[1] if max_prefix is None else max_prefix
    c.flags = flags
    return c


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def device_weights(W: dict, device="cuda"):
    """numpy weights (bf16 as uint16 bits) -> device tensors (bf16 kept as int16 bits;
    uint64 seeds kept as int64 bits)."""
    import torch
    out = {}
    for k, v in W.items():
        arr = v.view(np.int16) if v.dtype == np.uint16 else v.view(np.int64) if v.dtype == np.uint64 else v
        out[k] = torch.from_numpy(np.ascontiguousarray(arr)).to(device)
    return out


def device_inputs(I: dict, device="cuda"):
    return device_weights(I, device)


def lm_head_topk_noalloc(w_lm, a, k: int, stream=None):
    """LM-head top-k without a handle and without any device allocation inside the
    library (for callers that cannot allocate); outputs are allocated here by torch.
    The library reads w_lm as bf16 and a as float32: other dtypes are rejected here.
    If a kernel of the call gave up, every row comes back as id -1 and NaN logp / lse."""
    import torch
    if w_lm.dtype not in (torch.bfloat16, torch.int16) or w_lm.dim() != 2:
        raise EagleError(EAGLE_ERR_INVALID_ARG, "noalloc: w_lm must be a 2-D bf16 tensor (or its int16 bits)")
    if a.dtype != torch.float32 or a.dim() != 2 or a.shape[1] != w_lm.shape[1]:
        raise EagleError(EAGLE_ERR_INVALID_ARG, "noalloc: a must be float32 [N, d] with d = w_lm.shape[1]")
    if not (w_lm.is_contiguous() and a.is_contiguous()):
        raise EagleError(EAGLE_ERR_INVALID_ARG, "noalloc: w_lm and a must be contiguous")
    N, d = int(a.shape[0]), int(a.shape[1])
    ids = torch.empty((N, k), dtype=torch.int32, device=a.device)
    logp = torch.empty((N, k), dtype=torch.float32, device=a.device)
    lse = torch.empty((N,), dtype=torch.float32, device=a.device)
    st = None if stream is None else stream.cuda_stream
    _check(load().eagle_lm_head_topk_noalloc(_ptr(w_lm), int(w_lm.shape[0]), d, _ptr(a), N, k,
                                             _ptr(ids), _ptr(logp), _ptr(lse), st))
    return ids, logp, lse


class EagleDraft:
    """One handle of the C library bound to device weights (torch tensors)."""

    def __init__(self, cfg: DraftConfig, dW: dict, max_batch: int | None = None,
                 max_prefix: int | None = None, flags: int = 0):
        lib = load()
        self.cfg = cfg
        self._dW = dW  # keep the weights alive
        w = Weights(**{n: _ptr(dW.get(n)) for n, _ in Weights._fields_})
        self._ccfg = make_config(cfg, max_batch, max_prefix, flags)
        h = C.c_void_p()
        _check(lib.eagle_draft_create(C.byref(self._ccfg), C.byref(w), C.byref(h)))
        self.h = h
        info = Info()
        _check(lib.eagle_draft_query(self.h, C.byref(info)))
        self.info = {n: getattr(info, n) for n, _ in Info._fields_}

    def close(self):
        if getattr(self, "h", None):
            load().eagle_draft_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc_outputs(self, B: int, device="cuda"):
        import torch
        S = self.info["slots"]
        return {"tokens": torch.empty((B, S), dtype=torch.int32, device=device),
                "parents": torch.empty((B, S), dtype=torch.int32, device=device),
                "positions": torch.empty((B, S), dtype=torch.int32, device=device),
                "logv": torch.empty((B, S), dtype=torch.float32, device=device),
                "mask": torch.empty((B, S, S), dtype=torch.uint8, device=device)}

    def alloc_trace(self, device="cuda"):
        import torch
        c, i = self.cfg, self.info
        D, N, k = c.depth, i["n_max"], i["k_max"]
        Bm, hq = self._ccfg.max_batch, c.n_heads * c.head_dim
        f = dict(dtype=torch.float32, device=device)
        n = dict(dtype=torch.int32, device=device)
        return {"h": torch.zeros((D, N, c.d), **f), "q": torch.zeros((D, N, hq), **f),
                "attn": torch.zeros((D, N, hq), **f), "y": torch.zeros((D, N, c.d), **f),
                "a": torch.zeros((D, N, c.d), **f), "lse": torch.zeros((D, N), **f),
                "children": torch.full((D, N, k), -1, **n), "child_logp": torch.zeros((D, N, k), **f),
                "frontier": torch.full((D, Bm, i["f_max"]), -1, **n),
                "final_nodes": torch.full((Bm, i["slots"]), -1, **n),
                "tree_k": torch.zeros((Bm, i["rows"], c.n_kv_heads, c.head_dim), **f),
                "tree_v": torch.zeros((Bm, i["rows"], c.n_kv_heads, c.head_dim), **f)}

    def tree(self, dI: dict, out: dict | None = None, trace: dict | None = None, stream=None):
        """Enqueue one draft tree; returns the output tensors (device)."""
        B = int(dI["root_tok"].shape[0])
        out = self.alloc_outputs(B, dI["root_tok"].device) if out is None else out
        inp = Inputs(B=B, root_feat=_ptr(dI["root_feat"]), root_tok=_ptr(dI["root_tok"]),
                     k_cache=_ptr(dI["k_cache"]), v_cache=_ptr(dI["v_cache"]),
                     cu_seqlens=_ptr(dI["cu_seqlens"]), seeds=_ptr(dI.get("seeds")))
        o = Outputs(**{n: _ptr(out[n]) for n, _ in Outputs._fields_})
        tr = None if trace is None else C.byref(Trace(**{n: _ptr(trace.get(n)) for n in TRACE_FIELDS}))
        st = None if stream is None else stream.cuda_stream
        _check(load().eagle_draft_tree(self.h, C.byref(inp), C.byref(o), tr, st))
        return out

    def lm_head_topk(self, a, k: int, stream=None):
        import torch
        N = int(a.shape[0])
        ids = torch.empty((N, k), dtype=torch.int32, device=a.device)
        logp = torch.empty((N, k), dtype=torch.float32, device=a.device)
        lse = torch.empty((N,), dtype=torch.float32, device=a.device)
        st = None if stream is None else stream.cuda_stream
        _check(load().eagle_draft_lm_head_topk(self.h, _ptr(a), N, k, _ptr(ids), _ptr(logp), _ptr(lse), st))
        return ids, logp, lse

    def profile(self, enable: bool):
        _check(load().eagle_draft_profile(self.h, 1 if enable else 0))

    def profile_read(self) -> dict:
        """{kernel name: (total ms, launches)} since the last read (synchronises)."""
        ms = (C.c_float * KERNEL_KINDS)()
        n = (C.c_int32 * KERNEL_KINDS)()
        _check(load().eagle_draft_profile_read(self.h, ms, n))
        lib = load()
        return {lib.eagle_draft_kernel_name(i).decode(): (ms[i], n[i]) for i in range(KERNEL_KINDS) if n[i]}

    def set_wait_limit(self, cycles: int):
        _check(load().eagle_draft_set_wait_limit(self.h, int(cycles)))

    def check(self) -> int:
        """Synchronise; raise on a device error word or CUDA error."""
        w = C.c_uint32(0)
        st = load().eagle_draft_check(self.h, C.byref(w))
        if st != EAGLE_OK:
            raise EagleError(st, load().eagle_draft_last_error().decode())
        return w.value


class EagleVerify:
    """Handle of the target's verification pass over emitted trees (bf16 target layer)."""

    def __init__(self, cfg: DraftConfig, dWt: dict, dW: dict, max_batch: int, max_slots: int,
                 max_prefix: int | None = None, flags: int = 0):
        lib = load()
        self.cfg = cfg
        self._keep = (dWt, dW)
        c = VerifyConfig(d=cfg.d, n_heads=cfg.n_heads, n_kv_heads=cfg.n_kv_heads, head_dim=cfg.head_dim,
                         d_ff=cfg.d_ff, vocab=cfg.vocab, rms_eps=cfg.rms_eps, rope_theta=cfg.rope_theta,
                         dtype=DTYPE_BF16 if cfg.dtype == "bf16" else DTYPE_F32, max_batch=max_batch,
                         max_slots=max_slots, max_prefix=cfg.prefix[1] if max_prefix is None else max_prefix,
                         flags=flags)
        w = VerifyWeights(embed=_ptr(dW["embed"]), w_lm=_ptr(dW["w_lm"]),
                          **{n: _ptr(dWt[n]) for n in ("attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gate",
                                                       "w_up", "w_down", "final_norm")})
        h = C.c_void_p()
        _check(lib.eagle_verify_create(C.byref(c), C.byref(w), C.byref(h)))
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            load().eagle_verify_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def verify(self, tree: dict, cache: dict, cu_seqlens, accept: bool = True, hidden: bool = False,
               logits: bool = False, stream=None) -> dict:
        """tree: device tensors tokens / positions / parents [B,S] int32 and mask [B,S,S] uint8
        (as eagle_draft_tree emits them); cache: the target's k_cache / v_cache."""
        import torch
        B, S = (int(x) for x in tree["tokens"].shape)
        dev = tree["tokens"].device
        out = {"top_id": torch.empty((B, S), dtype=torch.int32, device=dev),
               "top_logp": torch.empty((B, S), dtype=torch.float32, device=dev),
               "lse": torch.empty((B, S), dtype=torch.float32, device=dev)}
        if hidden:
            out["hidden"] = torch.empty((B, S, self.cfg.d), dtype=torch.float32, device=dev)
        if logits:
            out["logits"] = torch.empty((B, S, self.cfg.vocab), dtype=torch.float32, device=dev)
        if accept:
            out["accept_len"] = torch.empty((B,), dtype=torch.int32, device=dev)
            out["accept_slots"] = torch.empty((B, S), dtype=torch.int32, device=dev)
            out["correction"] = torch.empty((B,), dtype=torch.int32, device=dev)
        inp = VerifyInputs(B=B, S=S, tokens=_ptr(tree["tokens"]), positions=_ptr(tree["positions"]),
                           mask=_ptr(tree["mask"]), parents=_ptr(tree.get("parents")),
                           k_cache=_ptr(cache["k_cache"]), v_cache=_ptr(cache["v_cache"]),
                           cu_seqlens=_ptr(cu_seqlens))
        o = VerifyOutputs(**{n: _ptr(out.get(n)) for n in VERIFY_OUTPUTS})
        st = None if stream is None else stream.cuda_stream
        _check(load().eagle_verify_tree(self.h, C.byref(inp), C.byref(o), st))
        return out

    def check(self) -> int:
        w = C.c_uint32(0)
        st = load().eagle_verify_check(self.h, C.byref(w))
        if st != EAGLE_OK:
            raise EagleError(st, load().eagle_draft_last_error().decode())
        return w.value


def speculative_accept(tree: dict, logits_target, logits_draft, seeds, stream=None) -> dict:
    """Multi-round speculative sampling over emitted trees (device tensors): tokens / parents
    [B,S] int32, logits [B,S,V] float32, seeds [B] (int64 bits of the uint64 seeds).
    Returns accept_len [B], accept_slots [B,S], correction [B] and the error word [1]."""
    import torch
    B, S = (int(x) for x in tree["tokens"].shape)
    V = int(logits_target.shape[-1])
    if logits_target.dtype != torch.float32 or logits_draft.dtype != torch.float32:
        raise EagleError(EAGLE_ERR_INVALID_ARG, "speculative_accept: logits must be float32")
    if tuple(logits_target.shape) != (B, S, V) or tuple(logits_draft.shape) != (B, S, V):
        raise EagleError(EAGLE_ERR_INVALID_ARG, "speculative_accept: logits must be [B, S, vocab]")
    dev = tree["tokens"].device
    out = {"accept_len": torch.empty((B,), dtype=torch.int32, device=dev),
           "accept_slots": torch.empty((B, S), dtype=torch.int32, device=dev),
           "correction": torch.empty((B,), dtype=torch.int32, device=dev),
           "err": torch.zeros((1,), dtype=torch.int32, device=dev)}
    st = None if stream is None else stream.cuda_stream
    _check(load().eagle_speculative_accept(B, S, V, _ptr(tree["tokens"]), _ptr(tree["parents"]),
                                           _ptr(logits_target.contiguous()), _ptr(logits_draft.contiguous()),
                                           _ptr(seeds), _ptr(out["accept_len"]), _ptr(out["accept_slots"]),
                                           _ptr(out["correction"]), _ptr(out["err"]), st))
    return out


def _ptr_array(ts):
    return (C.c_void_p * len(ts))(*[_ptr(t) for t in ts])


def device_dflash_weights(W: dict, device="cuda") -> dict:
    """DFlash weights (synth.make_dflash_weights) -> device tensors; per-layer lists kept."""
    top = device_weights({k: W[k] for k in ("embed", "w_lm", "final_norm")}, device)
    top["layers"] = [device_weights(L, device) for L in W["layers"]]
    return top


class EagleDFlash:
    """Handle of the DFlash block-parallel draft (bf16)."""

    def __init__(self, cfg, dW: dict, max_batch: int | None = None, max_prefix: int | None = None,
                 flags: int = 0):
        lib = load()
        self.cfg = cfg
        self._keep = dW
        c = DFlashConfigC(d=cfg.d, n_heads=cfg.n_heads, n_kv_heads=cfg.n_kv_heads, head_dim=cfg.head_dim,
                          d_ff=cfg.d_ff, vocab=cfg.vocab, rms_eps=cfg.rms_eps, rope_theta=cfg.rope_theta,
                          dtype=DTYPE_BF16 if cfg.dtype == "bf16" else DTYPE_F32, n_layers=cfg.layers,
                          gamma=cfg.gamma, k=cfg.k, mask_token=cfg.mask_id,
                          max_batch=cfg.B if max_batch is None else max_batch,
                          max_prefix=cfg.prefix[1] if max_prefix is None else max_prefix, flags=flags)
        L = dW["layers"]
        self._arrays = {n: _ptr_array([l[n] for l in L]) for n in
                        ("attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gate", "w_up", "w_down")}
        w = DFlashWeights(embed=_ptr(dW["embed"]), w_lm=_ptr(dW["w_lm"]), final_norm=_ptr(dW["final_norm"]),
                          **{n: C.cast(a, C.POINTER(C.c_void_p)) for n, a in self._arrays.items()})
        h = C.c_void_p()
        _check(lib.eagle_dflash_create(C.byref(c), C.byref(w), C.byref(h)))
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            load().eagle_dflash_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def draft(self, dI: dict, hidden: bool = False, stream=None) -> dict:
        """dI: anchor [B] int32, cu_seqlens [B+1], ctx_k / ctx_v lists of per-layer caches."""
        import torch
        B = int(dI["anchor"].shape[0])
        g, k, dev = self.cfg.gamma, self.cfg.k, dI["anchor"].device
        out = {"tokens": torch.empty((B, g, k), dtype=torch.int32, device=dev),
               "logp": torch.empty((B, g, k), dtype=torch.float32, device=dev),
               "lse": torch.empty((B, g), dtype=torch.float32, device=dev)}
        if hidden:
            out["hidden"] = torch.empty((B, g + 1, self.cfg.d), dtype=torch.float32, device=dev)
        ck, cv = _ptr_array(dI["ctx_k"]), _ptr_array(dI["ctx_v"])
        inp = DFlashInputs(B=B, anchor=_ptr(dI["anchor"]), ctx_k=C.cast(ck, C.POINTER(C.c_void_p)),
                           ctx_v=C.cast(cv, C.POINTER(C.c_void_p)), cu_seqlens=_ptr(dI["cu_seqlens"]))
        o = DFlashOutputs(**{n: _ptr(out.get(n)) for n in ("tokens", "logp", "lse", "hidden")})
        st = None if stream is None else stream.cuda_stream
        _check(load().eagle_dflash_draft(self.h, C.byref(inp), C.byref(o), st))
        return out

    def check(self) -> int:
        w = C.c_uint32(0)
        st = load().eagle_dflash_check(self.h, C.byref(w))
        if st != EAGLE_OK:
            raise EagleError(st, load().eagle_draft_last_error().decode())
        return w.value


# ------------------------------------------------------------- the caller's paged cache
# These calls run on `stream`, or on torch's current stream where none is given; tensors they
# allocate belong to that stream.  Tensors, caches and streams must be of the current device.  (The checks take a
# fast path first: a single-token step's calls are as short as their host time.)

def _bad(msg: str):
    raise EagleError(EAGLE_ERR_INVALID_ARG, msg)


_torch = None


def _here(stream):
    """(torch, current device, raw handle of the call's stream)"""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    dev = _torch.cuda.current_device()
    if stream is not None and stream.device_index != dev:
        _bad("the stream must be of the current CUDA device")
    return _torch, dev, (_torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)


def _tensor(t, name: str, dtype, shape, dev: int, contiguous: bool = True):
    """Refuses all but a tensor of device ``dev`` with this dtype and shape (None: any size)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and (not contiguous or t.is_contiguous()):
            s = t.shape
            if s == shape or (len(s) == len(shape) and all([w is None or w == n for w, n in zip(shape, s)])):
                return
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        _bad(f"{name} must be a {dtype} tensor")
    if t.get_device() != dev:
        _bad(f"{name} must be on the current CUDA device")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        _bad(f"{name} must have shape {tuple('*' if w is None else w for w in shape)}, not {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        _bad(f"{name} must be contiguous")


def _ints(t, name: str, n, dev: int) -> int:
    """A contiguous int32 vector (of n numbers, if n is given): its length."""
    if not (isinstance(t, _torch.Tensor) and t.dtype is _torch.int32 and t.dim() == 1 and t.get_device() == dev and t.is_contiguous()
            and (n is None or t.numel() == n)):
        _tensor(t, name, _torch.int32, (n,), dev)
    return t.numel()


def _rows(t, name: str, dtype, n, h, d, dev: int) -> int:
    """Rows [N, H, hd] (sizes n, h, d where given) whose heads are contiguous: the row stride in
    elements."""
    try:
        tn, th, td = t.shape
        s0, s1, s2 = t.stride()
        if t.dtype is dtype and t.get_device() == dev and (n is None or n == tn) and (h is None or h == th) and \
                (d is None or d == td) and ((s2 == 1 and (s1 == td or th == 1)) or tn == 0):
            return s0 if tn > 1 else th * td
    except (AttributeError, ValueError):
        pass
    _tensor(t, name, dtype, (n, h, d), dev, contiguous=False)
    _bad(f"{name}: the heads of a row must be contiguous")


def _new(like, shape, dtype, stream):
    """An uninitialised tensor that belongs to ``stream`` (None: the current one)."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=like.device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=like.device)


def _float_kind(t, name: str) -> int:
    d = getattr(t, "dtype", None)
    if d is _torch.bfloat16:
        return DTYPE_BF16
    if d is _torch.float32:
        return DTYPE_F32
    _bad(f"{name} must be a float32 or bfloat16 tensor")


def rope_frequencies(rot_dim: int, theta: float = 10000.0, linear: float = 1.0, banded: tuple | None = None,
                     ramped: tuple | None = None) -> list:
    """Inverse frequencies theta^(-2i/rot_dim), scaled for contexts longer than trained on.
    ``linear``: all divided by the factor (position interpolation).  ``banded`` (factor, low,
    high, original): waves longer than original/low positions are divided by the factor, those
    shorter than original/high kept, between them a blend linear in the turns within the original
    context (the rule of the Llama-3 family's long contexts).  ``ramped`` (factor, fast, slow,
    original): pairs that turn more than ``fast`` times within ``original`` positions are kept,
    those that turn less than ``slow`` times divided by the factor, between them a linear ramp
    over the pair index (NTK by parts: Peng et al., "YaRN", 2023).  The ramp's ends are whole
    indices, rounded outwards and kept within 0 .. rot_dim - 1: it may end behind the last pair,
    none of which is then divided whole."""
    import math
    if rot_dim < 2 or rot_dim % 2 or not theta > 0 or not linear > 0 or (banded and ramped):
        _bad("rope_frequencies: bad arguments")
    if banded and not (banded[0] > 0 and banded[2] > banded[1] >= 0 and banded[3] > 0):
        _bad("rope_frequencies: banded needs factor > 0, high > low >= 0, original > 0")
    if ramped and not (ramped[0] > 0 and ramped[1] > ramped[2] > 0 and ramped[3] > 0 and theta > 1):
        _bad("rope_frequencies: ramped needs factor > 0, fast > slow > 0, original > 0, theta > 1")
    w = [theta ** (-2.0 * i / rot_dim) / linear for i in range(rot_dim // 2)]
    if banded:
        factor, low, high, original = banded
        for i, f in enumerate(w):
            turns = original * f / (2 * math.pi)             # turns within the original context
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            w[i] = f * (keep + (1.0 - keep) / factor)
    if ramped:
        factor, fast, slow, original = ramped
        index = lambda turns: rot_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot_dim - 1)
        for i, f in enumerate(w):
            part = 1.0 if i >= hi else 0.0 if i <= lo else (i - lo) / (hi - lo)
            w[i] = f * (1.0 - part + part / factor)
    return w


class Rope:
    """Rotary positions (eagle_rope_t): the first ``rot_dim`` dims in half-split or interleaved
    pairs; ``inv_freq`` (rot_dim / 2 numbers, e.g. of rope_frequencies) replaces theta's powers."""

    def __init__(self, rot_dim: int, theta: float = 10000.0, interleaved: bool = False, inv_freq=None,
                 amplitude: float = 1.0):
        self.rot_dim = int(rot_dim)
        # (the powers of theta are taken once here rather than in every call)
        f = rope_frequencies(self.rot_dim, theta) if inv_freq is None else [float(x) for x in inv_freq]
        if 2 * len(f) != self.rot_dim:
            _bad("Rope: inv_freq must hold rot_dim / 2 numbers")
        self._freq = (C.c_double * len(f))(*f)
        self.c = RopeC(rot_dim=self.rot_dim, interleaved=1 if interleaved else 0, theta=float(theta),
                       inv_freq=self._freq, amplitude=float(amplitude))
        self.ref = C.byref(self.c)


def rotary(x, positions, rope: Rope, out=None, stream=None):
    """x [N, H, hd] (float32 or bfloat16) rotated at int32 positions [N]; out may be x."""
    torch, dev, st = _here(stream)
    kind = _float_kind(x, "x")
    ld = _rows(x, "x", x.dtype, None, None, None, dev)
    N, H, hd = x.shape
    _ints(positions, "positions", N, dev)
    if out is None:
        out = _new(x, (N, H, hd), x.dtype, stream)
        old = H * hd
    else:
        old = _rows(out, "out", x.dtype, N, H, hd, dev)
    if N:
        _check(load().eagle_rotary(kind, x.data_ptr(), ld, N, H, hd, positions.data_ptr(), rope.ref, out.data_ptr(), old, st))
    return out


def _cache_here(cache, dev: int):
    if cache.device_index != dev:
        _bad("the cache must be on the current CUDA device")


class KVCache:
    """Paged keys and values of one layer (eagle_kv_cache_t) over the caller's tensors:
    bf16 [pages, Hkv, page_size, hd], or uint8 codes [pages, Hkv, page_size, hd / 2] with uint8
    (e4m3) scales [pages, Hkv, page_size, hd / 16]; page_table int32 [B, max_pages]."""

    def __init__(self, k, v, page_table, k_scale=None, v_scale=None, k_global: float = 1.0, v_global: float = 1.0):
        torch, dev, _ = _here(None)
        f4 = getattr(k, "dtype", None) == torch.uint8
        _tensor(k, "k", torch.uint8 if f4 else torch.bfloat16, (None,) * 4, dev)
        _tensor(v, "v", k.dtype, tuple(k.shape), dev)
        _tensor(page_table, "page_table", torch.int32, (None, None), dev)
        P, H, ps, w = k.shape
        hd = 2 * w if f4 else w
        if f4:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _tensor(t, name, torch.uint8, (P, H, ps, hd // 16), dev)
        elif k_scale is not None or v_scale is not None:
            _bad("scales belong to a 4-bit cache")
        self.k, self.v, self.k_scale, self.v_scale, self.page_table = k, v, k_scale, v_scale, page_table
        self.kind, self.n_kv_heads, self.head_dim, self.device_index = (CACHE_F4 if f4 else CACHE_BF16), H, hd, dev
        self.err = torch.zeros((1,), dtype=torch.int32, device=k.device)
        self.c = KVCacheC(kind=self.kind, n_kv_heads=H, head_dim=hd, page_size=ps, num_pages=P,
                          max_pages=page_table.shape[1], k=_ptr(k), v=_ptr(v), k_scale=_ptr(k_scale),
                          v_scale=_ptr(v_scale), k_global=float(k_global), v_global=float(v_global),
                          page_table=_ptr(page_table))
        self.ref, self.err_ptr, self.max_requests = C.byref(self.c), self.err.data_ptr(), page_table.shape[0]

    @classmethod
    def empty(cls, num_pages: int, page_size: int, n_kv_heads: int, head_dim: int, page_table, four_bit: bool = False,
              k_global: float = 1.0, v_global: float = 1.0):
        """A pool of zeros on page_table's device."""
        import torch
        def z(w, dt):
            return torch.zeros((num_pages, n_kv_heads, page_size, w), dtype=dt, device=page_table.device)
        if not four_bit:
            return cls(z(head_dim, torch.bfloat16), z(head_dim, torch.bfloat16), page_table)
        return cls(z(head_dim // 2, torch.uint8), z(head_dim // 2, torch.uint8), page_table,
                   z(head_dim // 16, torch.uint8), z(head_dim // 16, torch.uint8), k_global, v_global)

    def check(self) -> int:
        """Synchronise; raise when a call on this cache recorded a device error, and clear it."""
        import torch
        torch.cuda.synchronize()
        w = int(self.err.item())
        if w:
            self.err.zero_()
            raise EagleError(EAGLE_ERR_DEVICE, f"device error word 0x{w:x}")
        return w


def kv_append(cache: KVCache, k, v, cu_rows, lens, positions=None, rope: Rope | None = None, q=None, q_out=None,
              stream=None):
    """Store a step's keys (rotated with a rope) and values [N, Hkv, hd] behind each request's
    lens[b] keys; returns the rotated queries when q [N, Hq, hd] is given (q_out may be q)."""
    torch, dev, st = _here(stream)
    H, hd = cache.n_kv_heads, cache.head_dim
    kind = _float_kind(k, "k")
    k_ld = _rows(k, "k", k.dtype, None, H, hd, dev)
    N = k.shape[0]
    v_ld = _rows(v, "v", k.dtype, N, H, hd, dev)
    B = _requests(cache, cu_rows, lens, dev)
    if rope is not None:
        _ints(positions, "positions", N, dev)
    Hq = q_ld = qo_ld = 0
    if q is not None:
        q_ld = _rows(q, "q", k.dtype, N, None, hd, dev)
        Hq = q.shape[1]
        if q_out is None:   # (rows of no request are not written)
            q_out, qo_ld = _new(q, (N, Hq, hd), k.dtype, stream), Hq * hd
        else:
            qo_ld = _rows(q_out, "q_out", k.dtype, N, Hq, hd, dev)
    if N:
        w = KVRows(B, N, cu_rows.data_ptr(), lens.data_ptr(), None if rope is None else positions.data_ptr(), kind, Hq,
                   k.data_ptr(), v.data_ptr(), _ptr(q), _ptr(q_out) if Hq else None, k_ld, v_ld, q_ld, qo_ld)
        _check(load().eagle_kv_append(cache.ref, C.byref(w), None if rope is None else rope.ref, cache.err_ptr, st))
    return q_out if Hq else None


def _requests(cache: KVCache, cu_rows, lens, dev: int) -> int:
    _cache_here(cache, dev)
    B = _ints(lens, "lens", None, dev)
    _ints(cu_rows, "cu_rows", B + 1, dev)
    if cache.max_requests < B:
        _bad("the page table has fewer rows than lens")
    return B


def kv_gather(cache: KVCache, cu_seqlens, total: int, k_out=None, v_out=None, stream=None):
    """The first cu_seqlens[b + 1] - cu_seqlens[b] keys and values of every request, packed bf16
    [total, Hkv, hd]: the k_cache / v_cache of EagleDraft.tree and EagleVerify.verify."""
    torch, dev, st = _here(stream)
    _cache_here(cache, dev)
    B, total = _ints(cu_seqlens, "cu_seqlens", None, dev) - 1, int(total)
    if B < 1 or total < 0 or cache.max_requests < B:
        _bad("kv_gather: cu_seqlens needs 1 .. page_table rows requests, total must not be negative")
    shape = (total, cache.n_kv_heads, cache.head_dim)
    if k_out is None:
        k_out = _new(cache.k, shape, torch.bfloat16, stream)
    else:
        _tensor(k_out, "k_out", torch.bfloat16, shape, dev)
    if v_out is None:
        v_out = _new(cache.k, shape, torch.bfloat16, stream)
    else:
        _tensor(v_out, "v_out", torch.bfloat16, shape, dev)
    _check(load().eagle_kv_gather(cache.ref, B, cu_seqlens.data_ptr(), total, k_out.data_ptr(), v_out.data_ptr(),
                                  cache.err_ptr, st))
    return k_out, v_out


def kv_accept(caches, lens, accept_len, accept_slots, new_lens=None, stream=None):
    """Keep the accepted path of a verified tree (appended behind lens[b] keys in slot order) in
    every cache of the list (one per layer, one shape and page table); returns the new lengths
    lens + 1 + accept_len (new_lens may be lens).  Device errors go to the first cache's word."""
    torch, dev, st = _here(stream)
    caches = [caches] if isinstance(caches, KVCache) else list(caches)
    if not caches:
        _bad("kv_accept: no caches")
    for c in caches:
        _cache_here(c, dev)
    _tensor(accept_slots, "accept_slots", torch.int32, (None, None), dev)
    B, S = accept_slots.shape
    _ints(lens, "lens", B, dev)
    _ints(accept_len, "accept_len", B, dev)
    if caches[0].max_requests < B:
        _bad("the page table has fewer rows than lens")
    if new_lens is None:
        new_lens = _new(lens, (B,), torch.int32, stream)
    else:
        _ints(new_lens, "new_lens", B, dev)
    n = len(caches)
    arr = C.byref(caches[0].c) if n == 1 else (KVCacheC * n)(*[c.c for c in caches])
    _check(load().eagle_kv_accept(arr, n, B, S, lens.data_ptr(), accept_len.data_ptr(), accept_slots.data_ptr(),
                                  new_lens.data_ptr(), caches[0].err_ptr, st))
    return new_lens


def kv_attention(cache: KVCache, q, cu_rows, lens, max_rows: int, max_len: int, mask=None, scale: float = 0.0, out=None,
                 lse=False, workspace=None, stream=None):
    """Attention of a step's rows (appended before) over the cache: bf16 q [N, Hq, hd]; row i of
    request b sees the lens[b] keys before the step and the step's rows j by mask[b, i, j] (uint8
    [B, S, S]) or j <= i.  max_rows / max_len bound one request's rows and keys.  Returns out,
    or (out, lse [N, Hq]) with lse=True or a tensor.  ``workspace``: a uint8 tensor to keep
    (at least kv_attention_workspace bytes); else one is taken from torch's allocator."""
    torch, dev, st = _here(stream)
    q_ld = _rows(q, "q", torch.bfloat16, None, None, cache.head_dim, dev)
    N, Hq, hd = q.shape
    B = _requests(cache, cu_rows, lens, dev)
    S = 0
    if mask is not None:
        S = mask.shape[-1]
        _tensor(mask, "mask", torch.uint8, (B, S, S), dev)
    if out is None:
        out, out_ld = _new(q, (N, Hq, hd), torch.bfloat16, stream), Hq * hd
    else:
        out_ld = _rows(out, "out", torch.bfloat16, N, Hq, hd, dev)
    if lse is True:
        lse = _new(q, (N, Hq), torch.float32, stream)
    elif lse is False:
        lse = None
    elif lse is not None:
        _tensor(lse, "lse", torch.float32, (N, Hq), dev)
    a = KVAttention(B, N, Hq, int(max_rows), int(max_len), S, cu_rows.data_ptr(), lens.data_ptr(), q.data_ptr(), q_ld,
                    _ptr(mask), float(scale), out.data_ptr(), out_ld, _ptr(lse))
    ref = C.byref(a)
    lib = load()
    need = lib.eagle_kv_attention_workspace(cache.ref, ref)
    if need < 0:
        _bad(lib.eagle_draft_last_error().decode())
    if need:
        if workspace is None:
            workspace = _new(q, (need,), torch.uint8, stream)
        else:
            _tensor(workspace, "workspace", torch.uint8, (None,), dev)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    if N:
        _check(lib.eagle_kv_attention(cache.ref, ref, cache.err_ptr, st))
    return out if lse is None else (out, lse)


def _outputs(q, out, lse, N, Hq, hd, dev, stream):
    """(out, its row stride, lse or None) of an attention call: given, or new."""
    if out is None:
        out, ld = _new(q, (N, Hq, hd), _torch.bfloat16, stream), Hq * hd
    else:
        ld = _rows(out, "out", _torch.bfloat16, N, Hq, hd, dev)
    if lse is True:
        lse = _new(q, (N, Hq), _torch.float32, stream)
    elif lse is False:
        lse = None
    elif lse is not None:
        _tensor(lse, "lse", _torch.float32, (N, Hq), dev)
    return out, ld, lse


def _workspace(a, need: int, workspace, like, dev: int, stream):
    """Gives the call's struct its workspace; returns the tensor, to be kept until the launch."""
    if need < 0:
        _bad(load().eagle_draft_last_error().decode())
    if need:
        if workspace is None:
            workspace = _new(like, (need,), _torch.uint8, stream)
        else:
            _tensor(workspace, "workspace", _torch.uint8, (None,), dev)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return workspace


def kv_cross_attention(cache: KVCache, q, cu_rows, lens, max_rows: int, max_len: int, scale: float = 0.0, out=None,
                       lse=False, workspace=None, stream=None):
    """Cross attention: rows cu_rows[b] .. cu_rows[b + 1] of bf16 q [N, Hq, hd] over all lens[b] keys
    in row b of the cache's page table (an encoder's states, a document; 0 keys give zeros and lse
    -inf).  max_rows / max_len bound one request's rows and keys.  out, lse and workspace as in
    kv_attention."""
    torch, dev, st = _here(stream)
    q_ld = _rows(q, "q", torch.bfloat16, None, None, cache.head_dim, dev)
    N, Hq, hd = q.shape
    B = _requests(cache, cu_rows, lens, dev)
    out, out_ld, lse = _outputs(q, out, lse, N, Hq, hd, dev, stream)
    a = KVCross(B, N, Hq, int(max_rows), int(max_len), cu_rows.data_ptr(), lens.data_ptr(), q.data_ptr(), q_ld, float(scale),
                out.data_ptr(), out_ld, _ptr(lse))
    ref = C.byref(a)
    lib = load()
    if N:
        workspace = _workspace(a, lib.eagle_kv_cross_attention_workspace(cache.ref, ref), workspace, q, dev, stream)
        _check(lib.eagle_kv_cross_attention(cache.ref, ref, cache.err_ptr, st))
    return out if lse is None else (out, lse)


def kv_cross_attention_workspace(cache: KVCache, n_heads: int, N: int, B: int, max_rows: int, max_len: int) -> int:
    """Bytes of workspace that kv_cross_attention needs for these sizes."""
    a = KVCross(B=B, N=N, n_heads=n_heads, max_rows=max_rows, max_len=max_len)
    need = load().eagle_kv_cross_attention_workspace(C.byref(cache.c), C.byref(a))
    if need < 0:
        _bad(load().eagle_draft_last_error().decode())
    return need


def kv_shared_attention(prefix: KVCache, cu_groups, prefix_lens, cache: KVCache, q, cu_rows, lens, max_group_rows: int,
                        max_prefix: int, max_rows: int, max_len: int, mask=None, scale: float = 0.0, out=None, lse=False,
                        workspace=None, stream=None):
    """Attention of requests behind shared prefixes: requests cu_groups[g] .. cu_groups[g + 1] see the
    prefix_lens[g] keys in row g of ``prefix``'s page table, computed once for all of them, and
    their own keys in ``cache`` as kv_attention takes them (lens, max_len and mask count own keys;
    the step's rows are appended to ``cache`` before, at positions behind the prefix).
    max_group_rows / max_prefix bound one group's rows and prefix.  Device errors go to ``cache``'s
    word.  out, lse and workspace as in kv_attention."""
    torch, dev, st = _here(stream)
    q_ld = _rows(q, "q", torch.bfloat16, None, None, cache.head_dim, dev)
    N, Hq, hd = q.shape
    B = _requests(cache, cu_rows, lens, dev)
    _cache_here(prefix, dev)
    n_groups = _ints(prefix_lens, "prefix_lens", None, dev)
    _ints(cu_groups, "cu_groups", n_groups + 1, dev)
    if prefix.max_requests < n_groups:
        _bad("the prefix's page table has fewer rows than prefix_lens")
    S = 0
    if mask is not None:
        S = mask.shape[-1]
        _tensor(mask, "mask", torch.uint8, (B, S, S), dev)
    out, out_ld, lse = _outputs(q, out, lse, N, Hq, hd, dev, stream)
    g = KVGroups(n_groups, cu_groups.data_ptr(), prefix_lens.data_ptr(), int(max_group_rows), int(max_prefix))
    a = KVAttention(B, N, Hq, int(max_rows), int(max_len), S, cu_rows.data_ptr(), lens.data_ptr(), q.data_ptr(), q_ld,
                    _ptr(mask), float(scale), out.data_ptr(), out_ld, _ptr(lse))
    gref, ref = C.byref(g), C.byref(a)
    lib = load()
    if N:
        need = lib.eagle_kv_shared_attention_workspace(prefix.ref, gref, cache.ref, ref)
        workspace = _workspace(a, need, workspace, q, dev, stream)
        _check(lib.eagle_kv_shared_attention(prefix.ref, gref, cache.ref, ref, cache.err_ptr, st))
    return out if lse is None else (out, lse)


def kv_shared_attention_workspace(prefix: KVCache, cache: KVCache, n_heads: int, N: int, n_groups: int, B: int,
                                  max_group_rows: int, max_prefix: int, max_rows: int, max_len: int) -> int:
    """Bytes of workspace that kv_shared_attention needs for these sizes, with a mask or without."""
    g = KVGroups(n_groups=n_groups, max_rows=max_group_rows, max_len=max_prefix)
    most = 0
    for slots in (0, max_rows) if 1 <= max_rows <= 64 else (0,):   # (a masked step is cut another way; the pointer is only told from null)
        a = KVAttention(B=B, N=N, n_heads=n_heads, max_rows=max_rows, max_len=max_len, mask=slots or None, mask_slots=slots)
        need = load().eagle_kv_shared_attention_workspace(C.byref(prefix.c), C.byref(g), C.byref(cache.c), C.byref(a))
        if need < 0:
            _bad(load().eagle_draft_last_error().decode())
        most = max(most, need)
    return most


def attention_merge(outs, lses, dtype=None, out=None, lse=False, stream=None):
    """Joins attention results of the same queries over disjoint keys: outs [N, H, hd] (float32 or
    bfloat16, at most 16), lses float32 [N, H] (-inf: the part adds nothing).  The result has
    ``dtype`` (the parts' if not given); out may be one of the parts.  Returns out, or (out, lse)
    with lse=True or a tensor."""
    torch, dev, st = _here(stream)
    outs, lses = list(outs), list(lses)
    n = len(outs)
    if not 1 <= n <= MAX_PARTS or len(lses) != n:
        _bad(f"attention_merge: need 1..{MAX_PARTS} parts, each with its lse")
    x = outs[0]
    kind = _float_kind(x, "outs")
    lds = [_rows(x, "outs", x.dtype, None, None, None, dev)]
    N, H, hd = x.shape
    for t in outs[1:]:
        lds.append(_rows(t, "outs", x.dtype, N, H, hd, dev))
    for t in lses:
        _tensor(t, "lses", torch.float32, (N, H), dev)
    if out is None:
        out, out_ld = _new(x, (N, H, hd), x.dtype if dtype is None else dtype, stream), H * hd
    else:
        if dtype is not None and out.dtype != dtype:
            _bad("attention_merge: out has another dtype")
        out_ld = _rows(out, "out", out.dtype, N, H, hd, dev)
    okind = _float_kind(out, "out")
    if lse is True:
        lse = _new(x, (N, H), torch.float32, stream)
    elif lse is False:
        lse = None
    elif lse is not None:
        _tensor(lse, "lse", torch.float32, (N, H), dev)
    a = AttentionParts(n, N, H, hd, kind, okind, (C.c_void_p * n)(*[t.data_ptr() for t in outs]), (C.c_int64 * n)(*lds),
                       (C.c_void_p * n)(*[t.data_ptr() for t in lses]), out.data_ptr(), out_ld, _ptr(lse))
    if N:
        _check(load().eagle_attention_merge(C.byref(a), st))
    return out if lse is None else (out, lse)


def kv_attention_workspace(cache: KVCache, n_heads: int, N: int, B: int, max_rows: int, max_len: int) -> int:
    """Bytes of workspace that kv_attention needs for these sizes."""
    a = KVAttention(B=B, N=N, n_heads=n_heads, max_rows=max_rows, max_len=max_len)
    need = load().eagle_kv_attention_workspace(C.byref(cache.c), C.byref(a))
    if need < 0:
        _bad(load().eagle_draft_last_error().decode())
    return need
