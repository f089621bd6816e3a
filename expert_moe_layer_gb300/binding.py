"""ctypes binding of libmoe.so (the C ABI in include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (used as plain device memory). The
functions take the same names and arguments as the C entry points and raise
``MoeError`` on a non-zero status. There is no fallback: if the library cannot
be loaded, every call fails loudly.

Inside ``with debug_library():`` the same functions call libmoe_debug.so,
the build whose kernels also check their own derived indices (see
``debug_take``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import threading

from . import _build

MOE_F32, MOE_BF16 = 0, 1
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_STATUS",
                6: "MOE_ERR_TIMEOUT"}
DEV_BAD_EXPERT_ID, DEV_CAP_OVERFLOW, DEV_TIMEOUT, DEV_BAD_SEGMENT = 0x1, 0x2, 0x4, 0x8
DEV_BAD_POSITION, DEV_BAD_SLOT, DEV_BAD_PAGE = 0x10, 0x20, 0x40
DEV_BAD_ROW, DEV_NO_PAGE = 0x80, 0x100


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        self.cuda_error = lib().moe_last_cuda_error() if status == 4 else 0
        why = f", CUDA error {self.cuda_error}" if self.cuda_error else ""
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({strerror(status)}{why})")


class MoeConfig(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int), ("top_k", ctypes.c_int),
                ("hidden_size", ctypes.c_int), ("intermediate_size", ctypes.c_int),
                ("renormalize", ctypes.c_int), ("use_grouped_topk", ctypes.c_int),
                ("num_expert_group", ctypes.c_int), ("topk_group", ctypes.c_int),
                ("routed_scaling_factor", ctypes.c_float),
                ("num_shared_experts", ctypes.c_int),
                ("shared_intermediate_size", ctypes.c_int),
                ("ep_size", ctypes.c_int), ("ep_rank", ctypes.c_int),
                ("act_dtype", ctypes.c_int), ("router_dtype", ctypes.c_int),
                ("scoring_func", ctypes.c_int), ("bias_mode", ctypes.c_int),
                ("max_replicas", ctypes.c_int), ("num_redundant_experts", ctypes.c_int)]


class AttnConfig(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("act_dtype", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("rope_layout", ctypes.c_int), ("rope_positions", ctypes.c_int),
                ("window", ctypes.c_int), ("softmax_scale", ctypes.c_float),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("kind", ctypes.c_int), ("factor", ctypes.c_double),
                ("original_positions", ctypes.c_double), ("slow_turns", ctypes.c_double),
                ("fast_turns", ctypes.c_double), ("attention_factor", ctypes.c_double)]


class KvCaches(ctypes.Structure):
    """Caches (one per layer) that the same page ids index (make_kv_caches)."""
    _fields_ = [("num_caches", ctypes.c_int), ("num_pages", ctypes.c_int64),
                ("caches", ctypes.POINTER(ctypes.c_void_p))]


class KvPool(ctypes.Structure):
    """A page table and its caches (make_kv_pool)."""
    _fields_ = [("page_table", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("num_rows", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("caches", KvCaches)]


class NormConfig(ctypes.Structure):
    _fields_ = [("hidden_size", ctypes.c_int), ("act_dtype", ctypes.c_int),
                ("residual_dtype", ctypes.c_int), ("kind", ctypes.c_int),
                ("post_norm", ctypes.c_int), ("gate", ctypes.c_int),
                ("residual_scale", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("eps", ctypes.c_float)]


class WorkspaceOffsets(ctypes.Structure):
    _fields_ = [("status", ctypes.c_size_t), ("topk_ids", ctypes.c_size_t),
                ("topk_w", ctypes.c_size_t), ("counts", ctypes.c_size_t),
                ("offsets", ctypes.c_size_t), ("sorted_ids", ctypes.c_size_t),
                ("inv_pos", ctypes.c_size_t), ("total", ctypes.c_size_t),
                ("cap", ctypes.c_int), ("block_m", ctypes.c_int)]


class DebugRecord(ctypes.Structure):
    _fields_ = [("count", ctypes.c_uint32), ("site", ctypes.c_uint32),
                ("index", ctypes.c_int64), ("bound", ctypes.c_int64)]


DEBUG_FILES = {1: "moe_api.cu", 2: "kernels_gemm.cu", 3: "kernels_gemm_pair.cu",
               4: "kernels_mlp_fused.cu", 5: "kernels_route.cu", 6: "kernels_align.cu"}


class Plan(ctypes.Structure):
    _fields_ = [("kernels", ctypes.c_int), ("fused_route", ctypes.c_int),
                ("router_tensor_cores", ctypes.c_int),
                ("router_partials", ctypes.c_int), ("align_kernels", ctypes.c_int),
                ("tile_rows", ctypes.c_int), ("gemm1_k_split", ctypes.c_int),
                ("cta_pairs", ctypes.c_int), ("fused_mlp", ctypes.c_int),
                ("gemm2_overlap", ctypes.c_int), ("combine_ring", ctypes.c_int)]


def make_config(num_experts, top_k, hidden_size, intermediate_size, renormalize=True,
                num_expert_group=0, topk_group=0, routed_scaling_factor=1.0,
                num_shared_experts=0, shared_intermediate_size=0, ep_size=1, ep_rank=0,
                act_dtype="bf16", router_dtype="bf16", scoring="softmax",
                bias_mode="logit", max_replicas=0, num_redundant_experts=0) -> MoeConfig:
    dt = {"bf16": MOE_BF16, "f32": MOE_F32}
    sc = {"softmax": 0, "sigmoid": 1}
    bm = {"logit": 0, "select": 1}
    return MoeConfig(num_experts, top_k, hidden_size, intermediate_size, int(bool(renormalize)),
                     int(num_expert_group > 0), num_expert_group, topk_group,
                     float(routed_scaling_factor), num_shared_experts,
                     shared_intermediate_size, ep_size, ep_rank, dt[act_dtype],
                     dt[router_dtype], sc[scoring], bm[bias_mode], max_replicas,
                     num_redundant_experts)


def make_attn_config(num_heads, num_kv_heads, head_dim, page_size=16, act_dtype="bf16",
                     rotary_dim=0, rope_layout="half", rope_positions=0, window=0,
                     softmax_scale=0.0, k_scale=1.0, v_scale=1.0) -> AttnConfig:
    dt = {"bf16": MOE_BF16, "f32": MOE_F32}
    lay = {"half": 0, "interleaved": 1}
    return AttnConfig(num_heads, num_kv_heads, head_dim, page_size, dt[act_dtype], rotary_dim,
                      lay[rope_layout], rope_positions, window, softmax_scale, k_scale, v_scale)


def make_rope_scaling(base=10000.0, kind="none", factor=1.0, original_positions=0, slow_turns=0.0,
                      fast_turns=0.0, attention_factor=0.0) -> RopeScaling:
    kinds = {"none": 0, "linear": 1, "ntk": 2, "parts": 3, "yarn": 4}
    return RopeScaling(base, kinds[kind], factor, original_positions, slow_turns, fast_turns,
                       attention_factor)


def make_norm_config(hidden_size, kind="rms", act_dtype="bf16", residual_dtype=None,
                     post_norm=False, gate="linear", residual_scale=1.0, weight_offset=0.0,
                     eps=1e-6) -> NormConfig:
    dt = {"bf16": MOE_BF16, "f32": MOE_F32}
    return NormConfig(hidden_size, dt[act_dtype], dt[residual_dtype or act_dtype],
                      {"rms": 0, "layer": 1}[kind], int(bool(post_norm)),
                      {"linear": 0, "sigmoid": 1}[gate], residual_scale, weight_offset, eps)


_libs: dict[bool, ctypes.CDLL] = {}  # debug build? -> loaded library
_use_debug = False
_lock = threading.Lock()
_VP, _SZ, _I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_I64 = ctypes.c_int64
_CFG = ctypes.POINTER(MoeConfig)
_ACFG = ctypes.POINTER(AttnConfig)
_POOL, _CACHES = ctypes.POINTER(KvPool), ctypes.POINTER(KvCaches)
_ROWS = [_VP, _I64, _I64]  # a strided [T, heads, D] tensor: pointer, token and head strides

_SIGS = {
    "moe_strerror": (ctypes.c_char_p, [_I]),
    "moe_validate_config": (_I, [_CFG]),
    "moe_align_cap": (_SZ, [_CFG, _I, _I]),
    "moe_route_workspace_size": (_SZ, [_CFG, _I]),
    "moe_route": (_I, [_CFG, _I, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_align_workspace_size": (_SZ, [_CFG, _I]),
    "moe_align_permute": (_I, [_CFG, _I, _VP, _VP, _I, _VP, _VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "moe_align_permute_noalloc": (_I, [_CFG, _I, _VP, _VP, _I, _VP, _VP, _VP, _VP, _I, _VP]),
    "moe_grouped_mlp_workspace_size": (_SZ, [_CFG, _I, _I]),
    "moe_grouped_mlp": (_I, [_CFG, _I, _VP, _VP, _VP, _VP, _I, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_combine": (_I, [_CFG, _I, _VP, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_workspace_size": (_SZ, [_CFG, _I]),
    "moe_workspace_layout": (_I, [_CFG, _I, ctypes.POINTER(WorkspaceOffsets)]),
    "moe_forward": (_I, [_CFG, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_forward_timed": (_I, [_CFG, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                               _SZ, _VP, ctypes.POINTER(ctypes.c_void_p),
                               ctypes.POINTER(ctypes.c_int)]),
    "moe_get_status": (_I, [_VP, _VP, ctypes.POINTER(ctypes.c_uint32)]),
    "moe_last_cuda_error": (_I, []),
    "moe_set_wait_limit_ns": (_I, [ctypes.c_uint64]),
    "moe_forward_plan": (_I, [_CFG, _I, ctypes.POINTER(Plan)]),
    "moe_ep_dispatch_workspace_size": (_SZ, [_CFG, _I]),
    "moe_ep_dispatch": (_I, [_CFG, _I] + [_VP] * 12 + [_SZ, _VP]),
    "moe_ep_expert_compute_workspace_size": (_SZ, [_CFG, _I]),
    "moe_ep_expert_compute": (_I, [_CFG, _I] + [_VP] * 7 + [_SZ, _VP]),
    "moe_ep_combine": (_I, [_CFG, _I] + [_VP] * 5 + [_SZ, _VP]),
    "moe_validate_attn_config": (_I, [_ACFG]),
    "moe_kv_page_bytes": (_SZ, [_ACFG]),
    "moe_rope_table": (_I, [_ACFG, _I, _VP, ctypes.POINTER(RopeScaling), _VP, _VP, _SZ, _VP]),
    "moe_rope": (_I, [_ACFG, _I, _I] + _ROWS + [_VP, _VP, _I, _VP, _VP, _SZ, _VP]),
    "moe_kv_append": (_I, [_ACFG, _I] + 3 * _ROWS + [_VP] * 5 + [_I64, _VP, _SZ, _VP]),
    "moe_kv_read": (_I, [_ACFG, _I, _VP, _VP, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "moe_kv_attention_workspace_size": (_SZ, [_ACFG, _I, _I, _I]),
    "moe_kv_attention": (_I, [_ACFG, _I, _I, _I] + _ROWS + [_VP] * 3 + [_I, _VP, _I64] +
                         [_VP, _VP, _VP, _SZ, _VP]),
    "moe_kv_attention_shared_workspace_size": (_SZ, [_ACFG] + [_I] * 5),
    "moe_kv_attention_shared": (_I, [_ACFG] + [_I] * 5 + _ROWS + [_VP] * 3 + [_I] + [_VP] * 3 +
                                [_I64] + [_VP, _VP, _VP, _SZ, _VP]),
    "moe_kv_pool_workspace_size": (_SZ, [_ACFG, _POOL, _I]),
    "moe_kv_fork": (_I, [_ACFG, _POOL, _I] + [_VP] * 4 + [_SZ, _VP]),
    "moe_kv_reserve": (_I, [_ACFG, _POOL, _I] + [_VP] * 4 + [_SZ, _VP]),
    "moe_kv_release": (_I, [_ACFG, _POOL, _I] + [_VP] * 3 + [_SZ, _VP]),
    "moe_kv_compact": (_I, [_ACFG, _POOL, _VP, _VP, _SZ, _VP]),
    "moe_kv_copy_pages": (_I, [_ACFG, _CACHES, _CACHES, _I, _VP, _VP, _VP, _SZ, _VP]),
    "moe_validate_norm_config": (_I, [ctypes.POINTER(NormConfig)]),
    "moe_norm": (_I, [ctypes.POINTER(NormConfig), _I, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _I64,
                      _I64] + [_VP] * 5 + [_SZ, _VP]),
    "moe_debug_build": (_I, []),
    "moe_debug_take": (_I, [ctypes.POINTER(DebugRecord)]),
    "moe_debug_selftest": (_I, [_VP]),
}


def header_functions() -> list[str]:
    """Names of the functions declared in include/moe.h."""
    with open(os.path.join(_build.INCLUDE, "moe.h")) as fh:
        text = fh.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", text)))


def lib(build: bool = True, debug: bool | None = None) -> ctypes.CDLL:
    """Load libmoe.so, or libmoe_debug.so inside ``debug_library()`` (or with
    debug=True), building it in place first if missing or stale."""
    dbg = _use_debug if debug is None else debug
    L = _libs.get(dbg)
    if L is not None:
        return L
    with _lock:
        L = _libs.get(dbg)
        if L is None:
            path = _build.lib_path(dbg)
            if build:
                _build.build(debug=dbg)
            if not os.path.exists(path):
                raise RuntimeError(f"{os.path.basename(path)} is not built; "
                                   "call __graft_entry__.build()")
            L = ctypes.CDLL(path)
            for name, (res, args) in _SIGS.items():
                f = getattr(L, name)
                f.restype, f.argtypes = res, args
            _libs[dbg] = L
    return L


@contextlib.contextmanager
def debug_library():
    """Route every call of this module to libmoe_debug.so for the duration
    (one thread at a time; not reentrant across threads)."""
    global _use_debug
    old = _use_debug
    _use_debug = True
    try:
        yield lib()
    finally:
        _use_debug = old


def strerror(status: int) -> str:
    return lib().moe_strerror(status).decode()


def _p(t):
    """Device pointer of a tensor (None -> NULL); integers pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libmoe takes device tensors; got one on " + str(t.device))
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


_current_stream = None  # (imports torch on first use)


def _stream(stream):
    if stream is None:
        global _current_stream
        if _current_stream is None:
            import torch
            raw, device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
            _current_stream = lambda: raw(device())  # noqa: E731
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(fn, rc):
    if rc != 0:
        raise MoeError(fn, rc)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def validate_config(cfg: MoeConfig) -> int:
    return lib().moe_validate_config(ctypes.byref(cfg))


def align_cap(cfg, T, block_m) -> int:
    return lib().moe_align_cap(ctypes.byref(cfg), T, block_m)


def route_workspace_size(cfg, T) -> int:
    return lib().moe_route_workspace_size(ctypes.byref(cfg), T)


def align_workspace_size(cfg, T) -> int:
    return lib().moe_align_workspace_size(ctypes.byref(cfg), T)


def grouped_mlp_workspace_size(cfg, T, cap) -> int:
    return lib().moe_grouped_mlp_workspace_size(ctypes.byref(cfg), T, cap)


def workspace_size(cfg, T) -> int:
    return lib().moe_workspace_size(ctypes.byref(cfg), T)


def workspace_layout(cfg, T) -> WorkspaceOffsets:
    out = WorkspaceOffsets()
    _check("moe_workspace_layout", lib().moe_workspace_layout(ctypes.byref(cfg), T,
                                                             ctypes.byref(out)))
    return out


def forward_plan(cfg, T) -> Plan:
    out = Plan()
    _check("moe_forward_plan", lib().moe_forward_plan(ctypes.byref(cfg), T, ctypes.byref(out)))
    return out


def ep_dispatch_workspace_size(cfg, T) -> int:
    return lib().moe_ep_dispatch_workspace_size(ctypes.byref(cfg), T)


def moe_ep_dispatch(cfg, T, x, topk_ids, topk_w, send_counts, send_offsets, send_pos, send_x,
                    send_ids, send_w, send_tok, ws, stream=None, phys_map=None):
    _check("moe_ep_dispatch", lib().moe_ep_dispatch(
        ctypes.byref(cfg), T, _p(x), _p(topk_ids), _p(topk_w), _p(phys_map), _p(send_counts),
        _p(send_offsets), _p(send_pos), _p(send_x), _p(send_ids), _p(send_w), _p(send_tok),
        _p(ws), _nbytes(ws), _stream(stream)))


def ep_expert_compute_workspace_size(cfg, R) -> int:
    return lib().moe_ep_expert_compute_workspace_size(ctypes.byref(cfg), R)


def moe_ep_expert_compute(cfg, R, recv_x, recv_ids, recv_w, w13, w2, y, ws, stream=None):
    _check("moe_ep_expert_compute", lib().moe_ep_expert_compute(
        ctypes.byref(cfg), R, _p(recv_x), _p(recv_ids), _p(recv_w), _p(w13), _p(w2), _p(y),
        _p(ws), _nbytes(ws), _stream(stream)))


def moe_ep_combine(cfg, T, ret, send_pos, shared_out, out, ws=None, stream=None):
    _check("moe_ep_combine", lib().moe_ep_combine(
        ctypes.byref(cfg), T, _p(ret), _p(send_pos), _p(shared_out), _p(out), _p(ws),
        _nbytes(ws), _stream(stream)))


def moe_route(cfg, T, x, router_w, router_bias, topk_ids, topk_w, ws, stream=None):
    _check("moe_route", lib().moe_route(ctypes.byref(cfg), T, _p(x), _p(router_w),
                                        _p(router_bias), _p(topk_ids), _p(topk_w), _p(ws),
                                        _nbytes(ws), _stream(stream)))


def moe_align_permute(cfg, T, topk_ids, expert_map, block_m, counts, offsets, sorted_ids,
                      inv_pos, cap, ws, stream=None):
    _check("moe_align_permute", lib().moe_align_permute(
        ctypes.byref(cfg), T, _p(topk_ids), _p(expert_map), block_m, _p(counts), _p(offsets),
        _p(sorted_ids), _p(inv_pos), cap, _p(ws), _nbytes(ws), _stream(stream)))


def moe_align_permute_noalloc(cfg, T, topk_ids, expert_map, block_m, counts, offsets,
                              sorted_ids, inv_pos, cap, stream=None):
    """moe_align_permute with its scratch in the library's static device array
    (for callers that cannot allocate a workspace)."""
    _check("moe_align_permute_noalloc", lib().moe_align_permute_noalloc(
        ctypes.byref(cfg), T, _p(topk_ids), _p(expert_map), block_m, _p(counts), _p(offsets),
        _p(sorted_ids), _p(inv_pos), cap, _stream(stream)))


def moe_grouped_mlp(cfg, T, x, sorted_ids, counts, offsets, cap, w13, w2, y_perm, ws,
                    stream=None):
    _check("moe_grouped_mlp", lib().moe_grouped_mlp(
        ctypes.byref(cfg), T, _p(x), _p(sorted_ids), _p(counts), _p(offsets), cap, _p(w13),
        _p(w2), _p(y_perm), _p(ws), _nbytes(ws), _stream(stream)))


def moe_combine(cfg, T, y_perm, cap, inv_pos, topk_w, shared_out, out, ws=None, stream=None):
    _check("moe_combine", lib().moe_combine(
        ctypes.byref(cfg), T, _p(y_perm), cap, _p(inv_pos), _p(topk_w), _p(shared_out),
        _p(out), _p(ws), _nbytes(ws), _stream(stream)))


def moe_forward(cfg, T, x, router_w, router_bias, w13, w2, shared_w13, shared_w2, expert_map,
                out, ws, stream=None):
    _check("moe_forward", lib().moe_forward(
        ctypes.byref(cfg), T, _p(x), _p(router_w), _p(router_bias), _p(w13), _p(w2),
        _p(shared_w13), _p(shared_w2), _p(expert_map), _p(out), _p(ws), _nbytes(ws),
        _stream(stream)))


def moe_forward_timed(cfg, T, x, router_w, router_bias, w13, w2, shared_w13, shared_w2,
                      expert_map, out, ws, events, stream=None) -> int:
    """moe_forward that records 8 torch.cuda.Event objects (or None) at the
    stage boundaries on the stream; returns the number of kernels launched."""
    handles = (ctypes.c_void_p * 8)()
    for i, ev in enumerate(events):
        handles[i] = None if ev is None else ev.cuda_event
    n = ctypes.c_int(0)
    _check("moe_forward_timed", lib().moe_forward_timed(
        ctypes.byref(cfg), T, _p(x), _p(router_w), _p(router_bias), _p(w13), _p(w2),
        _p(shared_w13), _p(shared_w2), _p(expert_map), _p(out), _p(ws), _nbytes(ws),
        _stream(stream), handles, ctypes.byref(n)))
    return n.value


# ------------------------------------------------------------------ attention
def _dtypes():
    """torch's types under the names used here (torch is imported on first use)."""
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32,
            "i64": torch.int64, "u8": torch.uint8, MOE_F32: torch.float32,
            MOE_BF16: torch.bfloat16}


_DT: dict = {}


def _dt(key):
    if not _DT:
        _DT.update(_dtypes())
    return _DT[key]


def _typed(name, t, key, shape):
    """Device pointer of a contiguous tensor of that type and shape (None
    passes through; a None in the shape is not checked)."""
    if t is None:
        return None
    # (what fits takes the short way: a call's checks cost as much as its launch)
    if t.dtype is _DT.get(key) and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not _dt(key):
        raise ValueError(f"{name} must be {_dt(key)}; got {t.dtype}")
    have = t.shape
    if have != shape and (len(have) != len(shape) or
                          any(n is not None and n != m for n, m in zip(shape, have))):
        raise ValueError(f"{name} must have shape {shape}; got {tuple(have)}")
    return _p(t)


def _rows(name, t, cfg, T, heads):
    """(pointer, token stride, head stride) of a [T, heads, head_dim] tensor
    whose channels are contiguous; tokens and heads may be strided."""
    if t is None:
        return None, 0, 0
    if t.dtype is not _dt(cfg.act_dtype):
        raise ValueError(f"{name} must be {_dt(cfg.act_dtype)}; got {t.dtype}")
    if t.shape != (T, heads, cfg.head_dim):
        raise ValueError(f"{name} must have shape {(T, heads, cfg.head_dim)}; "
                         f"got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("libmoe takes device tensors; got one on " + str(t.device))
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return t.data_ptr(), st, sh


def _cache(cache, cfg):
    """(pointer, pages) of a cache tensor [pages, kv heads, block bytes]."""
    block = cfg.page_size * cfg.head_dim * 9 // 8
    shape = cache.shape
    return _typed("cache", cache, "u8", (shape[0], cfg.num_kv_heads, block)), shape[0]


def validate_attn_config(cfg: AttnConfig) -> int:
    return lib().moe_validate_attn_config(ctypes.byref(cfg))


def kv_page_bytes(cfg: AttnConfig) -> int:
    return lib().moe_kv_page_bytes(ctypes.byref(cfg))


def kv_attention_workspace_size(cfg, num_seqs, T, max_q_len) -> int:
    return lib().moe_kv_attention_workspace_size(ctypes.byref(cfg), num_seqs, T, max_q_len)


def moe_rope_table(cfg, n, positions, scaling, table, ws=None, stream=None):
    _check("moe_rope_table", lib().moe_rope_table(
        ctypes.byref(cfg), n, _typed("positions", positions, "i32", (n,)),
        ctypes.byref(scaling), _typed("table", table, "f32", (n, cfg.rotary_dim)),
        _p(ws), _nbytes(ws), _stream(stream)))


def moe_rope(cfg, T, x, positions, table, out, inverse=False, ws=None, stream=None):
    heads = x.shape[1] if x.dim() == 3 else 0
    _check("moe_rope", lib().moe_rope(
        ctypes.byref(cfg), T, heads, *_rows("x", x, cfg, T, heads),
        _typed("positions", positions, "i32", (T,)),
        _typed("table", table, "f32", (cfg.rope_positions, cfg.rotary_dim)),
        int(bool(inverse)), _typed("out", out, cfg.act_dtype, (T, heads, cfg.head_dim)), _p(ws),
        _nbytes(ws), _stream(stream)))


def moe_kv_append(cfg, T, q, k, v, positions, slots, table, q_out, cache, ws=None, stream=None):
    _check("moe_kv_append", lib().moe_kv_append(
        ctypes.byref(cfg), T, *_rows("q", q, cfg, T, cfg.num_heads),
        *_rows("k", k, cfg, T, cfg.num_kv_heads), *_rows("v", v, cfg, T, cfg.num_kv_heads),
        _typed("positions", positions, "i32", (T,)),
        _typed("slots", slots, "i64", (T,)),
        _typed("table", table, "f32", (cfg.rope_positions, cfg.rotary_dim)),
        _typed("q_out", q_out, cfg.act_dtype, (T, cfg.num_heads, cfg.head_dim)),
        *_cache(cache, cfg), _p(ws), _nbytes(ws), _stream(stream)))


def moe_kv_read(cfg, N, slots, cache, k_out, v_out, ws=None, stream=None):
    shape = (N, cfg.num_kv_heads, cfg.head_dim)
    _check("moe_kv_read", lib().moe_kv_read(
        ctypes.byref(cfg), N, _typed("slots", slots, "i64", (N,)), *_cache(cache, cfg),
        _typed("k_out", k_out, cfg.act_dtype, shape), _typed("v_out", v_out, cfg.act_dtype, shape),
        _p(ws), _nbytes(ws), _stream(stream)))


def moe_kv_attention(cfg, num_seqs, T, max_q_len, q, q_offsets, seq_lens, page_table, cache, out,
                     lse, ws, stream=None):
    max_pages = page_table.shape[-1]
    _check("moe_kv_attention", lib().moe_kv_attention(
        ctypes.byref(cfg), num_seqs, T, max_q_len, *_rows("q", q, cfg, T, cfg.num_heads),
        _typed("q_offsets", q_offsets, "i32", (num_seqs + 1,)),
        _typed("seq_lens", seq_lens, "i32", (num_seqs,)),
        _typed("page_table", page_table, "i32", (num_seqs, max_pages)), max_pages,
        *_cache(cache, cfg), _typed("out", out, cfg.act_dtype, (T, cfg.num_heads, cfg.head_dim)),
        _typed("lse", lse, "f32", (T, cfg.num_heads)), _p(ws), _nbytes(ws),
        _stream(stream)))


def kv_attention_shared_workspace_size(cfg, num_seqs, T, max_q_len, num_groups,
                                       max_group_len) -> int:
    return lib().moe_kv_attention_shared_workspace_size(ctypes.byref(cfg), num_seqs, T, max_q_len,
                                                        num_groups, max_group_len)


def moe_kv_attention_shared(cfg, num_seqs, T, max_q_len, num_groups, max_group_len, q, q_offsets,
                            seq_lens, page_table, group_offsets, prefix_lens, cache, out, lse, ws,
                            stream=None):
    max_pages = page_table.shape[-1]
    _check("moe_kv_attention_shared", lib().moe_kv_attention_shared(
        ctypes.byref(cfg), num_seqs, T, max_q_len, num_groups, max_group_len,
        *_rows("q", q, cfg, T, cfg.num_heads),
        _typed("q_offsets", q_offsets, "i32", (num_seqs + 1,)),
        _typed("seq_lens", seq_lens, "i32", (num_seqs,)),
        _typed("page_table", page_table, "i32", (num_seqs, max_pages)), max_pages,
        _typed("group_offsets", group_offsets, "i32", (num_groups + 1,)),
        _typed("prefix_lens", prefix_lens, "i32", (num_groups,)), *_cache(cache, cfg),
        _typed("out", out, cfg.act_dtype, (T, cfg.num_heads, cfg.head_dim)),
        _typed("lse", lse, "f32", (T, cfg.num_heads)), _p(ws), _nbytes(ws), _stream(stream)))


# --------------------------------------------------------------- shared pages
def make_kv_caches(cfg, caches) -> KvCaches:
    """The caches (uint8 tensors [pages, kv heads, block bytes], one per layer)
    that the same page ids index. Keeps the tensors alive."""
    caches = list(caches)
    if not caches:
        raise ValueError("at least one cache")
    found = [_cache(c, cfg) for c in caches]
    if any(n != found[0][1] for _, n in found):
        raise ValueError("the caches must have the same number of pages; got "
                         f"{[n for _, n in found]}")
    array = (ctypes.c_void_p * len(found))(*[p for p, _ in found])
    out = KvCaches(len(found), found[0][1], array)
    out.keep = (caches, array)
    return out


def make_kv_pool(cfg, page_table, held, refs, caches) -> KvPool:
    """A pool over page_table [rows, max_pages], held [rows] and refs [pages]
    (int32) and its caches (tensors, or what make_kv_caches returned). Keeps the
    tensors alive."""
    if not isinstance(caches, KvCaches):
        caches = make_kv_caches(cfg, caches)
    rows, width = page_table.shape
    out = KvPool(_typed("page_table", page_table, "i32", (rows, width)),
                 _typed("held", held, "i32", (rows,)),
                 _typed("refs", refs, "i32", (caches.num_pages,)), rows, width, caches)
    out.keep = (page_table, held, refs, caches)
    return out


def kv_pool_workspace_size(cfg, pool, n=0) -> int:
    return lib().moe_kv_pool_workspace_size(ctypes.byref(cfg), ctypes.byref(pool), n)


def moe_kv_fork(cfg, pool, n, parents, children, tokens, ws=None, stream=None):
    _check("moe_kv_fork", lib().moe_kv_fork(
        ctypes.byref(cfg), ctypes.byref(pool), n, _typed("parents", parents, "i32", (n,)),
        _typed("children", children, "i32", (n,)), _typed("tokens", tokens, "i32", (n,)), _p(ws),
        _nbytes(ws), _stream(stream)))


def moe_kv_reserve(cfg, pool, n, rows, start, end, ws, stream=None):
    _check("moe_kv_reserve", lib().moe_kv_reserve(
        ctypes.byref(cfg), ctypes.byref(pool), n, _typed("rows", rows, "i32", (n,)),
        _typed("start", start, "i32", (n,)), _typed("end", end, "i32", (n,)), _p(ws),
        _nbytes(ws), _stream(stream)))


def moe_kv_release(cfg, pool, n, rows, keep=None, ws=None, stream=None):
    _check("moe_kv_release", lib().moe_kv_release(
        ctypes.byref(cfg), ctypes.byref(pool), n, _typed("rows", rows, "i32", (n,)),
        _typed("keep", keep, "i32", (n,)), _p(ws), _nbytes(ws), _stream(stream)))


def moe_kv_compact(cfg, pool, used, ws, stream=None):
    _check("moe_kv_compact", lib().moe_kv_compact(
        ctypes.byref(cfg), ctypes.byref(pool), _typed("used", used, "i32", (1,)), _p(ws),
        _nbytes(ws), _stream(stream)))


def moe_kv_copy_pages(cfg, src_caches, dst_caches, n, src, dst, ws=None, stream=None):
    _check("moe_kv_copy_pages", lib().moe_kv_copy_pages(
        ctypes.byref(cfg), ctypes.byref(src_caches), ctypes.byref(dst_caches), n,
        _typed("src", src, "i32", (n,)), _typed("dst", dst, "i32", (n,)), _p(ws), _nbytes(ws),
        _stream(stream)))


# ---------------------------------------------------------------------- norms
def validate_norm_config(cfg: NormConfig) -> int:
    return lib().moe_validate_norm_config(ctypes.byref(cfg))


def _norm_rows(name, t, dtype, T, H):
    """(pointer, row stride) of a [T, H] tensor whose channels are contiguous."""
    if t is None:
        return None, 0
    if t.dtype is _DT.get(dtype) and t.shape == (T, H) and t.is_cuda:
        st, sd = t.stride()
        if sd == 1:
            return t.data_ptr(), st
    if t.dtype is not _dt(dtype):
        raise ValueError(f"{name} must be {_dt(dtype)}; got {t.dtype}")
    if t.shape != (T, H):
        raise ValueError(f"{name} must have shape {(T, H)}; got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("libmoe takes device tensors; got one on " + str(t.device))
    st, sd = t.stride()
    if sd != 1 and H > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return t.data_ptr(), st


def _gate(gate, cfg, T):
    """(pointer, token stride, channel stride) of a gate [H], [T, 1] or [T, H]."""
    if gate is None:
        return None, 0, 0
    H = cfg.hidden_size
    if gate.dtype is not _dt(cfg.act_dtype):
        raise ValueError(f"gate must be {_dt(cfg.act_dtype)}; got {gate.dtype}")
    if not gate.is_cuda:
        raise ValueError("libmoe takes device tensors; got one on " + str(gate.device))
    if gate.shape == (H,):
        token, channel = 0, gate.stride(0)
    elif gate.shape == (T, H):
        token, channel = gate.stride()
    elif gate.shape == (T, 1):
        token, channel = gate.stride(0), 0
    else:
        raise ValueError(f"gate must have shape {(H,)}, {(T, 1)} or {(T, H)}; "
                         f"got {tuple(gate.shape)}")
    if H == 1:
        channel = 0
    if channel not in (0, 1):
        raise ValueError("the channels of the gate must be contiguous")
    return gate.data_ptr(), token, channel


def moe_norm(cfg, T, y, x, post_w, post_b, gate, pre_w, pre_b, x_out, h, ws=None, stream=None):
    H, act, res = cfg.hidden_size, cfg.act_dtype, cfg.residual_dtype
    vec, rows = (H,), (T, H)
    _check("moe_norm", lib().moe_norm(
        ctypes.byref(cfg), T, *_norm_rows("y", y, act, T, H), *_norm_rows("x", x, res, T, H),
        _typed("post_w", post_w, "f32", vec), _typed("post_b", post_b, "f32", vec),
        *_gate(gate, cfg, T), _typed("pre_w", pre_w, "f32", vec),
        _typed("pre_b", pre_b, "f32", vec), _typed("x_out", x_out, res, rows),
        _typed("h", h, act, rows), _p(ws), _nbytes(ws), _stream(stream)))


def moe_get_status(ws, stream=None) -> tuple[int, int]:
    """(status code, raw MOE_DEV_* flags); synchronises the stream."""
    flags = ctypes.c_uint32(0)
    rc = lib().moe_get_status(_p(ws), _stream(stream), ctypes.byref(flags))
    return rc, flags.value


def debug_build() -> bool:
    """True when the active library is libmoe_debug.so."""
    return bool(lib().moe_debug_build())


def debug_take() -> DebugRecord:
    """Synchronise the device, then read and clear the debug build's record
    of failed bounds checks (count, and site / index / bound of the first)."""
    rec = DebugRecord()
    _check("moe_debug_take", lib().moe_debug_take(ctypes.byref(rec)))
    return rec


def debug_site(site: int) -> str:
    """'file:line' of a record's site."""
    return f"{DEBUG_FILES.get(site >> 16, site >> 16)}:{site & 0xffff}"


def debug_selftest(stream=None) -> None:
    """Enqueue the debug build's one failing check (index 5, bound 4)."""
    _check("moe_debug_selftest", lib().moe_debug_selftest(_stream(stream)))


def set_wait_limit_ns(ns: int) -> None:
    """Time limit of the kernels' pipeline waits on the current device, in ns
    (0 restores the default of 1 s)."""
    _check("moe_set_wait_limit_ns", lib().moe_set_wait_limit_ns(int(ns)))
