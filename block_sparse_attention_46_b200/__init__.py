"""Python binding of liblf, the sm_100a hierarchical sparse attention library.

Argument marshalling only: every function below forwards to the C entry point of the
same name in ``liblf.so`` (declared in include/lf.h) with raw device pointers, host
slot lists and the current CUDA stream.  PyTorch provides device memory and streams; no
step of the attention path runs in Python or on the CPU.  If the library is missing or
does not load, every call raises.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import operator
import os
from typing import Optional, Sequence

import torch

__all__ = [
    "LfError", "LfShape", "load", "make_shape", "lf_compress", "lf_select_frames",
    "lf_select_blocks", "lf_block_sparse_attn", "lf_forward_chunk",
    "lf_attn_workspace_size", "lf_forward_workspace_size", "lf_device_status",
    "lf_select_chunk", "lf_select_workspace_size", "lf_block_sparse_attn_noalloc",
    "lf_noalloc_scratch_bytes", "lf_pooled_cache_bytes", "lf_pool_frames",
    "lf_select_chunk_cached", "lf_cag_schedule", "lf_select_chunk_1d",
    "lf_status_string", "lf_abi_version", "lf_debug_configure", "lf_select_current",
    "lf_quantize_e4m3", "lf_e4m3_head_scales", "lf_block_sparse_attn_e4m3",
    "lf_attn_backward_workspace_size", "lf_block_sparse_attn_backward", "LfRope", "make_rope",
    "lf_rope_frames", "lf_rope_backward_workspace_size", "lf_rope_frames_backward",
    "derived", "current_blocks", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblf.so")

LF_OK = 0
LF_ERR_INVALID_ARG = 1
LF_ERR_UNSUPPORTED = 2


class LfError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: liblf status {code} ({lf_status_string(code)})")


class LfShape(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d", ctypes.c_int32),
                ("tokens_per_frame", ctypes.c_int32), ("block", ctypes.c_int32),
                ("n_cur_frames", ctypes.c_int32), ("n_hist", ctypes.c_int32),
                ("n_sink", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("k_f", ctypes.c_int32), ("k_b", ctypes.c_int32), ("scale", ctypes.c_float),
                ("k_c", ctypes.c_int32)]


class LfRope(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d", ctypes.c_int32), ("n_frames", ctypes.c_int32),
                ("height", ctypes.c_int32), ("width", ctypes.c_int32),
                ("pairs_t", ctypes.c_int32), ("pairs_h", ctypes.c_int32),
                ("pairs_w", ctypes.c_int32), ("halves", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("base", ctypes.c_double)]


_lib: Optional[ctypes.CDLL] = None
_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_I32P = ctypes.POINTER(ctypes.c_int32)
_SHP = ctypes.POINTER(LfShape)
_RPP = ctypes.POINTER(LfRope)
_I32, _I64 = ctypes.c_int32, ctypes.c_int64

_SIGS = {
    "lf_compress": (ctypes.c_int, [_SHP, _P, _P, _I32P, _P, _P, _P, _P]),
    "lf_select_frames": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _P]),
    "lf_select_blocks": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _P, _P]),
    "lf_attn_workspace_size": (_SZ, [_SHP]),
    "lf_block_sparse_attn": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _P, _I32P, _I32P, _P, _P,
                                            _P, _P, _P, _SZ, _P]),
    "lf_select_current": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _SZ, _P]),
    "lf_forward_workspace_size": (_SZ, [_SHP]),
    "lf_select_workspace_size": (_SZ, [_SHP]),
    "lf_select_chunk": (ctypes.c_int, [_SHP, _P, _P, _I32P, _P, _P, _SZ, _P]),
    "lf_forward_chunk": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _P, _I32P, _I32P, _P, _SZ, _P,
                                        _P, _P, _P, _P]),
    "lf_device_status": (ctypes.c_int, [ctypes.c_int]),
    "lf_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "lf_abi_version": (ctypes.c_int, []),
    "lf_noalloc_scratch_bytes": (_SZ, []),
    "lf_debug_configure": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_int, ctypes.c_int]),
    "lf_block_sparse_attn_e4m3": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _P, _P, _P, _I32P, _I32P,
                                                 _P, _P, _P, _P, _P, _SZ, _P]),
    "lf_quantize_e4m3": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P,
                                        _P, _P, _P]),
    "lf_e4m3_head_scales": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p),
                                           ctypes.POINTER(ctypes.c_int64), ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "lf_pooled_cache_bytes": (_SZ, [_SHP]),
    "lf_cag_schedule": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                       ctypes.c_float, _I32P, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.POINTER(ctypes.c_float), _I32P, _I32P]),
    "lf_pool_frames": (ctypes.c_int, [_SHP, _P, _I32P, ctypes.c_int32, _P, _P]),
    "lf_select_chunk_cached": (ctypes.c_int, [_SHP, _P, _P, _I32P, _P, _P, _SZ, _P]),
    "lf_select_chunk_1d": (ctypes.c_int, [_SHP, _P, _P, _I32P, _P, _P, _SZ, _P]),
    "lf_attn_backward_workspace_size": (_SZ, [_SHP]),
    "lf_block_sparse_attn_backward": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _P, _I32P, _I32P] +
                                      [_P] * 11 + [_SZ, _P]),
    "lf_rope_frames": (ctypes.c_int, [_RPP, _P, _I64, _I32, _I32P, _I32P, _P, _P, _I32, _I32P,
                                      _P]),
    "lf_rope_backward_workspace_size": (_SZ, [_RPP]),
    "lf_rope_frames_backward": (ctypes.c_int, [_RPP, _P, _I64, _I32, _I32P, _I32P, _P, _P, _I32,
                                               _I32P, _P, _I64, _P, _P, _SZ, _P]),
    "lf_block_sparse_attn_noalloc": (ctypes.c_int, [_SHP, _P, _P, _P, _P, _P, _I32P, _I32P, _P,
                                                    _P, _P, _P]),
}


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads liblf.so (once) and declares its signatures.  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise FileNotFoundError(
                f"{path} is missing: build it with python -m block_sparse_attention_46_b200.build")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def make_shape(s) -> LfShape:
    """lf_shape from any object with the plain size fields (H, d, T, block, ...)."""
    return LfShape(s.H, s.d, s.T, s.block, s.n_cur_frames, s.n_hist, s.n_sink, s.n_slots,
                   s.k_f, s.k_b, s.scale, getattr(s, "k_c", 0))


def derived(s):
    """(n_bpf, n_qb, kf, kb) as the library derives them (for sizing output tensors)."""
    nbpf = -(-s.T // s.block)
    kf = min(s.k_f, s.n_hist) if s.n_hist > 0 else 0
    kb = min(s.k_b, nbpf) if s.n_hist > 0 else 0
    return nbpf, s.n_cur_frames * nbpf, kf, kb


def current_blocks(s) -> int:
    """kc, the current-chunk blocks kept per query block (0: the dense current chunk)."""
    nqb = s.n_cur_frames * -(-s.T // s.block)
    k_c = getattr(s, "k_c", 0)
    return min(k_c, nqb) if k_c > 0 else 0


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _slots(v: Sequence[int]):
    """Host list of int32 for a call, and the memory to keep alive during it.  ctypes alone would
    wrap what does not fit, silently."""
    try:
        n = array.array("i", v)                  # refuses what is no 32-bit integer
    except (TypeError, OverflowError):
        n = [int(x) for x in v]                  # 3.0 is one, 2.5 and 2^31 are not
        if not (-2 ** 31 <= min(n) and max(n) < 2 ** 31 and all(map(operator.eq, n, v))):
            raise ValueError(f"slots and positions are 32-bit integers, not {list(v)}") from None
    arr = (ctypes.c_int32 * max(len(n), 1))(*n)
    return arr, arr


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, where: str):
    if rc != LF_OK:
        raise LfError(rc, where)


def lf_status_string(code: int) -> str:
    return load().lf_status_string(code).decode()


def lf_abi_version() -> int:
    return load().lf_abi_version()


def lf_device_status(reset: bool = True) -> int:
    return load().lf_device_status(1 if reset else 0)


def lf_debug_configure(wait_limit_ns: int = 0, stall: int = 0, tail_split: bool = True):
    """Test hook: wait limit of the device waits, a stalled CTA (True: the first one), and whether
    the last partial wave of query tiles may be split (defaults restored by calling it with none)."""
    _check(load().lf_debug_configure(int(wait_limit_ns), int(stall), 1 if tail_split else 0),
           "lf_debug_configure")


def lf_compress(shape, q, k_cache, hist_slots, q_blk, k_blk, k_frm, stream=None):
    sh = make_shape(shape)
    hs, _keep = _slots(hist_slots)
    _check(load().lf_compress(ctypes.byref(sh), _ptr(q), _ptr(k_cache), hs, _ptr(q_blk),
                              _ptr(k_blk), _ptr(k_frm), _stream(stream)), "lf_compress")


def lf_select_frames(shape, q_blk, k_frm, frame_idx, frame_score=None, stream=None):
    sh = make_shape(shape)
    _check(load().lf_select_frames(ctypes.byref(sh), _ptr(q_blk), _ptr(k_frm), _ptr(frame_idx),
                                   _ptr(frame_score), _stream(stream)), "lf_select_frames")


def lf_select_blocks(shape, q_blk, k_blk, frame_idx, block_idx, block_score=None, stream=None):
    sh = make_shape(shape)
    _check(load().lf_select_blocks(ctypes.byref(sh), _ptr(q_blk), _ptr(k_blk), _ptr(frame_idx),
                                   _ptr(block_idx), _ptr(block_score), _stream(stream)),
           "lf_select_blocks")


def lf_select_workspace_size(shape) -> int:
    sh = make_shape(shape)
    return int(load().lf_select_workspace_size(ctypes.byref(sh)))


def lf_select_chunk(shape, q, k_cache, hist_slots, block_idx, workspace=None, stream=None):
    sh = make_shape(shape)
    hs, _keep = _slots(hist_slots)
    if workspace is None:
        workspace = torch.empty(max(lf_select_workspace_size(shape), 256), dtype=torch.uint8,
                                device=q.device)
    _check(load().lf_select_chunk(ctypes.byref(sh), _ptr(q), _ptr(k_cache), hs, _ptr(block_idx),
                                  _ptr(workspace), workspace.numel(), _stream(stream)),
           "lf_select_chunk")


def lf_select_chunk_1d(shape, q, k_cache, hist_slots, block_idx, workspace=None, stream=None):
    """One-dimensional selection (no frame stage): the kf*kb best blocks over all frames."""
    sh = make_shape(shape)
    hs, _keep = _slots(hist_slots)
    if workspace is None:
        workspace = torch.empty(max(lf_select_workspace_size(shape), 256), dtype=torch.uint8,
                                device=q.device)
    _check(load().lf_select_chunk_1d(ctypes.byref(sh), _ptr(q), _ptr(k_cache), hs,
                                     _ptr(block_idx), _ptr(workspace), workspace.numel(),
                                     _stream(stream)), "lf_select_chunk_1d")


def lf_select_current(shape, q, k_cur, cur_idx, workspace=None, stream=None):
    """Current-chunk block choice (shape.k_c >= 1): each query block's own block plus the
    k_c - 1 best-scoring other current blocks, into cur_idx [H, n_qb, kc]."""
    sh = make_shape(shape)
    if workspace is None:
        workspace = torch.empty(max(lf_forward_workspace_size(shape), 256), dtype=torch.uint8,
                                device=q.device)
    _check(load().lf_select_current(ctypes.byref(sh), _ptr(q), _ptr(k_cur), _ptr(cur_idx),
                                    _ptr(workspace), workspace.numel(), _stream(stream)),
           "lf_select_current")


def lf_pooled_cache_bytes(shape) -> int:
    sh = make_shape(shape)
    return int(load().lf_pooled_cache_bytes(ctypes.byref(sh)))


def lf_pool_frames(shape, k_cache, slots, k_pool, stream=None):
    """Block means of the keys of cache slots `slots` into the pooled-key cache k_pool
    (fp32 [n_slots, H, n_bpf, d])."""
    sh = make_shape(shape)
    sl, _keep = _slots(slots)
    _check(load().lf_pool_frames(ctypes.byref(sh), _ptr(k_cache), sl, len(slots), _ptr(k_pool),
                                 _stream(stream)), "lf_pool_frames")


def lf_select_chunk_cached(shape, q, k_pool, hist_slots, block_idx, workspace=None, stream=None):
    sh = make_shape(shape)
    hs, _keep = _slots(hist_slots)
    if workspace is None:
        workspace = torch.empty(max(lf_select_workspace_size(shape), 256), dtype=torch.uint8,
                                device=q.device)
    _check(load().lf_select_chunk_cached(ctypes.byref(sh), _ptr(q), _ptr(k_pool), hs,
                                         _ptr(block_idx), _ptr(workspace), workspace.numel(),
                                         _stream(stream)), "lf_select_chunk_cached")


def lf_cag_schedule(n_chunks, first, mean_sparsity, final_sparsity, n_hist=None, n_bpf=1,
                    kf_max=1):
    """Per-chunk keep ratios of the chunk-aware sparsity growth, and (if n_hist is given)
    the (k_f, k_b) budgets.  Host only.  Returns (keep, k_f, k_b); the last two are None
    without n_hist."""
    keep = (ctypes.c_float * n_chunks)()
    if n_hist is not None:
        nh = (ctypes.c_int32 * n_chunks)(*[int(x) for x in n_hist])
        kf = (ctypes.c_int32 * n_chunks)()
        kb = (ctypes.c_int32 * n_chunks)()
        args = (ctypes.cast(nh, _I32P), n_bpf, kf_max, keep, ctypes.cast(kf, _I32P),
                ctypes.cast(kb, _I32P))
    else:
        args = (None, n_bpf, kf_max, keep, None, None)
    _check(load().lf_cag_schedule(n_chunks, first, mean_sparsity, final_sparsity, *args),
           "lf_cag_schedule")
    if n_hist is None:
        return list(keep), None, None
    return list(keep), list(kf), list(kb)


def lf_attn_workspace_size(shape) -> int:
    sh = make_shape(shape)
    return int(load().lf_attn_workspace_size(ctypes.byref(sh)))


def lf_forward_workspace_size(shape) -> int:
    sh = make_shape(shape)
    return int(load().lf_forward_workspace_size(ctypes.byref(sh)))


def lf_block_sparse_attn(shape, q, k_cur, v_cur, k_cache, v_cache, hist_slots, sink_slots,
                         block_idx, out, lse=None, workspace=None, stream=None, cur_idx=None):
    sh = make_shape(shape)
    hs, _k1 = _slots(hist_slots)
    ss, _k2 = _slots(sink_slots)
    if workspace is None:
        workspace = torch.empty(max(lf_attn_workspace_size(shape), 256), dtype=torch.uint8,
                                device=q.device)
    _check(load().lf_block_sparse_attn(
        ctypes.byref(sh), _ptr(q), _ptr(k_cur), _ptr(v_cur), _ptr(k_cache), _ptr(v_cache), hs, ss,
        _ptr(block_idx), _ptr(cur_idx), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream(stream)), "lf_block_sparse_attn")


def lf_quantize_e4m3(x, x8, head_scale=None, row_scale=None, stream=None):
    """e4m3 codes of x [rows, H, d] bf16 into x8 (uint8, same shape): per head with the given
    scales [H], or per (row, head) with the scales written to row_scale [rows, H]."""
    rows, H, d = x.shape
    _check(load().lf_quantize_e4m3(_ptr(x), rows, H, d, _ptr(head_scale), _ptr(x8),
                                   _ptr(row_scale), _stream(stream)), "lf_quantize_e4m3")


def lf_e4m3_head_scales(xs, head_scale, stream=None):
    """Per-head power-of-two scales over the bf16 tensors xs (each [rows, H, d])."""
    n = len(xs)
    H, d = xs[0].shape[-2], xs[0].shape[-1]
    ptrs = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
    rows = (ctypes.c_int64 * n)(*[x.numel() // (H * d) for x in xs])
    for x in xs:
        _ptr(x)
    _check(load().lf_e4m3_head_scales(ptrs, rows, n, H, d, _ptr(head_scale), _stream(stream)),
           "lf_e4m3_head_scales")


def lf_block_sparse_attn_e4m3(shape, q8, q_scale, k_cur8, v_cur, k_cache8, v_cache, k_scale,
                              hist_slots, sink_slots, block_idx, out, lse=None, workspace=None,
                              stream=None, cur_idx=None):
    """(d) with e4m3 queries and keys (QK^T on the FP8 tensor cores), bf16 values."""
    sh = make_shape(shape)
    hs, _k1 = _slots(hist_slots)
    ss, _k2 = _slots(sink_slots)
    if workspace is None:
        workspace = torch.empty(max(lf_attn_workspace_size(shape), 256), dtype=torch.uint8,
                                device=q8.device)
    _check(load().lf_block_sparse_attn_e4m3(
        ctypes.byref(sh), _ptr(q8), _ptr(q_scale), _ptr(k_cur8), _ptr(v_cur), _ptr(k_cache8),
        _ptr(v_cache), _ptr(k_scale), hs, ss, _ptr(block_idx), _ptr(cur_idx), _ptr(out),
        _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)),
        "lf_block_sparse_attn_e4m3")


def lf_noalloc_scratch_bytes() -> int:
    return int(load().lf_noalloc_scratch_bytes())


def lf_block_sparse_attn_noalloc(shape, q, k_cur, v_cur, k_cache, v_cache, hist_slots,
                                 sink_slots, block_idx, out, lse=None, stream=None):
    """lf_block_sparse_attn without a workspace argument, for callers that cannot
    allocate device memory: the library's fixed scratch array is used instead (calls
    that overlap on the GPU must not share a device)."""
    sh = make_shape(shape)
    hs, _k1 = _slots(hist_slots)
    ss, _k2 = _slots(sink_slots)
    _check(load().lf_block_sparse_attn_noalloc(
        ctypes.byref(sh), _ptr(q), _ptr(k_cur), _ptr(v_cur), _ptr(k_cache), _ptr(v_cache), hs, ss,
        _ptr(block_idx), _ptr(out), _ptr(lse), _stream(stream)), "lf_block_sparse_attn_noalloc")


def lf_forward_chunk(shape, q, k_cur, v_cur, k_cache, v_cache, hist_slots, sink_slots,
                     out, lse=None, block_idx_out=None, workspace=None, stream=None,
                     cur_idx_out=None):
    sh = make_shape(shape)
    hs, _k1 = _slots(hist_slots)
    ss, _k2 = _slots(sink_slots)
    if workspace is None:
        workspace = torch.empty(max(lf_forward_workspace_size(shape), 256), dtype=torch.uint8,
                                device=q.device)
    _check(load().lf_forward_chunk(
        ctypes.byref(sh), _ptr(q), _ptr(k_cur), _ptr(v_cur), _ptr(k_cache), _ptr(v_cache), hs, ss,
        _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse), _ptr(block_idx_out),
        _ptr(cur_idx_out), _stream(stream)), "lf_forward_chunk")


# ------------------------------------------------------------------ gradient, rotary positions
# These calls are small next to what they launch only when their checks are: one look at each
# tensor, plain integers for pointers, the device switched only when it is another one.
def _arg(what, name, t, device, dtype, count=None):
    """Address of a contiguous tensor after checking what the C side cannot see of it: its
    device, type and number of elements.  None stays None."""
    if t is None:
        return None
    if t.device != device or t.dtype != dtype:
        raise ValueError(f"{what}: {name} is {t.dtype} on {t.device}, not {dtype} on {device}")
    if count is not None and t.numel() != count:
        raise ValueError(f"{what}: {name} has {t.numel()} elements, not {count}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous")
    return t.data_ptr()


def _on_gpu(what, name, t):
    if t is None or t.device.type != "cuda":
        raise ValueError(f"{what}: {name} must be a CUDA tensor")
    return t.device


def _device(device):
    """Makes `device` current for a call, if it is not."""
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream_handle(stream):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _workspace(what, workspace, size, device, stream):
    """(tensor, address, bytes): the caller's workspace, or one of size() bytes from the memory
    of the stream that the call runs on, which may be reused once that stream is past the call."""
    if workspace is None:
        n = size()
        if n == 0:
            return None, None, 0
        with torch.cuda.stream(stream):               # None: the current stream
            workspace = torch.empty(n, dtype=torch.uint8, device=device)
    return workspace, _arg(what, "workspace", workspace, device, torch.uint8), workspace.numel()


def lf_attn_backward_workspace_size(shape) -> int:
    sh = make_shape(shape)
    return int(load().lf_attn_backward_workspace_size(ctypes.byref(sh)))


def lf_block_sparse_attn_backward(shape, q, k_cur, v_cur, k_cache, v_cache, hist_slots,
                                  sink_slots, block_idx, out, dout, lse, dq, dk_cur, dv_cur,
                                  dk_cache=None, dv_cache=None, workspace=None, stream=None,
                                  cur_idx=None):
    """Gradient of lf_block_sparse_attn (or of the attention of lf_forward_chunk): dq, dk_cur
    and dv_cur, and with dk_cache and dv_cache the gradient into the listed cache slots, from
    the forward call's out and lse and the gradient dout of out."""
    what = "lf_block_sparse_attn_backward"
    sh = make_shape(shape)
    dev, bf, i32 = _on_gpu(what, "q", q), torch.bfloat16, torch.int32
    if len(hist_slots) != sh.n_hist or len(sink_slots) != sh.n_sink:
        raise ValueError(f"{what}: slot lists do not match the shape's frames")
    if sh.d < 1 or sh.block < 1:
        _check(LF_ERR_UNSUPPORTED, what)
    _, nqb, kf, kb = derived(shape)
    row = sh.H * sh.d
    chunk = sh.n_cur_frames * sh.tokens_per_frame * row
    cached = sh.n_slots * sh.tokens_per_frame * row if sh.n_hist + sh.n_sink > 0 else None
    cur = [_arg(what, n, t, dev, bf, chunk) for n, t in
           (("q", q), ("k_cur", k_cur), ("v_cur", v_cur), ("out", out), ("dout", dout),
            ("dq", dq), ("dk_cur", dk_cur), ("dv_cur", dv_cur))]
    cache = [_arg(what, n, t, dev, bf, cached) for n, t in
             (("k_cache", k_cache), ("v_cache", v_cache), ("dk_cache", dk_cache),
              ("dv_cache", dv_cache))]
    p_lse = _arg(what, "lse", lse, dev, torch.float32, chunk // sh.d)
    p_bi = _arg(what, "block_idx", block_idx, dev, i32, sh.H * nqb * kf * kb) if sh.n_hist else None
    kc = current_blocks(shape)
    p_ci = _arg(what, "cur_idx", cur_idx, dev, i32, sh.H * nqb * kc) if kc else None
    hs, _k1 = _slots(hist_slots)
    ss, _k2 = _slots(sink_slots)
    lib = load()
    with _device(dev):
        _ws, p_ws, n_ws = _workspace(
            what, workspace, lambda: lib.lf_attn_backward_workspace_size(ctypes.byref(sh)), dev, stream)
        _check(lib.lf_block_sparse_attn_backward(
            ctypes.byref(sh), cur[0], cur[1], cur[2], cache[0], cache[1], hs, ss, p_bi, p_ci,
            cur[3], cur[4], p_lse, cur[5], cur[6], cur[7], cache[2], cache[3], p_ws, n_ws,
            _stream_handle(stream)), what)


_NORMS = {None: 0, "head": 1, "token": 2, "row": 2}


def make_rope(H, d, n_frames, height, width, pairs, halves=False, norm=None, base=10000.0,
              eps=1e-6) -> LfRope:
    """lf_rope: heads, head dimension, frames and their token grid, channel pairs per axis
    (time, height, width), pairing, norm (None, "head" or "row", over the whole token)."""
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {list(_NORMS)}")
    sizes = [H, d, n_frames, height, width, *[int(p) for p in pairs]]
    if not (-2 ** 31 <= min(sizes) and max(sizes) < 2 ** 31):
        raise ValueError(f"sizes are 32-bit integers, not {sizes}")
    return LfRope(*sizes, 1 if halves else 0, _NORMS[norm], eps, base)


def _rope_tokens(H, d, T, t, name, device, contiguous):
    """(address, elements between tokens, frames) of bf16 tokens [..., H, d] whose leading
    dimensions are frames x tokens at one stride."""
    what = "lf_rope"
    if t.device != device or t.dtype != torch.bfloat16:
        raise ValueError(f"{what}: {name} is {t.dtype} on {t.device}, not bf16 on {device}")
    shape, row = t.shape, H * d
    n, rest = divmod(t.numel(), T * row)
    if len(shape) < 3 or shape[-2] != H or shape[-1] != d or rest:
        raise ValueError(f"{what}: {name} must be [frames, {T}, {H}, {d}] or [frames * {T}, {H}, {d}]")
    if t.is_contiguous():
        return t.data_ptr(), row, n
    if contiguous:
        raise ValueError(f"{what}: {name} must be contiguous")
    strides = t.stride()
    if (strides[-1] != 1 and d > 1) or (strides[-2] != d and H > 1):
        raise ValueError(f"{what}: a token's H * d channels of {name} must be contiguous")
    stride = step = None                              # None: only dimensions of one token yet
    for s, st in zip(shape[-3::-1], strides[-3::-1]):
        if s == 1:
            continue
        if step is None:
            if st < row:                              # broadcast or overlapping tokens
                raise ValueError(f"{what}: {name}'s tokens share memory")
            stride = step = st
        if st != step:
            raise ValueError(f"{what}: {name}'s tokens are not at one stride")
        step *= s
    return t.data_ptr(), row if stride is None else stride, n


def _frames(n_frames, v, name):
    if v is None:
        return None, None
    if len(v) != n_frames:
        raise ValueError(f"lf_rope: {name} needs one entry per frame")
    return _slots(v)


def lf_rope_frames(rope, x, out, frame_pos=None, weight=None, in_slots=None, out_slots=None,
                   stream=None):
    """Norm and rotary positions of n_frames frames of x [n_in, T, H, d] (tokens may lie
    inside a wider projection) into out [n_out, T, H, d], through optional slot lists."""
    dev = _on_gpu("lf_rope", "x", x)
    H, d, T, F, norm = rope.H, rope.d, rope.height * rope.width, rope.n_frames, rope.norm
    if H < 1 or d < 1 or T < 1:
        _check(LF_ERR_INVALID_ARG, "lf_rope_frames")
    px, xs, n_in = _rope_tokens(H, d, T, x, "x", dev, False)
    po, _, n_out = _rope_tokens(H, d, T, out, "out", dev, True)
    pw = _arg("lf_rope", "weight", weight, dev, torch.float32, d if norm == 1 else H * d)
    si, _k1 = _frames(F, in_slots, "in_slots")
    so, _k2 = _frames(F, out_slots, "out_slots")
    fp, _k3 = _frames(F, frame_pos, "frame_pos")
    with _device(dev):
        _check(load().lf_rope_frames(ctypes.byref(rope), px, xs, n_in, si, fp, pw, po, n_out, so,
                                     _stream_handle(stream)), "lf_rope_frames")


def lf_rope_backward_workspace_size(rope) -> int:
    return int(load().lf_rope_backward_workspace_size(ctypes.byref(rope)))


def lf_rope_frames_backward(rope, x, dout, dx, frame_pos=None, weight=None, dweight=None,
                            in_slots=None, out_slots=None, workspace=None, stream=None):
    """Gradient of lf_rope_frames: dx (x's frames and slots, its own token stride) and, with a
    norm, dweight, from dout.  x may be None without a norm."""
    dev = _on_gpu("lf_rope", "dx", dx)
    H, d, T, F, norm = rope.H, rope.d, rope.height * rope.width, rope.n_frames, rope.norm
    if H < 1 or d < 1 or T < 1:
        _check(LF_ERR_INVALID_ARG, "lf_rope_frames_backward")
    px, xs = None, 0
    pd, ds, n_in = _rope_tokens(H, d, T, dx, "dx", dev, False)
    if x is not None:
        px, xs, n_x = _rope_tokens(H, d, T, x, "x", dev, False)
        if n_x != n_in:
            raise ValueError("lf_rope: x and dx differ in frames")
    pg, _, n_out = _rope_tokens(H, d, T, dout, "dout", dev, True)
    n_w = d if norm == 1 else H * d
    pw = _arg("lf_rope", "weight", weight, dev, torch.float32, n_w)
    pdw = _arg("lf_rope", "dweight", dweight, dev, torch.float32, n_w)
    si, _k1 = _frames(F, in_slots, "in_slots")
    so, _k2 = _frames(F, out_slots, "out_slots")
    fp, _k3 = _frames(F, frame_pos, "frame_pos")
    lib = load()
    with _device(dev):
        _ws, p_ws, size = _workspace(
            "lf_rope", workspace, lambda: lib.lf_rope_backward_workspace_size(ctypes.byref(rope)),
            dev, stream)
        _check(lib.lf_rope_frames_backward(
            ctypes.byref(rope), px, xs, n_in, si, fp, pw, pg, n_out, so, pd, ds, pdw, p_ws, size,
            _stream_handle(stream)), "lf_rope_frames_backward")
