"""ctypes binding of libvkv (include/vkv.h): argument marshalling only (the paged cache
calls' in csrc/vkv_binding.cpp).

Every computation runs in the library's sm_100a kernels; this module turns
torch tensors into the C structs, passes the current CUDA stream and raises
on a non-OK status.  There is no fallback: if libvkv.so is missing or no
sm_100 device is present the calls raise.

Raw entry points with the C names: ``vkv_chunk_attn``, ``vkv_block_select``,
``vkv_block_select_workspace_size``, ``vkv_lse_merge``, ``vkv_latent_attn``,
``vkv_page_map``, ``vkv_page_append``, ``vkv_page_select``, ``vkv_page_attn``,
``vkv_status_string`` (and the other entry points of the header).
Convenience wrappers that allocate outputs with torch: ``chunk_attn_segments``,
``chunk_attn_block_sparse``, ``chunk_attn_ragged``, ``block_select``, ``lse_merge``,
``latent_attn``, the paged cache's ``page_map``, ``page_append``, ``page_select`` and
``page_attn``, and the others below.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from ctypes import POINTER, c_float, c_int32, c_int64, c_size_t, c_void_p

import numpy as np
import torch

from . import build

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvkv.so")
LIB_TEST_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvkv_test.so")

MODE_SEGMENTS, MODE_BLOCK_SPARSE, MODE_RAGGED = 0, 1, 2
MAX_BRANCHES, MAX_SEGMENTS = 2, 8
DEVERR_TIMEOUT, DEVERR_BAD_INDEX, DEVERR_BAD_OFFSETS, DEVERR_NO_SPACE = 1, 2, 3, 4
DTYPE_BF16, DTYPE_FP16, DTYPE_E4M3 = 0, 1, 2
PAGE_ATTN_CLEAR_BYTES = 4096  # VKV_PAGE_ATTN_CLEAR_BYTES in include/vkv.h
NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024  # VKV_NOALLOC_SCRATCH_BYTES in include/vkv.h
STATUS = {0: "VKV_OK", 1: "VKV_ERR_NULL", 2: "VKV_ERR_SHAPE", 3: "VKV_ERR_ALIGN", 4: "VKV_ERR_RANGE",
          5: "VKV_ERR_UNSUPPORTED", 6: "VKV_ERR_CUDA", 7: "VKV_ERR_WORKSPACE"}


class VkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({vkv_status_string(status)})")


class vkv_segment(ctypes.Structure):
    _fields_ = [("start", c_int32), ("len", c_int32)]


class vkv_tensor(ctypes.Structure):
    _fields_ = [("ptr", c_void_p), ("sb", c_int64), ("st", c_int64), ("sh", c_int64)]


class vkv_attn_args(ctypes.Structure):
    _fields_ = [
        ("mode", c_int32), ("B", c_int32), ("H", c_int32), ("Lq", c_int32), ("Lkv", c_int32),
        ("d", c_int32), ("scale", c_float),
        ("q", vkv_tensor), ("k", vkv_tensor), ("v", vkv_tensor),
        ("n_branches", c_int32),
        ("segs", POINTER(vkv_segment) * MAX_BRANCHES),
        ("n_segs", c_int32 * MAX_BRANCHES),
        ("block", c_int32),
        ("persist_idx", c_void_p), ("n_persist", c_int32),
        ("sel_idx", c_void_p), ("topk", c_int32), ("window_blk0", c_int32), ("n_win_blk", c_int32),
        ("cu_seqlens", c_void_p), ("cu_seqlens_host", POINTER(c_int32)),
        ("o", vkv_tensor * MAX_BRANCHES), ("lse", c_void_p * MAX_BRANCHES),
        ("o_merged", vkv_tensor), ("lse_merged", c_void_p),
        ("err_word", c_void_p),
        ("qblk_order", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("kbar", c_void_p), ("sel_out", c_void_p),
    ]


class vkv_select_args(ctypes.Structure):
    _fields_ = [
        ("B", c_int32), ("H", c_int32), ("d", c_int32), ("block", c_int32),
        ("Lq", c_int32), ("Lkv", c_int32), ("window_blk0", c_int32), ("n_win_blk", c_int32),
        ("topk", c_int32),
        ("q", vkv_tensor), ("k", vkv_tensor),
        ("out_idx", c_void_p), ("out_scores", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("err_word", c_void_p),
        ("out_order", c_void_p),
        ("kbar", c_void_p),
    ]


class vkv_head_rule(ctypes.Structure):
    _fields_ = [("policy", c_int32), ("param", c_int32)]


class vkv_compact_args(ctypes.Structure):
    _fields_ = [
        ("B", c_int32), ("H", c_int32), ("d", c_int32), ("frame_tokens", c_int32),
        ("hist_frames", c_int32), ("cur_frames", c_int32), ("recent_frames", c_int32),
        ("k_src", vkv_tensor), ("v_src", vkv_tensor),
        ("rules", POINTER(vkv_head_rule)),
        ("k_out", c_void_p), ("v_out", c_void_p), ("out_rows", c_int64),
        ("cu_seqlens", c_void_p), ("cu_seqlens_host", POINTER(c_int32)),
    ]


HEAD_FULL, HEAD_ANCHOR, HEAD_WAVE, HEAD_VEIL = 0, 1, 2, 3


class vkv_persist_args(ctypes.Structure):
    _fields_ = [
        ("B", c_int32), ("H", c_int32), ("d", c_int32), ("block", c_int32),
        ("Lq", c_int32), ("Lkv", c_int32),
        ("q", vkv_tensor), ("k", vkv_tensor),
        ("persist_idx", c_void_p), ("n_persist", c_int32),
        ("evict_blk0", c_int32), ("n_evict", c_int32),
        ("out_idx", c_void_p), ("out_scores", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("err_word", c_void_p),
    ]

class vkv_latent_args(ctypes.Structure):
    _fields_ = [
        ("B", c_int32), ("H", c_int32), ("Lq", c_int32), ("Lkv", c_int32),
        ("d_c", c_int32), ("d_rope", c_int32), ("scale", c_float),
        ("q", vkv_tensor), ("kv", vkv_tensor), ("kr", vkv_tensor), ("o", vkv_tensor),
        ("lse", c_void_p), ("err_word", c_void_p),
    ]

class vkv_page_map_args(ctypes.Structure):
    _fields_ = [
        ("R", c_int32), ("W", c_int32), ("page", c_int32), ("n_ring", c_int32), ("max_tokens", c_int32),
        ("reserved", c_int32),
        ("kv_len", c_void_p), ("new_len", c_void_p), ("table", c_void_p), ("table_stride", c_int64),
        ("ring", c_void_p), ("ring_pos", c_void_p), ("kv_len_out", c_void_p), ("ring_pos_out", c_void_p),
        ("slot", c_void_p), ("row", c_void_p), ("pos", c_void_p), ("cu", c_void_p), ("err_word", c_void_p),
    ]


class vkv_page_append_args(ctypes.Structure):
    _fields_ = [
        ("T", c_int32), ("Hkv", c_int32), ("d", c_int32), ("page", c_int32), ("n_pages", c_int32),
        ("x_dtype", c_int32), ("kv_dtype", c_int32), ("reserved", c_int32),
        ("k_new", vkv_tensor), ("v_new", vkv_tensor), ("k", vkv_tensor), ("v", vkv_tensor),
        ("slot", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p), ("kbar", c_void_p),
        ("err_word", c_void_p),
    ]


class vkv_page_select_args(ctypes.Structure):
    _fields_ = [
        ("R", c_int32), ("H", c_int32), ("Hkv", c_int32), ("d", c_int32), ("page", c_int32), ("n_pages", c_int32),
        ("W", c_int32), ("topk", c_int32), ("sink_pages", c_int32), ("local_pages", c_int32),
        ("q_dtype", c_int32), ("reserved", c_int32),
        ("q", vkv_tensor), ("kbar", c_void_p), ("table", c_void_p), ("table_stride", c_int64),
        ("kv_len", c_void_p), ("sel", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
        ("err_word", c_void_p),
    ]


class vkv_page_attn_args(ctypes.Structure):
    _fields_ = [
        ("R", c_int32), ("H", c_int32), ("Hkv", c_int32), ("d", c_int32), ("page", c_int32), ("n_pages", c_int32),
        ("W", c_int32), ("q_dtype", c_int32), ("kv_dtype", c_int32), ("scale", c_float), ("sink", c_int32),
        ("window", c_int32), ("topk", c_int32), ("reserved", c_int32),
        ("q", vkv_tensor), ("o", vkv_tensor), ("k", vkv_tensor), ("v", vkv_tensor),
        ("table", c_void_p), ("table_stride", c_int64), ("kv_len", c_void_p), ("sel", c_void_p),
        ("k_scale", c_void_p), ("v_scale", c_void_p), ("lse", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("err_word", c_void_p),
    ]


class vkv_schedule(ctypes.Structure):
    _fields_ = [
        ("n_ctas", c_int32), ("n_units", c_int32), ("n_pieces", c_int32), ("n_slots", c_int32),
        ("cta_begin", POINTER(c_int32)), ("cta_piece0", POINTER(c_int32)),
        ("units", POINTER(ctypes.c_uint32)), ("pieces", POINTER(ctypes.c_uint32)),
    ]


_lib = None
_test_lib = None


def lib() -> ctypes.CDLL:
    """Load libvkv.so (built in-tree by kv_cache_attention_chunk_b200.build); raise if absent."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


def test_lib() -> ctypes.CDLL:
    """Load the test build libvkv_test.so: the same library plus the test aids of
    include/vkv_test.h (vkv_debug_withhold_copy)."""
    global _test_lib
    if _test_lib is None:
        L = _load(LIB_TEST_PATH)
        L.vkv_debug_withhold_copy.argtypes = [c_int32]
        L.vkv_debug_withhold_copy.restype = c_int32
        L.vkv_debug_exp2_poly.argtypes = [c_void_p, c_void_p, c_int32, c_void_p]
        L.vkv_debug_exp2_poly.restype = c_int32
        _test_lib = L
    return _test_lib


@contextlib.contextmanager
def using_test_library():
    """Route the calls of this module through the test build while the block runs."""
    global _lib
    saved = lib()
    _lib = test_lib()
    try:
        yield _lib
    finally:
        _lib = saved


def _load(path: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m kv_cache_attention_chunk_b200.build`"
                           " (there is no fallback implementation)")
    L = ctypes.CDLL(path)
    L.vkv_chunk_attn.argtypes = [POINTER(vkv_attn_args), c_void_p]
    L.vkv_chunk_attn.restype = c_int32
    L.vkv_chunk_attn_workspace_size.argtypes = [POINTER(vkv_attn_args)]
    L.vkv_chunk_attn_workspace_size.restype = c_size_t
    L.vkv_debug_schedule.argtypes = [POINTER(vkv_attn_args), c_int32, c_int32, POINTER(vkv_schedule)]
    L.vkv_debug_schedule.restype = c_int32
    L.vkv_block_select.argtypes = [POINTER(vkv_select_args), c_void_p]
    L.vkv_block_select.restype = c_int32
    L.vkv_block_select_noalloc.argtypes = [POINTER(vkv_select_args), c_void_p]
    L.vkv_block_select_noalloc.restype = c_int32
    L.vkv_block_select_workspace_size.argtypes = [c_int32] * 6
    L.vkv_block_select_workspace_size.restype = c_size_t
    L.vkv_block_order.argtypes = [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p]
    L.vkv_block_order.restype = c_int32
    L.vkv_lse_merge.argtypes = [vkv_tensor, c_void_p, vkv_tensor, c_void_p, vkv_tensor, c_void_p,
                                c_int32, c_int32, c_int32, c_int32, c_void_p]
    L.vkv_lse_merge.restype = c_int32
    L.vkv_status_string.argtypes = [c_int32]
    L.vkv_status_string.restype = ctypes.c_char_p
    L.vkv_version.argtypes = []
    L.vkv_version.restype = c_int32
    L.vkv_abi_sizeof.argtypes = [c_int32]
    L.vkv_abi_sizeof.restype = c_int32
    L.vkv_block_pool.argtypes = [vkv_tensor, c_int32, c_int32, c_int32, c_int32, c_int32, c_int32, c_void_p,
                                 c_void_p]
    L.vkv_block_pool.restype = c_int32
    L.vkv_compact_rows.argtypes = [POINTER(vkv_compact_args)]
    L.vkv_compact_rows.restype = c_int64
    L.vkv_compact_cache.argtypes = [POINTER(vkv_compact_args), c_void_p]
    L.vkv_compact_cache.restype = c_int32
    L.vkv_persist_update_workspace_size.argtypes = [c_int32] * 7
    L.vkv_persist_update_workspace_size.restype = c_size_t
    L.vkv_persist_update.argtypes = [POINTER(vkv_persist_args), c_void_p]
    L.vkv_persist_update.restype = c_int32
    L.vkv_latent_attn.argtypes = [POINTER(vkv_latent_args), c_void_p]
    L.vkv_latent_attn.restype = c_int32
    for name in ("vkv_page_map", "vkv_page_append", "vkv_page_select", "vkv_page_attn"):
        fn = getattr(L, name)
        fn.argtypes = [c_void_p, c_void_p]
        fn.restype = c_int32
    L.page_entry = {name: ctypes.cast(getattr(L, "vkv_" + name), c_void_p).value
                    for name in ("page_map", "page_append", "page_select", "page_attn")}
    L.vkv_page_select_workspace_size.argtypes = [c_int32] * 3
    L.vkv_page_select_workspace_size.restype = c_size_t
    L.vkv_page_attn_workspace_size.argtypes = [c_int32] * 3
    L.vkv_page_attn_workspace_size.restype = c_size_t
    for i, st in enumerate((vkv_attn_args, vkv_select_args, vkv_tensor, vkv_segment, vkv_compact_args,
                            vkv_head_rule, vkv_persist_args, vkv_latent_args, vkv_schedule,
                            vkv_page_map_args, vkv_page_append_args, vkv_page_select_args, vkv_page_attn_args)):
        if L.vkv_abi_sizeof(i) != ctypes.sizeof(st):
            raise RuntimeError(f"ABI mismatch for {st.__name__}: C {L.vkv_abi_sizeof(i)} B, "
                               f"binding {ctypes.sizeof(st)} B")
    return L


# ---------------------------------------------------------------------------
# raw entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def vkv_status_string(status: int) -> str:
    return lib().vkv_status_string(int(status)).decode()


def vkv_chunk_attn(args: vkv_attn_args, stream: int | None) -> int:
    return int(lib().vkv_chunk_attn(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_chunk_attn_workspace_size(args: vkv_attn_args) -> int:
    return int(lib().vkv_chunk_attn_workspace_size(ctypes.byref(args)))


def vkv_debug_schedule(args: vkv_attn_args, n_sm: int, split: int, out: vkv_schedule) -> int:
    return int(lib().vkv_debug_schedule(ctypes.byref(args), int(n_sm), int(split), ctypes.byref(out)))


def attn_schedule(args: vkv_attn_args, n_sm: int, split: bool) -> dict:
    """The work schedule of vkv_chunk_attn for these arguments on `n_sm` SMs (host only):
    numpy arrays cta_begin, cta_piece0, units (uint32 codes), pieces ([n, 2] uint32) and n_slots."""
    cb = np.zeros(n_sm + 1, np.int32)
    cp = np.zeros(n_sm + 1, np.int32)
    un = np.zeros(6144, np.uint32)
    pc = np.zeros(2 * 384, np.uint32)
    out = vkv_schedule(0, 0, 0, 0, cb.ctypes.data_as(POINTER(c_int32)), cp.ctypes.data_as(POINTER(c_int32)),
                       un.ctypes.data_as(POINTER(ctypes.c_uint32)), pc.ctypes.data_as(POINTER(ctypes.c_uint32)))
    _check(vkv_debug_schedule(args, n_sm, 1 if split else 0, out), "vkv_debug_schedule")
    g = out.n_ctas
    return {"cta_begin": cb[:g + 1].copy(), "cta_piece0": cp[:g + 1].copy(), "units": un[:out.n_units].copy(),
            "pieces": pc[:2 * out.n_pieces].reshape(-1, 2).copy(), "n_slots": out.n_slots}


def vkv_block_select(args: vkv_select_args, stream: int | None) -> int:
    return int(lib().vkv_block_select(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_block_select_noalloc(args: vkv_select_args, stream: int | None) -> int:
    """vkv_block_select with the library's own fixed scratch array (no workspace argument)."""
    return int(lib().vkv_block_select_noalloc(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_block_order(sel_idx, out_order, BH, n_qblk, topk, stream: int | None) -> int:
    return int(lib().vkv_block_order(c_void_p(sel_idx), c_void_p(out_order), int(BH), int(n_qblk), int(topk),
                                     c_void_p(stream or 0)))


def block_order(sel_idx, out=None, stream=None):
    """Query-block order [B*H, nQblk] grouping similar selections, from a selection
    sel_idx (device int32 [B*H, nQblk, topk], e.g. the sel_out of chunk_attn_block_sparse
    with kbar), for a later call's qblk_order."""
    sel_idx = _contiguous(sel_idx, stream)
    BH, n_qblk, topk = sel_idx.shape
    order = out if out is not None else _new_outputs(sel_idx, stream, ((BH, n_qblk), torch.int32))[0]
    _check(vkv_block_order(sel_idx.data_ptr(), order.data_ptr(), BH, n_qblk, topk, _stream(stream)),
           "vkv_block_order")
    return order


def vkv_block_pool(x: vkv_tensor, B, L, H, d, blk0, n_blk, out, stream: int | None) -> int:
    return int(lib().vkv_block_pool(x, B, L, H, d, blk0, n_blk, c_void_p(out), c_void_p(stream or 0)))


def vkv_persist_update_workspace_size(B, H, Lq, n_persist, n_evict, block, d) -> int:
    return int(lib().vkv_persist_update_workspace_size(B, H, Lq, n_persist, n_evict, block, d))


def vkv_persist_update(args: vkv_persist_args, stream: int | None) -> int:
    return int(lib().vkv_persist_update(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_latent_attn(args: vkv_latent_args, stream: int | None) -> int:
    return int(lib().vkv_latent_attn(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_page_map(args: vkv_page_map_args, stream: int | None) -> int:
    return int(lib().vkv_page_map(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_page_append(args: vkv_page_append_args, stream: int | None) -> int:
    return int(lib().vkv_page_append(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_page_select(args: vkv_page_select_args, stream: int | None) -> int:
    return int(lib().vkv_page_select(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_page_attn(args: vkv_page_attn_args, stream: int | None) -> int:
    return int(lib().vkv_page_attn(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_page_select_workspace_size(R, Hkv, W) -> int:
    return int(lib().vkv_page_select_workspace_size(R, Hkv, W))


def vkv_page_attn_workspace_size(H, Hkv, d) -> int:
    return int(lib().vkv_page_attn_workspace_size(H, Hkv, d))


def vkv_debug_withhold_copy(n_calls: int) -> int:
    """Test aid of the test build (include/vkv_test.h): the next n_calls attention
    launches of libvkv_test.so withhold their first cache-tile copy."""
    return int(test_lib().vkv_debug_withhold_copy(int(n_calls)))


def vkv_compact_rows(args: vkv_compact_args) -> int:
    return int(lib().vkv_compact_rows(ctypes.byref(args)))


def vkv_compact_cache(args: vkv_compact_args, stream: int | None) -> int:
    return int(lib().vkv_compact_cache(ctypes.byref(args), c_void_p(stream or 0)))


def vkv_block_select_workspace_size(B, H, Lq, n_win_blk, block, d) -> int:
    return int(lib().vkv_block_select_workspace_size(B, H, Lq, n_win_blk, block, d))


def vkv_lse_merge(o_a: vkv_tensor, lse_a, o_b: vkv_tensor, lse_b, o_out: vkv_tensor, lse_out,
                  B, H, Lq, d, stream: int | None) -> int:
    return int(lib().vkv_lse_merge(o_a, c_void_p(lse_a), o_b, c_void_p(lse_b), o_out, c_void_p(lse_out),
                                   B, H, Lq, d, c_void_p(stream or 0)))


# ---------------------------------------------------------------------------
# torch helpers
# ---------------------------------------------------------------------------
def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _handle(di, stream):
    """The stream handle for a call on device `di` (-1, no GPU tensor: refused by the call)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(di) if di >= 0 else 0
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _stream_of(di, sh):
    """The torch stream of a handle on device `di`."""
    return torch.cuda.ExternalStream(sh, device=di) if sh else torch.cuda.default_stream(di)


def _made_on(x, stream, make):
    """make()'s tensors, on the device of `x`, for a call on `stream`: memory of that stream (what the current
    stream last used could still be written there), and not handed out again, once they are freed, before
    the current stream is done with what it has of them by then.  The caller orders the inputs before
    `stream`, and `stream` before what uses the results."""
    di = x.get_device()
    if stream is None or di < 0 or _handle(di, stream) == torch._C._cuda_getCurrentRawStream(di):
        return make()
    with torch.cuda.stream(_stream_of(di, _handle(di, stream))):
        out = make()
    for y in out:
        y.record_stream(torch.cuda.current_stream(di))
    return out


def _new_outputs(x, stream, *specs):
    """Tensors (shape, type) on the device of `x` for a call on `stream` to write."""
    return _made_on(x, stream, lambda: [torch.empty(shape, dtype=t, device=x.device) for shape, t in specs])


def _contiguous(x, stream):
    """`x`, or a copy that a call on `stream` may read, made there."""
    return x if x.is_contiguous() else _made_on(x, stream, lambda: [x.contiguous()])[0]


def tensor_desc(x: torch.Tensor) -> vkv_tensor:
    """[B, L, H, d] bf16 with a contiguous last axis -> vkv_tensor."""
    if x.dim() != 4 or x.dtype != torch.bfloat16 or x.stride(3) != 1:
        raise ValueError("expected a bf16 [B, L, H, d] tensor with contiguous d")
    return vkv_tensor(x.data_ptr(), x.stride(0), x.stride(1), x.stride(2))


def flat_desc(x: torch.Tensor) -> vkv_tensor:
    """[rows, d] bf16 with contiguous d -> vkv_tensor (row stride in st)."""
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.stride(1) != 1:
        raise ValueError("expected a bf16 [rows, d] tensor with contiguous d")
    return vkv_tensor(x.data_ptr(), 0, x.stride(0), 0)


def _check(status: int, what: str):
    if status != 0:
        raise VkvError(status, what)


def _base_args(mode, q, Lkv, d, scale, k_desc, v_desc, err):
    B, Lq, H, dq = q.shape
    if dq != d:
        raise ValueError("head dimension mismatch")
    a = vkv_attn_args()
    a.mode = mode
    a.B, a.H, a.Lq, a.Lkv, a.d = B, H, Lq, Lkv, d
    a.scale = float(scale if scale is not None else 1.0 / np.sqrt(d))
    a.q = tensor_desc(q)
    a.k = k_desc
    a.v = v_desc
    a.block = 64
    a.err_word = err.data_ptr() if err is not None else None
    return a


_attn_ws: dict = {}  # (device index, stream handle) -> uint8 device buffer, grown on demand


def _attn_workspace(a: vkv_attn_args, q: torch.Tensor, stream, split: bool, workspace):
    """Point the call at a key-axis split workspace: the caller's, or one kept per
    (device, stream) by this module; none when split is False or the schedule
    splits nothing.  Returns the buffer (kept alive by the caller until launch)."""
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
        return workspace
    if not split:
        return None
    need = vkv_chunk_attn_workspace_size(a)
    if need == 0:
        return None
    key = (q.device.index, _stream(stream))
    buf = _attn_ws.get(key)
    if buf is None or buf.numel() < need:
        buf, = _new_outputs(q, stream, (need, torch.uint8))
        _attn_ws[key] = buf
    a.workspace = buf.data_ptr()
    a.workspace_bytes = buf.numel()
    return buf


def _new_out(q, stream):
    B, Lq, H, d = q.shape
    return tuple(_new_outputs(q, stream, ((B, Lq, H, d), torch.bfloat16), ((B, H, Lq), torch.float32)))


def segments_args(q, k, v, branches, scale=None, err=None) -> vkv_attn_args:
    """vkv_attn_args of a SEGMENTS call, inputs filled in, outputs left empty (the
    segment arrays are kept alive by the returned struct)."""
    d = q.shape[3]
    a = _base_args(MODE_SEGMENTS, q, k.shape[1], d, scale, tensor_desc(k), tensor_desc(v), err)
    a.n_branches = len(branches)
    keep = []
    for i, br in enumerate(branches):
        arr = (vkv_segment * max(1, len(br)))(*[vkv_segment(int(s), int(n)) for s, n in br])
        keep.append(arr)
        a.segs[i] = ctypes.cast(arr, POINTER(vkv_segment))
        a.n_segs[i] = len(br)
    a._keep_segs = keep
    return a


def chunk_attn_segments(q, k, v, branches, scale=None, merged=True, err=None, stream=None, out=None,
                        split=True, workspace=None):
    """Dual-branch (or single-branch) chunk attention over token segments.

    branches: list (length 1 or 2) of lists of (start, len) cache-row segments.
    split: let the schedule cut units along the key axis (a workspace kept by this
    module; `workspace`, a device uint8 tensor, overrides it).
    Returns dict(o=[...], lse=[...], o_merged, lse_merged).
    """
    nb = len(branches)
    a = segments_args(q, k, v, branches, scale, err)
    res = out if out is not None else {}
    if out is None:
        res["o"], res["lse"] = [], []
        for _ in range(nb):
            o, l = _new_out(q, stream)
            res["o"].append(o)
            res["lse"].append(l)
        res["o_merged"], res["lse_merged"] = _new_out(q, stream) if (merged and nb == 2) else (None, None)
    for i in range(nb):
        a.o[i] = tensor_desc(res["o"][i])
        a.lse[i] = res["lse"][i].data_ptr()
    if res.get("o_merged") is not None:
        a.o_merged = tensor_desc(res["o_merged"])
        a.lse_merged = res["lse_merged"].data_ptr()
    sh = _stream(stream)
    ws = _attn_workspace(a, q, stream, split, workspace)  # noqa: F841 (alive until the launch)
    _check(vkv_chunk_attn(a, sh), "vkv_chunk_attn")
    return res


def chunk_attn_block_sparse(q, k, v, persist_idx, sel_idx, window_blk0, n_win_blk, scale=None,
                            err=None, stream=None, out=None, qblk_order=None, split=True, workspace=None,
                            kbar=None, topk=None, sel_out=None):
    """Persistent blocks + selected window blocks (device int32 index tensors).

    qblk_order (optional device int32 [B*H, nQblk]): query-block permutation that
    groups blocks with similar selections into the same units (from block_select).
    split / workspace: key-axis pieces, as in chunk_attn_segments.

    kbar (optional device fp32 [B*H, n_win_blk, d], from block_pool): the kernel
    selects the top-`topk` window blocks itself (sel_idx may then be None); the
    selection is written to sel_out (device int32 [B*H, nQblk, topk]) when given.
    """
    d = q.shape[3]
    a = _base_args(MODE_BLOCK_SPARSE, q, k.shape[1], d, scale, tensor_desc(k), tensor_desc(v), err)
    persist_idx = _contiguous(persist_idx, stream)
    a.persist_idx = persist_idx.data_ptr() if persist_idx.numel() else None
    a.n_persist = persist_idx.shape[-1]
    if kbar is not None:
        if topk is None:
            topk = sel_out.shape[-1] if sel_out is not None else sel_idx.shape[-1]
        if not (kbar.dtype == torch.float32 and kbar.is_contiguous()):
            raise ValueError("kbar must be a contiguous float32 tensor [B*H, n_win_blk, d]")
        a.kbar = kbar.data_ptr()
        if sel_out is not None:
            if not (sel_out.dtype == torch.int32 and sel_out.is_contiguous()):
                raise ValueError("sel_out must be a contiguous int32 tensor [B*H, nQblk, topk]")
            a.sel_out = sel_out.data_ptr()
        a.topk = int(topk)
    else:
        sel_idx = _contiguous(sel_idx, stream)
        a.sel_idx = sel_idx.data_ptr() if sel_idx.numel() else None
        a.topk = sel_idx.shape[-1]
    a.window_blk0 = int(window_blk0)
    a.n_win_blk = int(n_win_blk)
    if qblk_order is not None:
        qblk_order = _contiguous(qblk_order, stream)
        a.qblk_order = qblk_order.data_ptr()
    o, l = out if out is not None else _new_out(q, stream)
    a.o[0] = tensor_desc(o)
    a.lse[0] = l.data_ptr()
    sh = _stream(stream)
    ws = _attn_workspace(a, q, stream, split, workspace)  # noqa: F841 (alive until the launch)
    _check(vkv_chunk_attn(a, sh), "vkv_chunk_attn")
    return o, l


def chunk_attn_ragged(q, k_flat, v_flat, cu_seqlens, cu_seqlens_host=None, scale=None, err=None,
                      stream=None, out=None, split=True, workspace=None):
    """Ragged per-(batch, head) caches stored flattened with boundary offsets.

    With cu_seqlens_host the schedule knows each sequence's length and may cut
    long sequences' units along the key axis (split / workspace as in
    chunk_attn_segments)."""
    d = q.shape[3]
    a = _base_args(MODE_RAGGED, q, k_flat.shape[0], d, scale, flat_desc(k_flat), flat_desc(v_flat), err)
    a.cu_seqlens = cu_seqlens.data_ptr()
    host = None
    if cu_seqlens_host is not None:
        host = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
        a.cu_seqlens_host = host.ctypes.data_as(POINTER(c_int32))
    o, l = out if out is not None else _new_out(q, stream)
    a.o[0] = tensor_desc(o)
    a.lse[0] = l.data_ptr()
    sh = _stream(stream)
    ws = _attn_workspace(a, q, stream, split, workspace)  # noqa: F841 (alive until the launch)
    _check(vkv_chunk_attn(a, sh), "vkv_chunk_attn")
    return o, l


def block_select(q, k, window_blk0, n_win_blk, topk, workspace=None, scores=False, err=None, stream=None,
                 out_idx=None, order=False, out_order=None, kbar=None):
    """Top-K window blocks per 64-query block; returns (idx [B*H, nQblk, topk], scores or None).

    With order=True (or an out_order tensor) also returns the query-block order
    [B*H, nQblk] that groups blocks with similar selections: (idx, scores, order).
    kbar (optional device fp32 [B*H, n_win_blk, d], from block_pool) supplies the
    window blocks' representatives, so only the query blocks are pooled.
    """
    B, Lq, H, d = q.shape
    n_qblk = -(-Lq // 64)
    a = vkv_select_args()
    a.B, a.H, a.d, a.block = B, H, d, 64
    a.Lq, a.Lkv = Lq, k.shape[1]
    a.window_blk0, a.n_win_blk, a.topk = int(window_blk0), int(n_win_blk), int(topk)
    a.q = tensor_desc(q)
    a.k = tensor_desc(k)
    idx = out_idx if out_idx is not None else _new_outputs(q, stream, ((B * H, n_qblk, topk), torch.int32))[0]
    a.out_idx = idx.data_ptr()
    sc = None
    if scores:
        sc, = _new_outputs(q, stream, ((B * H, n_qblk, n_win_blk), torch.float32))
        a.out_scores = sc.data_ptr()
    need = vkv_block_select_workspace_size(B, H, Lq, n_win_blk, 64, d)
    if workspace is None:
        workspace, = _new_outputs(q, stream, (need, torch.uint8))
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.err_word = err.data_ptr() if err is not None else None
    if kbar is not None:
        kbar = _contiguous(kbar, stream)
        a.kbar = kbar.data_ptr()
    if order and out_order is None:
        out_order, = _new_outputs(q, stream, ((B * H, n_qblk), torch.int32))
    if out_order is not None:
        a.out_order = out_order.data_ptr()
    _check(vkv_block_select(a, _stream(stream)), "vkv_block_select")
    if out_order is not None:
        return idx, sc, out_order
    return idx, sc


def block_pool(x, blk0, n_blk, stream=None, out=None):
    """fp32 mean of each 64-row block [blk0, blk0 + n_blk) of x [B, L, H, d] -> [B*H, n_blk, d]."""
    B, L, H, d = x.shape
    o = out if out is not None else _new_outputs(x, stream, ((B * H, n_blk, d), torch.float32))[0]
    _check(vkv_block_pool(tensor_desc(x), B, L, H, d, int(blk0), int(n_blk), o.data_ptr(), _stream(stream)),
           "vkv_block_pool")
    return o


def lse_merge(o_a, lse_a, o_b, lse_b, stream=None, out=None):
    B, Lq, H, d = o_a.shape
    o, l = out if out is not None else _new_out(o_a, stream)
    _check(vkv_lse_merge(tensor_desc(o_a), lse_a.data_ptr(), tensor_desc(o_b), lse_b.data_ptr(),
                         tensor_desc(o), l.data_ptr(), B, H, Lq, d, _stream(stream)), "vkv_lse_merge")
    return o, l


def compact_cache(k, v, rules, frame_tokens, hist_frames, cur_frames, recent_frames, stream=None):
    """Head-aware compaction of a dense cache into a flattened ragged cache.

    k, v: device bf16 [B, L, H, d] with L = (hist_frames + cur_frames) * frame_tokens;
    rules: one (policy, param) per head (HEAD_FULL / HEAD_ANCHOR / HEAD_WAVE / HEAD_VEIL).
    Returns (k_flat [rows, d], v_flat, cu_seqlens on the device, cu_seqlens on the host).
    """
    B, L, H, d = k.shape
    a = vkv_compact_args()
    a.B, a.H, a.d = B, H, d
    a.frame_tokens, a.hist_frames, a.cur_frames, a.recent_frames = (int(frame_tokens), int(hist_frames),
                                                                     int(cur_frames), int(recent_frames))
    a.k_src = tensor_desc(k)
    a.v_src = tensor_desc(v)
    rr = (vkv_head_rule * H)(*[vkv_head_rule(int(p), int(x)) for p, x in rules])
    a.rules = ctypes.cast(rr, POINTER(vkv_head_rule))
    rows = vkv_compact_rows(a)
    if rows < 0:
        raise VkvError(-rows, "vkv_compact_rows")
    k_out, v_out, cu_dev = _new_outputs(k, stream, ((rows, d), k.dtype), ((rows, d), v.dtype), (B * H + 1, torch.int32))
    cu_host = np.zeros(B * H + 1, dtype=np.int32)
    a.k_out, a.v_out, a.out_rows = k_out.data_ptr(), v_out.data_ptr(), rows
    a.cu_seqlens = cu_dev.data_ptr()
    a.cu_seqlens_host = cu_host.ctypes.data_as(POINTER(c_int32))
    _check(vkv_compact_cache(a, _stream(stream)), "vkv_compact_cache")
    return k_out, v_out, cu_dev, cu_host


def persist_update(q, k, persist_idx, evict_blk0, n_evict, scores=False, err=None, stream=None, out_idx=None,
                   workspace=None):
    """Top-C of (persistent blocks + evicted window blocks) by <mean query, block mean>.

    q [B, Lq, H, d], k [B, Lkv, H, d] device bf16; persist_idx device int32 [B*H, C].
    Returns (new persistent ids [B*H, C] ascending, candidate scores [B*H, C + n_evict] or None).
    """
    B, Lq, H, d = q.shape
    persist_idx = _contiguous(persist_idx, stream)
    C = persist_idx.shape[-1]
    a = vkv_persist_args()
    a.B, a.H, a.d, a.block, a.Lq, a.Lkv = B, H, d, 64, Lq, k.shape[1]
    a.q, a.k = tensor_desc(q), tensor_desc(k)
    a.persist_idx, a.n_persist = persist_idx.data_ptr(), C
    a.evict_blk0, a.n_evict = int(evict_blk0), int(n_evict)
    idx = out_idx if out_idx is not None else _new_outputs(q, stream, ((B * H, C), torch.int32))[0]
    a.out_idx = idx.data_ptr()
    sc = None
    if scores:
        sc, = _new_outputs(q, stream, ((B * H, C + int(n_evict)), torch.float32))
        a.out_scores = sc.data_ptr()
    need = vkv_persist_update_workspace_size(B, H, Lq, C, int(n_evict), 64, d)
    if workspace is None:
        workspace, = _new_outputs(q, stream, (need, torch.uint8))
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    a.err_word = err.data_ptr() if err is not None else None
    _check(vkv_persist_update(a, _stream(stream)), "vkv_persist_update")
    return idx, sc


def latent_desc(x: torch.Tensor) -> vkv_tensor:
    """[B, L, w] bf16 cache rows with contiguous w -> vkv_tensor (sh unused)."""
    if x.dim() != 3 or x.dtype != torch.bfloat16 or x.stride(2) != 1:
        raise ValueError("expected a bf16 [B, L, w] tensor with contiguous w")
    return vkv_tensor(x.data_ptr(), x.stride(0), x.stride(1), 0)


def latent_attn(q, kv, d_c, scale=None, kr=None, err=None, stream=None, out=None, lse=True):
    """Latent attention over a head-shared cache (vkv_latent_attn).

    q [B, Lq, H, d_c + d_rope] absorbed queries; kv [B, Lkv, d_c (+ d_rope)] cached rows
    [c ; k_R]; kr optional [B, Lkv, d_rope] when the rotary keys are stored apart.
    Returns (latent output [B, Lq, H, d_c] bf16, LSE [B, H, Lq] fp32 or None).
    """
    B, Lq, H, dq = q.shape
    d_rope = dq - d_c
    a = vkv_latent_args()
    a.B, a.H, a.Lq, a.Lkv, a.d_c, a.d_rope = B, H, Lq, kv.shape[1], d_c, d_rope
    a.scale = float(scale if scale is not None else 1.0 / np.sqrt(dq))
    a.q = tensor_desc(q)
    if kv.shape[1] > 0:  # an empty cache is passed as a NULL pointer
        a.kv = latent_desc(kv)
        if kr is not None:
            a.kr = latent_desc(kr)
    if out is None:
        o, = _new_outputs(q, stream, ((B, Lq, H, d_c), torch.bfloat16))
        l = _new_outputs(q, stream, ((B, H, Lq), torch.float32))[0] if lse else None
    else:
        o, l = out
    a.o = tensor_desc(o)
    a.lse = l.data_ptr() if l is not None else None
    a.err_word = err.data_ptr() if err is not None else None
    _check(vkv_latent_attn(a, _stream(stream)), "vkv_latent_attn")
    return o, l


# ---------------------------------------------------------------------------
# paged cache: one query per row (request) over pages of tokens
# ---------------------------------------------------------------------------
# These calls run once per layer and token; their arguments are checked and marshalled by
# csrc/vkv_binding.cpp (a refused one is a ValueError), which calls the same entry points.
_page_attn_ws: dict = {}  # (device index, stream handle) -> uint8 buffer, cleared once (the call leaves it clear)
_NO_WORKSPACE = torch.empty(0, dtype=torch.uint8)
_page_select_ws: dict = {}  # (device index, stream handle) -> uint8 buffer, grown on demand


_binding = None


def _page_binding():
    global _binding
    if _binding is None:
        how = "build it with `python -m kv_cache_attention_chunk_b200.build`"
        if os.path.exists(build.BINDING) and not build.binding_fits():  # it would load, and read another torch's tensors
            raise RuntimeError(f"{build.BINDING} was built for another torch or Python: {how}")
        try:
            from . import _binding as b
        except ImportError as e:
            raise RuntimeError(f"the torch binding does not load ({e}): {how}") from e
        _binding = b
    return _binding


def _page_call(name, x, stream, *args):
    """One call on the device of `x`: with it current, on `stream`; raises VkvError on a non-OK status."""
    fn = getattr(_binding or _page_binding(), name)
    address = (_lib or lib()).page_entry[name]
    di = x.get_device()
    sh = _handle(di, stream)
    if di < 0 or di == torch._C._cuda_getDevice():
        status = fn(address, sh, *args)
    else:
        with torch.cuda.device(di):
            status = fn(address, sh, *args)
    if status:
        _check(status, "vkv_" + name)


def page_map(kv_len, new_len, block_table, ring, ring_pos, page_size, max_tokens, out=None, err=None, stream=None):
    """Pages and slots of one step's new tokens (vkv_page_map).

    kv_len, new_len: int32 [R] tokens held (-1: no request) and arriving (-1: the request
    ends).  block_table int32 [R, W] and ring int32 [n] (free page numbers, ring[t % n] for
    ring_pos[0] <= t < ring_pos[1]) are updated in place; ring_pos int64 [2].
    Returns (or fills `out`) dict(kv_len, ring [the new ring_pos], slot int64 [max_tokens],
    row, pos int32 [max_tokens], cu int32 [R + 1]; of a given `out` the last three may be
    missing); out["kv_len"] may be kv_len itself and out["ring"] ring_pos.  A step that does
    not fit changes nothing and sets err.
    """
    if out is None:
        R, i32, i64 = kv_len.shape[0], torch.int32, torch.int64
        out = dict(zip(("kv_len", "ring", "slot", "row", "pos", "cu"), _new_outputs(
            kv_len, stream, (R, i32), (2, i64), (max_tokens, i64), (max_tokens, i32), (max_tokens, i32), (R + 1, i32))))
    get = out.get
    _page_call("page_map", kv_len, stream, kv_len, new_len, block_table, ring, ring_pos, page_size, max_tokens,
               out["kv_len"], out["ring"], out["slot"], get("row"), get("pos"), get("cu"), err)
    return out


def page_append(k_new, v_new, slot, k_pages, v_pages, k_scale=None, v_scale=None, kbar=None, err=None, stream=None):
    """Write a step's keys and values [T, Hkv, d] into the pages at `slot` (vkv_page_append).

    k_pages, v_pages [n_pages, page, Hkv, d] of the type of k_new, or float8_e4m3fn (stored =
    x / scale, fp32 scales [Hkv]); kbar (optional fp32 [n_pages, Hkv, d]) receives the key
    mean of each page written to.  k_pages, v_pages and kbar do not overlap (two parts of one
    buffer, side by side, do not; one tensor may be both caches if it gets the same rows as both).
    """
    _page_call("page_append", k_pages, stream, k_new, v_new, slot, k_pages, v_pages, k_scale, v_scale, kbar, err)


def _new_workspace(di, need, clear):
    buf = torch.empty(need, dtype=torch.uint8, device=di)
    buf[:clear].zero_()
    return buf


def _page_workspace(kept, di, sh, need, clear):
    """A workspace of `need` bytes for a call on (device, stream): one kept by this module,
    or, while the stream is being captured, one of the graph's own (two captured graphs
    may be replayed at the same time, so they must not share it)."""
    if di < 0 or need <= 0:
        return _NO_WORKSPACE  # what makes the call refuse its arguments comes first
    if sh != torch._C._cuda_getCurrentRawStream(di) or di != torch._C._cuda_getDevice():
        # allocate, clear and ask about a capture on the stream that will use it
        with torch.cuda.stream(_stream_of(di, sh)):
            return _page_workspace(kept, di, sh, need, clear)
    if torch._C._cuda_isCurrentStreamCapturing():
        return _new_workspace(di, need, clear)
    buf = kept.get((di, sh))
    if buf is None or buf.numel() < need:
        buf = kept[di, sh] = _new_workspace(di, need, clear)
    return buf


def page_select(q, kbar, block_table, kv_len, page_size, topk, sink_pages=0, local_pages=0, err=None, stream=None,
                out=None, workspace=None):
    """The `topk` pages that each row and key head attends to (vkv_page_select).

    q [R, H, d]; kbar fp32 [n_pages, Hkv, d], the pages' key means (page_append keeps them).
    Returns int32 [R, Hkv, topk]: logical page numbers ascending, then -1 (`out` lies in none of the inputs).
    workspace: a uint8 tensor of vkv_page_select_workspace_size bytes (8 per row, key head and table
    column); without one, this module keeps the largest that a stream has needed, as long as it is loaded.
    """
    R, Hkv = q.shape[0], kbar.shape[1]
    sel = out if out is not None else _new_outputs(q, stream, ((R, Hkv, topk), torch.int32))[0]
    if workspace is None:
        di = q.get_device()
        workspace = _page_workspace(_page_select_ws, di, _handle(di, stream),
                                    vkv_page_select_workspace_size(R, Hkv, block_table.shape[1]), 0)
    _page_call("page_select", q, stream, q, kbar, block_table, kv_len, page_size, topk, sink_pages, local_pages, sel,
               workspace, err)
    return sel


def page_attn(q, k_pages, v_pages, block_table, kv_len, scale=None, sink=0, window=0, sel=None, k_scale=None,
              v_scale=None, err=None, stream=None, out=None, workspace=None):
    """Attention of one query per row over its paged cache (vkv_page_attn).

    q [R, H, d] bf16 or fp16; k_pages, v_pages [n_pages, page, Hkv, d] of q's type or
    float8_e4m3fn with fp32 scales [Hkv]; kv_len int32 [R] (-1: no request, its outputs are
    left as they were).  window > 0 keeps the first `sink` and the last `window` tokens; sel
    (from page_select) the selected pages.  Returns (o [R, H, d], lse fp32 [R, H]).
    workspace: a uint8 tensor of vkv_page_attn_workspace_size bytes whose first PAGE_ATTN_CLEAR_BYTES
    were zero before its first use.  Without one, calls that are being captured into a graph get one
    each and clear it in every replay (a kernel more per call): a captured step passes its own, the same
    to all its calls, and another one to each graph that may run beside it.
    o and lse (given as `out`) must not overlap one another or the inputs.
    """
    R, H, d = q.shape
    if out is None:
        out = _new_outputs(q, stream, ((R, H, d), q.dtype), ((R, H), torch.float32))
    o, lse = out
    if workspace is None:
        di = q.get_device()
        workspace = _page_workspace(_page_attn_ws, di, _handle(di, stream), _attn_need(H, k_pages.shape[2], d, di),
                                    PAGE_ATTN_CLEAR_BYTES)
    _page_call("page_attn", q, stream, q, k_pages, v_pages, block_table, kv_len, scale, sink, window, sel, k_scale, v_scale,
               o, lse, workspace, err)
    return o, lse


@functools.lru_cache(maxsize=256)
def _attn_need(H, Hkv, d, di):
    """vkv_page_attn_workspace_size on device `di` (it depends on the sizes and the device's SMs)."""
    with torch.cuda.device(di):
        return vkv_page_attn_workspace_size(H, Hkv, d)
