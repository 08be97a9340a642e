"""Python binding of the gbsort C ABI (include/gbsort.h).

Argument marshalling only: every function forwards torch tensors' device
pointers, sizes and the current CUDA stream to the entry point of the same
name in libgbsort.so; all sorting work runs in that library's kernels.  The
work buffer is a torch uint8 tensor that the caller may pass in and reuse
(it is allocated here, never inside the library).

The library is loaded on first use; if it is missing the call raises, so no
computation can silently happen elsewhere.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgbsort.so")

GBS_OK, GBS_ERR_INVALID_ARG, GBS_ERR_TEMP_TOO_SMALL, GBS_ERR_UNSUPPORTED, GBS_ERR_CUDA, GBS_ERR_TIMEOUT = range(6)
GBS_U32, GBS_I32, GBS_F32, GBS_U64, GBS_I64, GBS_F64 = range(6)
GBS_MAX_RADIX_KEYS = (1 << 32) - 1
GBS_MAX_SEGMENT_LEN = 16384

_DTYPE_KIND = {
    torch.uint32: GBS_U32,
    torch.int32: GBS_I32,
    torch.float32: GBS_F32,
    torch.uint64: GBS_U64,
    torch.int64: GBS_I64,
    torch.float64: GBS_F64,
}
GBS_ROW_F32, GBS_ROW_F16, GBS_ROW_BF16 = range(3)
GBS_MAX_EXPERTS, GBS_MAX_TOP_K, GBS_MAX_ROW_LEN = 1024, 256, 1 << 23
GBS_SCORE_SOFTMAX, GBS_SCORE_SIGMOID = range(2)
GBS_MAX_GROUPS, GBS_MAX_BEAMS, GBS_MAX_BEAM_OUT = 32, 32, 64
_ROW_TYPE = {torch.float32: GBS_ROW_F32, torch.float16: GBS_ROW_F16, torch.bfloat16: GBS_ROW_BF16}
_ID_TYPE = {torch.int32: GBS_I32, torch.int64: GBS_I64}
_KIND_BYTES = {GBS_U32: 4, GBS_I32: 4, GBS_F32: 4, GBS_U64: 8, GBS_I64: 8, GBS_F64: 8}

# every symbol the headers declare
EXPORTS = ("gbs_sort_keys", "gbs_sort_pairs", "gbs_segmented_sort", "gbs_digit_histograms", "gbs_get_status",
           "gbs_status_string", "gbs_version", "gbs_debug_set_lookback_fault", "gbs_debug_last_launch_count",
           "gbs_debug_radix_tile_keys", "gbs_debug_set_timing_events", "gbs_sort_keys_noalloc",
           "gbs_sort_keys_host", "gbs_segmented_sort_offsets", "gbs_sort_pairs64", "gbs_get_status_noalloc",
           "gbs_sort_keys_msd_bitonic", "gbs_debug_set_radix_bits", "gbs_sort_keys_host_batch",
           "gbs_expert_num_rows", "gbs_expert_sort", "gbs_expert_dispatch", "gbs_expert_gather", "gbs_expert_combine",
           "gbs_expert_combine_grad", "gbs_embedding_lookup", "gbs_embedding_grad", "gbs_debug_set_ring_fault",
           "gbs_expert_route", "gbs_expert_route_grad", "gbs_beam_select", "gbs_beam_reorder")
GBS_NOALLOC_MAX_KEYS = 1 << 20


class GbsError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)}")
        self.status = status


# absent where torch is built without CUDA: no tensor gets as far as their calls there
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_lib = None
_fast = None  # the row operators' compiled calls (csrc/rows_py.c), once the library is loaded; None: not built


def load(path: str | None = None):
    """Loads libgbsort.so (built by sorting_lsd_radix_gb300.build) and declares the prototypes."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"gbsort CUDA library not built: {p} is missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    vp, sz, i, u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32
    szp = ctypes.POINTER(ctypes.c_size_t)
    lib.gbs_sort_keys.argtypes = [vp, szp, i, vp, vp, sz, i, i, i, vp]
    lib.gbs_sort_keys.restype = i
    lib.gbs_sort_keys_host.argtypes = [vp, szp, i, vp, vp, sz, i, i, i, vp]
    lib.gbs_sort_keys_host_batch.restype = i
    lib.gbs_sort_keys_host_batch.argtypes = [vp, szp, i, ctypes.POINTER(vp), ctypes.POINTER(vp), szp, sz, i, i, i,
                                             vp]
    lib.gbs_sort_keys_host.restype = i
    lib.gbs_sort_pairs.argtypes = [vp, szp, i, vp, vp, vp, vp, sz, i, i, i, vp]
    lib.gbs_sort_pairs64.argtypes = [vp, szp, i, vp, vp, vp, vp, sz, i, i, i, vp]
    lib.gbs_sort_pairs64.restype = i
    lib.gbs_sort_pairs.restype = i
    lib.gbs_segmented_sort_offsets.argtypes = [vp, szp, i, vp, vp, sz, vp, i, vp]
    lib.gbs_segmented_sort_offsets.restype = i
    lib.gbs_segmented_sort.argtypes = [vp, szp, i, vp, vp, sz, sz, i, vp]
    lib.gbs_segmented_sort.restype = i
    lib.gbs_digit_histograms.argtypes = [vp, szp, i, vp, sz, i, i, i, vp, vp]
    lib.gbs_digit_histograms.restype = i
    lib.gbs_sort_keys_noalloc.argtypes = [i, vp, vp, sz, i, i, i, vp]
    lib.gbs_sort_keys_noalloc.restype = i
    lib.gbs_sort_keys_msd_bitonic.argtypes = [vp, szp, i, vp, vp, sz, i, vp]
    lib.gbs_sort_keys_msd_bitonic.restype = i
    lib.gbs_debug_set_radix_bits.argtypes = [i]
    lib.gbs_debug_set_radix_bits.restype = None
    lib.gbs_get_status_noalloc.argtypes = [vp]
    lib.gbs_get_status_noalloc.restype = i
    lib.gbs_get_status.argtypes = [vp, sz, vp]
    lib.gbs_get_status.restype = i
    lib.gbs_status_string.argtypes = [i]
    lib.gbs_status_string.restype = ctypes.c_char_p
    lib.gbs_version.argtypes = []
    lib.gbs_version.restype = ctypes.c_char_p
    lib.gbs_debug_set_lookback_fault.argtypes = [i, u32, u32]
    lib.gbs_debug_set_lookback_fault.restype = None
    lib.gbs_debug_set_ring_fault.argtypes = [i, u32]
    lib.gbs_debug_set_ring_fault.restype = None
    lib.gbs_debug_last_launch_count.argtypes = []
    lib.gbs_debug_last_launch_count.restype = i
    lib.gbs_debug_radix_tile_keys.argtypes = [i, i]
    lib.gbs_debug_radix_tile_keys.restype = sz
    lib.gbs_debug_set_timing_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), i]
    lib.gbs_debug_set_timing_events.restype = None
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.gbs_expert_num_rows.argtypes = [sz, sz, sz]
    lib.gbs_expert_num_rows.restype = sz
    order = [i, vp, sz, sz, sz, i64, sz, sz]  # ids, tokens, top_k, experts, first, row_align, num_rows
    lib.gbs_expert_sort.argtypes = [vp, szp] + order + [vp, vp, vp, vp, vp]
    lib.gbs_expert_sort.restype = i
    lib.gbs_expert_dispatch.argtypes = [vp, szp, i, vp, sz, sz] + order + [vp, sz, vp, vp, vp, vp, vp]
    lib.gbs_expert_dispatch.restype = i
    lib.gbs_expert_gather.argtypes = [i, vp, sz, sz, sz, sz, vp, vp, sz, vp, sz, vp]
    lib.gbs_expert_gather.restype = i
    lib.gbs_expert_combine.argtypes = [i, vp, sz, sz, vp, i, vp, sz, sz, sz, vp, sz, vp]
    lib.gbs_expert_combine.restype = i
    lib.gbs_expert_combine_grad.argtypes = [i, vp, sz, vp, sz, sz, vp, vp, i, vp, sz, sz, sz, vp, sz, vp, vp]
    lib.gbs_expert_combine_grad.restype = i
    lib.gbs_embedding_lookup.argtypes = [i, vp, sz, sz, i, vp, sz, i64, f32, sz, vp, sz, vp]
    lib.gbs_embedding_lookup.restype = i
    lib.gbs_embedding_grad.argtypes = [vp, szp, i, vp, sz, i, vp, sz, i64, i64, f32, sz, sz, i, vp, sz, i, vp]
    lib.gbs_embedding_grad.restype = i
    lib.gbs_expert_route.argtypes = [i, vp, sz, sz, sz, sz, i, vp, sz, sz, sz, i, f32, i, vp, i, vp, vp]
    lib.gbs_expert_route.restype = i
    lib.gbs_expert_route_grad.argtypes = [i, i, vp, vp, sz, sz, sz, sz, i, vp, i, i, f32, vp, sz, vp]
    lib.gbs_expert_route_grad.restype = i
    lib.gbs_beam_select.argtypes = [vp, szp, i, vp, sz, sz, sz, sz, vp, vp, ctypes.c_int32, sz, vp, vp, vp, vp]
    lib.gbs_beam_select.restype = i
    lib.gbs_beam_reorder.argtypes = [vp, szp, vp, szp, sz, sz, sz, sz, sz, sz, vp, vp]
    lib.gbs_beam_reorder.restype = i
    if path is None:
        _lib = lib
        _load_fast(lib)
    return lib


def _load_fast(lib):
    global _fast
    try:
        from . import _rows
    except ImportError:
        return
    _rows.setup((torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int64), _raw_stream, _current_device,
                tuple(ctypes.cast(f, ctypes.c_void_p).value for f in (
                    lib.gbs_expert_sort, lib.gbs_expert_dispatch, lib.gbs_expert_gather, lib.gbs_expert_combine,
                    lib.gbs_expert_combine_grad, lib.gbs_embedding_lookup, lib.gbs_embedding_grad)))
    _rows.setup_select(torch.bool, torch.uint8, tuple(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.gbs_expert_route, lib.gbs_expert_route_grad, lib.gbs_beam_select, lib.gbs_beam_reorder)))
    _fast = _rows


def status_string(status: int) -> str:
    try:
        return load().gbs_status_string(status).decode()
    except RuntimeError:
        return f"status {status}"


def gbs_version() -> str:
    return load().gbs_version().decode()


def _kind(t: torch.Tensor, key_type: int | None) -> int:
    if key_type is not None:
        if _KIND_BYTES[key_type] != t.element_size():
            raise ValueError("key_type does not match the tensor's element size")
        return key_type
    try:
        return _DTYPE_KIND[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported key dtype {t.dtype}; pass key_type for a reinterpreting view") from None


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr() if t is not None and t.numel() else 0)


def _check_tensor(t: torch.Tensor, n: int, what: str):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() != n:
        raise ValueError(f"{what} must hold {n} elements")


def _run(fn, args_after_temp, temp: torch.Tensor | None, what: str) -> torch.Tensor:
    """Work-buffer protocol: with a work buffer, run at once; without one, or if it is too small
    (GBS_ERR_TEMP_TOO_SMALL, nothing launched), query the size, allocate with torch and run."""
    if temp is not None and temp.numel():  # an empty buffer's address would be a query
        # a strided or expanded tensor has fewer bytes behind it than elements
        dev = temp.get_device()
        if dev < 0 or dev != _current_device() or not temp.is_contiguous():
            raise ValueError("temp must be a contiguous tensor on the current CUDA device")
        have = ctypes.c_size_t(temp.numel())
        st = fn(_ptr(temp), ctypes.byref(have), *args_after_temp)
        if st == GBS_OK:
            return temp
        if st != GBS_ERR_TEMP_TOO_SMALL:
            raise GbsError(st, what)
    need = ctypes.c_size_t(0)
    st = fn(None, ctypes.byref(need), *args_after_temp)
    if st != GBS_OK:
        raise GbsError(st, what)
    temp = torch.empty(max(need.value, 256), dtype=torch.uint8, device="cuda")
    have = ctypes.c_size_t(temp.numel())
    st = fn(_ptr(temp), ctypes.byref(have), *args_after_temp)
    if st != GBS_OK:
        raise GbsError(st, what)
    return temp


def temp_bytes(fn_name: str, *args) -> int:
    """Work-buffer size a call with these C-level arguments needs (no launch)."""
    need = ctypes.c_size_t(0)
    st = getattr(load(), fn_name)(None, ctypes.byref(need), *args)
    if st != GBS_OK:
        raise GbsError(st, fn_name)
    return need.value


def gbs_sort_keys(keys_in: torch.Tensor, keys_out: torch.Tensor | None = None, begin_bit: int = 0,
                  end_bit: int | None = None, descending: bool = False, temp: torch.Tensor | None = None,
                  key_type: int | None = None, stream=None, return_temp: bool = False):
    """Stable LSD radix sort of a CUDA tensor of keys by bits [begin_bit, end_bit) of their code.

    keys_out may be keys_in (in place); None allocates a new tensor."""
    kind = _kind(keys_in, key_type)
    n = keys_in.numel()
    _check_tensor(keys_in, n, "keys_in")
    if keys_out is None:
        keys_out = torch.empty_like(keys_in)
    _check_tensor(keys_out, n, "keys_out")
    if end_bit is None:
        end_bit = 8 * _KIND_BYTES[kind]
    args = (kind, _ptr(keys_in), _ptr(keys_out), n, begin_bit, end_bit, int(bool(descending)), _stream(stream))
    temp = _run(load().gbs_sort_keys, args, temp, "gbs_sort_keys")
    return (keys_out, temp) if return_temp else keys_out


def gbs_sort_keys_msd_bitonic(keys_in: torch.Tensor, keys_out: torch.Tensor | None = None,
                              descending: bool = False, temp: torch.Tensor | None = None,
                              key_type: int | None = None, stream=None, return_temp: bool = False):
    """Full-width key sort by MSD radix passes over the top 16 bits, then a bitonic sort of every
    bucket (the pages' hybrid; synchronises the stream once)."""
    kind = _kind(keys_in, key_type)
    n = keys_in.numel()
    _check_tensor(keys_in, n, "keys_in")
    if keys_out is None:
        keys_out = torch.empty_like(keys_in)
    _check_tensor(keys_out, n, "keys_out")
    args = (kind, _ptr(keys_in), _ptr(keys_out), n, int(bool(descending)), _stream(stream))
    temp = _run(load().gbs_sort_keys_msd_bitonic, args, temp, "gbs_sort_keys_msd_bitonic")
    return (keys_out, temp) if return_temp else keys_out


def gbs_sort_keys_host(keys_in: torch.Tensor, keys_out: torch.Tensor | None = None, begin_bit: int = 0,
                       end_bit: int | None = None, descending: bool = False, temp: torch.Tensor | None = None,
                       key_type: int | None = None, stream=None, return_temp: bool = False):
    """gbs_sort_keys on a CPU tensor: copy to the device, sort, copy back into keys_out (a CPU tensor;
    may be keys_in; None allocates one, page-locked when keys_in is).  Asynchronous on the stream:
    synchronise it before reading keys_out.  temp is the device work buffer (torch uint8)."""
    kind = _kind(keys_in, key_type)
    n = keys_in.numel()
    if keys_in.is_cuda or not keys_in.is_contiguous():
        raise ValueError("keys_in must be a contiguous CPU tensor")
    if keys_out is None:
        keys_out = torch.empty_like(keys_in, pin_memory=keys_in.is_pinned())
    if keys_out.is_cuda or not keys_out.is_contiguous() or keys_out.numel() != n:
        raise ValueError(f"keys_out must be a contiguous CPU tensor of {n} elements")
    if end_bit is None:
        end_bit = 8 * _KIND_BYTES[kind]
    args = (kind, _ptr(keys_in), _ptr(keys_out), n, begin_bit, end_bit, int(bool(descending)), _stream(stream))
    temp = _run(load().gbs_sort_keys_host, args, temp, "gbs_sort_keys_host")
    return (keys_out, temp) if return_temp else keys_out


def gbs_sort_keys_host_batch(keys_in: list, keys_out: list | None = None, begin_bit: int = 0,
                             end_bit: int | None = None, descending: bool = False, temp: torch.Tensor | None = None,
                             key_type: int | None = None, stream=None, return_temp: bool = False):
    """gbs_sort_keys_host on a list of CPU tensors of one dtype, with the copies of neighbouring arrays
    overlapped (see the C entry point).  keys_out: a list of CPU tensors of the same sizes (an entry may be
    the matching keys_in), or None to allocate them (page-locked when the inputs are).  Asynchronous on the
    stream: synchronise it before reading the outputs."""
    kind = _kind(keys_in[0], key_type) if keys_in else (GBS_U32 if key_type is None else key_type)
    for t in keys_in:
        if t.is_cuda or not t.is_contiguous() or t.dtype != keys_in[0].dtype:
            raise ValueError("keys_in must be contiguous CPU tensors of one dtype")
    if keys_out is None:
        keys_out = [torch.empty_like(t, pin_memory=t.is_pinned()) for t in keys_in]
    if len(keys_out) != len(keys_in):
        raise ValueError("keys_out must hold one tensor per input")
    for t, o in zip(keys_in, keys_out):
        if o.is_cuda or not o.is_contiguous() or o.numel() != t.numel() or o.dtype != t.dtype:
            raise ValueError("each keys_out entry must be a contiguous CPU tensor like its input")
    if end_bit is None:
        end_bit = 8 * _KIND_BYTES[kind]
    count = len(keys_in)
    ins = (ctypes.c_void_p * max(count, 1))(*[_ptr(t) for t in keys_in])
    outs = (ctypes.c_void_p * max(count, 1))(*[_ptr(t) for t in keys_out])
    ns = (ctypes.c_size_t * max(count, 1))(*[t.numel() for t in keys_in])
    args = (kind, ins, outs, ns, count, begin_bit, end_bit, int(bool(descending)), _stream(stream))
    temp = _run(load().gbs_sort_keys_host_batch, args, temp, "gbs_sort_keys_host_batch")
    return (keys_out, temp) if return_temp else keys_out


def gbs_sort_pairs(keys_in: torch.Tensor, vals_in: torch.Tensor, keys_out: torch.Tensor | None = None,
                   vals_out: torch.Tensor | None = None, begin_bit: int = 0, end_bit: int | None = None,
                   descending: bool = False, temp: torch.Tensor | None = None, key_type: int | None = None,
                   stream=None, return_temp: bool = False):
    """Stable LSD radix sort of (key, value) pairs with 4- or 8-byte values; returns (keys_out, vals_out)."""
    kind = _kind(keys_in, key_type)
    n = keys_in.numel()
    _check_tensor(keys_in, n, "keys_in")
    _check_tensor(vals_in, n, "vals_in")
    if vals_in.element_size() not in (4, 8):
        raise ValueError("values must be 4- or 8-byte elements")
    if keys_out is None:
        keys_out = torch.empty_like(keys_in)
    if vals_out is None:
        vals_out = torch.empty_like(vals_in)
    _check_tensor(keys_out, n, "keys_out")
    _check_tensor(vals_out, n, "vals_out")
    if end_bit is None:
        end_bit = 8 * _KIND_BYTES[kind]
    args = (kind, _ptr(keys_in), _ptr(keys_out), _ptr(vals_in), _ptr(vals_out), n, begin_bit, end_bit,
            int(bool(descending)), _stream(stream))
    fn = load().gbs_sort_pairs64 if vals_in.element_size() == 8 else load().gbs_sort_pairs
    temp = _run(fn, args, temp, "gbs_sort_pairs")
    return (keys_out, vals_out, temp) if return_temp else (keys_out, vals_out)


def gbs_segmented_sort(keys_in: torch.Tensor, num_segments: int, segment_len: int,
                       keys_out: torch.Tensor | None = None, descending: bool = False,
                       temp: torch.Tensor | None = None, key_type: int | None = None, stream=None,
                       return_temp: bool = False):
    """Sort each of num_segments consecutive segments of segment_len keys (bitonic network up to
    GBS_MAX_SEGMENT_LEN keys per segment, the radix sort segment by segment above)."""
    kind = _kind(keys_in, key_type)
    n = num_segments * segment_len
    _check_tensor(keys_in, n, "keys_in")
    if keys_out is None:
        keys_out = torch.empty_like(keys_in)
    _check_tensor(keys_out, n, "keys_out")
    args = (kind, _ptr(keys_in), _ptr(keys_out), num_segments, segment_len, int(bool(descending)), _stream(stream))
    temp = _run(load().gbs_segmented_sort, args, temp, "gbs_segmented_sort")
    return (keys_out, temp) if return_temp else keys_out


def gbs_segmented_sort_offsets(keys_in: torch.Tensor, offsets, keys_out: torch.Tensor | None = None,
                               descending: bool = False, temp: torch.Tensor | None = None,
                               key_type: int | None = None, stream=None, return_temp: bool = False):
    """Sorts each segment [offsets[s], offsets[s+1]) of keys_in independently (any lengths).

    offsets: host sequence of num_segments + 1 non-decreasing integers (list, numpy or CPU tensor).
    keys_out may be keys_in; None allocates a copy of keys_in, so keys outside the segments keep
    their values."""
    kind = _kind(keys_in, key_type)
    n = keys_in.numel()
    _check_tensor(keys_in, n, "keys_in")
    if isinstance(offsets, torch.Tensor):
        offsets = offsets.cpu().numpy()
    offs = np.ascontiguousarray(np.asarray(offsets, dtype=np.int64)).astype(np.uint64)
    if offs.ndim != 1 or offs.size < 1:
        raise ValueError("offsets must hold num_segments + 1 entries")
    if offs.size > 1 and int(offs[-1]) > n:
        raise ValueError("offsets reach past the end of keys_in")
    if keys_out is None:
        keys_out = keys_in.clone()
    _check_tensor(keys_out, n, "keys_out")
    args = (kind, _ptr(keys_in), _ptr(keys_out), offs.size - 1, ctypes.c_void_p(offs.ctypes.data),
            int(bool(descending)), _stream(stream))
    temp = _run(load().gbs_segmented_sort_offsets, args, temp, "gbs_segmented_sort_offsets")
    return (keys_out, temp) if return_temp else keys_out


def gbs_digit_histograms(keys: torch.Tensor, begin_bit: int = 0, end_bit: int | None = None,
                         descending: bool = False, temp: torch.Tensor | None = None,
                         key_type: int | None = None, stream=None) -> torch.Tensor:
    """[passes, 256] uint32 digit counts computed by the upfront-histogram kernel."""
    kind = _kind(keys, key_type)
    n = keys.numel()
    _check_tensor(keys, n, "keys")
    if end_bit is None:
        end_bit = 8 * _KIND_BYTES[kind]
    passes = (end_bit - begin_bit + 7) // 8
    hist = torch.zeros((max(passes, 1), 256), dtype=torch.int32, device="cuda")
    args = (kind, _ptr(keys), n, begin_bit, end_bit, int(bool(descending)), _ptr(hist), _stream(stream))
    _run(load().gbs_digit_histograms, args, temp, "gbs_digit_histograms")
    return hist[:passes]


# ---------------------------------------------------------------------------
# Row operators.  `stream` (a torch stream or a cudaStream_t handle) makes the
# call, and what it allocates, belong to that stream; the caller keeps tensors
# of other streams alive until it is done.  Matrices are 2-D with unit stride
# along a row and any stride between rows (0, as expand makes it, for inputs).
#
# A small call costs more on the host than on the GPU, so a call with plain
# arguments and all of its outputs goes through the compiled calls of _rows
# (_fast); whatever they do not take, and every refusal, is handled here.
# ---------------------------------------------------------------------------


def _finish(st: int, what: str) -> bool:
    """Whether a compiled call is done; an error it met is raised."""
    if st > 0:
        raise GbsError(st, what)
    return st == GBS_OK


def _on_stream(stream, fn, *args):
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return fn(*args)


def _refuse_devices(*tensors):
    if any(t is not None and not t.is_cuda for t in tensors):
        raise ValueError("the tensors must be CUDA tensors")
    raise ValueError("the tensors must be on one device, the current one")


def _matrix(t: torch.Tensor, what: str, rows: int, cols: int, dtype) -> int:
    """Row stride of a 2-D tensor of `rows` rows of `cols` values of `dtype`."""
    if t.dim() != 2 or t.size(0) != rows or t.size(1) != cols:
        raise ValueError(f"{what} must be [{rows}, {cols}], got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have unit stride along its rows")
    return t.stride(0)


def _vector(t: torch.Tensor, what: str, count: int, dtype):
    """A contiguous tensor of `count` values of `dtype`."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and hold {count} elements")


def _row_type(t: torch.Tensor, what: str) -> int:
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions, got {list(t.shape)}")
    try:
        return _ROW_TYPE[t.dtype]
    except KeyError:
        raise TypeError(f"{what} must be float32, float16 or bfloat16, got {t.dtype}") from None


def _id_type(t: torch.Tensor, what: str) -> int:
    if t.dtype not in _ID_TYPE:
        raise TypeError(f"{what} must be int32 or int64, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return _ID_TYPE[t.dtype]


def _int64(value: int, what: str) -> int:
    """ctypes would take the low 64 bits of any other."""
    if not -(1 << 63) <= value < 1 << 63:
        raise ValueError(f"{what} must be a signed integer of 64 bits, got {value}")
    return value


def _int32(value: int, what: str) -> int:
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError(f"{what} must be a signed integer of 32 bits, got {value}")
    return value


def _weight_type(weights: torch.Tensor, dtype, count: int) -> int:
    if weights.dtype not in (torch.float32, dtype):
        raise TypeError(f"weights must be float32 or {dtype}, got {weights.dtype}")
    _vector(weights, "weights", count, weights.dtype)
    return _ROW_TYPE[weights.dtype]


def _slots_out(t, what, tokens, top_k):
    """The dtype of a contiguous [tokens, top_k] tensor."""
    if tuple(t.shape) != (tokens, top_k) or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and [{tokens}, {top_k}], got {list(t.shape)}")
    return t.dtype


def gbs_expert_route(logits: torch.Tensor, top_k: int, score_type: int = GBS_SCORE_SOFTMAX,
                     bias: torch.Tensor | None = None, num_groups: int = 1, top_groups: int = 1, group_top: int = 1,
                     renormalise: bool = False, scale: float = 1.0, ids_out: torch.Tensor | None = None,
                     weights_out: torch.Tensor | None = None, stream=None):
    """A router's choice: (expert_ids, weights) [tokens, top_k] from logits [tokens, experts].  The best top_k by
    score + bias (score: softmax or sigmoid of the logits), best first, ties to the lowest expert; with num_groups
    only the experts of the top_groups groups whose group_top best choice values add up to the most.  weights are
    scale * score, with renormalise divided by the token's sum of them.  A logit or bias of -inf: never chosen; too
    few left: id -1, weight 0.  ids are int32 and weights float32 unless ids_out (int64) or weights_out (the logits'
    type) say otherwise."""
    if _fast is not None and stream is None and ids_out is not None and weights_out is not None:
        if _finish(_fast.route(logits, top_k, score_type, bias, num_groups, top_groups, group_top, renormalise, scale, ids_out,
                               weights_out), "gbs_expert_route"):
            return ids_out, weights_out
    if stream is not None:
        return _on_stream(stream, gbs_expert_route, logits, top_k, score_type, bias, num_groups, top_groups, group_top,
                          renormalise, scale, ids_out, weights_out)
    row_type, dtype, dev = _row_type(logits, "logits"), logits.dtype, logits.get_device()
    tokens, experts = logits.shape
    stride = _matrix(logits, "logits", tokens, experts, dtype)
    for value, what in ((top_k, "top_k"), (num_groups, "num_groups"), (top_groups, "top_groups")):
        if _int64(value, what) < 1:
            raise ValueError(f"{what} must be positive")
    _int64(group_top, "group_top")
    _int32(score_type, "score_type")
    b = None
    if bias is not None:
        _vector(bias, "bias", experts, torch.float32)
        b = bias.data_ptr()
    if ids_out is None:
        ids_out = torch.empty((tokens, top_k), dtype=torch.int32, device=logits.device)
    if weights_out is None:
        weights_out = torch.empty((tokens, top_k), dtype=torch.float32, device=logits.device)
    id_type = _ID_TYPE.get(_slots_out(ids_out, "ids_out", tokens, top_k))
    if id_type is None:
        raise TypeError(f"ids_out must be int32 or int64, got {ids_out.dtype}")
    if _slots_out(weights_out, "weights_out", tokens, top_k) not in (torch.float32, dtype):
        raise TypeError(f"weights_out must be float32 or {dtype}, got {weights_out.dtype}")
    if dev < 0 or dev != _current_device() or not (ids_out.get_device() == weights_out.get_device() == dev) or \
            (bias is not None and bias.get_device() != dev):
        _refuse_devices(logits, bias, ids_out, weights_out)
    st = load().gbs_expert_route(row_type, logits.data_ptr(), stride, tokens, experts, top_k, score_type, b, num_groups,
                                 top_groups, group_top, 1 if renormalise else 0, scale, id_type, ids_out.data_ptr(),
                                 _ROW_TYPE[weights_out.dtype], weights_out.data_ptr(), _raw_stream(dev))
    if st != GBS_OK:
        raise GbsError(st, "gbs_expert_route")
    return ids_out, weights_out


def gbs_expert_route_grad(d_weights: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor,
                          score_type: int = GBS_SCORE_SOFTMAX, renormalise: bool = False, scale: float = 1.0,
                          d_logits_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of gbs_expert_route's weights with respect to logits, from d_weights [tokens, top_k] (float32 or
    the logits' type) and the expert_ids that were chosen; ids outside the experts add nothing."""
    if _fast is not None and stream is None and d_logits_out is not None:
        if _finish(_fast.route_grad(d_weights, logits, expert_ids, score_type, renormalise, scale, d_logits_out),
                   "gbs_expert_route_grad"):
            return d_logits_out
    if stream is not None:
        return _on_stream(stream, gbs_expert_route_grad, d_weights, logits, expert_ids, score_type, renormalise, scale,
                          d_logits_out)
    row_type, dtype, dev = _row_type(logits, "logits"), logits.dtype, logits.get_device()
    tokens, experts = logits.shape
    stride = _matrix(logits, "logits", tokens, experts, dtype)
    if expert_ids.dim() != 2 or expert_ids.size(0) != tokens or expert_ids.size(1) < 1:
        raise ValueError(f"expert_ids must be [{tokens}, top_k], got {list(expert_ids.shape)}")
    _int32(score_type, "score_type")
    id_type, top_k = _id_type(expert_ids, "expert_ids"), expert_ids.size(1)
    if _slots_out(d_weights, "d_weights", tokens, top_k) not in (torch.float32, dtype):
        raise TypeError(f"d_weights must be float32 or {dtype}, got {d_weights.dtype}")
    if d_logits_out is None:
        d_logits_out = torch.empty((tokens, experts), dtype=dtype, device=logits.device)
    d_stride = _matrix(d_logits_out, "d_logits_out", tokens, experts, dtype)
    if dev < 0 or dev != _current_device() or not (
            d_weights.get_device() == expert_ids.get_device() == d_logits_out.get_device() == dev):
        _refuse_devices(d_weights, logits, expert_ids, d_logits_out)
    st = load().gbs_expert_route_grad(row_type, _ROW_TYPE[d_weights.dtype], d_weights.data_ptr(), logits.data_ptr(), stride,
                                      tokens, experts, top_k, id_type, expert_ids.data_ptr(), score_type,
                                      1 if renormalise else 0, scale, d_logits_out.data_ptr(), d_stride, _raw_stream(dev))
    if st != GBS_OK:
        raise GbsError(st, "gbs_expert_route_grad")
    return d_logits_out


def gbs_expert_num_rows(num_slots: int, num_experts: int, row_align: int = 1) -> int:
    """Rows that hold num_slots slots whatever their experts, each expert's rows starting at a multiple of
    row_align."""
    return load().gbs_expert_num_rows(num_slots, num_experts, row_align)


def _order(expert_ids, num_experts, row_align, num_rows, plan_out):
    """(tokens, top_k, num_rows, plan, device) of a call that makes an order."""
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [tokens, top_k]")
    if _int64(num_experts, "num_experts") < 1 or _int64(row_align, "row_align") < 1:
        raise ValueError("num_experts and row_align must be positive")
    tokens, top_k = expert_ids.shape
    dev = expert_ids.get_device()
    if plan_out is None:
        if num_rows is None:
            num_rows = tokens * top_k if row_align == 1 else \
                load().gbs_expert_num_rows(tokens * top_k, num_experts, row_align)
        plan_out = tuple(torch.empty(s, dtype=torch.int32, device=expert_ids.device)
                         for s in ((num_rows,), (tokens, top_k), (num_experts + 1,), (num_experts,)))
        return tokens, top_k, num_rows, plan_out, dev
    i32 = torch.int32
    slot_of_row, row_of_slot, offsets, counts = plan_out
    if num_rows is None:
        num_rows = slot_of_row.numel()
    for t, what, count in ((slot_of_row, "slot_of_row", num_rows), (row_of_slot, "row_of_slot", tokens * top_k),
                           (offsets, "offsets", num_experts + 1), (counts, "counts", num_experts)):
        if t.dtype is not i32 or t.numel() != count or not t.is_contiguous():
            _vector(t, what, count, i32)
        if t.get_device() != dev:
            _refuse_devices(expert_ids, *plan_out)
    return tokens, top_k, num_rows, plan_out, dev


def gbs_expert_sort(expert_ids: torch.Tensor, num_experts: int, first_expert: int = 0, row_align: int = 1,
                    num_rows: int | None = None, plan_out: tuple | None = None, temp: torch.Tensor | None = None,
                    stream=None, return_temp: bool = False):
    """The stable order of the slots (t, k) of expert_ids [tokens, top_k] by expert; returns
    (slot_of_row, row_of_slot, offsets, counts), int32.  Ids outside [first_expert, first_expert + num_experts)
    have no row (row_of_slot -1); rows without a slot have slot_of_row -1."""
    if _fast is not None and stream is None and plan_out is not None and temp is not None and num_rows is None:
        if _finish(_fast.sort(expert_ids, num_experts, first_expert, row_align, plan_out, temp), "gbs_expert_sort"):
            return (plan_out, temp) if return_temp else plan_out
    if stream is not None:
        return _on_stream(stream, gbs_expert_sort, expert_ids, num_experts, first_expert, row_align, num_rows, plan_out,
                          temp, None, return_temp)
    id_type = _id_type(expert_ids, "expert_ids")
    tokens, top_k, num_rows, plan, dev = _order(expert_ids, num_experts, row_align, num_rows, plan_out)
    if dev < 0 or dev != _current_device():
        _refuse_devices(expert_ids)
    a, b, c, d = plan
    temp = _run(load().gbs_expert_sort,
                (id_type, expert_ids.data_ptr(), tokens, top_k, num_experts, _int64(first_expert, "first_expert"), row_align,
                 num_rows, a.data_ptr(), b.data_ptr(), c.data_ptr(), d.data_ptr(), _raw_stream(dev)), temp, "gbs_expert_sort")
    return (plan, temp) if return_temp else plan


def gbs_expert_dispatch(x: torch.Tensor, expert_ids: torch.Tensor, num_experts: int, first_expert: int = 0,
                        row_align: int = 1, num_rows: int | None = None, rows_out: torch.Tensor | None = None,
                        plan_out: tuple | None = None, temp: torch.Tensor | None = None, stream=None,
                        return_temp: bool = False):
    """gbs_expert_sort, and the rows of x [tokens, row_len] in that order: returns (rows, plan) with
    rows[r] = x[t] for the slot (t, k) at row r, zeros in rows without a slot."""
    if _fast is not None and stream is None and rows_out is not None and plan_out is not None and temp is not None and \
            num_rows is None:
        if _finish(_fast.dispatch(expert_ids, num_experts, first_expert, row_align, plan_out, temp, x, rows_out),
                   "gbs_expert_dispatch"):
            return (rows_out, plan_out, temp) if return_temp else (rows_out, plan_out)
    if stream is not None:
        return _on_stream(stream, gbs_expert_dispatch, x, expert_ids, num_experts, first_expert, row_align, num_rows,
                          rows_out, plan_out, temp, None, return_temp)
    row_type, id_type = _row_type(x, "x"), _id_type(expert_ids, "expert_ids")
    tokens, top_k, num_rows, plan, dev = _order(expert_ids, num_experts, row_align, num_rows, plan_out)
    row_len, dtype = x.size(1), x.dtype
    x_stride = _matrix(x, "x", tokens, row_len, dtype)
    if rows_out is None:
        rows_out = x.new_empty((num_rows, row_len))
    rows_stride = _matrix(rows_out, "rows_out", num_rows, row_len, dtype)
    if dev < 0 or dev != _current_device() or x.get_device() != dev or rows_out.get_device() != dev:
        _refuse_devices(expert_ids, x, rows_out)
    a, b, c, d = plan
    temp = _run(load().gbs_expert_dispatch, (row_type, x.data_ptr(), x_stride, row_len, id_type, expert_ids.data_ptr(), tokens, top_k,
                      num_experts, _int64(first_expert, "first_expert"), row_align, num_rows, rows_out.data_ptr(), rows_stride,
                      a.data_ptr(), b.data_ptr(), c.data_ptr(), d.data_ptr(), _raw_stream(dev)), temp, "gbs_expert_dispatch")
    return (rows_out, plan, temp) if return_temp else (rows_out, plan)


def gbs_expert_gather(x: torch.Tensor, slot_of_row: torch.Tensor, row_of_slot: torch.Tensor,
                      rows_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The rows of x [tokens, row_len] in the order of an earlier gbs_expert_sort or gbs_expert_dispatch."""
    if _fast is not None and stream is None and rows_out is not None:
        if _finish(_fast.gather(x, slot_of_row, row_of_slot, rows_out), "gbs_expert_gather"):
            return rows_out
    if stream is not None:
        return _on_stream(stream, gbs_expert_gather, x, slot_of_row, row_of_slot, rows_out)
    if row_of_slot.dim() != 2:
        raise ValueError("row_of_slot must be [tokens, top_k]")
    row_type = _row_type(x, "x")
    (tokens, top_k), num_rows, row_len, dtype = row_of_slot.shape, slot_of_row.numel(), x.size(1), x.dtype
    x_stride = _matrix(x, "x", tokens, row_len, dtype)
    _vector(slot_of_row, "slot_of_row", num_rows, torch.int32)
    _vector(row_of_slot, "row_of_slot", tokens * top_k, torch.int32)
    if rows_out is None:
        rows_out = x.new_empty((num_rows, row_len))
    rows_stride = _matrix(rows_out, "rows_out", num_rows, row_len, dtype)
    dev = x.get_device()
    if dev < 0 or dev != _current_device() or not (slot_of_row.get_device() == row_of_slot.get_device() ==
                                                   rows_out.get_device() == dev):
        _refuse_devices(x, slot_of_row, row_of_slot, rows_out)
    st = load().gbs_expert_gather(row_type, x.data_ptr(), x_stride, tokens, top_k, row_len, slot_of_row.data_ptr(),
                                  row_of_slot.data_ptr(), num_rows, rows_out.data_ptr(), rows_stride, _raw_stream(dev))
    if st != GBS_OK:
        raise GbsError(st, "gbs_expert_gather")
    return rows_out


def gbs_expert_combine(rows: torch.Tensor, row_of_slot: torch.Tensor, weights: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum over k of weights[t, k] * rows[row_of_slot[t, k]], without the slots that have no row;
    weights None: ones (the gradient of gbs_expert_gather with respect to x)."""
    if _fast is not None and stream is None and out is not None:
        if _finish(_fast.combine(rows, row_of_slot, weights, out), "gbs_expert_combine"):
            return out
    if stream is not None:
        return _on_stream(stream, gbs_expert_combine, rows, row_of_slot, weights, out)
    row_type, dtype, dev = _row_type(rows, "rows"), rows.dtype, rows.get_device()
    if row_of_slot.dim() != 2:
        raise ValueError("row_of_slot must be [tokens, top_k]")
    (tokens, top_k), (num_rows, row_len), (rows_stride, step) = row_of_slot.shape, rows.shape, rows.stride()
    if step != 1 and row_len > 1:
        _matrix(rows, "rows", num_rows, row_len, dtype)
    if row_of_slot.dtype is not torch.int32 or not row_of_slot.is_contiguous():
        _vector(row_of_slot, "row_of_slot", tokens * top_k, torch.int32)
    weight_type, w = GBS_ROW_F32, None
    if weights is not None:
        weight_type, w = _weight_type(weights, dtype, tokens * top_k), weights.data_ptr()
        if weights.get_device() != dev:
            _refuse_devices(rows, weights)
    if out is None:
        out = rows.new_empty((tokens, row_len))
    out_stride = _matrix(out, "out", tokens, row_len, dtype)
    if dev < 0 or dev != _current_device() or row_of_slot.get_device() != dev or out.get_device() != dev:
        _refuse_devices(rows, row_of_slot, out)
    st = load().gbs_expert_combine(row_type, rows.data_ptr(), rows_stride, num_rows, row_of_slot.data_ptr(), weight_type,
                                   w, tokens, top_k, row_len, out.data_ptr(), out_stride, _raw_stream(dev))
    if st != GBS_OK:
        raise GbsError(st, "gbs_expert_combine")
    return out


def gbs_expert_combine_grad(d_out: torch.Tensor, rows: torch.Tensor, slot_of_row: torch.Tensor,
                            row_of_slot: torch.Tensor, weights: torch.Tensor | None,
                            d_rows_out: torch.Tensor | None = None, d_weights_out: torch.Tensor | None = None, stream=None):
    """The gradient of gbs_expert_combine: (d_rows, d_weights) from d_out [tokens, row_len]; weights None: ones, which
    have no gradient (d_weights None), and rows is not read."""
    if _fast is not None and stream is None and d_rows_out is not None and d_weights_out is not None and \
            weights is not None:
        if _finish(_fast.combine_grad(d_out, rows, slot_of_row, row_of_slot, weights, d_rows_out, d_weights_out),
                   "gbs_expert_combine_grad"):
            return d_rows_out, d_weights_out
    if stream is not None:
        return _on_stream(stream, gbs_expert_combine_grad, d_out, rows, slot_of_row, row_of_slot, weights, d_rows_out,
                          d_weights_out)
    row_type, dtype, dev = _row_type(rows, "rows"), rows.dtype, rows.get_device()
    if row_of_slot.dim() != 2:
        raise ValueError("row_of_slot must be [tokens, top_k]")
    (tokens, top_k), (num_rows, row_len), (rows_stride, step) = row_of_slot.shape, rows.shape, rows.stride()
    if step != 1 and row_len > 1:
        _matrix(rows, "rows", num_rows, row_len, dtype)
    d_out_stride = _matrix(d_out, "d_out", tokens, row_len, dtype)
    i32, slots = torch.int32, tokens * top_k
    if slot_of_row.dtype is not i32 or slot_of_row.numel() != num_rows or not slot_of_row.is_contiguous():
        _vector(slot_of_row, "slot_of_row", num_rows, i32)
    if row_of_slot.dtype is not i32 or not row_of_slot.is_contiguous():
        _vector(row_of_slot, "row_of_slot", slots, i32)
    weight_type, w, d_w = GBS_ROW_F32, None, None
    if weights is None:
        if d_weights_out is not None:
            raise ValueError("d_weights_out must be None without weights")
    else:
        weight_type = _weight_type(weights, dtype, slots)
        if d_weights_out is None:
            d_weights_out = torch.empty_like(weights)
        _vector(d_weights_out, "d_weights_out", slots, weights.dtype)
        if weights.get_device() != dev or d_weights_out.get_device() != dev:
            _refuse_devices(rows, weights, d_weights_out)
        w, d_w = weights.data_ptr(), d_weights_out.data_ptr()
    if d_rows_out is None:
        d_rows_out = rows.new_empty((num_rows, row_len))
    d_rows_stride = _matrix(d_rows_out, "d_rows_out", num_rows, row_len, dtype)
    if dev < 0 or dev != _current_device() or not (
            d_out.get_device() == slot_of_row.get_device() == row_of_slot.get_device() == d_rows_out.get_device() == dev):
        _refuse_devices(d_out, rows, slot_of_row, row_of_slot, d_rows_out)
    st = load().gbs_expert_combine_grad(
        row_type, d_out.data_ptr(), d_out_stride, rows.data_ptr(), rows_stride, num_rows, slot_of_row.data_ptr(),
        row_of_slot.data_ptr(), weight_type, w, tokens, top_k, row_len, d_rows_out.data_ptr(), d_rows_stride, d_w,
        _raw_stream(dev))
    if st != GBS_OK:
        raise GbsError(st, "gbs_expert_combine_grad")
    return d_rows_out, d_weights_out


def _by_id(t: torch.Tensor, ids: torch.Tensor, row_len: int, what: str) -> torch.Tensor:
    """t [*ids.shape, row_len] as a matrix with a row per id."""
    if tuple(t.shape) != (*ids.shape, row_len):
        raise ValueError(f"{what} must be {[*ids.shape, row_len]}, got {list(t.shape)}")
    try:
        return t.view(ids.numel(), row_len)
    except RuntimeError:
        raise ValueError(f"{what} must have evenly spaced rows") from None


def gbs_embedding_lookup(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, first_id: int = 0,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[..., :] = scale * table[ids[...] - first_id], zeros for ids outside the table [vocab, row_len]."""
    if _fast is not None and stream is None and out is not None:
        if _finish(_fast.lookup(table, ids, scale, first_id, out), "gbs_embedding_lookup"):
            return out
    if stream is not None:
        return _on_stream(stream, gbs_embedding_lookup, table, ids, scale, first_id, out)
    row_type, id_type, dtype, dev = _row_type(table, "table"), _id_type(ids, "ids"), table.dtype, table.get_device()
    (vocab, row_len), (table_stride, step), n = table.shape, table.stride(), ids.numel()
    if step != 1 and row_len > 1:
        _matrix(table, "table", vocab, row_len, dtype)
    if out is None:
        out = table.new_empty((*ids.shape, row_len))
    flat = out if ids.dim() == 1 else _by_id(out, ids, row_len, "out")
    out_stride = _matrix(flat, "out", n, row_len, dtype)
    if dev < 0 or dev != _current_device() or ids.get_device() != dev or flat.get_device() != dev:
        _refuse_devices(table, ids, out)
    st = load().gbs_embedding_lookup(row_type, table.data_ptr(), table_stride, vocab, id_type, ids.data_ptr(), n,
                                     _int64(first_id, "first_id"), scale, row_len, flat.data_ptr(), out_stride,
                                     _raw_stream(dev))
    if st != GBS_OK:
        raise GbsError(st, "gbs_embedding_lookup")
    return out


def gbs_embedding_grad(d_out: torch.Tensor, ids: torch.Tensor, grad: torch.Tensor, scale: float = 1.0,
                       first_id: int = 0, padding_id: int | None = None, accumulate: bool = False,
                       temp: torch.Tensor | None = None, stream=None, return_temp: bool = False):
    """grad[v] (+)= scale * sum of d_out[i] over ids[i] - first_id == v, into grad [vocab, row_len] (float32 or
    d_out's type).  accumulate False writes every row, True adds to the rows whose ids occur.  The id
    padding_id adds nothing (None or negative: no such id; it does not count from the table's end).  d_out is
    [*ids.shape, row_len].  Equal calls (the same values and sizes, rows aligned alike) give equal bits."""
    if _fast is not None and stream is None and temp is not None:
        if _finish(_fast.grad(d_out, ids, grad, scale, first_id, -1 if padding_id is None else padding_id,
                              1 if accumulate else 0, temp), "gbs_embedding_grad"):
            return (grad, temp) if return_temp else grad
    if stream is not None:
        return _on_stream(stream, gbs_embedding_grad, d_out, ids, grad, scale, first_id, padding_id, accumulate, temp,
                          None, return_temp)
    grad_type, id_type, dev = _row_type(grad, "grad"), _id_type(ids, "ids"), grad.get_device()
    (vocab, row_len), n, dtype = grad.shape, ids.numel(), d_out.dtype
    flat = d_out if ids.dim() == 1 else _by_id(d_out, ids, row_len, "d_out")
    row_type = _row_type(flat, "d_out")
    if grad_type != row_type and grad_type != GBS_ROW_F32:
        raise TypeError(f"grad must be float32 or {dtype}, got {grad.dtype}")
    d_out_stride = _matrix(flat, "d_out", n, row_len, dtype)
    grad_stride = _matrix(grad, "grad", vocab, row_len, grad.dtype)
    if dev < 0 or dev != _current_device() or flat.get_device() != dev or ids.get_device() != dev:
        _refuse_devices(d_out, ids, grad)
    padding_id = -1 if padding_id is None else _int64(padding_id, "padding_id")
    temp = _run(load().gbs_embedding_grad,
                (row_type, flat.data_ptr(), d_out_stride, id_type, ids.data_ptr(), n, _int64(first_id, "first_id"), padding_id,
                 scale, vocab, row_len, grad_type, grad.data_ptr(), grad_stride, 1 if accumulate else 0, _raw_stream(dev)),
                temp, "gbs_embedding_grad")
    return (grad, temp) if return_temp else grad


def gbs_beam_select(logits: torch.Tensor, scores: torch.Tensor, num_out: int | None = None,
                    finished: torch.Tensor | None = None, end_id: int = 0, out: tuple | None = None,
                    temp: torch.Tensor | None = None, stream=None, return_temp: bool = False):
    """A beam search's next beams: (scores, beams, tokens) [batch, num_out] (num_out None: as many as there are beams),
    the best of scores[b, i] + log_softmax(logits[b * beams + i])[token], best first, ties to the lowest beam and token.
    scores is float32 [batch, beams], -inf for a beam that does not exist; a finished beam (bool or uint8
    [batch, beams]) has one candidate, end_id at its score.  Where too few candidates are left, the score is -inf and
    beam and token are -1.  beams and tokens are int32."""
    if _fast is not None and stream is None and out is not None and temp is not None and num_out is not None:
        if _finish(_fast.beam_select(logits, scores, num_out, finished, end_id, out, temp), "gbs_beam_select"):
            return (out, temp) if return_temp else out
    if stream is not None:
        return _on_stream(stream, gbs_beam_select, logits, scores, num_out, finished, end_id, out, temp, None, return_temp)
    row_type, dtype, dev = _row_type(logits, "logits"), logits.dtype, logits.get_device()
    if scores.dim() != 2:
        raise ValueError(f"scores must be [batch, beams], got {list(scores.shape)}")
    (batch, beams), vocab = scores.shape, logits.size(1)
    _vector(scores, "scores", batch * beams, torch.float32)
    stride = _matrix(logits, "logits", batch * beams, vocab, dtype)
    done = None
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"finished must be bool or uint8, got {finished.dtype}")
        _vector(finished, "finished", batch * beams, finished.dtype)
        done = finished.data_ptr()
    if num_out is None:
        num_out = beams
    if _int64(num_out, "num_out") < 1:
        raise ValueError("num_out must be positive")
    _int32(end_id, "end_id")
    if out is None:
        out = tuple(torch.empty((batch, num_out), dtype=t, device=logits.device)
                    for t in (torch.float32, torch.int32, torch.int32))
    for t, what, kind in zip(out, ("scores_out", "beams_out", "tokens_out"), (torch.float32, torch.int32, torch.int32)):
        _vector(t, what, batch * num_out, kind)
    if dev < 0 or dev != _current_device() or scores.get_device() != dev or any(t.get_device() != dev for t in out) or \
            (finished is not None and finished.get_device() != dev):
        _refuse_devices(logits, scores, finished, *out)
    temp = _run(load().gbs_beam_select,
                (row_type, logits.data_ptr(), stride, batch, beams, vocab, scores.data_ptr(), done, end_id, num_out,
                 out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), _raw_stream(dev)), temp, "gbs_beam_select")
    return (out, temp) if return_temp else out


def _merged(sizes, *strides):
    """(size, strides) of neighbouring dimensions as few as they can be, in one or several tensors."""
    dims = []
    for size, *at in reversed(list(zip(sizes, *strides))):
        if size == 1:
            continue
        if dims and all(a == b * dims[-1][0] for a, b in zip(at, dims[-1][1])):
            dims[-1] = (dims[-1][0] * size, dims[-1][1])
        else:
            dims.append((size, at))
    return dims[::-1]


def gbs_beam_reorder(state: torch.Tensor, parents: torch.Tensor, dim: int = 0, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """state[..., b, j, ...] = state[..., b, parents[b, j], ...] in place, or into out (of parents' beams), for
    dimensions dim (batch) and dim + 1 (beams) of state.  parents is int32 [batch, beams]; a beam whose parent is
    outside [0, beams) is left as it is.  Any element type.  The dimensions before dim, and those after the beams down
    to the neighbouring values, must each merge into one (a cache [layers, batch, beams, heads, length, size] cut to
    [..., :n, :] does)."""
    if stream is not None:
        return _on_stream(stream, gbs_beam_reorder, state, parents, dim, out)
    to = state if out is None else out
    if _fast is not None and _finish(_fast.beam_reorder(state, parents, dim, to), "gbs_beam_reorder"):
        return to
    if not 0 <= dim < state.dim() - 1:
        raise ValueError(f"dim must be one of the dimensions before state's last, got {dim}")
    if parents.dim() != 2 or parents.size(0) != state.size(dim):
        raise ValueError(f"parents must be [{state.size(dim)}, beams], got {list(parents.shape)}")
    batch, into = parents.shape
    shape, beams = tuple(state.shape), state.size(dim + 1)
    _vector(parents, "parents", batch * into, torch.int32)
    if to.dtype != state.dtype:
        raise TypeError(f"out must be {state.dtype}, got {to.dtype}")
    if tuple(to.shape) != (*shape[:dim + 1], into, *shape[dim + 2:]):
        raise ValueError(f"{'parents' if out is None else 'out'} must have {'the beams of state' if out is None else [*shape[:dim + 1], into, *shape[dim + 2:]]}")
    s, t = state.stride(), to.stride()
    outer, inner = [], []
    if state.numel():  # an empty state's dimensions need not merge
        outer, inner = _merged(shape[:dim], s[:dim], t[:dim]), _merged(shape[dim + 2:], s[dim + 2:], t[dim + 2:])
    length = inner.pop()[0] if inner and inner[-1][1] == [1, 1] else 1
    if len(outer) > 1 or len(inner) > 1:
        raise ValueError("state's and out's dimensions do not merge into outer ones, segments and neighbouring values")
    many, (o_in, o_out) = outer[0] if outer else (1, (0, 0))
    segments, (g_in, g_out) = inner[0] if inner else (1, (0, 0))
    dev, size = state.get_device(), state.element_size()
    if dev < 0 or dev != _current_device() or parents.get_device() != dev or to.get_device() != dev:
        _refuse_devices(state, parents, to)
    strides = ctypes.c_size_t * 4
    st = load().gbs_beam_reorder(
        state.data_ptr(), strides(o_in * size, s[dim] * size, s[dim + 1] * size, g_in * size), to.data_ptr(),
        strides(o_out * size, t[dim] * size, t[dim + 1] * size, g_out * size), many if state.numel() else 0, batch, beams, into,
        segments, length * size, parents.data_ptr(), _raw_stream(dev))
    if st != GBS_OK:
        raise GbsError(st, "gbs_beam_reorder")
    return to


def gbs_sort_keys_noalloc(keys_in: torch.Tensor, keys_out: torch.Tensor, begin_bit: int = 0,
                          end_bit: int | None = None, descending: bool = False, key_type: int | None = None,
                          stream=None) -> torch.Tensor:
    """gbs_sort_keys without a work buffer, for callers that cannot allocate device memory.

    keys_out must be allocated by the caller (it may be keys_in); nothing is
    allocated here either.  n <= GBS_NOALLOC_MAX_KEYS; calls share one
    library-owned scratch array, so they must not overlap on the GPU."""
    kind = _kind(keys_in, key_type)
    n = keys_in.numel()
    _check_tensor(keys_in, n, "keys_in")
    _check_tensor(keys_out, n, "keys_out")
    if end_bit is None:
        end_bit = 8 * _KIND_BYTES[kind]
    st = load().gbs_sort_keys_noalloc(kind, _ptr(keys_in), _ptr(keys_out), n, begin_bit, end_bit,
                                      int(bool(descending)), _stream(stream))
    if st != GBS_OK:
        raise GbsError(st, "gbs_sort_keys_noalloc")
    return keys_out


def gbs_get_status_noalloc(stream=None) -> int:
    """Synchronises the stream; GBS_ERR_TIMEOUT if the last gbs_sort_keys_noalloc call on the
    current device timed out."""
    return load().gbs_get_status_noalloc(_stream(stream))


def gbs_get_status(temp: torch.Tensor, stream=None) -> int:
    """Synchronises the stream; GBS_ERR_TIMEOUT if the last call on this work buffer timed out."""
    return load().gbs_get_status(_ptr(temp), temp.numel(), _stream(stream))


def gbs_debug_set_lookback_fault(pass_index: int, tile: int, spin_limit: int) -> None:
    load().gbs_debug_set_lookback_fault(pass_index, tile, spin_limit)


def gbs_debug_set_ring_fault(chunk: int, spin_limit: int) -> None:
    load().gbs_debug_set_ring_fault(chunk, spin_limit)


def gbs_debug_set_radix_bits(bits: int) -> None:
    """8 (default) or 11: digit width of later keys-only radix sorts below 2^29 keys (test hook)."""
    load().gbs_debug_set_radix_bits(bits)


def gbs_debug_last_launch_count() -> int:
    return load().gbs_debug_last_launch_count()


_timing_keepalive = None


def gbs_debug_set_timing_events(events) -> None:
    """events: list of torch.cuda.Event(enable_timing=True), or None to switch the hook off.

    torch creates an event's CUDA handle on its first record, so unrecorded
    events are recorded once here first."""
    global _timing_keepalive
    if not events:
        _timing_keepalive = None
        load().gbs_debug_set_timing_events(None, 0)
        return
    for e in events:
        if not e.cuda_event:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _timing_keepalive = (arr, list(events))
    load().gbs_debug_set_timing_events(arr, len(events))


def gbs_debug_radix_tile_keys(key_bytes: int, pairs: bool = False, value_bytes: int | None = None) -> int:
    """Keys per radix tile; value_bytes (0, 4 or 8) overrides pairs (4-byte values)."""
    vb = value_bytes if value_bytes is not None else (4 if pairs else 0)
    return load().gbs_debug_radix_tile_keys(key_bytes, vb)
