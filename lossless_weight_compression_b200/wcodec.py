"""ctypes binding of libwcodec (include/wcodec.h), plus torch-tensor helpers.

The ``wc_*`` functions take the same arguments as the C functions (device
pointers as ints, sizes, a cudaStream_t as an int); they only marshal
arguments. Every step of compression and decompression runs in the library's
CUDA kernels; there is no Python or CPU fallback, and loading fails loudly if
``libwcodec.so`` has not been built (``python -m
lossless_weight_compression_b200.build_lib``).

The helpers below (``compress``, ``decompress``, ...) take torch tensors,
allocate outputs with torch and call the same entry points.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libwcodec.so")

WC_OK = 0
WC_ERR_INVALID_ARG = 1
WC_ERR_BUFFER_TOO_SMALL = 2
WC_ERR_CORRUPT_STREAM = 3
WC_ERR_CUDA = 4
WC_ERR_TIMEOUT = 5
WC_HEADER_BYTES = 128
WC_BATCH_MAX = 512
BLOCK_SIZES = (128, 256, 512, 1024, 2048, 4096)


class WcodecError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d)" % (what, wc_status_string(status), status))
        self.status = status


class wc_compress_item(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p),
        ("n", ctypes.c_uint64),
        ("block", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
        ("out", ctypes.c_void_p),
        ("out_capacity", ctypes.c_uint64),
        ("out_bytes", ctypes.c_void_p),
    ]


class wc_gemv_item(ctypes.Structure):
    _fields_ = [
        ("stream", ctypes.c_void_p),
        ("stream_bytes", ctypes.c_uint64),
        ("x", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("rows", ctypes.c_uint32),
        ("cols", ctypes.c_uint32),
        ("block", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
    ]


class wc_batch_item(ctypes.Structure):
    _fields_ = [
        ("stream", ctypes.c_void_p),
        ("stream_bytes", ctypes.c_uint64),
        ("out", ctypes.c_void_p),
        ("n", ctypes.c_uint64),
        ("block", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libwcodec.so (once). Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            "libwcodec.so is not built (%s); run `python -m lossless_weight_compression_b200."
            "build_lib`" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    u32, u64, vp, i = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int
    L.wc_bound.argtypes, L.wc_bound.restype = [u64, u32], u64
    L.wc_workspace_size.argtypes, L.wc_workspace_size.restype = [u64, u32], u64
    L.wc_compress.argtypes = [vp, u64, u32, vp, u64, vp, vp, u64, vp, vp]
    L.wc_compress.restype = i
    L.wc_decompress.argtypes = [vp, u64, vp, u64, u32, vp, vp]
    L.wc_decompress.restype = i
    L.wc_decompress_batch.argtypes = [ctypes.POINTER(wc_batch_item), u32, vp, vp]
    L.wc_decompress_batch.restype = i
    L.wc_stream_info.argtypes = [vp, u64, ctypes.POINTER(u64), ctypes.POINTER(u32),
                                 ctypes.POINTER(u64)]
    L.wc_stream_info.restype = i
    L.wc_status_string.argtypes, L.wc_status_string.restype = [i], ctypes.c_char_p
    L.wc_compress_batch_workspace_size.argtypes = [ctypes.POINTER(wc_compress_item), u32]
    L.wc_compress_batch_workspace_size.restype = u64
    L.wc_compress_batch.argtypes = [ctypes.POINTER(wc_compress_item), u32, vp, u64, vp, vp]
    L.wc_compress_batch.restype = i
    L.wc_gemv.argtypes = [vp, u64, u32, u32, u32, vp, u32, vp, vp, vp]
    L.wc_gemv.restype = i
    L.wc_gemv_batch.argtypes = [ctypes.POINTER(wc_gemv_item), u32, u32, vp, vp]
    L.wc_gemv_batch.restype = i
    L.wc_bound_fp32.argtypes, L.wc_bound_fp32.restype = [u64, u32], u64
    L.wc_compress_fp32.argtypes = [vp, u64, u32, vp, u64, vp, vp, u64, vp, vp]
    L.wc_compress_fp32.restype = i
    L.wc_decompress_fp32.argtypes = [vp, u64, vp, u64, u32, vp, vp]
    L.wc_decompress_fp32.restype = i
    L.wc_gemm.argtypes = [vp, u64, u32, u32, u32, vp, u32, vp, vp, vp]
    L.wc_gemm.restype = i
    L.wc_gemm_batch.argtypes = [ctypes.POINTER(wc_gemv_item), u32, u32, vp, vp]
    L.wc_gemm_batch.restype = i
    L.wc_gemm_batch_flags.argtypes = [ctypes.POINTER(wc_gemv_item), u32, u32, u32, vp, vp]
    L.wc_gemm_batch_flags.restype = i
    L.wc_bound_tans.argtypes, L.wc_bound_tans.restype = [u64, u32, u32], u64
    L.wc_compress_tans_batch_workspace_size.argtypes = [ctypes.POINTER(wc_compress_item), u32]
    L.wc_compress_tans_batch_workspace_size.restype = u64
    L.wc_compress_tans.argtypes = [vp, u64, u32, u32, vp, u64, vp, vp, u64, vp]
    L.wc_compress_tans.restype = i
    L.wc_compress_tans_batch.argtypes = [ctypes.POINTER(wc_compress_item), u32, u32, vp, u64, vp]
    L.wc_compress_tans_batch.restype = i
    L.wc_decompress_tans.argtypes = [vp, u64, vp, u64, u32, vp, vp]
    L.wc_decompress_tans.restype = i
    L.wc_decompress_tans_batch.argtypes = [ctypes.POINTER(wc_batch_item), u32, vp, vp]
    L.wc_decompress_tans_batch.restype = i
    L.wc_compress_noalloc.argtypes = [vp, u64, u32, vp, u64, vp, vp, vp]
    L.wc_compress_noalloc.restype = i
    L.wc_debug_compress_stalled.argtypes = [vp, u64, u32, vp, u64, vp, vp, u64, vp, u64, vp]
    L.wc_debug_compress_stalled.restype = i
    L.wc_bound_escape.argtypes, L.wc_bound_escape.restype = [u64, u32], u64
    L.wc_workspace_size_escape.argtypes, L.wc_workspace_size_escape.restype = [u64, u32], u64
    L.wc_compress_escape.argtypes = [vp, u64, u32, vp, u64, vp, vp, u64, vp, vp]
    L.wc_compress_escape.restype = i
    L.wc_decompress_escape.argtypes = [vp, u64, vp, u64, u32, vp, vp]
    L.wc_decompress_escape.restype = i
    L.wc_decompress_escape_batch.argtypes = [ctypes.POINTER(wc_batch_item), u32, vp, vp]
    L.wc_decompress_escape_batch.restype = i
    L.wc_compress_escape_batch_workspace_size.argtypes = [ctypes.POINTER(wc_compress_item), u32]
    L.wc_compress_escape_batch_workspace_size.restype = u64
    L.wc_compress_escape_batch.argtypes = [ctypes.POINTER(wc_compress_item), u32, vp, u64, vp, vp]
    L.wc_compress_escape_batch.restype = i
    L.wc_decompress_host.argtypes = [vp, u64, vp, u64, u32, u32, vp, vp]
    L.wc_decompress_host.restype = i
    L.wc_decompress_host_batch.argtypes = [ctypes.POINTER(wc_batch_item), u32, u32, vp, vp]
    L.wc_decompress_host_batch.restype = i
    L.wc_q4_bytes.argtypes, L.wc_q4_bytes.restype = [u64, u64, u32, u32], u64
    L.wc_q4_quantize.argtypes = [vp, u64, u64, u64, u32, u32, vp, u64, vp]
    L.wc_q4_quantize.restype = i
    L.wc_q4_pack.argtypes = [vp, vp, vp, u64, u64, u32, u32, vp, u64, vp]
    L.wc_q4_pack.restype = i
    L.wc_q4_dequantize.argtypes = [vp, u64, u64, u64, u32, u32, vp, u64, u32, vp, vp]
    L.wc_q4_dequantize.restype = i
    L.wc_q4_gemm.argtypes = [vp, u64, u64, u64, u32, u32, vp, u64, u64, vp, u64, vp, vp]
    L.wc_q4_gemm.restype = i
    L.wc_q4_gemm_experts.argtypes = [vp, u64, u32, u64, u64, u32, u32, vp, u64, u64, vp, vp, u64,
                                     vp, vp]
    L.wc_q4_gemm_experts.restype = i
    L.wc_moe_sort.argtypes, L.wc_moe_sort.restype = [vp, u64, u32, vp, vp, vp, vp], i
    L.wc_moe_gather.argtypes = [vp, u64, u64, u64, u64, u32, vp, vp, u64, u64, vp]
    L.wc_moe_gather.restype = i
    L.wc_moe_combine.argtypes = [vp, u64, u64, u64, u64, u64, u32, vp, vp, vp, u64, vp]
    L.wc_moe_combine.restype = i
    L.wc_moe_combine_backward.argtypes = [vp, u64, vp, u64, u64, u64, u64, u64, u32, vp, vp, vp, u64,
                                          vp, vp]
    L.wc_moe_combine_backward.restype = i
    _lib = L
    return L


# ---------------------------------------------------------------------------
# The C functions, same names and arguments
# ---------------------------------------------------------------------------
def wc_bound(n: int, block: int) -> int:
    return lib().wc_bound(n, block)


def wc_workspace_size(n: int, block: int) -> int:
    return lib().wc_workspace_size(n, block)


def wc_compress(d_in, n, block, d_out, out_capacity, d_out_bytes, d_workspace, workspace_bytes,
                d_status, stream) -> int:
    return lib().wc_compress(d_in, n, block, d_out, out_capacity, d_out_bytes, d_workspace,
                             workspace_bytes, d_status, stream)


def wc_compress_batch_workspace_size(items, count) -> int:
    return lib().wc_compress_batch_workspace_size(items, count)


def wc_compress_batch(items, count, d_workspace, workspace_bytes, d_status, stream) -> int:
    return lib().wc_compress_batch(items, count, d_workspace, workspace_bytes, d_status, stream)


def wc_compress_noalloc(d_in, n, block, d_out, out_capacity, d_out_bytes, d_status,
                        stream) -> int:
    """wc_compress without a workspace, for callers that cannot allocate device
    memory; its scratch is a fixed array in the library (n <= 2^30)."""
    return lib().wc_compress_noalloc(d_in, n, block, d_out, out_capacity, d_out_bytes, d_status,
                                     stream)


def wc_decompress(d_stream, stream_bytes, d_out, n, block, d_status, stream) -> int:
    return lib().wc_decompress(d_stream, stream_bytes, d_out, n, block, d_status, stream)


def wc_decompress_batch(items, count, d_status, stream) -> int:
    return lib().wc_decompress_batch(items, count, d_status, stream)


def wc_gemv(d_stream, stream_bytes, rows, cols, block, d_x, n_vec, d_y, d_status, stream) -> int:
    return lib().wc_gemv(d_stream, stream_bytes, rows, cols, block, d_x, n_vec, d_y, d_status,
                         stream)


def wc_gemv_batch(items, count, n_vec, d_status, stream) -> int:
    return lib().wc_gemv_batch(items, count, n_vec, d_status, stream)


def wc_bound_fp32(n, block) -> int:
    return lib().wc_bound_fp32(n, block)


def wc_compress_fp32(d_in, n, block, d_out, out_capacity, d_out_bytes, d_ws, ws_bytes, d_status,
                     stream) -> int:
    return lib().wc_compress_fp32(d_in, n, block, d_out, out_capacity, d_out_bytes, d_ws,
                                  ws_bytes, d_status, stream)


def wc_decompress_fp32(d_stream, stream_bytes, d_out, n, block, d_status, stream) -> int:
    return lib().wc_decompress_fp32(d_stream, stream_bytes, d_out, n, block, d_status, stream)


def wc_gemm(d_stream, stream_bytes, rows, cols, block, d_x, tokens, d_y, d_status, stream) -> int:
    return lib().wc_gemm(d_stream, stream_bytes, rows, cols, block, d_x, tokens, d_y, d_status,
                         stream)


def wc_bound_tans(n, chunk, table_log) -> int:
    return lib().wc_bound_tans(n, chunk, table_log)


def wc_compress_tans_batch_workspace_size(items, count) -> int:
    return lib().wc_compress_tans_batch_workspace_size(items, count)


def wc_compress_tans(d_in, n, chunk, table_log, d_out, out_capacity, d_out_bytes, d_ws, ws_bytes,
                     stream) -> int:
    return lib().wc_compress_tans(d_in, n, chunk, table_log, d_out, out_capacity, d_out_bytes,
                                  d_ws, ws_bytes, stream)


def wc_compress_tans_batch(items, count, table_log, d_ws, ws_bytes, stream) -> int:
    return lib().wc_compress_tans_batch(items, count, table_log, d_ws, ws_bytes, stream)


def wc_decompress_tans(d_stream, stream_bytes, d_out, n, chunk, d_status, stream) -> int:
    return lib().wc_decompress_tans(d_stream, stream_bytes, d_out, n, chunk, d_status, stream)


def wc_decompress_tans_batch(items, count, d_status, stream) -> int:
    return lib().wc_decompress_tans_batch(items, count, d_status, stream)


def wc_gemm_batch_flags(items, count, tokens, flags, d_status, stream) -> int:
    return lib().wc_gemm_batch_flags(items, count, tokens, flags, d_status, stream)


def wc_gemm_batch(items, count, tokens, d_status, stream) -> int:
    return lib().wc_gemm_batch(items, count, tokens, d_status, stream)


def wc_bound_escape(n, block) -> int:
    return lib().wc_bound_escape(n, block)


def wc_workspace_size_escape(n, block) -> int:
    return lib().wc_workspace_size_escape(n, block)


def wc_compress_escape(d_in, n, block, d_out, out_capacity, d_out_bytes, d_ws, ws_bytes, d_status,
                       stream) -> int:
    return lib().wc_compress_escape(d_in, n, block, d_out, out_capacity, d_out_bytes, d_ws,
                                    ws_bytes, d_status, stream)


def wc_decompress_escape(d_stream, stream_bytes, d_out, n, block, d_status, stream) -> int:
    return lib().wc_decompress_escape(d_stream, stream_bytes, d_out, n, block, d_status, stream)


def wc_decompress_escape_batch(items, count, d_status, stream) -> int:
    return lib().wc_decompress_escape_batch(items, count, d_status, stream)


WC_FLAG_ESCAPE = 2


def wc_compress_escape_batch_workspace_size(items, count) -> int:
    return lib().wc_compress_escape_batch_workspace_size(items, count)


def wc_compress_escape_batch(items, count, d_workspace, workspace_bytes, d_status, stream) -> int:
    return lib().wc_compress_escape_batch(items, count, d_workspace, workspace_bytes, d_status,
                                          stream)


def wc_decompress_host(h_stream, stream_bytes, d_out, n, block, flags, d_status, stream) -> int:
    return lib().wc_decompress_host(h_stream, stream_bytes, d_out, n, block, flags, d_status,
                                    stream)


def wc_decompress_host_batch(items, count, flags, d_status, stream) -> int:
    return lib().wc_decompress_host_batch(items, count, flags, d_status, stream)


WC_Q4_ZEROS = 1
WC_Q4_SCALES_FP16 = 2
WC_Q4_X_FP16 = 4
WC_Q4_Y_16BIT = 8
WC_DTYPE_BF16, WC_DTYPE_FP16, WC_DTYPE_FP32 = 0, 1, 2
WC_MOE_MAX_EXPERTS = 1024


def wc_q4_bytes(rows, cols, group, flags) -> int:
    return lib().wc_q4_bytes(rows, cols, group, flags)


def wc_q4_quantize(d_w, ld, rows, cols, group, flags, d_out, out_capacity, stream) -> int:
    return lib().wc_q4_quantize(d_w, ld, rows, cols, group, flags, d_out, out_capacity, stream)


def wc_q4_pack(d_codes, d_scales, d_zeros, rows, cols, group, flags, d_out, out_capacity,
               stream) -> int:
    return lib().wc_q4_pack(d_codes, d_scales, d_zeros, rows, cols, group, flags, d_out,
                            out_capacity, stream)


def wc_q4_dequantize(d_stream, stream_bytes, rows, cols, group, flags, d_out, ld, dtype, d_status,
                     stream) -> int:
    return lib().wc_q4_dequantize(d_stream, stream_bytes, rows, cols, group, flags, d_out, ld,
                                  dtype, d_status, stream)


def wc_q4_gemm(d_stream, stream_bytes, rows, cols, group, flags, d_x, ldx, tokens, d_y, ldy,
               d_status, stream) -> int:
    return lib().wc_q4_gemm(d_stream, stream_bytes, rows, cols, group, flags, d_x, ldx, tokens, d_y,
                            ldy, d_status, stream)


def wc_q4_gemm_experts(d_streams, stream_stride, experts, rows, cols, group, flags, d_x, ldx,
                       tokens, d_offsets, d_y, ldy, d_status, stream) -> int:
    return lib().wc_q4_gemm_experts(d_streams, stream_stride, experts, rows, cols, group, flags,
                                    d_x, ldx, tokens, d_offsets, d_y, ldy, d_status, stream)


def wc_moe_sort(d_ids, slots, experts, d_offsets, d_order, d_inverse, stream) -> int:
    return lib().wc_moe_sort(d_ids, slots, experts, d_offsets, d_order, d_inverse, stream)


def wc_moe_gather(d_x, ldx, tokens, top, cols, dtype, d_inverse, d_rows, ldr, rows, stream) -> int:
    return lib().wc_moe_gather(d_x, ldx, tokens, top, cols, dtype, d_inverse, d_rows, ldr, rows,
                               stream)


def wc_moe_combine(d_rows, ldr, rows, tokens, top, cols, dtype, d_inverse, d_weights, d_out, ldo,
                   stream) -> int:
    return lib().wc_moe_combine(d_rows, ldr, rows, tokens, top, cols, dtype, d_inverse, d_weights,
                                d_out, ldo, stream)


def wc_moe_combine_backward(d_dout, ldd, d_rows, ldr, rows, tokens, top, cols, dtype, d_inverse,
                            d_weights, d_drows, lddr, d_dweights, stream) -> int:
    return lib().wc_moe_combine_backward(d_dout, ldd, d_rows, ldr, rows, tokens, top, cols, dtype,
                                         d_inverse, d_weights, d_drows, lddr, d_dweights, stream)


def wc_stream_info(h_header: bytes):
    """Returns (status, n, block, total_bytes) parsed from a host copy of the header."""
    n, blk, tot = ctypes.c_uint64(), ctypes.c_uint32(), ctypes.c_uint64()
    buf = ctypes.create_string_buffer(bytes(h_header), len(h_header))
    rc = lib().wc_stream_info(ctypes.cast(buf, ctypes.c_void_p), len(h_header), ctypes.byref(n),
                              ctypes.byref(blk), ctypes.byref(tot))
    return rc, n.value, blk.value, tot.value


def wc_status_string(status: int) -> str:
    return lib().wc_status_string(status).decode()


def wc_debug_compress_stalled(d_in, n, block, d_out, out_capacity, d_out_bytes, d_workspace,
                              workspace_bytes, d_status, timeout_ns, stream) -> int:
    return lib().wc_debug_compress_stalled(d_in, n, block, d_out, out_capacity, d_out_bytes,
                                           d_workspace, workspace_bytes, d_status, timeout_ns,
                                           stream)


# ---------------------------------------------------------------------------
# torch helpers
# ---------------------------------------------------------------------------
def _stream_handle(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(rc: int, what: str):
    if rc != WC_OK:
        raise WcodecError(rc, what)


def as_words(x: torch.Tensor) -> torch.Tensor:
    """A 16-bit tensor (bf16 / int16 / uint16 / fp16) as contiguous flat int16 words."""
    if x.element_size() != 2:
        raise TypeError("wcodec compresses 16-bit words (BF16); got %s" % x.dtype)
    return x.contiguous().view(-1).view(torch.int16)


@dataclass
class Compressed:
    """A compressed tensor on the GPU: ``buffer`` holds ``wc_bound`` bytes of
    which the first ``nbytes`` (a device int64) are the stream."""
    buffer: torch.Tensor
    nbytes: torch.Tensor
    status: torch.Tensor
    n: int
    block: int
    shape: tuple
    dtype: torch.dtype
    escape: bool = False  # an escape-coded stream (header flags bit 1)

    def size(self) -> int:
        return int(self.nbytes.item())

    def stream(self) -> torch.Tensor:
        """The stream bytes (synchronises to read the size)."""
        return self.buffer[: self.size()]


def workspace_for(n: int, block: int, device) -> torch.Tensor:
    ws = wc_workspace_size(n, block)
    if ws == 0:
        raise WcodecError(WC_ERR_INVALID_ARG, "workspace size")
    return torch.empty((ws + 15) // 16 * 16, dtype=torch.uint8, device=device)


def compress(x: torch.Tensor, block: int = 1024, *, workspace: torch.Tensor | None = None,
             stream=None) -> Compressed:
    """Compress a CUDA tensor of BF16 (any 16-bit dtype is read as bit patterns)."""
    words = as_words(x)
    n = words.numel()
    cap = wc_bound(n, block)
    if cap == 0:
        raise WcodecError(WC_ERR_INVALID_ARG, "block size %r" % (block,))
    dev = words.device
    buf = torch.empty((cap + 15) // 16 * 16, dtype=torch.uint8, device=dev)
    nbytes = torch.zeros(1, dtype=torch.int64, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = workspace_for(n, block, dev)
    rc = wc_compress(words.data_ptr() if n else None, n, block, buf.data_ptr(), buf.numel(),
                     nbytes.data_ptr(), workspace.data_ptr(), workspace.numel(),
                     status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_compress")
    return Compressed(buf, nbytes, status, n, block, tuple(x.shape), x.dtype)


def decompress(stream_bytes: torch.Tensor, n: int, block: int, *, out: torch.Tensor | None = None,
               status: torch.Tensor | None = None, nbytes: int | None = None,
               stream=None) -> torch.Tensor:
    """Decode a stream (a uint8 CUDA tensor) into n BF16 values (``out`` if given)."""
    if out is None:
        out = torch.empty(n, dtype=torch.bfloat16, device=stream_bytes.device)
    words = out.view(-1)
    if words.numel() != n or not words.is_contiguous() or out.element_size() != 2:
        raise ValueError("out must be a contiguous 16-bit tensor of %d elements" % n)
    own_status = status is None
    if own_status:
        status = torch.zeros(1, dtype=torch.int32, device=stream_bytes.device)
    size = stream_bytes.numel() if nbytes is None else nbytes
    rc = wc_decompress(stream_bytes.data_ptr(), size, words.data_ptr() if n else None, n, block,
                       status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress")
    return out


def decompress_compressed(c: Compressed, out: torch.Tensor | None = None, status=None,
                          stream=None) -> torch.Tensor:
    """Decode a ``Compressed`` (plain or escape-coded) back into its original shape and dtype."""
    if out is None:
        out = torch.empty(c.shape, dtype=c.dtype, device=c.buffer.device)
    fn = decompress_escape if c.escape else decompress
    return fn(c.buffer, c.n, c.block, out=out, status=status, stream=stream)


class CompressBatch:
    """Reusable buffers and descriptors for compressing a fixed list of tensors
    in one call: ``run()`` enqueues one encoder launch per 512 tensors (five for
    escape-coded streams, ``escape=True``; five per 512 for tANS-coded streams,
    ``tans_log=R``, whose ``block`` is then the chunk size)."""

    def __init__(self, tensors, block=1024, escape=False, tans_log=None):
        self.escape = escape
        self.tans_log = tans_log
        if tans_log is not None:
            def bound(n, b):
                return wc_bound_tans(n, b, tans_log)
        else:
            bound = wc_bound_escape if escape else wc_bound
        self.words = [as_words(t) for t in tensors]
        dev = self.words[0].device if self.words else torch.device("cuda")
        k = len(self.words)
        self.blocks = list(block) if isinstance(block, (list, tuple)) else [block] * k
        self.buffers = [torch.empty((bound(w.numel(), b) + 15) // 16 * 16,
                                    dtype=torch.uint8, device=dev)
                        for w, b in zip(self.words, self.blocks)]
        self.nbytes = torch.zeros(max(1, k), dtype=torch.int64, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.items = (wc_compress_item * max(1, k))()
        for j, w in enumerate(self.words):
            it = self.items[j]
            it.in_ = w.data_ptr() if w.numel() else None
            it.n = w.numel()
            it.block = self.blocks[j]
            it.reserved = 0
            it.out = self.buffers[j].data_ptr()
            it.out_capacity = self.buffers[j].numel()
            it.out_bytes = self.nbytes[j:].data_ptr()
        if tans_log is not None:
            ws = wc_compress_tans_batch_workspace_size(self.items, k)
        else:
            ws = (wc_compress_escape_batch_workspace_size if escape
                  else wc_compress_batch_workspace_size)(self.items, k)
        if k and ws == 0:
            raise WcodecError(WC_ERR_INVALID_ARG, "workspace size")
        self.workspace = torch.empty(max(16, (ws + 15) // 16 * 16), dtype=torch.uint8, device=dev)
        self.count = k

    def run(self, stream=None):
        if self.tans_log is not None:
            rc = wc_compress_tans_batch(self.items, self.count, self.tans_log,
                                        self.workspace.data_ptr(), self.workspace.numel(),
                                        _stream_handle(stream))
            _check(rc, "wc_compress_tans_batch")
            return
        entry = wc_compress_escape_batch if self.escape else wc_compress_batch
        rc = entry(self.items, self.count, self.workspace.data_ptr(), self.workspace.numel(),
                   self.status.data_ptr(), _stream_handle(stream))
        _check(rc, entry.__name__)

    def sizes(self) -> list[int]:
        return self.nbytes[: self.count].cpu().tolist()


def make_batch(items) -> ctypes.Array:
    """items: iterable of (stream uint8 tensor, stream_bytes, out tensor, n, block)."""
    items = list(items)
    arr = (wc_batch_item * max(1, len(items)))()
    for k, (s, sb, o, n, b) in enumerate(items):
        arr[k].stream = s.data_ptr()
        arr[k].stream_bytes = sb
        arr[k].out = o.data_ptr() if n else None
        arr[k].n = n
        arr[k].block = b
        arr[k].reserved = 0
    return arr, len(items)


def decompress_batch(batch, status: torch.Tensor, stream=None):
    """Decode a batch made by ``make_batch`` in one launch per 512 tensors."""
    arr, count = batch
    rc = wc_decompress_batch(arr, count, status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress_batch")


def stream_info(header: bytes):
    rc, n, block, total = wc_stream_info(header)
    _check(rc, "wc_stream_info")
    return n, block, total


def gemv(stream_bytes: torch.Tensor, rows: int, cols: int, block: int, x: torch.Tensor, *,
         nbytes: int | None = None, y: torch.Tensor | None = None,
         status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x @ W.T with W (rows x cols BF16) given as its stream; x is (n_vec, cols)
    with n_vec in {1, 2, 4}; returns FP32 (n_vec, rows)."""
    xw = as_words(x).view(-1, cols)
    n_vec = xw.shape[0]
    if y is None:
        y = torch.empty((n_vec, rows), dtype=torch.float32, device=stream_bytes.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=stream_bytes.device)
    rc = wc_gemv(stream_bytes.data_ptr(), stream_bytes.numel() if nbytes is None else nbytes,
                 rows, cols, block, xw.data_ptr(), n_vec, y.data_ptr(), status.data_ptr(),
                 _stream_handle(stream))
    _check(rc, "wc_gemv")
    return y


def make_gemv_batch(items) -> tuple:
    """items: iterable of (stream uint8 tensor, stream_bytes, x (n_vec, cols), y (n_vec, rows), rows, cols, block)."""
    items = list(items)
    arr = (wc_gemv_item * max(1, len(items)))()
    for k, (s, sb, x, y, rows, cols, b) in enumerate(items):
        arr[k].stream = s.data_ptr()
        arr[k].stream_bytes = sb
        arr[k].x = x.data_ptr()
        arr[k].y = y.data_ptr()
        arr[k].rows, arr[k].cols, arr[k].block, arr[k].reserved = rows, cols, b, 0
    return arr, len(items)


def gemv_batch(batch, n_vec: int, status: torch.Tensor, stream=None):
    arr, count = batch
    rc = wc_gemv_batch(arr, count, n_vec, status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_gemv_batch")


GEMM_MAX_TOKENS = 128


def gemm(stream_bytes: torch.Tensor, rows: int, cols: int, block: int, x: torch.Tensor, *,
         nbytes: int | None = None, y: torch.Tensor | None = None,
         status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x @ W.T on the tensor cores with W (rows x cols BF16) given as its stream;
    x is (tokens, cols) BF16 with 1 <= tokens <= 128; returns FP32 (tokens, rows)."""
    xw = as_words(x).view(-1, cols)
    tokens = xw.shape[0]
    if y is None:
        y = torch.empty((tokens, rows), dtype=torch.float32, device=stream_bytes.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=stream_bytes.device)
    rc = wc_gemm(stream_bytes.data_ptr(), stream_bytes.numel() if nbytes is None else nbytes,
                 rows, cols, block, xw.data_ptr(), tokens, y.data_ptr(), status.data_ptr(),
                 _stream_handle(stream))
    _check(rc, "wc_gemm")
    return y


def gemm_batch(batch, tokens: int, status: torch.Tensor, stream=None, escape: bool = False):
    """batch from make_gemv_batch (x (tokens, cols), y (tokens, rows) per item);
    escape: the streams are escape-coded (every row whole blocks)."""
    arr, count = batch
    rc = wc_gemm_batch_flags(arr, count, tokens, WC_FLAG_ESCAPE if escape else 0,
                             status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_gemm_batch_flags")


def compress_fp32(x: torch.Tensor, block: int = 1024, *, workspace: torch.Tensor | None = None,
                  stream=None) -> Compressed:
    """Compress a CUDA tensor of 32-bit words (FP32, read as bit patterns)."""
    if x.element_size() != 4:
        raise TypeError("compress_fp32 takes 32-bit words; got %s" % x.dtype)
    words = x.contiguous().view(-1).view(torch.int32)
    n = words.numel()
    cap = wc_bound_fp32(n, block)
    if cap == 0:
        raise WcodecError(WC_ERR_INVALID_ARG, "block size %r" % (block,))
    dev = words.device
    buf = torch.empty((cap + 15) // 16 * 16, dtype=torch.uint8, device=dev)
    nbytes = torch.zeros(1, dtype=torch.int64, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = workspace_for(n, block, dev)
    rc = wc_compress_fp32(words.data_ptr() if n else None, n, block, buf.data_ptr(), buf.numel(),
                          nbytes.data_ptr(), workspace.data_ptr(), workspace.numel(),
                          status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_compress_fp32")
    return Compressed(buf, nbytes, status, n, block, tuple(x.shape), x.dtype)


def decompress_fp32(stream_bytes: torch.Tensor, n: int, block: int, *,
                    out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                    nbytes: int | None = None, stream=None) -> torch.Tensor:
    """Decode an FP32 stream into n FP32 values (``out`` if given)."""
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=stream_bytes.device)
    words = out.view(-1)
    if words.numel() != n or not words.is_contiguous() or out.element_size() != 4:
        raise ValueError("out must be a contiguous 32-bit tensor of %d elements" % n)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=stream_bytes.device)
    size = stream_bytes.numel() if nbytes is None else nbytes
    rc = wc_decompress_fp32(stream_bytes.data_ptr(), size, words.data_ptr() if n else None, n,
                            block, status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress_fp32")
    return out


# ---------------------------------------------------------------------------
# escape-coded streams (a window of 2^w - 1 exponents per block + exceptions)
# ---------------------------------------------------------------------------
def compress_escape(x: torch.Tensor, block: int = 1024, *, workspace: torch.Tensor | None = None,
                    stream=None) -> Compressed:
    """Compress a CUDA tensor of 16-bit words into an escape-coded stream."""
    words = as_words(x)
    n = words.numel()
    cap = wc_bound_escape(n, block)
    if cap == 0:
        raise WcodecError(WC_ERR_INVALID_ARG, "block size %r" % (block,))
    dev = words.device
    buf = torch.empty((cap + 15) // 16 * 16, dtype=torch.uint8, device=dev)
    nbytes = torch.zeros(1, dtype=torch.int64, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if workspace is None:
        ws = wc_workspace_size_escape(n, block)
        workspace = torch.empty((ws + 15) // 16 * 16, dtype=torch.uint8, device=dev)
    rc = wc_compress_escape(words.data_ptr() if n else None, n, block, buf.data_ptr(),
                            buf.numel(), nbytes.data_ptr(), workspace.data_ptr(),
                            workspace.numel(), status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_compress_escape")
    return Compressed(buf, nbytes, status, n, block, tuple(x.shape), x.dtype, escape=True)


def decompress_escape(stream_bytes: torch.Tensor, n: int, block: int, *,
                      out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      nbytes: int | None = None, stream=None) -> torch.Tensor:
    """Decode an escape-coded stream into n 16-bit values (``out`` if given)."""
    if out is None:
        out = torch.empty(n, dtype=torch.bfloat16, device=stream_bytes.device)
    words = out.view(-1)
    if words.numel() != n or not words.is_contiguous() or out.element_size() != 2:
        raise ValueError("out must be a contiguous 16-bit tensor of %d elements" % n)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=stream_bytes.device)
    size = stream_bytes.numel() if nbytes is None else nbytes
    rc = wc_decompress_escape(stream_bytes.data_ptr(), size, words.data_ptr() if n else None, n,
                              block, status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress_escape")
    return out


def decompress_escape_batch(batch, status: torch.Tensor, stream=None):
    """Decode escape-coded streams (a batch from ``make_batch``), one launch per 512."""
    arr, count = batch
    rc = wc_decompress_escape_batch(arr, count, status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress_escape_batch")


def decompress_host_batch(batch, status: torch.Tensor, escape: bool = False, stream=None):
    """Decode streams held in page-locked host memory (a batch from ``make_batch``
    whose stream tensors are pinned CPU tensors) straight into device outputs."""
    arr, count = batch
    rc = wc_decompress_host_batch(arr, count, WC_FLAG_ESCAPE if escape else 0,
                                  status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress_host_batch")


def decompress_tans_batch(batch, status: torch.Tensor, stream=None):
    """Decode tANS-coded streams (a batch from ``make_batch``, block = the chunk
    size), one launch per 256."""
    arr, count = batch
    rc = wc_decompress_tans_batch(arr, count, status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress_tans_batch")


def decompress_tans(stream_bytes: torch.Tensor, n: int, chunk: int, *,
                    out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                    nbytes: int | None = None, stream=None) -> torch.Tensor:
    """Decode a tANS-coded stream into n 16-bit values (``out`` if given)."""
    if out is None:
        out = torch.empty(n, dtype=torch.bfloat16, device=stream_bytes.device)
    words = out.view(-1)
    if words.numel() != n or not words.is_contiguous() or out.element_size() != 2:
        raise ValueError("out must be a contiguous 16-bit tensor of %d elements" % n)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=stream_bytes.device)
    size = stream_bytes.numel() if nbytes is None else nbytes
    rc = wc_decompress_tans(stream_bytes.data_ptr(), size, words.data_ptr() if n else None, n,
                            chunk, status.data_ptr(), _stream_handle(stream))
    _check(rc, "wc_decompress_tans")
    return out


# ---------------------------------------------------------------------------
# 4-bit streams with group scales, their products, and the expert routing. These
# run on the tensors' device and, unless `stream` is given, on its current
# stream; results are allocated on the stream that the work runs on.
# The products have no gradient and the routing's are functions of their own, so
# activations and weights that autograd would follow are refused. (Quantizing and
# packing take parameters: rounding has no gradient to lose.)
# ---------------------------------------------------------------------------
_DTYPES = {torch.bfloat16: WC_DTYPE_BF16, torch.float16: WC_DTYPE_FP16,
           torch.float32: WC_DTYPE_FP32}


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _raw_stream = torch._C._cuda_getCurrentRawStream  # a fiftieth of current_stream()'s time
else:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _here(t: torch.Tensor, stream) -> bool:
    """Whether t's device is the current one and its current stream is meant."""
    return t.is_cuda and stream is None and t.get_device() == _current_device()


@contextlib.contextmanager
def _there(device: torch.device, stream, *tensors):
    """Make ``device`` current, and ``stream`` (if given) the one that work is
    enqueued and tensors are allocated on. The call's own ``tensors`` (None among
    them) are then marked as used there, so that a caller may let go of them as
    soon as the call returns."""
    if device.type != "cuda":
        raise ValueError("wcodec works on CUDA tensors; got one on %s" % device)
    if stream is not None and stream.device != device:
        raise ValueError("stream is on %s, not on %s" % (stream.device, device))
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)


def _no_graph(what: str):
    """For a call some of whose tensors require grad: refused where autograd would
    follow them. Results here have no graph, and the gradient would be lost without
    a word."""
    if torch.is_grad_enabled():
        raise ValueError("%s records no autograd graph: call it under torch.no_grad(), or on detached tensors"
                         % what)


def _rows(t: torch.Tensor, cols: int, what: str, device=None) -> int:
    """Check a matrix of `cols` columns whose rows are dense (they may lie
    apart); returns the elements between rows."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols:
        raise ValueError("%s must be a matrix of %d columns; got %s" % (what, cols, tuple(shape)))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (what, t.device, device))
    rows = shape[0]
    if rows == 0 or cols == 0:
        return cols
    ld, inner = t.stride()
    if (cols > 1 and inner != 1) or (rows > 1 and ld < cols):
        raise ValueError("%s must have dense rows; got strides %s" % (what, t.stride()))
    return ld if rows > 1 else cols  # the stride of a single row means nothing


def _vector(t: torch.Tensor, shape: tuple, dtype: torch.dtype, what: str, device) -> torch.Tensor:
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (what, dtype, tuple(shape), device))
    return t


def _status_ptr(status: torch.Tensor | None, device):
    if status is None:
        return None
    if status.dtype != torch.int32 or status.numel() < 1 or status.device != device:
        raise ValueError("status must be an int32 tensor on %s" % device)
    return status.data_ptr()


@dataclass
class Q4Matrix:
    """A rows x cols matrix held as a 4-bit stream: ``buffer`` is its bytes
    (uint8), or (experts, bytes) for the matrices of several experts."""
    buffer: torch.Tensor
    rows: int
    cols: int
    group: int
    zeros: bool
    scale_dtype: torch.dtype

    def flags(self) -> int:
        if self.scale_dtype == torch.bfloat16:
            return WC_Q4_ZEROS if self.zeros else 0
        if self.scale_dtype == torch.float16:
            return WC_Q4_SCALES_FP16 + (WC_Q4_ZEROS if self.zeros else 0)
        raise TypeError("scales are BF16 or FP16; got %s" % self.scale_dtype)


def _q4_buffer(m: Q4Matrix, dims: int) -> torch.Tensor:
    b = m.buffer
    if b.dtype != torch.uint8 or b.dim() != dims or not (
            b.is_contiguous() or b.shape[-1] <= 1 or b.stride(-1) == 1):
        raise ValueError("a 4-bit stream is a dense uint8 tensor of %d dimension(s); got %s %s"
                         % (dims, b.dtype, tuple(b.shape)))
    return b


@functools.lru_cache(maxsize=256)
def _q4_size(rows: int, cols: int, group: int, flags: int) -> int:
    size = wc_q4_bytes(rows, cols, group, flags) if rows >= 0 and cols >= 0 else 0
    if size == 0:
        raise WcodecError(WC_ERR_INVALID_ARG, "4-bit stream of %r x %r in groups of %r"
                          % (rows, cols, group))
    return size


def _q4_out(m: Q4Matrix, size: int, like: torch.Tensor) -> torch.Tensor:
    if m.buffer is None:
        m.buffer = like.new_empty(size, dtype=torch.uint8)
    elif m.buffer.device != like.device:
        raise ValueError("out is on %s, not on %s" % (m.buffer.device, like.device))
    return _q4_buffer(m, 1)


def quantize_q4(w: torch.Tensor, group: int = 128, *, zeros: bool = False,
                out: torch.Tensor | None = None, stream=None) -> Q4Matrix:
    """Round a BF16 or FP16 matrix to a 4-bit stream with one scale of its type
    (and with ``zeros`` a zero point) per row and ``group`` columns."""
    if w.dtype != torch.bfloat16 and w.dtype != torch.float16:
        raise TypeError("quantize_q4 takes BF16 or FP16; got %s" % w.dtype)
    if w.dim() != 2:
        raise ValueError("w must be a matrix; got shape %s" % (tuple(w.shape),))
    rows, cols = w.shape
    ld = _rows(w, cols, "w")
    m = Q4Matrix(out, rows, cols, group, zeros, w.dtype)
    flags = m.flags()
    size = _q4_size(rows, cols, group, flags)
    if not _here(w, stream):
        with _there(w.device, stream, w, out):
            return quantize_q4(w, group, zeros=zeros, out=out)
    b = _q4_out(m, size, w)
    rc = lib().wc_q4_quantize(w.data_ptr(), ld, rows, cols, group, flags, b.data_ptr(), b.numel(),
                              _raw_stream(w.get_device()))
    _check(rc, "wc_q4_quantize")
    return m


def pack_q4(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None, *,
            group: int = 128, out: torch.Tensor | None = None, stream=None) -> Q4Matrix:
    """The stream of given codes (uint8, rows x cols, 0..15), scales (BF16 or
    FP16, rows x ceil(cols / group)) and zero points (uint8, as the scales)."""
    if codes.dim() != 2:
        raise ValueError("codes must be a matrix; got shape %s" % (tuple(codes.shape),))
    rows, cols = codes.shape
    m = Q4Matrix(out, rows, cols, group, zeros is not None, scales.dtype)
    flags = m.flags()
    size = _q4_size(rows, cols, group, flags)
    shape = (rows, -(-cols // group))
    _vector(codes, (rows, cols), torch.uint8, "codes", codes.device)
    _vector(scales, shape, scales.dtype, "scales", codes.device)
    if zeros is not None:
        _vector(zeros, shape, torch.uint8, "zeros", codes.device)
    if not _here(codes, stream):
        with _there(codes.device, stream, codes, scales, zeros, out):
            return pack_q4(codes, scales, zeros, group=group, out=out)
    b = _q4_out(m, size, codes)
    rc = lib().wc_q4_pack(codes.data_ptr(), scales.data_ptr(),
                          None if zeros is None else zeros.data_ptr(), rows, cols, group, flags,
                          b.data_ptr(), b.numel(), _raw_stream(codes.get_device()))
    _check(rc, "wc_q4_pack")
    return m


def dequantize_q4(m: Q4Matrix, dtype: torch.dtype = torch.bfloat16, *,
                  out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """The weights of a 4-bit stream, rounded once to ``dtype`` (BF16, FP16 or FP32)."""
    b = _q4_buffer(m, 1)
    rows, cols = m.rows, m.cols
    ld = cols
    if out is not None:
        ld = _rows(out, cols, "out", b.device)
        dtype = out.dtype
        if out.shape[0] != rows:
            raise ValueError("out must have %d rows" % rows)
    if dtype not in _DTYPES:
        raise TypeError("dequantize_q4 gives BF16, FP16 or FP32; got %s" % dtype)
    if out is not None and out.requires_grad:
        _no_graph("dequantize_q4")
    if not _here(b, stream):
        with _there(b.device, stream, b, out, status):
            return dequantize_q4(m, dtype, out=out, status=status)
    if out is None:
        out = b.new_empty((rows, cols), dtype=dtype)
    rc = lib().wc_q4_dequantize(b.data_ptr(), b.numel(), rows, cols, m.group, m.flags(),
                                out.data_ptr(), ld, _DTYPES[dtype], _status_ptr(status, b.device),
                                _raw_stream(b.get_device()))
    _check(rc, "wc_q4_dequantize")
    return out


def _q4_product_args(m: Q4Matrix, b, x, y, out_dtype):
    """Checks shared by the two products: (tokens, ldx, ldy, flags, result type)."""
    dt = x.dtype
    if dt == torch.bfloat16:
        flags = m.flags()
    elif dt == torch.float16:
        flags = m.flags() + WC_Q4_X_FP16
    else:
        raise TypeError("activations are BF16 or FP16; got %s" % dt)
    ldx = _rows(x, m.cols, "x", b.device)
    tokens = x.shape[0]
    ldy = m.rows
    if y is not None:
        ldy = _rows(y, m.rows, "y", b.device)
        out_dtype = y.dtype
        if y.shape[0] != tokens:
            raise ValueError("y must have %d rows" % tokens)
    if out_dtype != torch.float32:
        if out_dtype != dt:
            raise TypeError("the product is FP32 or has x's type; got %s" % out_dtype)
        flags += WC_Q4_Y_16BIT
    return tokens, ldx, ldy, flags, out_dtype


def gemm_q4(m: Q4Matrix, x: torch.Tensor, *, y: torch.Tensor | None = None,
            out_dtype: torch.dtype = torch.float32, status: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """y = x @ W.T with W held as a 4-bit stream; x is (tokens, cols) BF16 or
    FP16, y (tokens, rows) in FP32 or x's type."""
    b = _q4_buffer(m, 1)
    tokens, ldx, ldy, flags, out_dtype = _q4_product_args(m, b, x, y, out_dtype)
    if x.requires_grad or (y is not None and y.requires_grad):
        _no_graph("gemm_q4")
    if not _here(b, stream):
        with _there(b.device, stream, b, x, y, status):
            return gemm_q4(m, x, y=y, out_dtype=out_dtype, status=status)
    if y is None:
        y = x.new_empty((tokens, m.rows), dtype=out_dtype)
    rc = lib().wc_q4_gemm(b.data_ptr(), b.numel(), m.rows, m.cols, m.group, flags, x.data_ptr(),
                          ldx, tokens, y.data_ptr(), ldy,
                          None if status is None else _status_ptr(status, b.device),
                          _raw_stream(b.get_device()))
    _check(rc, "wc_q4_gemm")
    return y


def gemm_q4_experts(m: Q4Matrix, x: torch.Tensor, offsets: torch.Tensor, *,
                    y: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                    status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gemm_q4 over the matrices of m.buffer's experts: rows offsets[e] ..
    offsets[e + 1] - 1 of x take matrix e (offsets int32, as moe_sort gives
    them). The streams may lie apart, each a multiple of 16 bytes from the last. Rows outside every range are left as they were in ``y``."""
    b = _q4_buffer(m, 2)
    experts, size = b.shape
    _vector(offsets, (experts + 1,), torch.int32, "offsets", b.device)
    tokens, ldx, ldy, flags, out_dtype = _q4_product_args(m, b, x, y, out_dtype)
    need = _q4_size(m.rows, m.cols, m.group, flags & (WC_Q4_ZEROS | WC_Q4_SCALES_FP16))
    if size < need:  # (the stride between streams says nothing of the last one's length)
        raise WcodecError(WC_ERR_CORRUPT_STREAM, "streams of %d bytes each; one takes %d" % (size, need))
    if x.requires_grad or (y is not None and y.requires_grad):
        _no_graph("gemm_q4_experts")
    if not _here(b, stream):
        with _there(b.device, stream, b, x, offsets, y, status):
            return gemm_q4_experts(m, x, offsets, y=y, out_dtype=out_dtype, status=status)
    if y is None:
        y = x.new_empty((tokens, m.rows), dtype=out_dtype)
    rc = lib().wc_q4_gemm_experts(b.data_ptr(), b.stride(0) if experts > 1 else need, experts,
                                  m.rows, m.cols, m.group, flags, x.data_ptr(), ldx, tokens,
                                  offsets.data_ptr(), y.data_ptr(), ldy,
                                  None if status is None else _status_ptr(status, b.device),
                                  _raw_stream(b.get_device()))
    _check(rc, "wc_q4_gemm_experts")
    return y


@dataclass
class MoePlan:
    """Where each (token, choice) slot's row lies among the rows sorted by
    expert: offsets (experts + 1), order (slot of each sorted row, -1 behind
    them; may be None), inverse ((tokens, top), -1: dropped); all int32."""
    offsets: torch.Tensor
    order: torch.Tensor | None
    inverse: torch.Tensor


def moe_sort(ids: torch.Tensor, experts: int, *, stream=None) -> MoePlan:
    """The plan that sorts (token, choice) slots by expert: ids is (tokens, top)
    int32; ids outside 0..experts-1 are dropped."""
    if ids.dim() != 2 or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 tensor of shape (tokens, top)")
    if not 1 <= experts <= WC_MOE_MAX_EXPERTS:
        raise ValueError("1 to %d experts; got %r" % (WC_MOE_MAX_EXPERTS, experts))
    if not _here(ids, stream):
        with _there(ids.device, stream, ids):
            return moe_sort(ids, experts)
    slots = ids.numel()
    offsets = ids.new_empty(experts + 1)
    order = ids.new_empty(slots)
    inverse = ids.new_empty(ids.shape)
    rc = lib().wc_moe_sort(ids.data_ptr(), slots, experts, offsets.data_ptr(), order.data_ptr(),
                           inverse.data_ptr(), _raw_stream(ids.get_device()))
    _check(rc, "wc_moe_sort")
    return MoePlan(offsets, order, inverse)


def _moe_matrix(t: torch.Tensor, cols: int, what: str, like: torch.Tensor) -> int:
    """Check a matrix of the routing operators; returns the elements between rows."""
    if t.dtype not in _DTYPES or t.dtype != like.dtype:
        raise TypeError("%s must be BF16, FP16 or FP32 and of one type; got %s" % (what, t.dtype))
    return _rows(t, cols, what, like.device)


def _moe_inverse(plan: MoePlan, device) -> torch.Tensor:
    inv = plan.inverse
    if inv.dim() != 2:
        raise ValueError("plan.inverse must be (tokens, top)")
    return _vector(inv, inv.shape, torch.int32, "plan.inverse", device)


def moe_gather(x: torch.Tensor, plan: MoePlan, *, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """The rows of x (tokens, cols) sorted by expert: (tokens * top, cols), of
    which plan.offsets[-1] are written (the others are left as they were)."""
    inv = _moe_inverse(plan, x.device)
    tokens, top = inv.shape
    cols = x.shape[-1]
    ldx = _moe_matrix(x, cols, "x", x)
    if x.shape[0] != tokens:
        raise ValueError("x must have %d rows" % tokens)
    ldo = cols if out is None else _moe_matrix(out, cols, "out", x)
    if x.requires_grad or (out is not None and out.requires_grad):
        _no_graph("moe_gather")
    if not _here(x, stream):
        with _there(x.device, stream, x, inv, out):
            return moe_gather(x, plan, out=out)
    if out is None:
        out = x.new_empty((tokens * top, cols))
    rc = lib().wc_moe_gather(x.data_ptr(), ldx, tokens, top, cols, _DTYPES[x.dtype], inv.data_ptr(),
                             out.data_ptr(), ldo, out.shape[0], _raw_stream(x.get_device()))
    _check(rc, "wc_moe_gather")
    return out


def moe_combine(rows: torch.Tensor, plan: MoePlan, weights: torch.Tensor | None, *,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * rows[plan.inverse[t, j]] (weights FP32,
    None: all 1), in the type of rows."""
    device = rows.device
    inv = _moe_inverse(plan, device)
    tokens, top = inv.shape
    cols = rows.shape[-1]
    ldr = _moe_matrix(rows, cols, "rows", rows)
    if weights is not None:
        _vector(weights, inv.shape, torch.float32, "weights", device)
    ldo = cols
    if out is not None:
        ldo = _moe_matrix(out, cols, "out", rows)
        if out.shape[0] != tokens:
            raise ValueError("out must have %d rows" % tokens)
    if rows.requires_grad or (weights is not None and weights.requires_grad) or (out is not None and out.requires_grad):
        _no_graph("moe_combine")
    if not _here(rows, stream):
        with _there(device, stream, rows, inv, weights, out):
            return moe_combine(rows, plan, weights, out=out)
    if out is None:
        out = rows.new_empty((tokens, cols))
    rc = lib().wc_moe_combine(rows.data_ptr(), ldr, rows.shape[0], tokens, top, cols,
                              _DTYPES[rows.dtype], inv.data_ptr(),
                              None if weights is None else weights.data_ptr(), out.data_ptr(), ldo,
                              _raw_stream(rows.get_device()))
    _check(rc, "wc_moe_combine")
    return out


def moe_gather_backward(drows: torch.Tensor, plan: MoePlan, *, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """The gradient of x from that of moe_gather's rows: each token's rows summed."""
    return moe_combine(drows, plan, None, out=out, stream=stream)


def moe_combine_backward(dout: torch.Tensor, rows: torch.Tensor, plan: MoePlan,
                         weights: torch.Tensor | None, *, drows: torch.Tensor | None = None,
                         stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The gradients of moe_combine's rows and weights. Rows that no slot names
    are left as they were in ``drows``."""
    device = rows.device
    inv = _moe_inverse(plan, device)
    tokens, top = inv.shape
    cols = rows.shape[-1]
    ldr = _moe_matrix(rows, cols, "rows", rows)
    ldd = _moe_matrix(dout, cols, "dout", rows)
    if dout.shape[0] != tokens:
        raise ValueError("dout must have %d rows" % tokens)
    if weights is not None:
        _vector(weights, inv.shape, torch.float32, "weights", device)
    lddr = cols
    if drows is not None:
        lddr = _moe_matrix(drows, cols, "drows", rows)
        if drows.shape[0] != rows.shape[0]:
            raise ValueError("drows must have %d rows" % rows.shape[0])
    if dout.requires_grad or rows.requires_grad or (weights is not None and weights.requires_grad) or \
            (drows is not None and drows.requires_grad):
        _no_graph("moe_combine_backward")
    if not _here(rows, stream):
        with _there(device, stream, dout, rows, inv, weights, drows):
            return moe_combine_backward(dout, rows, plan, weights, drows=drows)
    if drows is None:
        drows = rows.new_empty((rows.shape[0], cols))
    dweights = rows.new_empty((tokens, top), dtype=torch.float32)
    rc = lib().wc_moe_combine_backward(
        dout.data_ptr(), ldd, rows.data_ptr(), ldr, rows.shape[0], tokens, top, cols,
        _DTYPES[rows.dtype], inv.data_ptr(), None if weights is None else weights.data_ptr(),
        drows.data_ptr(), lddr, dweights.data_ptr(), _raw_stream(rows.get_device()))
    _check(rc, "wc_moe_combine_backward")
    return drows, dweights
