"""Thin ctypes binding of libss_sampler.so (argument marshalling only).

Every computation runs in the HIP library; this module only turns torch device
tensors into the C ABI's pointers and sizes (include/ss_sampler.h) and passes
torch's current stream. It raises if the library is missing: there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libss_sampler.so")

SS_OK = 0
SS_ERR_INVALID_ARG = -1
SS_ERR_UNSUPPORTED = -2
SS_ERR_OUT_OF_MEMORY = -3
SS_ERR_HIP = -4
SS_F32 = 0
SS_BF16 = 1
SS_F16 = 2

EXPORTED = ("ss_sampler_create", "ss_sampler_destroy", "ss_status_string",
            "ss_sampler_workspace_bytes", "ss_sampler_set_launch_events", "ss_sample",
            "ss_spec_verify", "ss_spec_verify_scatter", "ss_tree_verify", "ss_lmhead_sample",
            "ss_lmhead_sample_params", "ss_sample_noalloc", "ss_spec_verify_probs",
            "ss_lmhead_quant_logits", "ss_cache_create", "ss_cache_destroy",
            "ss_cache_workspace_bytes", "ss_cache_reserve", "ss_cache_fork", "ss_cache_commit",
            "ss_cache_commit_reserved", "ss_cache_truncate", "ss_cache_copy_pages",
            "ss_cache_create_scaled", "ss_cache_write", "ss_cache_read", "ss_cache_attend",
            "ss_rotate")
NOALLOC_MAX_BATCH = 64
NOALLOC_MAX_ENTRIES = 1 << 23


class Config(ctypes.Structure):
    _fields_ = [("max_batch", ctypes.c_int32), ("vocab_size", ctypes.c_int32),
                ("max_draft", ctypes.c_int32), ("hidden_size", ctypes.c_int32),
                ("device", ctypes.c_int32)]


class CParams(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p),
                ("repetition_penalty", ctypes.c_void_p), ("frequency_penalty", ctypes.c_void_p),
                ("presence_penalty", ctypes.c_void_p), ("history_ids", ctypes.c_void_p),
                ("history_len", ctypes.c_void_p), ("history_stride", ctypes.c_int32),
                ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_len", ctypes.c_void_p), ("bias_stride", ctypes.c_int32),
                ("grammar_mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int32),
                ("request_ids", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("seed", ctypes.c_uint64)]


class CDebug(ctypes.Structure):
    _fields_ = [("processed_logits", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p),
                ("topk_stride", ctypes.c_int32), ("kept_count", ctypes.c_void_p),
                ("probs", ctypes.c_void_p), ("path", ctypes.c_void_p)]


class CSequences(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("capacity", ctypes.c_int32), ("len", ctypes.c_void_p)]


class CacheConfig(ctypes.Structure):
    _fields_ = [("num_planes", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("piece_bytes", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("max_batch", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("device", ctypes.c_int32)]


class CBlockTables(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("rows", ctypes.c_int32), ("ref", ctypes.c_void_p), ("len", ctypes.c_void_p)]


class CacheScales(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class SamplerError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


_lib = None


def load_library(path=None):
    """Load libss_sampler.so and declare its signatures (raises if absent)."""
    global _lib
    if _lib is not None:
        return _lib
    path = LIB_PATH if path is None else path
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (__graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    lib.ss_sampler_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(vp)]
    lib.ss_sampler_create.restype = i32
    lib.ss_sampler_destroy.argtypes = [vp]
    lib.ss_sampler_destroy.restype = None
    lib.ss_status_string.argtypes = [i32]
    lib.ss_status_string.restype = ctypes.c_char_p
    lib.ss_sampler_workspace_bytes.argtypes = [vp]
    lib.ss_sampler_workspace_bytes.restype = i64
    lib.ss_sampler_set_launch_events.argtypes = [vp, ctypes.POINTER(vp), i32]
    lib.ss_sampler_set_launch_events.restype = i32
    lib.ss_sample.argtypes = [vp, vp, i32, i64, i32, ctypes.POINTER(CParams), vp,
                              ctypes.POINTER(CDebug), vp]
    lib.ss_sample.restype = i32
    lib.ss_spec_verify.argtypes = [vp, vp, i32, i64, vp, i64, vp, i32, i32,
                                   ctypes.POINTER(CParams), vp, vp, vp]
    lib.ss_spec_verify.restype = i32
    lib.ss_spec_verify_scatter.argtypes = [vp, vp, i32, i64, vp, i64, vp, i32, i32,
                                           ctypes.POINTER(CParams), vp, vp,
                                           ctypes.POINTER(CSequences), vp]
    lib.ss_spec_verify_scatter.restype = i32
    lib.ss_tree_verify.argtypes = [vp, vp, i32, i64, vp, vp, i32, i32, ctypes.POINTER(CParams),
                                   vp, vp, vp, vp]
    lib.ss_tree_verify.restype = i32
    lib.ss_lmhead_sample.argtypes = [vp, vp, vp, i32, vp, vp, vp, u64, vp, vp, vp]
    lib.ss_lmhead_sample.restype = i32
    lib.ss_lmhead_sample_params.argtypes = [vp, vp, vp, i32, ctypes.POINTER(CParams), vp, vp, vp]
    lib.ss_lmhead_sample_params.restype = i32
    lib.ss_sample_noalloc.argtypes = [vp, i32, i64, i32, i32, ctypes.POINTER(CParams), vp, vp]
    lib.ss_sample_noalloc.restype = i32
    lib.ss_spec_verify_probs.argtypes = [vp, vp, i32, i64, vp, i64, vp, vp, vp, i32, i32, vp, vp,
                                         ctypes.POINTER(CSequences), vp]
    lib.ss_spec_verify_probs.restype = i32
    lib.ss_lmhead_quant_logits.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, vp, i32, i64, vp]
    lib.ss_lmhead_quant_logits.restype = i32
    tables = ctypes.POINTER(CBlockTables)
    lib.ss_cache_create.argtypes = [ctypes.POINTER(CacheConfig), ctypes.POINTER(vp),
                                    ctypes.POINTER(vp)]
    lib.ss_cache_create.restype = i32
    lib.ss_cache_destroy.argtypes = [vp]
    lib.ss_cache_destroy.restype = None
    lib.ss_cache_workspace_bytes.argtypes = [vp]
    lib.ss_cache_workspace_bytes.restype = i64
    lib.ss_cache_reserve.argtypes = [vp, tables, vp, vp, i32, vp, vp]
    lib.ss_cache_reserve.restype = i32
    lib.ss_cache_fork.argtypes = [vp, tables, vp, vp, i32, vp, vp]
    lib.ss_cache_fork.restype = i32
    lib.ss_cache_commit.argtypes = [vp, tables, vp, vp, i64, i32, vp, i32, i32, vp, vp]
    lib.ss_cache_commit.restype = i32
    lib.ss_cache_commit_reserved.argtypes = [vp, tables, vp, vp, i64, i32, vp, i32, i32, vp, vp, vp]
    lib.ss_cache_commit_reserved.restype = i32
    lib.ss_cache_truncate.argtypes = [vp, tables, vp, vp, i32, vp]
    lib.ss_cache_truncate.restype = i32
    lib.ss_cache_copy_pages.argtypes = [vp, vp, vp, vp, i32, vp, vp]
    lib.ss_cache_copy_pages.restype = i32
    lib.ss_cache_create_scaled.argtypes = [ctypes.POINTER(CacheConfig), ctypes.POINTER(vp),
                                           ctypes.POINTER(vp), ctypes.POINTER(CacheScales),
                                           ctypes.POINTER(vp)]
    lib.ss_cache_create_scaled.restype = i32
    # structures come as bytes: see _pack_heads
    lib.ss_rotate.argtypes = [i32, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp, i32, vp]
    lib.ss_rotate.restype = i32
    lib.ss_cache_write.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp]
    lib.ss_cache_write.restype = i32
    lib.ss_cache_read.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.ss_cache_read.restype = i32
    lib.ss_cache_attend.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, i32, ctypes.c_float, vp, vp]
    lib.ss_cache_attend.restype = i32
    _lib = lib
    return lib


def _check(fn, st):
    if st != SS_OK:
        raise SamplerError(fn, st, load_library().ss_status_string(st).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# torch's current stream as an address, without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream_on(stream, device):
    """The given stream, or the current one of a device that need not be current."""
    return _raw_stream(device) if stream is None else stream.cuda_stream


# torch's allocation of a contiguous array without the argument parser around it
# (0.7 us instead of 1.3 to 1.5); it allocates on the current device
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None),
                         "_empty_strided_cuda", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _empty_rows(n, m, like, dtype=torch.int32, stream=None):
    """An uninitialised [n, m] array (m None: [n]) on the device of `like`, for a call
    on `stream` (None: the current one)."""
    return _empty((n,) if m is None else (n, m), like, dtype, stream)


def _empty(shape, like, dtype, stream=None):
    """An uninitialised contiguous array on the device of `like`. What another stream
    writes is allocated there, so that its memory is never one that earlier work of
    the current stream still uses, and returns to that stream once neither is at
    work on it."""
    if stream is not None and stream.cuda_stream != _raw_stream(like.get_device()):
        device = like.device
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
        with torch.cuda.stream(stream):
            out = like.new_empty(shape, dtype=dtype)
        out.record_stream(torch.cuda.current_stream(device))
        return out
    if _empty_strided is not None and _current_device is not None and \
            _current_device() == like.get_device():
        if len(shape) == 1:
            return _empty_strided(shape, (1,), dtype)
        if len(shape) == 2:
            return _empty_strided(shape, (shape[1], 1), dtype)
        if len(shape) == 3:
            _, h, d = shape
            return _empty_strided(shape, (h * d, d, 1), dtype)
        if len(shape) == 4:
            _, n, h, d = shape
            return _empty_strided(shape, (n * h * d, h * d, d, 1), dtype)
    return like.new_empty(shape, dtype=dtype)


def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def _check_dev(t, name, dtypes, device):
    _require(isinstance(t, torch.Tensor), f"{name} must be a tensor")
    _require(t.is_cuda and t.device.index == device, f"{name} must live on cuda:{device}")
    _require(t.dtype in dtypes, f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def _check_vec(t, name, n, dtype, device):
    """A per-row array: at least n entries, unit stride (the ABI takes a bare pointer)."""
    if t is None:
        return
    _check_dev(t, name, (dtype,), device)
    _require(t.dim() == 1 and t.shape[0] >= n and (t.shape[0] <= 1 or t.stride(0) == 1),
             f"{name} must be a 1-D array of >= {n} entries with unit stride")


def _check_rows(t, name, n, dtypes, device):
    """A [rows, cols] matrix with unit column stride: the ABI takes its row stride."""
    _check_dev(t, name, dtypes, device)
    _require(t.dim() == 2 and t.shape[0] >= n, f"{name} must be 2-D with >= {n} rows")
    _require(t.shape[1] <= 1 or t.stride(1) == 1, f"{name} must have unit stride along its last dim")


_PROB_DTYPES = {torch.float32: SS_F32, torch.bfloat16: SS_BF16, torch.float16: SS_F16}


def _check_block(t, name, shape, dtype, device):
    """A contiguous array of exactly this shape; returns its address. A call that
    takes microseconds is checked by what costs least, the message formed on
    failure only."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.get_device() == device and t.is_contiguous()):
        _check_dev(t, name, (dtype,), device)
        raise ValueError(f"{name} must be a contiguous {list(shape)} array of {dtype}")
    return t.data_ptr()


def _check_array(t, name, n, device, dtype=torch.int32):
    """A 1-D array of at least n entries with unit stride; returns its address
    (None for None)."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and
            t.dim() == 1 and t.shape[0] >= n and t.is_contiguous()):
        _check_vec(t, name, n, dtype, device)  # a longer strided array of one entry passes
    return t.data_ptr()


def _check_rank3(t, name, shape, dtype, device):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and
            t.shape == shape):
        _check_dev(t, name, (dtype,), device)
        raise ValueError(f"{name} must be {list(shape)}")


_HALF_DTYPES = {torch.bfloat16: SS_BF16, torch.float16: SS_F16}

# ss_heads, ss_block_tables, ss_cache_step and ss_rotary as bytes, which ctypes passes by
# their address: a structure of its own takes 1 us a call, these 0.3
_pack_heads = struct.Struct("@P3q").pack
_pack_tables = struct.Struct("@PqixxxxPP").pack
_pack_step = struct.Struct("@iiPPPP").pack
_pack_rotary = struct.Struct("@Piid").pack


def _heads(t, name, shape, dtype, device):
    """A [B, N, heads, dim] array of 16-bit floats as the ABI takes it; shape None: any.
    The last dimension has unit stride, the others any. [T, heads, dim] is a batch of one."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and
            (shape is None or t.shape == shape)):
        _check_dev(t, name, (dtype,), device)
        raise ValueError(f"{name} must be {'[B, N, heads, dim]' if shape is None else list(shape)}")
    strides = t.stride()
    if strides[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dim")
    if t.is_contiguous():  # a dimension of one entry may have any stride: it is not stepped
        _, N, H, D = t.shape if len(strides) == 4 else (1, *t.shape)
        return _pack_heads(t.data_ptr(), N * H * D, H * D, D)
    b, n, h, _ = strides if len(strides) == 4 else (0, *strides)
    B, N, H, _ = t.shape if len(strides) == 4 else (1, *t.shape)
    return _pack_heads(t.data_ptr(), b if B > 1 else 0, n if N > 1 else 0, h if H > 1 else 0)


def _new_heads(shape, like, dtype, stream):
    """A new [..., N, heads, dim] array, and as the ABI takes it."""
    out = _empty(tuple(shape), like, dtype, stream)
    n, h, d = shape[-3:]
    h *= d
    return out, _pack_heads(out.data_ptr(), n * h, h, d)


def _out_heads(out, name, shape, like, dtype, stream):
    """The given output, of this shape and type, or a new one (None), and as the ABI takes it."""
    if out is None:
        return _new_heads(shape, like, dtype, stream)
    words = _heads(out, name, shape, dtype, like.get_device())
    _check_out_heads(out, name)
    return out, words


def _check_out_heads(t, name):
    """An output whose entries lie apart: strides, sorted, each span what lies within."""
    if t.is_contiguous():
        return
    span = t.shape[-1]
    for stride, n in sorted(zip(t.stride()[:-1], t.shape[:-1])):
        if n > 1:
            _require(stride >= span, f"{name} must not hold an entry twice")
            span += stride * (n - 1)


def _row_stride(t, name):
    """The one stride between the rows of a [B, R, V] array (row b * R + r)."""
    B, R, V = t.shape
    if t.is_contiguous():
        return V
    if V > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along V")
    stride = t.stride(1) if R > 1 else t.stride(0) if B > 1 else V
    if not ((B <= 1 or R == 0 or t.stride(0) == R * stride) and stride >= V):
        raise ValueError(f"{name} rows must be evenly spaced and must not overlap")
    return stride


@dataclass
class SamplingParams:
    """Per-request parameters as device tensors (None disables a feature)."""
    temperature: torch.Tensor
    top_k: torch.Tensor | None = None
    top_p: torch.Tensor | None = None
    min_p: torch.Tensor | None = None
    repetition_penalty: torch.Tensor | None = None
    frequency_penalty: torch.Tensor | None = None
    presence_penalty: torch.Tensor | None = None
    history_ids: torch.Tensor | None = None   # [B, H] int32
    history_len: torch.Tensor | None = None   # [B] int32
    bias_ids: torch.Tensor | None = None      # [B, NB] int32
    bias_values: torch.Tensor | None = None   # [B, NB] float32
    bias_len: torch.Tensor | None = None      # [B] int32
    grammar_mask: torch.Tensor | None = None  # [B, W] (or [B, G+1, W]) int32 view of uint32 words
    request_ids: torch.Tensor | None = None
    positions: torch.Tensor | None = None
    seed: int = 0

    def validate(self, B, V, device, mask_rows=None):
        """Check every tensor against what the C ABI can express for B rows of a
        V-entry vocabulary; mask_rows = G + 1 for a per-position [B, G+1, W]
        mask (verification). Raises ValueError; returns the mask row stride."""
        _require(self.temperature is not None, "temperature is required")
        _check_vec(self.temperature, "temperature", B, torch.float32, device)
        _check_vec(self.top_k, "top_k", B, torch.int32, device)
        for name in ("top_p", "min_p", "repetition_penalty", "frequency_penalty",
                     "presence_penalty"):
            _check_vec(getattr(self, name), name, B, torch.float32, device)
        _check_vec(self.request_ids, "request_ids", B, torch.int32, device)
        _check_vec(self.positions, "positions", B, torch.int32, device)
        if self.history_len is not None or self.history_ids is not None:
            _require(self.history_len is not None and self.history_ids is not None,
                     "history_ids and history_len go together")
            _check_rows(self.history_ids, "history_ids", B, (torch.int32,), device)
            _check_vec(self.history_len, "history_len", B, torch.int32, device)
        if self.bias_len is not None or self.bias_ids is not None or self.bias_values is not None:
            _require(self.bias_len is not None and self.bias_ids is not None and
                     self.bias_values is not None, "bias_ids, bias_values and bias_len go together")
            _check_rows(self.bias_ids, "bias_ids", B, (torch.int32,), device)
            _check_rows(self.bias_values, "bias_values", B, (torch.float32,), device)
            _require(self.bias_values.shape[1] >= self.bias_ids.shape[1] and
                     self.bias_values.stride(0) == self.bias_ids.stride(0),
                     "bias_values must share bias_ids' row stride (one stride in the ABI)")
            _check_vec(self.bias_len, "bias_len", B, torch.int32, device)
        mask_stride = 0
        if self.grammar_mask is not None:
            m = self.grammar_mask
            _check_dev(m, "grammar_mask", (torch.int32,), device)
            words = (V + 31) // 32
            _require(m.shape[-1] >= words and (m.shape[-1] <= 1 or m.stride(-1) == 1),
                     f"grammar_mask needs >= {words} unit-stride words per row")
            if mask_rows is None:
                _require(m.dim() == 2 and m.shape[0] >= B, "grammar_mask must be [B, words]")
                mask_stride = m.stride(0)
            else:
                _require(m.dim() == 3 and m.shape[0] >= B and m.shape[1] == mask_rows and
                         (B <= 1 or m.stride(0) == mask_rows * m.stride(1)),
                         "a verification grammar_mask must be [B, G+1, words] with rows "
                         "evenly spaced")
                mask_stride = m.stride(1)
        return mask_stride

    def to_c(self, mask_stride=None):
        c = CParams()
        c.temperature = _ptr(self.temperature)
        c.top_k = _ptr(self.top_k)
        c.top_p = _ptr(self.top_p)
        c.min_p = _ptr(self.min_p)
        c.repetition_penalty = _ptr(self.repetition_penalty)
        c.frequency_penalty = _ptr(self.frequency_penalty)
        c.presence_penalty = _ptr(self.presence_penalty)
        c.history_ids = _ptr(self.history_ids)
        c.history_len = _ptr(self.history_len)
        c.history_stride = 0 if self.history_ids is None else int(self.history_ids.stride(0))
        c.bias_ids = _ptr(self.bias_ids)
        c.bias_values = _ptr(self.bias_values)
        c.bias_len = _ptr(self.bias_len)
        c.bias_stride = 0 if self.bias_ids is None else int(self.bias_ids.stride(0))
        c.grammar_mask = _ptr(self.grammar_mask)
        if mask_stride is None:
            mask_stride = 0 if self.grammar_mask is None else int(self.grammar_mask.stride(-2))
        c.mask_stride = int(mask_stride)
        c.request_ids = _ptr(self.request_ids)
        c.positions = _ptr(self.positions)
        c.seed = int(self.seed) & 0xFFFFFFFFFFFFFFFF
        return c


@dataclass
class Debug:
    """Optional debug outputs of sample() (device tensors, None = not wanted)."""
    processed_logits: torch.Tensor | None = None
    topk_ids: torch.Tensor | None = None
    kept_count: torch.Tensor | None = None
    probs: torch.Tensor | None = None
    path: torch.Tensor | None = None

    @staticmethod
    def full(B, V, device, topk_stride=1024):
        return Debug(torch.empty(B, V, dtype=torch.float32, device=device),
                     torch.empty(B, topk_stride, dtype=torch.int32, device=device),
                     torch.empty(B, dtype=torch.int32, device=device),
                     torch.empty(B, V, dtype=torch.float32, device=device),
                     torch.empty(B, dtype=torch.int32, device=device))

    def to_c(self):
        d = CDebug()
        d.processed_logits = _ptr(self.processed_logits)
        d.topk_ids = _ptr(self.topk_ids)
        d.topk_stride = 0 if self.topk_ids is None else int(self.topk_ids.shape[-1])
        d.kept_count = _ptr(self.kept_count)
        d.probs = _ptr(self.probs)
        d.path = _ptr(self.path)
        return d


class Sampler:
    """Owns one ss_sampler handle (and its device workspace)."""

    def __init__(self, max_batch, vocab_size, max_draft=0, hidden_size=0, device=0):
        self.lib = load_library()
        cfg = Config(max_batch, vocab_size, max_draft, hidden_size, device)
        h = ctypes.c_void_p()
        _check("ss_sampler_create", self.lib.ss_sampler_create(ctypes.byref(cfg), ctypes.byref(h)))
        self.handle = h
        self.vocab_size = vocab_size
        self.hidden_size = hidden_size
        self.max_draft = max_draft
        self.device = device

    def close(self):
        if getattr(self, "handle", None):
            self.lib.ss_sampler_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()

    def workspace_bytes(self):
        return int(self.lib.ss_sampler_workspace_bytes(self.handle))

    def set_launch_events(self, events):
        """Bracket kernel k of the following calls with events[2k] / events[2k+1]
        (torch.cuda.Event objects; None clears). Each event must have been
        recorded once so that its HIP event exists."""
        if not events:
            _check("ss_sampler_set_launch_events",
                   self.lib.ss_sampler_set_launch_events(self.handle, None, 0))
            return
        arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
        _check("ss_sampler_set_launch_events",
               self.lib.ss_sampler_set_launch_events(self.handle, arr, len(events)))

    @staticmethod
    def _dtype(t):
        if t.dtype == torch.float32:
            return SS_F32
        if t.dtype == torch.bfloat16:
            return SS_BF16
        raise TypeError(f"unsupported logits dtype {t.dtype}")

    def sample(self, logits, params: SamplingParams, out=None, debug: Debug | None = None,
               stream=None):
        _check_rows(logits, "logits", 0, (torch.float32, torch.bfloat16), self.device)
        B, V = logits.shape
        _require(V == self.vocab_size, f"logits have {V} columns, the sampler {self.vocab_size}")
        if out is None:
            out = _empty_rows(B, None, logits, stream=stream)
        _check_vec(out, "out", B, torch.int32, self.device)
        if debug is not None:
            for name, cols in (("processed_logits", V), ("probs", V)):
                t = getattr(debug, name)
                if t is not None:
                    _check_rows(t, f"debug.{name}", B, (torch.float32,), self.device)
                    _require(t.shape[1] == V and (B <= 1 or t.stride(0) == V),
                             f"debug.{name} must be a contiguous [B, V] array")
            if debug.topk_ids is not None:
                _check_rows(debug.topk_ids, "debug.topk_ids", B, (torch.int32,), self.device)
                _require(B <= 1 or debug.topk_ids.stride(0) == debug.topk_ids.shape[1],
                         "debug.topk_ids must be contiguous")
            _check_vec(debug.kept_count, "debug.kept_count", B, torch.int32, self.device)
            _check_vec(debug.path, "debug.path", B, torch.int32, self.device)
        cp = params.to_c(params.validate(B, V, self.device))
        cd = debug.to_c() if debug is not None else None
        st = self.lib.ss_sample(self.handle, _ptr(logits), self._dtype(logits),
                                int(logits.stride(0)), B, ctypes.byref(cp), _ptr(out),
                                ctypes.byref(cd) if cd is not None else None, _stream(stream))
        _check("ss_sample", st)
        return out

    def spec_verify(self, target_logits, draft_probs, draft_tokens, params: SamplingParams,
                    out_tokens=None, out_num_accepted=None, stream=None, seq_tokens=None,
                    seq_len=None):
        """draft_probs None: a greedy draft (q one-hot at each draft token).
        seq_tokens [B, capacity] / seq_len [B] int32: append the emitted tokens
        to these per-request sequences on the device and advance seq_len
        (params.positions may be seq_len itself)."""
        _check_dev(target_logits, "target_logits", (torch.float32, torch.bfloat16), self.device)
        _require(target_logits.dim() == 3, "target_logits must be [B, G+1, V]")
        B, G1, V = target_logits.shape
        G = G1 - 1
        _require(V == self.vocab_size, f"target_logits have {V} columns, the sampler {self.vocab_size}")
        # the ABI addresses row b * (G + 1) + j at one row stride
        _require(target_logits.stride(2) == 1 and
                 (B <= 1 or target_logits.stride(0) == G1 * target_logits.stride(1)),
                 "target_logits rows must be evenly spaced with unit stride along V")
        if draft_probs is not None:
            _check_dev(draft_probs, "draft_probs", (torch.float32,), self.device)
            _require(draft_probs.dim() == 3 and tuple(draft_probs.shape) == (B, G, V) and
                     draft_probs.stride(2) == 1 and
                     (B <= 1 or draft_probs.stride(0) == G * draft_probs.stride(1)),
                     "draft_probs must be [B, G, V] with evenly spaced rows and unit stride "
                     "along V")
        _check_dev(draft_tokens, "draft_tokens", (torch.int32,), self.device)
        _require(tuple(draft_tokens.shape) == (B, G) and draft_tokens.is_contiguous(),
                 "draft_tokens must be a contiguous [B, G] int32 array")
        if out_tokens is None:
            out_tokens = _empty_rows(B, G1, target_logits, stream=stream)
        if out_num_accepted is None:
            out_num_accepted = _empty_rows(B, None, target_logits, stream=stream)
        _check_dev(out_tokens, "out_tokens", (torch.int32,), self.device)
        _require(tuple(out_tokens.shape) == (B, G1) and out_tokens.is_contiguous(),
                 "out_tokens must be a contiguous [B, G+1] int32 array")
        _check_vec(out_num_accepted, "out_num_accepted", B, torch.int32, self.device)
        cp = params.to_c(params.validate(B, V, self.device, mask_rows=G1))
        seq = None
        if seq_tokens is not None or seq_len is not None:
            _require(seq_tokens is not None and seq_len is not None,
                     "seq_tokens and seq_len go together")
            _check_rows(seq_tokens, "seq_tokens", B, (torch.int32,), self.device)
            _check_vec(seq_len, "seq_len", B, torch.int32, self.device)
            seq = CSequences(_ptr(seq_tokens), int(seq_tokens.stride(0)) if B > 1 else
                             int(seq_tokens.shape[1]), int(seq_tokens.shape[1]), _ptr(seq_len))
        dstride = 0 if draft_probs is None else int(draft_probs.stride(1))
        st = self.lib.ss_spec_verify_scatter(
            self.handle, _ptr(target_logits), self._dtype(target_logits),
            int(target_logits.stride(1)), _ptr(draft_probs), dstride, _ptr(draft_tokens), B, G,
            ctypes.byref(cp), _ptr(out_tokens), _ptr(out_num_accepted),
            ctypes.byref(seq) if seq is not None else None, _stream(stream))
        _check("ss_spec_verify_scatter", st)
        return out_tokens, out_num_accepted

    def tree_verify(self, target_logits, parents, tokens, params: SamplingParams, out_tokens=None,
                    out_nodes=None, out_num_accepted=None, stream=None):
        """Verify one draft tree per request: target_logits [B, N, V] (row n after
        the root path to node n), parents / tokens [B, N] int32. Returns
        (tokens [B, N], nodes [B, N], num_accepted [B])."""
        _check_dev(target_logits, "target_logits", (torch.float32, torch.bfloat16), self.device)
        _require(target_logits.dim() == 3, "target_logits must be [B, N, V]")
        B, N, V = target_logits.shape
        _require(V == self.vocab_size, f"target_logits have {V} columns, the sampler {self.vocab_size}")
        _require(target_logits.stride(2) == 1 and
                 (B <= 1 or target_logits.stride(0) == N * target_logits.stride(1)),
                 "target_logits rows must be evenly spaced with unit stride along V")
        for name, t in (("parents", parents), ("tokens", tokens)):
            _check_dev(t, name, (torch.int32,), self.device)
            _require(tuple(t.shape) == (B, N) and t.is_contiguous(),
                     f"{name} must be a contiguous [B, N] int32 array")
        if out_tokens is None:
            out_tokens = _empty_rows(B, N, target_logits, stream=stream)
        if out_nodes is None:
            out_nodes = _empty_rows(B, N, target_logits, stream=stream)
        if out_num_accepted is None:
            out_num_accepted = _empty_rows(B, None, target_logits, stream=stream)
        for name, t in (("out_tokens", out_tokens), ("out_nodes", out_nodes)):
            _check_dev(t, name, (torch.int32,), self.device)
            _require(tuple(t.shape) == (B, N) and t.is_contiguous(),
                     f"{name} must be a contiguous [B, N] int32 array")
        _check_vec(out_num_accepted, "out_num_accepted", B, torch.int32, self.device)
        cp = params.to_c(params.validate(B, V, self.device, mask_rows=N))
        st = self.lib.ss_tree_verify(self.handle, _ptr(target_logits), self._dtype(target_logits),
                                     int(target_logits.stride(1)), _ptr(parents), _ptr(tokens), B,
                                     N, ctypes.byref(cp), _ptr(out_tokens), _ptr(out_nodes),
                                     _ptr(out_num_accepted), _stream(stream))
        _check("ss_tree_verify", st)
        return out_tokens, out_nodes, out_num_accepted

    def lmhead_sample_params(self, hidden, weight, params: SamplingParams, out=None, path=None,
                             stream=None):
        """LM-head GEMM with the per-request pipeline (penalties, bias, mask,
        temperature, filters) before Gumbel-max sampling. path: optional [B]
        int32 that receives how each row was decided."""
        _check_dev(hidden, "hidden", (torch.bfloat16, torch.int16), self.device)
        _check_dev(weight, "weight", (torch.bfloat16, torch.int16), self.device)
        _require(hidden.dim() == 2 and hidden.is_contiguous(), "hidden must be a contiguous [B, K] array")
        B, K = hidden.shape
        _require(K == self.hidden_size, f"hidden has K = {K}, the sampler {self.hidden_size}")
        _require(tuple(weight.shape) == (self.vocab_size, K) and weight.is_contiguous(),
                 f"weight must be a contiguous [{self.vocab_size}, {K}] array")
        if out is None:
            out = _empty_rows(B, None, hidden, stream=stream)
        _check_vec(out, "out", B, torch.int32, self.device)
        _check_vec(path, "path", B, torch.int32, self.device)
        cp = params.to_c(params.validate(B, self.vocab_size, self.device))
        st = self.lib.ss_lmhead_sample_params(self.handle, _ptr(hidden), _ptr(weight), B,
                                              ctypes.byref(cp), _ptr(out), _ptr(path),
                                              _stream(stream))
        _check("ss_lmhead_sample_params", st)
        return out

    def lmhead_sample(self, hidden, weight, temperature, request_ids=None, positions=None,
                      seed=0, out=None, debug_logits=None, stream=None):
        _check_dev(hidden, "hidden", (torch.bfloat16, torch.int16), self.device)
        _check_dev(weight, "weight", (torch.bfloat16, torch.int16), self.device)
        _require(hidden.dim() == 2 and hidden.is_contiguous(), "hidden must be a contiguous [B, K] array")
        B, K = hidden.shape
        _require(K == self.hidden_size, f"hidden has K = {K}, the sampler {self.hidden_size}")
        _require(tuple(weight.shape) == (self.vocab_size, K) and weight.is_contiguous(),
                 f"weight must be a contiguous [{self.vocab_size}, {K}] array")
        _check_vec(temperature, "temperature", B, torch.float32, self.device)
        _check_vec(request_ids, "request_ids", B, torch.int32, self.device)
        _check_vec(positions, "positions", B, torch.int32, self.device)
        if out is None:
            out = _empty_rows(B, None, hidden, stream=stream)
        _check_vec(out, "out", B, torch.int32, self.device)
        if debug_logits is not None:
            _check_dev(debug_logits, "debug_logits", (torch.float32,), self.device)
            _require(tuple(debug_logits.shape) == (B, self.vocab_size) and debug_logits.is_contiguous(),
                     "debug_logits must be a contiguous [B, V] float32 array")
        st = self.lib.ss_lmhead_sample(self.handle, _ptr(hidden), _ptr(weight), B,
                                       _ptr(temperature), _ptr(request_ids), _ptr(positions),
                                       int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(out),
                                       _ptr(debug_logits), _stream(stream))
        _check("ss_lmhead_sample", st)
        return out


    def spec_verify_probs(self, target_probs, draft_probs, draft_tokens, uniforms, draft_len=None,
                          out_tokens=None, out_num_accepted=None, stream=None, seq_tokens=None,
                          seq_len=None):
        """Verify drafts against probability rows target_probs [B, G+1, V] (float32,
        bfloat16 or float16) with the caller's uniforms [B, G+1] float32 in
        [0, 1). draft_probs [B, G, V] of the same dtype, or None for greedy
        drafts; draft_len [B] int32: drafts of each request (None: G).
        seq_tokens / seq_len as in spec_verify. Returns (tokens [B, G+1],
        num_accepted [B])."""
        dev = self.device
        dtype = getattr(target_probs, "dtype", None)
        code = _PROB_DTYPES.get(dtype)
        if code is None or target_probs.get_device() != dev:
            _check_dev(target_probs, "target_probs", tuple(_PROB_DTYPES), dev)
        shape = target_probs.shape
        if len(shape) != 3 or shape[1] < 1:
            raise ValueError("target_probs must be [B, G+1, V]")
        B, G1, V = shape
        G = G1 - 1
        if V != self.vocab_size:
            raise ValueError(f"target_probs have {V} columns, the sampler {self.vocab_size}")
        tstride = V if target_probs.is_contiguous() else _row_stride(target_probs, "target_probs")
        dptr, dstride = None, 0
        if draft_probs is not None:
            _check_rank3(draft_probs, "draft_probs", (B, G, V), dtype, dev)
            dstride = V if draft_probs.is_contiguous() else _row_stride(draft_probs, "draft_probs")
            dptr = draft_probs.data_ptr()
        tokens = _check_block(draft_tokens, "draft_tokens", (B, G), torch.int32, dev)
        u = _check_block(uniforms, "uniforms", (B, G1), torch.float32, dev)
        n = _check_array(draft_len, "draft_len", B, dev)
        if out_tokens is None:
            out_tokens = _empty_rows(B, G1, uniforms, stream=stream)
        else:
            _check_block(out_tokens, "out_tokens", (B, G1), torch.int32, dev)
        if out_num_accepted is None:
            out_num_accepted = _empty_rows(B, None, uniforms, stream=stream)
        else:
            _check_array(out_num_accepted, "out_num_accepted", B, dev)
        seq = None
        if seq_tokens is not None or seq_len is not None:
            _require(seq_tokens is not None and seq_len is not None,
                     "seq_tokens and seq_len go together")
            _check_rows(seq_tokens, "seq_tokens", B, (torch.int32,), dev)
            _check_vec(seq_len, "seq_len", B, torch.int32, dev)
            _require(B <= 1 or seq_tokens.stride(0) >= seq_tokens.shape[1],
                     "seq_tokens rows must not overlap")
            seq = CSequences(_ptr(seq_tokens), int(seq_tokens.stride(0)) if B > 1 else
                             int(seq_tokens.shape[1]), int(seq_tokens.shape[1]), _ptr(seq_len))
        st = self.lib.ss_spec_verify_probs(
            self.handle, target_probs.data_ptr(), code, tstride, dptr, dstride, tokens, n, u, B, G,
            out_tokens.data_ptr(), out_num_accepted.data_ptr(),
            ctypes.byref(seq) if seq is not None else None, _stream_on(stream, dev))
        if st != SS_OK:
            _check("ss_spec_verify_probs", st)
        return out_tokens, out_num_accepted

    def lmhead_quant_logits(self, hidden, qweight, scales, group, zeros=None, out=None,
                            out_dtype=torch.float32, stream=None):
        """LM-head logits [B, V] of hidden [B, K] bfloat16 and 4-bit weights: qweight
        [V, K/2] uint8 (even k in the low nibble), scales [V, ceil(K/group)]
        float16 or bfloat16, zeros [V, ceil(groups/2)] uint8 nibbles (None: 8).
        out: [B, V] float32 or bfloat16 with unit column stride, else one of
        out_dtype is made."""
        dev, V, K = self.device, self.vocab_size, self.hidden_size
        if not (isinstance(hidden, torch.Tensor) and hidden.dtype is torch.bfloat16 and
                hidden.get_device() == dev):
            _check_dev(hidden, "hidden", (torch.bfloat16, torch.int16), dev)
        shape = hidden.shape
        if len(shape) != 2 or not hidden.is_contiguous():
            raise ValueError("hidden must be a contiguous [B, K] array")
        B = shape[0]
        if shape[1] != K:
            raise ValueError(f"hidden has K = {shape[1]}, the sampler {K}")
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        groups = -(-K // group)
        q = _check_block(qweight, "qweight", (V, K // 2), torch.uint8, dev)
        half = getattr(scales, "dtype", None) is torch.float16
        s = _check_block(scales, "scales", (V, groups), torch.float16 if half else torch.bfloat16, dev)
        z = None
        if zeros is not None:
            z = _check_block(zeros, "zeros", (V, (groups + 1) // 2), torch.uint8, dev)
        if out is None:
            if out_dtype is not torch.float32 and out_dtype is not torch.bfloat16:
                raise ValueError("out_dtype must be float32 or bfloat16")
            out = _empty_rows(B, V, hidden, out_dtype, stream)
            stride = V
        else:
            _check_rows(out, "out", B, (torch.float32, torch.bfloat16), dev)
            stride = out.stride(0) if B > 1 else V
            if out.shape != (B, V) or stride < V:
                raise ValueError("out must be [B, V] with rows that do not overlap")
        st = self.lib.ss_lmhead_quant_logits(
            self.handle, hidden.data_ptr(), q, s, SS_F16 if half else SS_BF16, z, group, B,
            out.data_ptr(), SS_BF16 if out.dtype is torch.bfloat16 else SS_F32, stride,
            _stream_on(stream, dev))
        if st != SS_OK:
            _check("ss_lmhead_quant_logits", st)
        return out


def sample_noalloc(logits, params: SamplingParams, out=None, stream=None):
    """ss_sample without a handle: the library's static per-GPU scratch serves
    as workspace, so the call allocates nothing when `out` is given (B rows of
    at most 64, B * V at most 2^23). Calls that overlap on one GPU race."""
    _require(isinstance(logits, torch.Tensor) and logits.is_cuda, "logits must be a device tensor")
    dev = logits.device.index
    _check_rows(logits, "logits", 0, (torch.float32, torch.bfloat16), dev)
    B, V = logits.shape
    if out is None:
        out = _empty_rows(B, None, logits, stream=stream)
    _check_vec(out, "out", B, torch.int32, dev)
    cp = params.to_c(params.validate(B, V, dev))
    with torch.cuda.device(dev):
        st = load_library().ss_sample_noalloc(_ptr(logits), Sampler._dtype(logits),
                                              int(logits.stride(0)), B, V, ctypes.byref(cp),
                                              _ptr(out), _stream(stream))
    _check("ss_sample_noalloc", st)
    return out
