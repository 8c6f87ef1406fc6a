"""ctypes binding of libspecverify.so (argument marshalling only).

Every step of the verify path runs in the library's CUDA kernels; this module
only turns torch tensors into device pointers and sizes, and the current torch
stream into a cudaStream_t.  There is no fallback: if the library is missing
or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libspecverify.so")

SPEC_OK = 0
SPEC_ERR_ARG = -1
SPEC_ERR_ALIGN = -2
SPEC_ERR_WORKSPACE = -3
SPEC_ERR_UNSUPPORTED = -4
SPEC_ERR_CUDA = -5
SPEC_KV_BF16 = 0
SPEC_KV_FP8_E4M3 = 1
SPEC_FLAG_CHECKED = 1
SPEC_STATUS_BAD_PAGE = 1
SPEC_STATUS_TIMEOUT = 2
SPEC_STATUS_NO_SLOT = 4
SPEC_STATUS_BAD_GROUPS = 8
WIDTH_POLICIES = {"fixed": 0, "ewma": 1, "doubling": 2}

EXPORTED = (
    "spec_verify_workspace_size", "spec_verify_attention",
    "spec_verify_status", "spec_accept_workspace_size", "spec_greedy_accept",
    "spec_last_error", "spec_version", "spec_verify_attention_noalloc",
    "spec_kv_append", "spec_greedy_accept_commit", "spec_prepare_next_block",
    "spec_stochastic_workspace_size", "spec_stochastic_accept",
    "spec_select_workspace_size", "spec_dflash2_select",
    "spec_verify_set_wait_limit", "spec_rope_append",
    "spec_verify_attention_shared", "spec_verify_shared_workspace_size",
    "spec_sample", "spec_norm_rope_append", "spec_chunk_attention",
    "spec_chunk_workspace_size", "spec_logprobs",
)
SELECT_MODES = {"greedy": 0, "map": 1}
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024
LOGPROB_MAX_TOP = 32


class SpecError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"spec_verify error {code}: {msg}")
        self.code = code


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("q_lens", ctypes.c_void_p)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("q_lens", ctypes.c_void_p),
                ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32),
                ("attn_factor", ctypes.c_float),
                ("q_strides", ctypes.c_int64 * 2),
                ("k_strides", ctypes.c_int64 * 2),
                ("v_strides", ctypes.c_int64 * 2)]


# The same struct as bytes: a ctypes structure with arrays takes four times as
# long to fill.
_ROPE_DESC = struct.Struct("@9iIP2if6q")
assert _ROPE_DESC.size == ctypes.sizeof(RopeDesc)


class NormDesc(ctypes.Structure):
    _fields_ = [("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


_NORM_DESC = struct.Struct("@i2f2P")
assert _NORM_DESC.size == ctypes.sizeof(NormDesc)


class SampleDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("row_stride", ctypes.c_int64)]


class LogprobDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("top", ctypes.c_int32),
                ("row_stride", ctypes.c_int64)]


_LOGPROB_DESC = struct.Struct("@4iq")
assert _LOGPROB_DESC.size == ctypes.sizeof(LogprobDesc)


class SelectDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("positions", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("top", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("mode", ctypes.c_int32)]


class WidthPolicy(ctypes.Structure):
    _fields_ = [("policy", ctypes.c_int32), ("q_max", ctypes.c_int32),
                ("min_width", ctypes.c_int32), ("mask_id", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("offset", ctypes.c_float)]


_lib = None


def load(path: str = LIB_PATH):
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} not found: build it with "
            "`python -m speculative_decoding_target_gb300.build`")
    lib = ctypes.CDLL(path)
    P, i32, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32
    sz = ctypes.c_size_t
    lib.spec_verify_workspace_size.argtypes = [ctypes.POINTER(AttnDesc)]
    lib.spec_verify_workspace_size.restype = sz
    lib.spec_verify_attention.argtypes = [
        ctypes.POINTER(AttnDesc), P, P, P, P, P, P, P, ctypes.c_float, P, P,
        sz, P]
    lib.spec_verify_attention.restype = ctypes.c_int
    lib.spec_verify_attention_noalloc.argtypes = [
        ctypes.POINTER(AttnDesc), P, P, P, P, P, P, P, ctypes.c_float, P, P]
    lib.spec_verify_attention_noalloc.restype = ctypes.c_int
    lib.spec_kv_append.argtypes = [ctypes.POINTER(AttnDesc), P, P, P, P, P,
                                   P, P, P, P, P, P, P]
    lib.spec_kv_append.restype = ctypes.c_int
    lib.spec_verify_shared_workspace_size.argtypes = [
        ctypes.POINTER(AttnDesc), i32]
    lib.spec_verify_shared_workspace_size.restype = sz
    lib.spec_verify_attention_shared.argtypes = [
        ctypes.POINTER(AttnDesc), P, P, P, P, P, P, P, i32, P, P,
        ctypes.c_float, P, P, sz, P]
    lib.spec_verify_attention_shared.restype = ctypes.c_int
    lib.spec_chunk_workspace_size.argtypes = [ctypes.POINTER(AttnDesc)]
    lib.spec_chunk_workspace_size.restype = sz
    lib.spec_chunk_attention.argtypes = lib.spec_verify_attention.argtypes
    lib.spec_chunk_attention.restype = ctypes.c_int
    lib.spec_sample.argtypes = [ctypes.POINTER(SampleDesc)] + [P] * 10
    lib.spec_sample.restype = ctypes.c_int
    lib.spec_logprobs.argtypes = [P] * 9
    lib.spec_logprobs.restype = ctypes.c_int
    lib.spec_rope_append.argtypes = [P] * 16
    lib.spec_rope_append.restype = ctypes.c_int
    lib.spec_norm_rope_append.argtypes = [P] * 17
    lib.spec_norm_rope_append.restype = ctypes.c_int
    lib.spec_verify_set_wait_limit.argtypes = [ctypes.c_int64]
    lib.spec_verify_set_wait_limit.restype = ctypes.c_int
    lib.spec_verify_status.argtypes = [P, ctypes.POINTER(u32), i32, P]
    lib.spec_verify_status.restype = ctypes.c_int
    lib.spec_accept_workspace_size.argtypes = [i32, i32]
    lib.spec_accept_workspace_size.restype = sz
    lib.spec_greedy_accept.argtypes = [P, P, i32, i32, i32, P, P, P, P, sz, P]
    lib.spec_greedy_accept.restype = ctypes.c_int
    lib.spec_greedy_accept_commit.argtypes = [P, P, P, i32, i32, i32, P, P, P,
                                              P, P, P, sz, P]
    lib.spec_greedy_accept_commit.restype = ctypes.c_int
    lib.spec_prepare_next_block.argtypes = [
        ctypes.POINTER(WidthPolicy), i32, P, P, P, P, P, P, i32, i32, i32, P,
        P, P, P, P, P, P]
    lib.spec_prepare_next_block.restype = ctypes.c_int
    lib.spec_stochastic_workspace_size.argtypes = [i32, i32, i32]
    lib.spec_stochastic_workspace_size.restype = sz
    lib.spec_stochastic_accept.argtypes = [P, P, P, P, i32, i32, i32, P, P, P,
                                           P, P, P, P, P, P, sz, P]
    lib.spec_stochastic_accept.restype = ctypes.c_int
    lib.spec_select_workspace_size.argtypes = [ctypes.POINTER(SelectDesc)]
    lib.spec_select_workspace_size.restype = sz
    lib.spec_dflash2_select.argtypes = [ctypes.POINTER(SelectDesc), P, P, P,
                                        P, P, P, P, P, P, P, P, sz, P]
    lib.spec_dflash2_select.restype = ctypes.c_int
    lib.spec_last_error.argtypes = []
    lib.spec_last_error.restype = ctypes.c_char_p
    lib.spec_version.argtypes = []
    lib.spec_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int):
    if rc != SPEC_OK:
        raise SpecError(rc, load().spec_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _at(t: Optional[torch.Tensor]):
    """Address of a tensor as ctypes takes it for a void pointer."""
    return None if t is None else t.data_ptr()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _expect(t: torch.Tensor, dtype, what: str, shape=None,
            contiguous: bool = False) -> None:
    """Refuse a tensor of another type, shape or layout before its address
    is taken."""
    if t.dtype is not dtype:
        raise SpecError(SPEC_ERR_ARG, f"{what} must be {dtype}, is {t.dtype}")
    if shape is not None and t.shape != shape:
        raise SpecError(SPEC_ERR_ARG, f"{what} must be {tuple(shape)}, is "
                                      f"{tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise SpecError(SPEC_ERR_ARG, f"{what} must be contiguous")


def _on_current_device(tensors, stream) -> int:
    """Check that every tensor (None: absent) and the stream belong to the
    current CUDA device, where the library launches on plain addresses; the
    stream's handle (None: the current stream)."""
    on = {t.get_device() for t in tensors if t is not None}  # -1: the host
    if -1 in on:
        raise SpecError(SPEC_ERR_ARG, "tensors must be on a CUDA device")
    now = torch.cuda.current_device()
    if on != {now}:
        raise SpecError(SPEC_ERR_ARG, f"tensors on devices {sorted(on)} in a "
                                      f"call on cuda:{now}, the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(now)
    if stream.device_index != now:
        raise SpecError(SPEC_ERR_ARG, "the stream is another device's")
    return stream.cuda_stream


def _packed(layout: struct.Struct, *values) -> bytes:
    """A descriptor's bytes; numbers that its fields cannot hold are refused."""
    try:
        return layout.pack(*values)
    except (struct.error, OverflowError) as e:
        raise SpecError(SPEC_ERR_ARG, f"a value out of range: {e}") from None


def _made_on(stream):
    """Allocate a call's own buffers for the stream that the call runs on:
    memory of another stream could be handed out again, when the buffer is
    dropped, before the call has run."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(
        stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """torch.empty on the call's stream (see _made_on)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _expect_pools(k_pages, v_pages, k_scales, v_scales, hkv: int,
                  d: int) -> bool:
    """Check a K/V page pool; returns whether it is FP8."""
    fp8 = k_pages.dtype == torch.uint8
    shape = (k_pages.shape[0], hkv, k_pages.shape[2], d)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    _expect(k_pages, dtype, "k_pages", shape, True)
    _expect(v_pages, dtype, "v_pages", shape, True)
    if fp8 and k_scales is not None and v_scales is not None:
        shape = shape[:3] + (d // 64,)
        _expect(k_scales, torch.float16, "k_scales", shape, True)
        _expect(v_scales, torch.float16, "v_scales", shape, True)
    return fp8


def _expect_optional(B: int, q_len: int, q_lens, positions=None,
                     cache_loc=None) -> None:
    if q_lens is not None:
        _expect(q_lens, torch.int32, "q_lens", (B,), True)
    if positions is not None:
        _expect(positions, torch.int32, "positions", (B, q_len), True)
    if cache_loc is not None:
        _expect(cache_loc, torch.int64, "cache_loc", (B, q_len), True)


def make_desc(*, batch, q_len, num_q_heads, num_kv_heads, head_dim,
              page_size, num_pages, max_pages_per_seq, kv_dtype="bf16",
              checked=False, q_lens: Optional[torch.Tensor] = None) -> AttnDesc:
    """q_lens: optional int32 device tensor [B] of per-request block rows."""
    return AttnDesc(batch, q_len, num_q_heads, num_kv_heads, head_dim,
                    page_size, num_pages, max_pages_per_seq,
                    SPEC_KV_BF16 if kv_dtype == "bf16" else SPEC_KV_FP8_E4M3,
                    SPEC_FLAG_CHECKED if checked else 0,
                    None if q_lens is None else q_lens.data_ptr())


def desc_for(q: torch.Tensor, k_pages: torch.Tensor,
             page_table: torch.Tensor, checked: bool = False,
             q_lens: Optional[torch.Tensor] = None) -> AttnDesc:
    B, q_len, hq, d = q.shape
    num_pages, hkv, ps, d2 = k_pages.shape
    assert d2 == d
    return make_desc(batch=B, q_len=q_len, num_q_heads=hq, num_kv_heads=hkv,
                     head_dim=d, page_size=ps, num_pages=num_pages,
                     max_pages_per_seq=page_table.shape[1],
                     kv_dtype="fp8" if k_pages.dtype == torch.uint8 else "bf16",
                     checked=checked, q_lens=q_lens)


def verify_workspace_size(desc: AttnDesc) -> int:
    n = load().spec_verify_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise SpecError(SPEC_ERR_ARG, load().spec_last_error().decode())
    return int(n)


def accept_workspace_size(rows: int, vocab: int) -> int:
    return int(load().spec_accept_workspace_size(rows, vocab))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator hands out 512-byte aligned blocks
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)


def verify_attention_into(desc: AttnDesc, q, k_pages, v_pages, k_scales,
                          v_scales, page_table, seq_lens, scale: float, out,
                          workspace: torch.Tensor, stream=None) -> None:
    _check(load().spec_verify_attention(
        ctypes.byref(desc), _ptr(q), _ptr(k_pages), _ptr(v_pages),
        _ptr(k_scales), _ptr(v_scales), _ptr(page_table), _ptr(seq_lens),
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(stream)))


def verify_attention(q, k_pages, v_pages, page_table, seq_lens, *,
                     scale: float, k_scales=None, v_scales=None,
                     out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     checked: bool = False, q_lens=None,
                     stream=None) -> torch.Tensor:
    """Verify attention on device tensors; returns out bf16 [B, q_len, Hq, D]
    (q_lens: optional int32 [B] rows per request of a block padded to
    q_len)."""
    desc = desc_for(q, k_pages, page_table, checked, q_lens)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = alloc_workspace(verify_workspace_size(desc), q.device)
    verify_attention_into(desc, q, k_pages, v_pages, k_scales, v_scales,
                          page_table, seq_lens, scale, out, workspace, stream)
    return out


def shared_workspace_size(desc: AttnDesc, groups: int) -> int:
    n = load().spec_verify_shared_workspace_size(ctypes.byref(desc), groups)
    if n == 0:
        raise SpecError(SPEC_ERR_ARG, load().spec_last_error().decode())
    return int(n)


def verify_attention_shared(q, k_pages, v_pages, page_table, seq_lens,
                            group_starts, shared_lens, *, scale: float,
                            k_scales=None, v_scales=None,
                            out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            checked: bool = False, q_lens=None,
                            stream=None) -> torch.Tensor:
    """Verify attention of requests that share cached prefixes: group n is
    requests group_starts[n] .. group_starts[n+1] - 1 (int32 [groups + 1]),
    whose first shared_lens[n] (int32 [groups]) tokens are the same cache
    entries; each shared part is computed once for its group.  Returns out
    bf16 [B, q_len, Hq, D]."""
    B, q_len, hq, d = q.shape
    _expect(q, torch.bfloat16, "q", contiguous=True)
    fp8 = _expect_pools(k_pages, v_pages, k_scales, v_scales,
                        k_pages.shape[1], d)
    groups = shared_lens.numel()
    _expect(page_table, torch.int32, "page_table", contiguous=True)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise SpecError(SPEC_ERR_ARG, f"page_table must have {B} rows")
    _expect(seq_lens, torch.int32, "seq_lens", (B,), True)
    _expect(shared_lens, torch.int32, "shared_lens", (groups,), True)
    _expect(group_starts, torch.int32, "group_starts", (groups + 1,), True)
    _expect_optional(B, q_len, q_lens)
    if out is None:
        with _made_on(stream):
            out = torch.empty_like(q)
    _expect(out, torch.bfloat16, "out", q.shape, True)
    on = _on_current_device((q, k_pages, v_pages, k_scales, v_scales,
                             page_table, seq_lens, group_starts, shared_lens,
                             q_lens, out, workspace), stream)
    desc = AttnDesc(B, q_len, hq, k_pages.shape[1], d, k_pages.shape[2],
                    k_pages.shape[0], page_table.shape[1],
                    SPEC_KV_FP8_E4M3 if fp8 else SPEC_KV_BF16,
                    SPEC_FLAG_CHECKED if checked else 0,
                    None if q_lens is None else q_lens.data_ptr())
    if workspace is None:
        with _made_on(stream):
            workspace = alloc_workspace(shared_workspace_size(desc, groups),
                                        q.device)
    rc = load().spec_verify_attention_shared(
        ctypes.byref(desc), _at(q), _at(k_pages), _at(v_pages), _at(k_scales),
        _at(v_scales), _at(page_table), _at(seq_lens), groups,
        _at(group_starts), _at(shared_lens), scale, _at(out), _at(workspace),
        workspace.numel(), on)
    if rc:
        _check(rc)
    return out


def chunk_workspace_size(desc: AttnDesc) -> int:
    n = load().spec_chunk_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise SpecError(SPEC_ERR_ARG, load().spec_last_error().decode())
    return int(n)


def chunk_attention(q, k_pages, v_pages, page_table, seq_lens, *,
                    scale: float, k_scales=None, v_scales=None,
                    out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    checked: bool = False, q_lens=None,
                    stream=None) -> torch.Tensor:
    """Attention of a chunk of new tokens (a prompt or a piece of one, already
    appended) over the paged cache, causal within the chunk: q bf16
    [B, q_len, Hq, 256] for any q_len, q_lens optional int32 [B] tokens per
    request of a chunk padded to q_len.  Returns out bf16 [B, q_len, Hq, 256].
    The weights are rounded to bf16 (fp16 for FP8 KV), but a chunk of at most
    16 tokens and 128 rows per KV head is a block of verify_attention."""
    B, q_len, hq, d = q.shape
    _expect(q, torch.bfloat16, "q", contiguous=True)
    fp8 = _expect_pools(k_pages, v_pages, k_scales, v_scales,
                        k_pages.shape[1], d)
    _expect(page_table, torch.int32, "page_table", contiguous=True)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise SpecError(SPEC_ERR_ARG, f"page_table must have {B} rows")
    _expect(seq_lens, torch.int32, "seq_lens", (B,), True)
    _expect_optional(B, q_len, q_lens)
    if out is None:
        with _made_on(stream):
            out = torch.empty_like(q)
    _expect(out, torch.bfloat16, "out", q.shape, True)
    on = _on_current_device((q, k_pages, v_pages, k_scales, v_scales,
                             page_table, seq_lens, q_lens, out, workspace),
                            stream)
    desc = AttnDesc(B, q_len, hq, k_pages.shape[1], d, k_pages.shape[2],
                    k_pages.shape[0], page_table.shape[1],
                    SPEC_KV_FP8_E4M3 if fp8 else SPEC_KV_BF16,
                    SPEC_FLAG_CHECKED if checked else 0,
                    None if q_lens is None else q_lens.data_ptr())
    if workspace is None:
        with _made_on(stream):
            workspace = alloc_workspace(chunk_workspace_size(desc), q.device)
    rc = load().spec_chunk_attention(
        ctypes.byref(desc), _at(q), _at(k_pages), _at(v_pages), _at(k_scales),
        _at(v_scales), _at(page_table), _at(seq_lens), scale, _at(out),
        _at(workspace), workspace.numel() * workspace.element_size(), on)
    if rc:
        _check(rc)
    return out


def verify_attention_noalloc(q, k_pages, v_pages, page_table, seq_lens, *,
                             scale: float, k_scales=None, v_scales=None,
                             out: Optional[torch.Tensor] = None,
                             q_lens=None, stream=None) -> torch.Tensor:
    """Verify attention with the library's fixed scratch instead of a
    workspace (for callers that cannot allocate device memory)."""
    desc = desc_for(q, k_pages, page_table, q_lens=q_lens)
    if out is None:
        out = torch.empty_like(q)
    _check(load().spec_verify_attention_noalloc(
        ctypes.byref(desc), _ptr(q), _ptr(k_pages), _ptr(v_pages),
        _ptr(k_scales), _ptr(v_scales), _ptr(page_table), _ptr(seq_lens),
        float(scale), _ptr(out), _stream(stream)))
    return out


def kv_append(k_new, v_new, k_pages, v_pages, page_table, seq_lens, *,
              k_scales=None, v_scales=None, positions=None, cache_loc=None,
              checked: bool = False, workspace=None, q_lens=None,
              stream=None):
    """Append the verify block's K/V (bf16 [B, q_len, Hkv, D]) to the paged
    pool in place (quantised on write for an FP8 pool); fills the optional
    positions (int32 [B, q_len]) and cache_loc (int64 [B, q_len])."""
    B, q_len, hkv, d = k_new.shape
    num_pages, hkv2, ps, _ = k_pages.shape
    desc = make_desc(batch=B, q_len=q_len, num_q_heads=hkv, num_kv_heads=hkv,
                     head_dim=d, page_size=ps, num_pages=num_pages,
                     max_pages_per_seq=page_table.shape[1],
                     kv_dtype="fp8" if k_pages.dtype == torch.uint8 else "bf16",
                     checked=checked, q_lens=q_lens)
    _check(load().spec_kv_append(
        ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(k_pages),
        _ptr(v_pages), _ptr(k_scales), _ptr(v_scales), _ptr(page_table),
        _ptr(seq_lens), _ptr(positions), _ptr(cache_loc), _ptr(workspace),
        _stream(stream)))


def _strides(t: torch.Tensor, what: str):
    """(request, token) strides of [B, q_len, H, 256] whose heads and channels
    are contiguous."""
    B, q_len, heads, d = t.shape
    request, token, head, channel = t.stride()
    if channel != 1 or (heads > 1 and head != d):
        raise SpecError(SPEC_ERR_ARG,
                        f"{what}: heads and channels must be contiguous")
    return request if B > 1 else 0, token if q_len > 1 else 0


def rope_append(q, k_new, v_new, freq, k_pages, v_pages, page_table, seq_lens,
                *, interleaved: bool = False, attn_factor: float = 1.0,
                q_out: Optional[torch.Tensor] = None, k_scales=None,
                v_scales=None, positions=None, cache_loc=None,
                checked: bool = False, workspace=None, q_lens=None,
                stream=None):
    """Rotate the block's queries and keys to their positions and append K/V
    to the paged pool in place (quantised on write for an FP8 pool).

    q bf16 [B, q_len, Hq, 256] (None: keys and values only), k_new / v_new
    bf16 [B, q_len, Hkv, 256], each possibly a view of one projection's
    output; freq float64 [rotary_dim / 2] radians per position
    (rope_frequencies).  Returns the rotated queries, bf16
    [B, q_len, Hq, 256] (q_out, which may be a contiguous q itself), or None.
    """
    return _rope_append(q, k_new, v_new, None, freq, k_pages, v_pages,
                        page_table, seq_lens, interleaved, attn_factor, q_out,
                        k_scales, v_scales, positions, cache_loc, checked,
                        workspace, q_lens, stream)


def norm_rope_append(q, k_new, v_new, q_weight, k_weight, freq, k_pages,
                     v_pages, page_table, seq_lens, *, eps: float = 1e-6,
                     weight_offset: float = 0.0, interleaved: bool = False,
                     attn_factor: float = 1.0,
                     q_out: Optional[torch.Tensor] = None, k_scales=None,
                     v_scales=None, positions=None, cache_loc=None,
                     checked: bool = False, workspace=None, q_lens=None,
                     stream=None):
    """rope_append with an RMS norm of every query and key head before its
    rotation: x / sqrt(mean(x^2) + eps) * (weight_offset + weight), weights
    bf16 or fp32 [256] (q_weight None with q None).  Returns the rotated
    queries, or None."""
    return _rope_append(q, k_new, v_new, (q_weight, k_weight, eps,
                                          weight_offset), freq, k_pages,
                        v_pages, page_table, seq_lens, interleaved,
                        attn_factor, q_out, k_scales, v_scales, positions,
                        cache_loc, checked, workspace, q_lens, stream)


def _rope_append(q, k_new, v_new, norm, freq, k_pages, v_pages, page_table,
                 seq_lens, interleaved, attn_factor, q_out, k_scales, v_scales,
                 positions, cache_loc, checked, workspace, q_lens, stream):
    shape = k_new.shape
    B, q_len, hkv, d = shape
    hq = 0 if q is None else q.shape[2]
    _expect(k_new, torch.bfloat16, "k_new")
    _expect(v_new, torch.bfloat16, "v_new", shape)
    _expect(freq, torch.float64, "freq", (freq.numel(),), contiguous=True)
    _expect(page_table, torch.int32, "page_table", contiguous=True)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise SpecError(SPEC_ERR_ARG, f"page_table must have {B} rows")
    _expect(seq_lens, torch.int32, "seq_lens", (B,), contiguous=True)
    if q is not None:
        q_shape = (B, q_len, hq, d)
        _expect(q, torch.bfloat16, "q", q_shape)
        if q_out is None:
            q_out = _empty(q_shape, torch.bfloat16, q.device, stream)
        else:
            _expect(q_out, torch.bfloat16, "q_out", q_shape, contiguous=True)
    q_w = k_w = None
    if norm is not None:
        q_w, k_w, eps, offset = norm
        if (k_w is None or (q_w is None) != (q is None)
                or k_w.dtype not in (torch.bfloat16, torch.float32)):
            raise SpecError(SPEC_ERR_ARG, "q_weight goes with q; weights are "
                                          "bf16 or fp32")
        _expect(k_w, k_w.dtype, "k_weight", (d,), contiguous=True)
        if q_w is not None:
            _expect(q_w, k_w.dtype, "q_weight", (d,), contiguous=True)
    fp8 = _expect_pools(k_pages, v_pages, k_scales, v_scales, hkv, d)
    _expect_optional(B, q_len, q_lens, positions, cache_loc)
    if (checked and workspace is not None
            and workspace.numel() * workspace.element_size() < 4):
        raise SpecError(SPEC_ERR_WORKSPACE, "workspace of fewer than 4 bytes")
    on = _on_current_device((q, k_new, v_new, freq, q_out, k_pages, v_pages,
                             k_scales, v_scales, page_table, seq_lens, q_lens,
                             positions, cache_loc, workspace, q_w, k_w),
                            stream)
    pages, _, page, _ = k_pages.shape
    desc = _packed(
        _ROPE_DESC,
        B, q_len, hq, hkv, d, page, pages, page_table.shape[1],
        SPEC_KV_FP8_E4M3 if fp8 else SPEC_KV_BF16,
        SPEC_FLAG_CHECKED if checked else 0,
        0 if q_lens is None else q_lens.data_ptr(), 2 * freq.shape[0],
        1 if interleaved else 0, attn_factor,
        *(_strides(q, "q") if q is not None else (0, 0)),
        *_strides(k_new, "k_new"), *_strides(v_new, "v_new"))
    args = (_at(q), k_new.data_ptr(), v_new.data_ptr(), freq.data_ptr(),
            q_out.data_ptr() if q is not None else None, k_pages.data_ptr(),
            v_pages.data_ptr(), _at(k_scales), _at(v_scales),
            page_table.data_ptr(), seq_lens.data_ptr(), _at(positions),
            _at(cache_loc), _at(workspace), on)
    if norm is None:
        rc = load().spec_rope_append(desc, *args)
    else:
        rc = load().spec_norm_rope_append(desc, _packed(
            _NORM_DESC, k_w.dtype == torch.bfloat16, eps, offset,
            0 if q_w is None else q_w.data_ptr(), k_w.data_ptr()), *args)
    if rc:
        _check(rc)
    return q_out


def set_wait_limit(cycles: int) -> None:
    """Main-loop wait bound (SM clock cycles) of the split kernels for calls
    with checked=True; 0 restores the default.  A test hook for the timeout
    path."""
    _check(load().spec_verify_set_wait_limit(int(cycles)))


def verify_status(workspace: torch.Tensor, clear: bool = True,
                  stream=None) -> int:
    st = ctypes.c_uint32(0)
    _check(load().spec_verify_status(_ptr(workspace), ctypes.byref(st),
                                     int(clear), _stream(stream)))
    return int(st.value)


def greedy_accept_into(logits, draft_ids, accept_len, next_token, out_tokens,
                       workspace: torch.Tensor, stream=None) -> None:
    B, q_len = draft_ids.shape
    _check(load().spec_greedy_accept(
        _ptr(logits), _ptr(draft_ids), B, q_len, logits.shape[-1],
        _ptr(accept_len), _ptr(next_token), _ptr(out_tokens),
        _ptr(workspace), workspace.numel(), _stream(stream)))


def greedy_accept_commit_into(logits, draft_ids, q_lens, seq_lens,
                              new_seq_lens, accept_len, next_token, out_tokens,
                              workspace: torch.Tensor, stream=None) -> None:
    B, q_len = draft_ids.shape
    _check(load().spec_greedy_accept_commit(
        _ptr(logits), _ptr(draft_ids), _ptr(q_lens), B, q_len,
        logits.shape[-1], _ptr(seq_lens), _ptr(new_seq_lens),
        _ptr(accept_len), _ptr(next_token), _ptr(out_tokens),
        _ptr(workspace), workspace.numel(), _stream(stream)))


def greedy_accept_commit(logits, draft_ids, q_lens, seq_lens, *,
                         workspace: Optional[torch.Tensor] = None,
                         stream=None):
    """Greedy accept with per-request widths and the committed cache length.
    Returns (accept_len, next_token, out_tokens, new_seq_lens)."""
    B, q_len = draft_ids.shape
    dev = logits.device
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    nxt = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, q_len), dtype=torch.int32, device=dev)
    new = torch.empty(B, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(
            accept_workspace_size(B * q_len, logits.shape[-1]), dev)
    greedy_accept_commit_into(logits, draft_ids, q_lens, seq_lens, new, acc,
                              nxt, toks, workspace, stream)
    return acc, nxt, toks, new


def width_policy(policy: str, q_max: int, *, min_width: int = 2,
                 alpha: float = 0.5, offset: float = 1.5,
                 mask_id: int = 0) -> WidthPolicy:
    return WidthPolicy(WIDTH_POLICIES[policy], q_max, min_width, mask_id,
                       alpha, offset)


def prepare_next_block_into(pol: WidthPolicy, q_lens, accept_len, next_token,
                            new_seq_lens, state, page_table, page_size: int,
                            num_pages: int, next_q_lens, next_seq_lens,
                            block_ids=None, positions=None, cache_loc=None,
                            status=None, stream=None) -> None:
    B = accept_len.shape[0]
    _check(load().spec_prepare_next_block(
        ctypes.byref(pol), B, _ptr(q_lens), _ptr(accept_len),
        _ptr(next_token), _ptr(new_seq_lens), _ptr(state), _ptr(page_table),
        page_table.shape[1], page_size, num_pages, _ptr(next_q_lens),
        _ptr(next_seq_lens), _ptr(block_ids), _ptr(positions),
        _ptr(cache_loc), _ptr(status), _stream(stream)))


def prepare_next_block(pol: WidthPolicy, q_lens, accept_len, next_token,
                       new_seq_lens, state, page_table, *, page_size: int,
                       num_pages: int, status=None, stream=None):
    """Next widths and next-block layout on the device (state updated in
    place).  Returns dict of next_q_lens, next_seq_lens, block_ids,
    positions, cache_loc."""
    B = accept_len.shape[0]
    dev = accept_len.device
    out = {"next_q_lens": torch.empty(B, dtype=torch.int32, device=dev),
           "next_seq_lens": torch.empty(B, dtype=torch.int32, device=dev),
           "block_ids": torch.empty((B, pol.q_max), dtype=torch.int32,
                                    device=dev),
           "positions": torch.empty((B, pol.q_max), dtype=torch.int32,
                                    device=dev),
           "cache_loc": torch.empty((B, pol.q_max), dtype=torch.int64,
                                    device=dev)}
    prepare_next_block_into(pol, q_lens, accept_len, next_token, new_seq_lens,
                            state, page_table, page_size, num_pages,
                            out["next_q_lens"], out["next_seq_lens"],
                            out["block_ids"], out["positions"],
                            out["cache_loc"], status, stream)
    return out


def stochastic_workspace_size(batch: int, q_len: int, vocab: int) -> int:
    return int(load().spec_stochastic_workspace_size(batch, q_len, vocab))


def stochastic_accept_into(logits, draft_ids, draft_probs, q_lens,
                           temperature, u_accept, u_sample, seq_lens,
                           new_seq_lens, accept_len, next_token, out_tokens,
                           workspace: torch.Tensor, stream=None) -> None:
    B, q_len = draft_ids.shape
    _check(load().spec_stochastic_accept(
        _ptr(logits), _ptr(draft_ids), _ptr(draft_probs), _ptr(q_lens), B,
        q_len, logits.shape[-1], _ptr(temperature), _ptr(u_accept),
        _ptr(u_sample), _ptr(seq_lens), _ptr(new_seq_lens), _ptr(accept_len),
        _ptr(next_token), _ptr(out_tokens), _ptr(workspace),
        workspace.numel(), _stream(stream)))


def stochastic_accept(logits, draft_ids, temperature, u_accept, u_sample, *,
                      draft_probs=None, q_lens=None, seq_lens=None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Rejection-sampling verify.  Returns (accept_len, next_token,
    out_tokens, new_seq_lens or None)."""
    B, q_len = draft_ids.shape
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    acc, nxt = torch.empty(B, **i32), torch.empty(B, **i32)
    toks = torch.empty((B, q_len), **i32)
    new = torch.empty(B, **i32) if seq_lens is not None else None
    if workspace is None:
        workspace = alloc_workspace(
            stochastic_workspace_size(B, q_len, logits.shape[-1]), dev)
    stochastic_accept_into(logits, draft_ids, draft_probs, q_lens,
                           temperature, u_accept, u_sample, seq_lens, new,
                           acc, nxt, toks, workspace, stream)
    return acc, nxt, toks, new


def _row_stride(logits: torch.Tensor, rows: int) -> int:
    """Elements from one row of logits [.., vocab] to the next."""
    vocab = logits.shape[-1]
    if logits.dim() == 2 and rows > 1 and logits.stride(1) == 1:
        stride = logits.stride(0)
    elif logits.is_contiguous():
        stride = vocab
    elif rows == 1 and (vocab == 1 or logits.stride(-1) == 1):
        stride = vocab
    else:
        try:                    # [.., vocab] of a padded vocabulary
            flat = logits.view(rows, vocab)
        except RuntimeError:
            flat = None
        if flat is None or (vocab > 1 and flat.stride(1) != 1):
            raise SpecError(SPEC_ERR_ARG, "logits rows must be contiguous and "
                                          "evenly spaced")
        stride = flat.stride(0)
    if rows > 1 and stride < vocab:
        raise SpecError(SPEC_ERR_ARG, "logits rows overlap")
    return stride


def sample(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None,
           probs: Optional[torch.Tensor] = None,
           filtered: Optional[torch.Tensor] = None,
           token: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The next token of every row of logits (fp32 or bf16 [.., vocab], rows
    contiguous, evenly spaced) from the uniforms u (fp32 [..]), with optional
    per-row temperature, top_p, min_p (fp32) and top_k (int32).  Fills the
    optional probs (the distribution drawn from) and filtered (the logits,
    -inf outside the kept set), fp32 of the logits' shape.  Returns token
    int32 [..]."""
    lead, vocab = logits.shape[:-1], logits.shape[-1]
    rows = u.numel()
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise SpecError(SPEC_ERR_ARG, f"logits are {logits.dtype}")
    if token is None:
        with _made_on(stream):
            token = torch.empty(lead, dtype=torch.int32, device=logits.device)
    for t, dtype, what in ((u, torch.float32, "u"),
                           (temperature, torch.float32, "temperature"),
                           (top_k, torch.int32, "top_k"),
                           (top_p, torch.float32, "top_p"),
                           (min_p, torch.float32, "min_p"),
                           (token, torch.int32, "token")):
        if t is not None:
            _expect(t, dtype, what, lead, True)
    for t, what in ((probs, "probs"), (filtered, "filtered")):
        if t is not None:
            _expect(t, torch.float32, what, logits.shape, True)
    on = _on_current_device((logits, u, temperature, top_k, top_p, min_p,
                             probs, filtered, token), stream)
    stride = _row_stride(logits, rows)
    desc = SampleDesc(rows, vocab, int(logits.dtype == torch.bfloat16),
                      stride)
    rc = load().spec_sample(
        ctypes.byref(desc), _at(logits), _at(temperature), _at(top_k),
        _at(top_p), _at(min_p), _at(u), _at(token), _at(probs), _at(filtered),
        on)
    if rc:
        _check(rc)
    return token


def logprobs(logits, token=None, *, temperature=None, top: int = 0,
             stream=None) -> dict:
    """Log probabilities of the given tokens (int32 [..], or None) under the
    rows of logits (fp32 or bf16 [.., vocab], rows contiguous, evenly spaced),
    with an optional per-row temperature (fp32 [..]).  Returns a dict of
    logprob fp32 [..] (with token), entropy fp32 [..], and with top > 0 the
    most likely tokens top_ids int32 [.., top] and their top_logprobs fp32
    [.., top].  Rows whose token lies outside the vocabulary are idle: zeros,
    ids -1."""
    lead, vocab = logits.shape[:-1], logits.shape[-1]
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise SpecError(SPEC_ERR_ARG, f"logits are {logits.dtype}")
    if token is not None:
        _expect(token, torch.int32, "token", lead, True)
    if temperature is not None:
        _expect(temperature, torch.float32, "temperature", lead, True)
    if not 0 <= top <= LOGPROB_MAX_TOP:     # before anything of that size is made
        raise SpecError(SPEC_ERR_ARG, f"top {top} outside [0, {LOGPROB_MAX_TOP}]")
    on = _on_current_device((logits, token, temperature), stream)
    rows = lead.numel()
    stride = _row_stride(logits, rows)
    desc = _packed(_LOGPROB_DESC, rows, vocab, logits.dtype == torch.bfloat16,
                   top, stride)
    dev, f32 = logits.device, torch.float32
    logprob = top_ids = top_logprobs = None
    if token is not None:
        logprob = _empty(lead, f32, dev, stream)
    entropy = _empty(lead, f32, dev, stream)
    if top > 0:
        top_ids = _empty((*lead, top), torch.int32, dev, stream)
        top_logprobs = _empty((*lead, top), f32, dev, stream)
    rc = load().spec_logprobs(
        desc, logits.data_ptr(), _at(token), _at(temperature), _at(logprob),
        entropy.data_ptr(), _at(top_ids), _at(top_logprobs), on)
    if rc:
        _check(rc)
    out = {} if token is None else {"logprob": logprob}
    out["entropy"] = entropy
    if top > 0:
        out["top_ids"], out["top_logprobs"] = top_ids, top_logprobs
    return out


def select_desc(cand_logits, code_a, hidden, *, top: int = 16,
                mode: str = "greedy") -> SelectDesc:
    B, P1, V = cand_logits.shape
    return SelectDesc(B, P1 + 1, V, top, code_a.shape[1], hidden.shape[2],
                      SELECT_MODES[mode])


def select_workspace_size(desc: SelectDesc) -> int:
    n = load().spec_select_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise SpecError(SPEC_ERR_ARG, load().spec_last_error().decode())
    return int(n)


def dflash2_select_into(desc: SelectDesc, cand_logits, boundary, hidden, w_h,
                        code_a, code_b, draft_ids, cand_ids, cand_logit,
                        trans, workspace: torch.Tensor, stream=None) -> None:
    _check(load().spec_dflash2_select(
        ctypes.byref(desc), _ptr(cand_logits), _ptr(boundary), _ptr(hidden),
        _ptr(w_h), _ptr(code_a), _ptr(code_b), _ptr(draft_ids),
        _ptr(cand_ids), _ptr(cand_logit), _ptr(trans), _ptr(workspace),
        workspace.numel(), _stream(stream)))


def dflash2_select(cand_logits, boundary, hidden, w_h, code_a, code_b, *,
                   top: int = 16, mode: str = "greedy",
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """DFlash2 candidate selection on device tensors.  Returns dict of
    draft_ids [B, P], cand_ids [B, P-1, K], cand_logit [B, P-1, K] and
    trans [B, P-1, K, K]."""
    desc = select_desc(cand_logits, code_a, hidden, top=top, mode=mode)
    B, P1 = cand_logits.shape[:2]
    dev = cand_logits.device
    out = {"draft_ids": torch.empty((B, P1 + 1), dtype=torch.int32,
                                    device=dev),
           "cand_ids": torch.empty((B, P1, top), dtype=torch.int32,
                                   device=dev),
           "cand_logit": torch.empty((B, P1, top), device=dev),
           "trans": torch.empty((B, P1, top, top), device=dev)}
    if workspace is None:
        workspace = alloc_workspace(select_workspace_size(desc), dev)
    dflash2_select_into(desc, cand_logits, boundary, hidden, w_h, code_a,
                        code_b, out["draft_ids"], out["cand_ids"],
                        out["cand_logit"], out["trans"], workspace, stream)
    return out


def greedy_accept(logits: torch.Tensor, draft_ids: torch.Tensor, *,
                  workspace: Optional[torch.Tensor] = None,
                  with_tokens: bool = True, stream=None):
    """Returns (accept_len [B], next_token [B], out_tokens [B, q_len] or None)."""
    B, q_len = draft_ids.shape
    dev = logits.device
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    nxt = torch.empty(B, dtype=torch.int32, device=dev)
    toks = (torch.empty((B, q_len), dtype=torch.int32, device=dev)
            if with_tokens else None)
    if workspace is None:
        workspace = alloc_workspace(
            accept_workspace_size(B * q_len, logits.shape[-1]), dev)
    greedy_accept_into(logits, draft_ids, acc, nxt, toks, workspace, stream)
    return acc, nxt, toks
