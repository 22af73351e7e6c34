"""Python binding of libsmcsd.so - the MI355X (gfx950) SMC-SD verify / resample / KV path.

Argument marshalling only: every step of the path runs in the library's HIP kernels.
Tensors must be device (HIP) tensors; this module checks placement, dtype, contiguity
and sizes so that no host pointer or short buffer reaches a kernel, passes raw pointers
and the current torch stream, and turns negative return codes into ``SmcsdError``.
There is no fallback: if the library is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsmcsd.so")

DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
MODE_SMC, MODE_SPS, MODE_SMC_RACE = 0, 1, 2  # MODE_SMC_RACE: SMC with the exponential-race bonus
OP_VERIFY_SMC, OP_VERIFY_SPS, OP_KV, OP_DRAFT, OP_KV_CHECK = 0, 1, 2, 3, 4
OP_TREE_ATTN, OP_LOGPROBS, OP_KV_FREE, OP_KV_COMPACT = 5, 6, 7, 8
KV_COPY_MAX_CACHES = 256
STATIC_SCRATCH_BYTES = 4 << 20  # smcsd_verify_static's per-GPU scratch array

ST_NAN_INPUT = 1
ST_EMPTY_ROW = 2
ST_NOSPACE = 4
ST_DEGENERATE_WEIGHTS = 8
ST_BAD_INPUT = 16
ST_KV_INCONSISTENT = 32
KV_CHECK_KINDS = 5
STREAM_READ_TILE_BYTES = 131072
KV_CHECK_NAMES = ("refcount != table references", "table id out of range",
                  "free-stack entry out of range or repeated", "referenced block on the free stack",
                  "unreferenced block not on the free stack")

EXPORTED = ("smcsd_version", "smcsd_status_string", "smcsd_workspace_bytes", "smcsd_verify",
            "smcsd_verify_static", "smcsd_draft_sample", "smcsd_resample", "smcsd_kv_reassign",
            "smcsd_resample_kv_reassign", "smcsd_step", "smcsd_kv_check", "smcsd_philox4x32_10",
            "smcsd_stream_read", "smcsd_kv_fork", "smcsd_kv_free", "smcsd_kv_compact",
            "smcsd_kv_copy", "smcsd_qk_norm_rope", "smcsd_tree_attention", "smcsd_token_logprobs")

_DT = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_DT_KV = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}


class SmcsdError(RuntimeError):
    pass


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libsmcsd.so and declare the C signatures (no GPU work)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise SmcsdError("libsmcsd.so is not built (%s); run __graft_entry__.build()" % path)
    lib = ctypes.CDLL(path)
    P, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                                 ctypes.c_float, ctypes.c_size_t)
    lib.smcsd_version.restype = i32
    lib.smcsd_status_string.argtypes = [i32]
    lib.smcsd_status_string.restype = ctypes.c_char_p
    lib.smcsd_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i64]
    lib.smcsd_workspace_bytes.restype = sz
    lib.smcsd_verify.argtypes = [P, P, i32, i64, i32, P, i32, i32, i32, i32, f32, f32, i32, u64,
                                 u64, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.smcsd_verify.restype = i32
    lib.smcsd_verify_static.argtypes = [P, P, i32, i64, i32, P, i32, i32, i32, i32, f32, f32, i32,
                                        u64, u64, P, P, P, P, P, P, P, P, P, P]
    lib.smcsd_verify_static.restype = i32
    lib.smcsd_draft_sample.argtypes = [P, i32, i64, i32, i32, f32, u64, u64, i32, P, P, P, P, sz, P]
    lib.smcsd_draft_sample.restype = i32
    lib.smcsd_resample.argtypes = [P, i32, i32, f32, u64, u64, P, P, P, P, P]
    lib.smcsd_resample.restype = i32
    lib.smcsd_kv_reassign.argtypes = [P, P, i32, i32, P, i32, i32, i64, i32, P, P, P, i64, P, P,
                                      P, P, sz, P]
    lib.smcsd_kv_reassign.restype = i32
    lib.smcsd_resample_kv_reassign.argtypes = [P, i32, i32, f32, u64, u64, P, P, P, P, i32, i32, i64,
                                               i32, P, P, P, i64, P, P, P, P, sz, P]
    lib.smcsd_resample_kv_reassign.restype = i32
    lib.smcsd_step.argtypes = [P, P, i32, i64, P, i32, i32, i32, i32, f32, f32, i32, f32, u64, u64,
                               P, P, P, P, P, P, P, P, P, P, P, i32, i32, i64, i32, P, P, P, i64,
                               P, P, P, P, sz, P, sz, P]
    lib.smcsd_step.restype = i32
    lib.smcsd_kv_check.argtypes = [P, i64, i32, i32, P, P, P, i64, P, P, P, sz, P]
    lib.smcsd_kv_check.restype = i32
    lib.smcsd_philox4x32_10.argtypes = [P, P, i32, P, P]
    lib.smcsd_philox4x32_10.restype = i32
    lib.smcsd_stream_read.argtypes = [P, i64, P, P]
    lib.smcsd_stream_read.restype = i32
    lib.smcsd_kv_fork.argtypes = [P, i32, i32, P, i32, P, i64, P, P]
    lib.smcsd_kv_fork.restype = i32
    lib.smcsd_kv_free.argtypes = [P, i64, P, i32, P, P, P, i64, P, P, sz, P]
    lib.smcsd_kv_free.restype = i32
    lib.smcsd_kv_compact.argtypes = [P, i64, i32, i32, P, P, P, i64, P, P, P, P, sz, P]
    lib.smcsd_kv_compact.restype = i32
    lib.smcsd_kv_copy.argtypes = [P, i32, i64, i32, i64, i64, i32, P, P, i64, i64, P, P]
    lib.smcsd_kv_copy.restype = i32
    lib.smcsd_qk_norm_rope.argtypes = [P, P, P, i32, i64, i64, i64, i32, i32, i32, i32, i32, P, P,
                                       f32, P, i64, i32, i32, P, P, P, P, i32, i32, i64, P, P, i64,
                                       i64, i64, P, P, P]
    lib.smcsd_qk_norm_rope.restype = i32
    lib.smcsd_tree_attention.argtypes = [P, i32, i64, P, P, i64, i64, i64, P, i32, i32, i64, P, P,
                                         P, i32, i32, i32, i32, i32, i32, f32, i64, P, P, P, P, sz,
                                         P]
    lib.smcsd_tree_attention.restype = i32
    lib.smcsd_token_logprobs.argtypes = [P, i32, i64, i32, i32, f32, P, i32, i32, P, P, P, P, P, P,
                                         P, sz, P]
    lib.smcsd_token_logprobs.restype = i32
    if path == LIB_PATH:
        _lib = lib
    return lib


def _L():
    return _lib if _lib is not None else load_library()


def _check(rc: int, what: str):
    if rc != 0:
        raise SmcsdError("%s failed: %s (%d)" % (what, _L().smcsd_status_string(rc).decode(), rc))


def status_string(code: int) -> str:
    return _L().smcsd_status_string(code).decode()


def version() -> int:
    return int(_L().smcsd_version())


def workspace_bytes(op: int, B: int, N: int, K: int = 0, V: int = 1, P: int = 0) -> int:
    return int(_L().smcsd_workspace_bytes(op, B, N, K, V, P))


def _dev(t: Optional[torch.Tensor], name: str, dtype=None, min_numel: int = 0,
         contiguous: bool = True):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SmcsdError("%s must be a device tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise SmcsdError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if contiguous and not t.is_contiguous():
        raise SmcsdError("%s must be contiguous" % name)
    if t.numel() < min_numel:
        raise SmcsdError("%s holds %d elements, needs %d" % (name, t.numel(), min_numel))
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def alloc_workspace(op: int, B: int, N: int, K: int = 0, V: int = 1, P: int = 0,
                    device=None) -> torch.Tensor:
    """Zero-filled device workspace of the size the library asks for."""
    n = workspace_bytes(op, B, N, K, V, P)
    if n == 0:
        raise SmcsdError("invalid workspace sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def verify(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: Optional[torch.Tensor],
           B: int, N: int, K: int, V: int, temperature: float, alpha: float, mode: int, seed: int,
           step: int, out_tokens: torch.Tensor, status: torch.Tensor, workspace: torch.Tensor,
           log_weights: Optional[torch.Tensor] = None, out_num_tokens=None, out_logp=None,
           out_logq=None, out_lse=None, lse_in=None, seq_step: int = 1,
           row_stride: Optional[int] = None, stream=None, logq_in=None) -> None:
    """smcsd_verify.  target [*, K+1, row_stride], draft [*, K, row_stride] (bf16 or fp32).
    mode: MODE_SMC (bonus by inverse CDF), MODE_SMC_RACE (bonus by the exponential race)
    or MODE_SPS.  With logq_in [*, K] fp32 (the draft's log q of its tokens; SMC modes)
    draft may be None."""
    if target.dtype not in _DT:
        raise SmcsdError("logits must be bfloat16 or float32")
    rs = V if row_stride is None else int(row_stride)
    S = B * N
    nsrc = (S - 1) * seq_step + 1 if S > 0 else 0
    tp = _dev(target, "target", target.dtype, nsrc * (K + 1) * rs - (rs - V) if S else 0)
    dp = _dev(draft, "draft", target.dtype, nsrc * K * rs - (rs - V) if S and K else 0) \
        if K > 0 and (draft is not None or logq_in is None) else None
    xp = _dev(draft_tokens, "draft_tokens", torch.int32, nsrc * K) if K > 0 else None
    lw = _dev(log_weights, "log_weights", torch.float32, S)
    rc = _L().smcsd_verify(
        tp, dp, _DT[target.dtype], rs, seq_step, xp, B, N, K, V, float(temperature), float(alpha),
        mode, int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _dev(lse_in, "lse_in", torch.float32, nsrc * (2 * K + 1)),
        _dev(logq_in, "logq_in", torch.float32, nsrc * K), lw,
        _dev(out_tokens, "out_tokens", torch.int32, S * (K + 1)),
        _dev(out_num_tokens, "out_num_tokens", torch.int32, S),
        _dev(out_logp, "out_logp", torch.float32, S * (K + 1)),
        _dev(out_logq, "out_logq", torch.float32, S * K),
        _dev(out_lse, "out_lse", torch.float32, S * (2 * K + 1)),
        _dev(status, "status", torch.int32, 1),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check(rc, "smcsd_verify")


def verify_static(target: torch.Tensor, draft: Optional[torch.Tensor],
                  draft_tokens: Optional[torch.Tensor], B: int, N: int, K: int, V: int,
                  temperature: float, alpha: float, mode: int, seed: int, step: int,
                  out_tokens: torch.Tensor, status: torch.Tensor,
                  log_weights: Optional[torch.Tensor] = None, out_num_tokens=None, out_logp=None,
                  out_logq=None, out_lse=None, lse_in=None, seq_step: int = 1,
                  row_stride: Optional[int] = None, stream=None, logq_in=None) -> None:
    """smcsd_verify_static: smcsd_verify with the library's own per-GPU scratch array instead
    of a workspace (for callers that cannot allocate); same arguments otherwise.  Calls that
    overlap in time on one GPU race on that array."""
    if target.dtype not in _DT:
        raise SmcsdError("logits must be bfloat16 or float32")
    rs = V if row_stride is None else int(row_stride)
    S = B * N
    nsrc = (S - 1) * seq_step + 1 if S > 0 else 0
    tp = _dev(target, "target", target.dtype, nsrc * (K + 1) * rs - (rs - V) if S else 0)
    dp = _dev(draft, "draft", target.dtype, nsrc * K * rs - (rs - V) if S and K else 0) \
        if K > 0 and (draft is not None or logq_in is None) else None
    xp = _dev(draft_tokens, "draft_tokens", torch.int32, nsrc * K) if K > 0 else None
    lw = _dev(log_weights, "log_weights", torch.float32, S)
    rc = _L().smcsd_verify_static(
        tp, dp, _DT[target.dtype], rs, seq_step, xp, B, N, K, V, float(temperature), float(alpha),
        mode, int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _dev(lse_in, "lse_in", torch.float32, nsrc * (2 * K + 1)),
        _dev(logq_in, "logq_in", torch.float32, nsrc * K), lw,
        _dev(out_tokens, "out_tokens", torch.int32, S * (K + 1)),
        _dev(out_num_tokens, "out_num_tokens", torch.int32, S),
        _dev(out_logp, "out_logp", torch.float32, S * (K + 1)),
        _dev(out_logq, "out_logq", torch.float32, S * K),
        _dev(out_lse, "out_lse", torch.float32, S * (2 * K + 1)),
        _dev(status, "status", torch.int32, 1), _stream(stream))
    _check(rc, "smcsd_verify_static")


def draft_sample(draft: torch.Tensor, n: int, V: int, temperature: float, seed: int, step: int,
                 pos: int, out_tokens: torch.Tensor, status: torch.Tensor, workspace: torch.Tensor,
                 out_logq: Optional[torch.Tensor] = None, row_stride: Optional[int] = None,
                 stream=None) -> None:
    """smcsd_draft_sample.  draft [n, row_stride] (bf16 or fp32) at one draft position."""
    if draft.dtype not in _DT:
        raise SmcsdError("logits must be bfloat16 or float32")
    rs = V if row_stride is None else int(row_stride)
    rc = _L().smcsd_draft_sample(
        _dev(draft, "draft", draft.dtype, n * rs - (rs - V) if n else 0), _DT[draft.dtype], rs, n,
        V, float(temperature), int(seed) & (2**64 - 1), int(step) & (2**64 - 1), int(pos),
        _dev(out_tokens, "out_tokens", torch.int32, n),
        _dev(out_logq, "out_logq", torch.float32, n), _dev(status, "status", torch.int32, 1),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check(rc, "smcsd_draft_sample")


def resample(log_weights: torch.Tensor, B: int, N: int, tau: float, seed: int, step: int,
             ancestors: torch.Tensor, ess: torch.Tensor, resampled: torch.Tensor,
             status: torch.Tensor, stream=None) -> None:
    """smcsd_resample over log_weights [B, N]."""
    rc = _L().smcsd_resample(
        _dev(log_weights, "log_weights", torch.float32, B * N), B, N, float(tau),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _dev(ancestors, "ancestors", torch.int32, B * N), _dev(ess, "ess", torch.float32, B),
        _dev(resampled, "resampled", torch.int32, B), _dev(status, "status", torch.int32, 1),
        _stream(stream))
    _check(rc, "smcsd_resample")


def kv_reassign(ancestors: torch.Tensor, resampled: torch.Tensor, B: int, N: int,
                block_tables: torch.Tensor, block_size: int, seq_len: int, reserve_tokens: int,
                refcounts: torch.Tensor, free_list: torch.Tensor, free_top: torch.Tensor,
                cow: torch.Tensor, cow_count: torch.Tensor, status: torch.Tensor,
                workspace: torch.Tensor, stream=None) -> None:
    """smcsd_kv_reassign.  block_tables [B*N, M_cap] int32; refcounts / free_list [P] int32."""
    if block_tables.dim() != 2 or block_tables.shape[0] != B * N:
        raise SmcsdError("block_tables must be [B*N, M_cap]")
    M_cap = block_tables.shape[1]
    P = refcounts.numel()
    rc = _L().smcsd_kv_reassign(
        _dev(ancestors, "ancestors", torch.int32, B * N), _dev(resampled, "resampled", torch.int32, B),
        B, N, _dev(block_tables, "block_tables", torch.int32), M_cap, block_size, int(seq_len),
        reserve_tokens, _dev(refcounts, "refcounts", torch.int32), _dev(free_list, "free_list",
                                                                       torch.int32, P),
        _dev(free_top, "free_top", torch.int32, 1), P, _dev(cow, "cow", torch.int32, 3 * B * N),
        _dev(cow_count, "cow_count", torch.int32, 1), _dev(status, "status", torch.int32, 1),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check(rc, "smcsd_kv_reassign")
    _debug_kv_check(block_tables, block_size, seq_len, reserve_tokens, refcounts, free_list,
                    free_top, "smcsd_kv_reassign", stream)


def resample_kv_reassign(log_weights: torch.Tensor, B: int, N: int, tau: float, seed: int,
                         step: int, ancestors: torch.Tensor, ess: torch.Tensor,
                         resampled: torch.Tensor, block_tables: torch.Tensor, block_size: int,
                         seq_len: int, reserve_tokens: int, refcounts: torch.Tensor,
                         free_list: torch.Tensor, free_top: torch.Tensor, cow: torch.Tensor,
                         cow_count: torch.Tensor, status: torch.Tensor, workspace: torch.Tensor,
                         stream=None) -> None:
    """smcsd_resample_kv_reassign: resample then kv_reassign in one launch fewer."""
    if block_tables.dim() != 2 or block_tables.shape[0] != B * N:
        raise SmcsdError("block_tables must be [B*N, M_cap]")
    M_cap = block_tables.shape[1]
    P = refcounts.numel()
    rc = _L().smcsd_resample_kv_reassign(
        _dev(log_weights, "log_weights", torch.float32, B * N), B, N, float(tau),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _dev(ancestors, "ancestors", torch.int32, B * N), _dev(ess, "ess", torch.float32, B),
        _dev(resampled, "resampled", torch.int32, B),
        _dev(block_tables, "block_tables", torch.int32), M_cap, block_size, int(seq_len),
        reserve_tokens, _dev(refcounts, "refcounts", torch.int32),
        _dev(free_list, "free_list", torch.int32, P), _dev(free_top, "free_top", torch.int32, 1), P,
        _dev(cow, "cow", torch.int32, 3 * B * N), _dev(cow_count, "cow_count", torch.int32, 1),
        _dev(status, "status", torch.int32, 1), _dev(workspace, "workspace", torch.uint8),
        workspace.numel(), _stream(stream))
    _check(rc, "smcsd_resample_kv_reassign")
    _debug_kv_check(block_tables, block_size, seq_len, reserve_tokens, refcounts, free_list,
                    free_top, "smcsd_resample_kv_reassign", stream)


def step(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: Optional[torch.Tensor],
         B: int, N: int, K: int, V: int, temperature: float, alpha: float, mode: int, tau: float,
         seed: int, step: int, log_weights: torch.Tensor, out_tokens: torch.Tensor,
         ancestors: torch.Tensor, ess: torch.Tensor, resampled: torch.Tensor,
         block_tables: torch.Tensor, block_size: int, seq_len: int, reserve_tokens: int,
         refcounts: torch.Tensor, free_list: torch.Tensor, free_top: torch.Tensor,
         cow: torch.Tensor, cow_count: torch.Tensor, status: torch.Tensor,
         verify_workspace: torch.Tensor, kv_workspace: torch.Tensor, out_num_tokens=None,
         out_logp=None, out_logq=None, out_lse=None, logq_in=None,
         row_stride: Optional[int] = None, stream=None) -> None:
    """smcsd_step: smcsd_verify (MODE_SMC or MODE_SMC_RACE) then smcsd_resample_kv_reassign
    in one call (the same bits); seq_len is the length after this round's K+1 tokens."""
    if target.dtype not in _DT:
        raise SmcsdError("logits must be bfloat16 or float32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B * N:
        raise SmcsdError("block_tables must be [B*N, M_cap]")
    rs = V if row_stride is None else int(row_stride)
    S = B * N
    M_cap = block_tables.shape[1]
    P = refcounts.numel()
    tp = _dev(target, "target", target.dtype, S * (K + 1) * rs - (rs - V) if S else 0)
    dp = _dev(draft, "draft", target.dtype, S * K * rs - (rs - V) if S and K else 0) \
        if K > 0 and (draft is not None or logq_in is None) else None
    xp = _dev(draft_tokens, "draft_tokens", torch.int32, S * K) if K > 0 else None
    rc = _L().smcsd_step(
        tp, dp, _DT[target.dtype], rs, xp, B, N, K, V, float(temperature), float(alpha), mode,
        float(tau), int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _dev(logq_in, "logq_in", torch.float32, S * K),
        _dev(log_weights, "log_weights", torch.float32, S),
        _dev(out_tokens, "out_tokens", torch.int32, S * (K + 1)),
        _dev(out_num_tokens, "out_num_tokens", torch.int32, S),
        _dev(out_logp, "out_logp", torch.float32, S * (K + 1)),
        _dev(out_logq, "out_logq", torch.float32, S * K),
        _dev(out_lse, "out_lse", torch.float32, S * (2 * K + 1)),
        _dev(ancestors, "ancestors", torch.int32, S), _dev(ess, "ess", torch.float32, B),
        _dev(resampled, "resampled", torch.int32, B),
        _dev(block_tables, "block_tables", torch.int32), M_cap, block_size, int(seq_len),
        reserve_tokens, _dev(refcounts, "refcounts", torch.int32),
        _dev(free_list, "free_list", torch.int32, P), _dev(free_top, "free_top", torch.int32, 1), P,
        _dev(cow, "cow", torch.int32, 3 * S), _dev(cow_count, "cow_count", torch.int32, 1),
        _dev(status, "status", torch.int32, 1),
        _dev(verify_workspace, "verify_workspace", torch.uint8), verify_workspace.numel(),
        _dev(kv_workspace, "kv_workspace", torch.uint8), kv_workspace.numel(), _stream(stream))
    _check(rc, "smcsd_step")
    _debug_kv_check(block_tables, block_size, seq_len, reserve_tokens, refcounts, free_list,
                    free_top, "smcsd_step", stream)


def kv_check(block_tables: torch.Tensor, slots: int, refcounts: torch.Tensor,
             free_list: torch.Tensor, free_top: torch.Tensor, violations: torch.Tensor,
             status: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """smcsd_kv_check: violations [KV_CHECK_KINDS] int32 receives the counts (KV_CHECK_NAMES);
    workspace from alloc_workspace(OP_KV_CHECK, 0, 0, P=P)."""
    if block_tables.dim() != 2:
        raise SmcsdError("block_tables must be [S, M_cap]")
    S, M_cap = block_tables.shape
    P = refcounts.numel()
    rc = _L().smcsd_kv_check(
        _dev(block_tables, "block_tables", torch.int32), S, M_cap, int(slots),
        _dev(refcounts, "refcounts", torch.int32), _dev(free_list, "free_list", torch.int32, P),
        _dev(free_top, "free_top", torch.int32, 1), P,
        _dev(violations, "violations", torch.int32, KV_CHECK_KINDS),
        _dev(status, "status", torch.int32, 1), _dev(workspace, "workspace", torch.uint8),
        workspace.numel(), _stream(stream))
    _check(rc, "smcsd_kv_check")


def _debug_kv_check(block_tables, block_size, seq_len, reserve_tokens, refcounts, free_list,
                    free_top, what, stream):
    """With SMCSD_DEBUG_CHECK=1 in the environment: smcsd_kv_check after a KV call, waited
    for, raising SmcsdError on any violation (debug runs only: it synchronises the stream)."""
    if os.environ.get("SMCSD_DEBUG_CHECK") != "1":
        return
    dev = block_tables.device
    P = refcounts.numel()
    ws = alloc_workspace(OP_KV_CHECK, 0, 0, P=P, device=dev)
    viol = torch.zeros(KV_CHECK_KINDS, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    slots = -(-(int(seq_len) + int(reserve_tokens)) // int(block_size))
    kv_check(block_tables, slots, refcounts, free_list, free_top, viol, st, ws, stream)
    counts = viol.cpu().tolist()
    if any(counts):
        raise SmcsdError("%s left an inconsistent KV state: %s" % (what, ", ".join(
            "%s: %d" % (n, c) for n, c in zip(KV_CHECK_NAMES, counts) if c)))


def philox4x32_10(counters: torch.Tensor, keys: torch.Tensor, out: torch.Tensor, stream=None):
    """Device Philox4x32-10 blocks: counters [n, 4], keys [n, 2] -> out [n, 4] (int32 views)."""
    n = counters.shape[0]
    rc = _L().smcsd_philox4x32_10(_dev(counters, "counters", torch.int32, 4 * n),
                                  _dev(keys, "keys", torch.int32, 2 * n), n,
                                  _dev(out, "out", torch.int32, 4 * n), _stream(stream))
    _check(rc, "smcsd_philox4x32_10")


def stream_read(buf: torch.Tensor, tile_xor: torch.Tensor, stream=None):
    """Reads every byte of the contiguous device tensor `buf` once (16-byte aligned, a
    multiple of 16 bytes) and writes the XOR of each STREAM_READ_TILE_BYTES tile's 32-bit
    words to tile_xor (int32, one word per tile): the achievable HBM read rate that the LSE
    pass is compared with."""
    if not isinstance(buf, torch.Tensor) or not buf.is_cuda or not buf.is_contiguous():
        raise SmcsdError("buf must be a contiguous device tensor")
    nbytes = buf.numel() * buf.element_size()
    ntiles = -(-nbytes // STREAM_READ_TILE_BYTES)
    rc = _L().smcsd_stream_read(ctypes.c_void_p(buf.data_ptr()), nbytes,
                                _dev(tile_xor, "tile_xor", torch.int32, ntiles), _stream(stream))
    _check(rc, "smcsd_stream_read")


# ---------------------------------------------------------------------------------------
# The serving operators around a round.  A call of theirs can be as short as a kernel of a
# few microseconds, so their checks take the common case in one condition per tensor.
# ---------------------------------------------------------------------------------------
def _addr(t, name: str, dtype, n: int, dev: int) -> Optional[int]:
    """The address of a contiguous tensor of `dtype` with at least n elements on device `dev`
    (None for None)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and t.numel() >= n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name, dtype, n)
    raise SmcsdError("%s is on device %d, the call runs on device %d" % (name, t.get_device(), dev))


def _need(t, name: str, dtype, n: int, dev: int) -> int:
    if t is None:
        raise SmcsdError("%s is missing" % name)
    return _addr(t, name, dtype, n, dev)


def _device_of(t, name: str) -> int:
    """The index of the device that holds t, which must be the current one: kernels are
    enqueued there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SmcsdError("%s must be a device tensor" % name)
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise SmcsdError("%s is on device %d, the current device is %d" %
                         (name, dev, torch.cuda.current_device()))
    return dev


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _queue(stream, dev: int) -> int:
    """The handle of `stream`, or of device `dev`'s current stream."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    if stream.device_index != dev:
        raise SmcsdError("the stream is on device %d, the tensors on device %d" %
                         (stream.device_index, dev))
    return stream.cuda_stream


def _tables(block_tables, rows: Optional[int], dev: int):
    """(address, rows, M_cap) of block tables [rows, M_cap]."""
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise SmcsdError("block_tables must be [S, M_cap]")
    n, m = block_tables.shape
    if rows is not None and n != rows:
        raise SmcsdError("block_tables must be [%d, M_cap]" % rows)
    return _addr(block_tables, "block_tables", torch.int32, 0, dev), n, m


def kv_fork(forked: torch.Tensor, B: int, N: int, block_tables: torch.Tensor,
            refcounts: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    """smcsd_kv_fork: the tables of the prompts with forked[b] != 0 from their particle 0's
    (admission of a prefilled prompt).  block_tables [B*N, M_cap], refcounts [P] in/out."""
    dev = _device_of(status, "status")
    T, _, M_cap = _tables(block_tables, B * N, dev)
    i32 = torch.int32
    rc = _L().smcsd_kv_fork(_need(forked, "forked", i32, B, dev), B, N, T, M_cap,
                            _need(refcounts, "refcounts", i32, 1, dev), refcounts.numel(),
                            _need(status, "status", i32, 1, dev), _queue(stream, dev))
    if rc:
        _check(rc, "smcsd_kv_fork")


def kv_free(freed: torch.Tensor, block_tables: torch.Tensor, refcounts: torch.Tensor,
            free_list: torch.Tensor, free_top: torch.Tensor, status: torch.Tensor,
            workspace: torch.Tensor, stream=None) -> None:
    """smcsd_kv_free: the sequences with freed[g] != 0 drop their blocks.  workspace from
    alloc_workspace(OP_KV_FREE, 0, 0, P=P)."""
    dev = _device_of(status, "status")
    T, S, M_cap = _tables(block_tables, None, dev)
    i32 = torch.int32
    R = _need(refcounts, "refcounts", i32, 1, dev)
    P = refcounts.numel()
    rc = _L().smcsd_kv_free(
        _need(freed, "freed", i32, S, dev), S, T, M_cap, R, _need(free_list, "free_list", i32, P, dev),
        _need(free_top, "free_top", i32, 1, dev), P, _need(status, "status", i32, 1, dev),
        _need(workspace, "workspace", torch.uint8, 0, dev), workspace.numel(), _queue(stream, dev))
    if rc:
        _check(rc, "smcsd_kv_free")
    _debug_kv_check(block_tables, 1, M_cap, 0, refcounts, free_list, free_top, "smcsd_kv_free",
                    stream)


def kv_compact(block_tables: torch.Tensor, block_size: int, refcounts: torch.Tensor,
               free_list: torch.Tensor, free_top: torch.Tensor, moves: torch.Tensor,
               move_count: torch.Tensor, status: torch.Tensor, workspace: torch.Tensor,
               stream=None) -> None:
    """smcsd_kv_compact: live blocks to the lowest ids; moves [P // 2, 3] and move_count are
    what kv_copy then runs on the data.  workspace from alloc_workspace(OP_KV_COMPACT, 0, 0,
    P=P)."""
    dev = _device_of(status, "status")
    T, S, M_cap = _tables(block_tables, None, dev)
    i32 = torch.int32
    R = _need(refcounts, "refcounts", i32, 1, dev)
    P = refcounts.numel()
    rc = _L().smcsd_kv_compact(
        T, S, M_cap, int(block_size), R, _need(free_list, "free_list", i32, P, dev),
        _need(free_top, "free_top", i32, 1, dev), P, _need(moves, "moves", i32, 3 * (P // 2), dev),
        _need(move_count, "move_count", i32, 1, dev), _need(status, "status", i32, 1, dev),
        _need(workspace, "workspace", torch.uint8, 0, dev), workspace.numel(), _queue(stream, dev))
    if rc:
        _check(rc, "smcsd_kv_compact")
    _debug_kv_check(block_tables, 1, M_cap, 0, refcounts, free_list, free_top, "smcsd_kv_compact",
                    stream)


def _pages(t, name: str, dtype, dev: int):
    """(shape, strides) of a cache seen as [P, block_size, Hkv, D]: rows of D contiguous
    elements, any strides between them."""
    try:
        shape, strides = t.shape, t.stride()
        if len(shape) == 4 and (dtype is None or t.dtype is dtype) and t.get_device() == dev and (
                strides[3] == 1 or shape[3] == 1):
            return shape, strides
    except AttributeError:
        pass
    _dev(t, name, dtype, contiguous=False)
    if t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] != 1):
        raise SmcsdError("%s must be [P, block_size, Hkv, D] with contiguous rows of D" % name)
    raise SmcsdError("%s is on device %d, the call runs on device %d" % (name, t.get_device(), dev))


def kv_copy(caches: Sequence[torch.Tensor], moves: torch.Tensor, count: torch.Tensor,
            status: torch.Tensor, stream=None) -> None:
    """smcsd_kv_copy: runs a list of (source, destination, tokens) entries, as kv_reassign
    (copy-on-write) and kv_compact write them, on every cache.  caches: tensors seen as
    [P, block_size, Hkv, D], all of one shape, type and layout; a [P, Hkv, block_size, D]
    cache is passed as its transpose(1, 2)."""
    n = len(caches)
    if n > KV_COPY_MAX_CACHES:
        raise SmcsdError("at most %d caches a call" % KV_COPY_MAX_CACHES)
    dev = _device_of(status, "status")
    if not isinstance(moves, torch.Tensor) or moves.dim() != 2 or moves.shape[1] != 3:
        raise SmcsdError("moves must be [capacity, 3]")
    i32 = torch.int32
    mp, cp, sp = (_need(moves, "moves", i32, 0, dev), _need(count, "count", i32, 1, dev),
                  _need(status, "status", i32, 1, dev))
    if n == 0:
        return
    shape, strides = _pages(caches[0], "caches[0]", None, dev)
    dtype = caches[0].dtype
    ptrs = (ctypes.c_void_p * n)()
    for i, c in enumerate(caches):
        if _pages(c, "caches[%d]" % i, dtype, dev) != (shape, strides):
            raise SmcsdError("caches must have one shape and layout")
        ptrs[i] = c.data_ptr()
    P, bs, H, D = shape
    e = caches[0].element_size()
    page, token, head = (s * e for s in strides[:3])
    # a token's heads in one piece, or a head's tokens
    if (H == 1 or head == D * e) and (bs == 1 or token == H * D * e):
        segments, seg, tok = 1, 0, H * D * e
    elif bs == 1 or token == D * e:
        segments, seg, tok = H, head, D * e
    else:
        raise SmcsdError("a token's heads, or a head's tokens, must be contiguous")
    rc = _L().smcsd_kv_copy(ptrs, n, page, segments, seg, tok, bs, mp, cp, moves.shape[0], P, sp,
                            _queue(stream, dev))
    if rc:
        _check(rc, "smcsd_kv_copy")


def _heads(t, name: str, S: int, R: int, D: int, dtype, dev: int):
    """(address, heads, stride between tokens) of [S, R, H, D] with each token's heads
    contiguous."""
    try:
        s, r, H, d = t.shape
        a, tok, h, e = t.stride()
        if R == 1:
            tok = a if S > 1 else H * D
        if s == S and r == R and d == D and t.dtype is dtype and t.get_device() == dev and (
                h == D or H == 1) and (e == 1 or D == 1) and (a == R * tok or S == 1):
            return t.data_ptr(), H, tok
    except (AttributeError, ValueError):
        pass
    _dev(t, name, dtype, contiguous=False)
    if t.dim() != 4 or t.shape[0] != S or t.shape[1] != R or t.shape[3] != D:
        raise SmcsdError("%s must be [%d, %d, heads, %d]" % (name, S, R, D))
    if t.get_device() != dev:
        raise SmcsdError("%s is on device %d, the call runs on device %d" % (name, t.get_device(), dev))
    raise SmcsdError("%s must hold each token's heads contiguously, tokens one stride apart" % name)


def _cache_pair(k_cache, v_cache, dtype, D: int, dev: int):
    """(P, block_size, Hkv, strides of page, token and head) of two caches of one layout."""
    kv = _pages(k_cache, "k_cache", dtype, dev)
    if _pages(v_cache, "v_cache", dtype, dev) != kv:
        raise SmcsdError("k_cache and v_cache must have one shape and layout")
    (P, bs, H, d), (page, token, head, _) = kv
    if d != D:
        raise SmcsdError("the caches' heads must have %d elements" % D)
    # the stride of an axis of one entry says nothing
    return P, bs, H, page if P > 1 else D, token if bs > 1 else D, head if H > 1 else D


def _kv_dtype(q):
    try:
        return _DT_KV[q.dtype]
    except (AttributeError, KeyError):
        raise SmcsdError("queries, keys and values must be bfloat16 or float16") from None


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, ctx_lens: torch.Tensor,
                 block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 q_out: torch.Tensor, status: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 cos_sin: Optional[torch.Tensor] = None, interleaved: bool = False,
                 positions: Optional[torch.Tensor] = None,
                 num_nodes: Optional[torch.Tensor] = None, stream=None) -> None:
    """smcsd_qk_norm_rope.  q [S, R, Hq, D], k, v [S, R, Hkv, D] (bf16 or f16; views into a
    fused projection will do), q_out [S, R, Hq, D]; k_cache, v_cache seen as [P, block_size,
    Hkv, D] with any strides between rows of D; cos_sin [max_pos, rot_dim] fp32 (None: no
    rotation), positions [S, R] int32 (None: ctx_lens + j), num_nodes [S] int32."""
    dev = _device_of(status, "status")
    dt = _kv_dtype(q)
    dtype = q.dtype
    if q.dim() != 4:
        raise SmcsdError("q must be [S, R, heads, D]")
    S, R, Hq, D = q.shape
    qp, _, qs = _heads(q, "q", S, R, D, dtype, dev)
    kp, Hkv, ks = _heads(k, "k", S, R, D, dtype, dev)
    vp, Hv, vs = _heads(v, "v", S, R, D, dtype, dev)
    P, bs, H, page, token, head = _cache_pair(k_cache, v_cache, dtype, D, dev)
    if Hv != Hkv or H != Hkv:
        raise SmcsdError("k, v and the caches must have the same heads (%d, %d, %d)" % (Hkv, Hv, H))
    max_pos, rot = 0, 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise SmcsdError("cos_sin must be [max_pos, rot_dim]")
        max_pos, rot = cos_sin.shape
    T, _, M_cap = _tables(block_tables, S, dev)
    i32 = torch.int32
    rc = _L().smcsd_qk_norm_rope(
        qp, kp, vp, dt, qs, ks, vs, S, R, Hq, Hkv, D, _addr(q_weight, "q_weight", dtype, D, dev),
        _addr(k_weight, "k_weight", dtype, D, dev), eps, _addr(cos_sin, "cos_sin", torch.float32, 0, dev),
        max_pos, rot, 1 if interleaved else 0, _addr(positions, "positions", i32, S * R, dev),
        _need(ctx_lens, "ctx_lens", i32, S, dev), _addr(num_nodes, "num_nodes", i32, S, dev), T, M_cap,
        bs, P, k_cache.data_ptr(), v_cache.data_ptr(), page, token, head,
        _need(q_out, "q_out", dtype, S * R * Hq * D, dev), _need(status, "status", i32, 1, dev),
        _queue(stream, dev))
    if rc:
        _check(rc, "smcsd_qk_norm_rope")


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, ctx_lens: torch.Tensor, B: int, N: int,
                   scale: float, out: torch.Tensor, status: torch.Tensor, workspace: torch.Tensor,
                   tree_mask: Optional[torch.Tensor] = None,
                   num_nodes: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   max_len: int = 0, stream=None) -> None:
    """smcsd_tree_attention.  q [B*N, R, Hq, D] (bf16 or f16); k_cache, v_cache seen as [P,
    block_size, Hkv, D] with any strides between rows of D; out [B*N, R, Hq, D]; tree_mask
    [B*N, R] int64 (bit j of row i: node i sees node j; None: a chain); lse [B*N, R, Hq]
    fp32.  workspace from alloc_workspace(OP_TREE_ATTN, B, N, K=R, V=Hq * D, P=Hkv)."""
    dev = _device_of(status, "status")
    dt = _kv_dtype(q)
    dtype = q.dtype
    if q.dim() != 4 or q.shape[0] != B * N:
        raise SmcsdError("q must be [B*N, R, Hq, D]")
    S, R, Hq, D = q.shape
    qp, _, qs = _heads(q, "q", S, R, D, dtype, dev)
    P, bs, Hkv, page, token, head = _cache_pair(k_cache, v_cache, dtype, D, dev)
    T, _, M_cap = _tables(block_tables, S, dev)
    i32 = torch.int32
    rc = _L().smcsd_tree_attention(
        qp, dt, qs, k_cache.data_ptr(), v_cache.data_ptr(), page, token, head, T, M_cap, bs, P,
        _need(ctx_lens, "ctx_lens", i32, S, dev), _addr(num_nodes, "num_nodes", i32, S, dev),
        _addr(tree_mask, "tree_mask", torch.int64, S * R, dev), B, N, R, Hq, Hkv, D, scale,
        max_len, _need(out, "out", dtype, S * R * Hq * D, dev),
        _addr(lse, "lse", torch.float32, S * R * Hq, dev), _need(status, "status", i32, 1, dev),
        _need(workspace, "workspace", torch.uint8, 0, dev), workspace.numel(), _queue(stream, dev))
    if rc:
        _check(rc, "smcsd_tree_attention")


def token_logprobs(logits: torch.Tensor, n: int, V: int, temperature: float, status: torch.Tensor,
                   workspace: torch.Tensor, tokens: Optional[torch.Tensor] = None,
                   out_logp: Optional[torch.Tensor] = None,
                   out_entropy: Optional[torch.Tensor] = None,
                   out_lse: Optional[torch.Tensor] = None,
                   top_ids: Optional[torch.Tensor] = None,
                   top_logp: Optional[torch.Tensor] = None, row_stride: Optional[int] = None,
                   stream=None) -> None:
    """smcsd_token_logprobs on logits [n, row_stride] (bf16 or fp32): tokens [n, C] int32 and
    out_logp [n, C]; out_entropy, out_lse [n]; top_ids and top_logp [n, k] (k = their second
    extent).  workspace from alloc_workspace(OP_LOGPROBS, n, 1, K=k, V=V)."""
    dev = _device_of(status, "status")
    dtype = getattr(logits, "dtype", None)
    if dtype not in _DT:
        raise SmcsdError("logits must be bfloat16 or float32")
    rs = V if row_stride is None else int(row_stride)
    C, k = 0, 0
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != n:
            raise SmcsdError("tokens must be [n, C]")
        C = tokens.shape[1]
    if top_ids is not None:
        if top_ids.dim() != 2 or top_ids.shape[0] != n:
            raise SmcsdError("top_ids must be [n, k]")
        k = top_ids.shape[1]
    if top_logp is not None:
        if top_logp.dim() != 2 or top_logp.shape[0] != n or (top_ids is not None and top_logp.shape[1] != k):
            raise SmcsdError("top_logp must be [n, k], with the k of top_ids")
        k = top_logp.shape[1]
    i32, f32 = torch.int32, torch.float32
    rc = _L().smcsd_token_logprobs(
        _need(logits, "logits", dtype, n * rs - (rs - V) if n else 0, dev), _DT[dtype], rs, n, V,
        temperature, _addr(tokens, "tokens", i32, n * C, dev), C, k,
        _addr(out_logp, "out_logp", f32, n * C, dev), _addr(out_entropy, "out_entropy", f32, n, dev),
        _addr(out_lse, "out_lse", f32, n, dev), _addr(top_ids, "top_ids", i32, n * k, dev),
        _addr(top_logp, "top_logp", f32, n * k, dev), _need(status, "status", i32, 1, dev),
        _need(workspace, "workspace", torch.uint8, 0, dev), workspace.numel(), _queue(stream, dev))
    if rc:
        _check(rc, "smcsd_token_logprobs")
