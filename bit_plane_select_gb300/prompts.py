"""Whole prompts, a key/value cache held in 4 bits, and scoring (declared in
``include/trit.h``).

Prompts of different lengths come as packed rows: their keys and values are
quantised into pages (``trit_kv4_append``), read back with those of earlier
turns (``trit_kv4_read``) and attended to (``trit_attn_prompt``); single tokens and
drafts attend to the pages themselves (``trit_attn_paged4``); ``trit_logprobs`` scores
given tokens.  Calls take jobs, as those of ``serving`` do.
"""
from __future__ import annotations

import ctypes

import torch

from . import lib
from .serving import (_DTYPE, ROPE_PAIRS, KvBatch, Rope, TritKvBatch, _f32, _i32, _i64, _Job, _p, _ptr, _token_rows,
                      _u32, _whole, _workspace)

__all__ = ["Kv4Cache", "Append4Job", "Read4Job", "Attn4Job", "PromptJob", "LogprobJob", "TritKv4Cache",
           "TritKv4AppendJob", "TritKv4ReadJob", "TritAttn4Job", "TritPromptJob", "TritLogprobJob", "trit_kv4_append",
           "trit_kv4_read", "trit_attn_paged4", "trit_attn4_workspace_bytes", "trit_attn_prompt", "trit_logprobs",
           "KV4_GROUP", "MAX_TOP"]

KV4_GROUP = 64
MAX_TOP = 64

_HALF = (torch.bfloat16, torch.float16)


class TritKv4Cache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("page_stride", _i64),
                ("head_stride", _i64), ("slot_stride", _i64), ("pages", _i32), ("heads", _i32),
                ("page_size", _i32), ("head_dim", _i32), ("reserved", _i64)]


class TritKv4AppendJob(ctypes.Structure):
    _fields_ = [("cache", TritKv4Cache), ("batch", TritKvBatch), ("q", _p), ("k", _p), ("v", _p),
                ("q_out", _p), ("starts", _p), ("cos", _p), ("sin", _p), ("q_gain", _p), ("k_gain", _p),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("rows", _i64), ("max_pos", _i64),
                ("eps", _f32), ("q_heads", _i32), ("rot", _i32), ("src_dtype", _i32), ("dtype", _i32),
                ("flags", _u32)]


class TritKv4ReadJob(ctypes.Structure):
    _fields_ = [("cache", TritKv4Cache), ("batch", TritKvBatch), ("k", _p), ("v", _p), ("starts", _p),
                ("rows", _i64), ("dtype", _i32), ("flags", _u32)]


class TritAttn4Job(ctypes.Structure):
    _fields_ = [("cache", TritKv4Cache), ("batch", TritKvBatch), ("q", _p), ("out", _p), ("lse", _p),
                ("workspace", _p), ("workspace_bytes", _i64), ("q_stride", _i64), ("scale", _f32),
                ("q_heads", _i32), ("dtype", _i32), ("out_dtype", _i32), ("flags", _u32), ("reserved", _i32)]


class TritPromptJob(ctypes.Structure):
    _fields_ = [("q", _p), ("k", _p), ("v", _p), ("out", _p), ("lse", _p), ("q_starts", _p), ("k_starts", _p),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("q_rows", _i64), ("k_rows", _i64),
                ("B", _i32), ("q_heads", _i32), ("heads", _i32), ("head_dim", _i32), ("dtype", _i32),
                ("out_dtype", _i32), ("scale", _f32), ("flags", _u32)]


class TritLogprobJob(ctypes.Structure):
    _fields_ = [("logits", _p), ("tokens", _p), ("logprob", _p), ("entropy", _p), ("top_tokens", _p),
                ("top_logprobs", _p), ("stride", _i64), ("rows", _i64), ("V", _i64), ("top_n", _i32),
                ("dtype", _i32), ("flags", _u32), ("reserved", _i32)]


class Kv4Cache:
    """One layer's paged cache in 4 bits: codes k and v [pages, heads, page_size,
    D/2] uint8 (columns 2i and 2i + 1 in the low and high half of byte i) and pairs
    k_scale and v_scale [pages, heads, page_size, D/64, 2] fp16, (s, z) of each 64
    columns: code c stands for s c + z.  All four lie alike (contiguous, or permuted
    from [pages, page_size, heads, ...])."""

    def __init__(self, k, v, k_scale, v_scale):
        if k.dim() != 4:
            raise ValueError("k must be [pages, heads, page_size, D/2]")
        pages, heads, page_size, half = k.shape
        groups = 2 * half // KV4_GROUP
        shape = (pages, heads, page_size, groups, 2)
        pointers = [_ptr(k, "k", (torch.uint8,)), _ptr(v, "v", (torch.uint8,), k.shape)]
        pointers += [_ptr(s, n, (torch.float16,), shape) for s, n in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        # strides in vectors; those of a dimension of one entry are of no account
        strides = [0 if n == 1 or not half else st // half for n, st in zip(k.shape[:3], k.stride()[:3])]
        for t, n, w in ((k, "k", half), (v, "v", half), (k_scale, "k_scale", 2 * groups), (v_scale, "v_scale", 2 * groups)):
            if any(size > 1 and st != s * w for size, st, s in zip(t.shape[:3], t.stride()[:3], strides)):
                raise ValueError(f"{n}: the cache's vectors must lie alike in all four tensors, each whole")
            if t.dim() == 5 and groups > 1 and t.stride(3) != 2:
                raise ValueError(f"{n}: a vector's pairs must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale, self.head_dim = k, v, k_scale, v_scale, 2 * half
        self.c = TritKv4Cache(*pointers, *strides, pages, heads, page_size, 2 * half, 0)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, head_dim: int, device="cuda"):
        """A cache of zeros."""
        codes = [torch.zeros((pages, heads, page_size, head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
        pairs = [torch.zeros((pages, heads, page_size, head_dim // KV4_GROUP, 2), dtype=torch.float16, device=device)
                 for _ in range(2)]
        return cls(*codes, *pairs)


def _packed_rows(t, name, dtypes, heads, D):
    """[rows, heads, D] or [rows, heads * D] with any row stride -> (pointer, rows, stride)."""
    if t.dim() == 2 and t.shape[1] == heads * D:
        t = t.unflatten(1, (heads, D))
    if t.dim() != 3 or tuple(t.shape[1:]) != (heads, D):
        raise ValueError(f"{name} must be [rows, {heads}, {D}] or [rows, {heads * D}]")
    if heads > 1 and t.stride(1) != D:
        raise ValueError(f"{name}: a row's heads must be contiguous")
    return _ptr(t, name, dtypes), t.shape[0], (t.stride(0) if t.shape[0] > 1 else heads * D)


class Append4Job(_Job):
    """The arguments of trit_kv4_append: a Kv4Cache, batch, rope, q (None: keys and
    values only), k, v (fp32 or the type of q_out; token rows may be strided views)
    and q_out of bf16 or fp16.  Without starts the rows are [B, T, ...] and q_out is
    [B, T, Hq, D]; with starts [B + 1] int32 they are packed, [rows, ...], and q_out is
    [rows, Hq, D]."""

    def __init__(self, cache: Kv4Cache, batch: KvBatch, rope: Rope, q, k, v, q_out, starts=None):
        B, T, D, heads = batch.B, batch.T, cache.head_dim, cache.k.shape[1]
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out come together")
        src = k.dtype
        dt = q_out.dtype if q_out is not None else torch.bfloat16 if src is torch.float32 else src
        if dt not in _HALF or src not in (torch.float32, dt):
            raise ValueError("q_out must be bfloat16 or float16, and k float32 or the same")
        rows = B * T if starts is None else k.shape[0]

        def of(t, name, h):
            if starts is None:
                return _token_rows(t, name, (src,), B, T, h, D)
            p, n, s = _packed_rows(t, name, (src,), h, D)
            if n != rows:
                raise ValueError(f"{name} must have {rows} rows")
            return p, s
        hq, qo, qs = 0, None, (None, 0)
        if q is not None:
            hq = q.numel() // max(1, rows * D)
            qs = of(q, "q", hq)
            qo = _whole(q_out, "q_out", (dt,), (B, T, hq, D) if starts is None else (rows, hq, D))
        (k_p, k_s), (v_p, v_s) = of(k, "k", heads), of(v, "v", heads)
        f = (torch.float32,)
        c = TritKv4AppendJob(cache.c, batch.c, qs[0], k_p, v_p, qo,
                             _whole(starts, "starts", (torch.int32,), (B + 1,), True), rope.p_cos, rope.p_sin,
                             _whole(rope.q_gain, "q_gain", f, (D,), True), _whole(rope.k_gain, "k_gain", f, (D,), True),
                             qs[1], k_s, v_s, rows, rope.max_pos, rope.eps, hq, rope.rot, _DTYPE[src], _DTYPE[dt],
                             ROPE_PAIRS if rope.pairs else 0)
        self.q_out = q_out
        self._bind("trit_kv4_append", k.device, c, cache, batch, rope, q, k, v, q_out, starts)


def trit_kv4_append(job: Append4Job, err_flag: torch.Tensor, stream=None):
    """Norm and rotate the new tokens' q and k, write q to q_out, quantise k and v into
    their cache slots (one launch).  Returns q_out."""
    job._call(err_flag, stream)
    return job.q_out


class Read4Job(_Job):
    """The arguments of trit_kv4_read: a Kv4Cache, batch (its tables, lens and prefix),
    k and v [rows, heads, D] bf16 or fp16, and starts [B + 1] int32, the first row
    of each sequence's prefix_len + lens[b] keys."""

    def __init__(self, cache: Kv4Cache, batch: KvBatch, k, v, starts):
        shape = (k.shape[0], cache.k.shape[1], cache.head_dim)
        c = TritKv4ReadJob(cache.c, batch.c, _whole(k, "k", _HALF, shape), _whole(v, "v", (k.dtype,), shape),
                           _whole(starts, "starts", (torch.int32,), (batch.B + 1,)), shape[0], _DTYPE[k.dtype], 0)
        self.k, self.v = k, v
        self._bind("trit_kv4_read", k.device, c, cache, batch, k, v, starts)


def trit_kv4_read(job: Read4Job, err_flag: torch.Tensor, stream=None):
    """Write the keys and values that the sequences see as packed rows.  Returns (k, v)."""
    job._call(err_flag, stream)
    return job.k, job.v


def trit_attn4_workspace_bytes(job: TritAttn4Job) -> int:
    """Bytes of the workspace of a job (its pointers are not read); -1 for
    sizes that are not supported."""
    return int(lib().trit_attn4_workspace_bytes(ctypes.byref(job)))


class Attn4Job(_Job):
    """The arguments of trit_attn_paged4: a Kv4Cache, batch, q (bf16 or fp16; token rows
    may be strided views) and out [B, T, Hq, D] (q's type or fp32), optionally lse
    [B, T, Hq] fp32; scale defaults to 1/sqrt(D).  The workspace is made here (or given:
    zeroed once, at least trit_attn4_workspace_bytes; jobs of any sizes may share one, one
    call at a time)."""

    def __init__(self, cache: Kv4Cache, batch: KvBatch, q, out, lse=None, scale=None, workspace=None):
        B, T, D, dt = batch.B, batch.T, cache.head_dim, q.dtype
        hq = q.numel() // max(1, B * T * D)
        q_p, q_s = _token_rows(q, "q", _HALF, B, T, hq, D)
        c = TritAttn4Job(cache.c, batch.c, q_p, _whole(out, "out", (dt, torch.float32), (B, T, hq, D)),
                         _whole(lse, "lse", (torch.float32,), (B, T, hq), True), None, 0, q_s,
                         float(D ** -0.5 if scale is None else scale), hq, _DTYPE[dt], _DTYPE[out.dtype], 0, 0)
        need = trit_attn4_workspace_bytes(c)
        if need < 0:
            raise ValueError("sizes outside the supported range")
        if workspace is None:
            workspace = _workspace(need, q.device)
        c.workspace = _whole(workspace, "workspace", (torch.uint8,), workspace.shape)
        c.workspace_bytes = workspace.numel()
        self.out, self.lse, self.workspace = out, lse, workspace
        self._bind("trit_attn_paged4", q.device, c, cache, batch, q, out, lse, workspace)


def trit_attn_paged4(job: Attn4Job, err_flag: torch.Tensor, stream=None):
    """Attention of the new tokens to the keys they see.  Returns out."""
    job._call(err_flag, stream)
    return job.out


class PromptJob(_Job):
    """The arguments of trit_attn_prompt: packed q [rows, Hq, D], k and v [keys, heads, D]
    (bf16 or fp16; rows may be strided views), out [rows, Hq, D] (their type or fp32),
    q_starts [B + 1] int32 and, where sequences have other keys than queries, k_starts
    [B + 1] int32; optionally lse [rows, Hq] fp32; scale defaults to 1/sqrt(D)."""

    def __init__(self, q, k, v, out, q_starts, k_starts=None, lse=None, scale=None):
        if q.dim() != 3 or k.dim() != 3:
            raise ValueError("q and k must be [rows, heads, D]")
        hq, D = q.shape[1:]
        heads, dt = k.shape[1], q.dtype
        q_p, q_rows, q_s = _packed_rows(q, "q", _HALF, hq, D)
        k_p, k_rows, k_s = _packed_rows(k, "k", (dt,), heads, D)
        v_p, v_rows, v_s = _packed_rows(v, "v", (dt,), heads, D)
        if v_rows != k_rows:
            raise ValueError("k and v must have as many rows")
        B, i32 = q_starts.numel() - 1, (torch.int32,)
        c = TritPromptJob(q_p, k_p, v_p, _whole(out, "out", (dt, torch.float32), (q_rows, hq, D)),
                          _whole(lse, "lse", (torch.float32,), (q_rows, hq), True), _whole(q_starts, "q_starts", i32, (B + 1,)),
                          _whole(k_starts, "k_starts", i32, (B + 1,), True), q_s, k_s, v_s, q_rows, k_rows, B, hq, heads, D,
                          _DTYPE[dt], _DTYPE[out.dtype], float(D ** -0.5 if scale is None else scale), 0)
        self.out, self.lse = out, lse
        self._bind("trit_attn_prompt", q.device, c, q, k, v, out, q_starts, k_starts, lse)


def trit_attn_prompt(job: PromptJob, err_flag: torch.Tensor, stream=None):
    """Causal attention of the packed prompts.  Returns out."""
    job._call(err_flag, stream)
    return job.out


class LogprobJob(_Job):
    """The arguments of trit_logprobs: logits [rows, V] (fp32, bf16 or fp16; rows may be
    strided), tokens [rows] int32 with logprob [rows] fp32 (-1: padding, 0), entropy [rows]
    fp32, top_tokens [rows, n] int32 with top_logprobs [rows, n] fp32; each pair, and
    entropy, may be None."""

    def __init__(self, logits, tokens=None, logprob=None, entropy=None, top_tokens=None, top_logprobs=None):
        if logits.dim() != 2 or logits.dtype not in _DTYPE:
            raise ValueError("logits must be [rows, V], float32, bfloat16 or float16")
        if (tokens is None) != (logprob is None) or (top_tokens is None) != (top_logprobs is None):
            raise ValueError("tokens and logprob, and top_tokens and top_logprobs, come together")
        rows, V = logits.shape
        n = 0 if top_tokens is None else top_tokens.shape[-1]
        f32, i32 = (torch.float32,), (torch.int32,)
        c = TritLogprobJob(_ptr(logits, "logits", (logits.dtype,)), _whole(tokens, "tokens", i32, (rows,), True),
                           _whole(logprob, "logprob", f32, (rows,), True), _whole(entropy, "entropy", f32, (rows,), True),
                           _whole(top_tokens, "top_tokens", i32, (rows, n), True),
                           _whole(top_logprobs, "top_logprobs", f32, (rows, n), True),
                           logits.stride(0) if rows > 1 else V, rows, V, n, _DTYPE[logits.dtype], 0, 0)
        self.outputs = logprob, entropy, top_tokens, top_logprobs
        self._bind("trit_logprobs", logits.device, c, logits, tokens, *self.outputs)


def trit_logprobs(job: LogprobJob, err_flag: torch.Tensor, stream=None):
    """Log probabilities of the tokens, entropies and the top alternatives.  Returns
    (logprob, entropy, top_tokens, top_logprobs)."""
    job._call(err_flag, stream)
    return job.outputs
