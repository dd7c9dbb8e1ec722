"""The decode step between the ternary products: a paged key/value cache with
its append, the attention that reads it, and the verification of drafted
tokens (declared in ``include/trit.h``).

A call takes a job -- the checked arguments and the workspace of one call site,
built once and used every step, as the prepared lists of the products are --
and launches on the current torch stream (or ``stream``).  Jobs hold their
tensors; a job must outlive the work enqueued from it.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, lib

__all__ = ["KvCache", "KvBatch", "Rope", "AppendJob", "AttnJob", "VerifyJob", "TritKvCache",
           "TritKvBatch", "TritKvAppendJob", "TritAttnJob", "TritVerifyJob", "trit_kv_append",
           "trit_attn_paged", "trit_attn_workspace_bytes", "trit_draft_verify", "ERR_INDEX", "ERR_EMPTY",
           "ROPE_PAIRS", "MAX_SEQUENCES"]

ERR_INDEX = 32
ERR_EMPTY = 64
ROPE_PAIRS = 1
MAX_SEQUENCES = 4096

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_p, _i64, _i32, _u32, _f32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32,
                              ctypes.c_float)


class TritKvCache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("page_stride", _i64), ("head_stride", _i64),
                ("slot_stride", _i64), ("pages", _i32), ("heads", _i32), ("page_size", _i32),
                ("head_dim", _i32), ("dtype", _i32), ("reserved", _i32)]


class TritKvBatch(ctypes.Structure):
    _fields_ = [("prefix_table", _p), ("table", _p), ("lens", _p), ("new_lens", _p),
                ("prefix_len", _i64), ("table_stride", _i64), ("prefix_pages", _i32),
                ("table_pages", _i32), ("B", _i32), ("T", _i32)]


class TritKvAppendJob(ctypes.Structure):
    _fields_ = [("cache", TritKvCache), ("batch", TritKvBatch), ("q", _p), ("k", _p), ("v", _p),
                ("q_out", _p), ("cos", _p), ("sin", _p), ("q_gain", _p), ("k_gain", _p),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("max_pos", _i64),
                ("eps", _f32), ("q_heads", _i32), ("rot", _i32), ("src_dtype", _i32),
                ("flags", _u32), ("reserved", _i32)]


class TritAttnJob(ctypes.Structure):
    _fields_ = [("cache", TritKvCache), ("batch", TritKvBatch), ("q", _p), ("out", _p),
                ("lse", _p), ("workspace", _p), ("workspace_bytes", _i64), ("q_stride", _i64),
                ("scale", _f32), ("q_heads", _i32), ("out_dtype", _i32), ("flags", _u32)]


class TritVerifyJob(ctypes.Structure):
    _fields_ = [("p", _p), ("q", _p), ("draft", _p), ("n_draft", _p), ("u", _p), ("race", _p),
                ("tokens", _p), ("accepted", _p), ("p_seq_stride", _i64),
                ("p_tok_stride", _i64), ("q_seq_stride", _i64), ("q_tok_stride", _i64),
                ("race_stride", _i64), ("V", _i64), ("B", _i32), ("T", _i32), ("dtype", _i32),
                ("flags", _u32)]


def _ptr(t, name, dtypes, shape=None, optional=False, inner=True):
    """The device pointer of t after checking device, type, shape and (inner) a
    unit last stride."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if inner and t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return ctypes.c_void_p(t.data_ptr())


def _whole(t, name, dtypes, shape, optional=False):
    p = _ptr(t, name, dtypes, shape, optional)
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return p


def _workspace(nbytes: int, device) -> torch.Tensor:
    """A zeroed workspace, complete before it is handed to any stream."""
    w = torch.zeros(nbytes, dtype=torch.uint8, device=device)
    torch.cuda.current_stream(w.device).synchronize()
    return w


class KvCache:
    """One layer's paged cache: k and v [pages, heads, page_size, D], bf16 or
    fp16, of the same strides (any, unit in D: a permuted [pages, page_size,
    heads, D] tensor will do)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 4:
            raise ValueError("k must be [pages, heads, page_size, D]")
        if k.stride() != v.stride():
            raise ValueError("k and v must have the same strides")
        kp = _ptr(k, "k", (torch.bfloat16, torch.float16))
        vp = _ptr(v, "v", (k.dtype,), k.shape)
        pages, heads, page_size, d = k.shape
        self.k, self.v = k, v
        self.c = TritKvCache(kp, vp, k.stride(0), k.stride(1), k.stride(2), pages, heads, page_size,
                             d, _DTYPE[k.dtype], 0)


class KvBatch:
    """Who reads and writes which pages: own page ids table [B, cols] int32, own
    lengths lens [B] int32 (new tokens included), at most T new tokens per
    sequence of which new_lens [B] int32 (all T by default) are valid, and
    the pages prefix_table int32 of the prefix_len keys every sequence shares.  The tables
    and lengths are read when the kernels run: update them in place between
    steps."""

    def __init__(self, table, lens, T: int, new_lens=None, prefix_table=None, prefix_len: int = 0):
        if table.dim() != 2:
            raise ValueError("table must be [B, cols]")
        B, cols = table.shape
        i32 = (torch.int32,)
        if prefix_len and prefix_table is None:
            raise ValueError("prefix_table is required with a prefix")
        npre = 0 if prefix_table is None else prefix_table.numel()
        self.keep = (table, lens, new_lens, prefix_table)
        self.B, self.T = B, int(T)
        pre = _whole(prefix_table, "prefix_table", i32, (npre,), True) if npre else None
        self.c = TritKvBatch(pre, _ptr(table, "table", i32), _whole(lens, "lens", i32, (B,)),
                             _whole(new_lens, "new_lens", i32, (B,), True), int(prefix_len),
                             table.stride(0) if B > 1 else max(cols, 1), npre, cols, B, int(T))


class Rope:
    """Rotation tables cos and sin [max_pos, rot/2] fp32 (None: no rotation),
    pairs=True for columns (2j, 2j+1) instead of (j, j + rot/2), and the optional
    head norms' gains [D] fp32 and eps."""

    def __init__(self, cos=None, sin=None, pairs: bool = False, q_gain=None, k_gain=None, eps: float = 1e-5):
        self.cos, self.sin, self.pairs = cos, sin, bool(pairs)
        self.q_gain, self.k_gain, self.eps = q_gain, k_gain, float(eps)
        f = (torch.float32,)
        self.max_pos, half = (0, 0) if cos is None else cos.shape
        self.rot = 2 * half
        self.p_cos = _whole(cos, "cos", f, (self.max_pos, half), True)
        self.p_sin = _whole(sin, "sin", f, (self.max_pos, half), cos is None)


def _token_rows(t, name, dtypes, B, T, heads, D):
    """[B, T, heads, D] (or [B*T, heads, D], [B*T, heads*D]) with any token
    stride -> (pointer, stride between tokens)."""
    if t.numel() != B * T * heads * D:
        raise ValueError(f"{name} must hold {B}x{T} tokens of {heads} heads of {D}")
    if t.dim() == 2 and t.shape == (B * T, heads * D):
        t = t.unflatten(1, (heads, D))
    if t.dim() == 4 and t.shape == (B, T, heads, D):
        if B > 1 and T > 1 and t.stride(0) != T * t.stride(1):
            raise ValueError(f"{name}: the tokens must be evenly spaced")
        step = t.stride(1) if T > 1 else t.stride(0)
    elif t.dim() == 3 and t.shape == (B * T, heads, D):
        step = t.stride(0)
    else:
        raise ValueError(f"{name} must be [B, T, heads, D], [B*T, heads, D] or [B*T, heads*D]")
    if heads > 1 and t.stride(-2) != D:
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return _ptr(t, name, dtypes), (step if B * T > 1 else heads * D)


class _Job:
    def _bind(self, name, device, c, *keep):
        self.c = c
        self._name = name
        self._fn = getattr(lib(), name)
        self._at = ctypes.addressof(c)
        self._device = device.index
        self._keep = keep

    def _call(self, err_flag, stream):
        """Launch on `stream` or the device's current stream (the raw handle: a
        Stream object per call would cost as much as the launch)."""
        if err_flag.dtype is not torch.int32 or not err_flag.is_cuda:
            raise ValueError("err_flag must be an int32 CUDA tensor")
        s = torch._C._cuda_getCurrentRawStream(self._device) if stream is None else stream.cuda_stream
        status = self._fn(self._at, err_flag.data_ptr(), s)
        if status:
            _check(status, self._name)


class AppendJob(_Job):
    """The arguments of trit_kv_append: cache, batch, rope, q (None: keys and
    values only), k, v (fp32 or the cache's type; token rows may be strided views
    of one buffer) and q_out [B, T, Hq, D] of the cache's type."""

    def __init__(self, cache: KvCache, batch: KvBatch, rope: Rope, q, k, v, q_out):
        B, T, D, Hkv, dt = batch.B, batch.T, cache.k.shape[3], cache.k.shape[1], cache.k.dtype
        src = k.dtype
        if src not in (torch.float32, dt):
            raise ValueError(f"k must be float32 or {dt}")
        hq, q_p, q_s, qo_p = 0, None, 0, None
        if q is not None:
            hq = q.numel() // max(1, B * T * D)
            q_p, q_s = _token_rows(q, "q", (src,), B, T, hq, D)
            qo_p = _whole(q_out, "q_out", (dt,), (B, T, hq, D))
        k_p, k_s = _token_rows(k, "k", (src,), B, T, Hkv, D)
        v_p, v_s = _token_rows(v, "v", (src,), B, T, Hkv, D)
        f = (torch.float32,)
        c = TritKvAppendJob(cache.c, batch.c, q_p, k_p, v_p, qo_p, rope.p_cos, rope.p_sin,
                            _whole(rope.q_gain, "q_gain", f, (D,), True),
                            _whole(rope.k_gain, "k_gain", f, (D,), True), q_s, k_s, v_s,
                            rope.max_pos, rope.eps, hq, rope.rot, _DTYPE[src],
                            ROPE_PAIRS if rope.pairs else 0, 0)
        self.q_out = q_out
        self._bind("trit_kv_append", k.device, c, cache, batch, rope, q, k, v, q_out)


def trit_kv_append(job: AppendJob, err_flag: torch.Tensor, stream=None):
    """Norm and rotate the new tokens' q and k, write q to q_out and k, v to their
    cache slots (one launch).  Returns q_out."""
    job._call(err_flag, stream)
    return job.q_out


def trit_attn_workspace_bytes(job: TritAttnJob) -> int:
    """Bytes of the workspace of a job (its pointers are not read); -1 for
    sizes that are not supported."""
    return int(lib().trit_attn_workspace_bytes(ctypes.byref(job)))


class AttnJob(_Job):
    """The arguments of trit_attn_paged: cache, batch, q (the cache's type;
    token rows may be strided views) and out [B, T, Hq, D] (the cache's type or
    fp32), optionally lse [B, T, Hq] fp32; scale defaults to 1/sqrt(D).  The
    workspace is made here (or given: zeroed once, at least
    trit_attn_workspace_bytes; jobs of any sizes may share one, one call at a time)."""

    def __init__(self, cache: KvCache, batch: KvBatch, q, out, lse=None, scale=None, workspace=None):
        B, T, D, dt = batch.B, batch.T, cache.k.shape[3], cache.k.dtype
        hq = q.numel() // max(1, B * T * D)
        q_p, q_s = _token_rows(q, "q", (dt,), B, T, hq, D)
        c = TritAttnJob(cache.c, batch.c, q_p, _whole(out, "out", (dt, torch.float32), (B, T, hq, D)),
                        _whole(lse, "lse", (torch.float32,), (B, T, hq), True), None, 0, q_s,
                        float(D ** -0.5 if scale is None else scale), hq, _DTYPE[out.dtype], 0)
        need = trit_attn_workspace_bytes(c)
        if need < 0:
            raise ValueError("sizes outside the supported range")
        if workspace is None:
            workspace = _workspace(need, q.device)
        c.workspace = _whole(workspace, "workspace", (torch.uint8,), workspace.shape)
        c.workspace_bytes = workspace.numel()
        self.out, self.lse, self.workspace = out, lse, workspace
        self._bind("trit_attn_paged", q.device, c, cache, batch, q, out, lse, workspace)


def trit_attn_paged(job: AttnJob, err_flag: torch.Tensor, stream=None):
    """Attention of the new tokens to the keys they see.  Returns out."""
    job._call(err_flag, stream)
    return job.out


class VerifyJob(_Job):
    """The arguments of trit_draft_verify: target probabilities p [B, T+1, V]
    and draft probabilities q [B, T, V] (fp32, bf16 or fp16), draft [B, T] int32,
    u [B, T] and race [B, V] fp32, out tokens [B, T+1] and accepted [B] int32."""

    def __init__(self, p, q, draft, u, race, tokens, accepted, n_draft=None):
        if q.dim() != 3:
            raise ValueError("q must be [B, T, V]")
        B, T, V = q.shape
        dt, i32, f32 = (q.dtype,), (torch.int32,), (torch.float32,)
        if q.dtype not in _DTYPE:
            raise ValueError("q must be float32, bfloat16 or float16")
        self.tokens, self.accepted = tokens, accepted
        c = TritVerifyJob(_ptr(p, "p", dt, (B, T + 1, V)), _ptr(q, "q", dt), _whole(draft, "draft", i32, (B, T)),
                          _whole(n_draft, "n_draft", i32, (B,), True), _whole(u, "u", f32, (B, T)),
                          _ptr(race, "race", f32, (B, V)), _whole(tokens, "tokens", i32, (B, T + 1)),
                          _whole(accepted, "accepted", i32, (B,)),
                          p.stride(0), p.stride(1), q.stride(0), q.stride(1), race.stride(0), V, B, T,
                          _DTYPE[q.dtype], 0)
        self._bind("trit_draft_verify", q.device, c, p, q, draft, u, race, tokens, accepted, n_draft)


def trit_draft_verify(job: VerifyJob, err_flag: torch.Tensor, stream=None):
    """Keep drafts, draw the token after them.  Returns (tokens, accepted)."""
    job._call(err_flag, stream)
    return job.tokens, job.accepted
