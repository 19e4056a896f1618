"""The target model's side of a speculative step (include/dflash.h).

A step gives the target some new rows of every sequence.  Per target layer
:func:`append` normalises and rotates the rows' queries and keys and puts keys
and values into the layer's paged cache, and :func:`attention` attends over
that cache, with a prefix that all sequences share read once for the batch.
After the target's lm_head :func:`verify_tokens` decides which drafted tokens
stand and draws the next one, and :func:`next_step` makes the next step's tables
from that.  The cache is one of 16-bit rows (:class:`PagedCache`) or of rows
rounded to 4 bits (:class:`PagedCache4`).

Argument marshalling only, as in :mod:`.dflash`: the work is in the library's
CUDA kernels and there is no fallback.  Calls run on ``stream`` (default: the
current stream of the tensors' device) and return without waiting.  Lengths,
row starts and block tables are device tensors that the kernels read, so a
captured step replays with whatever they hold then.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence, Tuple, Union

import torch

from . import dflash
from .dflash import BF16, ERR_INVALID_ARG, ERR_UNSUPPORTED, F16, F32, DflashError, _check

_append_args, _packed_append_args, _attention_args, _verify_args, _next_step_args = (
    dflash.packer(c) for c in (dflash.AppendArgs, dflash.PackedAppendArgs, dflash.AttentionArgs, dflash.VerifyArgs,
                               dflash.NextStepArgs))
_STATUS_BYTES = 4096     # what every attention workspace starts with
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _refuse(msg: str, code: int = ERR_INVALID_ARG):
    raise DflashError(code, msg)


def _dtype(t: torch.Tensor, what: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        _refuse(f"{what}: dtype {t.dtype} is not supported", ERR_UNSUPPORTED)
    return d


def _cuda(device: torch.device, what: str) -> torch.device:
    if device.type != "cuda":
        _refuse(f"{what} is on {device}, expected a CUDA device")
    return device


def _vector(device: torch.device, what: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype = torch.int32) -> int:
    """Device pointer of a tensor of this shape whose rows are contiguous."""
    if t.get_device() != device.index:
        _refuse(f"{what} is on {t.device}, expected {device}")
    if t.dtype is not dtype or t.shape != shape:
        _refuse(f"{what} is {t.dtype} {tuple(t.shape)}, expected {dtype} {tuple(shape)}")
    if not t.is_contiguous() and shape[-1] > 1 and t.stride(-1) != 1:
        _refuse(f"{what} must be contiguous in its last dimension")
    return t.data_ptr()


def _scale(scale: Optional[float]) -> float:
    """The attention's scale as the f32 it is passed as, where 0 stands for the default."""
    if scale is None:
        return 0.0
    s = ctypes.c_float(scale).value
    if not 0 < s < float("inf"):
        _refuse("scale must be positive, and finite, in f32")
    return s


@contextlib.contextmanager
def _on(device: torch.device, stream: Optional[torch.cuda.Stream]):
    """The device (and the caller's stream, if any) made current."""
    if stream is None:
        with torch.cuda.device(device):
            yield
        return
    if stream.device != device:
        _refuse(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):     # makes its device current too; outputs are allocated on it
        yield


def _stream(device: torch.device) -> int:
    """Handle of the device's current stream.  (The public calls for this and
    for the current device take 2 us of a call's 15; tensors on the device
    exist by now, so CUDA is initialised.)"""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _used(stream: Optional[torch.cuda.Stream], *tensors):
    """The caller named a stream: its tensors, which may belong to another
    one, are not to be reused before the call has run."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _elsewhere(device: torch.device, stream: Optional[torch.cuda.Stream]) -> bool:
    return stream is not None or torch._C._cuda_getDevice() != device.index


class Rope:
    """RoPE frequencies over the first ``rot_dim`` elements of a head: plain, or
    YaRN with ``yarn_factor`` > 1 (the drafter's formulas), or given ones
    (``inv_freq``, rot_dim / 2 numbers, with ``mscale`` as the factor on cosine and
    sine).  Elements j and j + rot_dim / 2 are a pair, as in the drafter, or 2j and
    2j + 1 (``interleaved``)."""

    def __init__(self, rot_dim: int, theta: float = 1e6, yarn_factor: float = 1.0, yarn_original_max_pos: int = 0,
                 yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0, *, interleaved: bool = False,
                 inv_freq: Optional[Sequence[float]] = None, mscale: Optional[float] = None):
        self.rot_dim = int(rot_dim)
        self.interleaved = int(bool(interleaved))
        self.inv_freq = (ctypes.c_double * max(1, self.rot_dim // 2))()
        self.ptr = ctypes.addressof(self.inv_freq)
        if inv_freq is not None:
            if len(inv_freq) != self.rot_dim // 2 or self.rot_dim < 2 or self.rot_dim % 2:
                _refuse("inv_freq must have rot_dim / 2 numbers")
            self.inv_freq[:] = [float(f) for f in inv_freq]
            if not all(map(math.isfinite, self.inv_freq)):
                _refuse("frequencies must be finite")
            self.mscale = self.mscale64 = 1.0 if mscale is None else float(mscale)
            return
        if mscale is not None:
            _refuse("mscale goes with inv_freq")
        ms = ctypes.c_double(0)
        _check(dflash.load_library().dflash_rope_frequencies(
            self.rot_dim, float(theta), float(yarn_factor), int(yarn_original_max_pos), float(yarn_beta_fast),
            float(yarn_beta_slow), self.inv_freq, ctypes.byref(ms)))
        self.mscale = ms.value
        # the same, not rounded to a float: rows are rounded to 4 bits from what 64 bits give
        self.mscale64 = 0.1 * math.log(yarn_factor) + 1.0 if yarn_factor > 1 else 1.0


def _workspace_bytes(cache, entry: str, n_rows: int, n_heads: int) -> int:
    key = (n_rows, n_heads)
    got = cache._ws.get(key)
    if got is None:
        n = ctypes.c_size_t(0)
        lib = dflash.load_library()
        with torch.cuda.device(cache.device):
            _check(getattr(lib, entry)(cache.ref, n_rows, n_heads, ctypes.byref(n)))
        if len(cache._ws) > 64:
            cache._ws = {}      # another thread may be about to look into the old one
        got = cache._ws[key] = n.value
    return got


class PagedCache:
    """A target layer's paged cache: k and v ``[n_pages, page_size, n_kv_heads,
    head_dim]`` (bf16 or f16), any strides whose last is 1 (a
    ``[n_pages, n_kv_heads, page_size, head_dim]`` pool passes its transpose)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        self.device = _cuda(k.device, "k cache")
        self.index = self.device.index
        if k.dim() != 4 or v.device != k.device or v.dtype != k.dtype or k.shape != v.shape or k.stride() != v.stride():
            _refuse("k and v caches must be alike: [n_pages, page_size, n_kv_heads, head_dim], device, dtype, strides")
        if k.stride(3) != 1:
            _refuse("head elements of the caches must be contiguous")
        self.k, self.v, self.dtype, self.tensors = k, v, k.dtype, (k, v)
        self.n_kv_heads, self.head_dim = k.shape[2], k.shape[3]
        # the stride of a dimension of one element is never used
        st = [s if n > 1 else max(self.head_dim, 8) for s, n in zip(k.stride(), k.shape)]
        self.c = dflash.PagedCacheDesc(k=k.data_ptr(), v=v.data_ptr(), dtype=_dtype(k, "cache"), n_pages=k.shape[0],
                                       page_size=k.shape[1], n_kv_heads=k.shape[2], head_dim=k.shape[3],
                                       page_stride=st[0], row_stride=st[1], head_stride=st[2])
        self.ref = ctypes.byref(self.c)
        self._ws = {}

    def workspace_bytes(self, n_rows: int, n_heads: int) -> int:
        """Workspace of :func:`attention` for up to n_rows rows."""
        return _workspace_bytes(self, "dflash_step_attention_workspace", n_rows, n_heads)


class PagedCache4:
    """A target layer's paged cache in 4 bits: codes k and v uint8 ``[n_pages,
    page_size, n_kv_heads, head_dim / 2]`` (two a byte, the even element in the low
    half) and scales ``[n_pages, page_size, n_kv_heads, head_dim / 16]``
    (float8_e4m3fn, or uint8), each any strides whose last is 1; the scales of a
    head's rows of a page lie together (``[n_pages, n_kv_heads, page_size,
    head_dim / 16]`` pools pass their transposes).  An element is e2m1 code x e4m3
    scale of its 16 x ``unit`` (powers of two).  ``dtype``: of queries, results and
    rounded rows."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, *,
                 dtype: torch.dtype = torch.bfloat16, k_unit: float = 1.0, v_unit: float = 1.0):
        self.device = _cuda(k.device, "k cache")
        self.index = self.device.index
        alike = all(a.device == k.device and a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
                    for a, b in ((v, k), (v_scale, k_scale)))
        if k.dim() != 4 or not alike or k_scale.device != k.device:
            _refuse("k and v must be alike: [n_pages, page_size, n_kv_heads, head_dim / 2], device, dtype, strides; "
                    "their scales too")
        if k.dtype != torch.uint8 or k_scale.dtype not in (torch.uint8, torch.float8_e4m3fn):
            _refuse("codes must be uint8, scales float8_e4m3fn or uint8", ERR_UNSUPPORTED)
        d = 2 * k.shape[3]
        if k_scale.shape != (*k.shape[:3], d // 16):
            _refuse(f"scales must be {(*k.shape[:3], d // 16)}")
        if (k.stride(3) != 1 and d > 2) or (k_scale.stride(3) != 1 and d > 16):
            _refuse("the bytes of a head row must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale, self.dtype = k, v, k_scale, v_scale, dtype
        self.n_kv_heads, self.head_dim, self.page_size = k.shape[2], d, k.shape[1]
        code = _DTYPES.get(dtype)
        if code is None:
            _refuse(f"dtype {dtype} is not supported", ERR_UNSUPPORTED)
        # the stride of a dimension of one element is never used
        st = [s if n > 1 else max(d // 2, 16) for s, n in zip(k.stride(), k.shape)]
        sc = [s if n > 1 else max(d // 16 * k.shape[1], 16) for s, n in zip(k_scale.stride(), k.shape)]
        try:
            units = ctypes.c_float(k_unit), ctypes.c_float(v_unit)
        except TypeError:
            _refuse("units must be numbers")
        if (units[0].value, units[1].value) != (k_unit, v_unit):
            _refuse("units must be powers of two")
        self.tensors = (k, v, k_scale, v_scale)
        self.c = dflash.PackedCacheDesc(
            k=k.data_ptr(), v=v.data_ptr(), k_scale=k_scale.data_ptr(), v_scale=v_scale.data_ptr(), dtype=code,
            n_pages=k.shape[0], page_size=k.shape[1], n_kv_heads=k.shape[2], head_dim=d, page_stride=st[0],
            row_stride=st[1], head_stride=st[2], scale_page_stride=sc[0], scale_row_stride=sc[1],
            scale_head_stride=sc[2], k_unit=k_unit, v_unit=v_unit)
        self.ref = ctypes.byref(self.c)
        self._ws = {}

    @classmethod
    def zeros(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device, **kw) -> "PagedCache4":
        """A cache of zeros, each head's rows of a page together."""
        k, v, ks, vs = (torch.zeros((n_pages, n_kv_heads, page_size, n), dtype=torch.uint8, device=device)
                        .transpose(1, 2) for n in (head_dim // 2, head_dim // 2, head_dim // 16, head_dim // 16))
        return cls(k, v, ks.view(torch.float8_e4m3fn), vs.view(torch.float8_e4m3fn), **kw)

    def workspace_bytes(self, n_rows: int, n_heads: int) -> int:
        """Workspace of :func:`attention` for up to n_rows rows."""
        return _workspace_bytes(self, "dflash_step_attention_packed_workspace", n_rows, n_heads)


AnyCache = Union[PagedCache, PagedCache4]


class Step:
    """The rows of a step: sequence i owns rows ``row_start[i] ..
    row_start[i+1]-1`` and, with them, ``kv_len[i]`` keys at the pages
    ``block_table[i]``, behind the ``prefix_len`` keys at ``prefix_pages``
    that all sequences share.  int32 device tensors; block_table may be one
    row of pages expanded to all sequences, but its rows may not overlap."""

    def __init__(self, row_start: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor,
                 prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0):
        self.device = dev = _cuda(row_start.device, "row_start")
        if row_start.dim() != 1 or row_start.shape[0] < 2 or block_table.dim() != 2:
            _refuse("row_start must be [n_seq + 1] and block_table [n_seq, pages]")
        n, cols = row_start.shape[0] - 1, block_table.shape[1]
        rs = _vector(dev, "row_start", row_start, (n + 1,))
        kl = _vector(dev, "kv_len", kv_len, (n,))
        bt = _vector(dev, "block_table", block_table, (n, cols)) if cols else 0
        self.prefix_pages = 0 if prefix_pages is None else prefix_pages.shape[0]
        pp = _vector(dev, "prefix_pages", prefix_pages, (self.prefix_pages,)) if self.prefix_pages else 0
        self.tensors = (row_start, kv_len, block_table, prefix_pages)
        self.prefix_len = int(prefix_len)
        # the stride of a dimension of one row is never used
        self.fields = (rs, kl, bt, cols, block_table.stride(0) if n > 1 else cols, self.prefix_len, pp)
        self.n_seq = n
        self._refs = {}

    def rows(self, cache: AnyCache, n_rows: int):
        """This step's descriptor for buffers of n_rows rows."""
        if self.device != cache.device:
            _refuse(f"the step is on {self.device}, the cache on {cache.device}")
        if self.prefix_len > self.prefix_pages * cache.c.page_size:
            _refuse("prefix_pages does not hold prefix_len keys")
        ref = self._refs.get(n_rows)
        if ref is None:
            if len(self._refs) > 64:
                self._refs = {}
            ref = self._refs[n_rows] = ctypes.byref(dflash.StepDesc(self.n_seq, n_rows, *self.fields))
        return ref


def _rows(cache: AnyCache, what: str, t: torch.Tensor, n_rows: Optional[int] = None, heads: Optional[int] = None):
    """(rows, heads, row stride) of a [n_rows, heads, head_dim] tensor with contiguous heads."""
    shape, st, d = t.shape, t.stride(), cache.head_dim
    if t.get_device() != cache.index:
        _refuse(f"{what} is on {t.device}, the cache on {cache.device}")
    if len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads) or (
            n_rows is not None and shape[0] != n_rows):
        _refuse(f"{what} has shape {tuple(shape)}")
    n, h = shape[0], shape[1]
    if n and (st[2] != 1 or (h > 1 and st[1] != d)):
        _refuse(f"{what}: the heads of a row must be contiguous")
    return n, h, (st[0] if n > 1 else h * d)


def append(cache: AnyCache, step: Step, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, *,
           rope: Optional[Rope] = None, q_gain: Optional[torch.Tensor] = None,
           k_gain: Optional[torch.Tensor] = None, eps: float = 1e-6, positions: Optional[torch.Tensor] = None,
           q_out: Optional[torch.Tensor] = None, k_values: Optional[torch.Tensor] = None,
           v_values: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
           ) -> Optional[torch.Tensor]:
    """Head norms (where there is a gain) and RoPE of the step's queries and
    keys; keys and values go into the cache, the queries are returned.

    q, k, v ``[n_rows, heads, head_dim]`` in the cache's dtype or f32, with
    any row stride (views of one fused projection will do); gains f32
    ``[head_dim]``; positions int32 ``[n_rows]`` (default: prefix_len plus the
    row's own key index); q may be None.  ``q_out`` may be q itself.  A
    :class:`PagedCache4` takes the rows rounded to 4 bits; ``k_values`` and
    ``v_values`` ``[n_rows, n_kv_heads, head_dim]`` (not k or v themselves) then get
    what they stand for."""
    dev = cache.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            q_out = append(cache, step, q, k, v, rope=rope, q_gain=q_gain, k_gain=k_gain, eps=eps,
                           positions=positions, q_out=q_out, k_values=k_values, v_values=v_values)
        _used(stream, *cache.tensors, *step.tensors, q, k, v, q_gain, k_gain, positions, q_out, k_values, v_values)
        return q_out
    n, _, ks = _rows(cache, "k", k, None, cache.n_kv_heads)
    _, _, vs = _rows(cache, "v", v, n, cache.n_kv_heads)
    dt = k.dtype
    if v.dtype is not dt or (q is not None and q.dtype is not dt):
        _refuse("q, k and v must have one dtype")
    hq = qp = qs = qop = qos = 0
    if q is not None:
        _, hq, qs = _rows(cache, "q", q, n)
        qp = q.data_ptr()
        if q_out is None:
            q_out = torch.empty_like(q, dtype=cache.dtype, memory_format=torch.contiguous_format)
            qos = hq * cache.head_dim
        else:
            if q_out.dtype != cache.dtype:
                _refuse("q_out must have the cache's dtype")
            _, _, qos = _rows(cache, "q_out", q_out, n, hq)
        qop = q_out.data_ptr()
    elif q_out is not None:
        _refuse("q_out without q")
    head = (cache.head_dim,)
    rot, freq, ms, inter = (0, 0, 1.0, 0) if rope is None else (rope.rot_dim, rope.ptr, rope.mscale, rope.interleaved)
    qg = 0 if q_gain is None else _vector(dev, "q_gain", q_gain, head, torch.float32)
    kg = 0 if k_gain is None else _vector(dev, "k_gain", k_gain, head, torch.float32)
    pos = 0 if positions is None else _vector(dev, "positions", positions, (n,))
    if isinstance(cache, PagedCache4):
        out = [0, 0, 0, 0]
        for i, (what, t) in enumerate((("k_values", k_values), ("v_values", v_values))):
            if t is not None:
                if t.dtype is not cache.dtype:
                    _refuse(f"{what} must have the cache's dtype")
                out[2 + i] = _rows(cache, what, t, n, cache.n_kv_heads)[2]
                out[i] = t.data_ptr()
        a = _packed_append_args(_dtype(k, "rows"), hq, qp, k.data_ptr(), v.data_ptr(), qs, ks, vs, qg, kg, eps, rot,
                                freq, ms if rope is None else rope.mscale64, pos, qop, qos, inter, *out)
        rc = dflash.load_library().dflash_step_append_packed(cache.ref, step.rows(cache, n), a, _stream(dev))
    else:
        if k_values is not None or v_values is not None:
            _refuse("k_values and v_values go with a 4-bit cache")
        a = _append_args(_dtype(k, "rows"), hq, qp, k.data_ptr(), v.data_ptr(), qs, ks, vs, qg, kg, eps, rot, freq, ms,
                         pos, qop, qos)
        lib = dflash.load_library()
        call = lib.dflash_step_append_interleaved if inter else lib.dflash_step_append
        rc = call(cache.ref, step.rows(cache, n), a, _stream(dev))
    if rc:
        _check(rc)
    return q_out


def attention(cache: AnyCache, step: Step, q: torch.Tensor, *, scale: Optional[float] = None, causal: bool = True,
              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
              ) -> Tuple[torch.Tensor, torch.Tensor]:
    """softmax(scale q K^T) V of the step's rows over [shared prefix ; own
    keys], with the log-sum-exp ``[n_rows, n_heads]`` (f32) beside it.

    q ``[n_rows, n_heads, head_dim]`` in the cache's dtype (normed and
    rotated).  ``causal``: a row sees own keys up to its own; else all of
    them.  Rows without keys give zeros and -inf.  ``workspace``: uint8, at
    least ``cache.workspace_bytes(n_rows, n_heads)``; calls that share one
    must not overlap (default: a fresh one)."""
    dev = cache.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            out, lse = attention(cache, step, q, scale=scale, causal=causal, out=out, lse=lse, workspace=workspace)
        _used(stream, *cache.tensors, *step.tensors, q, out, lse, workspace)
        return out, lse
    n, hq, qs = _rows(cache, "q", q)
    if q.dtype is not cache.dtype:
        _refuse("q must have the cache's dtype")
    ref, need = step.rows(cache, n), cache.workspace_bytes(n, hq)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        os = hq * cache.head_dim
    else:
        if out.dtype != q.dtype:
            _refuse("out must have the cache's dtype")
        _, _, os = _rows(cache, "out", out, n, hq)
    if lse is None:
        lse = torch.empty((n, hq), dtype=torch.float32, device=dev)
    else:
        _vector(dev, "lse", lse, (n, hq), torch.float32)
        if not lse.is_contiguous():
            _refuse("lse must be contiguous")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _vector(dev, "workspace", workspace, (workspace.numel(),), torch.uint8)
    a = _attention_args(hq, 1 if causal else 0, _scale(scale), q.data_ptr(), qs, out.data_ptr(), os,
                        lse.data_ptr())
    lib = dflash.load_library()
    call = lib.dflash_step_attention_packed if isinstance(cache, PagedCache4) else lib.dflash_step_attention
    rc = call(cache.ref, ref, a, workspace.data_ptr(), workspace.numel(), _stream(dev))
    if rc:
        _check(rc)
    return out, lse


def attention_status(workspace: torch.Tensor, stream: Optional[torch.cuda.Stream] = None):
    """Wait for the stream; raise if a bounded device-side wait of the last
    attention on this workspace gave up."""
    dev = _cuda(workspace.device, "workspace")
    _vector(dev, "workspace", workspace, (workspace.numel(),), torch.uint8)
    if workspace.numel() < _STATUS_BYTES:
        _refuse(f"a workspace of {workspace.numel()} bytes is not one of the attention's")
    with _on(dev, stream):
        _check(dflash.load_library().dflash_step_attention_status(workspace.data_ptr(), _stream(dev)))


def verify_tokens(draft: torch.Tensor, target_probs: torch.Tensor, u_accept: torch.Tensor, u_token: torch.Tensor, *,
                  draft_probs: Optional[torch.Tensor] = None, n_draft: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Which drafted tokens stand, and the token behind them.

    draft int32 ``[n_seq, k]`` (the greedy block of :meth:`Drafter.draft_tokens`,
    or tokens drawn from ``draft_probs`` ``[n_seq, k, vocab]``); target_probs
    ``[n_seq, k + 1, vocab]`` f32, bf16 or f16; u_accept ``[n_seq, k]`` and
    u_token ``[n_seq]`` uniform in [0, 1); n_draft int32 ``[n_seq]`` where
    sequences drafted fewer than k.  Returns int32 tokens ``[n_seq, k + 1]``
    (accepted drafts, the next token, then -1) and the accepted counts."""
    dev = _cuda(target_probs.device, "target_probs")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            got = verify_tokens(draft, target_probs, u_accept, u_token, draft_probs=draft_probs, n_draft=n_draft)
        _used(stream, draft, target_probs, u_accept, u_token, draft_probs, n_draft)
        return got
    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        _refuse("target_probs must be [n_seq, k + 1, vocab]")
    n, k1, vocab = target_probs.shape
    k, dt, ts = k1 - 1, target_probs.dtype, target_probs.stride()
    dp = dss = drs = 0
    if draft_probs is not None and k:
        dp = _vector(dev, "draft_probs", draft_probs, (n, k, vocab), dt)
        dss, drs = draft_probs.stride(0), draft_probs.stride(1) if k > 1 else vocab
    d = _vector(dev, "draft", draft, (n, k)) if k else 0
    ua = _vector(dev, "u_accept", u_accept, (n, k), torch.float32) if k else 0
    tokens = torch.empty((n, k1), dtype=torch.int32, device=dev)
    accepted = torch.empty(n, dtype=torch.int32, device=dev)
    a = _verify_args(
        n, k, vocab, _dtype(target_probs, "target_probs"), d, draft.stride(0),
        0 if n_draft is None else _vector(dev, "n_draft", n_draft, (n,)),
        _vector(dev, "target_probs", target_probs, (n, k1, vocab), dt), ts[0], ts[1] if k else vocab, dp, dss, drs,
        ua, u_accept.stride(0), _vector(dev, "u_token", u_token, (n,), torch.float32), tokens.data_ptr(),
        accepted.data_ptr())
    rc = dflash.load_library().dflash_verify_tokens(a, _stream(dev))
    if rc:
        _check(rc)
    return tokens, accepted


class PagePool:
    """The pages and sequences of a server, on the device: a stack of free page
    ids (``free`` int32 ``[places]``, the first ``n_free`` ``[1]`` of them in use),
    and of every sequence its pages (``block_table`` int32 ``[n_seq, pages]``), keys
    (``kv_len`` ``[n_seq]``) and the last step's rows (``row_start`` ``[n_seq + 1]``).
    All layers' caches go by the same pages.  :func:`next_step` moves it on."""

    def __init__(self, free: torch.Tensor, n_free: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor,
                 row_start: torch.Tensor, *, page_size: int, prefix_pages: Optional[torch.Tensor] = None,
                 prefix_len: int = 0, _ticket: Optional[torch.Tensor] = None):
        self.device = dev = _cuda(free.device, "free")
        if free.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] < 1:
            _refuse("free must be [places] and block_table [n_seq, pages]")
        n, cols = block_table.shape
        self.n_seq, self.page_size, self.prefix_len = n, int(page_size), int(prefix_len)
        self.free, self.n_free, self.block_table, self.kv_len, self.row_start = free, n_free, block_table, kv_len, row_start
        self.prefix_pages = prefix_pages
        if n > 1 and cols and block_table.stride(0) < cols:
            _refuse("the rows of block_table overlap")
        self._pages = (_vector(dev, "block_table", block_table, (n, cols)) if cols else 0,
                       _vector(dev, "free", free, (free.shape[0],)) if free.shape[0] else 0)
        self._lengths = tuple(_vector(dev, w, x, (m,)) for w, x, m in (
            ("kv_len", kv_len, n), ("row_start", row_start, n + 1), ("n_free", n_free, 1)))
        self._shape = (cols, free.shape[0])
        self._stride = block_table.stride(0) if n > 1 else cols
        self.ticket = torch.zeros(1, dtype=torch.int32, device=dev) if _ticket is None else _ticket
        self._step = None

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_seq: int, table_cols: int, device, *, reserved: int = 0,
              **kw) -> "PagePool":
        """A pool of sequences without keys; pages ``reserved .. n_pages - 1`` are free."""
        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)

        free = torch.arange(n_pages - 1, reserved - 1, -1, dtype=torch.int32, device=device)
        return cls(free, torch.full((1,), n_pages - reserved, dtype=torch.int32, device=device),
                   ints(n_seq, table_cols), ints(n_seq), ints(n_seq + 1), page_size=page_size, **kw)

    def beside(self) -> "PagePool":
        """The same pages with lengths of their own, for a step planned beside this one."""
        return PagePool(self.free, torch.empty_like(self.n_free), self.block_table, torch.empty_like(self.kv_len),
                        torch.empty_like(self.row_start), page_size=self.page_size, prefix_pages=self.prefix_pages,
                        prefix_len=self.prefix_len, _ticket=self.ticket)

    @property
    def step(self) -> Step:
        """The step that the pool's lengths are of."""
        if self._step is None:
            self._step = Step(self.row_start, self.kv_len, self.block_table, self.prefix_pages, self.prefix_len)
        return self._step


def next_step(pool: PagePool, rows: torch.Tensor, *, n_rows: Optional[int] = None,
              n_accepted: Optional[torch.Tensor] = None, keep: Optional[torch.Tensor] = None,
              out: Optional[PagePool] = None, slots: Optional[torch.Tensor] = None,
              positions: Optional[torch.Tensor] = None, sequences: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> PagePool:
    """The next step's lengths, row starts and pages, from what stands of the last
    one and the rows that are asked for.

    rows int32 ``[n_seq]``.  Of a sequence's keys stand ``keep`` int32 ``[n_seq]``
    where it is given and not negative (0: the sequence is over); else, where
    ``n_accepted`` (:func:`verify_tokens`) is and is not negative, all but the last
    step's rejected drafts; else all.  Sequences get their rows in order while pages
    and ``n_rows`` (default: the length of the tensors below) last, and behind that
    none: ``row_start`` says what was given.  For every row, where wanted: its place
    in the cache ``slots`` int64 (page * page_size + row of the page), ``positions``
    int32 and whose it is, ``sequences`` int32, all ``[n_rows]``.

    The lengths go to ``out`` (default: the pool itself; or a pool ``beside`` it,
    which leaves this one to be planned again), which is returned: its ``step`` is what
    :func:`append` and :func:`attention` take."""
    dev = pool.device
    out = pool if out is None else out
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            next_step(pool, rows, n_rows=n_rows, n_accepted=n_accepted, keep=keep, out=out, slots=slots,
                      positions=positions, sequences=sequences)
        _used(stream, pool.free, pool.block_table, pool.ticket, pool.n_free, pool.kv_len, pool.row_start, out.n_free,
              out.kv_len, out.row_start, rows, n_accepted, keep, slots, positions, sequences)
        return out
    if out is not pool and (out._pages != pool._pages or out.ticket is not pool.ticket):
        _refuse("out must be the pool or one beside it")
    n = (pool.n_seq,)
    given = [t for t in (slots, positions, sequences) if t is not None]
    if n_rows is None:
        if not given:
            _refuse("n_rows is needed where no tensor has that length")
        n_rows = given[0].shape[0]
    of_rows = [0 if t is None else _vector(dev, w, t, (n_rows,), dt) for w, t, dt in (
        ("slots", slots, torch.int64), ("positions", positions, torch.int32), ("sequences", sequences, torch.int32))]
    table, free = pool._pages
    kv_len, row_start, n_free = pool._lengths
    a = _next_step_args(
        pool.n_seq, pool.page_size, *pool._shape, n_rows, pool.prefix_len, pool._stride, kv_len, row_start, n_free,
        _vector(dev, "rows", rows, n), 0 if n_accepted is None else _vector(dev, "n_accepted", n_accepted, n),
        0 if keep is None else _vector(dev, "keep", keep, n), table, free, *out._lengths, *of_rows,
        pool.ticket.data_ptr())
    rc = dflash.load_library().dflash_next_step(a, _stream(dev))
    if rc:
        _check(rc)
    return out
