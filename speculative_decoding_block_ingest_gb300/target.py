"""The target model's side of a speculative step (include/dflash.h).

A step gives the target some new rows of every sequence.  Per target layer
:func:`append` normalises and rotates the rows' queries and keys and puts keys
and values into the layer's paged cache, and :func:`attention` attends over
that cache, with a prefix that all sequences share read once for the batch.
After the target's lm_head :func:`verify_tokens` decides which drafted tokens
stand and draws the next one.

Argument marshalling only, as in :mod:`.dflash`: the work is in the library's
CUDA kernels and there is no fallback.  Calls run on ``stream`` (default: the
current stream of the tensors' device) and return without waiting.  Lengths,
row starts and block tables are device tensors that the kernels read, so a
captured step replays with whatever they hold then.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import dflash
from .dflash import BF16, ERR_INVALID_ARG, ERR_UNSUPPORTED, F16, F32, DflashError, _check

_append_args, _attention_args, _verify_args = (
    dflash.packer(c) for c in (dflash.AppendArgs, dflash.AttentionArgs, dflash.VerifyArgs))
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
    """RoPE frequencies over the first ``rot_dim`` elements of a head (halves
    paired, as in the drafter): plain, or YaRN with ``yarn_factor`` > 1."""

    def __init__(self, rot_dim: int, theta: float = 1e6, yarn_factor: float = 1.0, yarn_original_max_pos: int = 0,
                 yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0):
        self.rot_dim = int(rot_dim)
        self.inv_freq = (ctypes.c_double * max(1, self.rot_dim // 2))()
        self.ptr = ctypes.addressof(self.inv_freq)
        ms = ctypes.c_double(0)
        _check(dflash.load_library().dflash_rope_frequencies(
            self.rot_dim, float(theta), float(yarn_factor), int(yarn_original_max_pos), float(yarn_beta_fast),
            float(yarn_beta_slow), self.inv_freq, ctypes.byref(ms)))
        self.mscale = ms.value


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
        self.k, self.v, self.dtype = k, v, k.dtype
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
        key = (n_rows, n_heads)
        got = self._ws.get(key)
        if got is None:
            n = ctypes.c_size_t(0)
            lib = dflash.load_library()
            with torch.cuda.device(self.device):
                _check(lib.dflash_step_attention_workspace(self.ref, n_rows, n_heads, ctypes.byref(n)))
            if len(self._ws) > 64:
                self._ws = {}      # another thread may be about to look into the old one
            got = self._ws[key] = n.value
        return got


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

    def rows(self, cache: PagedCache, n_rows: int):
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


def _rows(cache: PagedCache, what: str, t: torch.Tensor, n_rows: Optional[int] = None, heads: Optional[int] = None):
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


def append(cache: PagedCache, step: Step, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, *,
           rope: Optional[Rope] = None, q_gain: Optional[torch.Tensor] = None,
           k_gain: Optional[torch.Tensor] = None, eps: float = 1e-6, positions: Optional[torch.Tensor] = None,
           q_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
           ) -> Optional[torch.Tensor]:
    """Head norms (where there is a gain) and RoPE of the step's queries and
    keys; keys and values go into the cache, the queries are returned.

    q, k, v ``[n_rows, heads, head_dim]`` in the cache's dtype or f32, with
    any row stride (views of one fused projection will do); gains f32
    ``[head_dim]``; positions int32 ``[n_rows]`` (default: prefix_len plus the
    row's own key index); q may be None.  ``q_out`` may be q itself."""
    dev = cache.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            q_out = append(cache, step, q, k, v, rope=rope, q_gain=q_gain, k_gain=k_gain, eps=eps,
                           positions=positions, q_out=q_out)
        _used(stream, cache.k, cache.v, *step.tensors, q, k, v, q_gain, k_gain, positions, q_out)
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
    a = _append_args(
        _dtype(k, "rows"), hq, qp, k.data_ptr(), v.data_ptr(), qs, ks, vs,
        0 if q_gain is None else _vector(dev, "q_gain", q_gain, head, torch.float32),
        0 if k_gain is None else _vector(dev, "k_gain", k_gain, head, torch.float32), eps,
        0 if rope is None else rope.rot_dim, 0 if rope is None else rope.ptr, 1.0 if rope is None else rope.mscale,
        0 if positions is None else _vector(dev, "positions", positions, (n,)), qop, qos)
    rc = dflash.load_library().dflash_step_append(cache.ref, step.rows(cache, n), a, _stream(dev))
    if rc:
        _check(rc)
    return q_out


def attention(cache: PagedCache, step: Step, q: torch.Tensor, *, scale: Optional[float] = None, causal: bool = True,
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
        _used(stream, cache.k, cache.v, *step.tensors, q, out, lse, workspace)
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
    rc = dflash.load_library().dflash_step_attention(cache.ref, ref, a, workspace.data_ptr(), workspace.numel(),
                                                     _stream(dev))
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
