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

import ctypes
from typing import Optional, Tuple

import torch

from . import dflash
from .dflash import BF16, ERR_INVALID_ARG, ERR_UNSUPPORTED, F16, F32, DflashError, _check

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _refuse(msg: str, code: int = ERR_INVALID_ARG):
    raise DflashError(code, msg)


def _dtype(t: torch.Tensor, what: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        _refuse(f"{what}: dtype {t.dtype} is not supported", ERR_UNSUPPORTED)
    return d


def _on(device: torch.device, what: str, t: torch.Tensor, dtype=None, dim: Optional[int] = None):
    if t.device != device or device.type != "cuda":
        _refuse(f"{what} is on {t.device}, expected the cache's CUDA device ({device})")
    if dtype is not None and t.dtype != dtype:
        _refuse(f"{what} has dtype {t.dtype}, expected {dtype}")
    if dim is not None and t.dim() != dim:
        _refuse(f"{what} has {t.dim()} dimensions, expected {dim}")


def _index(device: torch.device, what: str, t: torch.Tensor, dim: int) -> int:
    """Device pointer of an int32 tensor whose last dimension is contiguous."""
    _on(device, what, t, torch.int32, dim)
    if t.numel() and t.stride(-1) != 1 and t.shape[-1] > 1:
        _refuse(f"{what} must be contiguous in its last dimension")
    return t.data_ptr()


class _Launch:
    """The device and stream of one call: makes the device current, allocates
    outputs on the call's stream, and tells the allocator of tensors that
    belong to another one."""

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        self.device, self.stream = device, stream
        self.ctx = None

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device != self.device:
                _refuse(f"stream is on {self.stream.device}, the tensors on {self.device}")
            self.ctx = torch.cuda.stream(self.stream)     # makes its device current too
        elif torch.cuda.current_device() != self.device.index:
            self.ctx = torch.cuda.device(self.device)
        if self.ctx is not None:
            self.ctx.__enter__()
        self.ptr = ctypes.c_void_p(torch.cuda.current_stream(self.device).cuda_stream)
        return self

    def uses(self, *tensors):
        if self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


class Rope:
    """RoPE frequencies over the first ``rot_dim`` elements of a head (halves
    paired, as in the drafter): plain, or YaRN with ``yarn_factor`` > 1."""

    def __init__(self, rot_dim: int, theta: float = 1e6, yarn_factor: float = 1.0, yarn_original_max_pos: int = 0,
                 yarn_beta_fast: float = 32.0, yarn_beta_slow: float = 1.0):
        self.rot_dim = int(rot_dim)
        self.inv_freq = (ctypes.c_double * max(1, self.rot_dim // 2))()
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
        _on(k.device, "k cache", k, dim=4)
        _on(k.device, "v cache", v, k.dtype, 4)
        if k.shape != v.shape or k.stride() != v.stride():
            _refuse("k and v caches must have one shape and strides")
        self.k, self.v = k, v
        self.device = k.device
        self.n_kv_heads, self.head_dim = k.shape[2], k.shape[3]
        if k.stride(3) != 1:
            _refuse("head elements of the caches must be contiguous")
        # the stride of a dimension of one element is never used
        st = [s if n > 1 else max(self.head_dim, 8) for s, n in zip(k.stride(), k.shape)]
        self.c = dflash.PagedCacheDesc(k=k.data_ptr(), v=v.data_ptr(), dtype=_dtype(k, "cache"), n_pages=k.shape[0],
                                       page_size=k.shape[1], n_kv_heads=k.shape[2], head_dim=k.shape[3],
                                       page_stride=st[0], row_stride=st[1], head_stride=st[2])
        self._ws = {}

    def workspace_bytes(self, n_rows: int, n_heads: int) -> int:
        """Workspace of :func:`attention` for up to n_rows rows."""
        key = (n_rows, n_heads)
        if key not in self._ws:
            n = ctypes.c_size_t(0)
            with torch.cuda.device(self.device):
                _check(dflash.load_library().dflash_step_attention_workspace(ctypes.byref(self.c), n_rows, n_heads,
                                                                             ctypes.byref(n)))
            if len(self._ws) > 64:
                self._ws.clear()
            self._ws[key] = n.value
        return self._ws[key]


class Step:
    """The rows of a step: sequence i owns rows ``row_start[i] ..
    row_start[i+1]-1`` and, with them, ``kv_len[i]`` keys at the pages
    ``block_table[i]``, behind the ``prefix_len`` keys at ``prefix_pages``
    that all sequences share.  int32 device tensors."""

    def __init__(self, row_start: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor,
                 prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0):
        dev = row_start.device
        rs, kl = _index(dev, "row_start", row_start, 1), _index(dev, "kv_len", kv_len, 1)
        bt = _index(dev, "block_table", block_table, 2)
        n = kv_len.shape[0]
        if row_start.shape[0] != n + 1 or block_table.shape[0] != n:
            _refuse("row_start, kv_len and block_table disagree about the number of sequences")
        pp = _index(dev, "prefix_pages", prefix_pages, 1) if prefix_pages is not None else None
        self.tensors = (row_start, kv_len, block_table, prefix_pages)
        self.device = dev
        self.prefix_pages = 0 if prefix_pages is None else prefix_pages.shape[0]
        cols = block_table.shape[1]
        self.c = dflash.StepDesc(n_seq=n, n_rows=0, row_start=rs, kv_len=kl, block_table=bt, table_cols=cols,
                                 table_stride=max(block_table.stride(0), cols) if n > 1 else cols,
                                 prefix_len=int(prefix_len), prefix_pages=pp)

    def rows(self, cache: PagedCache, n_rows: int):
        """This step's descriptor for buffers of n_rows rows."""
        if self.device != cache.device:
            _refuse(f"the step is on {self.device}, the cache on {cache.device}")
        if self.c.prefix_len > self.prefix_pages * cache.c.page_size:
            _refuse("prefix_pages does not hold prefix_len keys")
        d = dflash.StepDesc.from_buffer_copy(self.c)
        d.n_rows = n_rows
        return d


def _rows(cache: PagedCache, what: str, t: torch.Tensor, heads: Optional[int] = None, n_rows: Optional[int] = None):
    """Row stride of a [n_rows, heads, head_dim] tensor with contiguous heads."""
    _on(cache.device, what, t, dim=3)
    n, h, d = t.shape
    if d != cache.head_dim or (heads is not None and h != heads) or (n_rows is not None and n != n_rows):
        _refuse(f"{what} has shape {tuple(t.shape)}")
    if t.numel() and (t.stride(2) != 1 or (h > 1 and t.stride(1) != d)):
        _refuse(f"{what}: the heads of a row must be contiguous")
    return t.stride(0) if n > 1 else h * d


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
    kv = cache.n_kv_heads
    ks = _rows(cache, "k", k, kv)
    n_rows = k.shape[0]
    vs = _rows(cache, "v", v, kv, n_rows)
    if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        _refuse("q, k and v must have one dtype")
    a = dflash.AppendArgs(dtype=_dtype(k, "rows"), k=k.data_ptr(), v=v.data_ptr(), k_stride=ks, v_stride=vs, eps=eps)
    for name, g in (("q_gain", q_gain), ("k_gain", k_gain)):
        if g is not None:
            _on(cache.device, name, g, torch.float32, 1)
            if g.shape[0] != cache.head_dim or not g.is_contiguous():
                _refuse(f"{name} must be a contiguous [head_dim] tensor")
            setattr(a, name, g.data_ptr())
    if rope is not None:
        a.rot_dim, a.inv_freq, a.mscale = rope.rot_dim, ctypes.cast(rope.inv_freq, dflash.PDOUBLE), rope.mscale
    if positions is not None:
        a.positions = _index(cache.device, "positions", positions, 1)
        if positions.shape[0] != n_rows:
            _refuse("positions must have one entry per row")
    with _Launch(cache.device, stream) as call:
        if q is not None:
            a.n_heads, a.q, a.q_stride = q.shape[1], q.data_ptr(), _rows(cache, "q", q, n_rows=n_rows)
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=cache.k.dtype, device=cache.device)
            elif q_out.dtype != cache.k.dtype:
                _refuse("q_out must have the cache's dtype")
            a.q_out, a.q_out_stride = q_out.data_ptr(), _rows(cache, "q_out", q_out, q.shape[1], n_rows)
        elif q_out is not None:
            _refuse("q_out without q")
        s = step.rows(cache, n_rows)
        _check(dflash.load_library().dflash_step_append(ctypes.byref(cache.c), ctypes.byref(s), ctypes.byref(a),
                                                        call.ptr))
        call.uses(cache.k, cache.v, *step.tensors, q, k, v, q_gain, k_gain, positions, q_out)
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
    qs = _rows(cache, "q", q)
    n_rows, n_heads = q.shape[:2]
    if q.dtype != cache.k.dtype:
        _refuse("q must have the cache's dtype")
    s = step.rows(cache, n_rows)
    need = cache.workspace_bytes(n_rows, n_heads)
    with _Launch(cache.device, stream) as call:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=cache.device)
        elif out.dtype != q.dtype:
            _refuse("out must have the cache's dtype")
        if lse is None:
            lse = torch.empty(n_rows, n_heads, dtype=torch.float32, device=cache.device)
        _on(cache.device, "lse", lse, torch.float32, 2)
        if tuple(lse.shape) != (n_rows, n_heads) or not lse.is_contiguous():
            _refuse("lse must be a contiguous [n_rows, n_heads] tensor")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
        _on(cache.device, "workspace", workspace, torch.uint8, 1)
        a = dflash.AttentionArgs(n_heads=n_heads, causal=1 if causal else 0, scale=0.0 if scale is None else scale,
                                 q=q.data_ptr(), q_stride=qs, out=out.data_ptr(),
                                 out_stride=_rows(cache, "out", out, n_heads, n_rows), lse=lse.data_ptr())
        if scale is not None and not scale > 0:
            _refuse("scale must be positive")
        _check(dflash.load_library().dflash_step_attention(
            ctypes.byref(cache.c), ctypes.byref(s), ctypes.byref(a), ctypes.c_void_p(workspace.data_ptr()),
            workspace.numel(), call.ptr))
        call.uses(cache.k, cache.v, *step.tensors, q, out, lse, workspace)
    return out, lse


def attention_status(workspace: torch.Tensor, stream: Optional[torch.cuda.Stream] = None):
    """Wait for the stream; raise if a bounded device-side wait of the last
    attention on this workspace gave up."""
    with _Launch(workspace.device, stream) as call:
        _check(dflash.load_library().dflash_step_attention_status(ctypes.c_void_p(workspace.data_ptr()), call.ptr))


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
    dev = target_probs.device
    _on(dev, "target_probs", target_probs, dim=3)
    n, k1, vocab = target_probs.shape
    _on(dev, "draft", draft, torch.int32, 2)
    _on(dev, "u_accept", u_accept, torch.float32, 2)
    _on(dev, "u_token", u_token, torch.float32, 1)
    if tuple(draft.shape) != (n, k1 - 1) or tuple(u_accept.shape) != (n, k1 - 1) or u_token.shape[0] != n:
        _refuse("draft, u_accept, u_token and target_probs disagree about n_seq or k")
    for name, t in (("draft", draft), ("u_accept", u_accept), ("u_token", u_token), ("target_probs", target_probs)):
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            _refuse(f"{name} must be contiguous in its last dimension")
    a = dflash.VerifyArgs(n_seq=n, k=k1 - 1, vocab=vocab, dtype=_dtype(target_probs, "target_probs"),
                          draft=draft.data_ptr(), draft_stride=draft.stride(0), target_probs=target_probs.data_ptr(),
                          target_seq_stride=target_probs.stride(0),
                          target_row_stride=target_probs.stride(1) if k1 > 1 else vocab,
                          u_accept=u_accept.data_ptr(), u_accept_stride=u_accept.stride(0),
                          u_token=u_token.data_ptr())
    if draft_probs is not None:
        _on(dev, "draft_probs", draft_probs, target_probs.dtype, 3)
        if tuple(draft_probs.shape) != (n, k1 - 1, vocab) or (vocab > 1 and draft_probs.stride(2) != 1):
            _refuse("draft_probs must be [n_seq, k, vocab] with contiguous rows")
        a.draft_probs, a.draft_seq_stride = draft_probs.data_ptr(), draft_probs.stride(0)
        a.draft_row_stride = draft_probs.stride(1) if k1 > 2 else vocab
    if n_draft is not None:
        a.n_draft = _index(dev, "n_draft", n_draft, 1)
        if n_draft.shape[0] != n:
            _refuse("n_draft must have one entry per sequence")
    with _Launch(dev, stream) as call:
        tokens = torch.empty(n, k1, dtype=torch.int32, device=dev)
        accepted = torch.empty(n, dtype=torch.int32, device=dev)
        a.tokens, a.n_accepted = tokens.data_ptr(), accepted.data_ptr()
        _check(dflash.load_library().dflash_verify_tokens(ctypes.byref(a), call.ptr))
        call.uses(draft, target_probs, u_accept, u_token, draft_probs, n_draft)
    return tokens, accepted
