"""Plain 64-bit forms of the target-step operators for the tests (numpy / torch
on the CPU), and the error bounds that follow from the kernels' roundings."""
from __future__ import annotations

import math

import numpy as np
import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative


def make_step(rows, kv, page, *, prefix=0, seed=0, spare=2, extra_rows=0):
    """(row_start, kv_len, table, prefix_pages, n_pages) with pages in random order; unused entries are -7."""
    g = torch.Generator().manual_seed(seed)
    n_own = [-(-n // page) for n in kv]
    n_pre = -(-prefix // page)
    n_pages = sum(n_own) + n_pre + spare
    order = torch.randperm(n_pages, generator=g).tolist()
    pre, order = order[:n_pre], order[n_pre:]
    table = torch.full((len(rows), max(n_own + [1])), -7, dtype=torch.int32)
    for i, n in enumerate(n_own):
        table[i, :n] = torch.tensor(order[:n], dtype=torch.int32)
        order = order[n:]
    starts = np.concatenate([[0], np.cumsum(rows)]).tolist()
    return starts, list(kv), table, torch.tensor(pre, dtype=torch.int32), n_pages


def rope_freqs(rot, theta, yarn=None):
    j = np.arange(rot // 2, dtype=np.float64)
    inv = theta ** (-2 * j / rot)
    if yarn is None:
        return inv, 1.0
    factor, orig, fast, slow = yarn
    corr = [rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(theta)) for t in (fast, slow)]
    lo, hi = max(math.floor(corr[0]), 0), min(math.ceil(corr[1]), rot - 1)
    ramp = np.clip((j - lo) / max(hi - lo, 0.001), 0, 1)
    return inv * ((1 - ramp) + ramp / factor), 0.1 * math.log(factor) + 1


def head_rows(x, gain, eps, pos, inv, mscale):
    """Norm and rotation of [n, heads, d] in 64 bits; also the scale of each element's f32 error (the rotated pair's
    length)."""
    x = x.double().cpu().numpy()
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain.double().cpu().numpy()
    h = len(inv)
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * inv
    c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
    a, b = x[..., :h], x[..., h:2 * h]
    y = np.concatenate([a * c - b * s, b * c + a * s, x[..., 2 * h:]], -1)
    pair = np.hypot(a, b) * mscale
    return y, np.concatenate([pair, pair, np.abs(x[..., 2 * h:])], -1)


def attend(q, ks, vs, *, scale, visible):
    """q [t, G, d], keys and values [n, d], visible [t, n] (all f64 numpy): o, lse, A = sum p |v| and the bound of a
    score's error in f32."""
    t, G, d = q.shape
    n = ks.shape[0]
    o, lse, A = np.zeros((t, G, d)), np.full((t, G), -np.inf), np.zeros((t, G, d))
    ds = 0.0
    if n == 0:
        return o, lse, A, ds
    s = np.einsum("tgd,nd->tgn", q, ks) * scale
    ds = d * 2.0 ** -23 * scale * float(np.einsum("tgd,nd->tgn", np.abs(q), np.abs(ks)).max())
    s = np.where(visible[:, None], s, -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - np.where(np.isinf(m), 0.0, m))
    l = p.sum(-1, keepdims=True)
    some = l[..., 0] > 0
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isinf(m), 0.0, m) + np.log(l))[..., 0]
    p = p / np.where(l == 0, 1.0, l)
    o = np.einsum("tgn,nd->tgd", p, vs)
    A = np.einsum("tgn,nd->tgd", p, np.abs(vs))
    return np.where(some[..., None], o, 0.0), lse, A, ds


def attend_step(q, kc, vc, starts, kv, table, pre, prefix, page, *, causal, scale):
    """Every row of a step: (o, tol_o, lse, tol_lse), f64 numpy.  Only keys that exist are read."""
    n_rows, hq, d = q.shape
    hkv = kc.shape[2]
    G = hq // hkv
    half = EPS[q.dtype]
    qn, kn, vn = (x.double().cpu().numpy() for x in (q, kc, vc))
    o, lse = np.zeros((n_rows, hq, d)), np.full((n_rows, hq), -np.inf)
    to, tl = np.zeros((n_rows, hq, d)), np.zeros((n_rows, hq))

    def gather(x, pages, n, h):
        j = np.arange(n)
        return x[np.asarray(pages)[j // page], j % page, h] if n else np.zeros((0, d))

    for i in range(len(kv)):
        r0, r1, n = starts[i], starts[i + 1], kv[i]
        t = r1 - r0
        if t == 0:
            continue
        vis = np.ones((t, prefix + n), dtype=bool)
        if causal:
            vis[:, prefix:] = np.arange(n)[None] <= (n - t + np.arange(t))[:, None]
        for h in range(hkv):
            hs = slice(h * G, (h + 1) * G)
            ks = np.concatenate([gather(kn, pre.numpy(), prefix, h), gather(kn, table[i].numpy(), n, h)])
            vs = np.concatenate([gather(vn, pre.numpy(), prefix, h), gather(vn, table[i].numpy(), n, h)])
            a, b, A, ds = attend(qn[r0:r1, hs], ks, vs, scale=scale, visible=vis)
            o[r0:r1, hs], lse[r0:r1, hs] = a, b
            # softmax weights rounded to the cache's type, the result too; scores off by ds (weights and their sum,
            # and once more for the partial maxima's exp2); f32 sums over n keys; f16 weights below its normal range
            # are off by up to 2^-25 of a weight of at least 1
            vmax = np.abs(vs).max() if vs.size else 0.0
            tiny = (prefix + n) * 2.0 ** -25 * vmax if q.dtype == torch.float16 else 0.0
            to[r0:r1, hs] = half * (A + np.abs(a)) * 1.01 + (4 * ds + (prefix + n + 64) * 2.0 ** -23) * A + tiny + 1e-30
            tl[r0:r1, hs] = 2 * ds + (prefix + n + 64) * 2.0 ** -24 + 2.0 ** -22 * np.where(np.isinf(b), 0, np.abs(b))
    return o, to, lse, tl


def weights(x):
    x = x.double().cpu().numpy()
    return np.where((x > 0) & np.isfinite(x), x, 0.0)


def verify(draft, tp, ua, ut, dp=None, nd=None):
    """Tokens and accepted counts by the definition, one sequence at a time."""
    draft = draft.cpu().numpy()
    n, k = draft.shape
    V = tp.shape[2]
    tokens, taken = np.full((n, k + 1), -1), np.zeros(n, dtype=int)
    ua, ut = ua.double().cpu().numpy(), ut.double().cpu().numpy()
    for i in range(n):
        m = k if nd is None else min(max(int(nd[i]), 0), k)
        j = 0
        while j < m:
            x = draft[i, j]
            if not 0 <= x < V:
                break
            p = weights(tp[i, j])[x]
            q = 1.0 if dp is None else weights(dp[i, j])[x]
            if not ua[i, j] * q < p:
                break
            tokens[i, j] = x
            j += 1
        w = weights(tp[i, j])
        if j < m:
            if dp is None:
                r = w.copy()
                if 0 <= draft[i, j] < V:
                    r[draft[i, j]] = 0
            else:
                r = np.maximum(w - weights(dp[i, j]), 0)
            if r.sum() > 0:
                w = r
        c = np.cumsum(w)
        u = ut[i] if ut[i] > 0 else 0.0
        hit = np.nonzero(c > min(u, 1.0) * c[-1])[0]
        pos = np.nonzero(w > 0)[0]
        tokens[i, j] = hit[0] if len(hit) else (pos[-1] if len(pos) else 0)
        taken[i] = j
    return tokens, taken
