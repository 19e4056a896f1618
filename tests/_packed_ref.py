"""Plain 64-bit forms of the operators over a 4-bit cache and of the next
step's tables (numpy / torch on the CPU), and error bounds."""
from __future__ import annotations

import numpy as np
import torch

import _target_ref as R

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
NAN = 0x7F


def nearest(x, values):
    """Index of the nearest value, ties to the even index."""
    mid = (values[1:] + values[:-1]) / 2
    below, upto = np.searchsorted(mid, x, side="left"), np.searchsorted(mid, x, side="right")
    return np.where(below == upto, below, below + below % 2)


def pack(x, unit=1.0):
    """(codes uint8 [..., d / 2], scales uint8 [..., d / 16], the values they stand for) of rows [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, 16) / unit
    top = np.abs(b).max(-1)
    fine = np.isfinite(top)
    sc = np.where(fine, nearest(np.where(fine, top, 0.0) / 6, E4M3), NAN)
    s = np.where(fine, E4M3[np.minimum(sc, len(E4M3) - 1)], np.nan)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where((s > 0)[..., None], np.abs(b) / np.where(s > 0, s, 1.0)[..., None], 0.0)
    mag = nearest(q, E2M1)
    code = np.where(fine[..., None], mag + 8 * np.signbit(b), 0).reshape(x.shape).astype(np.uint8)
    value = (E2M1[mag] * np.where(np.signbit(b), -1.0, 1.0) * s[..., None] * unit).reshape(x.shape)
    return code[..., ::2] | code[..., 1::2] << 4, sc.astype(np.uint8), value


def values(code, scale, unit=1.0):
    """What codes and scales (uint8 arrays) stand for."""
    n = np.stack([code & 15, code >> 4], -1).reshape(*code.shape[:-1], -1)
    s = torch.from_numpy(np.ascontiguousarray(scale)).view(torch.float8_e4m3fn).double().numpy()
    return np.where(n & 8, -1.0, 1.0) * E2M1[n & 7] * np.repeat(s, 16, axis=-1) * unit


def rotate(x, gain, eps, pos, inv, mscale, interleaved):
    """Norm and RoPE in 64 bits, and the length of each element's pair; R.head_rows with the elements in another order."""
    if not interleaved:
        return R.head_rows(x, gain, eps, pos, inv, mscale)
    h, d = len(inv), x.shape[-1]
    order = np.concatenate([np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2), np.arange(2 * h, d)])
    y, size = R.head_rows(x[..., torch.from_numpy(order)], None if gain is None else gain[torch.from_numpy(order)], eps,
                          pos, inv, mscale)
    back = np.argsort(order)
    return y[..., back], size[..., back]


def attend_step(q, kc, vc, starts, kv, table, pre, prefix, page, *, causal, scale):
    """R.attend_step over f64 values [n_pages, page, hkv, d], softmax weights in f16: (o, tol_o, lse, tol_lse)."""
    n_rows, hq, d = q.shape
    hkv = kc.shape[2]
    G, half = hq // hkv, R.EPS[q.dtype]
    qn = q.double().cpu().numpy()
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
            ks, vs = (np.concatenate([gather(x, pre.numpy(), prefix, h), gather(x, table[i].numpy(), n, h)])
                      for x in (kc, vc))
            a, b, A, ds = R.attend(qn[r0:r1, hs], ks, vs, scale=scale, visible=vis)
            o[r0:r1, hs], lse[r0:r1, hs] = a, b
            # weights rounded to f16 (half a step, 2^-11; at 2^7 times their size, so that 2^-32 of the largest is
            # lost at the low end), the result to its type; scores off by ds (weights and their sum, and once more
            # for the partial maxima's exp2); f32 sums over n keys.  A result below f16's normal range is off by half of
            # its smallest step.
            vmax = np.abs(vs).max() if vs.size else 0.0
            to[r0:r1, hs] = (2.0 ** -11 * A * 1.01 + half * np.abs(a) * 1.01 + (4 * ds + (prefix + n + 64) * 2.0 ** -23) * A
                             + (prefix + n) * 2.0 ** -31 * vmax + (2.0 ** -25 if q.dtype == torch.float16 else 0) + 1e-30)
            tl[r0:r1, hs] = 2 * ds + (prefix + n + 64) * 2.0 ** -24 + 2.0 ** -22 * np.where(np.isinf(b), 0, np.abs(b))
    return o, to, lse, tl


def next_step(kv_len, row_start, rows, table, free, n_free, page, n_rows, prefix=0, accepted=None, keep=None):
    """The tables of the next step with a stack, one sequence after the other; `table` and `free` (numpy) change."""
    cols, n = table.shape[1], len(kv_len)

    def pages(x):
        return -(-x // page)

    kept = []
    for i, length in enumerate(kv_len):
        t = row_start[i + 1] - row_start[i]
        if keep is not None and keep[i] >= 0:
            kept.append(min(keep[i], length))
        elif accepted is not None and accepted[i] >= 0:
            kept.append(length - t + min(t, 1 + accepted[i]))
        else:
            kept.append(length)
    want = [t if t > 0 and pages(k + t) <= cols else 0 for k, t in zip(kept, rows)]
    room = n_free + sum(max(0, pages(a) - pages(k + t)) for a, k, t in zip(kv_len, kept, want))
    given, taken, used = [], 0, 0
    for i, t in enumerate(want):
        taken += max(0, pages(kept[i] + t) - pages(kv_len[i]))
        used += t
        given.append(t if taken <= room and used <= n_rows else 0)
    new = [k + t for k, t in zip(kept, given)]
    top = n_free
    for i in reversed(range(n)):
        for col in reversed(range(pages(new[i]), pages(kv_len[i]))):
            free[top] = table[i, col]
            top += 1
    starts, slots, positions, sequences = [0], [], [], []
    for i, t in enumerate(given):
        for col in range(pages(kv_len[i]), pages(new[i])):
            top -= 1
            table[i, col] = free[top]
        for j in range(kept[i], new[i]):
            slots.append(int(table[i, j // page]) * page + j % page)
            positions.append(prefix + j)
            sequences.append(i)
        starts.append(starts[-1] + t)
    return new, starts, top, slots, positions, sequences
