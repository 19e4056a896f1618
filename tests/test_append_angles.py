"""Codes of keys at far positions on the GPU: the angle is position times
frequency as exact numbers, not as a product that was rounded on the way."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import _packed_ref as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BITS = 400


def pi_bits(bits):
    """pi times 2^bits, rounded down (Machin's formula)."""
    one = 1 << (bits + 32)

    def arctan_inverse(x):
        term, total, n = one // x, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total

    return 4 * (4 * arctan_inverse(5) - arctan_inverse(239)) >> 32


PI = Fraction(pi_bits(BITS), 1 << BITS)


def turn(pos, f):
    """pos times f in turns, in [-1/2, 1/2), as a float."""
    t = pos * Fraction(f) / (2 * PI)
    return float(t - (t + Fraction(1, 2)).__floor__())


def rounded_turn(pos, f):
    """The same from f / (2 pi) as a double, of which 64 bits behind the point are kept."""
    t = f / (2.0 * np.pi)
    bits = int((t - np.floor(t)) * 2.0 ** 64) * pos % 2 ** 64
    return (bits if bits < 2 ** 63 else bits - 2 ** 64) * 2.0 ** -64


def between(exact, rounded, border, other):
    """f32 (a, b) whose rotation's first element lies on one side of the border at one angle, and on the other at the other."""
    c0, s0, c1, s1 = np.cos(exact), np.sin(exact), np.cos(rounded), np.sin(rounded)
    a = np.float32(border * c0 + other * s0) + np.arange(-120, 121, dtype=np.float32) * np.float32(2.0 ** -22)
    b = np.float32(other * c0 - border * s0) + np.arange(-120, 121, dtype=np.float32) * np.float32(2.0 ** -22)
    a, b = (x.astype(np.float64) for x in np.meshgrid(a, b))
    e, r = a * c0 - b * s0 - border, a * c1 - b * s1 - border
    score = np.where(e * r < 0, np.minimum(np.abs(e), np.abs(r)), 0.0)
    i = np.unravel_index(np.argmax(score), score.shape)
    return (a[i], b[i]) if score[i] > 0 else None


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("n", [7, 1400])     # eight warps a row, and one
def test_codes_at_far_positions(n, interleaved):
    from speculative_decoding_block_ingest_gb300 import target as T
    d, half = 128, 64
    rng = np.random.default_rng(5)
    freqs = np.exp(-np.linspace(0.0, 3.0, half))
    freqs[1:4] = [3.0, 17.25, 0.806]
    pos = [(1 << 24) - 1 - 3 * i for i in range(n)]
    angle = {}
    for p in pos[:7]:
        angle[p] = [(2 * np.pi * turn(p, f), 2 * np.pi * rounded_turn(p, f)) for f in freqs]
    x, y, crafted = np.zeros((n, d)), np.zeros((n, d)), 0
    for i, p in enumerate(pos):
        if p not in angle:                    # rows in the same places again: the first rows' angles
            pos[i] = p = pos[i % 7]
            x[i], y[i] = x[i % 7], y[i % 7]
            continue
        for j in range(half):
            exact, rounded = angle[p][j]
            first, second = (2 * j, 2 * j + 1) if interleaved else (j, half + j)
            got = None
            if j % 8 == 0:                    # the largest of its block: scale 1
                got = (6 * np.cos(exact) + 6 * np.sin(exact), 6 * np.cos(exact) - 6 * np.sin(exact))
            elif abs(exact - rounded) > 1e-10:
                got = between(exact, rounded, rng.choice([1.25, 1.75, 2.5, -2.5, 3.5]), rng.choice([-4.7, 4.4]))
                crafted += got is not None
            a, b = (np.float32(v) for v in (got or rng.uniform(-3, 3, 2)))
            x[i, first], x[i, second] = a, b
            a, b = float(a), float(b)
            y[i, first] = a * np.cos(exact) - b * np.sin(exact)
            y[i, second] = b * np.cos(exact) + a * np.sin(exact)
    assert crafted > 100
    cache = T.PagedCache4.zeros(-(-n // 64), 64, 1, d, DEV)
    step = T.Step(torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                  torch.arange(-(-n // 64), dtype=torch.int32, device=DEV)[None])
    k = torch.from_numpy(x).float().to(DEV)[:, None]
    T.append(cache, step, None, k, k, positions=torch.tensor(pos, dtype=torch.int32, device=DEV),
             rope=T.Rope(d, inv_freq=freqs.tolist(), interleaved=interleaved))
    c, s, _ = P.pack(y)
    codes, scales = (m.flatten(0, 1)[:n, 0].cpu().numpy() for m in (cache.k, cache.k_scale.view(torch.uint8)))
    assert np.array_equal(scales, s)
    assert np.array_equal(codes, c)
