"""Attention over a 4-bit cache on the GPU by the kernel for few query rows:
scales, units and queries that its own conversions see, against 64-bit forms.

Every step here has at most 8 query rows of a kv head and sequence on average
(one tile of rows) or at most 16 (two)."""
import numpy as np
import pytest
import torch

import _packed_ref as P
import _target_ref as R
from test_packed_attention import BF, DEV, HF, T, close, f64, i32, pools  # noqa: F401

pytestmark = pytest.mark.gpu

# rows, kv, hq, hkv, d, page, causal, prefix: key counts that are no multiple of 32
ONE = ([1, 3, 2, 1], [300, 77, 400, 33], 4, 2, 128, 64, True, 0)
ONE_PREFIX = ([1, 3, 2, 1], [300, 77, 400, 33], 3, 1, 64, 16, True, 301)
TWO = ([3, 4, 1, 2], [301, 70, 45, 1], 10, 2, 128, 16, True, 0)
TWO_PREFIX = ([1, 1], [170, 90], 16, 1, 64, 32, True, 45)
STEPS = pytest.mark.parametrize("case", [ONE, ONE_PREFIX, TWO, TWO_PREFIX], ids=["8", "8-prefix", "16", "16-prefix"])


def few(case, dt, seed, mem=None):
    rows, kv, hq, hkv, d, page, causal, prefix = case
    assert sum(rows) * (hq // hkv) <= 16 * len(rows)
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=seed)
    mem = pools(n_pages, page, hkv, d, hnd=bool(seed % 2), seed=seed + 1) if mem is None else mem(n_pages, page, hkv, d)
    q = torch.randn(starts[-1], hq, d, generator=torch.Generator().manual_seed(seed + 2))
    return starts, kv, table, pre, mem, q


def run(T, case, parts, q, units=(1.0, 1.0), **kw):  # noqa: F811
    starts, kv, table, pre, mem, _ = parts
    cache = T.PagedCache4(*mem, dtype=q.dtype, k_unit=units[0], v_unit=units[1])
    ws = torch.empty(cache.workspace_bytes(q.shape[0], q.shape[1]), dtype=torch.uint8, device=DEV)
    got = T.attention(cache, T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), case[7]), q, causal=case[6],
                      workspace=ws, **kw)
    T.attention_status(ws)
    return got


def want(case, parts, q, units=(1.0, 1.0), scale=None):
    starts, kv, table, pre, mem, _ = parts
    return P.attend_step(q, *f64(mem, units), starts, kv, table, pre, case[7], case[5], causal=case[6],
                         scale=scale or case[4] ** -0.5)


@STEPS
@pytest.mark.parametrize("k_unit,scale", [(1.0, None), (2.0 ** -22, None), (2.0 ** -60, None), (1.0, 2.0 ** -28),
                                          (2.0 ** 20, 2.0 ** -100), (2.0 ** -60, 2.0 ** 50)])
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
def test_query_rows_of_zeros_and_tiny_ones(T, case, k_unit, scale, dt):  # noqa: F811
    """A row whose scores are all zero (or lost beside 1) weighs its keys alike, whatever its masked keys hold."""
    parts = few(case, dt, 31)
    q = parts[5]
    small = [0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -100, 2.0 ** -60] if dt == BF else [0.0, 2.0 ** -24, 2.0 ** -14]
    for i in range(q.shape[0]):
        for h in range(q.shape[1]):
            q[i, h] *= small[(i + h) % len(small)]
    q = q.to(dt).to(DEV)
    close(*run(T, case, parts, q, (k_unit, 0.5), scale=scale), want(case, parts, q, (k_unit, 0.5), scale))


@STEPS
def test_large_query_rows_over_keys_of_zeros(T, case):  # noqa: F811
    """Scores of 0 however large the row and the scale are."""
    parts = few(case, BF, 35)
    q = (torch.sign(parts[5]) * 2.0 ** 127).to(BF).to(DEV)
    for m in parts[4][::2]:
        m.zero_()
    close(*run(T, case, parts, q, scale=2.0 ** 40), want(case, parts, q, scale=2.0 ** -100))   # (any: 0 in 64 bits too)


@pytest.mark.parametrize("case", [ONE, ONE_PREFIX, TWO, TWO_PREFIX, ([40], [300], 4, 2, 128, 64, True, 0)],
                         ids=["8", "8-prefix", "16", "16-prefix", "many"])
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
def test_scores_far_below_any_other(T, case, dt):  # noqa: F811
    """Rows all of whose scores lie below -1e30 (and are exact floats) have keys all the same."""
    rows, kv, hq, hkv, d, page, causal, prefix = case
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=41)
    mem = pools(n_pages, page, hkv, d, seed=42)
    mem[0].zero_()
    mem[0][..., 0] = 6                       # 4 times a scale of 0.5, and zeros
    mem[2].fill_(0x30)
    q = torch.zeros(starts[-1], hq, d)
    q[..., 0] = -2.0 ** (110 if dt == BF else 14)
    scale = 2.0 ** (0 if dt == BF else 96)
    q = q.to(dt).to(DEV)
    parts = (starts, kv, table, pre, mem, q)
    o, lse = (x.double().cpu().numpy() for x in run(T, case, parts, q, scale=scale))
    # 64-bit results of equal scores; f16 weights of 1 are exact: f32 sums and the rounding to the type
    wo, _, wl, _ = want(case, (starts, kv, table, pre, [torch.zeros_like(mem[0])] + mem[1:], q), q, scale=1.0)
    n = prefix + max(kv)
    assert np.all(np.abs(o - wo) <= R.EPS[dt] * np.abs(wo) + (n + 64) * 2.0 ** -23 * 6 + (2.0 ** -25 if dt == HF else 0))
    none = np.isinf(wl)                      # rows before any key
    assert np.all(lse[none] == -np.inf) and np.all(np.abs(lse[~none] + 2.0 ** 111) <= 2.0 ** -22 * 2.0 ** 111)


@STEPS
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
def test_units_a_scale_and_strided_rows(T, case, dt):  # noqa: F811
    """Large scores, a scale of the caller's, units of both sides, queries and results inside wider rows."""
    parts = few(case, dt, 51)
    q0 = parts[5]
    n, hq, d = q0.shape
    wide = torch.zeros(n, hq + 2, d, dtype=dt, device=DEV)
    q = wide[:, :hq]
    q.copy_(3 * q0)
    out = torch.full((n, hq + 3, d), 5.0, dtype=dt, device=DEV)
    units = (4.0, 2.0 ** -9)
    got = run(T, case, parts, q, units, scale=0.125, out=out[:, :hq])
    close(*got, want(case, parts, q, units, 0.125))
    assert bool((out[:, hq:] == 5).all())


@STEPS
def test_bf16_queries_outside_the_range_of_f16(T, case):  # noqa: F811
    """Rows 2^20 and 2^-20 times as large, heads of both sizes in one row, and codes and scales over their whole range."""
    hkv, d = case[3], case[4]
    rng = np.random.default_rng(52)

    def any_bytes(n_pages, page, hkv, d):
        mem = [torch.from_numpy(rng.integers(0, 256, (n_pages, page, hkv, d // 2), dtype=np.uint8)).to(DEV) for _ in range(2)]
        return mem + [torch.from_numpy(rng.integers(0, 0x7F, (n_pages, hkv, page, d // 16), dtype=np.uint8)).to(DEV)
                      .transpose(1, 2) for _ in range(2)]

    parts = few(case, BF, 53, any_bytes)
    q = parts[5]
    for i in range(q.shape[0]):
        for h in range(q.shape[1]):
            q[i, h] *= (2.0 ** 20, 2.0 ** -20, 1.0)[(2 * i + h) % 3]
    q = q.to(BF).to(DEV)
    close(*run(T, case, parts, q, scale=2.0 ** -28), want(case, parts, q, scale=2.0 ** -28))
    # and rows of one size far from 1, whose scores a scale brings back
    for size in (2.0 ** 100, 2.0 ** -60):
        x = (parts[5].sign() * size).to(BF).to(DEV)
        scale = float(2.0 ** -10 / size / 32)
        close(*run(T, case, parts, x, scale=scale), want(case, parts, x, scale=scale))


@pytest.mark.parametrize("case", [ONE, TWO_PREFIX, ([40, 9], [300, 700], 4, 2, 128, 64, True, 129),
                                  ([1] * 20, [400 + 77 * i for i in range(20)], 16, 2, 128, 64, True, 1500),
                                  ([1, 60], [3000, 900], 8, 1, 64, 16, True, 0)],
                         ids=["few", "few-prefix", "many", "decoding", "both"])
def test_results_are_the_same_bits_every_time(T, case):  # noqa: F811
    rows, kv, hq, hkv, d, page, causal, prefix = case
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=61)
    parts = (starts, kv, table, pre, pools(n_pages, page, hkv, d, seed=62), None)
    q = torch.randn(starts[-1], hq, d, generator=torch.Generator().manual_seed(63)).to(BF).to(DEV)
    o, lse = run(T, case, parts, q)
    close(o, lse, want(case, parts, q))
    for _ in range(20):
        a, b = run(T, case, parts, q)
        assert torch.equal(a, o) and torch.equal(b, lse)
