"""Attention over a 4-bit cache on the GPU against 64-bit forms."""
import random

import numpy as np
import pytest
import torch

import _packed_ref as P
import _target_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def T():
    from speculative_decoding_block_ingest_gb300 import target
    return target


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def pools(n_pages, page, hkv, d, *, hnd=False, pad=0, seed=0):
    """Codes and scales of normal rows, as [n_pages, page, hkv, bytes] views (`pad` bytes behind a head's codes, and its
    scales of a page)."""
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(2):
        c, s, _ = P.pack(rng.standard_normal((n_pages, page, hkv, d), dtype=np.float32))
        out.append((c, s))
    mem = []
    for c, _ in out:
        x = np.pad(c, [(0, 0)] * 3 + [(0, pad)])
        x = torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3) if hnd else x)).to(DEV)[..., :d // 2]
        mem.append(x.transpose(1, 2) if hnd else x)
    for _, s in out:      # a head's rows of a page together
        x = np.pad(s.transpose(0, 2, 1, 3).reshape(n_pages, hkv, -1), [(0, 0)] * 2 + [(0, pad)])
        x = torch.from_numpy(x).to(DEV)[..., :page * d // 16]
        mem.append(x.unflatten(2, (page, d // 16)).transpose(1, 2))
    return mem      # k, v, k_scale, v_scale


def f64(mem, units=(1.0, 1.0)):
    k, v, ks, vs = (m.cpu().numpy() for m in mem)
    return P.values(k, ks, units[0]), P.values(v, vs, units[1])


def close(o, lse, want):
    wo, to, wl, tl = want
    e = np.abs(o.double().cpu().numpy() - wo)
    assert np.all(e <= to), (float(np.max(e / to)), np.unravel_index(np.argmax(e / to), e.shape))
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isinf(l), np.isinf(wl)) and np.all(l[np.isinf(l)] < 0)
    f = ~np.isinf(wl)
    assert np.all(np.abs(l[f] - wl[f]) <= tl[f])


def attend_case(T, case, seed=0, units=(1.0, 1.0), **kw):
    rows, kv, hq, hkv, d, page, dt, causal, prefix, hnd = case
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=seed)
    mem = pools(n_pages, page, hkv, d, hnd=hnd, pad=16 if seed % 2 else 0, seed=seed + 1)
    # what lies behind the last keys, and on pages nobody names, is NaN
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    for pages, n in [(pre, prefix)] + [(table[i], n) for i, n in enumerate(kv)]:
        j = torch.arange(n)
        used[pages[j // page].long(), j % page] = True
    for m in mem[2:]:
        m.masked_fill_(~used.to(DEV)[:, :, None, None], P.NAN)
    g = torch.Generator().manual_seed(seed + 2)
    q = torch.randn(starts[-1], hq, d, generator=g).to(dt).to(DEV)
    cache = T.PagedCache4(*mem, dtype=dt, k_unit=units[0], v_unit=units[1])
    step = T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), prefix)
    ws = torch.empty(cache.workspace_bytes(starts[-1], hq), dtype=torch.uint8, device=DEV)
    o, lse = T.attention(cache, step, q, causal=causal, workspace=ws, **kw)
    T.attention_status(ws)
    return (starts, kv, table, pre, mem, q, step, cache), o, lse


def expect(case, got, units=(1.0, 1.0), scale=None):
    (starts, kv, table, pre, mem, q, _, _), o, lse = got
    d = case[4]
    close(o, lse, P.attend_step(q, *f64(mem, units), starts, kv, table, pre, case[8], case[5], causal=case[7],
                                scale=scale or d ** -0.5))


ATTEND = [
    # rows, kv, hq, hkv, d, page, dtype, causal, prefix, hnd
    ([1], [1], 1, 1, 64, 16, BF, True, 0, False),
    ([1], [777], 32, 4, 128, 64, BF, True, 0, True),
    ([2], [130], 8, 1, 128, 64, HF, True, 0, True),
    ([16], [3000], 8, 2, 128, 256, BF, True, 0, False),
    ([1, 17, 0, 5], [300, 17, 9, 130], 12, 4, 64, 16, HF, True, 2053, True),
    ([4, 4, 4], [4, 129, 257], 10, 2, 64, 32, BF, True, 127, False),
    ([3, 40], [2, 10], 8, 1, 128, 16, BF, True, 0, False),          # rows before any key: nothing to see
    ([3, 2], [0, 0], 4, 4, 128, 16, BF, True, 0, False),            # no keys at all
    ([3, 2], [0, 2], 4, 4, 128, 16, BF, True, 33, False),
    ([200, 1, 65], [200, 500, 400], 6, 2, 128, 64, BF, True, 0, False),   # two tiles and more
    ([130], [1000], 4, 1, 64, 64, HF, True, 300, True),
    ([33, 70], [40, 600], 5, 1, 128, 32, BF, False, 129, False),    # every own key
    ([2, 1], [50, 60], 64, 1, 64, 16, BF, True, 256, False),        # 64 heads share a kv head
    ([9], [700], 7, 7, 64, 16, BF, True, 128, False),
    ([1] * 70, [3 * i + 1 for i in range(70)], 4, 2, 128, 16, BF, True, 500, False),
    ([1], [513], 16, 1, 128, 16, HF, False, 1, True),
    ([1, 2, 1], [1, 2, 90], 3, 3, 128, 128, BF, True, 5, False),
    ([5, 3], [640, 3], 3, 1, 64, 32, BF, True, 0, False),
]


@pytest.mark.parametrize("case", ATTEND, ids=[f"{i}" for i in range(len(ATTEND))])
def test_attention(T, case):
    expect(case, attend_case(T, case))


def test_random_steps(T):
    r = random.Random(21)
    for seed in range(16):
        hkv, n = r.choice([1, 2, 4]), r.randint(1, 9)
        rows = [r.choice([0, 1, 1, r.randint(1, 20), r.randint(1, 90)]) for _ in range(n)]
        kv = [t + r.choice([0, r.randint(0, 40), r.randint(0, 700)]) for t in rows]
        rows[0], kv[0] = max(rows[0], 1), max(kv[0], 1)
        case = (rows, kv, hkv * r.choice([1, 2, 3, 8]), hkv, r.choice([64, 128]), r.choice([16, 32, 64, 128, 256]),
                r.choice([BF, HF]), r.random() < 0.7, r.choice([0, r.randint(1, 600)]), r.random() < 0.5)
        expect(case, attend_case(T, case, seed=100 + seed))


@pytest.mark.parametrize("case", [
    # enough blocks for every CTA to go round its rings several times, in every mode
    ([2], [60000], 8, 8, 128, 64, BF, True, 0, False),
    ([1, 3], [41000, 20001], 8, 8, 64, 128, HF, True, 1000, True),
    ([90, 1, 2], [9000, 15000, 11000], 32, 4, 128, 64, BF, True, 3000, False),
    ([3, 9], [20000, 30000], 32, 4, 128, 64, HF, True, 0, True),
    ([1] * 300, [5 + i % 380 for i in range(300)], 4, 4, 128, 16, BF, True, 0, False),
    # a batch of many places, most of them without rows
    ([2 if i % 97 == 5 else 0 for i in range(4096)], [300 if i % 97 == 5 else i % 3 for i in range(4096)], 8, 2, 64,
     16, BF, True, 200, False),
    # many more rows than the CTAs' last items have: merged by CTA
    ([1500, 3, 900, 0, 1], [1500, 2000, 950, 10, 1], 32, 4, 64, 64, HF, True, 0, False),
    ([1400, 700], [1400, 900], 24, 2, 128, 16, BF, False, 0, True),
    # one kv head: rows with a part in every CTA
    ([3], [50000], 4, 1, 128, 64, BF, True, 0, False),
    ([1, 0, 2, 1], [400, 7, 300, 1], 2, 1, 64, 32, HF, True, 40000, False),
    ([1] * 64, [400 + 37 * i for i in range(64)], 16, 2, 128, 64, BF, True, 1500, True),
], ids=["single", "single-d64", "pair-and-single", "few-and-many", "many-short", "many-empty", "prompts",
        "prompts-not-causal", "one-head", "one-head-prefix", "decoding"])
def test_long(T, case):
    expect(case, attend_case(T, case, seed=40))


def test_many_short_sequences_and_a_long_one(T):
    # more rows than the merge goes over one by one, the items of both kernels cut by the CTAs' shares
    rows, kv = [3] * 400 + [40], [3 + 7 * i % 61 for i in range(399)] + [5000, 2500]
    case = (rows, kv, 32, 8, 64, 16, BF, True, 0, False)
    expect(case, attend_case(T, case, seed=77))


def test_units_scale_and_strided_rows(T):
    """Large scores, a scale of the caller's, units of both sides, queries and results inside wider rows."""
    case = ([20, 1, 3], [900, 77, 400], 6, 2, 128, 64, BF, True, 300, True)
    starts, kv, table, pre, n_pages = R.make_step(case[0], case[1], 64, prefix=300, seed=3)
    units = (4.0, 2.0 ** -9)
    mem = pools(n_pages, 64, 2, 128, hnd=True, seed=4)
    g = torch.Generator().manual_seed(5)
    wide = (3 * torch.randn(24, 8, 128, generator=g)).to(BF).to(DEV)
    q = wide[:, :6]
    out = torch.zeros(24, 9, 128, dtype=BF, device=DEV)
    step = T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), 300)
    o, lse = T.attention(T.PagedCache4(*mem, k_unit=4.0, v_unit=2.0 ** -9), step, q, scale=0.125, out=out[:, :6])
    close(o, lse, P.attend_step(q, *f64(mem, units), starts, kv, table, pre, 300, 64, causal=True, scale=0.125))
    assert bool((out[:, 6:] == 0).all())


def test_large_and_small_queries(T):
    """bf16 queries outside f16's range, and codes and scales over their whole range."""
    starts, kv, table, pre, n_pages = R.make_step([2, 20], [100, 80], 16, seed=2)
    rng = np.random.default_rng(7)
    mem = [torch.from_numpy(rng.integers(0, 256, (n_pages, 16, 1, 64), dtype=np.uint8)).to(DEV) for _ in range(2)]
    mem += [torch.from_numpy(rng.integers(0, 0x7F, (n_pages, 16, 1, 8), dtype=np.uint8)).to(DEV) for _ in range(2)]
    q = torch.randn(22, 4, 128, generator=torch.Generator().manual_seed(3))
    q[::3] *= 2.0 ** 20
    q[1::3] *= 2.0 ** -20
    q = q.to(BF).to(DEV)
    k64, v64 = f64(mem)
    scale = float(2.0 ** -28)
    o, lse = T.attention(T.PagedCache4(*mem), T.Step(i32(starts), i32(kv), table.to(DEV)), q, scale=scale)
    close(o, lse, P.attend_step(q, k64, v64, starts, kv, table, pre, 0, 16, causal=True, scale=scale))


@pytest.mark.parametrize("rows", [1, 2, 40])
def test_scales_that_are_nan(T, rows):
    """NaN blocks of the step's later rows do not reach the earlier ones; a row that sees one has NaN in its 16
    elements only, or throughout where it is a key's."""
    kv, d = 400, 128
    starts, kv_, table, pre, n_pages = R.make_step([rows], [kv], 64, prefix=130, seed=6)
    mem = pools(n_pages, 64, 1, d, seed=7)
    q = torch.randn(rows, 4, d, generator=torch.Generator().manual_seed(8)).to(BF).to(DEV)
    step = T.Step(i32(starts), i32(kv_), table.to(DEV), pre.to(DEV), 130)
    wo, to, wl, tl = P.attend_step(q, *f64(mem), starts, kv_, table, pre, 130, 64, causal=True, scale=d ** -0.5)

    def at(key):
        return int(table[0, key // 64]), key % 64

    first = kv - rows
    seen = first + rows // 2                  # this row and those behind it see the NaN value
    p, r = at(seen)
    mem[3][p, r, 0, 2] = P.NAN
    mem[3][p, r, 0, 7] = 0xFF
    p, r = at(kv - 1)                         # the last row's own key
    if rows > 1:
        mem[2][p, r, 0, 3] = P.NAN
    o, lse = (x.double().cpu().numpy() for x in T.attention(T.PagedCache4(*mem), step, q))
    n0, n1 = rows // 2, rows - 1 if rows > 1 else 1
    ok = np.ones(d, dtype=bool)
    ok[32:48] = ok[112:] = False
    assert np.all(np.abs(o - wo)[:n0] <= to[:n0])
    assert np.all(np.abs(o - wo)[n0:n1][..., ok] <= to[n0:n1][..., ok])
    assert np.isnan(o[n0:n1][..., ~ok]).all()
    assert np.all(np.abs(lse - wl)[:n1] <= tl[:n1])
    if rows > 1:
        assert np.isnan(o[n1]).all() and np.isnan(lse[n1]).all()


def test_rows_behind_the_last_sequence(T):
    starts, kv, table, pre, n_pages = R.make_step([2, 3, 30], [70, 20, 90], 16, seed=9)
    mem = pools(n_pages, 16, 2, 64, seed=10)
    q = torch.randn(39, 4, 64, generator=torch.Generator().manual_seed(11)).to(HF).to(DEV)
    out, lse = torch.full((39, 4, 64), 3.0, dtype=HF, device=DEV), torch.full((39, 4), 3.0, device=DEV)
    T.attention(T.PagedCache4(*mem, dtype=HF), T.Step(i32(starts), i32(kv), table.to(DEV)), q, out=out, lse=lse)
    want = P.attend_step(q[:35], *f64(mem), starts, kv, table, pre, 0, 16, causal=True, scale=64 ** -0.5)
    close(out[:35], lse[:35], want)
    assert bool((out[35:] == 3).all()) and bool((lse[35:] == 3).all())


def test_lengths_past_the_table_and_missing_pages(T):
    """A length past the block table reads the keys it has room for; a page outside the pool reads as zeros."""
    mem = pools(4, 16, 1, 64, seed=12)
    q = torch.randn(22, 2, 64, generator=torch.Generator().manual_seed(13)).to(BF).to(DEV)
    table = torch.tensor([[2, 0], [1, 77], [3, -5]], dtype=torch.int32)
    starts = [0, 1, 2, 22]
    o, lse = T.attention(T.PagedCache4(*mem), T.Step(i32(starts), i32([1000, 20, 30]), table.to(DEV)), q, causal=False)
    zero = [torch.cat([m, torch.zeros_like(m[:1])]) for m in mem]
    table[1, 1] = table[2, 1] = 4
    want = P.attend_step(q, *f64(zero), starts, [32, 20, 30], table, torch.zeros(0, dtype=torch.int32), 0, 16,
                         causal=False, scale=0.125)
    close(o, lse, want)


def test_no_rows(T):
    mem = pools(2, 16, 1, 64)
    q = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    o, lse = T.attention(T.PagedCache4(*mem), T.Step(i32([0, 0]), i32([5]), i32([[0]])), q)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)


def test_starts_that_decrease_stay_inside(T):
    """Results are unspecified; the buffers' surroundings are not."""
    mem = pools(8, 16, 2, 64, seed=1)
    for starts in ([0, 9, 3, 12], [5, 2, 1, 0], [0, 1 << 30, -4, 12]):
        out, lse = torch.full((32, 4, 64), 3.0, dtype=BF, device=DEV), torch.full((32, 4), 3.0, device=DEV)
        q = torch.randn(12, 4, 64, device=DEV).to(BF)
        ws = torch.full((T.PagedCache4(*mem).workspace_bytes(12, 4) + 4096,), 77, dtype=torch.uint8, device=DEV)
        n = ws.numel() - 4096
        T.attention(T.PagedCache4(*mem), T.Step(i32(starts), i32([50, 40, 30]), i32([[0, 1, 2, 3]] * 3)), q,
                    out=out[10:22], lse=lse[10:22], workspace=ws[:n])
        torch.cuda.synchronize()
        for x in (out, lse):
            assert bool((x[:10] == 3).all()) and bool((x[22:] == 3).all())
        assert bool((ws[n:] == 77).all())


def test_repeats_bit_for_bit_and_replays(T):
    """Two calls agree in every bit; a captured step replays with the lengths its tensors hold then."""
    case = ATTEND[4]
    (starts, kv, table, pre, mem, q, step, cache), o, lse = attend_case(T, case, seed=20)
    o2, l2 = T.attention(cache, step, q)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    kv_len = i32(kv)
    step = T.Step(i32(starts), kv_len, table.to(DEV), pre.to(DEV), 2053)
    out, lse = torch.empty_like(q), torch.empty_like(lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    T.attention(cache, step, q, out=out, lse=lse, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        T.attention(cache, step, q, out=out, lse=lse)
    for lens in (kv, [200, 17, 3, 60]):
        kv_len.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        close(out, lse, P.attend_step(q, *f64(mem), starts, lens, table, pre, 2053, 16, causal=True, scale=0.125))


def test_pools_in_any_order_and_in_one(T):
    """K above V in memory, codes and scales each way, both in one pool side by side, and one buffer for both."""
    rows, kv = [1, 2, 1], [300, 90, 1000]
    for d, page in ((128, 64), (64, 16)):
        starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, seed=1)
        mem = pools(n_pages, page, 2, d, seed=2)
        q = torch.randn(4, 8, d, generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
        step = T.Step(i32(starts), i32(kv), table.to(DEV))
        k64, v64 = f64(mem)
        want = {}
        for swap in (False, True):
            a, b = (v64, k64) if swap else (k64, v64)
            want[swap] = P.attend_step(q, a, b, starts, kv, table, pre, 0, page, causal=True, scale=d ** -0.5)
        want["k"] = P.attend_step(q, k64, k64, starts, kv, table, pre, 0, page, causal=True, scale=d ** -0.5)
        both = torch.stack([m.transpose(1, 2).contiguous() for m in mem[:2]], 1).transpose(2, 3)
        sboth = torch.stack([m.transpose(1, 2).contiguous() for m in mem[2:]], 1).transpose(2, 3)
        for key, pool in ((False, mem), (True, [mem[1], mem[0], mem[3], mem[2]]), ("k", [mem[0], mem[0], mem[2], mem[2]]),
                          (False, [both[:, 0], both[:, 1], sboth[:, 0], sboth[:, 1]]),
                          (True, [both[:, 1], both[:, 0], mem[3], mem[2]])):
            o, lse = T.attention(T.PagedCache4(*pool), step, q)
            close(o, lse, want[key])


def test_calls_on_two_streams_at_once(T):
    case = ([1, 20, 3], [900, 700, 50], 8, 2, 128, 64, BF, True, 200, True)
    (starts, kv, table, pre, mem, q, step, cache), o, lse = attend_case(T, case, seed=30)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[T.attention(cache, step, q, stream=s) for _ in range(5)] for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for calls in got:
        for a, b in calls:
            assert torch.equal(a, o) and torch.equal(b, lse)


def test_offsets_past_32_bits(T):
    """Pools of more than 2^32 bytes of codes."""
    page, hkv, d = 256, 8, 128
    n_pages = (1 << 32) // (page * hkv * 64) + 40
    mem = [torch.zeros(n_pages, page, hkv, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    mem += [torch.zeros(n_pages, hkv, page, 8, dtype=torch.uint8, device=DEV).transpose(1, 2) for _ in range(2)]
    small = pools(4, page, hkv, d, seed=3)
    for m, x in zip(mem, small):
        m[-4:] = x
    for rows in ([2], [40]):
        q = torch.randn(rows[0], 16, d, generator=torch.Generator().manual_seed(4)).to(BF).to(DEV)
        t = n_pages - 4 + torch.tensor([[2, 0, 3]], dtype=torch.int32)
        o, lse = T.attention(T.PagedCache4(*mem), T.Step(i32([0, rows[0]]), i32([700]), t.to(DEV)), q)
        want = P.attend_step(q, *f64(small), [0, rows[0]], [700], t - (n_pages - 4), torch.zeros(0, dtype=torch.int32), 0,
                             page, causal=True, scale=d ** -0.5)
        close(o, lse, want)
