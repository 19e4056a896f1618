"""The target model's step operators on the GPU against 64-bit plain forms:
paged append with head norms and RoPE, attention with a shared prefix, and
verification of drafted tokens."""
import math

import numpy as np
import pytest
import torch

import _target_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def T():
    from speculative_decoding_block_ingest_gb300 import target
    return target


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def caches(n_pages, page, hkv, d, dt, *, hnd=False, seed=0, pad=0):
    """k and v pools (with `pad` unused elements behind every head row) as [n_pages, page, hkv, d] views."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        shape = (n_pages, hkv, page, d + pad) if hnd else (n_pages, page, hkv, d + pad)
        x = torch.randn(*shape, generator=g).to(dt).to(DEV)[..., :d]
        out.append(x.transpose(1, 2) if hnd else x)
    return out


# ------------------------------------------------------------------ append
APPEND = [
    # rows, kv, hq, hkv, d, rot, page, in, cache, norm, yarn, hnd, fused, prefix
    ([1], [1], 1, 1, 64, 64, 16, BF, BF, True, False, False, False, 0),
    ([1], [1000], 32, 4, 128, 128, 64, BF, BF, True, False, False, True, 0),
    ([5, 0, 17, 1], [5, 40, 100, 1], 32, 8, 128, 128, 16, F4, BF, True, True, True, False, 16383),
    ([3, 2], [700, 2], 6, 2, 64, 32, 128, HF, HF, False, False, False, True, 70),
    ([40, 33], [40, 200], 5, 5, 128, 64, 32, F4, HF, True, True, True, True, 1),
    ([9], [9], 3, 1, 128, 0, 256, BF, BF, True, False, False, False, 0),
    ([2] * 300, [7] * 300, 2, 1, 64, 16, 16, BF, BF, True, False, False, False, 5),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"{i}" for i in range(len(APPEND))])
def test_append(T, case):
    rows, kv, hq, hkv, d, rot, page, ti, tc, norm, yarn, hnd, fused, prefix = case
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=1)
    kc, vc = caches(n_pages, page, hkv, d, tc, hnd=hnd, pad=8)
    k0, v0 = kc.clone(), vc.clone()
    n = starts[-1]
    g = torch.Generator().manual_seed(2)
    if fused:
        x = torch.randn(n, (hq + 2 * hkv) * d, generator=g).to(ti).to(DEV)
        q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([hq * d, hkv * d, hkv * d], 1))
    else:
        q, k, v = (torch.randn(n, h, d, generator=g).to(ti).to(DEV) for h in (hq, hkv, hkv))
    qg, kg = ((1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)) if norm else (None, None)
    y4 = (32.0, 8192, 32.0, 1.0)
    rope = None
    inv, ms = np.zeros(0), 1.0
    if rot:
        rope = T.Rope(rot, 1e6, *y4) if yarn else T.Rope(rot, 1e4)
        inv, ms = R.rope_freqs(rot, 1e6, y4) if yarn else R.rope_freqs(rot, 1e4)
    step = T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), prefix)
    qo = T.append(T.PagedCache(kc, vc), step, q, k, v, rope=rope, q_gain=qg, k_gain=kg, eps=1e-6)
    torch.cuda.synchronize()
    pos, dst = [], []
    for i, t in enumerate(rows):
        for own in range(kv[i] - t, kv[i]):
            pos.append(prefix + own)
            dst.append((int(table[i, own // page]), own % page))
    half = R.EPS[tc]
    for got, src, gain in ((qo, q, qg), (torch.stack([kc[a, b] for a, b in dst]), k, kg)):
        want, size = R.head_rows(src, gain, 1e-6, pos, inv, ms)
        # one rounding to the cache's type; norm, angle (2^-25 of a turn) and rotation in f32
        tol = half * np.abs(want) + 1e-6 * size + (2.0 ** -25 if tc == HF else 0)
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    assert torch.equal(torch.stack([vc[a, b] for a, b in dst]), v.to(tc))
    # nothing else of the caches changed
    for a, b in dst:
        k0[a, b], v0[a, b] = kc[a, b], vc[a, b]
    assert torch.equal(k0, kc) and torch.equal(v0, vc)


def test_append_far_positions_and_given_ones(T):
    """Explicit positions up to 2^30: the angle keeps its accuracy."""
    d, pos = 128, [0, 1, 131071, 1 << 20, (1 << 30) + 12345]
    kc, vc = caches(2, 16, 1, d, HF)
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(5, h, d, generator=g).to(HF).to(DEV) for h in (2, 1))
    step = T.Step(i32([0, 5]), i32([5]), i32([[1]]))
    qo = T.append(T.PagedCache(kc, vc), step, q, k, k, rope=T.Rope(d, 1e6), positions=i32(pos))
    inv, ms = R.rope_freqs(d, 1e6)
    want, size = R.head_rows(q, None, 0, pos, inv, ms)
    # turns = p * f / 2 pi in f64: its error of 2^-53 * 2^30 / 6 turns is far below f32's
    assert np.all(np.abs(qo.double().cpu().numpy() - want) <= R.EPS[HF] * np.abs(want) + 1e-6 * size + 2.0 ** -25)


def test_append_leaves_what_no_row_names(T):
    """Rows behind the last sequence, rows before key 0, past the block table and on a page that does not exist."""
    d = 64
    kc, vc = caches(3, 16, 1, d, BF)
    k0, v0 = kc.clone(), vc.clone()
    g = torch.Generator().manual_seed(4)
    n = 12
    q, k, v = (torch.randn(n, 1, d, generator=g).to(BF).to(DEV) for _ in range(3))
    # seq 0: 3 rows, 2 keys (first row has none); seq 1: 4 rows ending at key 34 of a 2-page table; seq 2: page 9 of 3
    step = T.Step(i32([0, 3, 7, 9]), i32([2, 34, 2]), i32([[0, -7], [1, 2], [9, -7]]))
    qo = torch.full((n, 1, d), 7.0, dtype=BF, device=DEV)
    T.append(T.PagedCache(kc, vc), step, q, k, v, q_out=qo)
    torch.cuda.synchronize()
    for src, own, page, at in ((1, 0, 0, 0), (2, 1, 0, 1), (3, 30, 2, 14), (4, 31, 2, 15)):
        k0[page, at], v0[page, at] = k[src], v[src]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    assert torch.equal(qo[:9], q[:9]) and bool((qo[9:] == 7).all())


def test_append_in_place_and_without_queries(T):
    d = 128
    kc, vc = caches(2, 16, 2, d, BF)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, 8 * d, generator=g).to(BF).to(DEV)
    q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([4 * d, 2 * d, 2 * d], 1))
    step = T.Step(i32([0, 4]), i32([4]), i32([[1]]))
    rope, gain = T.Rope(d), torch.ones(d, device=DEV)
    c = T.PagedCache(kc, vc)
    want = T.append(c, step, q, k, v, rope=rope, q_gain=gain)
    k1, v1 = kc.clone(), vc.clone()
    kc.zero_(), vc.zero_()
    assert T.append(c, step, None, k, v, rope=rope) is None
    assert torch.equal(kc[1, :4], k1[1, :4]) and torch.equal(vc[1, :4], v1[1, :4])
    T.append(c, step, q, k, v, rope=rope, q_gain=gain, q_out=q)
    assert torch.equal(q, want)


# ------------------------------------------------------------------ attention
ATTEND = [
    # rows, kv, hq, hkv, d, page, dtype, causal, prefix, hnd
    ([1], [1], 1, 1, 64, 16, BF, True, 0, False),
    ([1], [777], 32, 4, 128, 64, BF, True, 0, False),
    ([1], [128], 8, 1, 128, 128, HF, True, 0, False),
    ([16], [16], 8, 2, 128, 64, BF, True, 0, True),
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
]


def attend_case(T, case, seed=0, **kw):
    rows, kv, hq, hkv, d, page, dt, causal, prefix, hnd = case
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=seed)
    kc, vc = caches(n_pages, page, hkv, d, dt, hnd=hnd, seed=seed + 1)
    # what lies behind the last keys, and on pages nobody names, is NaN
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    for pages, n in [(pre, prefix)] + [(table[i], n) for i, n in enumerate(kv)]:
        for j in range(n):
            used[int(pages[j // page]), j % page] = True
    for c in (kc, vc):
        c.masked_fill_(~used.to(DEV)[:, :, None, None], float("nan"))
    g = torch.Generator().manual_seed(seed + 2)
    q = torch.randn(starts[-1], hq, d, generator=g).to(dt).to(DEV)
    step = T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), prefix)
    ws = torch.empty(T.PagedCache(kc, vc).workspace_bytes(starts[-1], hq), dtype=torch.uint8, device=DEV)
    o, lse = T.attention(T.PagedCache(kc, vc), step, q, causal=causal, workspace=ws, **kw)
    T.attention_status(ws)
    return (starts, kv, table, pre, kc, vc, q, step), o, lse


def close(o, lse, want):
    wo, to, wl, tl = want
    e = np.abs(o.double().cpu().numpy() - wo)
    assert np.all(e <= to), (float(np.max(e / to)), np.unravel_index(np.argmax(e / to), e.shape))
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isinf(l), np.isinf(wl)) and np.all(l[np.isinf(l)] < 0)
    f = ~np.isinf(wl)
    assert np.all(np.abs(l[f] - wl[f]) <= tl[f])


@pytest.mark.parametrize("case", ATTEND, ids=[f"{i}" for i in range(len(ATTEND))])
def test_attention(T, case):
    rows, _, hq, hkv, d, page, dt, causal, prefix, hnd = case
    (starts, kv, table, pre, kc, vc, q, _), o, lse = attend_case(T, case)
    close(o, lse, R.attend_step(q, kc, vc, starts, kv, table, pre, prefix, page, causal=causal, scale=d ** -0.5))


def test_attention_random_steps(T):
    import random
    r = random.Random(11)
    for seed in range(12):
        hkv, n = r.choice([1, 2, 4]), r.randint(1, 9)
        rows = [r.choice([0, 1, r.randint(1, 20), r.randint(1, 90)]) for _ in range(n)]
        kv = [t + r.choice([0, r.randint(0, 40), r.randint(0, 700)]) for t in rows]
        rows[0], kv[0] = max(rows[0], 1), max(kv[0], 1)
        case = (rows, kv, hkv * r.choice([1, 2, 3, 8]), hkv, r.choice([64, 128]), r.choice([16, 32, 64, 128, 256]),
                r.choice([BF, HF]), r.random() < 0.7, r.choice([0, r.randint(1, 600)]), r.random() < 0.5)
        (starts, kv, table, pre, kc, vc, q, _), o, lse = attend_case(T, case, seed=100 + seed)
        close(o, lse, R.attend_step(q, kc, vc, starts, kv, table, pre, case[8], case[5], causal=case[7],
                                    scale=case[4] ** -0.5))


@pytest.mark.parametrize("case", [
    # enough blocks for every CTA to go round its ring of K and V tiles several times, in every mode
    ([2], [60000], 8, 8, 128, 64, BF, True, 0, False),
    ([1, 3], [41000, 20001], 8, 8, 64, 128, HF, True, 1000, True),
    ([90, 1, 2], [9000, 15000, 11000], 32, 4, 128, 64, BF, True, 3000, False),
    ([1] * 300, [5 + i % 380 for i in range(300)], 4, 4, 128, 16, BF, True, 0, False),
    # a batch of many places, most of them without rows
    ([2 if i % 97 == 5 else 0 for i in range(4096)], [300 if i % 97 == 5 else i % 3 for i in range(4096)], 8, 2, 64,
     16, BF, True, 200, False),
    # many more rows than the CTAs' last items have: merged by CTA
    ([1500, 3, 900, 0, 1], [1500, 2000, 950, 10, 1], 32, 4, 64, 64, HF, True, 0, False),
    ([1400, 700], [1400, 900], 24, 2, 128, 16, BF, False, 0, True),
    # one kv head: rows with a part in every CTA, more than 32 for each of a merging block's warps
    ([3], [50000], 4, 1, 128, 64, BF, True, 0, False),
    ([1, 0, 2, 1], [400, 7, 300, 1], 2, 1, 64, 32, HF, True, 40000, False),
], ids=["single", "single-d64", "pair-and-single", "many-short", "many-empty", "prompts", "prompts-not-causal",
        "one-head", "one-head-prefix"])
def test_attention_long(T, case):
    rows, _, hq, hkv, d, page, dt, causal, prefix, hnd = case
    (starts, kv, table, pre, kc, vc, q, _), o, lse = attend_case(T, case, seed=40)
    close(o, lse, R.attend_step(q, kc, vc, starts, kv, table, pre, prefix, page, causal=causal, scale=d ** -0.5))


def test_attention_large_scores_scale_and_strided_rows(T):
    """Scores far apart (the running maximum moves often), a scale of the caller's, queries and results inside wider
    rows."""
    starts, kv, table, pre, n_pages = R.make_step([20, 3], [900, 400], 64, prefix=300, seed=3)
    kc, vc = caches(n_pages, 64, 2, 128, BF, seed=4)
    g = torch.Generator().manual_seed(5)
    wide = (3 * torch.randn(23, 8, 128, generator=g)).to(BF).to(DEV)
    q = wide[:, :6]
    out = torch.zeros(23, 9, 128, dtype=BF, device=DEV)
    step = T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), 300)
    o, lse = T.attention(T.PagedCache(kc, vc), step, q, scale=0.5, out=out[:, :6])
    want = R.attend_step(q, kc, vc, starts, kv, table, pre, 300, 64, causal=True, scale=0.5)
    close(o, lse, want)
    assert bool((out[:, 6:] == 0).all())


def test_attention_values_that_are_not_finite_in_masked_places(T):
    """NaN and infinite keys and values of the step's later rows do not reach the earlier ones; a row that sees such a
    value has NaN in that element only."""
    rows, kv, d = [40], [400], 128
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, 64, prefix=130, seed=6)
    kc, vc = caches(n_pages, 64, 1, d, BF, seed=7)
    g = torch.Generator().manual_seed(8)
    q = torch.randn(40, 4, d, generator=g).to(BF).to(DEV)
    step = T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), 130)
    want = R.attend_step(q, kc, vc, starts, kv, table, pre, 130, 64, causal=True, scale=d ** -0.5)

    def at(key):
        return int(table[0, key // 64]), key % 64

    p, r = at(380)                       # step row 20
    vc[p, r, 0, 5] = float("nan")
    vc[p, r, 0, 70] = float("inf")
    p, r = at(399)                       # the last row's own key
    kc[p, r] = float("nan")
    o, lse = T.attention(T.PagedCache(kc, vc), step, q)
    o = o.double().cpu().numpy()
    wo, to, wl, _ = want
    assert np.all(np.abs(o - wo)[:20] <= to[:20])
    ok = np.ones(d, dtype=bool)
    ok[[5, 70]] = False
    assert np.all(np.abs(o - wo)[20:39][..., ok] <= to[20:39][..., ok])
    assert np.isnan(o[20:39][..., ~ok]).all()
    assert np.isnan(o[39]).all() and np.isnan(lse[39].cpu().numpy()).all()
    assert np.isfinite(lse[:39].cpu().numpy()).all()


def test_attention_rows_behind_the_last_sequence(T):
    starts, kv, table, pre, n_pages = R.make_step([2, 3], [70, 20], 16, seed=9)
    kc, vc = caches(n_pages, 16, 2, 64, HF, seed=10)
    q = torch.randn(9, 4, 64, generator=torch.Generator().manual_seed(11)).to(HF).to(DEV)
    out, lse = torch.full((9, 4, 64), 3.0, dtype=HF, device=DEV), torch.full((9, 4), 3.0, device=DEV)
    T.attention(T.PagedCache(kc, vc), T.Step(i32(starts), i32(kv), table.to(DEV)), q, out=out, lse=lse)
    want = R.attend_step(q[:5], kc, vc, starts, kv, table, pre, 0, 16, causal=True, scale=64 ** -0.5)
    close(out[:5], lse[:5], want)
    assert bool((out[5:] == 3).all()) and bool((lse[5:] == 3).all())


def test_attention_lengths_past_the_table_and_missing_pages(T):
    """A length past the block table reads the keys it has room for; a page outside the pool reads as zeros."""
    kc, vc = caches(4, 16, 1, 64, BF, seed=12)
    q = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(13)).to(BF).to(DEV)
    table = torch.tensor([[2, 0], [1, 77]], dtype=torch.int32)
    o, lse = T.attention(T.PagedCache(kc, vc), T.Step(i32([0, 1, 2]), i32([1000, 20]), table.to(DEV)), q)
    kz, vz = torch.cat([kc, torch.zeros_like(kc[:1])]), torch.cat([vc, torch.zeros_like(vc[:1])])
    table[1, 1] = 4
    want = R.attend_step(q, kz, vz, [0, 1, 2], [32, 20], table, torch.zeros(0, dtype=torch.int32), 0, 16, causal=False,
                         scale=0.125)
    close(o, lse, want)


def test_attention_repeats_bit_for_bit_and_replays(T):
    """Two calls agree in every bit; a captured step replays with the lengths its tensors hold then."""
    case = ATTEND[5]
    (starts, kv, table, pre, kc, vc, q, step), o, lse = attend_case(T, case, seed=20)
    o2, l2 = T.attention(T.PagedCache(kc, vc), step, q)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    kv_len, cache = i32(kv), T.PagedCache(kc, vc)
    step = T.Step(i32(starts), kv_len, table.to(DEV), pre.to(DEV), 2053)
    out, lse = torch.empty_like(q), torch.empty_like(lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        T.attention(cache, step, q, out=out, lse=lse)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        T.attention(cache, step, q, out=out, lse=lse)
    shorter = [200, 17, 3, 60]
    for lens in (kv, shorter):
        kv_len.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        want = R.attend_step(q, kc, vc, starts, lens, table, pre, 2053, 16, causal=True, scale=64 ** -0.5)
        close(out, lse, want)


def test_attention_with_room_for_one_block_of_keys(T):
    """A block table of at most 128 keys (nothing to merge) and a wider one of the same keys: the same bits."""
    rows, kv = [1, 0, 17, 4, 2], [128, 3, 17, 2, 0]
    starts, kv, table, _, n_pages = R.make_step(rows, kv, 32, seed=14)
    assert table.shape[1] == 4
    kc, vc = caches(n_pages, 32, 2, 128, BF, seed=15)
    q = torch.randn(starts[-1] + 2, 10, 128, generator=torch.Generator().manual_seed(16)).to(BF).to(DEV)
    cache, got = T.PagedCache(kc, vc), []
    for extra in (0, 1):
        wide = torch.cat([table, table[:, :extra]], 1)
        out, lse = torch.full_like(q, 3), torch.full((len(q), 10), 3.0, device=DEV)
        ws = torch.empty(cache.workspace_bytes(len(q), 10), dtype=torch.uint8, device=DEV)
        T.attention(cache, T.Step(i32(starts), i32(kv), wide.to(DEV)), q, out=out, lse=lse, workspace=ws)
        T.attention_status(ws)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    out, lse = got[0]
    n = starts[-1]
    close(out[:n], lse[:n], R.attend_step(q[:n], kc, vc, starts, kv, table, torch.zeros(0, dtype=torch.int32), 0, 32,
                                          causal=True, scale=128 ** -0.5))
    assert bool((out[n:] == 3).all()) and bool((lse[n:] == 3).all())


def test_two_calls_at_once(T):
    """Calls on two streams, each with a workspace of its own, as they would run one after the other."""
    calls = [attend_case(T, ATTEND[i], seed=30 + i) for i in (5, 13)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for i, ((_, _, _, _, kc, vc, q, step), _, _) in enumerate(calls):
            got[i].append(T.attention(T.PagedCache(kc, vc), step, q, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (_, o, lse) in enumerate(calls):
        assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in got[i])


def test_operators_on_another_stream(T):
    """Inputs made on one stream, the call on another, ordered by the caller."""
    case = ATTEND[4]
    s = torch.cuda.Stream()
    (starts, kv, table, pre, kc, vc, q, step), o, lse = attend_case(T, case, seed=21)
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = T.attention(T.PagedCache(kc, vc), step, q, stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    # append and verification, with tensors that go out of use before they have run
    k, v = (torch.randn(q.shape[0], 2, 128, device=DEV).to(BF) for _ in range(2))
    c = T.PagedCache(kc, vc)
    want = T.append(c, step, q, k, v, rope=T.Rope(128))
    args = [t.to(DEV) if t is not None else None for t in verify_case(4, 5, 30000, F4, False, True, seed=2)]
    ref = T.verify_tokens(*args[:4], draft_probs=args[4], n_draft=args[5])
    gone = [t.clone() for t in (q, k, v)]
    gone2 = [t.clone() if t is not None else None for t in args]
    s.wait_stream(torch.cuda.current_stream())
    got = T.append(c, step, *gone, rope=T.Rope(128), stream=s)
    tok = T.verify_tokens(*gone2[:4], draft_probs=gone2[4], n_draft=gone2[5], stream=s)
    del gone, gone2
    torch.zeros(1 << 22, device=DEV).fill_(7)      # may take over memory that was let go
    s.synchronize()
    assert torch.equal(tok[0], ref[0]) and torch.equal(tok[1], ref[1])
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------ verification
def verify_case(n, k, V, dt, greedy, ragged, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, k + 1, V, generator=g)
    tp = torch.softmax(3 * z, -1).to(dt)
    y = 0.97 * z[:, :k] + 0.25 * torch.randn(n, k, V, generator=g)
    dp = None if greedy else torch.softmax(3 * y, -1).to(dt)
    if greedy or k == 0:
        draft = y.argmax(-1).to(torch.int32) if k else torch.zeros(n, 0, dtype=torch.int32)
    else:
        draft = torch.multinomial(dp.float().flatten(0, 1), 1, generator=g).view(n, k).to(torch.int32)
    nd = torch.randint(0, k + 1, (n,), generator=g).to(torch.int32) if ragged else None
    return draft, tp, torch.rand(n, k, generator=g), torch.rand(n, generator=g), dp, nd


def run_verify(T, draft, tp, ua, ut, dp=None, nd=None):
    d = lambda t: None if t is None else t.to(DEV)
    tok, acc = T.verify_tokens(d(draft), d(tp), d(ua), d(ut), draft_probs=d(dp), n_draft=d(nd))
    torch.cuda.synchronize()
    return tok.cpu().numpy(), acc.cpu().numpy()


@pytest.mark.parametrize("n,k,V,dt,greedy,ragged", [
    (1, 15, 32768, F4, True, False), (7, 5, 1000, F4, False, True), (3, 15, 100003, F4, False, True),
    (5, 4, 50001, BF, False, False), (4, 3, 65536, HF, False, True), (2, 40, 517, F4, True, True),
    (9, 1, 1, F4, True, False), (6, 2, 17, F4, False, False), (8, 0, 4099, F4, True, False),
    (2, 1, 262144, BF, True, False), (2, 2, 300001, F4, False, False),
    (3, 2, 70013, F4, False, False), (3, 2, 70014, F4, False, True), (5, 3, 40007, HF, False, False),
    (4, 2, 90010, BF, False, False), (300, 2, 3001, F4, False, True), (160, 1, 20011, BF, False, False),
])
def test_verify(T, n, k, V, dt, greedy, ragged):
    args = verify_case(n, k, V, dt, greedy, ragged, seed=n * 1000 + k)
    tok, acc = run_verify(T, *args)
    wt, wa = R.verify(*args)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)


def test_verify_many_draws(T):
    """2048 draws over 10^5 tokens: sums as exact as 64 bits give, not one neighbour taken instead."""
    V = 100001
    draft, tp, _, _, dp, _ = verify_case(2, 1, V, F4, False, False, seed=77)
    n = 1024
    for i in range(2):
        g = torch.Generator().manual_seed(i)
        big = [draft[i:i + 1].expand(n, 1), tp[i:i + 1].expand(n, 2, V), torch.rand(n, 1, generator=g),
               torch.rand(n, generator=g), dp[i:i + 1].expand(n, 1, V)]
        tok, acc = run_verify(T, *big)
        p, q, x = R.weights(tp[i]), R.weights(dp[i, 0]), int(draft[i, 0])
        take = big[2].double().numpy()[:, 0] * q[x] < p[0, x]
        cums = [np.cumsum(np.maximum(p[0] - q, 0)), np.cumsum(p[1])]
        want = [np.searchsorted(cums[int(t)], u * cums[int(t)][-1], side="right")
                for t, u in zip(take, big[3].double().numpy())]
        assert np.array_equal(acc, take.astype(int))
        assert np.array_equal(tok[np.arange(n), acc], want)


def test_verify_borders(T):
    """Drafts outside the vocabulary, u at its ends and past them, nothing left of p - q, rows without weight, NaN,
    infinite and negative entries."""
    V, k = 1000, 2
    tp, dp = torch.zeros(10, k + 1, V), torch.zeros(10, k, V)
    tp[:, :, 100:200] = 0.01
    dp[:, :, 150:250] = 0.01
    draft = torch.full((10, k), 160, dtype=torch.int32)
    ua, ut = torch.full((10, k), 0.5), torch.full((10,), 0.5)
    draft[0, 0], draft[1, 0] = -1, V                       # rejected
    draft[2, 0], ut[2] = 210, 0.0                          # p(x) = 0: rejected; the first index with weight
    draft[3, 0], ut[3] = 210, 1.0                          # the last one
    draft[4, 0], ut[4] = 210, float("nan")                 # as 0
    dp[5, 0] = tp[5, 0]
    ua[5, 0] = 1.0                                         # rejected with p = q: drawn from p
    tp[6, 0] = 0                                           # rejected, and p has no weight
    tp[7, 0, 100:150] = float("nan")
    tp[7, 0, 5], tp[7, 0, 6], draft[7, 0] = float("inf"), -1.0, 210
    ut[8], ut[9] = 1.0 - 2.0 ** -24, -3.0                  # all taken: from the last row
    dp[7, 0, 100:] = 0
    tok, acc = run_verify(T, draft, tp, ua, ut, dp)
    wt, wa = R.verify(draft, tp, ua, ut, dp)
    assert np.array_equal(acc, wa)
    assert np.array_equal(tok, wt)
    assert tok[2, 0] == 100 and tok[3, 0] == 149 and tok[6, 0] == 0


def test_verify_views(T):
    """The block of draft_tokens without its anchor, rows padded to a wider vocabulary, the same draft twice."""
    n, k, V = 3, 15, 5000
    draft, tp, ua, ut, _, _ = verify_case(n, k, V, F4, True, False, seed=9)
    draft[:, 3] = draft[:, 2]
    block = torch.cat([torch.zeros(n, 1, dtype=torch.int32), draft], 1).to(DEV)
    wide = torch.full((n, k + 1, V + 37), 9.0, device=DEV)
    wide[..., :V] = tp.to(DEV)
    tok, acc = T.verify_tokens(block[:, 1:], wide[..., :V], ua.to(DEV), ut.to(DEV))
    wt, wa = R.verify(draft, tp, ua, ut)
    assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)


def test_append_many_sequences(T):
    """More sequences than a warp looks at in one go, most of them without rows."""
    n, d = 2500, 64
    rows = [3 if i % 7 == 0 else 0 for i in range(n)]
    kv = [t + i % 4 for i, t in enumerate(rows)]
    starts, kv, table, _, n_pages = R.make_step(rows, kv, 16, seed=8)
    kc, vc = caches(n_pages, 16, 1, d, HF)
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(starts[-1], 1, d, generator=g).to(HF).to(DEV) for _ in range(2))
    T.append(T.PagedCache(kc, vc), T.Step(i32(starts), i32(kv), table.to(DEV)), None, k, v)
    own = [(int(table[i, j // 16]), j % 16) for i, t in enumerate(rows) for j in range(kv[i] - t, kv[i])]
    p, r = (torch.tensor(x, device=DEV) for x in zip(*own))
    assert torch.equal(kc[p, r], k) and torch.equal(vc[p, r], v)


def test_bad_device_arrays_stay_in_bounds(T):
    """Lengths, row starts and page ids outside their ranges: nothing outside the buffers is touched, nothing hangs."""
    d, rows = 64, 8
    kc, vc = caches(4, 16, 2, d, BF, seed=3)
    q = torch.randn(rows, 4, d, generator=torch.Generator().manual_seed(4)).to(BF).to(DEV)
    kv = torch.randn(rows, 2, d, generator=torch.Generator().manual_seed(5)).to(BF).to(DEV)
    big = 2 ** 31 - 1
    for starts, lens, pages in [([0, 100, 200], [5, 5], [[0], [1]]), ([0, 8, 3], [5, 5], [[0], [1]]),
                                ([-5, 4, 8], [-3, big], [[0], [1]]), ([0, 4, 8], [16, 16], [[-1], [big]]),
                                ([8, 8, 8], [16, 16], [[0], [1]]), ([5, 0, 8], [3, big], [[99], [-big]])]:
        guard = torch.full((rows + 16, 4, d), 5.0, dtype=BF, device=DEV)
        cache, step = T.PagedCache(kc, vc), T.Step(i32(starts), i32(lens), i32(pages), i32([7, -1]), 20)
        T.append(cache, step, q, kv, kv, q_out=guard[:rows])
        out = torch.full((rows + 16, 4, d), 5.0, dtype=BF, device=DEV)
        ws = torch.empty(cache.workspace_bytes(rows, 4), dtype=torch.uint8, device=DEV)
        T.attention(cache, step, q, out=out[:rows], workspace=ws)
        T.attention_status(ws)
        assert bool((out[rows:] == 5).all()) and bool((guard[rows:] == 5).all())
