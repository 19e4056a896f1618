"""More of the step operators on the GPU: the calls their documentation allows and tests/test_target_step.py does not
make."""
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


def inputs(T, rows, kv, hq, hkv, d, page, dt, prefix=0, seed=0):
    """(starts, table, prefix pages, k, v, q, step) of random values, all on the GPU but the index lists."""
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    k, v = (torch.randn(n_pages, page, hkv, d, generator=g).to(dt).to(DEV) for _ in range(2))
    q = torch.randn(starts[-1], hq, d, generator=g).to(dt).to(DEV)
    return starts, table, pre, k, v, q, T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), prefix)


def close(o, lse, want):
    wo, to, wl, tl = want
    assert np.all(np.abs(o.double().cpu().numpy() - wo) <= to)
    assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= tl)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("d,dt", [(64, HF), (128, BF)])
def test_items_of_two_streams_merge_the_same_every_time(T, d, dt):
    """Few rows of many lengths: each item's even and odd blocks are two accumulators, read across the two streams
    right behind their last product.  Every call gives the same bits, and the right ones."""
    kv = [129 + 97 * i % 1400 for i in range(150)]
    rows = [1 + i % 2 for i in range(150)]
    starts, table, pre, k, v, q, step = inputs(T, rows, kv, 8, 2, d, 64, dt, seed=1)
    cache = T.PagedCache(k, v)
    first = T.attention(cache, step, q)
    for _ in range(60):
        o, lse = T.attention(cache, step, q)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    close(*first, R.attend_step(q, k, v, starts, kv, table, pre, 0, 64, causal=True, scale=d ** -0.5))


@pytest.mark.parametrize("rows", [1, 256], ids=["single", "pair"])
@pytest.mark.parametrize("drop", [20, 22.7, 25.5, 28])
def test_f16_keys_far_below_the_largest_still_count(T, rows, drop):
    """One key, then 131071 whose weights are 2^-drop of its own: the tail is up to an eighth of the sum, and half or
    all of it goes through one running maximum.  (All sequences read the same pages; what they return is one row.)"""
    n, page, d, n_seq = 131072, 256, 64, 304 // (1 if rows == 1 else 2)
    k, v = (torch.zeros(n // page, page, 1, d, dtype=HF, device=DEV) for _ in range(2))
    half = torch.tensor(drop * math.log(2) / 2).to(HF)          # scores a * (+-half) / 8 with a = 8
    k[..., 0], v[:] = -half, 1
    v[..., 1::2] = -0.75
    k[0, 0, 0, 0], v[0, 0] = half, 0
    q = torch.zeros(n_seq * rows, 1, d, dtype=HF, device=DEV)
    q[..., 0] = 8
    table = i32([list(range(n // page))]).expand(n_seq, n // page)
    step = T.Step(i32([i * rows for i in range(n_seq + 1)]), i32([n] * n_seq), table)
    o, lse = T.attention(T.PagedCache(k, v), step, q, causal=False)
    w = math.exp(-2 * float(half))
    l = 1 + (n - 1) * w
    tail = (n - 1) * w / l
    want = torch.where(torch.arange(d) % 2 == 0, tail, -0.75 * tail).double()
    # the result's rounding and the weights' (2^-11 each, on values of one sign), scores of at most 10 after three
    # roundings in f32 and their exponentials (2^-17 in all), sums of n terms in f32, 2^-32 of the largest weight a key
    tol = (2.0 ** -10 * 1.01 + 2.0 ** -17 + (n + 64) * 2.0 ** -23) * want.abs() + n * 2.0 ** -32 / l
    e = (o[:, 0].double().cpu() - want).abs()
    assert bool((e <= tol).all()), (float(e.max()), tail)
    want_lse = float(half) + math.log(l)
    assert float((lse.double().cpu() - want_lse).abs().max()) <= (n + 64) * 2.0 ** -24 + 2.0 ** -20 * abs(want_lse)


@pytest.mark.parametrize("rows,kv,hq,hkv,prefix", [
    ([600], [8000], 1, 1, 0), ([600], [8000], 4, 1, 0), ([2000], [2000], 32, 2, 0),
    ([16], [300], 4, 1, 700), ([16] * 4, [300] * 4, 32, 4, 700), ([16] * 10, [300] * 10, 32, 4, 700),
], ids=["block", "warp", "by-cta", "prefix-block", "prefix-warp", "prefix-half-warp"])
def test_values_that_are_not_finite_reach_rows_through_any_merge(T, rows, kv, hq, hkv, prefix):
    """A NaN or infinite value, or a NaN key, whose part of the keys weighs nothing beside the rest (120 below the
    largest score) is seen all the same."""
    d, page = 64, 64
    starts, table, pre, k, v, q, step = inputs(T, rows, kv, hq, hkv, d, page, BF, prefix=prefix, seed=3)
    q[:] = 0
    q[..., 0] = 8
    n, t = kv[0], rows[0]
    # own keys from here on score 120 less than the others and the prefix's
    turn = 0 if prefix else n - t if n > t else 1000
    bad = n - t + 5 if n > t else 1100
    k[pre.long().to(DEV), ..., 0] = 60.0
    for i in range(len(rows)):
        j = torch.arange(n)
        p, r = table[i][j // page].long(), j % page
        k[p, r, :, 0] = torch.where(j < turn, 60.0, -60.0).to(BF).to(DEV)[:, None]
    want = R.attend_step(q, k, v, starts, kv, table, pre, prefix, page, causal=True, scale=d ** -0.5)
    for i in range(len(rows)):
        at = int(table[i, bad // page]), bad % page
        v[at][:, 3], v[at][:, 7] = float("nan"), float("inf")
        k[int(table[i, (n - 1) // page]), (n - 1) % page] = float("nan")     # the last row's own key
    o, lse = T.attention(T.PagedCache(k, v), step, q)
    o, lse, (wo, to, wl, tl) = o.double().cpu().numpy(), lse.double().cpu().numpy(), want
    own = np.concatenate([n - t + np.arange(t)] * len(rows))                 # each row's own key
    last = own == n - 1
    assert np.isnan(o[last]).all() and np.isnan(lse[last]).all()
    assert np.all(np.abs(lse - wl)[~last] <= tl[~last])
    sees = np.zeros(o.shape, dtype=bool)
    sees[own >= bad, :, 3] = sees[own >= bad, :, 7] = True
    assert not np.isfinite(o[sees]).any()
    sees[last] = True
    assert np.all(np.abs(o - wo)[~sees] <= to[~sees])


def test_status_of_what_is_no_workspace_is_refused(T):
    """A tensor shorter than the words it would be read for, or not the bytes a call was given."""
    from speculative_decoding_block_ingest_gb300.dflash import DflashError
    ok = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    T.attention_status(ok)
    for bad in (ok[:4095], ok[:0], ok.view(torch.int32), ok.view(2, 2048), torch.zeros(16384, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(DflashError):
            T.attention_status(bad)
    # the smallest workspace there is holds them
    k = torch.zeros(1, 16, 1, 64, dtype=BF, device=DEV)
    assert T.PagedCache(k, k.clone()).workspace_bytes(0, 1) >= 4096


class Guarded:
    """Buffers inside larger ones; what lies on either side has to stay."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype, value):
        n, pad = math.prod(shape), 512
        flat = torch.full((n + 2 * pad,), value, dtype=dtype, device=DEV)
        self.all.append((flat, n, pad, value))
        return flat[pad:pad + n].view(shape)

    def untouched(self):
        return all(bool((f[:p] == x).all()) and bool((f[p + n:] == x).all()) for f, n, p, x in self.all)


BIG = 2 ** 31 - 1
BAD_SMALL = [([0, 100, 200], [5, 5], [[0], [1]]), ([0, 8, 3], [5, 5], [[0], [1]]), ([-5, 4, 8], [-3, BIG], [[0], [1]]),
             ([0, 4, 8], [16, 16], [[-1], [BIG]]), ([8, 8, 8], [16, 16], [[0], [1]]),
             ([5, 0, 8], [3, BIG], [[99], [-BIG]]), ([0, 4, 8], [16, 3], [[2], [2]])]
FAR = 5000
BAD_LARGE = [([0, FAR] * 6 + [0], [200] * 12, [[i % 8, 1, 2, -4] for i in range(12)]),
             ([-9, 2500, BIG], [BIG, 4000], [[0, 1, 2, 3], [4, 77, 6, 7]]),
             ([0, 4000, 3999, FAR], [250, 250, 250], [[0, 1, 2, 3]] * 3), ([FAR, 0, 0], [9, 9], [[0, 1, 2, 3]] * 2),
             ([0, 10, FAR], [-BIG, 256], [[0, 1, 2, 3], [4, 5, 6, 7]])]


@pytest.mark.parametrize("starts,lens,pages,prefix,rows,page,heads",
                         [(*c, p, 8, 16, 4) for c in BAD_SMALL for p in (20, 0)]
                         + [(*c, p, FAR, 64, 8) for c in BAD_LARGE for p in (0, 150)])
def test_bad_device_arrays_write_nothing_else(T, starts, lens, pages, prefix, rows, page, heads):
    """Row starts, lengths and pages out of range, through every way of merging: buffers keep their surroundings, the
    caches every row that no (sequence, key) in range names."""
    d, hkv = 64, 2
    new, g = Guarded(), torch.Generator().manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)
    kc, vc = (new((8, page, hkv, d), BF, 5.0) for _ in range(2))
    kc.copy_(rnd(*kc.shape)), vc.copy_(rnd(*vc.shape))
    before = kc.clone(), vc.clone()
    q, kv = rnd(rows, heads, d), rnd(rows, hkv, d)
    cache, step = T.PagedCache(kc, vc), T.Step(i32(starts), i32(lens), i32(pages), i32([7, -1, BIG]), prefix)
    T.append(cache, step, q, kv, kv, q_out=new(q.shape, BF, 5.0))
    torch.cuda.synchronize()
    s = [min(max(x, 0), rows) for x in starts]
    falls = s[0] != 0 or any(b < a for a, b in zip(s, s[1:]))      # rows of no known sequence
    named = torch.zeros(8, page, dtype=torch.bool)
    for i, n in enumerate(lens):
        own = range(len(pages[i]) * page) if falls else range(max(n, 0) - (s[i + 1] - s[i]), max(n, 0))
        for j in own:
            if 0 <= j < len(pages[i]) * page and 0 <= pages[i][j // page] < 8:
                named[pages[i][j // page], j % page] = True
    for c, b in zip((kc, vc), before):
        assert torch.equal(c[~named.to(DEV)], b[~named.to(DEV)])
    need = cache.workspace_bytes(rows, heads)
    ws, out, lse = new((need,), torch.uint8, 90), new(q.shape, BF, 5.0), new((rows, heads), F4, 5.0)
    kept = kc.clone(), vc.clone()
    for causal in (True, False):
        T.attention(cache, step, q, out=out, lse=lse, workspace=ws, causal=causal)
        T.attention_status(ws)
    assert torch.equal(kc, kept[0]) and torch.equal(vc, kept[1])
    assert new.untouched()
    if not falls:
        assert bool((out[s[-1]:] == 5).all()) and bool((lse[s[-1]:] == 5).all())


# ------------------------------------------------------------------ offsets past 32 bits
FAR_ROW = 1_200_000_000      # elements between rows: the third starts behind 2^31


def test_append_and_attention_far_into_large_pools(T):
    """Pages, query rows and results whose offsets pass 2^31 elements, both layouts of the pool."""
    n_pages, page, hkv, d, hq = 20011, 256, 8, 64, 16           # 2.6e9 elements each
    for hnd in (False, True):
        shape = (n_pages, hkv, page, d) if hnd else (n_pages, page, hkv, d)
        kc, vc = (torch.empty(*shape, dtype=BF, device=DEV) for _ in range(2))
        if hnd:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        table = torch.tensor([[n_pages - 1, 3, 17000], [16500, 19999, 0]], dtype=torch.int32)
        rows, kv, starts = [2, 1], [600, 700], [0, 2, 3]
        g = torch.Generator().manual_seed(11)
        for p in table.flatten().tolist():
            kc[p], vc[p] = (torch.randn(page, hkv, d, generator=g).to(BF).to(DEV) for _ in range(2))
        wide = torch.empty(2 * FAR_ROW + hq * d, dtype=BF, device=DEV)
        q = wide.as_strided((3, hq, d), (FAR_ROW, d, 1))
        q.copy_(torch.randn(3, hq, d, generator=g).to(BF))
        k, v = (torch.randn(3, hkv, d, generator=g).to(BF).to(DEV) for _ in range(2))
        cache, step = T.PagedCache(kc, vc), T.Step(i32(starts), i32(kv), table.to(DEV))
        assert T.append(cache, step, q, k, v, q_out=q) is q          # in place, no norm and no rotation
        for row, (i, own) in enumerate([(0, 598), (0, 599), (1, 699)]):
            p = int(table[i, own // page])
            assert torch.equal(kc[p, own % page], k[row]) and torch.equal(vc[p, own % page], v[row])
        far = torch.empty(2 * FAR_ROW + hq * d, dtype=BF, device=DEV).as_strided((3, hq, d), (FAR_ROW, d, 1))
        o, lse = T.attention(cache, step, q, out=far)
        used = table.flatten().tolist()
        small = torch.arange(6, dtype=torch.int32).view(2, 3)
        close(o, lse, R.attend_step(q, kc[used], vc[used], starts, kv, small, torch.zeros(0, dtype=torch.int32), 0, page,
                                    causal=True, scale=d ** -0.5))
        del kc, vc, cache, wide, far, q, o


def test_verify_rows_far_apart(T):
    n, k, V = 3, 2, 5003
    g = torch.Generator().manual_seed(12)
    tp, dp = (torch.softmax(3 * torch.randn(n, m, V, generator=g), -1) for m in (k + 1, k))
    draft = tp[:, :k].argmax(-1).to(torch.int32)
    ua, ut = torch.rand(n, k, generator=g), torch.rand(n, generator=g)
    far = []
    for x, (s0, s1) in ((tp, (FAR_ROW, 100_000_001)), (dp, (FAR_ROW + 3, 2 ** 27))):
        buf = torch.empty((n - 1) * s0 + (x.shape[1] - 1) * s1 + V, device=DEV)
        far.append(buf.as_strided(x.shape, (s0, s1, 1)))
        far[-1].copy_(x)
    tok, acc = T.verify_tokens(draft.to(DEV), far[0], ua.to(DEV), ut.to(DEV), draft_probs=far[1])
    wt, wa = R.verify(draft, tp, ua, ut, dp)
    assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)


def test_steps_without_rows(T):
    """A step of no rows, and buffers whose sequences have none."""
    kc, vc = (torch.ones(2, 16, 2, 64, dtype=BF, device=DEV) for _ in range(2))
    cache = T.PagedCache(kc, vc)
    for n in (0, 5):
        step = T.Step(i32([0, 0, 0]), i32([3, 0]), i32([[0], [1]]), i32([1]), 7)
        q, k = torch.ones(n, 4, 64, dtype=BF, device=DEV), torch.zeros(n, 2, 64, dtype=BF, device=DEV)
        out, lse = torch.full_like(q, 3), torch.full((n, 4), 3.0, device=DEV)
        ws = torch.full((cache.workspace_bytes(n, 4),), 90, dtype=torch.uint8, device=DEV)
        T.append(cache, step, q, k, k, rope=T.Rope(64))
        T.attention(cache, step, q, out=out, lse=lse, workspace=ws)
        T.attention_status(ws)
        assert bool((kc == 1).all()) and bool((vc == 1).all()) and bool((out == 3).all()) and bool((lse == 3).all())


# ------------------------------------------------------------------ verification
def drawn(T, tp, ut):
    """Tokens drawn from the rows of tp [n, V] (no drafts), into memory that holds -7."""
    import ctypes
    from speculative_decoding_block_ingest_gb300 import dflash
    n, V = tp.shape
    tok, acc = torch.full((n,), -7, dtype=torch.int32, device=DEV), torch.full((n,), -7, dtype=torch.int32, device=DEV)
    a = dflash.VerifyArgs(n_seq=n, k=0, vocab=V, dtype=dflash.F32, target_probs=tp.data_ptr(), target_seq_stride=V,
                          target_row_stride=V, u_token=ut.data_ptr(), tokens=tok.data_ptr(), n_accepted=acc.data_ptr())
    assert dflash.load_library().dflash_verify_tokens(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert bool((acc == 0).all())
    return tok.cpu().numpy()


def check_draws(tp, ut, tok):
    """Every token has weight, and u * total lies on its step but for the sums' error (2^-44, and 2^-39 of the 64-bit
    sums here)."""
    w = tp.double().cpu().numpy()
    c = np.cumsum(w, 1)
    i = np.arange(len(w))
    assert ((tok >= 0) & (tok < w.shape[1])).all(), tok[(tok < 0) | (tok >= w.shape[1])]
    th, eps = ut.double().cpu().numpy() * c[:, -1], 2.0 ** -38
    assert (w[i, tok] > 0).all()
    assert (c[i, tok] >= th * (1 - eps)).all() and (c[i, tok] - w[i, tok] <= th * (1 + eps)).all()


def test_verify_thresholds_next_to_the_border_of_a_run(T):
    """Rows whose halves weigh the same and u = 1/2: sums taken in different orders fall on both sides of the
    threshold, at the end of the entries that a warp, a CTA or a search step has."""
    g = torch.Generator().manual_seed(1)
    x = torch.exp(4 * torch.randn(2048, 4096, generator=g))
    half = torch.full((2048,), 0.5, device=DEV)
    for y in (x.flip(1), x, x[:, torch.randperm(4096, generator=g)]):
        tp = torch.cat([x, y], 1).to(DEV)
        check_draws(tp, half, drawn(T, tp, half))


def test_verify_thresholds_next_to_entries_without_weight(T):
    """The same with nothing but zeros between the halves: the runs there are never drawn from, nor is entry 0."""
    V = 16384
    half = torch.full((32,), 0.5, device=DEV)
    for m in (256, 700, 1536, 2048, 3333, 6000):
        for seed in range(12):
            g = torch.Generator().manual_seed(seed)
            x = torch.exp(4 * torch.randn(32, m, generator=g))
            tp = torch.zeros(32, V)
            tp[:, 1:m + 1], tp[:, V - m:] = x, x[:, torch.randperm(m, generator=g)]
            tp = tp.to(DEV)
            check_draws(tp, half, drawn(T, tp, half))


@pytest.mark.parametrize("dt", [F4, BF, HF])
def test_verify_accepts_tiny_probabilities_by_their_product(T, dt):
    """u q < p where u q has bits below the smallest float: equal probabilities are always accepted."""
    n, V = 400, 64
    g = torch.Generator().manual_seed(5)
    one = {F4: 2.0 ** -149, BF: 2.0 ** -133, HF: 2.0 ** -24}[dt]
    tp = torch.full((n, 2, V), 0.01, dtype=torch.float64)
    dp = torch.full((n, 1, V), 0.01, dtype=torch.float64)
    draft = torch.randint(0, V, (n, 1), generator=g).to(torch.int32)
    i = torch.arange(n)
    p, q = torch.randint(1, 5, (2, n), generator=g).double() * one
    q[::2] = p[::2]
    tp[i, 0, draft[:, 0].long()], dp[i, 0, draft[:, 0].long()] = p, q
    args = [draft, tp.to(dt), torch.rand(n, 1, generator=g), torch.rand(n, generator=g), dp.to(dt)]
    args[2][:20] = 1 - 2.0 ** -24
    tok, acc = T.verify_tokens(*(t.to(DEV) for t in args[:4]), draft_probs=args[4].to(DEV))
    wt, wa = R.verify(*args)
    assert bool((wa[::2] == 1).all())
    assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)
