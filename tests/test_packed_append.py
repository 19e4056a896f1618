"""Appending to a 4-bit cache on the GPU: every code and scale against the
definition in 64 bits, and RoPE in interleaved pairs in both kinds of cache."""
import numpy as np
import pytest
import torch

import _packed_ref as P
import _target_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
Y4 = (32.0, 8192, 32.0, 1.0)


@pytest.fixture(scope="module")
def T():
    from speculative_decoding_block_ingest_gb300 import target
    return target


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def pools(n_pages, page, hkv, d, *, hnd=False, pad=0, seed=0):
    """Random bytes of the four pools as [n_pages, page, hkv, bytes] views: `pad` unused bytes behind a head's codes, and
    behind its scales of a page."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        shape = (n_pages, hkv, page, d // 2 + pad) if hnd else (n_pages, page, hkv, d // 2 + pad)
        x = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).to(DEV)[..., :d // 2]
        out.append(x.transpose(1, 2) if hnd else x)
    for _ in range(2):
        n = page * d // 16
        x = torch.randint(0, 256, (n_pages, hkv, n + pad), generator=g, dtype=torch.uint8).to(DEV)[..., :n]
        out.append(x.unflatten(2, (page, d // 16)).transpose(1, 2))
    return out


CASES = [
    # rows, kv, hq, hkv, d, rot, page, in, out, norm, yarn, interleaved, hnd, prefix, units
    ([1], [1], 1, 1, 64, 64, 16, BF, BF, True, False, False, False, 0, (1.0, 1.0)),
    ([1], [1000], 32, 4, 128, 128, 64, BF, BF, True, False, True, True, 0, (1.0, 1.0)),
    ([5, 0, 17, 1], [5, 40, 100, 1], 32, 8, 128, 128, 16, F4, BF, True, True, False, True, 16383, (0.25, 4.0)),
    ([3, 2], [700, 2], 6, 2, 64, 32, 128, HF, HF, False, False, True, False, 70, (1.0, 2.0 ** -12)),
    ([40, 33], [40, 200], 5, 5, 128, 64, 32, F4, HF, True, True, True, True, 1, (1.0, 1.0)),
    ([9], [9], 3, 1, 128, 0, 256, BF, BF, True, False, False, False, 0, (1.0, 1.0)),
    ([2] * 300, [7] * 300, 2, 1, 64, 16, 16, BF, BF, True, False, False, False, 5, (1.0, 1.0)),   # blocks across lanes
    ([7, 2], [7, 30], 4, 2, 128, 48, 16, HF, HF, True, False, True, False, 3, (1.0, 1.0)),
    ([7, 2], [7, 30], 4, 2, 128, 112, 16, F4, BF, False, False, False, True, 3, (1.0, 1.0)),
    ([1300, 1], [1300, 2000], 8, 2, 128, 128, 64, BF, BF, True, False, False, True, 0, (1.0, 1.0)),   # a warp a row
    ([900, 800], [900, 900], 4, 4, 64, 64, 16, F4, HF, False, True, True, False, 9, (2.0, 0.5)),
    # many rows, queries, keys and values in one pass of a warp
    ([1300, 3], [1300, 9], 1, 1, 128, 128, 16, HF, HF, True, True, False, True, 0, (1.0, 1.0)),
    ([3, 1500], [40, 1500], 3, 3, 64, 32, 32, F4, BF, False, False, True, False, 2, (0.5, 1.0)),
    ([700] * 3, [700, 900, 701], 2, 5, 64, 16, 64, BF, BF, True, False, False, True, 1, (1.0, 2.0 ** 20)),
]


def inputs(case, seed=2):
    rows, kv, hq, hkv, d, rot, page, ti, to, norm, yarn, inter, hnd, prefix, units = case
    n = sum(rows)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, (hq + 2 * hkv) * d, generator=g)
    x[:, -hkv * d:] *= units[1]
    q, k, v = (t.unflatten(1, (-1, d)) for t in x.to(ti).to(DEV).split([hq * d, hkv * d, hkv * d], 1))
    qg, kg = ((1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)) if norm else (None, None)
    return q, k, v, qg, kg


def stored(pool, dst):
    return torch.stack([pool[a, b] for a, b in dst]).cpu().numpy()


@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_append(T, case):
    rows, kv, hq, hkv, d, rot, page, ti, to, norm, yarn, inter, hnd, prefix, units = case
    starts, kv, table, pre, n_pages = R.make_step(rows, kv, page, prefix=prefix, seed=1)
    mem = pools(n_pages, page, hkv, d, hnd=hnd, pad=16)
    before = [m.clone() for m in mem]
    q, k, v, qg, kg = inputs(case)
    theta, y = (1e6, Y4) if yarn else (1e4, None)
    rope = T.Rope(rot, theta, *(y or ()), interleaved=inter) if rot else None
    inv, ms = R.rope_freqs(rot, theta, y) if rot else (np.zeros(0), 1.0)
    cache = T.PagedCache4(*mem, dtype=to, k_unit=units[0], v_unit=units[1])
    step = T.Step(i32(starts), i32(kv), table.to(DEV), pre.to(DEV), prefix)
    n = starts[-1]
    kval, vval = (torch.empty(n, hkv, d, dtype=to, device=DEV) for _ in range(2))
    qo = T.append(cache, step, q, k, v, rope=rope, q_gain=qg, k_gain=kg, eps=1e-6, k_values=kval, v_values=vval)
    torch.cuda.synchronize()
    pos, dst = [], []
    for i, t in enumerate(rows):
        for own in range(kv[i] - t, kv[i]):
            pos.append(prefix + own)
            dst.append((int(table[i, own // page]), own % page))
    want, size = P.rotate(q, qg, 1e-6, pos, inv, ms, inter)
    # one rounding to the type; norm, angle (2^-25 of a turn) and rotation in f32
    tol = R.EPS[to] * np.abs(want) + 1e-6 * size + (2.0 ** -25 if to == HF else 0)
    assert np.all(np.abs(qo.double().cpu().numpy() - want) <= tol)
    ky, _ = P.rotate(k, kg, 1e-6, pos, inv, ms, inter)
    for y, unit, codes, scales, val in ((ky, units[0], mem[0], mem[2], kval),
                                        (v.double().cpu().numpy(), units[1], mem[1], mem[3], vval)):
        c, s, x = P.pack(y, unit)
        assert np.array_equal(stored(scales, dst), s)
        assert np.array_equal(stored(codes, dst), c)
        assert torch.equal(val.cpu(), torch.from_numpy(x).to(to))     # 6 bits: exact, or f16's range
    # nothing else of the pools changed
    for m, b in zip(mem, before):
        for p, r in dst:
            b[p, r] = m[p, r]
        assert torch.equal(m, b)


def test_interleaved_pairs_in_a_16_bit_cache(T):
    """The same call into a cache of rows: pairs 2j, 2j + 1."""
    for rows, hq, hkv, d, rot, ti, to in (([1], 4, 2, 128, 128, BF, BF), ([3, 4], 5, 1, 64, 32, F4, HF),
                                          ([1500], 2, 1, 128, 48, HF, HF)):
        starts, kv, table, pre, n_pages = R.make_step(rows, [t + 9 for t in rows], 16, seed=3)
        g = torch.Generator().manual_seed(4)
        q, k, v = (torch.randn(starts[-1], h, d, generator=g).to(ti).to(DEV) for h in (hq, hkv, hkv))
        gain = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
        kc, vc = (torch.zeros(n_pages, 16, hkv, d, dtype=to, device=DEV) for _ in range(2))
        step = T.Step(i32(starts), i32(kv), table.to(DEV))
        qo = T.append(T.PagedCache(kc, vc), step, q, k, v, rope=T.Rope(rot, 1e4, interleaved=True), q_gain=gain,
                      k_gain=gain)
        pos = [own for i, t in enumerate(rows) for own in range(kv[i] - t, kv[i])]
        dst = [(int(table[i, own // 16]), own % 16) for i, t in enumerate(rows) for own in range(kv[i] - t, kv[i])]
        inv, ms = R.rope_freqs(rot, 1e4)
        for got, x in ((qo.double().cpu().numpy(), q), (torch.stack([kc[a, b] for a, b in dst]).double().cpu().numpy(), k)):
            want, size = P.rotate(x, gain, 1e-6, pos, inv, ms, True)
            assert np.all(np.abs(got - want) <= R.EPS[to] * np.abs(want) + 1e-6 * size + (2.0 ** -25 if to == HF else 0))
        assert torch.equal(torch.stack([vc[a, b] for a, b in dst]), v.to(to))


def test_given_frequencies_and_far_positions(T):
    """Frequencies and a factor of the caller's; explicit positions up to 2^20."""
    d, pos = 128, [0, 1, 131071, 1 << 20, 5]
    mem = pools(2, 16, 1, d)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(5, h, d, generator=g).to(HF).to(DEV) for h in (2, 1, 1))
    inv = np.exp(-np.linspace(0.0, 9.0, 64))
    step = T.Step(i32([0, 5]), i32([5]), i32([[1]]))
    T.append(T.PagedCache4(*mem, dtype=HF), step, q, k, v, positions=i32(pos),
             rope=T.Rope(d, inv_freq=inv.tolist(), mscale=1.25))
    y, _ = R.head_rows(k, None, 0, pos, inv, 1.25)
    c, s, _ = P.pack(y)
    assert np.array_equal(mem[0][1, :5].cpu().numpy(), c) and np.array_equal(mem[2][1, :5].cpu().numpy(), s)


def rows_as_they_are(T, x, dt, unit=1.0):
    """Codes, scales and values of given value rows [n, 128]."""
    n = x.shape[0]
    mem = pools(-(-n // 16), 16, 1, 128)
    val = torch.empty(n, 1, 128, dtype=dt if dt != F4 else BF, device=DEV)
    step = T.Step(i32([0, n]), i32([n]), torch.arange(-(-n // 16), dtype=torch.int32)[None].to(DEV))
    x = x.to(dt).to(DEV)[:, None]
    T.append(T.PagedCache4(*mem, dtype=val.dtype, v_unit=unit), step, None, x, x, v_values=val)
    codes, scales = (m.flatten(0, 1)[:n, 0].cpu().numpy() for m in (mem[1], mem[3]))
    same = [torch.equal(a.flatten(0, 1)[:n], b.flatten(0, 1)[:n]) for a, b in ((mem[0], mem[1]), (mem[2], mem[3]))]
    if unit == 1.0:       # keys without norm and rotation are rounded like values
        assert all(same)
    return codes, scales, val[:, 0]


@pytest.mark.parametrize("dt", [BF, HF, F4], ids=["bf16", "f16", "f32"])
def test_ties_and_neighbours(T, dt):
    """Elements on the border between two codes, one step of their type to either side, and scales on theirs."""
    eps = {BF: 2.0 ** -7, HF: 2.0 ** -10, F4: 2.0 ** -23}[dt]
    rows = []
    for s in (0.5, 0.5625, 0.8125, 0.9375, 7.0, 2.0 ** -6):
        for step in (0.0, eps, -eps):
            mid = (P.E2M1[1:] + P.E2M1[:-1]) / 2
            m, e = np.frexp(s * mid)
            x = np.ldexp(m + step * 0.5, e)                       # the neighbour of a value with few bits
            row = np.concatenate([[6 * s], x, -x, [0.0]])
            rows.append(np.concatenate([row] * 8))
    for m in range(8, 16):                                        # 6 times a scale's border
        for step in (0.0, eps, -eps):
            top = 6 * (m + 0.5) / 8
            fr, e = np.frexp(top)
            row = np.concatenate([[np.ldexp(fr + step * 0.5, e)], np.linspace(-top, top, 15) * 0.9])
            rows.append(np.concatenate([row] * 8))
    x = torch.from_numpy(np.array(rows)).to(dt)
    codes, scales, _ = rows_as_they_are(T, x, dt)
    c, s, _ = P.pack(x.double().numpy())
    assert np.array_equal(scales, s)
    assert np.array_equal(codes, c)


@pytest.mark.parametrize("dt", [BF, HF, F4], ids=["bf16", "f16", "f32"])
def test_zeros_small_large_and_not_finite_values(T, dt):
    g = torch.Generator().manual_seed(9)
    x = torch.randn(20, 128, generator=g)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= 1e-5                       # below half of the smallest scale: zeros with their signs
    x[3] *= 2.0 ** -9                  # scales below their normal range
    x[4, 3] = 60000.0                  # beyond 6 * 448: the scale stays at its largest
    x[5] *= 3000.0
    x[6, 17] = float("nan")
    x[7, 40] = float("inf")
    x[8, 41] = -float("inf")
    x[9, 63:65] = float("nan")
    if dt != HF:
        x[10] = 3e38 * torch.sign(x[10])
        x[11] *= 1e-38
    x = x.to(dt)
    codes, scales, val = rows_as_they_are(T, x, dt)
    c, s, y = P.pack(x.double().numpy())
    assert np.array_equal(scales, s) and np.array_equal(codes, c)
    got = val.double().cpu().numpy()
    want = torch.from_numpy(y).to(val.dtype).double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    # units move the range
    for unit in (2.0 ** -20, 2.0 ** 12):
        codes, scales, _ = rows_as_they_are(T, x, dt, unit)
        c, s, _ = P.pack(x.double().numpy(), unit)
        assert np.array_equal(scales, s) and np.array_equal(codes, c)


def test_normed_keys_next_to_borders(T):
    """Keys whose norm and rotation land within f32's error of a border: many rows, all codes those of 64 bits."""
    n, d = 20000, 128
    g = torch.Generator().manual_seed(12)
    k = torch.randint(-3, 4, (n, 1, d), generator=g).to(BF).to(DEV)     # few values: quotients repeat, some on borders
    mem = pools(-(-n // 64), 64, 1, d)
    step = T.Step(i32([0, n]), i32([n]), torch.arange(-(-n // 64), dtype=torch.int32)[None].to(DEV))
    gain = torch.ones(d, device=DEV)
    T.append(T.PagedCache4(*mem), step, None, k, k, k_gain=gain, rope=T.Rope(64, 1e4))
    inv, ms = R.rope_freqs(64, 1e4)
    y, _ = R.head_rows(k, gain, 1e-6, range(n), inv, ms)
    c, s, _ = P.pack(y)
    assert np.array_equal(mem[2].flatten(0, 1)[:n].cpu().numpy(), s)
    assert np.array_equal(mem[0].flatten(0, 1)[:n].cpu().numpy(), c)


def test_codes_do_not_depend_on_the_rows_beside_them(T):
    """A row alone (eight warps) and among two thousand (one warp) has the same bits."""
    case = ([2000], [2000], 2, 2, 128, 128, 64, BF, BF, True, False, False, True, 0, (1.0, 1.0))
    q, k, v, qg, kg = inputs(case)
    rope = T.Rope(128, 1e6)
    a, b = pools(32, 64, 2, 128, hnd=True, seed=5), pools(32, 64, 2, 128, hnd=True, seed=6)
    table = torch.arange(32, dtype=torch.int32)[None].to(DEV)
    T.append(T.PagedCache4(*a), T.Step(i32([0, 2000]), i32([2000]), table), q, k, v, rope=rope, q_gain=qg, k_gain=kg)
    for r0 in range(0, 2000, 37):
        r1 = min(r0 + 37, 2000)
        T.append(T.PagedCache4(*b), T.Step(i32([0, r1 - r0]), i32([r1]), table), None, k[r0:r1], v[r0:r1], rope=rope,
                 k_gain=kg)
    for x, y in zip(a, b):
        assert torch.equal(x.transpose(1, 2).flatten(2, 3)[:31], y.transpose(1, 2).flatten(2, 3)[:31])


def test_leaves_what_no_row_names(T):
    """Rows behind the last sequence, before key 0, past the block table and on a page that does not exist."""
    d = 64
    mem = pools(3, 16, 1, d)
    before = [m.clone() for m in mem]
    g = torch.Generator().manual_seed(4)
    n = 12
    q, k, v = (torch.randn(n, 1, d, generator=g).to(BF).to(DEV) for _ in range(3))
    # seq 0: 3 rows, 2 keys (first row has none); seq 1: 4 rows ending at key 34 of a 2-page table; seq 2: page 9 of 3
    step = T.Step(i32([0, 3, 7, 9]), i32([2, 34, 2]), i32([[0, -7], [1, 2], [9, -7]]))
    qo, kv, vv = (torch.full((n, 1, d), 7.0, dtype=BF, device=DEV) for _ in range(3))
    T.append(T.PagedCache4(*mem), step, q, k, v, q_out=qo, k_values=kv, v_values=vv)
    torch.cuda.synchronize()
    written = {1: (0, 0), 2: (0, 1), 3: (2, 14), 4: (2, 15)}
    for src, (page, at) in written.items():
        for x, m, s, val in ((k, 0, 2, kv), (v, 1, 3, vv)):
            c, sc, y = P.pack(x[src].double().cpu().numpy())
            assert np.array_equal(mem[m][page, at].cpu().numpy(), c) and np.array_equal(mem[s][page, at].cpu().numpy(), sc)
            assert torch.equal(val[src].cpu(), torch.from_numpy(y).to(BF))
        for b, m in zip(before, mem):
            b[page, at] = m[page, at]
    assert all(torch.equal(a, b) for a, b in zip(mem, before))
    rest = [i for i in range(n) if i not in written]
    assert bool((kv[rest] == 7).all()) and bool((vv[rest] == 7).all())
    assert torch.equal(qo[:9], q[:9]) and bool((qo[9:] == 7).all())


def test_offsets_past_32_bits(T):
    """A pool of more than 2^32 bytes of codes."""
    page, hkv, d = 256, 8, 128
    n_pages = (1 << 32) // (page * hkv * 64) + 40
    mem = [torch.zeros(n_pages, page, hkv, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    mem += [torch.zeros(n_pages, hkv, page, 8, dtype=torch.uint8, device=DEV).transpose(1, 2) for _ in range(2)]
    g = torch.Generator().manual_seed(6)
    k = torch.randn(3, hkv, d, generator=g).to(BF).to(DEV)
    T.append(T.PagedCache4(*mem), T.Step(i32([0, 3]), i32([3]), i32([[n_pages - 1]])), None, k, k)
    c, s, _ = P.pack(k.double().cpu().numpy())
    assert np.array_equal(mem[0][-1, :3].cpu().numpy(), c) and np.array_equal(mem[3][-1, :3].cpu().numpy(), s)
    assert not mem[0][:-1].any() and not mem[1][:, 3:].any()


def test_queries_in_place_another_stream_and_a_graph(T):
    case = ([3, 2], [60, 40], 4, 2, 128, 128, 16, BF, BF, True, False, True, False, 0, (1.0, 1.0))
    starts, kv, table, _, n_pages = R.make_step(case[0], case[1], 16, seed=7)
    q, k, v, qg, kg = inputs(case)
    kw = dict(rope=T.Rope(128, 1e6, interleaved=True), q_gain=qg, k_gain=kg)
    a, b = pools(n_pages, 16, 2, 128, seed=8), pools(n_pages, 16, 2, 128, seed=8)
    kv_len = i32(kv)
    step = T.Step(i32(starts), kv_len, table.to(DEV))
    q1 = T.append(T.PagedCache4(*a), step, q, k, v, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qc = q.contiguous()
    cache = T.PagedCache4(*b)
    assert T.append(cache, step, qc, k, v, q_out=qc, stream=s, **kw) is qc
    s.synchronize()
    assert torch.equal(q1, qc) and all(torch.equal(x, y) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        T.append(cache, step, None, k, v, **kw)
    kv_len.sub_(7)              # the captured call reads the lengths of the replay
    graph.replay()
    T.append(T.PagedCache4(*a), step, None, k, v, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
