"""The next step's tables on the GPU against a stack and a loop."""
import random

import numpy as np
import pytest
import torch

import _packed_ref as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def T():
    from speculative_decoding_block_ingest_gb300 import target
    return target


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def state(seed, n, page, longest, prev, spare, cols_extra=1):
    """A server in the middle of its work: lengths, rows of the last step, table (unused entries -7), stack, height."""
    r = random.Random(seed)
    rows = [r.randint(0, prev) for _ in range(n)]
    kv = [t + r.choice([0, r.randint(0, longest)]) for t in rows]
    held = [-(-x // page) for x in kv]
    cols = max(held + [1]) + cols_extra
    order = list(range(sum(held) + spare))
    r.shuffle(order)
    table = np.full((n, cols), -7, dtype=np.int32)
    for i, h in enumerate(held):
        table[i, :h] = order[:h]
        order = order[h:]
    free = np.full(sum(held) + spare, -9, dtype=np.int32)
    free[:spare] = order
    return kv, np.concatenate([[0], np.cumsum(rows)]).tolist(), table, free, spare


def run(T, kv, starts, table, free, n_free, page, rows, n_rows, prefix=0, accepted=None, keep=None, beside=False):
    t, f = i32(table), i32(free)
    pool = T.PagePool(f, i32([n_free]), t, i32(kv), i32(starts), page_size=page, prefix_len=prefix)
    slots = torch.full((n_rows,), -3, dtype=torch.int64, device=DEV)
    pos, seqs = (torch.full((n_rows,), -3, dtype=torch.int32, device=DEV) for _ in range(2))
    kw = dict(n_accepted=None if accepted is None else i32(accepted), keep=None if keep is None else i32(keep),
              slots=slots, positions=pos, sequences=seqs, out=pool.beside() if beside else None)
    out = T.next_step(pool, i32(rows), **kw)
    if beside:       # the lengths it started from are still there: the same again
        assert out is not pool and pool.kv_len.tolist() == kv and pool.row_start.tolist() == starts
        first = [x.clone() for x in (out.kv_len, out.row_start, out.n_free, t, f, slots)]
        T.next_step(pool, i32(rows), **kw)
        assert all(torch.equal(a, b) for a, b in zip(first, (out.kv_len, out.row_start, out.n_free, t, f, slots)))
    return pool, out, slots, pos, seqs


def check(T, st, page, rows, n_rows, prefix=0, accepted=None, keep=None, beside=False):
    kv, starts, table, free, n_free = st
    pool, out, slots, pos, seqs = run(T, kv, starts, table, free, n_free, page, rows, n_rows, prefix, accepted, keep, beside)
    wt, wf = table.copy(), free.copy()
    new, ws, top, wslots, wpos, wseqs = P.next_step(kv, starts, rows, wt, wf, n_free, page, n_rows, prefix, accepted, keep)
    n = ws[-1]
    assert out.kv_len.tolist() == new and out.row_start.tolist() == ws and out.n_free.tolist() == [top]
    assert np.array_equal(out.block_table.cpu().numpy(), wt) and np.array_equal(out.free.cpu().numpy(), wf)
    assert slots[:n].tolist() == wslots and pos[:n].tolist() == wpos and seqs[:n].tolist() == wseqs
    assert bool((slots[n:] == -3).all()) and bool((pos[n:] == -3).all()) and bool((seqs[n:] == -3).all())
    return new, ws, wt, wf, top


CASES = [
    # sequences, page, longest, last rows, spare pages, rows asked for, room for rows, verified, over
    (1, 16, 40, 1, 4, 1, 1, False, 0.0),
    (1, 256, 9, 9, 0, 1, 5, True, 0.0),
    (8, 64, 700, 16, 40, 16, 128, True, 0.1),
    (33, 16, 200, 5, 100, 33, 2000, True, 0.3),
    (256, 32, 300, 17, 300, 17, 4352, True, 0.0),
    (257, 16, 90, 3, 5, 40, 9000, True, 0.2),          # pages run out
    (1000, 128, 500, 16, 900, 16, 7000, True, 0.1),    # room for rows runs out
    (1024, 16, 300, 9, 4000, 40, 9000, True, 0.1),     # sizes at which the CTAs change
    (1025, 32, 300, 9, 900, 40, 30000, True, 0.1),
    (2049, 16, 90, 5, 6000, 20, 50000, True, 0.2),
    (4096, 16, 60, 2, 3000, 1, 4096, False, 0.05),
    (4096, 16, 100, 17, 500, 90, 300000, True, 0.4),
    (3, 16, 30000, 0, 3000, 9000, 30000, False, 0.3),
    (5, 16, 0, 0, 10, 0, 4, False, 0.0),               # nothing there, nothing asked for
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
@pytest.mark.parametrize("beside", [False, True], ids=["inplace", "beside"])
def test_next_step(T, case, beside):
    n, page, longest, prev, spare, ask, n_rows, verified, over = case
    for seed in range(3):
        st = state(seed, n, page, longest, prev, spare, cols_extra=0 if seed == 1 else 2)
        r = random.Random(100 + seed)
        rows = [r.randint(0, ask) for _ in range(n)]
        acc = [r.randint(-1, max(t - 1, 0)) for t in np.diff(st[1])] if verified else None
        keep = [0 if r.random() < over else r.choice([-1, -5, r.randint(0, longest + 1)]) for _ in range(n)] if over else None
        check(T, st, page, rows, n_rows, prefix=seed * 17, accepted=acc, keep=keep, beside=beside)


def test_many_steps_in_place(T):
    """Steps one after the other, each from where the last one left off; at the end all pages are back."""
    r = random.Random(5)
    n, page, cols = 40, 16, 24
    free = np.arange(300, dtype=np.int32)[::-1].copy()
    st = ([0] * n, [0] * (n + 1), np.full((n, cols), -7, dtype=np.int32), free, 300)
    pool = T.PagePool.empty(300, page, n, cols, DEV, prefix_len=3)
    pool.block_table.fill_(-7)
    assert pool.free.tolist() == free.tolist()
    for turn in range(30):
        rows = [r.choice([0, 1, 16, 16, r.randint(0, 120)]) for _ in range(n)]
        acc = [r.randint(0, 15) for _ in range(n)]
        keep = [0 if r.random() < 0.1 else -1 for _ in range(n)]
        if turn == 29:
            rows, keep = [0] * n, [0] * n
        wt, wf = st[2].copy(), st[3].copy()
        new, ws, top, slots, _, _ = P.next_step(st[0], st[1], rows, wt, wf, st[4], page, 900, 3, acc, keep)
        got = torch.zeros(900, dtype=torch.int64, device=DEV)
        assert T.next_step(pool, i32(rows), n_accepted=i32(acc), keep=i32(keep), slots=got) is pool
        assert pool.kv_len.tolist() == new and pool.row_start.tolist() == ws and pool.n_free.tolist() == [top]
        assert np.array_equal(pool.block_table.cpu().numpy(), wt) and np.array_equal(pool.free.cpu().numpy(), wf)
        assert got[:ws[-1]].tolist() == slots and len(set(slots)) == len(slots)
        live = [p for i, x in enumerate(new) for p in wt[i, :-(-x // page)].tolist()] + wf[:top].tolist()
        assert sorted(live) == list(range(300))        # every page is somebody's or free, once
        st = (new, ws, wt, wf, top)
    assert st[4] == 300 and int(pool.ticket) == 0


def test_giving_back_restores_the_stack(T):
    st = state(7, 50, 16, 200, 0, 200)
    kv, starts, table, free, n_free = st
    new, ws, wt, wf, top = check(T, st, 16, [33] * 50, 2000)
    assert top < n_free
    _, _, _, wf2, top2 = check(T, (new, ws, wt, wf, top), 16, [0] * 50, 0, keep=kv)
    assert top2 == n_free and np.array_equal(wf2[:n_free], free[:n_free])


def test_lengths_and_heights_out_of_range(T):
    """Garbage in the arrays stays inside the buffers (guards around table and stack), and ends."""
    n, page, cols, places = 300, 16, 5, 100
    big = (1 << 31) - 1
    for seed in range(4):
        r = random.Random(seed)
        wild = lambda: r.choice([0, 1, 70, 80, 81, big, big - 100, -1, -big])
        mem = torch.full((n + 2, cols + 4), -11, dtype=torch.int32, device=DEV)
        mem[1:-1, 2:-2] = i32(np.arange(n * cols).reshape(n, cols))
        stack = torch.full((places + 20,), -11, dtype=torch.int32, device=DEV)
        stack[10:-10] = 3
        starts = [wild() for _ in range(n + 1)]
        pool = T.PagePool(stack[10:-10], i32([wild()]), mem[1:-1, 2:-2], i32([wild() for _ in range(n)]), i32(starts),
                          page_size=page, prefix_len=big - 2000)
        slots = torch.full((1000 + 20,), -11, dtype=torch.int64, device=DEV)
        T.next_step(pool, i32([wild() for _ in range(n)]), n_accepted=i32([wild() for _ in range(n)]),
                    keep=i32([wild() for _ in range(n)]), slots=slots[10:-10])
        torch.cuda.synchronize()
        assert bool((slots[:10] == -11).all()) and bool((slots[-10:] == -11).all())
        assert bool((stack[:10] == -11).all()) and bool((stack[-10:] == -11).all())
        assert bool((mem[0] == -11).all()) and bool((mem[-1] == -11).all())
        assert bool((mem[:, :2] == -11).all()) and bool((mem[:, -2:] == -11).all())
        assert 0 <= int(pool.n_free) <= places
        assert 0 <= int(pool.kv_len.min()) and int(pool.kv_len.max()) <= cols * page
        d = pool.row_start.diff()
        assert int(pool.row_start[0]) == 0 and bool((d >= 0).all()) and int(pool.row_start[-1]) <= 1000


def test_without_row_tensors_on_a_stream_and_in_a_graph(T):
    st = state(3, 20, 16, 100, 4, 60)
    kv, starts, table, free, n_free = st
    wt, wf = table.copy(), free.copy()
    new, ws, top, _, _, _ = P.next_step(kv, starts, [7] * 20, wt, wf, n_free, 16, 500)
    pool = T.PagePool(i32(free), i32([n_free]), i32(table), i32(kv), i32(starts), page_size=16)
    out, rows, s = pool.beside(), i32([7] * 20), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    T.next_step(pool, rows, n_rows=500, out=out, stream=s)
    s.synchronize()
    assert out.kv_len.tolist() == new and out.row_start.tolist() == ws and out.n_free.tolist() == [top]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        T.next_step(pool, rows, n_rows=500)
    # in place: every replay is a step of its own
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert pool.kv_len.tolist() == new and pool.row_start.tolist() == ws and pool.n_free.tolist() == [top]
        assert np.array_equal(pool.block_table.cpu().numpy(), wt)
        new, ws, top, _, _, _ = P.next_step(new, ws, [7] * 20, wt, wf, top, 16, 500)
