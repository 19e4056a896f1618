"""The pieces the attention of a step is cut into (host logic only): every key
block of every item exactly once, equal shares, and the CTA ranges the merge
relies on."""
import ctypes
import random

import pytest

from speculative_decoding_block_ingest_gb300 import build, dflash

KEYS = 128


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(dflash.LIB_PATH):
        build.build()
    return dflash.load_library()


def i32(v):
    return (ctypes.c_int32 * max(1, len(v)))(*v)


def plan(rows, kv, *, hq, hkv, prefix=0, page=64, causal=True, n_cta=152, cols=None, n_rows=None, room=1 << 20):
    starts = [0]
    for t in rows:
        starts.append(starts[-1] + t)
    rs, kl, dummy = i32(starts), i32(kv), i32([0])
    addr = ctypes.addressof
    cache = dflash.PagedCacheDesc(dtype=dflash.BF16, page_size=page, n_kv_heads=hkv, head_dim=128)
    cols = -(-max(kv) // page) if cols is None else cols
    step = dflash.StepDesc(n_seq=len(rows), n_rows=starts[-1] if n_rows is None else n_rows, row_start=addr(rs),
                           kv_len=addr(kl), block_table=addr(dummy), table_cols=cols, table_stride=cols,
                           prefix_len=prefix, prefix_pages=addr(dummy))
    n = ctypes.c_int32(0)
    out = (dflash.StepPiece * room)()
    rc = dflash.load_library().dflash_step_attention_plan(ctypes.byref(cache), ctypes.byref(step), hq, int(causal),
                                                          n_cta, ctypes.byref(n), out, room)
    assert rc == 0, dflash.load_library().dflash_last_error()
    return [{f: getattr(out[i], f) for f, _ in dflash.StepPiece._fields_} for i in range(n.value)]


def items(rows, kv, *, hq, hkv, prefix=0, page=64, causal=True, cols=None):
    """{(segment, seq, kv head, first row): (tokens, blocks)} from the definition."""
    pair = 2 * (128 // (hq // hkv))
    room = 10 ** 9 if cols is None else cols * page
    want, total = {}, sum(rows)       # in the pieces' order
    if prefix:
        for h in range(hkv):
            for r in range(0, total, pair):
                want[(0, -1, h, r)] = (min(pair, total - r), -(-prefix // KEYS))
    start = 0
    for i, (t, n) in enumerate(zip(rows, kv)):
        for h in range(hkv):
            for r in range(0, t, pair):
                seen = n - t + min(r + pair, t) if causal else n
                want[(1, i, h, start + r)] = (min(pair, t - r), -(-min(max(seen, 0), room) // KEYS))
        start += t
    return want


def ends(rows):
    return 6 + min(rows, 128) // 16


def check(rows, kv, n_cta=152, **kw):
    pieces = plan(rows, kv, n_cta=n_cta, **kw)
    want = items(rows, kv, **kw)
    G = kw["hq"] // kw["hkv"]
    start, pos, weight = {}, 0, {}     # an item's blocks, then its ends
    for key, (tokens, blocks) in want.items():           # prefix first, then by sequence, head and rows
        start[key] = pos
        weight[key] = 4 if tokens > 128 // G else 3
        pos += ends(tokens * G) + weight[key] * blocks
    C = min(n_cta, max(pos // 6, 1)) if pos else 0
    q, more = divmod(pos, C) if C else (0, 0)
    share = [(c * q + min(c, more), (c + 1) * q + min(c + 1, more)) for c in range(C)]
    got, ctas = {}, {}
    for p in pieces:
        key = (p["segment"], p["seq"], p["kv_head"], p["row0"])
        tokens, blocks = want[key]
        assert p["n_tokens"] == tokens and 0 <= p["block0"] <= p["block1"] <= blocks
        a, b = share[p["cta"]]
        assert p["first"] == (a <= start[key] < b)
        assert [i for i in range(blocks) if a <= start[key] + weight[key] * i < b] \
            == list(range(p["block0"], p["block1"]))      # the blocks that start in the CTA's share
        assert p["block0"] < p["block1"] or blocks == 0
        got.setdefault(key, []).append((p["block0"], p["block1"], p["first"]))
        ctas.setdefault(key, []).append((p["cta"], p["first"], p["last_cta"]))
    assert set(got) == set(want)
    for key, parts in got.items():
        at = 0
        for i, (b0, b1, first) in enumerate(parts):      # pieces come in CTA order
            assert first == (i == 0) and b0 == at
            at = b1
        assert at == want[key][1]
        c = [x for x, _, _ in ctas[key]]
        assert c == list(range(c[0], c[0] + len(c)))     # one CTA after the other
        assert ctas[key][0][2] == c[-1] and all(x[2] == -1 for x in ctas[key][1:])
        assert len(parts) == 1 or want[key][1] > 1       # one block: one piece
    # a CTA continues at most one item (its first)
    assert {p["cta"] for p in pieces} <= set(range(C))
    for c in range(C):
        mine = [p for p in pieces if p["cta"] == c]
        assert all(p["first"] for p in mine[1:])


@pytest.mark.parametrize("rows,kv,kw", [
    ([1], [1], dict(hq=4, hkv=1)),
    ([1], [777], dict(hq=32, hkv=4)),
    ([16], [131016], dict(hq=32, hkv=8)),
    ([1] * 64, list(range(1, 6401, 100)), dict(hq=32, hkv=4, prefix=4096)),
    ([16] * 32, [1024] * 32, dict(hq=32, hkv=4, prefix=16384)),
    ([0, 5, 0, 17, 1, 0], [0, 5, 300, 2000, 1, 0], dict(hq=12, hkv=4, prefix=129, page=16)),
    ([3, 40], [2, 10], dict(hq=8, hkv=1)),                       # rows before any key
    ([4, 4], [0, 0], dict(hq=8, hkv=8, cols=0)),                 # no keys at all
    ([1000, 1, 513], [1000, 5000, 800], dict(hq=6, hkv=2)),      # long prompts: many tiles
    ([1000, 1], [1500, 700], dict(hq=5, hkv=1, causal=False, prefix=1)),
    ([7, 9], [500, 400], dict(hq=64, hkv=1, cols=5, page=64)),   # lengths past the block table
])
def test_every_block_once_in_equal_shares(rows, kv, kw):
    for n_cta in (1, 2, 7, 152):
        check(rows, kv, n_cta=n_cta, **kw)


def test_random_steps():
    r = random.Random(5)
    for _ in range(60):
        hkv = r.choice([1, 2, 3, 4, 8])
        n = r.randint(1, 40)
        rows = [r.choice([0, 1, 1, r.randint(1, 20), r.randint(1, 300)]) for _ in range(n)]
        kv = [t + r.choice([0, r.randint(0, 100), r.randint(0, 5000)]) for t in rows]
        check(rows, kv, n_cta=r.choice([1, 5, 148, 152]), hq=hkv * r.randint(1, 64), hkv=hkv,
              prefix=r.choice([0, 0, 1, 128, r.randint(1, 3000)]), causal=r.random() < 0.7)


def test_no_rows_no_pieces():
    assert plan([0, 0], [10, 0], hq=4, hkv=1, prefix=100) == []


def test_refusals():
    lib = dflash.load_library()
    n = ctypes.c_int32(0)
    cache = dflash.PagedCacheDesc(dtype=dflash.BF16, page_size=64, n_kv_heads=2, head_dim=128)
    rs, kl = i32([0, 1]), i32([1000])
    step = dflash.StepDesc(n_seq=1, n_rows=1, row_start=ctypes.addressof(rs), kv_len=ctypes.addressof(kl),
                           block_table=ctypes.addressof(rs), table_cols=16, table_stride=16)
    out = (dflash.StepPiece * 1)()

    def call(c=cache, s=step, heads=4, cap=1, n_cta=8):
        return lib.dflash_step_attention_plan(ctypes.byref(c), ctypes.byref(s), heads, 1, n_cta, ctypes.byref(n), out,
                                              cap)

    assert call() == dflash.ERR_CAPACITY and n.value > 1
    assert call(heads=3) == dflash.ERR_INVALID_ARG
    assert call(heads=2 * 65) == dflash.ERR_UNSUPPORTED
    assert call(n_cta=0) == dflash.ERR_INVALID_ARG
    # 2^24 rows over 2^29 keys: more units of work than one call takes
    big = dflash.StepDesc(n_seq=1, n_rows=1 << 24, row_start=ctypes.addressof(rs), kv_len=ctypes.addressof(kl),
                          block_table=ctypes.addressof(rs), table_cols=1 << 23, table_stride=1 << 23)
    assert call(s=big) == dflash.ERR_UNSUPPORTED
    assert lib.dflash_last_error().decode() != ""
