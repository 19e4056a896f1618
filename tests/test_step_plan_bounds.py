"""What the attention's plan does with row starts that decrease and with key counts next to 2^31 (host logic only:
the same code plans on the device)."""
import ctypes

import pytest

from speculative_decoding_block_ingest_gb300 import build, dflash


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(dflash.LIB_PATH):
        build.build()
    return dflash.load_library()


def plan(lib, starts, kv, *, n_rows, hq, hkv, cols, page=64, prefix=0, causal=False, n_cta=148, room=1 << 20):
    rs, kl = ((ctypes.c_int32 * len(x))(*x) for x in (starts, kv))
    at = ctypes.addressof(rs)
    cache = dflash.PagedCacheDesc(dtype=dflash.BF16, page_size=page, n_kv_heads=hkv, head_dim=128)
    step = dflash.StepDesc(n_seq=len(kv), n_rows=n_rows, row_start=at, kv_len=ctypes.addressof(kl), block_table=at,
                           table_cols=cols, table_stride=cols, prefix_len=prefix, prefix_pages=at)
    n, out = ctypes.c_int32(0), (dflash.StepPiece * room)()
    rc = lib.dflash_step_attention_plan(ctypes.byref(cache), ctypes.byref(step), hq, int(causal), n_cta,
                                        ctypes.byref(n), out, room)
    return rc, [out[i] for i in range(min(n.value, room))]


@pytest.mark.parametrize("starts,kv,kw", [
    # the units of all sequences pass 2^31 although no sequence's do
    ([0, 8192] * 2048 + [0], [261760] * 4096, dict(n_rows=8192, hq=8, hkv=8, cols=4090)),
    ([0, 1 << 20] * 2048 + [0], [1024] * 4096, dict(n_rows=1 << 20, hq=8, hkv=8, cols=16, prefix=100)),
    ([0, 8, 3], [5, 5], dict(n_rows=8, hq=4, hkv=2, cols=1, prefix=20)),
    ([8, 0, 8], [50, 50], dict(n_rows=8, hq=4, hkv=2, cols=1)),
    ([0, 4, 2, 8], [50, 50, 50], dict(n_rows=8, hq=4, hkv=2, cols=1)),
])
def test_decreasing_row_starts_plan_nothing(lib, starts, kv, kw):
    """Rows are then unspecified; a plan that went on would count units past 32 bits and name CTAs that do not
    exist, whose partial rows lie behind the workspace."""
    rc, pieces = plan(lib, starts, kv, **kw)
    assert rc == dflash.OK
    assert all(p.cta < 148 and p.last_cta < 148 for p in pieces)
    assert pieces == []


def test_starts_outside_the_buffer_are_bounded_first(lib):
    """Clamped to [0, n_rows] these do not decrease: they are rows like others."""
    rc, pieces = plan(lib, [-5, 4, 200, 300], [9, 9, 9], n_rows=8, hq=4, hkv=2, cols=1)
    assert rc == dflash.OK
    assert {(p.seq, p.row0, p.n_tokens) for p in pieces} == {(0, 0, 4), (1, 4, 4)}


@pytest.mark.parametrize("kw", [dict(prefix=2 ** 31 - 1, cols=0), dict(prefix=2 ** 31 - 100, cols=0),
                                dict(prefix=2 ** 31 - 1 - 64, cols=1), dict(prefix=0, cols=2 ** 25 - 1)])
def test_key_counts_whose_last_block_passes_31_bits_are_refused(lib, kw):
    """A block or a page that ends behind key 2^31 - 1 has no 32-bit index."""
    rc, _ = plan(lib, [0, 1], [2 ** 31 - 1], n_rows=1, hq=1, hkv=1, **kw)
    assert rc == dflash.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(prefix=2 ** 31 - 257, cols=0), dict(prefix=0, cols=2 ** 25 - 5),
                                dict(prefix=2 ** 30, cols=2 ** 24 - 5)])
def test_the_largest_key_counts(lib, kw):
    kv = kw["cols"] * 64
    rc, pieces = plan(lib, [0, 1], [2 ** 31 - 1], n_rows=1, hq=1, hkv=1, **kw)
    assert rc == dflash.OK
    for seg, keys in ((0, kw["prefix"]), (1, kv)):
        at = 0
        for p in (x for x in pieces if x.segment == seg):
            assert p.block0 == at
            at = p.block1
        assert at == -(-keys // 128)
