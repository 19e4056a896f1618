"""Block tables that are views: one row of pages for every sequence, rows inside a wider table, rows that overlap."""
import pytest
import torch

import _target_ref as R
from speculative_decoding_block_ingest_gb300 import build, dflash, target

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(dflash.LIB_PATH):
        build.build()
    return dflash.load_library()


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def views():
    """(table, the row stride a kernel has to use)"""
    wide = torch.arange(40, dtype=torch.int32).view(4, 10)
    return [(wide[:, 2:5], 10), (wide[::2, :4], 20), (wide[1:2].expand(3, 10), 0), (wide[:1, :1].expand(5, 1), 0),
            (wide[:, :0], 10), (wide[:1], 10), (wide.as_strided((3, 4), (2, 1)), 2)]


@pytest.mark.parametrize("case", range(len(views())))
def test_stride_is_the_tensors_own(case, monkeypatch):
    """The binding describes a table as it lies in memory (on the host: only the device checks are left out)."""
    monkeypatch.setattr(target, "_cuda", lambda device, what: device)
    monkeypatch.setattr(target, "_vector", lambda device, what, t, *a: t.data_ptr())
    table, stride = views()[case]
    n = table.shape[0]
    z = torch.zeros(n + 1, dtype=torch.int32)
    assert target.Step(z, z[:n], table).fields[3:5] == (table.shape[1], stride)


@pytest.mark.parametrize("stride,ok", [(0, True), (4, True), (9, True), (3, False), (1, False), (-4, False)])
def test_rows_that_overlap_are_refused(lib, stride, ok):
    """One row for all sequences is a table, rows that overlap are not (the plan makes the checks of every call)."""
    import ctypes
    arr = (ctypes.c_int32 * 4)(0, 1, 2, 3)
    at = ctypes.addressof(arr)
    cache = dflash.PagedCacheDesc(dtype=dflash.BF16, page_size=64, n_kv_heads=1, head_dim=128)
    step = dflash.StepDesc(n_seq=3, n_rows=3, row_start=at, kv_len=at, block_table=at, table_cols=4,
                           table_stride=stride)
    n, out = ctypes.c_int32(0), (dflash.StepPiece * 64)()
    rc = lib.dflash_step_attention_plan(ctypes.byref(cache), ctypes.byref(step), 4, 1, 8, ctypes.byref(n), out, 64)
    assert rc == (dflash.OK if ok else dflash.ERR_INVALID_ARG)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["expanded", "sliced"])
def test_attention_over_a_viewed_table(kind):
    """Three sequences over the same pages, and tables that are columns of wider ones, as from a table of their own;
    the memory around the viewed entries names pages of NaN."""
    page, d, rows, kv = 16, 64, [2, 1, 3], [70, 70, 41]
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(9, page, 2, d, generator=g).to(BF) for _ in range(2))
    k[5:], v[5:] = float("nan"), float("nan")
    q = torch.randn(6, 4, d, generator=g).to(BF)
    starts, own = [0, 2, 3, 6], torch.tensor([[3, 0, 4, 1, 2]] * 3, dtype=torch.int32)
    wide = torch.full((3, 12), 7, dtype=torch.int32, device=DEV)
    if kind == "expanded":
        wide[0, :5] = own[0].to(DEV)
        table = wide[:1, :5].expand(3, 5)
    else:
        own[1], own[2] = own[1].flip(0), own[2].roll(1)
        wide[:, 4:9] = own.to(DEV)
        table = wide[:, 4:9]
    step = target.Step(i32(starts), i32(kv), table)
    o, lse = target.attention(target.PagedCache(k.to(DEV), v.to(DEV)), step, q.to(DEV))
    wo, to, wl, tl = R.attend_step(q, k, v, starts, kv, own, torch.zeros(0, dtype=torch.int32), 0, page, causal=True,
                                   scale=d ** -0.5)
    assert (abs(o.double().cpu().numpy() - wo) <= to).all()
    assert (abs(lse.double().cpu().numpy() - wl) <= tl).all()


@pytest.mark.gpu
def test_append_through_a_viewed_table():
    """Two sequences that append to different rows of the same page list, and columns of a wider table."""
    d = 64
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(5, 1, d, generator=g).to(BF).to(DEV) for _ in range(2))
    wide = torch.full((2, 9), 6, dtype=torch.int32, device=DEV)
    wide[0, :3] = i32([2, 0, 1])
    for table, at in ((wide[:1, :3].expand(2, 3), [(2, 3), (2, 4), (0, 9), (0, 10), (0, 11)]),
                      (wide[:, 1:3], [(0, 3), (0, 4), (6, 9), (6, 10), (6, 11)])):
        kc, vc = (torch.zeros(8, 16, 1, d, dtype=BF, device=DEV) for _ in range(2))
        # sequence 0 ends at key 5 of its table, sequence 1 at key 28 (expanded) or 12
        lens = [5, 28] if at[2][0] == 0 else [5, 12]
        target.append(target.PagedCache(kc, vc), target.Step(i32([0, 2, 5]), i32(lens), table), None, k, v)
        kw, vw = torch.zeros_like(kc), torch.zeros_like(vc)
        for i, (p, r) in enumerate(at):
            kw[p, r], vw[p, r] = k[i], v[i]
        assert torch.equal(kc, kw) and torch.equal(vc, vw)
