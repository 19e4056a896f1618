"""What the 4-bit cache's calls and the next step's refuse, and that the
binding's structures are the header's (CPU only: nothing here launches)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from speculative_decoding_block_ingest_gb300 import dflash, target
from test_target_refusals import (CAP, INV, P, STEP, UNS, append_args, attention_args, lib, ref,  # noqa: F401
                                  step)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def packed(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, dtype=dflash.BF16, n_pages=4, page_size=64, n_kv_heads=2, head_dim=128,
             page_stride=64 * 128, row_stride=128, head_stride=64, scale_page_stride=64 * 16, scale_row_stride=8,
             scale_head_stride=512, k_unit=1.0, v_unit=1.0)
    a.update(kw)
    return dflash.PackedCacheDesc(**a)


def packed_append(**kw):
    rows = append_args()
    a = {n: getattr(rows, n) for n, _ in dflash.AppendArgs._fields_}
    a.update(k_values=P, v_values=P, k_values_stride=256, v_values_stride=256)
    a.update(kw)
    return dflash.PackedAppendArgs(**a)


def next_args(**kw):
    a = dict(n_seq=3, page_size=16, table_cols=4, n_pages=10, n_rows=5, prefix_len=7, table_stride=4)
    a.update({n: P for n, t in dflash.NextStepArgs._fields_ if t is ctypes.c_void_p})
    a.update(kw)
    return dflash.NextStepArgs(**a)


CACHE = [(dict(dtype=dflash.F32), UNS), (dict(head_dim=96), UNS), (dict(head_dim=32), UNS), (dict(page_size=8), UNS),
         (dict(page_size=48), UNS), (dict(n_kv_heads=0), INV), (dict(n_pages=0), INV), (dict(k=None), INV),
         (dict(v_scale=None), INV), (dict(v=P + 8), INV), (dict(k_scale=P + 4), INV), (dict(row_stride=120), INV),
         (dict(head_stride=48), INV), (dict(page_stride=0), INV), (dict(scale_row_stride=16), UNS),
         (dict(scale_head_stride=504), INV), (dict(scale_head_stride=256), INV), (dict(scale_page_stride=-8), INV), (dict(k_unit=0.0), INV),
         (dict(k_unit=0.75), INV), (dict(v_unit=float("nan")), INV), (dict(v_unit=2.0 ** 90), INV),
         (dict(k_unit=2.0 ** -80), INV), (dict(k_unit=-1.0), INV)]


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_refused(lib, kw, code):  # noqa: F811
    c, s = packed(**kw), step()
    assert lib.dflash_step_append_packed(ref(c), ref(s), ref(packed_append()), None) == code
    assert lib.dflash_step_attention_packed(ref(c), ref(s), ref(attention_args()), P, 1 << 40, None) == code
    assert lib.dflash_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", STEP)
def test_step_refused(lib, kw, code):  # noqa: F811
    c, s = packed(), step(**kw)
    assert lib.dflash_step_append_packed(ref(c), ref(s), ref(packed_append()), None) == code
    assert lib.dflash_step_attention_packed(ref(c), ref(s), ref(attention_args()), P, 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=dflash.F16), UNS), (dict(n_heads=-1), INV), (dict(rot_dim=8), INV), (dict(rot_dim=144), INV),
    (dict(inv_freq=None), INV), (dict(mscale=float("nan")), INV), (dict(k_gain=P, eps=0.0), INV), (dict(k=None), INV),
    (dict(q_out=None), INV), (dict(k_stride=255), INV), (dict(k_values=P), INV), (dict(v_values=P), INV), (dict(k_values=P + 8), INV), (dict(k_values_stride=128), INV),
    (dict(v_values_stride=260), INV)])
def test_append_refused(lib, kw, code):  # noqa: F811
    assert lib.dflash_step_append_packed(ref(packed()), ref(step()), ref(packed_append(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_heads=3), INV), (dict(n_heads=130), UNS), (dict(scale=-1.0), INV), (dict(q=None), INV),
    (dict(q_stride=508), INV), (dict(out_stride=256), INV)])
def test_attention_refused(lib, kw, code):  # noqa: F811
    assert lib.dflash_step_attention_packed(ref(packed()), ref(step()), ref(attention_args(**kw)), P, 1 << 40,
                                            None) == code


def test_null_arguments_refused(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    assert lib.dflash_step_append_packed(None, ref(step()), ref(packed_append()), None) == INV
    assert lib.dflash_step_append_packed(ref(packed()), None, ref(packed_append()), None) == INV
    assert lib.dflash_step_append_packed(ref(packed()), ref(step()), None, None) == INV
    assert lib.dflash_step_attention_packed(ref(packed()), ref(step()), None, P, 1 << 40, None) == INV
    assert lib.dflash_step_attention_packed(ref(packed()), ref(step()), ref(attention_args()), None, 1, None) == INV
    assert lib.dflash_step_attention_packed_workspace(None, 1, 4, ctypes.byref(n)) == INV
    assert lib.dflash_step_attention_packed_workspace(ref(packed()), 1, 4, None) == INV
    assert lib.dflash_step_attention_packed_workspace(ref(packed()), 1, 3, ctypes.byref(n)) == INV
    assert lib.dflash_next_step(None, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=0), INV), (dict(n_seq=4097), INV), (dict(page_size=8), UNS), (dict(page_size=100), UNS),
    (dict(n_rows=-1), INV), (dict(n_rows=(1 << 24) + 1), INV), (dict(n_pages=-1), INV), (dict(table_cols=-1), INV),
    (dict(prefix_len=-1), INV), (dict(table_stride=3), INV), (dict(table_cols=1 << 27, table_stride=1 << 27), INV),
    (dict(n_seq=4096, table_cols=1 << 20, table_stride=1 << 20), INV), (dict(prefix_len=(1 << 31) - 300), INV),
    (dict(kv_len=None), INV), (dict(row_start=None), INV), (dict(n_free=None), INV), (dict(rows=None), INV),
    (dict(block_table=None), INV), (dict(free_pages=None), INV), (dict(kv_len_out=None), INV),
    (dict(row_start_out=None), INV), (dict(n_free_out=None), INV), (dict(ticket=None), INV)])
def test_next_step_refused(lib, kw, code):  # noqa: F811
    assert lib.dflash_next_step(ref(next_args(**kw)), None) == code
    assert lib.dflash_last_error().decode() != ""


@pytest.mark.parametrize("cls", [dflash.AppendArgs, dflash.PackedAppendArgs, dflash.NextStepArgs])
def test_packed_bytes_are_the_structure(cls):
    floats = (ctypes.c_float, ctypes.c_double)
    values = [i + 0.5 if t in floats else 1000 + i for i, (_, t) in enumerate(cls._fields_)]
    got = cls.from_buffer_copy(dflash.packer(cls)(*values))
    assert [getattr(got, n) for n, _ in cls._fields_] == values


def test_structures_are_the_headers(tmp_path):
    """Sizes and places of the fields as a C compiler sees them."""
    pairs = [("dflash_append_args", dflash.AppendArgs, ""), ("dflash_packed_cache", dflash.PackedCacheDesc, ""),
             ("dflash_packed_append_args", dflash.PackedAppendArgs, "rows."),
             ("dflash_next_step_args", dflash.NextStepArgs, "")]
    lines, want = [], []
    inner = {n for n, _ in dflash.AppendArgs._fields_}
    for name, cls, prefix in pairs:
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            if f.startswith("_"):
                continue
            at = prefix + f if prefix and f in inner else f
            lines.append(f'printf("%zu\\n", offsetof({name}, {at}));')
            want.append(getattr(cls, f).offset)
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "dflash.h"\nint main(void) {\n' + "\n".join(lines)
                   + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split()
    assert list(map(int, got)) == want


def test_binding_refuses(lib):  # noqa: F811
    z8, z32 = torch.zeros(2, 16, 1, 32, dtype=torch.uint8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(dflash.DflashError):
        target.PagedCache4(z8, z8, z8[..., :4], z8[..., :4])          # host tensors
    with pytest.raises(dflash.DflashError):
        target.PagePool(z32, z32[:1], z32.view(2, 2), z32[:2], z32[:3], page_size=16)
    for bad in (dict(inv_freq=[1.0] * 3), dict(inv_freq=[float("nan")] * 4), dict(mscale=1.0)):
        with pytest.raises(dflash.DflashError):
            target.Rope(8, **bad)
    r = target.Rope(8, inv_freq=[1.0, 0.5, 0.25, 0.125], mscale=1.5, interleaved=True)
    assert list(r.inv_freq) == [1.0, 0.5, 0.25, 0.125] and r.mscale == 1.5 and r.interleaved == 1


def test_yarn_factor_in_64_bits(lib):  # noqa: F811
    r = target.Rope(128, 1e6, 32.0, 8192)
    assert ctypes.c_float(r.mscale64).value == r.mscale and target.Rope(128).mscale64 == 1.0


def test_reference_rounding():
    """The tests' own 64-bit rounding: every code and scale is its own nearest; borders go to the even code."""
    import numpy as np

    import _packed_ref as R4
    e = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e, R4.E4M3)
    assert np.array_equal(R4.nearest(R4.E2M1, R4.E2M1), np.arange(8))
    assert R4.nearest(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), R4.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6]
    x = np.random.default_rng(1).standard_normal((5, 128))
    c, s, y = R4.pack(x, 0.5)
    assert np.array_equal(R4.values(c, s, 0.5), y)
    assert np.abs(y - x).max() <= np.abs(x).max() / 6 * 1.07


def test_header_names_no_digits():
    """The list of exports is checked against names of letters."""
    text = open(os.path.join(ROOT, "include", "dflash.h")).read()
    assert not re.findall(r"\bdflash_\w*\d\w*\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
