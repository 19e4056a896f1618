"""Callers of the 16-bit append that were built when its arguments ended with
the stride of q_out: what lies behind them is not read."""
import ctypes
import os
import subprocess

import pytest
import torch

from speculative_decoding_block_ingest_gb300 import dflash
from test_target_refusals import INV, P, UNS, append_args, cache, lib, ref, step  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIELDS = ("dtype", "n_heads", "q", "k", "v", "q_stride", "k_stride", "v_stride", "q_gain", "k_gain", "eps", "rot_dim",
          "inv_freq", "mscale", "positions", "q_out", "q_out_stride")


def test_size_of_the_arguments(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "dflash.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu\\n", sizeof(dflash_append_args), offsetof(dflash_append_args, q_out_stride), '
                   'offsetof(dflash_packed_append_args, k_values));\nreturn 0;\n}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split()
    assert got == ["128", "120", "136"]
    assert [n for n, _ in dflash.AppendArgs._fields_] == list(FIELDS)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=dflash.F16), UNS), (dict(n_heads=-1), INV), (dict(rot_dim=8), INV), (dict(inv_freq=None), INV),
    (dict(k_gain=P, eps=0.0), INV), (dict(q_out=None), INV), (dict(k_stride=255), INV)])
def test_interleaved_pairs_are_refused_alike(lib, kw, code):  # noqa: F811
    assert lib.dflash_step_append_interleaved(ref(cache()), ref(step()), ref(append_args(**kw)), None) == code
    assert lib.dflash_step_append_interleaved(ref(cache()), ref(step()), None, None) == INV
    assert lib.dflash_step_append_interleaved(None, ref(step()), ref(append_args()), None) == INV


@pytest.mark.gpu
@pytest.mark.parametrize("behind", [0, 1, 0xFF])
def test_what_lies_behind_the_arguments(behind):
    from speculative_decoding_block_ingest_gb300 import target as T
    dev = "cuda:0"

    class Args(ctypes.Structure):
        _fields_ = [f for f in dflash.AppendArgs._fields_ if f[0] in FIELDS]

    g = torch.Generator().manual_seed(1)
    n, hq, d = 5, 2, 64
    q, k, v = (torch.randn(n, h, d, generator=g).to(torch.bfloat16).to(dev) for h in (hq, 1, 1))
    rope = T.Rope(d, 1e4)
    rows = T.Step(*(torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, n], [9], [[1]])))
    want = [torch.zeros(2, 16, 1, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    wq = T.append(T.PagedCache(*want), rows, q, k, v, rope=rope)
    got = [torch.zeros_like(x) for x in want]
    gq = torch.empty_like(q)
    a = Args(dtype=dflash.BF16, n_heads=hq, q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), q_stride=hq * d, k_stride=d,
             v_stride=d, eps=1e-6, rot_dim=d, inv_freq=rope.ptr, mscale=1.0, q_out=gq.data_ptr(), q_out_stride=hq * d)
    raw = bytes(a) + bytes([behind]) * 16
    assert ctypes.sizeof(Args) == 128
    pages = T.PagedCache(*got)
    rc = dflash.load_library().dflash_step_append(pages.ref, rows.rows(pages, n), raw,
                                                  torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(gq, wq) and all(torch.equal(x, y) for x, y in zip(got, want))
