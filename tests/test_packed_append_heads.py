"""Appending rows of many heads to a 4-bit cache on the GPU: a warp passes over
a row's heads more than 32 times, with codes on borders in every pass."""
import numpy as np
import pytest
import torch

import _packed_ref as P
import _target_ref as R
from test_packed_append import BF, DEV, F4, T, i32, pools, stored  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,rot,ti,inter", [
    (128, 8, 128, 128, BF, False), (128, 128, 128, 64, BF, True), (0, 160, 128, 0, F4, False), (260, 20, 64, 64, BF, False),
    (1, 256, 64, 32, BF, True)])
@pytest.mark.parametrize("n", [3, 1300])     # eight warps a row, and one
def test_many_heads(T, hq, hkv, d, rot, ti, inter, n):  # noqa: F811
    g = torch.Generator().manual_seed(71)
    # few values: quotients repeat, and many lie on borders; rows as one projection gives them
    distinct = min(n, 40)
    x = torch.randint(-3, 4, (distinct, (hq + 2 * hkv) * d), generator=g).to(ti).to(DEV)
    x = x.repeat(-(-n // distinct), 1)[:n]
    q, k, v = (t.unflatten(1, (-1, d)) if t.shape[1] else None for t in x.split([hq * d, hkv * d, hkv * d], 1))
    gain = torch.ones(d, device=DEV)
    page = 64
    starts, kv, table, _, n_pages = R.make_step([n], [n + 5], page, seed=72)
    mem = pools(n_pages, page, hkv, d, hnd=True)
    rope = T.Rope(rot, 1e4, interleaved=inter) if rot else None
    pos = [i % distinct for i in range(n)]
    qo = T.append(T.PagedCache4(*mem), T.Step(i32(starts), i32(kv), table.to(DEV)), q, k, v, rope=rope, q_gain=gain,
                  k_gain=gain, positions=i32(pos))
    inv, ms = R.rope_freqs(rot, 1e4) if rot else (np.zeros(0), 1.0)
    pages = [(int(table[0, j // page]), j % page) for j in range(5, n + 5)]
    ky, _ = P.rotate(k[:distinct], gain, 1e-6, pos[:distinct], inv, ms, inter)
    again = np.arange(n) % distinct
    for y, codes, scales in ((ky, mem[0], mem[2]), (v[:distinct].double().cpu().numpy(), mem[1], mem[3])):
        c, s, _ = P.pack(y)
        assert np.array_equal(stored(scales, pages), s[again])
        assert np.array_equal(stored(codes, pages), c[again])
    if q is not None:
        want, size = P.rotate(q[:distinct], gain, 1e-6, pos[:distinct], inv, ms, inter)
        tol = R.EPS[BF] * np.abs(want) + 1e-6 * size
        assert np.all(np.abs(qo.double().cpu().numpy() - want[again]) <= tol[again])
