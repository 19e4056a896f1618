"""Attention over a 4-bit cache on the GPU: what a call may read of its
surroundings when row starts are not what they should be."""
import pytest
import torch

from test_packed_attention import BF, DEV, HF, T, i32, pools  # noqa: F401

pytestmark = pytest.mark.gpu


def bad_starts(n_seq, rows, how):
    """Row starts of n_seq sequences that end at `rows`: two of them swapped, or not from 0."""
    s = [round(i * rows / n_seq) for i in range(n_seq + 1)]
    if how == "decrease":
        s[1], s[2] = s[2] + 1, s[1]
    else:
        s[0] = s[1] = max(s[1], 1)
    return s


@pytest.mark.parametrize("how", ["decrease", "not-from-0"])
@pytest.mark.parametrize("n_seq,rows,hq,hkv,d,dt,prefix", [
    (3, 12, 4, 2, 64, BF, 0),          # a block of the merge for a row and head
    (300, 400, 8, 1, 128, HF, 0),      # a warp
    (1300, 1400, 6, 2, 64, BF, 0),     # half a warp
    (3, 12, 2, 1, 128, BF, 40),        # with a prefix: both kernels
], ids=["block", "warp", "half-warp", "prefix"])
def test_parts_are_read_from_the_workspace_only(T, how, n_seq, rows, hq, hkv, d, dt, prefix):  # noqa: F811
    """Rows that no piece names find in the workspace what was there: here CTAs and places that exist in no plan.  Results
    are unspecified, but nothing behind the workspace has a part in them."""
    mem = pools(16, 16, hkv, d, seed=1)
    cache = T.PagedCache4(*mem, dtype=dt)
    starts = bad_starts(n_seq, rows, how)
    pages = torch.arange(12, dtype=torch.int32)[None].to(DEV)
    step = T.Step(i32(starts), i32([190 - i % 70 for i in range(n_seq)]), pages.expand(n_seq, 12),
                  i32([12, 13, 14]), prefix)
    q = torch.randn(rows, hq, d, generator=torch.Generator().manual_seed(2)).to(dt).to(DEV)
    n = cache.workspace_bytes(rows, hq)
    n_cta = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    for first in (n_cta - 2, 0):
        for place in (255, 127, 17):
            got = []
            for behind in (1000.0, -7.0):
                ws = i32([first, n_cta - 1, place, 0]).repeat(n // 16 + 1024).view(torch.uint8)
                ws[n:].view(torch.float32).fill_(behind)
                out, lse = torch.full((rows, hq, d), 3.0, dtype=dt, device=DEV), torch.full((rows, hq), 3.0, device=DEV)
                T.attention(cache, step, q, out=out, lse=lse, workspace=ws[:n])
                torch.cuda.synchronize()
                assert bool((ws[n:].view(torch.float32) == behind).all())
                got.append((out.view(torch.int16), lse.view(torch.int32)))
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
