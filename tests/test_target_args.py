"""Arguments of the target-step calls that the kernels take in fewer bits than the caller gives (CPU only)."""
import ctypes

import pytest

from speculative_decoding_block_ingest_gb300 import dflash, target
from test_target_refusals import P, append_args, cache, lib, ref, step  # noqa: F401 (lib is a fixture)


@pytest.mark.parametrize("kw", [dict(q_gain=P, eps=1e-60), dict(k_gain=P, eps=1e-46), dict(q_gain=P, eps=float("nan")),
                                dict(mscale=1e300), dict(mscale=-1e39)])
def test_numbers_that_are_no_floats_are_refused(lib, kw):  # noqa: F811
    """An eps of 0 in f32 would make NaN of a row of zeros, an infinite factor of every row."""
    assert lib.dflash_step_append(ref(cache()), ref(step()), ref(append_args(**kw)), None) == dflash.ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [1e-50, 0.0, -1.0, 1e39, float("nan"), float("inf")])
def test_a_scale_that_is_no_float_is_refused(scale):
    """0 stands for the default, which a tiny scale must not become."""
    with pytest.raises(dflash.DflashError) as e:
        target._scale(scale)
    assert e.value.code == dflash.ERR_INVALID_ARG


def test_scales():
    assert target._scale(None) == 0.0 and target._scale(0.125) == 0.125
    assert target._scale(1e-40) == ctypes.c_float(1e-40).value > 0
