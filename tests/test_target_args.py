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


def test_two_threads_ask_for_workspaces(lib, monkeypatch):  # noqa: F811
    """Sizes are kept for some shapes at a time; a thread that makes room takes no other thread's answer away."""
    import contextlib
    import threading

    class Lib:
        def dflash_step_attention_workspace(self, ref, rows, heads, n):
            n._obj.value = 1000 * rows + heads
            return 0

    monkeypatch.setattr(target.dflash, "load_library", Lib)
    monkeypatch.setattr(target.torch.cuda, "device", lambda d: contextlib.nullcontext())

    class Others(dict):
        """Between storing an answer and reading it, other threads fill the table and clear it."""

        def __setitem__(self, key, value):
            dict.__setitem__(self, key, value)
            self.clear()

    c = object.__new__(target.PagedCache)
    c.device, c.ref, c._ws = None, None, Others()
    assert c.workspace_bytes(3, 4) == 3004
    c._ws, bad = {}, []

    def ask(first):
        for i in range(first, first + 500):
            if c.workspace_bytes(i, 8) != 1000 * i + 8:
                bad.append(i)

    threads = [threading.Thread(target=ask, args=(100 * i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == [] and len(c._ws) <= 66 + len(threads)
