"""What the target-step entry points refuse, and with which code (CPU only:
every call here is refused before it would launch)."""
import ctypes

import pytest
import torch

from speculative_decoding_block_ingest_gb300 import build, dflash

INV, CAP, UNS = dflash.ERR_INVALID_ARG, dflash.ERR_CAPACITY, dflash.ERR_UNSUPPORTED
P = 1 << 20      # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(dflash.LIB_PATH):
        build.build()
    return dflash.load_library()


def cache(**kw):
    a = dict(k=P, v=P, dtype=dflash.BF16, n_pages=4, page_size=64, n_kv_heads=2, head_dim=128, page_stride=64 * 256,
             row_stride=256, head_stride=128)
    a.update(kw)
    return dflash.PagedCacheDesc(**a)


def step(**kw):
    a = dict(n_seq=2, n_rows=3, row_start=P, kv_len=P, block_table=P, table_cols=2, table_stride=2, prefix_len=10,
             prefix_pages=P)
    a.update(kw)
    return dflash.StepDesc(**a)


INV_FREQ = (ctypes.c_double * 64)(*[1.0] * 64)


def append_args(**kw):
    a = dict(dtype=dflash.BF16, n_heads=4, q=P, k=P, v=P, q_stride=512, k_stride=256, v_stride=256, eps=1e-6,
             rot_dim=128, inv_freq=ctypes.addressof(INV_FREQ), mscale=1.0, q_out=P, q_out_stride=512)
    a.update(kw)
    return dflash.AppendArgs(**a)


def attention_args(**kw):
    a = dict(n_heads=4, causal=1, scale=0.0, q=P, q_stride=512, out=P, out_stride=512, lse=P)
    a.update(kw)
    return dflash.AttentionArgs(**a)


def verify_args(**kw):
    a = dict(n_seq=2, k=3, vocab=1000, dtype=dflash.F32, draft=P, draft_stride=3, target_probs=P,
             target_seq_stride=4000, target_row_stride=1000, draft_probs=P, draft_seq_stride=3000,
             draft_row_stride=1000, u_accept=P, u_accept_stride=3, u_token=P, tokens=P, n_accepted=P)
    a.update(kw)
    return dflash.VerifyArgs(**a)


def ref(x):
    return None if x is None else ctypes.byref(x)


CACHE = [(dict(dtype=dflash.F32), UNS), (dict(dtype=dflash.FP8), UNS), (dict(head_dim=96), UNS),
         (dict(head_dim=256), UNS), (dict(page_size=8), UNS), (dict(page_size=48), UNS), (dict(page_size=512), UNS),
         (dict(n_kv_heads=0), INV), (dict(n_pages=0), INV), (dict(k=None), INV), (dict(v=P + 8), INV),
         (dict(row_stride=252), INV), (dict(head_stride=120), INV), (dict(page_stride=0), INV),
         (dict(page_stride=-64), INV), (dict(row_stride=64), INV)]
STEP = [(dict(n_seq=0), INV), (dict(n_seq=4097), INV), (dict(n_rows=-1), INV), (dict(n_rows=(1 << 24) + 1), INV),
        (dict(row_start=None), INV), (dict(kv_len=None), INV), (dict(block_table=None), INV),
        (dict(table_cols=-1), INV), (dict(table_stride=1), INV), (dict(prefix_len=-1), INV),
        (dict(prefix_pages=None), INV), (dict(table_cols=1 << 26, table_stride=1 << 26), INV)]


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_refused(lib, kw, code):
    c, s = cache(**kw), step()
    assert lib.dflash_step_append(ref(c), ref(s), ref(append_args()), None) == code
    assert lib.dflash_step_attention(ref(c), ref(s), ref(attention_args()), P, 1 << 40, None) == code
    assert lib.dflash_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", STEP)
def test_step_refused(lib, kw, code):
    c, s = cache(), step(**kw)
    assert lib.dflash_step_append(ref(c), ref(s), ref(append_args()), None) == code
    assert lib.dflash_step_attention(ref(c), ref(s), ref(attention_args()), P, 1 << 40, None) == code


def test_null_descriptors_refused(lib):
    n = ctypes.c_size_t(0)
    assert lib.dflash_step_append(None, ref(step()), ref(append_args()), None) == INV
    assert lib.dflash_step_append(ref(cache()), None, ref(append_args()), None) == INV
    assert lib.dflash_step_append(ref(cache()), ref(step()), None, None) == INV
    assert lib.dflash_step_attention(ref(cache()), ref(step()), None, P, 1 << 40, None) == INV
    assert lib.dflash_step_attention_workspace(None, 1, 4, ctypes.byref(n)) == INV
    assert lib.dflash_step_attention_workspace(ref(cache()), 1, 4, None) == INV
    assert lib.dflash_step_attention_status(None, None) == INV
    assert lib.dflash_step_attention_plan(None, ref(step()), 4, 1, 8, None, None, 0) == INV
    assert lib.dflash_verify_tokens(None, None) == INV
    assert lib.dflash_rope_frequencies(128, 1e6, 1.0, 0, 32.0, 1.0, None, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=dflash.F16), UNS), (dict(dtype=dflash.FP8), UNS), (dict(n_heads=-1), INV), (dict(rot_dim=8), INV),
    (dict(rot_dim=144), INV), (dict(inv_freq=None), INV), (dict(mscale=float("nan")), INV),
    (dict(q_gain=P, eps=0.0), INV), (dict(k_gain=P + 4), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(q=None), INV), (dict(q_out=None), INV), (dict(k=P + 2), INV), (dict(k_stride=255), INV),
    (dict(v_stride=128), INV), (dict(q_stride=504), INV), (dict(q_out_stride=516), INV),
    (dict(dtype=dflash.F32, k_stride=258), INV)])
def test_append_refused(lib, kw, code):
    assert lib.dflash_step_append(ref(cache()), ref(step()), ref(append_args(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_heads=0), INV), (dict(n_heads=3), INV), (dict(n_heads=130), UNS), (dict(scale=-1.0), INV),
    (dict(scale=float("inf")), INV), (dict(q=None), INV), (dict(out=None), INV), (dict(q=P + 2), INV),
    (dict(q_stride=508), INV), (dict(out_stride=256), INV)])
def test_attention_refused(lib, kw, code):
    assert lib.dflash_step_attention(ref(cache()), ref(step()), ref(attention_args(**kw)), P, 1 << 40, None) == code


def test_attention_workspace_refused(lib):
    call = lib.dflash_step_attention
    assert call(ref(cache()), ref(step()), ref(attention_args()), None, 1 << 40, None) == INV
    assert call(ref(cache()), ref(step()), ref(attention_args()), P + 128, 1 << 40, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=0), INV), (dict(k=-1), INV), (dict(vocab=0), INV), (dict(dtype=dflash.FP8), UNS),
    (dict(draft=None), INV), (dict(target_probs=None), INV), (dict(u_accept=None), INV), (dict(u_token=None), INV),
    (dict(tokens=None), INV), (dict(n_accepted=None), INV), (dict(target_row_stride=999), INV),
    (dict(draft_row_stride=999), INV), (dict(target_seq_stride=-1), INV), (dict(target_probs=P + 2), INV),
    (dict(draft_probs=P + 1, dtype=dflash.BF16), INV)])
def test_verify_refused(lib, kw, code):
    assert lib.dflash_verify_tokens(ref(verify_args(**kw)), None) == code


@pytest.mark.parametrize("args", [(0, 1e6, 1.0, 0, 32.0, 1.0), (63, 1e6, 1.0, 0, 32.0, 1.0),
                                  (64, 1.0, 1.0, 0, 32.0, 1.0), (64, 1e6, 0.5, 4096, 32.0, 1.0),
                                  (64, 1e6, 4.0, 0, 32.0, 1.0), (64, 1e6, 4.0, 4096, 0.0, 1.0),
                                  (64, 1e6, float("nan"), 4096, 32.0, 1.0)])
def test_rope_refused(lib, args):
    out, ms = (ctypes.c_double * 64)(), ctypes.c_double(0)
    assert lib.dflash_rope_frequencies(*args, out, ctypes.byref(ms)) == INV


def test_rope_frequencies(lib):
    """The drafter's formulas: plain powers, and the YaRN remap with its factor on cos and sin."""
    import numpy as np
    from _target_ref import rope_freqs
    from speculative_decoding_block_ingest_gb300 import target
    for rot, theta, yarn in ((128, 1e6, None), (64, 1e4, None), (2, 10.0, None), (128, 1e6, (32.0, 8192, 32.0, 1.0))):
        r = target.Rope(rot, theta, *(yarn or ()))
        inv, ms = rope_freqs(rot, theta, yarn)
        assert np.allclose(np.array(r.inv_freq[:rot // 2]), inv, rtol=1e-14)
        assert r.mscale == pytest.approx(ms, rel=1e-7)      # held in f32 by the drafter


def test_binding_refuses_host_tensors(lib):
    from speculative_decoding_block_ingest_gb300 import target
    k = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(dflash.DflashError):
        target.PagedCache(k, k)
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(dflash.DflashError):
        target.Step(z, z[:1], torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(dflash.DflashError):
        target.verify_tokens(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2, 8), torch.zeros(1, 1),
                             torch.zeros(1))


@pytest.mark.parametrize("cls", [dflash.AppendArgs, dflash.AttentionArgs, dflash.VerifyArgs])
def test_packed_arguments_are_the_structure(cls):
    floats = (ctypes.c_float, ctypes.c_double)
    values = [i + 0.5 if t in floats else 1000 + i for i, (_, t) in enumerate(cls._fields_)]
    got = cls.from_buffer_copy(dflash.packer(cls)(*values))
    assert [getattr(got, n) for n, _ in cls._fields_] == values
    with pytest.raises(dflash.DflashError) as e:       # n_seq, n_heads or dtype past 32 bits
        dflash.packer(cls)(1 << 31, *values[1:])
    assert e.value.code == dflash.ERR_INVALID_ARG
