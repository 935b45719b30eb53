"""The paged softmax-attention entry points' refusals that need no GPU: what
kda_attn_create and calls without a context reject before any CUDA call."""
import ctypes
import math

import pytest

import kda_delta_rule_token_gb300 as kda
from kda_delta_rule_token_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.load()


def _create(lib, freqs=None, gammas=(None, None), scales=(None, None), **change):
    f = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, cache_type=0, rotary_dim=0,
             rope_interleaved=0, rms_eps=1e-6, softmax_scale=0.1)
    f.update(change)
    cfg = kda._AttnConfig(*f.values())
    out = ctypes.c_void_p(1)
    arr = (ctypes.c_double * len(freqs))(*freqs) if freqs else None
    status = lib.kda_attn_create(ctypes.byref(cfg), arr, *gammas, *scales, ctypes.byref(out))
    assert out.value is None
    return status


@pytest.mark.parametrize("change", [
    dict(num_q_heads=0), dict(num_kv_heads=0), dict(num_q_heads=7), dict(rms_eps=-1.0), dict(rms_eps=math.nan),
    dict(rms_eps=math.inf), dict(softmax_scale=0.0), dict(softmax_scale=-1.0), dict(softmax_scale=math.nan),
    dict(softmax_scale=math.inf), dict(cache_type=2), dict(cache_type=-1), dict(rotary_dim=-16),
    dict(rotary_dim=8), dict(rotary_dim=144), dict(rotary_dim=32), dict(cache_type=1)])
def test_create_refuses_arguments(lib, change):
    assert _create(lib, **change) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_create_refuses_frequencies(lib, bad):
    assert _create(lib, rotary_dim=16, freqs=[1.0] * 7 + [bad]) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(head_dim=64), dict(head_dim=256), dict(page_size=0), dict(page_size=8), dict(page_size=48),
    dict(page_size=256), dict(num_q_heads=258)])
def test_create_refuses_unsupported(lib, change):
    assert _create(lib, **change) == kda.KDA_ERR_UNSUPPORTED


def test_create_refuses_alignment(lib):
    assert _create(lib, gammas=(20, None)) == kda.KDA_ERR_ALIGNMENT
    assert _create(lib, gammas=(None, 24)) == kda.KDA_ERR_ALIGNMENT
    assert _create(lib, cache_type=1, scales=(18, 16)) == kda.KDA_ERR_ALIGNMENT
    assert _create(lib, cache_type=1, scales=(16, 19)) == kda.KDA_ERR_ALIGNMENT


def test_calls_without_a_context(lib):
    n = None
    out = ctypes.c_void_p()
    assert lib.kda_attn_create(n, n, n, n, n, n, ctypes.byref(out)) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_attn_create(n, n, n, n, n, n, n) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_attn_bind_cache(n, 1, 16, 16) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_attn_plan(n, 1, 1, 16, 16, 16, 1, 16, 16, 1, 16, 16, 16, 16, 16, n) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_attn_append(n, 1, 16, 128, 16, 128, 16, 128, 16, 16, 16, n) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_attn_workspace_bytes(n) == 0
    assert lib.kda_attn_decode(n, 1, 16, 16, 1, 16, n, 16, 0, n, 16, 1 << 30, n) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_attn_prefill(n, 1, 1, 16, 16, 16, 1, 16, n, 16, 0, n, 16, 1 << 30, n) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_attn_sync_status(n, n) == kda.KDA_ERR_INVALID_ARG
    lib.kda_attn_destroy(n)  # ignored


def test_binding_refuses_a_wrong_number_of_frequencies(lib):
    with pytest.raises(ValueError):
        kda.kda_attn_create(8, 2, page_size=16, rotary_dim=32, inv_freq=[1.0] * 15)


def test_binding_refuses_heads_that_are_not_dense(lib):
    import torch
    t = torch.zeros(4, 128, 8, dtype=torch.bfloat16).transpose(1, 2)
    with pytest.raises(ValueError):
        kda.kda_attn_append(None, 4, t, t, t, None, None, t)
