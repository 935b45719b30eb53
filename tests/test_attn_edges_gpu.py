"""The paged softmax-attention operators at their edges: pages and offsets that
are not valid, requests refused by the plan, requests without tokens, and the
accuracy that each path's weights are held to."""
import math
import statistics

import pytest
import torch

import attn_ref as ref
import kda_delta_rule_token_gb300 as kda
from test_attn_gpu import BF, D, DEV, Layer, _lib, check, i32, queries, run_attend, verify  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("held", [-1, -2, -2 ** 31])
def test_held_pages_below_zero_are_reported(page, held):
    """A token whose page the table does not hold is never taken for one to leave unstored."""
    hq, hkv = 2, 1
    layer = Layer(hq, hkv, page, pages=4)
    for row in (page - 1, page - 2, 0):
        c = i32([row])
        table = i32([[held, held]])
        cu, kv, pos, info = i32([0, 0]), i32([0]), i32([0]), i32([0] * 4)
        slots = torch.zeros(1, dtype=torch.int64, device=DEV)
        # row 0: the page is taken from the free list, whose entry is as bad.
        kda.kda_attn_plan(layer.attn, 1, 1, c, i32([1]), i32([held, held]), i32([2]), table, cu, kv, pos, slots, info)
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
        assert slots.item() < -1
        q, k = torch.ones(1, hq, D, dtype=BF, device=DEV), torch.ones(1, hkv, D, dtype=BF, device=DEV)
        before = layer.k.view(torch.int16).clone()
        kda.kda_attn_append(layer.attn, 1, q, k, k, pos, slots, q)
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
        assert torch.equal(layer.k.view(torch.int16), before)
    layer.done()


def _timed(call, n=15):
    call()
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1000)
    return statistics.median(times)


def test_a_refused_chunk_is_written_by_all():
    """A long chunk that the plan refused (its length is 0, its rows still stand in
    the step) beside requests of few rows: 67 MB of zeros, which the whole device
    writes in some 20 us beside the call's other 150, and one of its SMs not within 1000."""
    new, kv, hq, hkv = [2] * 300 + [4096], [100] * 300 + [0], 64, 32
    layer = Layer(hq, hkv, 16)
    layer.fill(kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = queries(layer, cu[-1])
    o, lse = run_attend(layer, q, kv, cu)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert bool((o.t[600:] == 0).all()) and bool((lse.t[600:] == -math.inf).all())
    assert o.intact() and lse.intact()
    cu_t, kv_t = i32(cu), i32(kv)
    us = _timed(lambda: kda.kda_attn_prefill(layer.attn, 301, cu[-1], cu_t, q, layer.table, kv_t, o.t, layer.ws.t, lse=lse.t))
    print(f"\n  {us:.0f} us")
    assert us < 400
    layer.done()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lse", [False, True])
def test_several_refused_requests(f32, lse):
    """Short and long requests without keys among others, more of them than a CTA has threads."""
    new = [(5 * i) % 9 for i in range(300)] + [200, 0, 130, 3]
    kv = [0 if i % 3 else 20 + i for i in range(300)] + [0, 0, 0, 50]
    layer = Layer(4, 2, 16)
    layer.fill(kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = queries(layer, cu[-1] + 3)
    o, l = run_attend(layer, q, kv, cu, None, f32, lse)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    N = cu[-1]
    want, wl, bound, lb = ref.attend(q[:N], layer.k, layer.v, layer.table_list, kv, cu, 16, D ** -0.5)
    check(o.t[:N], want, bound if f32 else bound * (1 + ref.UBF) + ref.UBF * want.abs(), "o")
    if lse:
        none = wl == -math.inf
        assert torch.equal(l.t[:N] == -math.inf, none)
    assert bool((o.t[N:].view(torch.uint8) == 0x5A).all())
    assert o.intact()
    layer.done()


def test_offsets_that_claim_rows_twice():
    """Row offsets that are not ascending and claim more token tiles than there are rows: reported, nothing written."""
    layer = Layer(128, 1, 16)
    layer.fill([100] * 5)
    q = queries(layer, 100)
    o, lse = run_attend(layer, q, [100] * 5, [0, 100, 0, 100, 0, 100])
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
    assert bool((o.t.view(torch.uint8) == 0x5A).all()) and o.intact() and lse.intact()
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    verify(layer, q, [100] * 5, [0, 30, 30, 77, 90, 100])
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("tail", [1, 200])
def test_cut_calls_with_empty_requests_at_the_end(tail, e4m3):
    """The walk over requests ends with the last one that has tokens."""
    new = [64, 0, 300, 300] + [0] * tail
    kv = [20000, 7, 300, 400] + [0, 9] * tail
    kv = kv[: len(new)]
    layer = Layer(8, 4, 32, e4m3)
    layer.fill(kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    verify(layer, queries(layer, cu[-1]), kv, cu)
    layer.done()


# (query heads, key heads, new tokens, keys, e4m3): paths whose weights are two bf16 parts or f16
FINE = [
    (8, 2, None, [9, 17, 31, 64], False), (24, 1, None, [9, 17, 40], False), (40, 1, None, [8, 33], False),
    (8, 2, [3, 5, 8], [9, 17, 40], False), (2, 2, [4, 1], [9, 5], False),
    (8, 2, None, [9, 17, 31, 64], True), (24, 1, None, [9, 17, 40], True), (8, 2, [3, 5, 8], [9, 17, 40], True),
    (8, 2, [40], [60], True), (128, 1, [9, 3], [33, 12], True),
]


@pytest.mark.parametrize("hq,hkv,new,kv,e4m3", FINE)
def test_weights_as_fine_as_stated(hq, hkv, new, kv, e4m3, monkeypatch):
    """fp32 outputs within the weights' own rounding: 2^-16 (two bf16 parts: what
    the second leaves, 2^-8 of 2^-8), or 2^-11 (f16).  Few keys and small logits,
    so that the other terms of the bound stay below it."""
    layer = Layer(hq, hkv, 16, e4m3)
    layer.fill(kv)
    cu = None
    if new is not None:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
    q = queries(layer, len(kv) if cu is None else cu[-1], 0.05)
    o, lse = run_attend(layer, q, kv, cu, None, True)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    monkeypatch.setattr(ref, "UBF", 2.0 ** -11 if e4m3 else 2.0 ** -16)
    want, wl, bound, lb = ref.attend(q, layer.k, layer.v, layer.table_list, kv, cu, 16, D ** -0.5, layer.ks, layer.vs)
    if e4m3 and cu is not None and max(new) * hq // hkv > 32:
        # Queries as two e4m3 parts: a logit off by 2^-17 of the row's largest channel per unit of the keys' sum.
        keys = (layer.k.float().nan_to_num(0.0) * layer.ks.view(1, -1, 1, 1)).abs().sum(-1).amax()
        off = D ** -0.5 * 2.0 ** -17 * q.double().abs().amax(-1) * keys
        top = (layer.v.float().nan_to_num(0.0) * layer.vs.view(1, -1, 1, 1)).abs().amax()
        bound = bound + (torch.expm1(2 * off) * top)[..., None]
    check(o.t, want, bound, "o")
    layer.done()
