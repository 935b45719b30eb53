"""Attention over caches, queries and gates that hold NaN or infinities: what a
row sees shows in its outputs, what it does not see has no effect, and neither
depends on how a call is cut between CTAs."""
import math

import pytest
import torch

import attn_ref as ref
import kda_delta_rule_token_gb300 as kda
from test_attn_gpu import BF, D, DEV, F8, Layer, _lib, check, queries, run_attend  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_of(kv, cu):
    """Request, and keys seen, of every packed row."""
    req, sees = [], []
    for b, n in enumerate(kv):
        new = 1 if cu is None else cu[b + 1] - cu[b]
        req += [b] * new
        sees += [n - new + 1 + i for i in range(new)]
    return torch.tensor(req, device=DEV), torch.tensor(sees, device=DEV)


def poison(layer, cache, b, key, head, channel, value=math.nan):
    at = (layer.table_list[b][key // layer.page], head, key % layer.page, channel)
    if layer.e4m3:
        cache.view(torch.uint8)[at] = 0x7F
    else:
        cache[at] = value


def finite(cache):
    """The cache with 0 for NaN and infinities (and for whatever no request's keys hold)."""
    x = cache.float()
    return torch.where(x.isfinite(), x, 0).to(cache.dtype)


def expect(layer, q, kv, cu, gate=None):
    """Values and bounds, were everything finite.  Over an e4m3 cache with the
    bound of queries held as two e4m3 parts (off by up to 2^-17 of the row's
    largest channel)."""
    args = (layer.table_list, kv, cu, layer.page, D ** -0.5, layer.ks, layer.vs, gate)
    q = torch.where(q.float().isfinite(), q.float(), 0).to(BF)
    k, v = finite(layer.k), finite(layer.v)
    want, wl, bound, lb = ref.attend(q, k, v, *args)
    if layer.e4m3 and cu is not None:
        G = layer.hq // layer.hkv
        mag = lambda c, s: (c.float() * s.view(1, -1, 1, 1)).abs()
        keys = mag(k, layer.ks).sum(-1).amax((0, 2)).repeat_interleave(G)
        top = mag(v, layer.vs).amax((0, 2, 3)).repeat_interleave(G).double()
        off = D ** -0.5 * 2.0 ** -17 * q.double().abs().amax(-1) * keys.double()
        bound, lb = bound + (torch.expm1(2 * off) * top)[..., None], lb + off
    return want, wl, bound, lb


# (new tokens, keys, query heads, key heads, page): decode where new is None
CALLS = {
    "decode": (None, [300, 77, 1000], 8, 2, 64),
    "decode_cut": (None, [30000, 5], 8, 2, 16),
    "few": ([5, 3, 7], [300, 40, 77], 8, 2, 16),
    "few_cut": ([8, 2], [20001, 9], 8, 2, 32),
    "prompt": ([150], [700], 4, 2, 16),
    "prompt_cut": ([128], [32768], 8, 2, 64),
}


def make(call, e4m3):
    new, kv, hq, hkv, page = CALLS[call]
    layer = Layer(hq, hkv, page, e4m3, seed=len(call))
    layer.fill(kv)
    cu = None
    if new is not None:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
    return layer, kv, cu, queries(layer, len(kv) if cu is None else cu[-1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("call", CALLS)
def test_nan_keys_and_queries(call, e4m3):
    """A NaN in a key makes every row that sees it NaN, and no other; a NaN
    in a query row that row alone."""
    layer, kv, cu, q = make(call, e4m3)
    req, sees = rows_of(kv, cu)
    G = layer.hq // layer.hkv
    want, wl, bound, lb = expect(layer, q, kv, cu)
    last = kv[0] - 1
    # An early key of head 0 that every row of request 0 sees, or (second turn) one that only its last row does.
    for key in (last // 3, last):
        keep = layer.k.clone()
        poison(layer, layer.k, 0, key, 0, 70)
        bad_q = q.clone()
        row = 1 if cu is None else cu[1] - 2
        bad_q[row, G, 5] = math.nan                       # first query head of key head 1
        hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
        hit[:, :G] = ((req == 0) & (sees > key))[:, None]
        hit[row, G] = True
        o, lse = run_attend(layer, bad_q, kv, cu, None, True)
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
        assert bool(o.t[hit].isnan().all()), "a row that sees NaN is not NaN"
        check(o.t[~hit], want[~hit], bound[~hit], "o")
        layer.k.copy_(keep)
    layer.done()


@pytest.mark.parametrize("call", ["prompt", "prompt_cut"])
def test_infinite_queries_over_e4m3(call):
    """A query row with an infinity comes out as NaN, alone, however the call is cut."""
    layer, kv, cu, q = make(call, True)
    want, wl, bound, lb = expect(layer, q, kv, cu)
    q[5, 1, 7], q[80, 2, 100] = math.inf, -math.inf
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[5, 1] = hit[80, 2] = True
    o, lse = run_attend(layer, q, kv, cu, None, True)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert bool(o.t[hit].isnan().all())
    check(o.t[~hit], want[~hit], bound[~hit], "o beside NaN rows")
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("call", CALLS)
def test_lse_of_nan_rows(call, e4m3):
    """lse is NaN where the logits are: -infinity says that a row sees no key."""
    layer, kv, cu, q = make(call, e4m3)
    req, sees = rows_of(kv, cu)
    G = layer.hq // layer.hkv
    want, wl, bound, lb = expect(layer, q, kv, cu)
    key = kv[0] // 2
    poison(layer, layer.k, 0, key, 1, 3)
    row = 1 if cu is None else cu[1] - 2
    q[row, 0, 100] = math.nan
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[:, G:] = ((req == 0) & (sees > key))[:, None]
    hit[row, 0] = True
    o, lse = run_attend(layer, q, kv, cu)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert bool(lse.t[hit].isnan().all())
    check(lse.t[~hit], wl[~hit], lb[~hit], "lse")
    layer.done()


class LargeQueries(Layer):
    """Keys and values of different sizes."""

    def values(self, n, scale, sigma):
        return super().values(n, scale, sigma if scale is self.ks else 1.0)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("up", [102, 110, 124])
def test_large_queries_over_e4m3(call, up):
    """Queries near 2^up (the largest bf16 are near 2^128) on keys near 2^-up: logits of ordinary size."""
    new, kv, hq, hkv, page = CALLS[call]
    layer = LargeQueries(hq, hkv, page, True, seed=up)
    layer.ks.fill_(2.0 ** (4 - up))
    layer.fill(kv, sigma=2.0 ** -up)
    cu = None
    if new is not None:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
    q = (queries(layer, len(kv) if cu is None else cu[-1]).float() * 2.0 ** up).to(BF)
    q[::3] = (q[::3].float() * 2.0 ** -up).to(BF)      # rows of ordinary size beside them
    assert bool(q.float().isfinite().all())
    want, wl, bound, lb = expect(layer, q, kv, cu)
    o, lse = run_attend(layer, q, kv, cu, None, True)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    check(o.t, want, bound, "o")
    check(lse.t, wl, lb, "lse")
    layer.done()


GATED = {
    "decode": (None, [300, 0, 77], 8, 2),
    "few": ([5, 3, 0, 7], [2, 300, 0, 0], 8, 2),            # rows that see no key, a request without keys
    "prompt": ([90, 40], [20, 300], 8, 2),
    "prompt_cut": ([128, 64], [60, 30000], 8, 2),
    "refused": ([3, 300, 2, 4], [50, 0, 3, 1], 8, 2),
    "refused_all": ([600, 300], [700, 0], 8, 2),
}


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("call", GATED)
def test_rows_without_keys_do_not_read_their_gate(call, f32, e4m3):
    """o is zero there whatever the gate holds: unused rows are often not written at all."""
    new, kv, hq, hkv = GATED[call]
    layer = Layer(hq, hkv, 16, e4m3)
    layer.fill(kv)
    cu = None
    if new is not None:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
    req, sees = rows_of(kv, cu)
    q = queries(layer, len(req))
    gate = torch.randn(len(req), hq, D, generator=layer.g, device=DEV)
    want, wl, bound, lb = expect(layer, q, kv, cu, gate)
    gate[sees <= 0] = math.nan
    o, lse = run_attend(layer, q, kv, cu, gate, f32)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert bool((o.t[sees <= 0] == 0).all()) and bool((lse.t[sees <= 0] == -math.inf).all())
    if not f32:
        bound = bound * (1 + ref.UBF) + ref.UBF * want.abs()
    check(o.t[sees > 0], want[sees > 0], bound[sees > 0], "o")
    layer.done()


VALUES = {
    "few_two_tiles": ([5, 3, 8], [300, 40, 77], 8, 2),          # two warps to a tile, each with rows of its own
    "few_turns": ([4, 2, 8], [300, 40, 65], 8, 2),              # or by turns, beside one that needs both
    "few_one": ([7, 9], [129, 9], 4, 4),
    "few_cut": ([8, 2], [20001, 9], 8, 2),
    "prompt": ([150, 40], [700, 41], 4, 2),
    "prompt_wide": ([300], [300], 2, 2),                        # 128 tokens to a row tile
    "prompt_deep": ([20], [520], 64, 1),                        # two tokens to a row tile
    "prompt_rounds": ([700, 650], [900, 650], 16, 8),
    "prompt_cut": ([128], [32768], 8, 2),
    "prompt_short": ([64, 33, 50], [64, 33, 90], 8, 2),         # the request ends in the tile
}


@pytest.mark.parametrize("e4m3,page", [(False, 16), (False, 128), (True, 32), (True, 64)])
@pytest.mark.parametrize("form", ["plain", "gate", "f32"])
@pytest.mark.parametrize("call", VALUES)
def test_values_that_a_row_does_not_see(call, form, e4m3, page):
    """NaN and infinities in the values of later tokens of the same chunk leave
    the rows before them as they are; the rows that see one have it in that channel only."""
    new, kv, hq, hkv = VALUES[call]
    layer = Layer(hq, hkv, page, e4m3, seed=len(call))
    layer.fill(kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    G = hq // hkv
    req, sees = rows_of(kv, cu)
    q = queries(layer, cu[-1])
    gate = torch.randn(cu[-1], hq, D, generator=layer.g, device=DEV) if form == "gate" else None
    want, wl, bound, lb = expect(layer, q, kv, cu, gate)
    hit = torch.zeros(want.shape, dtype=torch.bool, device=DEV)
    for b, n in enumerate(kv):
        t = new[b]
        spots = [(n - 1, 0, 0, math.nan), (n - 1, hkv - 1, 127, -math.inf), (n - 1 - t // 2, 0, 65, math.inf),
                 (n - t, hkv - 1, 30, math.nan)]
        for key, head, channel, value in spots[: 4 if b == 0 else 2]:
            poison(layer, layer.v, b, key, head, channel, value)
            hit[:, head * G:(head + 1) * G, channel] |= ((req == b) & (sees > key))[:, None]
    o, lse = run_attend(layer, q, kv, cu, gate, form == "f32")
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    if form != "f32":
        bound = bound * (1 + ref.UBF) + ref.UBF * want.abs()
    assert not o.t[hit].isfinite().any()
    check(o.t[~hit], want[~hit], bound[~hit], "o")
    check(lse.t, wl, lb, "lse")
    assert o.intact()
    layer.done()


def test_values_behind_a_prompt_of_clean_ones():
    """A call after one with NaN values, and requests beside the one that has them, are as ever."""
    layer = Layer(8, 2, 16)
    kv, cu = [400, 500], [0, 200, 500]
    layer.fill(kv)
    q = queries(layer, 500)
    clean, _ = run_attend(layer, q, kv, cu)
    torch.cuda.synchronize()
    keep = layer.v.clone()
    poison(layer, layer.v, 0, 399, 0, 9)
    o, _ = run_attend(layer, q, kv, cu)
    torch.cuda.synchronize()
    assert bool(o.t[199, :4, 9].isnan().all())
    # Bit for bit, but for the channels that are added again (four to a lane, those of key head 0 before the last row).
    same = torch.ones(500, 8, D, dtype=torch.bool, device=DEV)
    same[:200, :4, 8:12] = False
    assert torch.equal(o.t[same].view(torch.int16), clean.t[same].view(torch.int16))
    want, wl, bound, lb = expect(layer, q, kv, cu)
    again = ~same
    again[199, :4, 9] = False
    check(o.t[again], want[again], (bound * (1 + ref.UBF) + ref.UBF * want.abs())[again], "added again")
    layer.v.copy_(keep)
    o, _ = run_attend(layer, q, kv, cu)
    torch.cuda.synchronize()
    assert torch.equal(o.t.view(torch.int16), clean.t.view(torch.int16))
    layer.done()
