"""The paged softmax-attention operators at their edges: pages and offsets that
are not valid, requests refused by the plan."""
import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from test_attn_gpu import BF, D, DEV, Layer, _lib, i32  # noqa: F401

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
