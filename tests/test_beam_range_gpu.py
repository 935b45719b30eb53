"""Beam selection at the ends of its range: vocabularies next to 2^31, scores far from 0."""
import math

import pytest
import torch

import beam_ref
import kda_delta_rule_token_gb300 as kda
from test_beam_gpu import DEV, SLACK, Ctx, make, select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [2 ** 31 - 4096, 2 ** 31 - 4095, 2 ** 31 - 2, 2 ** 31 - 1])
def test_workspace_next_to_the_largest_vocabulary(V):
    """As much as for one a little smaller: a part and `num` candidates for every CTA."""
    with Ctx() as ctx:
        for groups, num in ((1, 1), (3, 64)):
            near = kda.kda_beam_select_workspace_bytes(ctx, groups, 1, 2 ** 31 - 8192, num)
            assert kda.kda_beam_select_workspace_bytes(ctx, groups, 1, V, num) == near < 1 << 20


@pytest.mark.parametrize("bf16", [False, True])
def test_largest_vocabulary(bf16):
    V = 2 ** 31 - 1
    x = torch.empty(1, V, dtype=torch.bfloat16 if bf16 else torch.float32, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    want = {V - 1: 20.0, 0: 19.5, V - 5000: 19.0, 2 ** 30 + 1: 18.5}
    for at, value in want.items():
        x[0, at] = value
    with Ctx() as ctx:
        s, t, r = select(ctx, x, torch.zeros(1, 1, device=DEV), 4)
        assert kda.kda_sync_status(ctx) == kda.KDA_OK
    total = sum(float(c.double().exp().sum()) for c in x[0].split(1 << 27))
    assert t[0].tolist() == list(want) and r[0].tolist() == [0] * 4
    for got, value in zip(s[0].tolist(), want.values()):
        exact = value - math.log(total)
        assert abs(got - exact) <= SLACK + 2.0 ** -23 * abs(exact)
