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


@pytest.mark.parametrize("far", [1e30, -1e30, 3e38, -3e38])
@pytest.mark.parametrize("K,V,num", [(1, 5000, 4), (3, 1000, 8), (2, 3, 5), (5, 40000, 64)])
def test_scores_far_from_zero(K, V, num, far):
    """All 64-bit scores of a group are equal there: the lower beam's come first, of a beam those of the larger logits,
    of equal logits the lower tokens, however many parts the row was cut into."""
    x, scores = make(2, K, V, seed=K + V)
    x[:, V // 2] = x[:, 0]                   # equal logits as well
    scores[:] = far
    with Ctx() as ctx:
        s, t, r = select(ctx, x, scores, num)
    assert bool((s == scores[0, 0]).all())
    for g in range(2):
        want = []
        for k in range(K):
            best = x[g * K + k].double().sort(descending=True, stable=True).indices[:num]
            want += [(g * K + k, v) for v in best.tolist()]
        assert list(zip(r[g].tolist(), t[g].tolist())) == want[:num]


def test_marks_of_beams_that_do_not_count():
    """Scores of -1e30 for all beams but one, and a vocabulary with few open tokens: the beam that counts first, then the
    others by their own logits."""
    x, scores = make(1, 3, 600, seed=4)
    x[:, 4:] = -math.inf
    scores[:] = -1e30
    scores[0, 0] = -2.0
    with Ctx() as ctx:
        s, t, r = select(ctx, x, scores, 7)
    y = beam_ref.scores64(x, scores, None, 0)
    assert r[0].tolist() == [0] * 4 + [1] * 3
    assert t[0, 4:].tolist() == x[1, :4].sort(descending=True).indices[:3].tolist()
    assert t[0, :4].tolist() == y[0, 0].sort(descending=True, stable=True).indices[:4].tolist()
    assert bool((s[0, 4:] == scores[0, 1]).all())


@pytest.mark.parametrize("K,V,num", [(1, 9000, 4), (3, 30000, 8), (4, 4097, 33)])
def test_logits_closer_than_scores(K, V, num):
    """Logits about 0 that differ by less than 64 bits of a score hold: the largest ones all the same."""
    gen = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randn(2 * K, V, generator=gen, device=DEV) * 1e-25
    scores = -torch.arange(2 * K, device=DEV, dtype=torch.float32).view(2, K)   # beams that are far apart
    with Ctx() as ctx:
        s, t, r = select(ctx, x, scores, num)
    for g in range(2):
        best = x[g * K].sort(descending=True, stable=True).indices[:num]
        assert t[g].tolist() == best.tolist() and r[g].tolist() == [g * K] * num
