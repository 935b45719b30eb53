"""Plain 64-bit forms of beam selection and of what its results may be off by."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def scores64(logits, scores, done, end_token):
    """[groups, beams, vocab]: the scores of all continuations, NaN as -infinity."""
    G, K = scores.shape
    x = logits[:G * K].to(F64).view(G, K, -1)
    most = x.amax(2, keepdim=True)
    most = torch.where(most.isinf(), torch.zeros_like(most), most)
    y = (x - most) - (x - most).exp().sum(2, keepdim=True).log() + scores.to(F64)[..., None]
    if done is not None:
        only = torch.full_like(y, -math.inf)
        only[..., end_token] = scores.to(F64)
        y = torch.where(done.bool()[..., None], only, y)
    return torch.where(y.isnan(), torch.full_like(y, -math.inf), y)


def best(y, num):
    """(scores, beams, tokens) [groups, num] of the highest, of equal ones those of the lowest index."""
    G, K, V = y.shape
    s, at = y.reshape(G, K * V).sort(dim=1, descending=True, stable=True)
    return s[:, :num], at[:, :num] // V, at[:, :num] % V


def places(beams):
    """Of one group's chosen beams, best first: the place that each continuation comes to."""
    n, place, left = len(beams), [None] * len(beams), []
    for i, k in enumerate(beams):
        if k in beams[:i]:
            left.append(i)
        else:
            place[i] = k
    free = [p for p in range(n) if p not in place]
    for i, p in zip(left, free):
        place[i] = p
    return place


def check(got, y, num, keep, slack):
    """Compares (out_scores, out_tokens, out_rows) [groups, num] with the formula.  `slack`: how far a
    score may be off beside its own rounding to fp32.  Tokens and beams have to be the formula's wherever
    their score is further than that from the scores beside it that another beam has."""
    G, K, V = y.shape
    s, k, v = best(y, min(num + 1, K * V))
    for g in range(G):
        want = list(zip(s[g].tolist(), k[g].tolist(), v[g].tolist()))
        have = list(zip(*(t[g].tolist() for t in got)))
        have = [(a, r - g * K, t) for a, t, r in have]
        if keep:
            # Back to the order of the scores; the places follow from the beams chosen.
            place = places([w[1] for w in want[:num]])
            have = [have[p] for p in place]
        for i in range(num):
            (ws, wk, wv), (hs, hk, hv) = want[i], have[i]
            assert 0 <= hk < K and 0 <= hv < V
            if ws == -math.inf or math.isinf(hs):
                assert hs == ws
            else:
                assert abs(hs - ws) <= slack + 2.0 ** -23 * abs(ws), (g, i, hs, ws)
                # What was chosen has the score that is said.
                own = y[g, hk, hv].item()
                assert abs(hs - own) <= slack + 2.0 ** -23 * abs(own), (g, i, hs, own)
            near = [j for j in (i - 1, i + 1) if 0 <= j < len(want) and want[j][1] != wk
                    and want[j][0] != ws and abs(want[j][0] - ws) <= 2 * slack]
            if not near:
                assert (hk, hv) == (wk, wv), (g, i, have[i], want[i])
