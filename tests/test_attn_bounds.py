"""The bounds that the attention tests hold fp32 outputs to, against mistakes
planted in a plain form: weights held in fewer bits than stated fall outside."""
import pytest
import torch

import attn_ref as ref

D = ref.D
BF = torch.bfloat16


def _case(hq, hkv, kv, seed=0):
    """Few keys and small logits, as in the tests of the weights' accuracy."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // 16) for n in kv]
    k, v = (torch.randn(sum(pages), hkv, 16, D, generator=g).to(BF) for _ in range(2))
    table, at = [], 0
    for n in pages:
        table.append(list(range(at, at + n)))
        at += n
    return (torch.randn(len(kv), hq, D, generator=g) * 0.05).to(BF), k, v, table


def _outputs(q, k, v, table, kv, rounded):
    """Attention with weights exp(z - max) passed through `rounded`, sums of the weights as they were."""
    G = q.shape[1] // k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64)
    for b, n in enumerate(kv):
        for h in range(q.shape[1]):
            kk, vv = (c[table[b], h // G].double().reshape(-1, D)[:n] for c in (k, v))
            z = kk @ q[b, h].double() * D ** -0.5
            p = torch.exp(z - z.max())
            o[b, h] = rounded(p) @ vv / p.sum()
    return o


def _bf16(p):
    return p.to(BF).double()


def _two_bf16(p):
    return _bf16(p) + _bf16(p - _bf16(p))


def _f16(p):
    return p.half().double()


@pytest.mark.parametrize("rounded,step,inside", [
    (_two_bf16, 2.0 ** -16, True), (_bf16, 2.0 ** -16, False),
    (_f16, 2.0 ** -11, True), (_bf16, 2.0 ** -11, False), (_bf16, 2.0 ** -8, True)])
@pytest.mark.parametrize("hq,hkv,kv", [(8, 2, [9, 17, 31, 64]), (24, 1, [9, 17, 40])])
def test_bound_tells_the_weights_bits(hq, hkv, kv, rounded, step, inside, monkeypatch):
    q, k, v, table = _case(hq, hkv, kv)
    monkeypatch.setattr(ref, "UBF", step)
    want, _, bound, _ = ref.attend(q, k, v, table, kv, None, 16, D ** -0.5)
    off = (_outputs(q, k, v, table, kv, rounded) - want).abs()
    assert bool((off <= bound).all()) == inside
