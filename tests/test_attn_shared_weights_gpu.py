"""How fine the softmax weights of kda_attn_decode_shared are, by the kernel that takes a group's prefix."""
import pytest

import attn_ref as ref
from test_attn_gpu import queries
from test_attn_shared_gpu import build, verify

pytestmark = pytest.mark.gpu

# Rows per key head of a group, and of the call, that stand in one bf16 part: 2^-8; two parts: 2^-16; f16: 2^-11.
CASES = [
    # groups, hq, hkv, page, e4m3, bits
    ([(3, 64)], 8, 2, 16, False, 16), ([(8, 128)], 8, 2, 16, False, 16), ([(2, 192)], 16, 1, 64, False, 16),
    ([(4, 128), (30, 64)], 4, 4, 32, False, 8), ([(16, 128), (17, 64)], 1, 1, 16, False, 8), ([(16, 128), (16, 64), (1, 9)], 1, 1, 16, False, 16),
    ([(4, 192), (4, 128), (4, 64)], 4, 1, 16, False, 16), ([(9, 128)], 8, 2, 16, False, 8), ([(40, 192)], 5, 1, 32, False, 8),
    ([(3, 64)], 128, 1, 64, False, 8), ([(3, 64)], 8, 2, 32, True, 11), ([(40, 128)], 8, 2, 32, True, 11), ([(40, 192)], 16, 1, 64, True, 11),
]


@pytest.mark.parametrize("groups,hq,hkv,page,e4m3,bits", CASES)
def test_weights_as_fine_as_stated(groups, hq, hkv, page, e4m3, bits, monkeypatch):
    """fp32 outputs within the weights' own rounding.  Few keys and small logits, so that the other terms of the bound
    stay below it (test_attn_bounds.py: weights of one bf16 part fall outside that of two)."""
    layer, lens = build(groups, 1, hq, hkv, page, e4m3, seed=sum(p for _, p in groups), ragged=False)
    monkeypatch.setattr(ref, "UBF", 2.0 ** -bits)
    verify(layer, queries(layer, len(lens), 0.05), lens, f32=True)
    layer.done()
