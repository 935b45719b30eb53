"""The example of a hybrid model's two layers: prompts followed by single
tokens agree with whole prompts."""
import importlib.util
import os

import pytest

import kda_delta_rule_token_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache_type,page", [(kda.KDA_CACHE_BF16, 16), (kda.KDA_CACHE_E4M3, 64)])
@pytest.mark.parametrize("lengths", [(200, 37, 1000), (5, 64)])
def test_hybrid_decode(lengths, cache_type, page):
    from kda_delta_rule_token_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # bf16 roundings between the steps (x, q, k, v, o: 2^-8 each, over two
    # layers of sums that average them) and, in the KDA layer, of the prompt's
    # tf32 products: within four of the largest value's.
    assert example.main(lengths=lengths, cache_type=cache_type, page_size=page) <= 4 * 2.0 ** -8
