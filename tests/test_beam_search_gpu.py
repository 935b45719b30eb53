"""Selection, reordering, forking and shared attention together: a beam search over a hybrid model whose
scores are those of the same tokens in requests that share nothing."""
import importlib.util
import os

import pytest

import kda_delta_rule_token_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from kda_delta_rule_token_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_decode.py")
    spec = importlib.util.spec_from_file_location("beam_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("cache_type,page", [(kda.KDA_CACHE_BF16, 16), (kda.KDA_CACHE_E4M3, 64)])
@pytest.mark.parametrize("lengths,beams,steps", [((37,), 1, 5), ((200, 5, 1000), 4, 20), ((64, 500), 16, 35), ((300,), 48, 9)])
def test_search(example, lengths, beams, steps, cache_type, page):
    # The two ways differ in the attention layer alone, whose outputs are off by up to 2^-8 of their mean
    # value (weights in bf16), below 1 for keys and values of variance 1; W_o's and the head's rows, of norm 1,
    # average them to logits off by 2^-8 in standard deviation, four of which 1000 tokens pass, and a
    # log-probability is off by twice its largest logit's: 2^-5 a step.  A beam that went on from another's
    # state would be off by its logits themselves, about 1 a step.
    assert example.main(lengths=lengths, beams=beams, steps=steps, cache_type=cache_type, page_size=page) <= steps * 2.0 ** -5


def test_search_that_ends(example):
    """Beams that come to their end keep their score and their tokens."""
    assert example.main(lengths=(20, 33), beams=8, steps=15, vocab=12, end=3) <= 15 * 2.0 ** -5
