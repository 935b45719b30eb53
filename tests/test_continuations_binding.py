"""Types that the bindings of the calls for several continuations of one prompt refuse, since the library would take
them for others, and tensors too short for the call (on a recording stand-in for the library)."""
import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from test_continuations_abi import BF, D, ints, lib, rec, select  # noqa: F401


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, torch.int64, torch.uint8])
def test_select_refuses_logits_that_are_neither_fp32_nor_bf16(rec, dtype):  # noqa: F811
    with pytest.raises(ValueError):
        select(torch.zeros(6, 50).to(dtype))
    assert not rec.calls


def test_select_takes_both_types_and_the_raw_view(rec):  # noqa: F811
    for dtype in (torch.float32, BF, torch.int16, torch.uint16):
        select(torch.zeros(6, 50).to(dtype))
    assert [a[5] for _, a in rec.calls] == [0, 1, 1, 1]
