"""Types that the bindings of the calls for several continuations of one prompt refuse, since the library would take
them for others, and tensors too short for the call (on a recording stand-in for the library)."""
import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from test_continuations_abi import BF, D, fork, ints, lib, rec, select  # noqa: F401


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, torch.int64, torch.uint8])
def test_select_refuses_logits_that_are_neither_fp32_nor_bf16(rec, dtype):  # noqa: F811
    with pytest.raises(ValueError):
        select(torch.zeros(6, 50).to(dtype))
    assert not rec.calls


def test_select_takes_both_types_and_the_raw_view(rec):  # noqa: F811
    for dtype in (torch.float32, BF, torch.int16, torch.uint16):
        select(torch.zeros(6, 50).to(dtype))
    assert [a[5] for _, a in rec.calls] == [0, 1, 1, 1]


def shared(B=3, **change):
    args = dict(q=torch.zeros(3, 4, D, dtype=BF), block_table=ints(3, 7), kv_lens=ints(3), groups=2, cu_groups=ints(3),
                prefix_lens=ints(2), o=torch.zeros(3, 4, D, dtype=BF))
    args.update(change)
    kda.kda_attn_decode_shared(1, B, **args, workspace=16, workspace_bytes=1 << 30, stream=0)


LONG = torch.int64


@pytest.mark.parametrize("change", [
    dict(cu_groups=torch.zeros(3, dtype=LONG)), dict(prefix_lens=torch.zeros(2, dtype=LONG)), dict(kv_lens=torch.zeros(3, dtype=LONG)),
    dict(block_table=torch.zeros(3, 7, dtype=LONG)), dict(cu_groups=ints(2)), dict(prefix_lens=ints(1)), dict(kv_lens=ints(2)),
    dict(block_table=ints(2, 7)), dict(q=torch.zeros(3, 4, D)), dict(q=torch.zeros(3, 4, D, dtype=torch.float16)),
    dict(q=torch.zeros(2, 4, D, dtype=BF)), dict(o=torch.zeros(3, 4, D, dtype=torch.float16)), dict(o=torch.zeros(3, 4, D), o_f32=False),
    dict(o_f32=True), dict(o=torch.zeros(2, 4, D, dtype=BF)), dict(o=torch.zeros(3, 4, D, dtype=torch.float64)),
    dict(gate_logit=torch.zeros(3, 4, D, dtype=BF)), dict(gate_logit=torch.zeros(2, 4, D)), dict(lse=torch.zeros(3, 4, dtype=torch.float64)),
    dict(lse=torch.zeros(2))])
def test_shared_decode_refuses_types_and_short_tensors(rec, change):  # noqa: F811
    with pytest.raises(ValueError):
        shared(**change)
    assert not rec.calls


def test_shared_decode_takes_what_it_may_be_given(rec):  # noqa: F811
    shared()
    shared(q=torch.zeros(5, 4, D, dtype=torch.int16), o=torch.zeros(4, 4, D), gate_logit=torch.zeros(3, 4, D), lse=torch.zeros(3, 4))
    shared(q=16, o=16, o_f32=True, kv_lens=16, block_table=16, cu_groups=16, prefix_lens=16, max_pages=9)
    shared(groups=0, cu_groups=None, prefix_lens=None, block_table=ints(3, 20)[:, 3:7])
    shared(groups=5)     # for the library to refuse
    shared(B=-1)
    assert [a[11] for _, a in rec.calls] == [0, 1, 1, 0, 0, 0] and [a[4] for _, a in rec.calls][2:4] == [9, 20]


@pytest.mark.parametrize("change", [
    dict(S=torch.zeros(2, 1, D, D)), dict(conv_state=torch.zeros(2, 3, 3 * D)), dict(S=torch.zeros(3, 1, D, D, dtype=torch.float64)),
    dict(conv_state=torch.zeros(3, 3, 3 * D, dtype=BF)), dict(S_out=torch.zeros(2, 1, D, D), conv_out=torch.zeros(3, 3, 3 * D)),
    dict(S_out=torch.zeros(3, 1, D, D), conv_out=torch.zeros(2, 3, 3 * D)),
    dict(S_out=torch.zeros(3, 1, D, D), conv_out=torch.zeros(3, 3, 3 * D, dtype=torch.float64)), dict(conv_state=torch.zeros(3, 3 * D, 3).transpose(1, 2))])
def test_reorder_refuses_short_tensors_and_other_types(rec, change):  # noqa: F811
    args = dict(S=torch.zeros(3, 1, D, D), conv_state=torch.zeros(3, 3, 3 * D))
    args.update(change)
    with pytest.raises(ValueError):
        kda.kda_beam_reorder(1, 3, ints(3), args.pop("S"), args.pop("conv_state"), stream=0, **args)
    assert not rec.calls


@pytest.mark.parametrize("change", [
    dict(block_table=torch.zeros(3, 7, dtype=LONG)), dict(new_table=torch.zeros(3, 7, dtype=LONG)), dict(free_count=torch.zeros(1, dtype=LONG)),
    dict(block_table=ints(2, 7)), dict(new_table=ints(2, 7)), dict(free_count=ints(0))])
def test_fork_refuses_types_and_short_tensors(rec, change):  # noqa: F811
    with pytest.raises(ValueError):
        fork(**change)
    assert not rec.calls


def test_fork_takes_addresses(rec):  # noqa: F811
    fork(block_table=16, new_table=32, free_count=48, max_pages=7)
    fork(block_table=ints(5, 7), new_table=ints(4, 7), free_count=ints(3))
    assert [(a[4], a[5], a[10]) for _, a in rec.calls[:1]] == [(16, 7, 32)] and len(rec.calls) == 2
