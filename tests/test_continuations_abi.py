"""What the calls for several continuations of one prompt refuse without a GPU, and what their Python
bindings make of tensors' shapes, strides and types (on a recording stand-in for the library)."""
import pytest
import torch

import beam_ref
import fork_ref
import kda_delta_rule_token_gb300 as kda
from kda_delta_rule_token_gb300 import build

D = 128
BF = torch.bfloat16


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib():
    build.build()
    return kda.load()


@pytest.fixture
def rec(lib, monkeypatch):
    r = Recorder()
    monkeypatch.setattr(kda, "load", lambda path=None: r)
    return r


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_calls_without_a_context(lib):
    n, bad = None, kda.KDA_ERR_INVALID_ARG
    assert lib.kda_beam_select_workspace_bytes(n, 1, 1, 1, 1) == 0
    assert lib.kda_beam_select(n, 1, 1, 1, 16, 0, 1, 16, n, 0, 1, 0, 16, 16, 16, 16, 1 << 20, n) == bad
    assert lib.kda_beam_reorder(n, 1, 16, 16, 16, 16, 16, 0, n) == bad
    assert lib.kda_attn_fork_workspace_bytes(n, 1, 1) == 0
    assert lib.kda_attn_fork(n, 1, *[16] * 3, 1, 16, 16, 1, *[16] * 8, 1 << 20, n) == bad
    assert lib.kda_attn_copy_pages(n, 1, 16, 16, 16, n) == bad
    assert lib.kda_attn_shared_workspace_bytes(n, 1) == 0
    assert lib.kda_attn_decode_shared(n, 1, 16, 16, 1, 16, 0, n, n, n, 16, 0, n, 16, 1 << 30, n) == bad


# ---------------------------------------------------------------- binding


def select(logits=None, scores=None, outs=None, **more):
    logits = torch.zeros(6, 50) if logits is None else logits
    scores = torch.zeros(2, 3) if scores is None else scores
    outs = (torch.zeros(2, 4), ints(2, 4), ints(2, 4)) if outs is None else outs
    kda.kda_beam_select(1, 2, 3, logits, scores, 4, *outs, 16, workspace_bytes=1 << 20, stream=0, **more)


def test_select_takes_rows_at_any_stride(rec):
    select(torch.zeros(6, 64)[:, :50])
    select(torch.zeros(18, 50, dtype=BF)[::3])
    select(torch.zeros(9, 50, dtype=torch.int16))
    assert [(a[3], a[5], a[6]) for _, a in rec.calls] == [(50, 0, 64), (50, 1, 150), (50, 1, 50)]


@pytest.mark.parametrize("change", [
    dict(logits=torch.zeros(50, 6).t()), dict(logits=torch.zeros(5, 50)), dict(logits=torch.zeros(2, 3, 50)),
    dict(scores=torch.zeros(2, 3, dtype=torch.float64)), dict(scores=torch.zeros(2, 6)[:, ::2]), dict(scores=torch.zeros(5)),
    dict(done=ints(2, 3)), dict(done=torch.zeros(5, dtype=torch.uint8)),
    dict(outs=(torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.int64), ints(2, 4))),
    dict(outs=(torch.zeros(2, 3), ints(2, 4), ints(2, 4)))])
def test_select_refuses_tensors(rec, change):
    with pytest.raises(ValueError):
        select(**change)
    assert not rec.calls


def test_reorder_in_place_and_elsewhere(rec):
    S, conv = torch.zeros(3, 1, D, D, dtype=BF), torch.zeros(3, 3, 3 * D)
    kda.kda_beam_reorder(1, 3, ints(3), S, conv, stream=0)
    other = torch.zeros_like(S), torch.zeros_like(conv)
    kda.kda_beam_reorder(1, 3, ints(3), S, conv, S_out=other[0], conv_out=other[1], stream=0)
    (_, a), (_, b) = rec.calls
    assert a[3] == a[5] and a[4] == a[6] and a[7] == 1
    assert b[5:7] == (other[0].data_ptr(), other[1].data_ptr())
    for wrong in (dict(rows=torch.zeros(3, dtype=torch.int64)), dict(rows=ints(2)), dict(S=S.transpose(2, 3)),
                  dict(S_out=torch.zeros(3, 1, D, D))):
        with pytest.raises(ValueError):
            kda.kda_beam_reorder(1, 3, wrong.pop("rows", ints(3)), wrong.pop("S", S), conv, stream=0, **wrong)
    assert len(rec.calls) == 2


def fork(**change):
    args = dict(rows=ints(3), kv_lens=ints(3), block_table=ints(3, 7), page_refs=ints(9), free_pages=ints(9), free_count=ints(1),
                new_table=ints(3, 7), new_lens=ints(3), copy_src=ints(3), copy_dst=ints(3), copy_rows=ints(3), info=ints(4))
    args.update(change)
    kda.kda_attn_fork(1, 3, **args, workspace=16, workspace_bytes=1 << 20, stream=0)


def test_fork_takes_tables_of_one_pitch(rec):
    fork()
    fork(block_table=ints(3, 20)[:, :7], new_table=ints(3, 20)[:, 5:12])
    fork(max_pages=7, block_table=ints(21), new_table=ints(21), free_capacity=4)
    assert [(a[5], a[8]) for _, a in rec.calls] == [(7, 9), (20, 9), (7, 4)]


@pytest.mark.parametrize("change", [
    dict(new_table=ints(3, 8)), dict(block_table=ints(7, 3).t(), new_table=ints(7, 3).t()), dict(rows=torch.zeros(3)[:2]),
    dict(rows=torch.zeros(3, dtype=torch.int64)), dict(kv_lens=ints(2)), dict(copy_src=ints(6)[::2]), dict(info=ints(3)),
    dict(new_lens=torch.zeros(3, dtype=torch.int64)), dict(page_refs=torch.zeros(9, dtype=torch.uint8)), dict(free_capacity=10)])
def test_fork_refuses_tensors(rec, change):
    with pytest.raises(ValueError):
        fork(**change)
    assert not rec.calls


def test_shared_decode_refuses_tensors(rec):
    q, o = torch.zeros(3, 4, D, dtype=BF), torch.zeros(3, 4, D, dtype=BF)

    def call(q=q, o=o, table=ints(3, 7), cu=ints(2), prefix=ints(1), **more):
        kda.kda_attn_decode_shared(1, 3, q, table, ints(3), 1, cu, prefix, o, 16, workspace_bytes=1 << 30, stream=0, **more)

    call()
    for wrong in (dict(q=torch.zeros(4, 3, D, dtype=BF).transpose(0, 1)), dict(o=torch.zeros(3, 4, 2 * D, dtype=BF)[..., ::2]),
                  dict(table=ints(7, 3).t()), dict(cu=ints(4)[::2]), dict(lse=torch.zeros(4, 3).t()),
                  dict(gate_logit=torch.zeros(4, 3, D).transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**wrong)
    assert len(rec.calls) == 1


# ---------------------------------------------------------------- the plain forms


def test_places():
    assert beam_ref.places([0, 1, 2, 3]) == [0, 1, 2, 3]
    assert beam_ref.places([2, 2, 2, 2]) == [2, 0, 1, 3]
    assert beam_ref.places([3, 1, 3, 1]) == [3, 1, 0, 2]


def test_fork_of_a_prompt():
    """One prompt of 20 tokens in pages of 16 to three beams, one of which ends."""
    table, refs, free = [[5, 6], [-1, -1], [-1, -1]], [0] * 8, [0, 1, 2, 3, 4, 7, -1, -1]
    new = [[-1, -1] for _ in range(3)]
    lens, copies, info = fork_ref.fork([0, 0, 0], [20, 0, 0], table, refs, free, 6, new, 16)
    assert lens == [20, 20, 20] and new == [[5, 6], [5, 7], [5, 4]] and info == [0, 2, 4, 0]
    assert copies == [(-1, -1, 0), (6, 7, 4), (6, 4, 4)] and refs[5] == 2
    last = [[-1, -1] for _ in range(3)]
    lens, copies, info = fork_ref.fork([0, 0, 2], lens, new, refs, free, 4, last, 16)
    # Beam 1 lets go of its copy, which beam 0's second child takes.
    assert last == [[5, 6], [5, 7], [5, 4]] and info == [1, 1, 4, 0] and copies[1] == (6, 7, 4) and refs[5] == 2
