"""What the Python binding of the paged softmax-attention operators makes of
tensors' shapes and strides, on a recording stand-in for the library."""
import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from kda_delta_rule_token_gb300 import build

D = 128
BF = torch.bfloat16
BIG = 1 << 30


class Recorder:
    """Takes the place of the loaded library: notes the arguments, returns KDA_OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    build.build()
    kda.load()
    rec = Recorder()
    monkeypatch.setattr(kda, "load", lambda path=None: rec)
    return rec


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def heads(n, h, dtype=BF):
    return torch.zeros(n, h, D, dtype=dtype)


def decode(q=None, table=None, o=None, **more):
    q = heads(3, 4) if q is None else q
    table = ints(3, 7) if table is None else table
    kda.kda_attn_decode(1, 3, q, table, ints(3), torch.zeros_like(heads(3, 4)) if o is None else o, 16, workspace_bytes=BIG,
                        stream=0, **more)


def prefill(q=None, table=None, o=None, **more):
    q = heads(3, 4) if q is None else q
    table = ints(3, 7) if table is None else table
    kda.kda_attn_prefill(1, 3, 3, ints(4), q, table, ints(3), heads(3, 4) if o is None else o, 16, workspace_bytes=BIG, stream=0,
                         **more)


def plan(table):
    kda.kda_attn_plan(1, table.shape[0] if table.dim() == 2 else 1, 1, ints(1), ints(1), ints(4), ints(1), table, ints(2), ints(1),
                      ints(1), torch.zeros(1, dtype=torch.int64), ints(4), stream=0)


BAD_TABLES = {
    "transposed": lambda: ints(7, 3).t(),
    "every other": lambda: ints(3, 14)[:, ::2],
    "one-dimensional": lambda: ints(7),
    "three-dimensional": lambda: ints(3, 7, 1),
    "one row for all": lambda: ints(1, 7).expand(3, 7),
}


@pytest.mark.parametrize("table", BAD_TABLES)
@pytest.mark.parametrize("call", [decode, prefill, plan])
def test_tables_that_are_not_rows(lib, call, table):
    with pytest.raises(ValueError, match="block_table"):
        call(table=BAD_TABLES[table]())
    assert not lib.calls


@pytest.mark.parametrize("table,pitch", [
    (lambda: ints(3, 7), 7), (lambda: ints(3, 20)[:, 5:12], 20), (lambda: ints(9, 7)[::3], 21),
    (lambda: ints(1, 7), 7), (lambda: ints(7, 1).t(), 7), (lambda: ints(2, 9)[:1, :4], 9), (lambda: ints(3, 1), 1)])
@pytest.mark.parametrize("call", [decode, prefill, plan])
def test_pitch_of_a_table(lib, call, table, pitch):
    call(table=table())
    (name, args), = lib.calls
    assert args[9 if name == "kda_attn_plan" else 4 if name == "kda_attn_decode" else 6] == pitch


def test_a_pitch_that_is_given_stands(lib):
    decode(table=ints(21), max_pages=7)
    assert lib.calls[0][1][4] == 7


LOOSE = {
    "a slice of a fused projection": lambda: torch.zeros(3, 8, D, dtype=BF)[:, :4],
    "transposed heads": lambda: torch.zeros(4, 3, D, dtype=BF).transpose(0, 1),
    "every other channel": lambda: torch.zeros(3, 4, 2 * D, dtype=BF)[..., ::2],
    "one row for all": lambda: torch.zeros(1, 4, D, dtype=BF).expand(3, 4, D),
}


@pytest.mark.parametrize("loose", LOOSE)
@pytest.mark.parametrize("call", [decode, prefill])
@pytest.mark.parametrize("arg", ["q", "o", "gate_logit", "lse"])
def test_tensors_that_are_not_dense(lib, call, arg, loose):
    with pytest.raises(ValueError, match=arg):
        call(**{arg: LOOSE[loose]()})
    assert not lib.calls


def test_dense_tensors_and_addresses_pass(lib):
    whole = heads(9, 4)
    for call in (decode, prefill):
        call(q=whole[3:6], o=whole[6:], lse=torch.zeros(3, 4), gate_logit=heads(3, 4, torch.float32))
        call(q=4096, o=8192, o_f32=False, gate_logit=None)
        call(q=torch.zeros(1, 8, D, dtype=BF)[:, :4], o=heads(1, 4))       # one token: dense
    assert len(lib.calls) == 6


def append(q, k, v, out, n=None, **more):
    kda.kda_attn_append(1, q.shape[0] if n is None else n, q, k, v, ints(4), torch.zeros(4, dtype=torch.int64), out, stream=0, **more)


def strides(lib):
    args = lib.calls[-1][1]
    return args[3], args[5], args[7]


def test_token_strides(lib):
    fused = torch.zeros(5, 8 * D + 24, dtype=BF)
    q, k, v = (t.unflatten(1, (-1, D)) for t in fused[:, :-24].split([4 * D, 2 * D, 2 * D], 1))
    append(q, k, v, heads(5, 4))
    assert strides(lib) == (8 * D + 24,) * 3
    # One token: how far the next one would be means nothing.
    q, k = torch.zeros(4, 1, D, dtype=BF).transpose(0, 1), torch.zeros(1, 2, D, dtype=BF).as_strided((1, 2, D), (8, D, 1))
    append(q, k, heads(1, 2), heads(1, 4))
    assert strides(lib) == (4 * D, 2 * D, 2 * D)
    # One head: nor does how far the next head would be.
    one = torch.zeros(5, 3 * D, dtype=BF)
    append(*(t.unsqueeze(1) for t in one.split(D, 1)), heads(5, 1))
    assert strides(lib) == (3 * D,) * 3
    append(heads(5, 4), heads(5, 2), heads(5, 2), heads(5, 4), q_stride=1024, v_stride=2048)
    assert strides(lib) == (1024, 2 * D, 2048)


def test_append_refuses_a_result_that_is_not_dense(lib):
    fused = torch.zeros(5, 8, D, dtype=BF)
    with pytest.raises(ValueError, match="q_out"):
        append(heads(5, 4), heads(5, 2), heads(5, 2), fused[:, :4])
    assert not lib.calls
