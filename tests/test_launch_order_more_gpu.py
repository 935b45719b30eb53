"""More of what the operators for several continuations read behind work that still runs: reordering in place, forks of
tables too wide for one launch, keys, values and block tables; and which launches the shared attention makes."""
import random

import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from test_attn_gpu import BF, D, DEV, Layer, i32, queries
from test_attn_shared_gpu import attend, build, verify
from test_beam_gpu import Ctx
from test_launch_order_gpu import Case

pytestmark = pytest.mark.gpu


def reorder_in_place():
    ctx, B = Ctx(2), 40
    S, conv, rows = torch.zeros(B, 2, D, D, device=DEV), torch.zeros(B, 3, 6 * D, device=DEV), i32(list(range(B)))
    final = [b - b % 3 if b % 5 else b for b in range(B)]
    final = i32([r if final[r] == r else b for b, r in enumerate(final)])
    return Case([(S, torch.randn_like(S)), (conv, torch.randn_like(conv)), (rows, final)],
                lambda: kda.kda_beam_reorder(ctx.ctx, B, rows, S, conv), [S, conv], lambda: kda.kda_destroy(ctx.ctx))


def fork(width):
    def make_case():
        page, B = 16, 12
        layer, rng = Layer(2, 1, page), random.Random(width)
        lens = [rng.randint(0, width * page) for _ in range(B)]
        layer.fill(lens, width=width)
        used = {p for row, n in zip(layer.table_list, lens) for p in row[:-(-n // page)]}
        spare = [p for p in range(layer.pages) if p not in used]
        free, refs = i32([0] * layer.pages), i32([3] * layer.pages)
        n, kv, rows = i32([0]), i32([0] * B), i32(list(range(B)))
        good = layer.table.clone()
        layer.table.zero_()
        new, out, info = torch.zeros_like(good), [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(4)], i32([0] * 4)
        ws = torch.empty(kda.kda_attn_fork_workspace_bytes(layer.attn, B, width), dtype=torch.uint8, device=DEV)
        return Case([(rows, i32([b // 2 for b in range(B)])), (refs, torch.zeros_like(refs)), (layer.table, good), (kv, i32(lens)),
                     (free, i32(spare + [0] * (layer.pages - len(spare)))), (n, i32([len(spare)]))],
                    lambda: kda.kda_attn_fork(layer.attn, B, rows, kv, layer.table, refs, free, n, new, *out, info, ws),
                    [new, *out, info, refs, free], layer.done)
    return make_case


def shared(narrow, n, e4m3):
    """Keys, values and the table come late: what kda_attn_append and kda_attn_fork write just before the call."""
    def make_case():
        layer, lens = build([(n, 300), (3, 50)], 9, 8, 2, 16, e4m3, narrow=narrow)
        B = len(lens)
        q, o = queries(layer, B), torch.zeros(B, 8, D, dtype=BF, device=DEV)
        ws = torch.empty(kda.kda_attn_shared_workspace_bytes(layer.attn, B), dtype=torch.uint8, device=DEV)
        late = [c.view(torch.int16) if not e4m3 else c.view(torch.uint8) for c in (layer.k, layer.v)] + [layer.table]
        pairs = [(t, t.clone()) for t in late]
        for t in late:
            t.zero_()
        args = (i32(lens), 2, i32([0, n, B]), i32([300, 50]))
        return Case(pairs, lambda: kda.kda_attn_decode_shared(layer.attn, B, q, layer.table, *args, o, ws), [o], layer.done)
    return make_case


CASES = {"reorder in place": reorder_in_place, "fork 40": fork(40), "fork 256": fork(256), "fork 300": fork(300)}
CASES.update({f"shared {'narrow' if w else 'wide'} {n} {'e4m3' if e else 'bf16'}": shared(w, n, e)
              for w, n in ((True, 5), (False, 5), (False, 40)) for e in (False, True)})


@pytest.mark.parametrize("how", ["kernels", "copies"])
@pytest.mark.parametrize("name", CASES)
def test_reads_what_is_written_before(name, how):
    case = CASES[name]()
    case.reset()
    case.write(how)
    torch.cuda.synchronize()
    case.call()
    want = case.results()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()

    def run():
        torch.cuda._sleep(2_000_000)
        case.write(how)
        case.call()

    def same():
        return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(case.results(), want))

    for _ in range(3):
        case.reset()
        run()
        assert same(), "eager"
    case.reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for _ in range(3):
        case.reset()
        graph.replay()
        assert same(), "captured"
    del graph
    case.done()


def launches(layer, q, lens):
    before = kda.kda_launch_count()
    attend(layer, q, lens)
    return kda.kda_launch_count() - before


@pytest.mark.parametrize("groups", [[(2, 256)], [(4, 517)], [(2, 15), (3, 16), (4, 17), (2, 128), (5, 300)], [(33, 129)], [(30, 40), (3, 200)]],
                         ids=lambda g: "_".join(f"{n}x{p}" for n, p in g))
@pytest.mark.parametrize("hq,hkv,page,e4m3", [(8, 2, 16, False), (8, 2, 32, True)])
def test_narrow_tables_take_two_launches(groups, hq, hkv, page, e4m3):
    layer, lens = build(groups, 1, hq, hkv, page, e4m3, narrow=True)
    q = queries(layer, len(lens))
    assert launches(layer, q, lens) == 2
    verify(layer, q, lens)
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,many", [(8, 0), (9, 1)])
def test_tables_at_the_limit(n, many, e4m3):
    """Tables for 24 MB of keys and values take two launches, wider ones three, or four where a call can have more than
    32 rows per key head."""
    hkv, page = 2, 16
    limit = (24 << 20) // (n * hkv * page * D * (2 if e4m3 else 4))
    for width, want in ((limit, 2), (limit + 1, 3 + many)):
        layer, lens = Layer(8, hkv, page, e4m3), [200 + b for b in range(n)]
        layer.fill(lens, width=width)
        layer.groups = [(0, n, 0)]
        assert launches(layer, queries(layer, n), lens) == want
        layer.done()
