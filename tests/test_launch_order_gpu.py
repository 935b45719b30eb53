"""The operators for several continuations start while what is before them in the stream still ends: what
that writes is what they read, behind kernels, copies and other streams, eager and captured."""
import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from test_attn_gpu import BF, D, DEV, Layer, i32, queries
from test_attn_shared_gpu import build
from test_beam_gpu import Ctx, make

pytestmark = pytest.mark.gpu


class Case:
    """`pairs`: (tensor that the call reads or changes, what it is to hold); `before`: what it held."""

    def __init__(self, pairs, call, outs, done):
        self.pairs, self.call, self.outs, self.done = pairs, call, outs, done
        self.before = [live.clone() for live, _ in pairs]

    def reset(self):
        for (live, _), old in zip(self.pairs, self.before):
            live.copy_(old)
        for out in self.outs:
            out.zero_()

    def write(self, how):
        for live, value in self.pairs:
            if how == "copies":
                live.copy_(value)
            else:
                torch.maximum(value, value, out=live)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.outs]


def select():
    x, scores = make(9, 4, 20000, seed=1)
    y, _ = make(9, 4, 20000, seed=2)
    ctx = Ctx()
    ws = torch.empty(kda.kda_beam_select_workspace_bytes(ctx.ctx, 9, 4, 20000, 4), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(9, 4, dtype=t, device=DEV) for t in (torch.float32, torch.int32, torch.int32)]
    return Case([(x, y)], lambda: kda.kda_beam_select(ctx.ctx, 9, 4, x, scores, 4, *outs, ws), outs, lambda: kda.kda_destroy(ctx.ctx))


def reorder():
    ctx, B = Ctx(2), 40
    S, conv = torch.randn(B, 2, D, D, device=DEV), torch.randn(B, 3, 6 * D, device=DEV)
    S_out, conv_out = torch.zeros_like(S), torch.zeros_like(conv)
    rows, final = i32(list(range(B))), i32([b // 3 for b in range(B)])
    return Case([(S, torch.randn_like(S)), (conv, torch.randn_like(conv)), (rows, final)],
                lambda: kda.kda_beam_reorder(ctx.ctx, B, rows, S, conv, S_out=S_out, conv_out=conv_out), [S_out, conv_out],
                lambda: kda.kda_destroy(ctx.ctx))


def fork():
    layer, B, width = Layer(2, 1, 16), 24, 40
    lens = [20 * b % 300 for b in range(B)]
    layer.fill(lens, width=width)
    free = i32([0] * 256)
    refs, n = torch.zeros(layer.pages, dtype=torch.int32, device=DEV), i32([0])
    used = {p for row, k in zip(layer.table_list, lens) for p in row[:-(-k // 16)]}
    spare = [p for p in range(layer.pages) if p not in used]
    rows, kv = i32(list(range(B))), i32(lens)
    new, out = torch.zeros_like(layer.table), [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(4)]
    info = i32([0] * 4)
    ws = torch.empty(kda.kda_attn_fork_workspace_bytes(layer.attn, B, width), dtype=torch.uint8, device=DEV)
    return Case([(rows, i32([b // 2 for b in range(B)])), (refs, refs.clone()), (free, i32(spare + [0] * (256 - len(spare)))),
                 (n, i32([len(spare)]))],
                lambda: kda.kda_attn_fork(layer.attn, B, rows, kv, layer.table, refs, free, n, new, *out, info, ws),
                [new, *out, info], layer.done)


def copy_pages():
    layer = Layer(4, 2, 32)
    layer.fill([32] * 12, spare=12)
    src, dst, rows = i32([-1] * 12), i32([0] * 12), i32([0] * 12)
    order = torch.randperm(layer.pages, generator=torch.Generator().manual_seed(1)).tolist()
    caches = [layer.k, layer.v]
    pairs = [(src, i32(order[:12])), (dst, i32(order[12:24])), (rows, i32([1 + 2 * i for i in range(12)]))]
    case = Case(pairs + [(c, c.clone()) for c in caches], lambda: kda.kda_attn_copy_pages(layer.attn, 12, src, dst, rows), caches, layer.done)
    return case


def shared(narrow, n):
    def make_case():
        layer, lens = build([(n, 300), (3, 50)], 9, 8, 2, 16, False, narrow=narrow)
        B = len(lens)
        q, o = queries(layer, B), torch.zeros(B, 8, D, dtype=BF, device=DEV)
        ws = torch.empty(kda.kda_attn_shared_workspace_bytes(layer.attn, B), dtype=torch.uint8, device=DEV)
        kv, cu, prefix = i32([0] * B), i32([0, 0, 0]), i32([0, 0])
        return Case([(q, queries(layer, B, 2.0)), (kv, i32(lens)), (cu, i32([0, n, B])), (prefix, i32([300, 50]))],
                    lambda: kda.kda_attn_decode_shared(layer.attn, B, q, layer.table, kv, 2, cu, prefix, o, ws), [o], layer.done)
    return make_case


CASES = {"select": select, "reorder": reorder, "fork": fork, "copy_pages": copy_pages, "shared few": shared(False, 5),
         "shared many": shared(False, 40), "shared narrow": shared(True, 5)}


@pytest.mark.parametrize("how", ["kernels", "copies"])
@pytest.mark.parametrize("name", CASES)
def test_reads_what_is_written_before(name, how):
    case = CASES[name]()
    case.reset()
    case.write(how)
    torch.cuda.synchronize()
    case.call()
    want = case.results()
    side, event = torch.cuda.Stream(), torch.cuda.Event()

    def same():
        return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(case.results(), want))

    def run(streams):
        torch.cuda._sleep(2_000_000)
        if streams == 1:
            case.write(how)
        else:   # written by another stream, while this one is busy with something else
            event.record()
            with torch.cuda.stream(side):
                side.wait_event(event)
                torch.cuda._sleep(2_000_000)
                case.write(how)
                event.record()
            torch.cuda._sleep(200_000)
            torch.cuda.current_stream().wait_event(event)
        case.call()

    for streams in (1, 2):
        for _ in range(2):
            case.reset()
            run(streams)
            assert same(), ("eager", streams)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        case.reset()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            run(streams)
        for _ in range(3):
            case.reset()
            graph.replay()
            assert same(), ("captured", streams)
        del graph
    case.done()


def test_calls_in_a_row():
    """Each call reads what the one before it wrote: a step of a search, many times over."""
    ctx, G, K, V, B = Ctx(2), 3, 4, 5000, 12
    gen = torch.Generator(device=DEV).manual_seed(5)
    xs = [torch.randn(B, V, generator=gen, device=DEV) for _ in range(6)]
    S, conv = torch.randn(B, 2, D, D, generator=gen, device=DEV), torch.randn(B, 3, 6 * D, generator=gen, device=DEV)
    ws = torch.empty(kda.kda_beam_select_workspace_bytes(ctx.ctx, G, K, V, K), dtype=torch.uint8, device=DEV)

    def search(sync):
        states, scores = [(S.clone(), conv.clone()), (torch.empty_like(S), torch.empty_like(conv))], torch.zeros(G, K, device=DEV)
        for x in xs * 4:
            out = [torch.empty(G, K, dtype=t, device=DEV) for t in (torch.float32, torch.int32, torch.int32)]
            kda.kda_beam_select(ctx.ctx, G, K, x, scores, K, *out, ws)
            if sync:
                torch.cuda.synchronize()
            kda.kda_beam_reorder(ctx.ctx, B, out[2].view(-1), *states[0], S_out=states[1][0], conv_out=states[1][1])
            if sync:
                torch.cuda.synchronize()
            states.reverse()
            scores = out[0]
        return scores, *states[0]

    want = search(True)
    for _ in range(3):
        for a, b in zip(search(False), want):
            assert torch.equal(a, b)
    kda.kda_destroy(ctx.ctx)
