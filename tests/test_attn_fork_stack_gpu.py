"""The stack of free pages behind a fork, from what a list of pages would hold."""
import random

import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from test_attn_fork_gpu import DEV, Layer, i32

pytestmark = pytest.mark.gpu


def stack_after(stack, freed, wants, room):
    """Pages that the copies get, in order, what the stack holds then, and how many pages are lost."""
    stack = stack + freed
    taken = [stack.pop() for _ in range(min(wants, len(stack)))]
    return taken, stack[:room], max(len(stack) - room, 0)


@pytest.mark.parametrize("width", [3, 300])   # in one launch, and in two
@pytest.mark.parametrize("have,room", [(0, 0), (0, 1), (2, 2), (2, 3), (1, 4), (2, 4), (2, 7), (3, 3)])
@pytest.mark.parametrize("ends,wants", [(1, 0), (1, 1), (1, 3), (2, 2), (3, 1), (3, 2), (2, 4), (3, 5), (3, 6)])
def test_stack_with_little_room(ends, wants, have, room, width):
    """`ends` requests of one page end, request 0 goes on `wants` times more: its copies take freed pages first, and a
    page is lost only if the stack has no room for it once they have theirs."""
    page, B = 16, 1 + max(ends, wants)
    layer = Layer(40, page=page)
    table = [[30, 31] + [-1] * (width - 2)] + [[10 + b] + [-1] * (width - 1) for b in range(1, B)]
    lens = [20] + [5 if b <= ends else 0 for b in range(1, B)]
    rows = [0] + [0 if b <= wants else -1 for b in range(1, B)]
    stack, freed = [4, 5, 6][:have], [10 + b for b in range(1, ends + 1)]
    taken, left, lost = stack_after(stack, freed, wants, room)
    free = torch.full((room + 16,), -5, dtype=torch.int32, device=DEV)
    free[:have] = i32(stack)
    refs, new = torch.zeros(40, dtype=torch.int32, device=DEV), torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    outs, info = [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(4)], i32([0] * 4)
    ws = torch.empty(kda.kda_attn_fork_workspace_bytes(layer.attn, B, width), dtype=torch.uint8, device=DEV)
    kda.kda_attn_fork(layer.attn, B, i32(rows), i32(lens), i32(table), refs, free, i32([have]), new, *outs, info, ws, free_capacity=room)
    status = kda.kda_attn_sync_status(layer.attn)
    assert info.tolist() == [ends, len(taken), len(left), wants - len(taken)]
    assert free[:len(left)].tolist() == left and bool((free[room:] == -5).all())
    assert status == (kda.KDA_ERR_INVALID_ARG if lost else kda.KDA_OK)
    assert outs[2][1:1 + len(taken)].tolist() == taken and new[1:1 + len(taken), 1].tolist() == taken
    assert refs.tolist() == [len(taken) if p == 30 else 0 for p in range(40)]
    layer.done()


@pytest.mark.parametrize("B,width", [(3, 2), (9, 40), (20, 250), (7, 256), (7, 257), (4, 1000)])
def test_count_carried_on_in_place(B, width):
    """free_count in info[2], where the call before left it: the same as with a count of its own, eager and captured."""
    page, rng = 16, random.Random(B * width)
    layer = Layer(B * width, page=page)
    order = list(range(B * width))
    rng.shuffle(order)
    lens0 = [rng.randint(1, width * page) for _ in range(B)]
    table0, at = torch.full((B, width), -1, dtype=torch.int32, device=DEV), 0
    for b, n in enumerate(lens0):
        need = -(-n // page)
        table0[b, :need] = i32(order[at:at + need])
        at += need
    steps = [i32([rng.randrange(B) for _ in range(B)]) for _ in range(5)] + [i32([-1] * B)]
    free0 = i32(order[at:] + [-1] * at)
    ws = torch.empty(kda.kda_attn_fork_workspace_bytes(layer.attn, B, width), dtype=torch.uint8, device=DEV)

    def walk(in_place):
        tables, lens = [table0.clone(), torch.full_like(table0, -1)], [i32(lens0), i32([0] * B)]
        refs, free, info = torch.zeros(B * width, dtype=torch.int32, device=DEV), free0.clone(), i32([0, 0, B * width - at, 0])
        copies = [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3)]

        def go():
            for i, rows in enumerate(steps):
                count = info[2:3] if in_place else info[2:3].clone()
                kda.kda_attn_fork(layer.attn, B, rows, lens[i % 2], tables[i % 2], refs, free, count, tables[1 - i % 2], lens[1 - i % 2], *copies, info, ws)
        return go, (*tables, *lens, refs, free, info, *copies)

    go, want = walk(False)
    go()
    assert want[6].tolist()[2] == B * width and kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    for _ in range(5):
        go, got = walk(True)
        go()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    go, got = walk(True)
    before = [t.clone() for t in got]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        for t, old in zip(got, before):
            t.copy_(old)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    layer.done()
