"""The operators for several continuations at their largest numbers of requests, beams and continuations."""
import pytest
import torch

import kda_delta_rule_token_gb300 as kda
from test_attn_fork_gpu import Layer as Pages
from test_attn_gpu import D, DEV, Guard, Layer, i32, queries
from test_beam_gpu import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [2, 256, 257])
def test_fork_of_the_most_requests(width):
    """16384 requests of two pages, of every four of which the first goes on as all four."""
    B, page = 16384, 16
    layer = Pages(2 * B, page=page)
    order = torch.randperm(2 * B, generator=torch.Generator().manual_seed(width)).to(torch.int32).to(DEV)
    table = torch.full((B, width), 2 ** 30, dtype=torch.int32, device=DEV)
    table[:, :2] = order.view(B, 2)
    at = torch.arange(B, device=DEV)
    lens = (page + 1 + at % (page - 1)).to(torch.int32)
    rows = (at - at % 4).to(torch.int32)
    refs, free, new = torch.zeros(2 * B, dtype=torch.int32, device=DEV), torch.full((2 * B,), -1, dtype=torch.int32, device=DEV), torch.full_like(table, -1)
    out, info = [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(4)], i32([0] * 4)
    ws = torch.empty(kda.kda_attn_fork_workspace_bytes(layer.attn, B, width), dtype=torch.uint8, device=DEV)
    kda.kda_attn_fork(layer.attn, B, rows, lens, table, refs, free, i32([0]), new, *out, info, ws)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    ends = at % 4 > 0
    freed = torch.cat([table[ends, 0], table[ends, 1]])       # the first pages of all, then the second
    wants = int(ends.sum())
    taken = freed.flip(0)[:wants]
    assert info.tolist() == [2 * wants, wants, wants, 0]
    assert torch.equal(free[:wants], freed[:wants])
    want = table[rows.long(), :2].clone()
    want[ends, 1] = taken
    assert torch.equal(new[:, :2], want) and bool((new[:, 2:] == -1).all())
    assert torch.equal(out[0], lens[rows.long()])
    assert torch.equal(out[2][ends], taken) and torch.equal(out[1][ends], table[rows.long(), 1][ends])
    assert torch.equal(out[3][ends], (lens[rows.long()] % page)[ends]) and bool((out[1][~ends] == -1).all())
    held = torch.zeros(2 * B, dtype=torch.int32, device=DEV)
    held[table[~ends, 0].long()] = 3
    assert torch.equal(refs, held)
    layer.done()


@pytest.mark.parametrize("hq,hkv,e4m3", [(4, 1, False), (2, 2, True)])
@pytest.mark.parametrize("B,size", [(2048, 3), (2049, 1), (5000, 3), (5000, 40), (16384, 2)])
def test_shared_attention_of_many_requests(B, size, hq, hkv, e4m3):
    """Against the decode of the same requests; groups of `size`, some of them without keys or too short for their prefix."""
    page, prefix = 16, 32
    lens = [0 if b % 11 == 3 else 20 if b % 13 == 5 else prefix + 1 + b % 30 for b in range(B)]
    layer = Layer(hq, hkv, page, e4m3, seed=B + size)
    layer.fill(lens, width=max(4, (30 << 20) // (B * hkv * page * D * 2) + 1))
    cu = list(range(0, B, size)) + [B]
    table = layer.table
    for g, end in zip(cu, cu[1:]):   # the prefix's pages of the first request that has them are everybody's
        lead = next((b for b in range(g, end) if lens[b] >= prefix), None)
        for b in range(g, end) if lead is not None else ():
            if lens[b] >= prefix:
                layer.table_list[b][:2] = layer.table_list[lead][:2]
    table = i32(layer.table_list)
    q, kv = queries(layer, B), i32(lens)
    o, lse = [Guard((B, hq, D), torch.float32) for _ in range(2)], [Guard((B, hq), torch.float32) for _ in range(2)]
    ws = Guard((kda.kda_attn_shared_workspace_bytes(layer.attn, B),), torch.uint8, fill=0xFF)
    before = kda.kda_launch_count()
    kda.kda_attn_decode_shared(layer.attn, B, q, table, kv, len(cu) - 1, i32(cu), i32([prefix] * (len(cu) - 1)), o[0].t, ws.t, lse=lse[0].t)
    assert kda.kda_launch_count() - before == 4
    kda.kda_attn_decode(layer.attn, B, q, table, kv, o[1].t, layer.ws.t, lse=lse[1].t)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert all(t.intact() for t in (*o, *lse, ws))
    # Values below 8 (normal, 128 channels of few keys), weights of one bf16 part at most, both sums in fp32.
    assert float((o[0].t - o[1].t).abs().max()) <= 8 * (2.0 ** -8 + 2.0 ** -10)
    none = lse[1].t == -torch.inf
    assert torch.equal(none, lse[0].t == -torch.inf) and bool((o[0].t[none] == 0).all())
    assert float((lse[0].t - lse[1].t)[~none].abs().max()) <= 1e-4
    layer.done()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("G,K,V,num", [(1, 64, 64, 64), (5, 64, 5000, 64), (200, 64, 300, 64), (2, 64, 33000, 63), (3, 63, 9001, 64)])
def test_most_beams_and_continuations(G, K, V, num, bf16):
    x, scores = make(G, K, V, bf16, seed=V)
    run(x, scores, num, keep=num == K)
