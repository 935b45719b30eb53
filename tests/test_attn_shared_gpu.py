"""Attention of requests that share a prefix on a GB300, against the plain 64-bit form, which knows
nothing of sharing."""
import math

import pytest
import torch

import attn_ref as ref
import kda_delta_rule_token_gb300 as kda
from test_attn_gpu import BF, D, DEV, Guard, Layer, check, i32, queries

pytestmark = pytest.mark.gpu


def share(layer, groups, lens):
    """fill()'s requests with the whole pages of each group's prefix one request's, the page that a prefix
    ends in a copy.  groups: (first, end, prefix).  The pages that nobody has any more are NaN."""
    page = layer.page
    caches = [c.view(torch.uint8) if layer.e4m3 else c for c in (layer.k, layer.v)]
    for first, end, prefix in groups:
        long = [b for b in range(first, end) if lens[b] >= prefix]
        if not long or prefix <= 0:
            continue
        lead = layer.table_list[long[0]]
        for b in range(first, end):
            row = layer.table_list[b]
            for j in range(-(-min(prefix, lens[b]) // page)):
                if b == long[0]:
                    continue
                rows = min(page, prefix - j * page)
                if rows == page and (j + 1) * page <= lens[b]:
                    for c in caches:
                        c[row[j]] = 0x7F if layer.e4m3 else math.nan
                    row[j] = lead[j]
                else:
                    for c in caches:
                        c[row[j], :, :min(rows, lens[b] - j * page)] = c[lead[j], :, :min(rows, lens[b] - j * page)]
    layer.table = i32(layer.table_list)
    layer.groups = groups


def attend(layer, q, lens, groups=None, gate=None, f32=False, ws=None, stream=None, want_lse=True):
    B = len(lens)
    o, lse = Guard((B, layer.hq, D), torch.float32 if f32 else BF), Guard((B, layer.hq), torch.float32)
    ws = ws or Guard((kda.kda_attn_shared_workspace_bytes(layer.attn, B),), torch.uint8, fill=0xFF)
    groups = layer.groups if groups is None else groups
    cu = [g[0] for g in groups] + [groups[-1][1]] if groups else [0]
    kda.kda_attn_decode_shared(layer.attn, B, q, layer.table, i32(lens), len(groups), i32(cu), i32([g[2] for g in groups]), o.t,
                               ws.t, gate_logit=gate, lse=lse.t if want_lse else None, stream=stream)
    assert o.intact() and lse.intact() and ws.intact()
    return o.t, lse.t


def verify(layer, q, lens, status=kda.KDA_OK, **more):
    o, lse = attend(layer, q, lens, **more)
    assert kda.kda_attn_sync_status(layer.attn) == status
    gate, f32 = more.get("gate"), more.get("f32", False)
    want, wl, bound, lb = ref.attend(q, layer.k, layer.v, layer.table_list, lens, None, layer.page, D ** -0.5, layer.ks, layer.vs, gate)
    # The two results meet with weights that are off by what their lse are, by the two exponentials and the quotient.
    values = layer.v.float()
    if layer.vs is not None:
        values = values * layer.vs.view(1, -1, 1, 1)
    most = values.nan_to_num(0.0, 0.0, 0.0).abs().max()
    weights = 2 * lb + 4 * ref.U32 * wl.abs().nan_to_num(posinf=0.0) + 2.0 ** -20
    bound = bound + weights[..., None] * most
    if not f32:
        bound = bound * (1 + ref.UBF) + ref.UBF * want.abs()
    check(o, want, bound, "o")
    none = wl == -math.inf
    assert torch.equal(lse == -math.inf, none) and bool((o[none] == 0).all())
    check(lse.masked_fill(none, 0), wl.masked_fill(none, 0), (2 * lb + weights).masked_fill(none, 1), "lse")


def wide(layer, B):
    """Columns of a block table that is too wide for the call to pass over its groups."""
    return (30 << 20) // (B * layer.hkv * layer.page * D * (2 if layer.e4m3 else 4)) + 1


def build(groups, own, hq, hkv, page, e4m3, seed=0, ragged=True, narrow=False):
    """groups: (requests, prefix); lens = prefix + own, different from request to request."""
    lens, spans, at = [], [], 0
    for i, (n, prefix) in enumerate(groups):
        lens += [prefix + (own + 7 * b + i if ragged else own) for b in range(n)]
        spans.append((at, at + n, prefix))
        at += n
    layer = Layer(hq, hkv, page, e4m3, seed=seed)
    fill(layer, lens, narrow=narrow)
    share(layer, spans, lens)
    return layer, lens


def fill(layer, lens, narrow=False, **more):
    least = max(1, -(-max(lens) // layer.page))
    layer.fill(lens, width=least if narrow else max(least, wide(layer, len(lens))), **more)


HEADS = [(1, 1, 16, False), (8, 2, 16, False), (32, 8, 64, False), (5, 1, 32, False), (16, 1, 128, False), (40, 1, 16, False),
         (128, 1, 16, False), (1, 1, 16, True), (8, 2, 32, True), (12, 4, 16, True), (16, 1, 64, True), (33, 1, 128, True)]
GROUPS = [
    [(1, 100)],                                  # nothing to share
    [(2, 256)], [(3, 1)], [(4, 517)],
    [(2, 15), (3, 16), (4, 17), (2, 128), (5, 300)],
    [(33, 129)], [(64, 1000)], [(130, 640)],
    [(1, 40), (40, 200), (2, 3000), (8, 64)],
]


WIDE = {40, 128, 33, 32}   # heads that the plain form takes long for: the last and a small case


@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: "_".join(f"{n}x{p}" for n, p in g))
@pytest.mark.parametrize("hq,hkv,page,e4m3", HEADS)
def test_groups(groups, hq, hkv, page, e4m3):
    if hq in WIDE and groups not in (GROUPS[3], GROUPS[-1]):
        return
    layer, lens = build(groups, 1, hq, hkv, page, e4m3, seed=hq + page)
    verify(layer, queries(layer, len(lens)), lens)
    layer.done()


@pytest.mark.parametrize("groups", GROUPS[1:], ids=lambda g: "_".join(f"{n}x{p}" for n, p in g))
@pytest.mark.parametrize("hq,hkv,page,e4m3", [(8, 2, 16, False), (8, 2, 32, True)])
def test_narrow_tables(groups, hq, hkv, page, e4m3):
    """Calls that are small enough to pass over their groups."""
    layer, lens = build(groups, 1, hq, hkv, page, e4m3, narrow=True)
    verify(layer, queries(layer, len(lens)), lens)
    layer.groups = [(0, 2, 5), (1 << 20, 1, 5)]
    o, _ = attend(layer, queries(layer, len(lens)), lens)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
    layer.done()


@pytest.mark.parametrize("hq,hkv,page,e4m3", [(8, 2, 16, False), (16, 1, 64, False), (8, 2, 32, True), (64, 4, 16, True)])
@pytest.mark.parametrize("n,prefix", [(2, 30000), (9, 20011), (40, 9000)])
def test_long_prefixes(n, prefix, hq, hkv, page, e4m3):
    layer, lens = build([(n, prefix)], 3, hq, hkv, page, e4m3)
    verify(layer, queries(layer, n), lens)
    layer.done()


@pytest.mark.parametrize("hq,hkv,page,e4m3", [(8, 2, 16, False), (16, 1, 128, True)])
@pytest.mark.parametrize("n", [4, 40])
def test_requests_without_keys_and_short_ones(n, hq, hkv, page, e4m3):
    """Some have none of the prefix, the first among them, some a part of it, some exactly it."""
    prefix = 512
    lens = [prefix + 3 * b for b in range(n)] * 2
    lens[0], lens[1], lens[2] = 0, prefix - 1, prefix
    lens[n], lens[n + 1], lens[n + 3] = 17, prefix, 1
    layer = Layer(hq, hkv, page, e4m3)
    fill(layer, lens)
    share(layer, [(0, n, prefix), (n, 2 * n, prefix)], lens)
    verify(layer, queries(layer, 2 * n), lens)
    layer.done()


@pytest.mark.parametrize("n", [4, 40])
def test_groups_of_one_long_request(n):
    """All but one short: nothing is shared; then no request has keys."""
    prefix = 512
    lens = [prefix - 1] * n + [prefix + 9] + [0] * (n - 1)
    layer = Layer(8, 2, 16)
    fill(layer, lens)
    share(layer, [(0, n, prefix), (n, 2 * n, prefix)], lens)
    verify(layer, queries(layer, 2 * n), lens)
    verify(layer, queries(layer, 2 * n), [0] * (2 * n))
    layer.done()


@pytest.mark.parametrize("what", ["none", "null", "gaps", "empty", "zero", "negative", "beyond"])
def test_what_groups_may_say(what):
    layer, lens = build([(3, 200), (5, 333), (40, 128)], 5, 8, 2, 16, False)
    q = queries(layer, len(lens))
    if what == "null":
        o = torch.empty(len(lens), 8, D, dtype=BF, device=DEV)
        ws = torch.empty(kda.kda_attn_shared_workspace_bytes(layer.attn, len(lens)), dtype=torch.uint8, device=DEV)
        kda.kda_attn_decode_shared(layer.attn, len(lens), q, layer.table, i32(lens), 0, None, None, o, ws)
        plain = torch.empty_like(o)
        kda.kda_attn_decode(layer.attn, len(lens), q, layer.table, i32(lens), plain, layer.ws.t)
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
        check(o, plain.double(), 2 * ref.UBF * plain.double().abs() + 1e-4, "o")
        return layer.done()
    layer.groups = {
        "none": [], "gaps": [(1, 3, 200), (3, 8, 333)], "empty": [(0, 3, 200), (3, 3, 500), (3, 8, 333), (8, 48, 100)],
        "zero": [(0, 3, 0), (3, 8, 333), (8, 48, 15)], "negative": [(0, 3, -7), (3, 8, 333), (8, 48, -2 ** 31)],
        "beyond": [(0, 3, 2 ** 31 - 1), (3, 8, 333), (8, 48, 10 ** 6)]}[what]
    verify(layer, q, lens)
    layer.done()


@pytest.mark.parametrize("cu", [[0, 8, 3, 48], [-1, 3, 8, 48], [0, 3, 8, 49], [2 ** 31 - 1, 3, 8, 48], [0, -2 ** 31, 8, 48]])
def test_offsets_that_are_not_ascending(cu):
    """Reported, and the results are the requests' own."""
    layer, lens = build([(3, 200), (5, 333), (40, 128)], 5, 8, 2, 16, False)
    layer.groups = [(a, b, 128) for a, b in zip(cu, cu[1:])]
    verify(layer, queries(layer, len(lens)), lens, status=kda.KDA_ERR_INVALID_ARG)
    layer.done()


@pytest.mark.parametrize("cu,status", [([0, 1], kda.KDA_OK), ([0, 2], kda.KDA_ERR_INVALID_ARG), ([-1, 1], kda.KDA_ERR_INVALID_ARG)])
def test_offsets_of_a_call_of_one_cta(cu, status):
    layer = Layer(1, 1, 16)
    fill(layer, [10], narrow=True)
    layer.groups = [(cu[0], cu[1], 5)]
    verify(layer, queries(layer, 1), [10], status=status)
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n", [4, 70])
def test_gate(n, f32, e4m3):
    layer, lens = build([(n, 400), (2, 100)], 1, 24, 3, 32, e4m3)
    lens[1] = 0
    gate = torch.randn(len(lens), 24, D, generator=layer.g, device=DEV) * 4
    gate[1] = math.nan       # of a row without keys: not read
    verify(layer, queries(layer, len(lens)), lens, gate=gate, f32=f32)
    attend(layer, queries(layer, len(lens)), lens, want_lse=False)
    layer.done()


@pytest.mark.parametrize("sigma,qs", [(1e-30, 1e-30), (1.0, 60.0), (30.0, 30.0), (1e4, 1e-4)])
@pytest.mark.parametrize("n", [4, 40])
def test_value_ranges(n, sigma, qs):
    lens = [640 + 5 * b for b in range(n)]
    layer = Layer(8, 2, 16)
    fill(layer, lens, sigma=sigma)
    share(layer, [(0, n, 600)], lens)
    verify(layer, queries(layer, n, qs), lens)
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [4, 40])
def test_nan_and_infinity(n, e4m3):
    """What a row sees shows, what it does not see has no effect."""
    page, prefix = 32, 256
    lens = [prefix + 20 + b for b in range(n)] + [200, 300]
    layer = Layer(8, 2, page, e4m3)
    fill(layer, lens)
    share(layer, [(0, n + 2, prefix)], lens)
    q = queries(layer, n + 2)
    clean, _ = attend(layer, q, lens)

    def put(cache, b, key, head, channel):
        c = cache.view(torch.uint8) if e4m3 else cache
        c[layer.table_list[b][key // page], head, key % page, channel] = 0x7F if e4m3 else math.nan

    # A value in the prefix, key 250, head 1: all rows of head 1 but the short request's, channel 5.
    put(layer.v, 3, 250, 1, 5)
    o, lse = attend(layer, q, lens)
    want = torch.zeros_like(clean, dtype=torch.bool)
    want[:, 4:, 5] = True
    want[n] = False
    assert torch.equal(o.isnan(), want) and not lse.isnan().any()
    # A key of request 1's own: its rows of head 0, all channels.
    put(layer.k, 1, prefix + 20, 0, 0)
    o, lse = attend(layer, q, lens)
    want[1, :4] = True
    assert torch.equal(o.isnan(), want)
    assert torch.equal(lse.isnan().nonzero()[:, 0].unique(), torch.tensor([1], device=DEV)) and int(lse.isnan().sum()) == 4
    # A key of the prefix that the short request does not reach: every long request's.
    put(layer.k, 0, 250, 0, 127)
    o, lse = attend(layer, q, lens)
    seen = torch.ones(n + 2, dtype=torch.bool, device=DEV)
    seen[n] = False
    assert bool(lse[:, :4].isnan().all(1)[seen].all()) and not o[n].isnan().any()
    assert torch.equal(o[n].float(), clean[n].float())
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,prefix", [(4, 217), (40, 217), (40, 16), (40, 400)])
def test_own_keys_behind_a_prefix_do_not_reach_the_others(n, prefix, e4m3):
    """The request whose table row names the prefix's pages has NaN in all keys and values behind it."""
    page = 16
    lens = [prefix + 30 + b for b in range(n)]
    layer = Layer(8, 2, page, e4m3)
    fill(layer, lens)
    share(layer, [(0, n, prefix)], lens)
    q = queries(layer, n)
    clean, cl = attend(layer, q, lens)
    for c in (layer.k, layer.v):
        c = c.view(torch.uint8) if e4m3 else c
        for key in range(prefix, -(-lens[0] // page) * page):
            c[layer.table_list[0][key // page], :, key % page] = 0x7F if e4m3 else math.nan
    o, lse = attend(layer, q, lens)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert bool(o[0].isnan().all()) and bool(lse[0].isnan().all())
    assert torch.equal(o[1:].view(torch.int16), clean[1:].view(torch.int16)) and torch.equal(lse[1:], cl[1:])
    layer.done()


def test_two_calls_at_once():
    """Two contexts, workspaces and streams."""
    made, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed, e4m3 in ((3, False), (4, True)):
        layer, lens = build([(40, 900), (5, 300)], 9, 16, 2, 16, e4m3, seed=seed)
        q = queries(layer, 45)
        want, _ = attend(layer, q, lens)
        ws = torch.empty(kda.kda_attn_shared_workspace_bytes(layer.attn, 45), dtype=torch.uint8, device=DEV)
        made.append((layer, q, (i32(lens), 2, i32([0, 40, 45]), i32([900, 300])), want, torch.zeros_like(want), ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for (layer, q, args, _, o, ws), s in zip(made, streams):
            kda.kda_attn_decode_shared(layer.attn, 45, q, layer.table, *args, o, ws, stream=s)
    torch.cuda.synchronize()
    for layer, _, _, want, o, _ in made:
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))
        layer.done()


@pytest.mark.parametrize("n", [4, 40])
def test_pages_outside_the_cache(n):
    layer, lens = build([(n, 300)], 40, 8, 2, 16, False)
    good = layer.table.clone()
    for b, j in ((0, 3), (n - 1, 20)):
        for bad in (-1, layer.pages, 2 ** 31 - 1, -2 ** 31):
            layer.table = good.clone()
            layer.table[b, j] = bad
            o, _ = attend(layer, queries(layer, n), lens)
            assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
            assert bool(torch.isfinite(o).all())
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cuts,prefix,hq,hkv", [([256], 4000, 64, 4), ([64, 128, 192, 256], 2000, 32, 8), ([8] * 32, 1000, 32, 8)])
def test_large_batches_against_decode(cuts, prefix, hq, hkv, e4m3):
    if len(cuts) == 32:
        cuts = list(range(8, 257, 8))
    spans = [(a, b, prefix - 10 * i) for i, (a, b) in enumerate(zip([0] + cuts, cuts))]
    lens = []
    for a, b, p in spans:
        lens += [p + 5 + 3 * (r % 50) for r in range(a, b)]
    layer = Layer(hq, hkv, 32, e4m3)
    fill(layer, lens)
    share(layer, spans, lens)
    q = queries(layer, 256)
    o, lse = attend(layer, q, lens, f32=True)
    plain, pl = Guard((256, hq, D), torch.float32), Guard((256, hq), torch.float32)
    kda.kda_attn_decode(layer.attn, 256, q, layer.table, i32(lens), plain.t, layer.ws.t, lse=pl.t)
    again, _ = attend(layer, q, lens, f32=True)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert torch.equal(o, again)
    # Weights in bf16 (2^-8 each) or f16 against the decode's: relative 2-norms well below that.
    off = ((o - plain.t).double().norm() / plain.t.double().norm()).item()
    assert off <= ref.UBF, off
    assert float((lse - pl.t).abs().max()) <= 1e-4
    layer.done()


def test_captured_and_on_another_stream():
    """Two graphs over one workspace, replayed in turn."""
    layers, graphs, outs = [], [], []
    stream = torch.cuda.Stream()
    ws = None
    for seed, n in ((1, 5), (2, 44)):
        layer, lens = build([(n, 300 + seed)], 9, 8, 2, 16, False, seed=seed)
        q, o = queries(layer, n), torch.zeros(n, 8, D, dtype=BF, device=DEV)
        args = (i32(lens), 1, i32([0, n]), i32([300 + seed]))
        ws = ws if ws is not None else torch.empty(kda.kda_attn_shared_workspace_bytes(layer.attn, 64), dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            kda.kda_attn_decode_shared(layer.attn, n, q, layer.table, *args, o, ws)
        layers.append((layer, lens, q, args))
        graphs.append(g)
        outs.append(o)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (layer, lens, q, _), o in zip(layers, outs):
        now, _ = attend(layer, q, lens)
        assert torch.equal(now.view(torch.int16), o.view(torch.int16))
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
        layer.done()


def test_refusals():
    layer, lens = build([(4, 100)], 1, 8, 2, 16, False)
    q, o = queries(layer, 4), torch.full((4, 8, D), 7.0, dtype=BF, device=DEV)
    ws = torch.empty(kda.kda_attn_shared_workspace_bytes(layer.attn, 4), dtype=torch.uint8, device=DEV)
    cu, prefix, kv = i32([0, 4]), i32([100]), i32(lens)

    def refused(status, B=4, groups=1, cu=cu, prefix=prefix, ws=ws, **more):
        before = kda.kda_launch_count()
        with pytest.raises(kda.KDAError) as e:
            kda.kda_attn_decode_shared(layer.attn, B, q, layer.table, kv, groups, cu, prefix, o, ws, **more)
        assert e.value.status == status and kda.kda_launch_count() == before
        torch.cuda.synchronize()
        assert bool((o == 7).all())

    bad, align = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_ALIGNMENT
    refused(bad, B=-1)
    refused(bad, groups=-1)
    refused(bad, groups=5)
    refused(bad, cu=None)
    refused(bad, prefix=None)
    refused(bad, ws=ws[:-256])
    refused(bad, max_pages=0)
    odd = torch.zeros(64, dtype=torch.uint8, device=DEV)
    refused(align, cu=odd[2:].data_ptr())
    refused(align, prefix=odd[2:].data_ptr())
    refused(align, ws=torch.empty(ws.numel() + 64, dtype=torch.uint8, device=DEV)[8:])
    assert kda.kda_attn_shared_workspace_bytes(layer.attn, 0) == 0
    kda.kda_attn_decode_shared(layer.attn, 0, q, layer.table, kv, 0, None, None, o, ws)
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,held", [(5, 0x3C), (40, 0x3C), (40, 0), (40, 0xFF)])
def test_a_copy_that_never_comes(n, held, e4m3, monkeypatch):
    """The bounded waits on it run out, whatever the workspace held: reported once, nothing written outside, and the
    device works on."""
    spans, lens = [(0, n, 300)], [320 + b for b in range(n)]

    def layer_of():
        layer = Layer(8, 2, 16, e4m3)
        fill(layer, lens)
        share(layer, spans, lens)
        return layer

    monkeypatch.setenv("KDA_FAULT_INJECT", "attn_drop")
    layer = layer_of()
    monkeypatch.delenv("KDA_FAULT_INJECT")
    ws = Guard((kda.kda_attn_shared_workspace_bytes(layer.attn, n),), torch.uint8, fill=held)
    attend(layer, queries(layer, n), lens, ws=ws)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_TIMEOUT
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    layer.done()
    again = layer_of()
    verify(again, queries(again, n), lens)
    again.done()


def test_injected_launch_failure(monkeypatch):
    for name in ("attn_decode_shared", "all"):
        monkeypatch.setenv("KDA_FAULT_INJECT", name)
        layer = Layer(4, 2, 16)
        monkeypatch.delenv("KDA_FAULT_INJECT")
        layer.fill([20])
        o = torch.full((1, 4, D), 7.0, dtype=BF, device=DEV)
        ws = torch.empty(kda.kda_attn_shared_workspace_bytes(layer.attn, 1), dtype=torch.uint8, device=DEV)
        before = kda.kda_launch_count()
        with pytest.raises(kda.KDAError) as e:
            kda.kda_attn_decode_shared(layer.attn, 1, queries(layer, 1), layer.table, i32([20]), 0, None, None, o, ws)
        assert e.value.status == kda.KDA_ERR_CUDA and "injected" in kda.kda_last_error_detail()
        assert kda.kda_launch_count() == before
        torch.cuda.synchronize()
        assert bool((o == 7).all())
        layer.done()
