"""The operators of several continuations of one prompt, as they are timed and compared.

Beam search, and several samples of one prompt, run many requests that share their first tokens and
that take over one another's state from step to step, in a model of KDA layers (a recurrent state per
request) and softmax-attention layers (pages of a key/value cache).  Four operators serve a step:

* select   the best continuations of each group of beams, over beams and vocabulary
* reorder  the recurrent states and convolution windows of the beams that were chosen
* fork     pages of the cache shared, released and copied as beams take over one another
* shared   attention of one new token per request where groups of requests share a prefix

Each has a plain form in elementary torch operations and the calls of the framework's kernels.
Sizes, lengths and which beam goes on come from the case alone, values and the order of pages from the
seed.
"""
import math
import random

import torch

own = False

HEAD = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One prompt with four beams: the smallest step of a search, where latency counts.
        {"name": "select_g1_k4_v32000", "op": "select", "groups": 1, "beams": 4, "vocab": 32000, "bf16": False, "num": 4, "places": True, "done": 0, "open": 0},
        # Sixteen prompts, bf16 logits of an odd vocabulary, twice the beams asked for, some beams at their end.
        {"name": "select_g16_k8_v131071_bf16", "op": "select", "groups": 16, "beams": 8, "vocab": 131071, "bf16": True, "num": 16, "places": False, "done": 9, "open": 0},
        # The largest batch of beams, fp32 logits.
        {"name": "select_g64_k8_v131072", "op": "select", "groups": 64, "beams": 8, "vocab": 131072, "bf16": False, "num": 8, "places": True, "done": 0, "open": 0},
        # The state of four beams of one prompt in a layer of 32 heads.
        {"name": "reorder_b4_h32", "op": "reorder", "B": 4, "beams": 4, "heads": 32, "bf16": False, "whole": False},
        # Decode batch of 64 sequences and 32 heads in groups of eight beams.
        {"name": "reorder_b64_h32", "op": "reorder", "B": 64, "beams": 8, "heads": 32, "bf16": False, "whole": False},
        # 256 sequences of 64 heads with 16-bit states, into another buffer in the order of their scores.
        {"name": "reorder_b256_h64_bf16", "op": "reorder", "B": 256, "beams": 4, "heads": 64, "bf16": True, "whole": True},
        # Four beams of one prompt: latency.
        {"name": "fork_b4_l1000", "op": "fork", "B": 4, "beams": 4, "prefix": 1000, "more": 200, "hkv": 8, "page": 16, "e4m3": False},
        # 256 requests in beams of eight behind long prompts, an 8-bit cache in pages of 128.
        {"name": "fork_b256_l8191_e4m3", "op": "fork", "B": 256, "beams": 8, "prefix": 8191, "more": 500, "hkv": 8, "page": 128, "e4m3": True},
        # Four beams behind a short prompt.
        {"name": "shared_g1_b4_l517", "op": "shared", "groups": 1, "B": 4, "prefix": 517, "more": 60, "hq": 32, "hkv": 8, "page": 16, "e4m3": False, "idle": 0},
        # Thirty-two prompts with eight beams each.
        {"name": "shared_g32_b256_l4100", "op": "shared", "groups": 32, "B": 256, "prefix": 4100, "more": 200, "hq": 32, "hkv": 8, "page": 16, "e4m3": False, "idle": 0},
        # 64 samples of one long prompt, a few at their end.
        {"name": "shared_g1_b64_l8192", "op": "shared", "groups": 1, "B": 64, "prefix": 8192, "more": 256, "hq": 32, "hkv": 8, "page": 64, "e4m3": False, "idle": 3},
        # The largest: 256 requests behind four long documents, 8-bit cache, sixteen query heads to a key head.
        {"name": "shared_g4_b256_l16300_e4m3", "op": "shared", "groups": 4, "B": 256, "prefix": 16300, "more": 500, "hq": 64, "hkv": 4, "page": 32, "e4m3": True, "idle": 5},
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["select", "select", "reorder", "fork", "shared", "shared", "shared"])
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
        vocab = _spread(rng, 1000, 200000)
        groups = _spread(rng, 1, max(1, min(64, (1 << 26) // (beams * vocab))))
        num = rng.choice([beams, beams, 2 * beams, _spread(rng, 1, 64)])
        return {"op": op, "groups": groups, "beams": beams, "vocab": vocab, "bf16": rng.random() < 0.5, "num": num,
                "places": num == beams and rng.random() < 0.7, "done": rng.randint(0, groups * beams // 3),
                "open": rng.choice([0, 0, 0, 3, 50])}
    beams = rng.choice([2, 3, 4, 5, 8, 16])
    if op == "reorder":
        heads = rng.choice([1, 2, 8, 32, 64])
        bf16 = rng.random() < 0.4
        groups = _spread(rng, 1, max(1, min(256, (16384 if bf16 else 8192) // heads) // beams))
        return {"op": op, "B": groups * beams, "beams": beams, "heads": heads, "bf16": bf16, "whole": rng.random() < 0.4}
    hkv, page, e4m3 = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128]), rng.random() < 0.4
    if op == "fork":
        B = beams * _spread(rng, 1, 256 // beams)
        return {"op": op, "B": B, "beams": beams, "prefix": _spread(rng, 1, 8191), "more": _spread(rng, 1, 500), "hkv": hkv, "page": page, "e4m3": e4m3}
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    while hq > 64:
        hq -= hkv
    B = _spread(rng, 1, 256)
    groups = _spread(rng, 1, min(B, 64))
    most = max(64, min(65536, (1 << 24) // (B * hkv)))
    return {"op": op, "groups": groups, "B": B, "prefix": _spread(rng, 1, most), "more": _spread(rng, 1, 300), "hq": hq, "hkv": hkv, "page": page,
            "e4m3": e4m3, "idle": rng.randint(0, B // 8)}


def _rng(case):
    return random.Random(" ".join("%s=%s" % (k, v) for k, v in sorted(case.items()) if k != "name"))


def _rows(case):
    """Which beam every beam goes on from.  In place: half of a group's beams or more go on where they are and the
    others take over one of them; else any beam of the group from any."""
    rng, K, rows = _rng(case), case["beams"], []
    for g in range(0, case["B"], K):
        if case.get("whole"):
            rows += [g + rng.randrange(K) for _ in range(K)]
            continue
        stay = sorted(rng.sample(range(K), rng.randint((K + 1) // 2, max(1, K - 1))))
        rows += [g + k if k in stay else g + rng.choice(stay) for k in range(K)]
    return rows


def _pages(n, page):
    return -(-n // page)


def _requests(case):
    """(first request, prefix length) of every group, and the lengths of all requests."""
    rng, B, P, more = _rng(case), case["B"], case["prefix"], case["more"]
    if case["op"] == "fork":
        K = case["beams"]
        groups = [(g, P if g == 0 else rng.randint(max(1, P // 2), P)) for g in range(0, B, K)]
        lens = []
        for g, p in groups:  # beams of a group are of one length
            lens += [p + rng.randint(1, more)] * K
        return groups, lens
    cuts = sorted(rng.sample(range(1, B), case["groups"] - 1))
    groups = [(g, P if g == 0 else rng.randint(max(1, P // 2), P)) for g in [0] + cuts]
    lens = []
    for (g, p), end in zip(groups, cuts + [B]):
        lens += [p + rng.randint(1, more) for _ in range(g, end)]
    for b in rng.sample(range(B), case["idle"]):
        lens[b] = 0
    return groups, lens


# ---------------------------------------------------------------- inputs

class Context:
    """The framework's context of a KDA layer."""

    def __init__(self, heads):
        import kda_delta_rule_token_gb300 as kda
        self.kda = kda
        f = dict(device="cuda")
        self.params = (torch.zeros(3, heads * HEAD, 4, **f), torch.zeros(heads, HEAD, **f), torch.zeros(heads, HEAD, **f), torch.ones(heads, HEAD, **f))
        self.ctx = kda.kda_create(heads, *self.params)

    def __del__(self):
        self.kda.kda_destroy(self.ctx)


class Handle:
    """The framework's context of a softmax-attention layer, with its cache bound."""

    def __init__(self, case, s):
        import kda_delta_rule_token_gb300 as kda
        self.kda = kda
        self.attn = kda.kda_attn_create(
            case.get("hq", case["hkv"]), case["hkv"], page_size=case["page"],
            cache_type=kda.KDA_CACHE_E4M3 if case["e4m3"] else kda.KDA_CACHE_BF16, rotary_dim=0,
            k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), softmax_scale=HEAD ** -0.5)
        kda.kda_attn_bind_cache(self.attn, s["k_cache"].shape[0], s["k_cache"], s["v_cache"])

    def __del__(self):
        self.kda.kda_attn_destroy(self.attn)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _fill(shape, e4m3, gen, scale):
    """Random cache contents: normal values, or e4m3 values that stand for normal ones at `scale`."""
    if not e4m3:
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
    step = max(1, (1 << 28) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        x = torch.randn(out[i:i + step].shape, generator=gen, device="cuda", dtype=torch.float32)
        out[i:i + step] = (x / scale.view(1, -1, 1, 1)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return out


def _prepare_select(case, gen, s):
    G, K, V, n = case["groups"], case["beams"], case["vocab"], case["num"]
    x = 3 * torch.randn(G * K, V, generator=gen, device="cuda")
    if case["open"]:  # a grammar leaves about so many tokens of the vocabulary open
        x.masked_fill_(torch.rand(G * K, V, generator=gen, device="cuda") * V > case["open"], -math.inf)
    s["logits"] = x.to(torch.bfloat16) if case["bf16"] else x
    s["scores"] = -20 * torch.rand(G, K, generator=gen, device="cuda")
    s["scores"][:1, 1:] = -math.inf  # a search that begins: its beams are still alike, one of them counts
    s["done"] = torch.zeros(G, K, dtype=torch.uint8, device="cuda")
    s["done"].view(-1)[torch.randperm(G * K, generator=gen, device="cuda")[:case["done"]]] = 1
    s["end"] = 2
    s["out"] = tuple(torch.empty(G, n, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
    if own:
        s["ctx"] = c = Context(1)
        s["workspace"] = torch.empty(c.kda.kda_beam_select_workspace_bytes(c.ctx, G, K, V, n), dtype=torch.uint8, device="cuda")


def _prepare_reorder(case, gen, s):
    B, H = case["B"], case["heads"]
    s["S"] = torch.randn(B, H, HEAD, HEAD, generator=gen, device="cuda", dtype=torch.bfloat16 if case["bf16"] else torch.float32)
    s["conv"] = torch.randn(B, 3, 3 * H * HEAD, generator=gen, device="cuda")
    s["rows"] = _i32(_rows(case))
    if case["whole"]:
        s["S_out"], s["conv_out"] = torch.empty_like(s["S"]), torch.empty_like(s["conv"])
    if own:
        s["ctx"] = Context(H)


def _prepare_cache(case, gen, s):
    """Block table, pages and cache: the whole pages of a group's prefix are shared, all others a request's own."""
    page, hkv, B = case["page"], case["hkv"], case["B"]
    groups, lens = _requests(case)
    ends = [g for g, _ in groups[1:]] + [B]
    width = max(1, max(_pages(n, page) for n in lens), max(p // page for _, p in groups))
    table, pool, copies = [], 0, []
    for (g, p), end in zip(groups, ends):
        shared = list(range(pool, pool + p // page))
        pool += len(shared)
        for b in range(g, end):
            mine = max(0, _pages(lens[b], page) - len(shared))
            table.append(shared + list(range(pool, pool + mine)) + [-1] * (width - len(shared) - mine))
            if mine and p % page:  # the page that the prefix ends in: a copy of its rows
                copies.append((pool, p % page, g))
            pool += mine
    spare = B + 5
    order = torch.randperm(pool + spare, generator=gen, device="cuda").to(torch.int32)
    t = _i32(table)
    s["table"] = torch.where(t >= 0, order[t.clamp(min=0)], -1).to(torch.int32)
    s["free"] = torch.cat([order[pool:], torch.full((pool,), -1, dtype=torch.int32, device="cuda")])
    s["free_count"] = _i32([spare])
    s["kv_lens"] = _i32(lens)
    if case["e4m3"]:
        s["k_scale"] = torch.rand(hkv, generator=gen, device="cuda") * 0.01 + 0.01
        s["v_scale"] = torch.rand(hkv, generator=gen, device="cuda") * 0.01 + 0.01
    for name in ("k", "v"):
        s[name + "_cache"] = c = _fill((pool + spare, hkv, page, HEAD), case["e4m3"], gen, s.get(name + "_scale"))
        raw, first = c.view(torch.uint8) if case["e4m3"] else c, {}
        for to, rows, g in copies:
            src = first.setdefault(g, to)
            if src != to:
                raw[order[to], :, :rows] = raw[order[src], :, :rows]
    if own:
        s["handle"] = Handle(case, s)
    return groups, lens, pool + spare


def _prepare_fork(case, gen, s):
    page, B = case["page"], case["B"]
    groups, lens, pages = _prepare_cache(case, gen, s)
    held = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    flat = s["table"].reshape(-1).long()
    held.index_add_(0, torch.where(flat >= 0, flat, pages), torch.ones_like(flat, dtype=torch.int32))
    s["refs_before"] = (held[:pages] - 1).clamp(min=0).contiguous()  # further holders of a page
    s["refs"] = torch.empty_like(s["refs_before"])
    s["rows"] = _i32(_rows(case))
    s["new_table"] = torch.full_like(s["table"], -1)
    s["new_lens"] = torch.empty_like(s["kv_lens"])
    s["copies"] = torch.empty(3, B, dtype=torch.int32, device="cuda")
    s["info"] = torch.empty(4, dtype=torch.int32, device="cuda")
    if own:
        h = s["handle"]
        s["workspace"] = torch.empty(h.kda.kda_attn_fork_workspace_bytes(h.attn, B, s["table"].shape[1]), dtype=torch.uint8, device="cuda")


def _prepare_shared(case, gen, s):
    B, hq = case["B"], case["hq"]
    groups, lens, _ = _prepare_cache(case, gen, s)
    s["cu_groups"] = _i32([g for g, _ in groups] + [B])
    s["prefix_lens"] = _i32([p for _, p in groups])
    s["q"] = (1.5 * torch.randn(B, hq, HEAD, generator=gen, device="cuda")).to(torch.bfloat16)
    s["o"] = torch.empty(B, hq, HEAD, device="cuda", dtype=torch.bfloat16)
    if own:
        h = s["handle"]
        s["workspace"] = torch.empty(h.kda.kda_attn_shared_workspace_bytes(h.attn, B), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    {"select": _prepare_select, "reorder": _prepare_reorder, "fork": _prepare_fork, "shared": _prepare_shared}[case["op"]](case, gen, s)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_select(s):
    c, h = s["case"], s["ctx"]
    scores, tokens, rows = s["out"]
    h.kda.kda_beam_select(h.ctx, c["groups"], c["beams"], s["logits"], s["scores"], c["num"], scores, tokens, rows, s["workspace"],
                          done=s["done"], end_token=s["end"], keep_places=c["places"])
    return scores, tokens, rows


def _own_reorder(s):
    c, h = s["case"], s["ctx"]
    if c["whole"]:
        h.kda.kda_beam_reorder(h.ctx, c["B"], s["rows"], s["S"], s["conv"], S_out=s["S_out"], conv_out=s["conv_out"])
        return s["S_out"], s["conv_out"]
    h.kda.kda_beam_reorder(h.ctx, c["B"], s["rows"], s["S"], s["conv"])
    return s["S"], s["conv"]


def _own_fork(s):
    c, h = s["case"], s["handle"]
    s["refs"].copy_(s["refs_before"])  # which the call changes: every pass begins with the same holders
    src, dst, rows = s["copies"].unbind(0)
    h.kda.kda_attn_fork(h.attn, c["B"], s["rows"], s["kv_lens"], s["table"], s["refs"], s["free"], s["free_count"], s["new_table"],
                        s["new_lens"], src, dst, rows, s["info"], s["workspace"])
    h.kda.kda_attn_copy_pages(h.attn, c["B"], src, dst, rows)
    return s["new_table"], s["new_lens"], s["refs"], s["free"], s["copies"], s["info"], s["k_cache"], s["v_cache"]


def _own_shared(s):
    c, h = s["case"], s["handle"]
    h.kda.kda_attn_decode_shared(h.attn, c["B"], s["q"], s["table"], s["kv_lens"], c["groups"], s["cu_groups"], s["prefix_lens"], s["o"], s["workspace"])
    return s["o"]


def _plain_select(s):
    c = s["case"]
    G, K, V, n = c["groups"], c["beams"], c["vocab"], c["num"]
    # In 64 bits: which of two beams' close candidates is the better one hangs on the last bits.
    x = s["logits"].double()
    most = x.amax(1, keepdim=True)
    most = torch.where(most.isinf(), 0, most)
    x = x - ((x - most).exp().sum(1, keepdim=True).log() + most) + s["scores"].view(-1, 1)
    # A beam at its end goes on in one way, at the score that it has.
    token = torch.arange(V, device="cuda")
    x = torch.where(s["done"].view(-1, 1) == 0, x, torch.where(token == s["end"], s["scores"].view(-1, 1).double(), -math.inf))
    x = torch.where(x.isnan(), -math.inf, x).view(G, K * V)
    # The n largest, of equal ones those of the lowest index.
    last = x.topk(n).values[:, -1:]
    above, equal = x > last, x == last
    take = above | (equal & (equal.cumsum(1) <= n - above.sum(1, keepdim=True)))
    at = x.new_zeros(G, n + 1, dtype=torch.int64)
    at.scatter_(1, torch.where(take, take.cumsum(1) - 1, n), torch.arange(K * V, device="cuda").expand(G, -1))
    at = at[:, :n]
    score, order = x.gather(1, at).sort(dim=1, descending=True, stable=True)
    at = at.gather(1, order)
    beam, token = at // V, at % V
    if c["places"]:
        # A beam's best continuation takes the beam's place, the others the places that are left.
        nth = torch.arange(n, device="cuda")
        first = ~((beam[:, :, None] == beam[:, None]) & (nth < nth[:, None])).any(2)
        taken = torch.zeros(G, n, dtype=torch.int64, device="cuda").scatter_add_(1, beam, first.long())
        left = taken.sort(dim=1, stable=True).indices
        place = torch.where(first, beam, left.gather(1, ((~first).cumsum(1) - 1).clamp(min=0)))
        score, token, beam = (torch.empty_like(t).scatter_(1, place, t) for t in (score, token, beam))
    rows = beam + K * torch.arange(G, device="cuda")[:, None]
    return score.float(), token.to(torch.int32), rows.to(torch.int32)


def _plain_reorder(s):
    rows = s["rows"].long()
    S, conv = s["S"][rows], s["conv"][rows]
    if s["case"]["whole"]:
        return s["S_out"].copy_(S), s["conv_out"].copy_(conv)
    return s["S"].copy_(S), s["conv"].copy_(conv)


def _plain_fork(s):
    c = s["case"]
    B, page, W = c["B"], c["page"], s["table"].shape[1]
    rows, lens, table = s["rows"].long(), s["kv_lens"].long(), s["table"].long()
    pages = s["refs_before"].numel()
    b, col = torch.arange(B, device="cuda"), torch.arange(W, device="cuda")
    children = torch.zeros(B, dtype=torch.int64, device="cuda").index_add_(0, rows, torch.ones_like(rows))
    first = torch.full((B,), B, device="cuda").scatter_reduce_(0, rows, b, "amin")[rows] == b
    used, whole = (lens + page - 1) // page, lens // page
    # Pages that go on with several requests have more holders, those of requests that end fewer.
    refs = torch.cat([s["refs_before"].long(), s["refs_before"].new_zeros(1).long()])
    more = (children[:, None] > 1) & (col < whole[:, None])
    refs.index_add_(0, torch.where(more, table, pages).reshape(-1), (children[:, None] - 1).expand(B, W).reshape(-1))
    gone = (children[:, None] == 0) & (col < used[:, None])
    at = torch.where(gone, table, pages).t().reshape(-1)  # by index in the row, then by request
    refs.index_add_(0, at, torch.full_like(at, -1))
    nth = torch.arange(B * W, device="cuda")
    last = torch.full((pages + 1,), -1, device="cuda").scatter_reduce_(0, at, nth, "amax")[at]
    push = (at < pages) & (refs[at] < 0) & (last == nth)
    count, freed = s["free_count"].long(), push.sum()
    free = torch.cat([s["free"].long(), s["free"].new_zeros(1).long()])
    free.scatter_(0, torch.where(push, count + push.cumsum(0) - 1, free.numel() - 1), at)
    refs = refs[:pages].clamp(min=0)
    # Requests after the first of a beam get their own copy of its last page, where that is partly full.
    part = (lens % page)[rows]
    need = ~first & (part > 0)
    fresh = free[(count + freed - need.cumsum(0)).clamp(min=0)]
    source = table[rows, whole[rows].clamp(max=W - 1)]
    new = torch.where(col < used[rows][:, None], table[rows], s["new_table"].long())
    new = torch.where(need[:, None] & (col == whole[rows][:, None]), fresh[:, None], new)
    src, dst, part = torch.where(need, source, -1), torch.where(need, fresh, -1), torch.where(need, part, 0)
    taken = need.sum()
    info = torch.stack([freed, taken, (count + freed - taken)[0], torch.zeros_like(taken)])
    # The copies' rows; where there is none to make, none of a page that stays as it is.
    row = torch.arange(page, device="cuda") < part[:, None]
    fro, to = torch.where(need, src, table[rows, 0]), torch.where(need, dst, table[rows, 0])
    for name in ("k_cache", "v_cache"):
        raw = s[name].view(torch.uint8) if c["e4m3"] else s[name]
        raw[to] = torch.where(row[:, None, :, None], raw[fro], raw[to])
    i32 = torch.int32
    return (new.to(i32), lens[rows].to(i32), refs.to(i32), free[:-1].to(i32), torch.stack([src, dst, part]).to(i32), info.to(i32), s["k_cache"], s["v_cache"])


def _plain_gather(cache, table, scale):
    """[B, kv heads, padded length, 128] in 32 bits."""
    x = cache.view(torch.uint8)[table.clamp(min=0).long()].view(cache.dtype) if scale is not None else cache[table.clamp(min=0).long()]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3).float()
    return x if scale is None else x.mul_(scale[None, :, None, None])


def _plain_shared(s):
    c = s["case"]
    k, v = _plain_gather(s["k_cache"], s["table"], s.get("k_scale")), _plain_gather(s["v_cache"], s["table"], s.get("v_scale"))
    q = s["q"].float().view(c["B"], c["hkv"], -1, HEAD)
    seen = torch.arange(k.shape[2], device="cuda") < s["kv_lens"][:, None, None]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(HEAD ** -0.5).masked_fill_(~seen[:, None], -math.inf)
    most = x.amax(-1, keepdim=True)
    x.sub_(torch.where(most == -math.inf, 0, most)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total == 0, 1, total)
    return o.view(c["B"], c["hq"], HEAD).to(torch.bfloat16)


_own = {"select": _own_select, "reorder": _own_reorder, "fork": _own_fork, "shared": _own_shared}
_plain = {"select": _plain_select, "reorder": _plain_reorder, "fork": _plain_fork, "shared": _plain_shared}


# ---------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    if op == "select":
        G, K, V, n = case["groups"], case["beams"], case["vocab"], case["num"]
        rows = G * K - case["done"]
        return {"bytes": rows * V * (2 if case["bf16"] else 4) + 5 * G * K + 12 * G * n, "flops": 4 * rows * V}
    if op == "reorder":
        rows, H = _rows(case), case["heads"]
        one = H * HEAD * HEAD * (2 if case["bf16"] else 4) + 9 * H * HEAD * 4
        moved = [r for b, r in enumerate(rows) if case["whole"] or r != b]
        return {"bytes": (len(set(moved)) + len(moved)) * one + 4 * len(rows), "flops": 0}
    page, hkv, es = case["page"], case["hkv"], 1 if case["e4m3"] else 2
    groups, lens = _requests(case)
    if op == "fork":
        rows = _rows(case)
        entries = sum(_pages(lens[r], page) for r in rows)
        times = [rows.count(b) for b in range(len(rows))]
        touched = sum(_pages(n, page) for n, t in zip(lens, times) if t != 1)
        copied = sum(lens[r] % page for b, r in enumerate(rows) if rows.index(r) != b)
        return {"bytes": 8 * entries + 12 * touched + 12 * len(rows) + 2 * 2 * copied * hkv * HEAD * es, "flops": 0}
    ends = [g for g, _ in groups[1:]] + [case["B"]]
    keys = entries = 0
    for (g, p), end in zip(groups, ends):
        here = [n for n in lens[g:end] if n]
        if here:
            keys += p + sum(n - p for n in here)
            entries += p // page + sum(_pages(n, page) - p // page for n in here)
    return {"bytes": 2 * keys * hkv * HEAD * es + 4 * entries + 2 * case["B"] * case["hq"] * HEAD * 2,
            "flops": 4 * sum(lens) * case["hq"] * HEAD}


def exact(case, seed):
    """The outputs in 64 bits, a group or a request after another; whole numbers have no such value."""
    op = case["op"]
    if op == "fork":
        return None  # page numbers, and rows copied as they are
    s = prepare(case, seed)
    if op == "reorder":
        S, conv = s["S"].clone(), s["conv"].clone()
        for b, r in enumerate(_rows(case)):
            S[b].copy_(s["S"][r])
            conv[b].copy_(s["conv"][r])
        return S, conv
    f64 = torch.float64
    if op == "select":
        G, K, V, n = case["groups"], case["beams"], case["vocab"], case["num"]
        out = torch.empty(G, n, dtype=f64, device="cuda")
        for g in range(G):
            rows = torch.log_softmax(s["logits"][g * K:(g + 1) * K].to(f64), 1) + s["scores"][g, :, None].to(f64)
            for k in range(K):
                if s["done"][g, k]:
                    rows[k] = -math.inf
                    rows[k, s["end"]] = s["scores"][g, k].to(f64)
            best = rows.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf).flatten().sort(dim=0, descending=True, stable=True)
            score, beam = best.values[:n].tolist(), (best.indices[:n] // V).tolist()
            if case["places"]:
                place, left = {}, []
                for i, k in enumerate(beam):
                    if k in place:
                        left.append(i)
                    else:
                        place[k] = i
                score = [score[place[k] if k in place else left.pop(0)] for k in range(n)]
            out[g] = torch.tensor(score, dtype=f64)
        return out, None, None
    page, hkv = case["page"], case["hkv"]
    G = case["hq"] // hkv
    out = torch.zeros(case["B"], case["hq"], HEAD, dtype=f64, device="cuda")
    for b, n in enumerate(_requests(case)[1]):
        if not n:
            continue
        pages = s["table"][b, :_pages(n, page)].long()
        k, v = (s[name].view(torch.uint8 if case["e4m3"] else torch.bfloat16)[pages].view(s[name].dtype).to(f64).transpose(0, 1).reshape(hkv, -1, HEAD)[:, :n]
                for name in ("k_cache", "v_cache"))
        if case["e4m3"]:
            k, v = k * s["k_scale"].to(f64)[:, None, None], v * s["v_scale"].to(f64)[:, None, None]
        z = torch.einsum("hgd,hnd->hgn", s["q"][b].to(f64).view(hkv, G, HEAD), k) / math.sqrt(HEAD)
        out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(z, 2), v).reshape(case["hq"], HEAD)
    return out
