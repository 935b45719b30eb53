"""The paged softmax-attention operators, as they are timed and compared.

Softmax-attention layers stand between KDA layers in a hybrid model.  Four operators serve one such
layer from a paged key/value cache (heads of 128, cache [pages][kv heads][page][128], bf16 or e4m3):

* plan     page allocation, block table, token positions and cache slots from the requests' lengths
* append   RMS norm of every q and k head, rotary position, k and v into their cache slots
* decode   attention of one new token per request over its cached keys
* prefill  causal attention of a chunk of new tokens per request over its cached keys

Each has a plain form in elementary torch operations and the call of the framework's kernel.
Lengths come from the case alone, values and the order of pages from the seed.
"""
import math
import random

import torch

own = False

HEAD = 128
EPS = 1e-6
BASE = 10000.0
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of 64 running requests, a few idle slots: called once per generated token.
        {"name": "plan_decode_b64", "op": "plan", "B": 64, "len": 8192, "new": 1, "page": 16, "idle": 3, "short": False},
        # A step that mixes prompts in chunks with decoding requests, the pool too small for all of them.
        {"name": "plan_mixed_b256", "op": "plan", "B": 256, "len": 16384, "new": 2048, "page": 64, "idle": 9, "short": True},
        # The smallest step there is: one request, one token.
        {"name": "append_b1_bf16", "op": "append", "N": 1, "hq": 32, "hkv": 8, "page": 16, "e4m3": False, "rot": 128, "inter": False, "pos": 4096},
        # One token of each of 256 requests into an 8-bit cache, half of the head rotated, far positions.
        {"name": "append_b256_e4m3", "op": "append", "N": 256, "hq": 64, "hkv": 8, "page": 64, "e4m3": True, "rot": 64, "inter": True, "pos": 1000000},
        # A packed batch of prompts.
        {"name": "append_n16381_bf16", "op": "append", "N": 16381, "hq": 32, "hkv": 8, "page": 16, "e4m3": False, "rot": 128, "inter": False, "pos": 16381},
        # One request with a short context: latency.
        {"name": "decode_b1_l517_bf16", "op": "decode", "B": 1, "len": 517, "hq": 32, "hkv": 8, "page": 16, "e4m3": False, "idle": 0},
        # A running batch with ragged contexts and idle slots.
        {"name": "decode_b64_l8192_bf16", "op": "decode", "B": 64, "len": 8192, "hq": 32, "hkv": 8, "page": 16, "e4m3": False, "idle": 2},
        # One request with a very long context and few heads: split over its length.
        {"name": "decode_b1_l262139_bf16", "op": "decode", "B": 1, "len": 262139, "hq": 32, "hkv": 4, "page": 64, "e4m3": False, "idle": 0},
        # The largest batch, 8-bit cache, sixteen query heads to a key head.
        {"name": "decode_b256_l8192_e4m3", "op": "decode", "B": 256, "len": 8192, "hq": 64, "hkv": 4, "page": 32, "e4m3": True, "idle": 5},
        # A few proposed tokens per request to verify against ragged contexts.
        {"name": "prefill_b32_t5_bf16", "op": "prefill", "B": 32, "new": 5, "len": 4096, "hq": 32, "hkv": 8, "page": 16, "e4m3": False},
        # One whole prompt.
        {"name": "prefill_b1_t8191_bf16", "op": "prefill", "B": 1, "new": 8191, "len": 8191, "hq": 32, "hkv": 8, "page": 16, "e4m3": False},
        # Ragged prompt chunks behind cached prefixes, 8-bit cache.
        {"name": "prefill_b6_t2048_e4m3", "op": "prefill", "B": 6, "new": 2048, "len": 6000, "hq": 64, "hkv": 8, "page": 64, "e4m3": True},
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "prefill", "prefill"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _spread(rng, 1, 256)
        return {"op": op, "B": B, "len": _spread(rng, 64, 16384), "new": _spread(rng, 1, 2048), "page": page,
                "idle": rng.randint(0, B // 4), "short": rng.random() < 0.3}
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    while hq > 64:
        hq -= hkv
    e4m3 = rng.random() < 0.4
    if op == "append":
        return {"op": op, "N": _spread(rng, 1, 16381), "hq": min(hq, 32), "hkv": min(hkv, hq, 32), "page": page,
                "e4m3": e4m3, "rot": rng.choice([32, 64, 96, 128]), "inter": rng.random() < 0.5,
                "pos": _spread(rng, 20000, 1000000)} if hq <= 32 else {
                "op": op, "N": _spread(rng, 1, 8192), "hq": hq, "hkv": hkv, "page": page, "e4m3": e4m3,
                "rot": 128, "inter": rng.random() < 0.5, "pos": _spread(rng, 20000, 1000000)}
    if op == "decode":
        B = _spread(rng, 1, 256)
        most = min(262139, 256 * 8192 * 4 // (B * hkv) // (1 if e4m3 else 2))
        return {"op": op, "B": B, "len": _spread(rng, 1, most), "hq": hq, "hkv": hkv, "page": page, "e4m3": e4m3,
                "idle": rng.randint(0, B // 4)}
    B = _spread(rng, 1, 32)
    new = _spread(rng, 1, 4096)
    most = 1 << 26  # query-key pairs over all requests: those of the listed prompt
    new = max(1, min(new, int(math.sqrt(most / B))))
    return {"op": op, "B": B, "new": new, "len": max(new, min(_spread(rng, new, 32768), most // (B * new))), "hq": min(hq, 32) // hkv * hkv,
            "hkv": hkv, "page": page, "e4m3": e4m3}


def _lens(case):
    """(cached before, new) tokens of every request; from the case alone."""
    rng = random.Random("%s %d %d %d" % (case["op"], case["B"], case["len"], case.get("new", 1)))
    B, L, idle = case["B"], case["len"], case.get("idle", 0)
    gone = set(rng.sample(range(B), idle)) if idle else set()
    cached, new = [], []
    for b in range(B):
        if case["op"] == "decode":  # the length that the token sees, its own key among them
            n = L if b == 0 else rng.randint(max(1, L // 8), L)
            cached.append(0 if b in gone else n - 1)
            new.append(0 if b in gone else 1)
        elif case["op"] == "prefill":
            t = case["new"] if b == 0 or case["new"] < 8 else rng.randint(1, case["new"])
            n = L if b == 0 else rng.randint(t, L)
            cached.append(n - t)
            new.append(t)
        else:
            t = 1 if case["new"] == 1 or rng.random() < 0.7 else rng.randint(1, case["new"])
            cached.append(rng.randint(0, L))
            new.append(0 if b in gone else t)
    return cached, new


def _pages(n, page):
    return -(-n // page)


def _table_width(case):
    c, n = _lens(case)
    return max(1, max(_pages(a + b, case["page"]) for a, b in zip(c, n)))


# ---------------------------------------------------------------- inputs

class Handle:
    """The framework's attention context of one layer, with its cache bound."""

    def __init__(self, case, s):
        import kda_delta_rule_token_gb300 as kda
        self.kda = kda
        hq, hkv = case.get("hq", 1), case.get("hkv", 1)
        self.attn = kda.kda_attn_create(
            hq, hkv, page_size=case["page"],
            cache_type=kda.KDA_CACHE_E4M3 if case.get("e4m3") else kda.KDA_CACHE_BF16,
            rotary_dim=case.get("rot", HEAD), rope_interleaved=case.get("inter", False),
            inv_freq=_inv_freq(case.get("rot", HEAD)), q_gamma=s.get("q_gamma"), k_gamma=s.get("k_gamma"),
            k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), rms_eps=EPS, softmax_scale=HEAD ** -0.5)
        if "k_cache" in s:
            kda.kda_attn_bind_cache(self.attn, s["k_cache"].shape[0], s["k_cache"], s["v_cache"])

    def __del__(self):
        self.kda.kda_attn_destroy(self.attn)


def _inv_freq(rot):
    return [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]


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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op, page = case["op"], case["page"]
    if op != "plan":
        hkv = case["hkv"]
        if case["e4m3"]:
            s["k_scale"] = torch.rand(hkv, generator=gen, device="cuda") * 0.01 + 0.01
            s["v_scale"] = torch.rand(hkv, generator=gen, device="cuda") * 0.01 + 0.01

    if op == "append":
        N, hq = case["N"], case["hq"]
        s["qkv"] = torch.randn(N, hq + 2 * hkv, HEAD, generator=gen, device="cuda", dtype=torch.bfloat16)
        s["q_gamma"] = 1 + 0.2 * torch.randn(HEAD, generator=gen, device="cuda")
        s["k_gamma"] = 1 + 0.2 * torch.randn(HEAD, generator=gen, device="cuda")
        pages = _pages(N, page) + 3
        s["slots"] = torch.randperm(pages * page, generator=gen, device="cuda")[:N] if N <= 256 else (
            torch.randperm(pages, generator=gen, device="cuda")[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:N].contiguous()
        s["positions"] = (torch.randint(0, case["pos"], (N,), generator=gen, device="cuda") if N <= 256 else
                          torch.arange(case["pos"] - N, case["pos"], device="cuda")).to(torch.int32)
        s["k_cache"] = _fill((pages, hkv, page, HEAD), case["e4m3"], gen, s.get("k_scale"))
        s["v_cache"] = _fill((pages, hkv, page, HEAD), case["e4m3"], gen, s.get("v_scale"))
        s["q_out"] = torch.empty(N, hq, HEAD, device="cuda", dtype=torch.bfloat16)
        s["inv_freq"] = torch.tensor(_inv_freq(case["rot"]), dtype=torch.float64, device="cuda")
        if own:
            s["handle"] = Handle(case, s)
        return s

    cached, new = _lens(case)
    B, width = case["B"], _table_width(case)
    s["width"] = width
    held = [_pages(c if op == "plan" else c + n, page) for c, n in zip(cached, new)]
    pool = sum(_pages(c + n, page) for c, n in zip(cached, new)) + 8
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    ends = _i32(held).cumsum(0)
    col = torch.arange(width, device="cuda")
    at = (ends - _i32(held))[:, None] + col
    s["table"] = torch.where(col < _i32(held)[:, None], order[at.clamp(max=pool - 1)], -1).to(torch.int32)
    if op == "plan":
        taken = sum(held)
        s["cached"], s["new"] = _i32(cached), _i32(new)
        s["N"] = sum(new)
        s["free"] = order[taken:].contiguous()
        need = pool - 8 - taken
        s["free_count"] = _i32([need // 2 if case["short"] else need + 5])
        s["cu"] = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        s["kv_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["positions"] = torch.empty(s["N"], dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(s["N"], dtype=torch.int64, device="cuda")
        s["info"] = torch.empty(4, dtype=torch.int32, device="cuda")
        if own:
            s["handle"] = Handle(case, s)
        return s

    hq = case["hq"]
    s["k_cache"] = _fill((pool, hkv, page, HEAD), case["e4m3"], gen, s.get("k_scale"))
    s["v_cache"] = _fill((pool, hkv, page, HEAD), case["e4m3"], gen, s.get("v_scale"))
    s["kv_lens"] = _i32([c + n for c, n in zip(cached, new)])
    s["N"] = B if op == "decode" else sum(new)
    s["new_max"] = max(new)
    s["q"] = (1.5 * torch.randn(s["N"], hq, HEAD, generator=gen, device="cuda")).to(torch.bfloat16)
    s["cu"] = _i32([0] + new).cumsum(0).to(torch.int32)
    s["o"] = torch.empty(s["N"], hq, HEAD, device="cuda", dtype=torch.bfloat16)
    if own:
        s["handle"] = h = Handle(case, s)
        s["workspace"] = torch.empty(h.kda.kda_attn_workspace_bytes(h.attn), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_plan(s):
    h = s["handle"]
    h.kda.kda_attn_plan(h.attn, s["case"]["B"], s["N"], s["cached"], s["new"], s["free"], s["free_count"], s["table"],
                        s["cu"], s["kv_lens"], s["positions"], s["slots"], s["info"])
    return s["table"], s["cu"], s["kv_lens"], s["positions"], s["slots"], s["info"]


def _own_append(s):
    h, c, qkv = s["handle"], s["case"], s["qkv"]
    hq, hkv = c["hq"], c["hkv"]
    h.kda.kda_attn_append(h.attn, c["N"], qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], s["positions"], s["slots"], s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_decode(s):
    h = s["handle"]
    h.kda.kda_attn_decode(h.attn, s["N"], s["q"], s["table"], s["kv_lens"], s["o"], s["workspace"])
    return s["o"]


def _own_prefill(s):
    h = s["handle"]
    h.kda.kda_attn_prefill(h.attn, s["case"]["B"], s["N"], s["cu"], s["q"], s["table"], s["kv_lens"], s["o"], s["workspace"])
    return s["o"]


def _plain_plan(s):
    page, N, table = s["case"]["page"], s["N"], s["table"].clone()
    cached, new, free, count = s["cached"].long(), s["new"].long(), s["free"].long(), s["free_count"].long()
    before, after = (cached + page - 1) // page, (cached + new + page - 1) // page
    ends = new.cumsum(0)
    fits = (after <= s["width"]) & (ends <= N)
    need = torch.where(fits, after - before, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= count))
    taken = torch.where(ok & (need > 0), upto, 0).max().reshape(1)
    kv = torch.where(ok, cached + new, 0)
    token = torch.arange(N, device="cuda")
    req = torch.searchsorted(ends, token, right=True)
    pos = cached[req] + token - (ends - new)[req]
    # The page of each token: one that the request holds, or one from the free list's end.
    fresh = pos // page - before[req]
    from_free = free[(count - 1 - ((upto - need)[req] + fresh)).clamp(0, free.numel() - 1)]
    held = table[req, (pos // page).clamp(max=s["width"] - 1)].long()
    at = torch.where(fresh >= 0, from_free, held)
    slots = torch.where(ok[req], at * page + pos % page, -1)
    # The new pages into the table.
    col = torch.arange(s["width"], device="cuda")
    nth = col - before[:, None]
    put = ok[:, None] & (nth >= 0) & (col < after[:, None])
    entry = free[(count - 1 - ((upto - need)[:, None] + nth)).clamp(0, free.numel() - 1)]
    table = torch.where(put, entry, table.long()).to(torch.int32)
    cu = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    info = torch.cat([ends[-1:], taken, count - taken, (~ok).sum().reshape(1)]).to(torch.int32)
    return table, cu, kv.to(torch.int32), pos.to(torch.int32), slots, info


def _plain_norm_rotate(x, gamma, cos, sin, case):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * gamma
    rot = case["rot"]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["inter"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if case["inter"] else torch.cat([c, d], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_store(cache, x, slots, scale):
    """Rows x [N, heads, 128] into the cache's slots."""
    page = cache.shape[2]
    if scale is None:
        cache[slots // page, :, slots % page] = x.to(cache.dtype)
    else:
        x = (x * (1 / scale)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache.view(torch.uint8)[slots // page, :, slots % page] = x.view(torch.uint8)


def _plain_append(s):
    c, qkv = s["case"], s["qkv"]
    hq, hkv = c["hq"], c["hkv"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _plain_norm_rotate(qkv[:, :hq], s["q_gamma"], cos, sin, c).to(torch.bfloat16)
    k = _plain_norm_rotate(qkv[:, hq:hq + hkv], s["k_gamma"], cos, sin, c)
    _plain_store(s["k_cache"], k, s["slots"], s.get("k_scale"))
    _plain_store(s["v_cache"], qkv[:, hq + hkv:].float(), s["slots"], s.get("v_scale"))
    return q, s["k_cache"], s["v_cache"]


def _plain_gather(cache, table, scale):
    """[B, kv heads, padded length, 128] in 32 bits."""
    x = cache.view(torch.uint8)[table.clamp(min=0).long()].view(cache.dtype) if scale is not None else cache[table.clamp(min=0).long()]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3).float()
    return x if scale is None else x.mul_(scale[None, :, None, None])


def _plain_attend(q, k, v, seen):
    """Softmax attention of q [B, kv heads, rows, 128]; seen [B, 1 or rows, keys] says which keys a row sees."""
    x = torch.matmul(q, k.transpose(2, 3)).mul_(HEAD ** -0.5).masked_fill_(~seen[:, None], -math.inf)
    most = x.amax(-1, keepdim=True)
    x.sub_(torch.where(most == -math.inf, 0, most)).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.matmul(x, v) / torch.where(total == 0, 1, total)


def _plain_decode(s):
    c = s["case"]
    k, v = _plain_gather(s["k_cache"], s["table"], s.get("k_scale")), _plain_gather(s["v_cache"], s["table"], s.get("v_scale"))
    q = s["q"].float().view(c["B"], c["hkv"], -1, HEAD)
    seen = torch.arange(k.shape[2], device="cuda") < s["kv_lens"][:, None, None]
    return _plain_attend(q, k, v, seen).view(c["B"], c["hq"], HEAD).to(torch.bfloat16)


def _plain_prefill(s):
    c, T = s["case"], s["new_max"]
    B, hkv, G = c["B"], c["hkv"], c["hq"] // c["hkv"]
    k, v = _plain_gather(s["k_cache"], s["table"], s.get("k_scale")), _plain_gather(s["v_cache"], s["table"], s.get("v_scale"))
    cu, t = s["cu"].long(), torch.arange(T, device="cuda")
    new = cu[1:] - cu[:-1]
    # Requests padded to the longest chunk.
    q = s["q"][(cu[:-1, None] + t).clamp(max=s["N"] - 1)].float()
    q = q.view(B, T, hkv, G, HEAD).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * T, HEAD)
    last = (s["kv_lens"] - new)[:, None] + t  # the last key that token t sees
    seen = torch.arange(k.shape[2], device="cuda") <= last[:, :, None]
    o = _plain_attend(q, k, v, seen.repeat(1, G, 1))
    o = o.view(B, hkv, G, T, HEAD).permute(0, 3, 1, 2, 4).reshape(B * T, c["hq"], HEAD)
    # Packed again.
    token = torch.arange(s["N"], device="cuda")
    req = torch.searchsorted(cu[1:], token, right=True)
    return o[req * T + token - cu[req]].to(torch.bfloat16)


_own = {"plan": _own_plan, "append": _own_append, "decode": _own_decode, "prefill": _own_prefill}
_plain = {"plan": _plain_plan, "append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}


# ---------------------------------------------------------------- work and exact values

def work(case):
    op, page = case["op"], case["page"]
    if op == "append":
        es, heads = 1 if case["e4m3"] else 2, case["hq"] + 2 * case["hkv"]
        row = heads * HEAD * 2 + case["hq"] * HEAD * 2 + 2 * case["hkv"] * HEAD * es + 12
        return {"bytes": case["N"] * row, "flops": case["N"] * (case["hq"] + case["hkv"]) * HEAD * 8}
    cached, new = _lens(case)
    tokens, B = sum(new), case["B"]
    if op == "plan":
        fresh = sum(_pages(c + n, page) - _pages(c, page) for c, n in zip(cached, new))
        return {"bytes": 4 * (2 * B + 2 * B + 1 + 5) + 12 * tokens + 8 * fresh, "flops": 10 * tokens}
    es = 1 if case["e4m3"] else 2
    kv = sum((c + n if n else 0) for c, n in zip(cached, new))
    table = 4 * sum(_pages(c + n, page) for c, n in zip(cached, new))
    rows = B if op == "decode" else tokens
    # Query-key pairs: token t of n new ones behind c cached sees c + t + 1 keys.
    pairs = sum(c * n + n * (n + 1) // 2 for c, n in zip(cached, new))
    return {"bytes": 2 * kv * case["hkv"] * HEAD * es + table + 2 * rows * case["hq"] * HEAD * 2,
            "flops": 4 * pairs * case["hq"] * HEAD}


def exact(case, seed):
    """The outputs in 64 bits, one request and one head after another."""
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    page, hkv = case["page"], case["hkv"]
    G = case["hq"] // hkv
    f64 = torch.float64
    if case["op"] == "append":
        N, rot = case["N"], case["rot"]
        half = rot // 2
        theta = torch.outer(s["positions"].to(f64), torch.tensor([BASE ** (-i / half) for i in range(half)], dtype=f64, device="cuda"))
        first = [2 * i for i in range(half)] if case["inter"] else list(range(half))
        second = [2 * i + 1 for i in range(half)] if case["inter"] else list(range(half, rot))

        def head(h, gamma):
            x = s["qkv"][:, h].to(f64)
            x = x / ((x ** 2).sum(1, keepdim=True) / HEAD + EPS).sqrt() * gamma.to(f64)
            z = torch.complex(x[:, first], x[:, second]) * torch.polar(torch.ones_like(theta), theta)
            x[:, first], x[:, second] = z.real, z.imag
            return x

        q = torch.stack([head(h, s["q_gamma"]) for h in range(case["hq"])], 1)
        out = [q]
        for name, scale, base in (("k_cache", "k_scale", case["hq"]), ("v_cache", "v_scale", case["hq"] + hkv)):
            cache = s[name].to(f64)
            for h in range(hkv):
                x = head(base + h, s["k_gamma"]) if name == "k_cache" else s["qkv"][:, base + h].to(f64)
                if case["e4m3"]:
                    x = (x / s[scale][h].to(f64)).clamp(-E4M3_MAX, E4M3_MAX)
                flat = cache[:, h].reshape(-1, HEAD)
                flat[s["slots"]] = x
                cache[:, h] = flat.view(-1, page, HEAD)
            out.append(cache)
        return tuple(out)

    out = torch.zeros(s["N"], case["hq"], HEAD, dtype=f64, device="cuda")
    cached, new = _lens(case)
    begin = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        rows = slice(b, b + 1) if case["op"] == "decode" else slice(begin, begin + n)
        begin += n
        if not n:
            continue
        pages = s["table"][b, :_pages(c + n, page)].long()
        sees = (torch.arange(c + n, device="cuda")[None] - torch.arange(n, device="cuda")[:, None]) <= c
        for h in range(hkv):
            k, v = (s[name].view(torch.uint8 if case["e4m3"] else torch.bfloat16)[pages, h].view(s[name].dtype).to(f64).reshape(-1, HEAD)[:c + n]
                    for name in ("k_cache", "v_cache"))
            if case["e4m3"]:
                k, v = k * s["k_scale"][h].to(f64), v * s["v_scale"][h].to(f64)
            for g in range(G):
                z = s["q"][rows, h * G + g].to(f64) @ k.T / math.sqrt(HEAD)
                w = torch.softmax(torch.where(sees, z, torch.full_like(z, -math.inf)), 1)
                out[rows, h * G + g] = w @ v
    return out
