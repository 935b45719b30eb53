"""The paged softmax-attention operators against their plain 64-bit forms.

Outputs lie between guard regions, caches hold NaN and infinity wherever no
request's keys lie, and block tables hold ids outside the cache wherever no
page is mapped: a kernel that looked there would show it.
"""
import math
import random

import pytest
import torch

import attn_ref as ref
import kda_delta_rule_token_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
BF = torch.bfloat16
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_delta_rule_token_gb300 import build
    build.build()
    kda.load()


class Guard:
    """A tensor of any type inside a buffer whose margins hold a byte pattern."""

    def __init__(self, shape, dtype, fill=0x5A):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        self.buf = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
        self.buf[4096:4096 + n] = fill
        self.t = self.buf[4096:4096 + n].view(dtype).view(shape)
        self.n = n

    def intact(self):
        return bool((self.buf[:4096] == 0xA5).all()) and bool((self.buf[4096 + self.n:] == 0xA5).all())


def inv_freq(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Layer:
    def __init__(self, hq, hkv, page, e4m3=False, pages=None, seed=0, rot=0, **more):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.hq, self.hkv, self.page, self.e4m3 = hq, hkv, page, e4m3
        self.ks = self.vs = None
        if e4m3:
            self.ks = torch.rand(hkv, generator=self.g, device=DEV) * 0.02 + 0.01
            self.vs = torch.rand(hkv, generator=self.g, device=DEV) * 0.02 + 0.01
        more.setdefault("inv_freq", inv_freq(rot) if rot else None)
        self.attn = kda.kda_attn_create(hq, hkv, page_size=page, rotary_dim=rot, k_scale=self.ks, v_scale=self.vs,
                                        cache_type=kda.KDA_CACHE_E4M3 if e4m3 else kda.KDA_CACHE_BF16, **more)
        self.ws = Guard((max(16, kda.kda_attn_workspace_bytes(self.attn)),), torch.uint8)
        if pages:
            self.caches(pages)

    def caches(self, pages):
        """Two caches of nothing but NaN and infinities."""
        self.pages = pages
        shape = (pages, self.hkv, self.page, D)
        if self.e4m3:
            self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
        else:
            self.k, self.v = (torch.full(shape, bad, dtype=BF, device=DEV) for bad in (math.nan, math.inf))
            self.v[::2] = math.nan
        kda.kda_attn_bind_cache(self.attn, pages, self.k, self.v)

    def values(self, n, scale, sigma):
        x = torch.randn(n, self.hkv, D, generator=self.g, device=DEV) * sigma
        return x.to(BF) if not self.e4m3 else (x / scale[:, None]).clamp(-448, 448).to(F8)

    def fill(self, lens, sigma=1.0, width=None, spare=3):
        """Random keys and values for requests of these lengths; their block table."""
        need = [-(-max(n, 0) // self.page) for n in lens]
        width = width or max(1, max(need))
        self.caches(sum(need) + spare)
        order = torch.randperm(self.pages, generator=self.g, device=DEV).tolist()
        bad = random.Random(5)
        table = []
        for n in need:
            held, order = order[:n], order[n:]
            table.append(held + [bad.choice([-1, self.pages, 2 ** 31 - 1, -2 ** 31])] * (width - n))
        for b, n in enumerate(lens):
            if n <= 0:
                continue
            at = torch.arange(n, device=DEV)
            pg = torch.tensor(table[b], device=DEV)[at // self.page]
            for cache, s in ((self.k, self.ks), (self.v, self.vs)):
                x = self.values(n, s, sigma)
                cache.view(torch.uint8 if self.e4m3 else BF)[pg, :, at % self.page] = x.view(torch.uint8) if self.e4m3 else x
        self.table_list, self.table = table, i32(table)
        return self.table

    def done(self):
        assert self.ws.intact()
        kda.kda_attn_destroy(self.attn)


def check(got, want, bound, what):
    assert got.shape == want.shape
    out = (got.double() - want).abs()
    assert not torch.isnan(got.double()).any(), what
    over = (out > bound)
    worst = (out / bound.clamp(min=1e-300)).max().item()
    print(f"\n  {what}: worst {worst:.3f} of its bound")
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} outside, worst {worst:.2f} of the bound"


# ------------------------------------------------------------------ plan

PLANS = [
    dict(page=16, cache=[0], new=[1], free=4, width=2),
    dict(page=16, cache=[15, 16, 17, 0, 5], new=[1, 1, 1, 0, 0], free=9, width=4),
    dict(page=64, cache=[0, 63, 64, 100], new=[200, 1, 65, 28], free=20, width=8),
    dict(page=128, cache=[0, 0, 0], new=[0, 0, 0], free=0, width=1),
    dict(page=32, cache=[0, 10, 90, 31], new=[65, 3, 40, 2], free=4, width=8),          # the pool runs out
    dict(page=16, cache=[0, 100, 3], new=[40, 20, 4], free=50, width=7),                # the table's width runs out
    dict(page=16, cache=[-1, 5, 7], new=[2, -3, 4], free=50, width=7),                  # negative lengths
    dict(page=16, cache=[2 ** 31 - 1, 0], new=[2 ** 31 - 1, 3], free=9, width=7, rows=40),  # sums past 2^31
    dict(page=16, cache=[0, 0, 1], new=[9, 9, 9], free=9, width=7, rows=20),            # more tokens than rows
    dict(page=16, cache=[0, 0], new=[3, 4], free=9, width=7, rows=12),                  # more rows than tokens
]


def _plan(page, cache, new, free, width, rows=None, count=None, seed=3):
    B = len(cache)
    N = sum(max(n, 0) for n in new) if rows is None else rows
    rng = random.Random(seed)
    pool = list(range(1000, 1000 + max(1, free)))
    rng.shuffle(pool)
    count = free if count is None else count
    table = [[rng.randrange(0, 900) for _ in range(width)] for _ in range(B)]
    layer = Layer(1, 1, page)
    outs = {n: Guard((k,), torch.int32) for n, k in (("cu", B + 1), ("kv", B), ("info", 4))}
    outs["pos"], outs["slots"] = Guard((N,), torch.int32), Guard((N,), torch.int64)
    gt = Guard((B, width), torch.int32)
    gt.t.copy_(i32(table))
    kda.kda_attn_plan(layer.attn, B, N, i32(cache), i32(new), i32(pool), i32([count]), gt.t, outs["cu"].t,
                      outs["kv"].t, outs["pos"].t, outs["slots"].t, outs["info"].t)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    cu, kv, pos, slots, info = ref.plan(cache, new, pool, count, table, page, N)
    assert outs["cu"].t.tolist() == cu
    assert outs["kv"].t.tolist() == kv
    assert outs["info"].t.tolist() == info
    assert outs["pos"].t.tolist() == [p - 2 ** 32 if p >= 2 ** 31 else p for p in pos]
    assert outs["slots"].t.tolist() == slots
    assert gt.t.tolist() == table
    assert gt.intact() and all(g.intact() for g in outs.values())
    layer.done()
    return info


@pytest.mark.parametrize("case", PLANS, ids=lambda c: f"p{c['page']}_b{len(c['cache'])}_f{c['free']}")
def test_plan(case):
    if case["cache"][0] == 2 ** 31 - 1:
        case = dict(case, new=[5, 3])   # position past 2^31 belongs to a request that is not admitted
    _plan(**case)


@pytest.mark.parametrize("count", [-5, 0, 3, 1 << 30])
def test_plan_free_count_is_clamped(count):
    _plan(page=16, cache=[0, 20, 3], new=[40, 1, 1], free=6, width=8, count=count)


@pytest.mark.parametrize("B,page,short", [(511, 16, False), (513, 64, True), (4096, 32, True), (16384, 16, False)])
def test_plan_many_requests(B, page, short):
    rng = random.Random(B)
    cache = [rng.randrange(0, 500) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 1, rng.randrange(1, 90)]) for _ in range(B)]
    need = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(cache, new))
    info = _plan(page, cache, new, need // 2 if short else need, 64)
    assert (info[3] > 0) == short


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("N,hq,hkv,page,e4m3,rot,inter,gammas", [
    (1, 1, 1, 16, False, 128, False, "qk"),
    (3, 5, 5, 32, False, 64, True, "qk"),
    (17, 8, 2, 64, True, 96, False, "q"),
    (5, 7, 1, 128, True, 16, True, "k"),
    (33, 32, 8, 16, False, 0, False, "qk"),
    (2500, 4, 2, 16, False, 128, True, ""),
    (1301, 16, 1, 16, True, 32, False, "qk"),
    (3001, 3, 3, 64, False, 112, False, "qk"),
])
def test_append(N, hq, hkv, page, e4m3, rot, inter, gammas):
    g = torch.Generator(device=DEV).manual_seed(N)
    gam = {n: 1 + 0.3 * torch.randn(D, generator=g, device=DEV) if n in gammas else None for n in "qk"}
    layer = Layer(hq, hkv, page, e4m3, rot=rot, rope_interleaved=inter, q_gamma=gam["q"], k_gamma=gam["k"])
    pages = -(-N // page) + 2
    layer.caches(pages)
    pad = 24
    fused = torch.randn(N, (hq + 2 * hkv) * D + pad, generator=g, device=DEV).to(BF) * 3
    q, k, v = (t.unflatten(1, (-1, D)) for t in fused[:, :-pad].split([hq * D, hkv * D, hkv * D], 1))
    pos = torch.randint(0, 2 ** 31 - 1, (N,), generator=g, device=DEV).to(torch.int32)
    pos[: N // 2] %= 5000
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:N].contiguous()
    if N > 4:
        slots[N // 3] = -1
    out = Guard((N, hq, D), BF)
    before = [c.view(torch.uint8).clone() for c in (layer.k, layer.v)]
    kda.kda_attn_append(layer.attn, N, q, k, v, pos, slots, out.t)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    want, err = ref.norm_rotate(q, gam["q"], pos, inv_freq(rot) if rot else (), rot, inter, 1e-6)
    check(out.t, want, ref.UBF * want.abs() + err, "q")
    keep = slots >= 0
    pg, row = slots[keep] // page, slots[keep] % page
    want, err = ref.norm_rotate(k, gam["k"], pos, inv_freq(rot) if rot else (), rot, inter, 1e-6)
    want, err = want[keep], err[keep]
    got_k, got_v = (c.view(torch.uint8)[pg, :, row].view(c.dtype) for c in (layer.k, layer.v))
    if e4m3:
        s = layer.ks.double()[:, None]
        want, err = (want / s).clamp(-448, 448), err / s
        check(got_k.float(), want, 2.0 ** -4 * want.abs() + 2.0 ** -10 + 1.1 * err, "k")
        stored = (v[keep].float() * (1 / layer.vs)[:, None]).clamp(-448, 448).to(F8)
        assert torch.equal(got_v.view(torch.uint8), stored.view(torch.uint8))
    else:
        check(got_k, want, ref.UBF * want.abs() + err, "k")
        assert torch.equal(got_v.view(torch.int16), v[keep].contiguous().view(torch.int16))
    # Every other slot is as it was.
    for c, old in zip((layer.k, layer.v), before):
        now = c.view(torch.uint8).clone()
        now[pg, :, row] = old[pg, :, row]
        assert torch.equal(now, old)
    assert out.intact()
    layer.done()


def test_append_in_place_and_slots_outside():
    N, hq, hkv, page = 9, 4, 2, 16
    layer = Layer(hq, hkv, page, pages=2, rot=64)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(N, h, D, generator=g, device=DEV).to(BF) for h in (hq, hkv, hkv))
    pos = torch.arange(N, device=DEV, dtype=torch.int32)
    slots = torch.tensor([0, 31, 32, -2, 2 ** 40, -1, -2 ** 62, 5, 6], device=DEV)
    first = torch.empty_like(q)
    kda.kda_attn_append(layer.attn, N, q, k, v, pos, slots, first)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
    assert "outside the cache" in kda.kda_last_error_detail()
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    rows = layer.v.permute(0, 2, 1, 3).reshape(32, hkv, D)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < 32:
            assert torch.equal(rows[s], v[t])
    untouched = [s for s in range(32) if s not in (0, 31, 5, 6)]
    assert not torch.isfinite(rows[untouched].float()).any()
    slots = torch.where((slots >= 0) & (slots < 32), slots, -1)
    kda.kda_attn_append(layer.attn, N, q, k, v, pos, slots, q)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert torch.equal(q.view(torch.int16), first.view(torch.int16))
    layer.done()


@pytest.mark.parametrize("N,hq,hkv,e4m3,inter", [
    (701, 8, 2, False, False), (4999, 6, 3, True, False), (6001, 5, 1, False, True), (9002, 4, 4, True, True)])
def test_append_does_not_depend_on_the_call(N, hq, hkv, e4m3, inter):
    """A token's values are the same in a long call, whose warps' ranges cut tokens, and in short ones."""
    page = 32
    g = torch.Generator(device=DEV).manual_seed(N)
    gam = 1 + 0.3 * torch.randn(D, generator=g, device=DEV)
    layer = Layer(hq, hkv, page, e4m3, pages=-(-N // page), rot=64, rope_interleaved=inter, q_gamma=gam, k_gamma=gam)
    q, k, v = (torch.randn(N, h, D, generator=g, device=DEV).to(BF) for h in (hq, hkv, hkv))
    pos = torch.randint(0, 2 ** 31 - 1, (N,), generator=g, device=DEV).to(torch.int32)
    slots = torch.randperm(N, generator=g, device=DEV)
    out = torch.empty_like(q)
    kda.kda_attn_append(layer.attn, N, q, k, v, pos, slots, out)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    caches = [c.view(torch.uint8).clone() for c in (layer.k, layer.v)]
    again = torch.empty_like(q)
    for t in list(range(0, N, 509)) + [N - 3]:
        n = min(7, N - t)
        kda.kda_attn_append(layer.attn, n, q[t:], k[t:], v[t:], pos[t:], slots[t:], again[t:])
        assert torch.equal(again[t:t + n].view(torch.int16), out[t:t + n].view(torch.int16))
    for c, old in zip((layer.k, layer.v), caches):
        assert torch.equal(c.view(torch.uint8), old)
    layer.done()


# ------------------------------------------------------- decode, prefill

def run_attend(layer, q, kv_lens, cu=None, gate=None, f32=False, want_lse=True, stream=None):
    N, hq, _ = q.shape
    o = Guard((N, hq, D), torch.float32 if f32 else BF)
    lse = Guard((N, hq), torch.float32) if want_lse else None
    args = dict(gate_logit=gate, lse=lse.t if lse else None, stream=stream)
    if cu is None:
        kda.kda_attn_decode(layer.attn, N, q, layer.table, i32(kv_lens), o.t, layer.ws.t, **args)
    else:
        kda.kda_attn_prefill(layer.attn, len(kv_lens), N, i32(cu), q, layer.table, i32(kv_lens), o.t, layer.ws.t, **args)
    return o, lse


def verify(layer, q, kv_lens, cu=None, gate=None, f32=False, what="o"):
    o, lse = run_attend(layer, q, kv_lens, cu, gate, f32)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    want, wl, bound, lb = ref.attend(q, layer.k, layer.v, layer.table_list, kv_lens, cu, layer.page,
                                     D ** -0.5, layer.ks, layer.vs, gate)
    if not f32:
        bound = bound * (1 + ref.UBF) + ref.UBF * want.abs()
    check(o.t, want, bound, what)
    none = wl == -math.inf
    assert torch.equal(lse.t == -math.inf, none)
    check(lse.t.masked_fill(none, 0), wl.masked_fill(none, 0), lb.masked_fill(none, 1), what + " lse")
    assert bool((o.t[none] == 0).all())
    assert o.intact() and lse.intact()
    return o


def queries(layer, n, sigma=1.5):
    return (torch.randn(n, layer.hq, D, generator=layer.g, device=DEV) * sigma).to(BF)


EDGES = [1, 0, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 0, 511, 1000]


@pytest.mark.parametrize("hq,hkv,page,e4m3", [
    (1, 1, 16, False), (8, 2, 16, False), (32, 4, 32, False), (5, 1, 64, False), (16, 1, 128, False),
    (17, 1, 16, False), (40, 1, 64, False), (128, 1, 16, False), (3, 3, 16, False),
    (1, 1, 16, True), (8, 2, 32, True), (16, 1, 64, True), (24, 1, 128, True), (6, 2, 16, True), (100, 1, 16, True)])
def test_decode_lengths(hq, hkv, page, e4m3):
    layer = Layer(hq, hkv, page, e4m3, seed=hq + page)
    layer.fill(EDGES, width=70)
    verify(layer, queries(layer, len(EDGES)), EDGES)
    layer.done()


@pytest.mark.parametrize("lens,hq,hkv,page,e4m3", [
    ([1], 8, 2, 16, False), ([0], 8, 2, 16, False), ([0, 0, 0], 4, 4, 32, True), ([517], 32, 8, 16, False),
    ([40003], 16, 1, 64, False), ([30011], 8, 1, 16, True), ([9000, 1, 0, 12345], 32, 2, 128, False),
    ([700] * 300, 2, 1, 16, False), (list(range(0, 600)), 4, 2, 32, True)])
def test_decode_batches(lens, hq, hkv, page, e4m3):
    layer = Layer(hq, hkv, page, e4m3, seed=len(lens))
    layer.fill(lens)
    verify(layer, queries(layer, len(lens)), lens)
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_decode_gate(e4m3, f32):
    lens = [300, 0, 77, 1025, 4096]
    layer = Layer(24, 3, 16, e4m3)
    layer.fill(lens)
    gate = torch.randn(len(lens), 24, D, generator=layer.g, device=DEV) * 4
    verify(layer, queries(layer, len(lens)), lens, gate=gate, f32=f32)
    layer.done()


@pytest.mark.parametrize("sigma,qs", [(1e-30, 1e-30), (1.0, 60.0), (30.0, 30.0), (1e4, 1e-4)])
@pytest.mark.parametrize("prefill", [False, True])
def test_value_ranges(sigma, qs, prefill):
    """Weights from uniform to one-hot, values small and large; growing maxima along the keys."""
    lens = [900, 64, 5000]
    layer = Layer(8, 2, 16)
    layer.fill(lens, sigma=sigma)
    cu = [0, 40, 104, 174] if prefill else None
    verify(layer, queries(layer, 174 if prefill else 3, qs), lens, cu)
    layer.done()


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_growing_logits(prefill, e4m3):
    """Every key beats all keys before it by far: the running maximum changes at every step."""
    n = 1500
    layer = Layer(4, 1, 16, e4m3)
    layer.fill([n])
    ramp = (torch.arange(n, device=DEV) * 0.4).view(n, 1, 1).expand(n, 1, D) / D
    ramp = ramp / layer.ks.view(1, 1, 1) if e4m3 else ramp
    at = torch.arange(n, device=DEV)
    pg = torch.tensor(layer.table_list[0], device=DEV)[at // 16]
    x = ramp.clamp(-448, 448).to(layer.k.dtype)
    layer.k.view(torch.uint8 if e4m3 else BF)[pg, :, at % 16] = x.view(torch.uint8) if e4m3 else x
    N = 100 if prefill else 1
    q = torch.full((N, 4, D), 10.0, device=DEV).to(BF)
    q[:, 1] = -10
    verify(layer, q, [n], [0, N] if prefill else None)
    layer.done()


CHUNKS = [
    dict(new=[1], kv=[1]),
    dict(new=[5, 3, 0, 1], kv=[5, 300, 40, 77]),
    dict(new=[127, 128, 129, 2], kv=[127, 128, 129, 2]),
    dict(new=[64, 33], kv=[1000, 333]),
    dict(new=[600], kv=[2049]),
    dict(new=[7, 9, 20], kv=[0, 4, 20]),                       # rows that see no key
    dict(new=[1] * 40, kv=list(range(40))),
    dict(new=[3], kv=[20001]),
    dict(new=[300, 0, 0, 270], kv=[300, 5, 0, 4000]),
]


@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: f"n{sum(c['new'])}_l{max(c['kv'])}_b{len(c['kv'])}")
@pytest.mark.parametrize("hq,hkv,page,e4m3", [
    (1, 1, 16, False), (8, 2, 16, False), (5, 1, 32, False), (16, 2, 64, False), (128, 1, 128, False),
    (6, 2, 16, True), (8, 1, 128, True), (3, 3, 32, True), (33, 1, 16, True)])
def test_prefill(case, hq, hkv, page, e4m3):
    layer = Layer(hq, hkv, page, e4m3, seed=hq)
    layer.fill(case["kv"], width=max(1, -(-max(case["kv"]) // page)))
    cu = [0]
    for n in case["new"]:
        cu.append(cu[-1] + n)
    verify(layer, queries(layer, cu[-1]), case["kv"], cu)
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
def test_prefill_gate_f32_and_unused_rows(e4m3):
    layer = Layer(12, 3, 32, e4m3)
    kv, cu = [200, 90], [0, 130, 150]
    layer.fill(kv)
    q = queries(layer, 157)
    gate = torch.randn(157, 12, D, generator=layer.g, device=DEV) * 4
    o, lse = run_attend(layer, q, kv, cu, gate, True)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    want, wl, bound, lb = ref.attend(q[:150], layer.k, layer.v, layer.table_list, kv, cu, 32, D ** -0.5,
                                     layer.ks, layer.vs, gate[:150])
    check(o.t[:150], want, bound, "o")
    check(lse.t[:150], wl, lb, "lse")
    assert bool((o.t[150:].view(torch.uint8) == 0x5A).all()) and bool((lse.t[150:].view(torch.uint8) == 0x5A).all())
    layer.done()


def test_prefill_long_prompt():
    layer = Layer(8, 2, 16)
    layer.fill([3001])
    verify(layer, queries(layer, 3001), [3001], [0, 3001])
    layer.done()


@pytest.mark.parametrize("new,kv,hq,hkv,page,e4m3", [
    # more (token tile, key head) segments than SMs: dealt in rounds
    ([2500], [2500], 32, 16, 16, False),
    ([900, 40, 700, 1, 1100], [900, 3000, 800, 2000, 1300], 16, 8, 64, True),
    # one long segment among many short ones: the keys are cut
    ([64, 300, 300], [20000, 300, 400], 8, 4, 32, False),
    ([40] * 12 + [70], [300] * 12 + [17000], 8, 4, 16, True),
    # a long mean length with single tokens, empty requests and unseen rows among them
    ([1, 900, 0, 3, 700, 40], [3000, 900, 50, 0, 2000, 20], 8, 2, 16, False),
    ([1, 900, 0, 3, 700, 40], [3000, 900, 50, 0, 2000, 20], 8, 2, 64, True),
    ([50], [0], 4, 1, 16, False),
    # more requests than threads look at once, small and large chunks mixed
    ([(7 * i) % 50 for i in range(300)], [(7 * i) % 50 + (13 * i) % 200 for i in range(300)], 4, 1, 16, False),
])
def test_prefill_schedules(new, kv, hq, hkv, page, e4m3):
    layer = Layer(hq, hkv, page, e4m3, seed=len(new))
    layer.fill(kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    verify(layer, queries(layer, cu[-1]), kv, cu)
    layer.done()


@pytest.mark.parametrize("e4m3,page", [(False, 16), (False, 64), (True, 16), (True, 128)])
@pytest.mark.parametrize("scale", [1, 40])
def test_prefill_one_and_two_row_tiles(e4m3, page, scale):
    """Requests of up to 16 rows and of 17 to 32 side by side, in one part and in many."""
    new = [4, 5, 1, 8, 0, 2, 6, 4, 4, 7, 3, 8]
    kv = [scale * x + n for x, n in zip([31, 33, 1, 70, 9, 16, 63, 64, 0, 100, 15, 129], new)]
    layer = Layer(8, 2, page, e4m3, seed=scale)
    layer.fill(kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    verify(layer, queries(layer, cu[-1]), kv, cu)
    layer.done()


def test_prefill_e4m3_wide_queries():
    """Channels far below their row's largest, whose low bits the e4m3 parts of a
    query do not hold: a channel is off by at most 2^-17 of that largest, so a
    logit by that times the keys' absolute sum, lse by as much and a weight by the
    factor exp(twice that).  Rows with an infinity come out as NaN, alone."""
    n, kv, hq, hkv, page = 150, 700, 4, 2, 16
    layer = Layer(hq, hkv, page, True)
    layer.fill([kv])
    q = queries(layer, n).float()
    q = (q * torch.exp2(torch.randint(-14, 1, q.shape, generator=layer.g, device=DEV).float())).to(BF)
    bad = q.clone()
    bad[5, 1, 7] = math.inf
    bad[80, 2, 100] = -math.inf
    args = (layer.k, layer.v, layer.table_list, [kv], [0, n], page, D ** -0.5, layer.ks, layer.vs, None)
    want, wl, bound, lb = ref.attend(q, *args)
    pages = torch.tensor(layer.table_list[0], device=DEV)[: -(-kv // page)]
    rows = lambda c, s: (c[pages].double().transpose(0, 1).reshape(hkv, -1, D)[:, :kv] * s.double().view(hkv, 1, 1)).abs()
    keys = rows(layer.k, layer.ks).sum(-1).amax(-1).repeat_interleave(hq // hkv)       # [Hq]
    top = rows(layer.v, layer.vs).amax((1, 2)).repeat_interleave(hq // hkv)
    off = D ** -0.5 * 2.0 ** -17 * q.double().abs().amax(-1) * keys
    bound, lb = bound + (torch.expm1(2 * off) * top)[..., None], lb + off
    o, lse = run_attend(layer, q, [kv], [0, n], None, True)
    check(o.t, want, bound, "o")
    check(lse.t, wl, lb, "lse")
    o, _ = run_attend(layer, bad, [kv], [0, n], None, True)
    hit = torch.zeros(n, hq, dtype=torch.bool, device=DEV)
    hit[5, 1] = hit[80, 2] = True
    assert bool(o.t[hit].isnan().all())
    check(o.t[~hit], want[~hit], bound[~hit], "o beside NaN rows")
    layer.done()


def test_prefill_more_segments_than_are_weighed():
    """64 query heads to a key head: four tokens to a segment, 5000 segments."""
    new = [500] * 40
    layer = Layer(64, 1, 16)
    layer.fill(new)
    verify(layer, queries(layer, 20000), new, [500 * i for i in range(41)])
    layer.done()


def test_prefill_of_single_tokens_is_decode():
    """Both entry points on the same tokens, within both bounds of the same exact value."""
    lens = [400, 1, 77]
    layer = Layer(8, 2, 16)
    layer.fill(lens)
    q = queries(layer, 3)
    verify(layer, q, lens)
    verify(layer, q, lens, [0, 1, 2, 3])
    layer.done()


@pytest.mark.parametrize("prefill", [False, True])
def test_repeats_are_bit_identical_on_streams_and_in_graphs(prefill):
    lens = [3000, 17, 0, 1200]
    layer = Layer(16, 2, 16)
    layer.fill(lens)
    cu = [0, 50, 60, 60, 260] if prefill else None
    q = queries(layer, 260 if prefill else 4)
    first, _ = run_attend(layer, q, lens, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    second, _ = run_attend(layer, q, lens, cu, stream=side)
    side.synchronize()
    assert torch.equal(first.t.view(torch.int16), second.t.view(torch.int16))
    lens_t, cu_t = i32(lens), i32(cu or [0])
    o = torch.zeros(q.shape, dtype=BF, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if prefill:
            kda.kda_attn_prefill(layer.attn, 4, 260, cu_t, q, layer.table, lens_t, o, layer.ws.t)
        else:
            kda.kda_attn_decode(layer.attn, 4, q, layer.table, lens_t, o, layer.ws.t)
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first.t.view(torch.int16), o.view(torch.int16))
    # The captured call follows its lengths: shorter ones on replay.
    lens_t.copy_(i32([100, 17, 0, 300]))
    graph.replay()
    torch.cuda.synchronize()
    again, _ = run_attend(layer, q, [100, 17, 0, 300], cu)
    torch.cuda.synchronize()
    assert torch.equal(again.t.view(torch.int16), o.view(torch.int16))
    layer.done()


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_outside_the_cache_are_reported(prefill, e4m3):
    lens = [200, 300, 100]
    layer = Layer(4, 2, 16, e4m3)
    layer.fill(lens)
    cu = [0, 10, 30, 35] if prefill else None
    q = queries(layer, 35 if prefill else 3)
    good, _ = run_attend(layer, q, lens, cu)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    for bad in (-1, layer.pages, 2 ** 31 - 1, -2 ** 31):
        t = layer.table.clone()
        t[1, 3] = bad
        keep, layer.table = layer.table, t
        o, _ = run_attend(layer, q, lens, cu)
        layer.table = keep
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
        rows = [*range(10), *range(30, 35)] if prefill else [0, 2]
        assert torch.equal(o.t[rows].view(torch.int16), good.t[rows].view(torch.int16))
        assert torch.isfinite(o.t.float()).all()
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    layer.done()


def test_lengths_past_the_table_are_clamped():
    layer = Layer(4, 2, 16)
    layer.fill([64, 64])
    q = queries(layer, 2)
    full, _ = run_attend(layer, q, [64, 64])
    o, _ = run_attend(layer, q, [2 ** 31 - 1, -7])
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert torch.equal(o.t[0], full.t[0]) and bool((o.t[1] == 0).all())
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_32_bits(e4m3):
    """Pages at the far end of a cache whose element offsets pass 2^32."""
    hkv, page = 8, 128
    layer = Layer(8, hkv, page, e4m3)
    pages = (1 << 32) // (hkv * page * D) + 40
    layer.pages = pages
    layer.k, layer.v = (torch.zeros(pages, hkv, page, D, dtype=torch.uint8 if e4m3 else BF, device=DEV).view(F8 if e4m3 else BF)
                        for _ in range(2))
    kda.kda_attn_bind_cache(layer.attn, pages, layer.k, layer.v)
    n = 300
    layer.table_list = [[pages - 1, 3, pages - 20]]
    layer.table = i32(layer.table_list)
    at = torch.arange(n, device=DEV)
    slots = torch.tensor(layer.table_list[0], device=DEV)[at // page] * page + at % page
    k, v = (torch.randn(n, hkv, D, generator=layer.g, device=DEV).to(BF) for _ in range(2))
    q = queries(layer, n)
    kda.kda_attn_append(layer.attn, n, q, k, v, at.to(torch.int32), slots, q)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    if not e4m3:
        assert torch.equal(layer.v[pages - 1, :, 5], v[5])
    verify(layer, q[:1].contiguous(), [n])
    verify(layer, q, [n], [0, n])
    layer.done()


# ------------------------------------------------------------- refusals

def test_refusals_with_a_context():
    layer = Layer(4, 2, 16, pages=4)
    lib, a, n = kda.load(), layer.attn, None
    need = kda.kda_attn_workspace_bytes(a)
    launches = kda.kda_launch_count()
    bare = kda.kda_attn_create(4, 2, page_size=16, rotary_dim=0)
    INV, ALI = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_ALIGNMENT

    def dec(ctx=a, B=1, q=16, t=16, mp=1, kv=16, gate=n, o=16, lse=n, ws=16, wb=need):
        return lib.kda_attn_decode(ctx, B, q, t, mp, kv, gate, o, 0, lse, ws, wb, n)

    def pre(ctx=a, B=1, N=1, cu=16, q=16, t=16, mp=1, kv=16, gate=n, o=16, lse=n, ws=16, wb=need):
        return lib.kda_attn_prefill(ctx, B, N, cu, q, t, mp, kv, gate, o, 0, lse, ws, wb, n)

    for f in (dec, pre):
        assert f(B=0) == kda.KDA_OK and f(B=-1) == INV
        for bad in (dict(q=n), dict(t=n), dict(kv=n), dict(o=n), dict(ws=n), dict(mp=0), dict(mp=-3), dict(mp=1 << 28),
                    dict(wb=need - 1), dict(ctx=bare)):
            assert f(**bad) == INV, bad
        for bad in (dict(q=24), dict(o=8), dict(gate=20), dict(ws=8), dict(t=18), dict(kv=17), dict(lse=18)):
            assert f(**bad) == ALI, bad
    assert pre(N=0) == kda.KDA_OK and pre(N=-1) == INV and pre(cu=n) == INV and pre(cu=18) == ALI

    def app(ctx=a, N=1, q=16, qs=512, k=16, ks=256, v=16, vs=256, pos=16, sl=16, out=32):
        return lib.kda_attn_append(ctx, N, q, qs, k, ks, v, vs, pos, sl, out, n)

    assert app(N=0) == kda.KDA_OK
    for bad in (dict(N=-1), dict(q=n), dict(k=n), dict(v=n), dict(pos=n), dict(sl=n), dict(out=n), dict(qs=504),
                dict(ks=248), dict(vs=0), dict(vs=-256), dict(ctx=bare), dict(q=32, qs=520)):
        assert app(**bad) == INV, bad
    for bad in (dict(q=24), dict(k=24), dict(v=24), dict(out=24), dict(qs=516), dict(ks=260), dict(vs=258), dict(pos=18), dict(sl=20)):
        assert app(**bad) == ALI, bad

    def plan(B=1, N=1, c=16, w=16, f=16, cap=1, cnt=16, t=16, mp=1, cu=16, kv=16, pos=16, sl=16, info=16):
        return lib.kda_attn_plan(a, B, N, c, w, f, cap, cnt, t, mp, cu, kv, pos, sl, info, n)

    assert plan(B=0) == kda.KDA_OK and plan(B=16385) == kda.KDA_ERR_UNSUPPORTED
    for bad in (dict(B=-1), dict(N=-1), dict(c=n), dict(w=n), dict(f=n), dict(cap=-1), dict(cnt=n), dict(t=n), dict(mp=0),
                dict(mp=1 << 28), dict(cu=n), dict(kv=n), dict(pos=n), dict(sl=n), dict(info=n)):
        assert plan(**bad) == INV, bad
    for bad in (dict(c=18), dict(w=18), dict(f=18), dict(cnt=18), dict(t=18), dict(cu=18), dict(kv=18), dict(pos=18), dict(sl=20), dict(info=18)):
        assert plan(**bad) == ALI, bad

    assert lib.kda_attn_bind_cache(bare, 0, 16, 16) == INV
    assert lib.kda_attn_bind_cache(bare, 1 << 30, 16, 16) == INV
    assert lib.kda_attn_bind_cache(bare, 1, n, 16) == INV
    assert lib.kda_attn_bind_cache(bare, 1, 16, 24) == ALI
    assert kda.kda_launch_count() == launches
    kda.kda_attn_destroy(bare)
    layer.done()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("prefill", [False, True])
def test_a_copy_that_never_comes(prefill, e4m3, monkeypatch):
    """The bounded waits on it run out: reported once, nothing written outside, and the device works on."""
    lens, cu = [700, 300], [0, 90, 130] if prefill else None
    monkeypatch.setenv("KDA_FAULT_INJECT", "attn_drop")
    layer = Layer(8, 2, 16, e4m3)
    monkeypatch.delenv("KDA_FAULT_INJECT")
    layer.fill(lens)
    q = queries(layer, 130 if prefill else 2)
    o, lse = run_attend(layer, q, lens, cu)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_TIMEOUT
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert o.intact() and lse.intact()
    layer.done()
    again = Layer(8, 2, 16, e4m3)
    again.fill(lens)
    verify(again, queries(again, 130 if prefill else 2), lens, cu)
    again.done()


@pytest.mark.parametrize("name", ["attn_plan", "attn_append", "attn_decode", "attn_prefill", "all"])
def test_injected_launch_failure(name, monkeypatch):
    monkeypatch.setenv("KDA_FAULT_INJECT", name)
    layer = Layer(4, 2, 16)
    layer.fill([20])
    monkeypatch.delenv("KDA_FAULT_INJECT")
    q = queries(layer, 1)
    o = torch.full_like(q, 7.0)
    k = torch.ones(1, 2, D, dtype=BF, device=DEV)
    one, slots = i32([1]), torch.zeros(1, dtype=torch.int64, device=DEV)
    calls = {
        "attn_plan": lambda: kda.kda_attn_plan(layer.attn, 1, 1, one, one, one, one, layer.table.clone(), i32([0, 0]), i32([0]), i32([0]), slots.clone(), i32([0] * 4)),
        "attn_append": lambda: kda.kda_attn_append(layer.attn, 1, q, k, k, one, slots, o),
        "attn_decode": lambda: kda.kda_attn_decode(layer.attn, 1, q, layer.table, i32([20]), o, layer.ws.t),
        "attn_prefill": lambda: kda.kda_attn_prefill(layer.attn, 1, 1, i32([0, 1]), q, layer.table, i32([20]), o, layer.ws.t),
    }
    for which, call in calls.items():
        if name in (which, "all"):
            o.fill_(7.0)
            before = kda.kda_launch_count()
            with pytest.raises(kda.KDAError) as ei:
                call()
            assert ei.value.status == kda.KDA_ERR_CUDA and "injected" in kda.kda_last_error_detail()
            assert kda.kda_launch_count() == before
            torch.cuda.synchronize()
            assert bool((o == 7.0).all())
        else:
            call()
    layer.done()
