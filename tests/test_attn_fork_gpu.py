"""Forked, released and copied pages on a GB300, against the fork's plain form."""
import math
import random

import pytest
import torch

import fork_ref
import kda_delta_rule_token_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
BF = torch.bfloat16
F8 = torch.float8_e4m3fn


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Layer:
    def __init__(self, pages, hkv=1, page=16, e4m3=False, seed=0):
        self.scale = torch.ones(hkv, device=DEV)
        self.attn = kda.kda_attn_create(hkv, hkv, page_size=page, rotary_dim=0, k_scale=self.scale, v_scale=self.scale,
                                        cache_type=kda.KDA_CACHE_E4M3 if e4m3 else kda.KDA_CACHE_BF16)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.raw = torch.randint(0, 256, (2, pages, hkv, page, D * (1 if e4m3 else 2)), generator=gen, device=DEV, dtype=torch.uint8)
        self.pages, self.page = pages, page
        self.k, self.v = (self.raw[i].view(F8 if e4m3 else BF) for i in range(2))
        kda.kda_attn_bind_cache(self.attn, pages, self.k, self.v)

    def done(self):
        kda.kda_attn_destroy(self.attn)


class Guarded:
    """int32 outputs between guards."""

    def __init__(self, *shape, fill=-77):
        n = math.prod(shape)
        self.buf = torch.full((n + 128,), 0x5A5A5A5A, dtype=torch.int32, device=DEV)
        self.t = self.buf[64:64 + n].view(*shape)
        self.t.fill_(fill)

    def intact(self):
        return bool((self.buf[:64] == 0x5A5A5A5A).all()) and bool((self.buf[-64:] == 0x5A5A5A5A).all())


def call(layer, rows, lens, table, refs, free, count, pitch=None, status=kda.KDA_OK, stream=None):
    """One call and its plain form, compared; returns the plain form's outputs as lists."""
    B, width = len(rows), len(table[0])
    pitch = pitch or width
    old = torch.full((B, pitch), 2 ** 30, dtype=torch.int32, device=DEV)
    old[:, :width] = i32(table)
    new, nl, src, dst, cr, info = (Guarded(*s) for s in ((B, pitch), (B,), (B,), (B,), (B,), (4,)))
    g_refs, g_free = Guarded(len(refs)), Guarded(max(1, len(free)))
    g_refs.t.copy_(i32(refs))
    g_free.t[:len(free)] = i32(free)
    ws = Guarded(kda.kda_attn_fork_workspace_bytes(layer.attn, B, width) // 4, fill=-1)
    kda.kda_attn_fork(layer.attn, B, i32(rows), i32(lens), old[:, :width], g_refs.t, g_free.t, i32([count]), new.t[:, :width], nl.t,
                      src.t, dst.t, cr.t, info.t, ws.t, free_capacity=len(free), stream=stream) if pitch == width else \
        kda.kda_attn_fork(layer.attn, B, i32(rows), i32(lens), old, g_refs.t, g_free.t, i32([count]), new.t, nl.t, src.t, dst.t, cr.t,
                          info.t, Guarded(kda.kda_attn_fork_workspace_bytes(layer.attn, B, pitch) // 4).t, free_capacity=len(free))
    assert kda.kda_attn_sync_status(layer.attn, stream) == status
    assert all(x.intact() for x in (new, nl, src, dst, cr, info, g_refs, g_free, ws))
    want_table = [[-77] * pitch for _ in range(B)]
    want_refs, want_free = list(refs), list(free)
    wide = [r + [2 ** 30] * (pitch - width) for r in table]
    want_lens, copies, want_info = fork_ref.fork(rows, lens, wide, want_refs, want_free, count, want_table, layer.page)
    assert info.t.tolist() == want_info
    assert nl.t.tolist() == want_lens
    assert list(zip(src.t.tolist(), dst.t.tolist(), cr.t.tolist())) == copies
    assert g_refs.t.tolist() == want_refs
    assert g_free.t[:len(free)].tolist() == want_free
    got = new.t.tolist()
    for b, r in enumerate(rows):
        if 0 <= r < B and want_lens[b] == 0 and lens[r] > 0:
            continue   # a refused request's row says nothing
        assert got[b] == want_table[b], b
    return want_table, want_lens, want_refs, want_free, copies, want_info


def holders(table, lens, page, pages):
    held = [0] * pages
    for row, n in zip(table, lens):
        for x in row[: -(-n // page)]:
            held[x] += 1
    return held


class Model:
    """Requests that grow and fork, by the plain form alone."""

    def __init__(self, B, width, page, pages, seed):
        self.rng = random.Random(seed)
        self.B, self.width, self.page, self.pages = B, width, page, pages
        self.free = list(range(pages))
        self.rng.shuffle(self.free)
        self.count = pages
        self.table, self.lens, self.refs = [[-1] * width for _ in range(B)], [0] * B, [0] * pages

    def grow(self, b, n):
        need = -(-(self.lens[b] + n) // self.page) - -(-self.lens[b] // self.page)
        if self.lens[b] + n > self.width * self.page or need > self.count:
            return
        at = -(-self.lens[b] // self.page)
        for i in range(need):
            self.count -= 1
            self.table[b][at + i] = self.free[self.count]
        self.lens[b] += n

    def step(self, layer, rows, **more):
        self.table, self.lens, self.refs, self.free, copies, info = call(layer, rows, self.lens, self.table, self.refs, self.free, self.count, **more)
        self.count = info[2]
        held = holders(self.table, self.lens, self.page, self.pages)
        assert [max(h - 1, 0) for h in held] == self.refs
        assert sorted(self.free[:self.count]) == [p for p, h in enumerate(held) if h == 0]
        return copies, info


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,width,seed", [(1, 1, 0), (2, 3, 1), (4, 40, 2), (9, 33, 3), (33, 70, 4), (70, 5, 5), (256, 9, 6), (300, 34, 7), (6, 256, 8), (6, 257, 9)])
def test_requests_that_grow_and_fork(B, width, page, seed):
    m = Model(B, width, page, B * width, seed)
    layer = Layer(m.pages, page=page)
    for turn in range(6):
        for b in range(B):
            if turn < 2 or m.lens[b]:
                m.grow(b, m.rng.choice([0, 1, page - 1, page, 2 * page + 3, m.rng.randint(1, width * page)]))
        kind = m.rng.choice(["any", "beams", "one", "same"])
        if kind == "any":
            rows = [m.rng.randint(-1, B - 1) for _ in range(B)]
        elif kind == "one":
            rows = [m.rng.randrange(B)] * B
        elif kind == "same":
            rows = list(range(B))
        else:
            stay = [b for b in range(B) if m.rng.random() < 0.6] or [0]
            rows = [b if b in stay else m.rng.choice(stay + [-1]) for b in range(B)]
        m.step(layer, rows)
    m.step(layer, [-1] * B)
    assert m.count == m.pages
    layer.done()


def test_prompt_kept_by_somebody_else():
    """A page that is held outside of the table is not freed."""
    layer = Layer(8)
    table, refs = [[3, 4, -1], [3, 5, -1]], [0, 0, 0, 2, 0, 0, 0, 0]
    out = call(layer, [-1, -1], [20, 32], table, refs, [0, 1, 2, 6, 7, -1, -1, -1], 5)
    assert out[2][3] == 0 and out[3][:7] == [0, 1, 2, 6, 7, 4, 5] and out[5] == [2, 0, 7, 0]
    layer.done()


@pytest.mark.parametrize("have", [0, 1, 2, 5])
def test_pages_run_short(have):
    """Requests whose copies find no page hold nothing; freed pages count."""
    page, B = 16, 7
    layer = Layer(40)
    table = [[10 + b, 20 + b, 30 + b] for b in range(B)]
    lens = [33, 40, 17, 48, 5, 1, 0]
    rows = [0, 0, 0, 3, 3, 0, 3]          # three copies of request 0's last page; 1, 2, 4 and 5 end
    _, _, refs, _, _, info = call(layer, rows, lens, table, [0] * 40, list(range(8)) + [-1] * 32, have)
    assert info[0] == 3 + 2 + 1 + 1 and info[3] == 0
    rows, lens = [0, 0, 0, 0, 0, 0, 0], [33, 0, 0, 0, 0, 0, 0]
    _, new_lens, refs, _, _, info = call(layer, rows, lens, table, [0] * 40, list(range(8)) + [-1] * 32, have)
    assert info[3] == 6 - have and sum(n > 0 for n in new_lens) == have + 1 and refs[10] == refs[20] == have
    layer.done()


def test_rows_that_there_are_not():
    layer = Layer(20)
    table = [[b, 5 + b] for b in range(5)]
    call(layer, [0, 5, -2, 2 ** 31 - 1, 0], [20, 16, 3, 32, 9], table, [0] * 20, [10, 11, 12] + [-1] * 17, 3, status=kda.KDA_ERR_INVALID_ARG)
    layer.done()


def test_pages_outside_the_cache():
    """Copied as they are, counted nowhere; a copy from or to one is no copy."""
    layer = Layer(20)
    for bad in (-1, 20, 2 ** 31 - 1, -2 ** 31):
        table = [[bad, 5], [1, bad], [2, 7]]
        for rows in ([0, 0, 2], [1, 1, 2], [2, 2, 2]):
            call(layer, rows, [32, 32, 32], table, [0] * 20, [10, 11] + [-1] * 18, 2, status=kda.KDA_ERR_INVALID_ARG)
        call(layer, [2, 1, 2], [0, 16, 20], table, [0] * 20, [10, bad] + [-1] * 18, 2, status=kda.KDA_ERR_INVALID_ARG)
    layer.done()


def test_lengths_are_clamped():
    layer = Layer(20)
    call(layer, [0, 1, 0], [2 ** 31 - 1, -5, 40], [[1, 2], [3, 4], [5, 6]], [0] * 20, [10] + [-1] * 19, 1)
    layer.done()


def test_holders_miscounted():
    """Two requests let go of a page that one is said to hold: freed once, and reported."""
    layer = Layer(20)
    B = 2
    refs, free, new = i32([0] * 20), i32([9] + [-1] * 19), torch.full((B, 1), -1, dtype=torch.int32, device=DEV)
    outs = [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(4)]
    info = i32([0] * 4)
    ws = torch.empty(kda.kda_attn_fork_workspace_bytes(layer.attn, B, 1), dtype=torch.uint8, device=DEV)
    kda.kda_attn_fork(layer.attn, B, i32([-1, -1]), i32([16, 16]), i32([[4], [4]]), refs, free, i32([1]), new, *outs, info, ws)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
    assert info.tolist() == [1, 0, 2, 0] and free.tolist()[:3] == [9, 4, -1] and refs.tolist() == [0] * 20
    # No room for what is freed.
    kda.kda_attn_fork(layer.attn, B, i32([-1, -1]), i32([16, 16]), i32([[4], [5]]), refs, free, i32([1]), new, *outs, info, ws, free_capacity=2)
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
    assert info.tolist() == [2, 0, 2, 0] and free.tolist()[:3] == [9, 4, -1]
    layer.done()


@pytest.mark.parametrize("B", [1000, 3000])
def test_many_requests(B):
    """All of one prompt, most of which end at once."""
    page, rng = 16, random.Random(B)
    layer = Layer(B + 20, page=page)
    table = [[0, 1, 2, 10 + b] for b in range(B)]
    refs = [B - 1] * 3 + [0] * (B + 17)
    free = [3, 4, 5, 6, 7, 8, 9] + [-1] * (B + 13)
    stay = sorted(rng.sample(range(B), 11))
    rows = [rng.choice(stay) if rng.random() < 0.3 else -1 for _ in range(B)]
    call(layer, rows, [3 * page + 1 + b % page for b in range(B)], table, refs, free, 7)
    layer.done()


def test_wide_table_and_stream():
    B, width, page = 5, 3001, 16
    layer = Layer(B * width, page=page)
    order = list(range(B * width))
    random.Random(1).shuffle(order)
    table = [order[b * width:(b + 1) * width] for b in range(B)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        call(layer, [1, 1, 3, 3, -1], [width * page, 40000, 17, width * page - 1, 31], table, [0] * (B * width), [-1] * (B * width), 0, stream=stream)
    call(layer, [1, 1, 3, 3, -1], [200, 400, 17, 333, 31], [t[:30] for t in table], [0] * (B * width), [-1] * (B * width), 0, pitch=64)
    layer.done()


# ---------------------------------------------------------------- copies


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv,page", [(1, 16), (3, 32), (8, 64), (2, 128), (16, 16)])
def test_copy(hkv, page, e4m3):
    layer = Layer(50, hkv, page, e4m3, seed=page)
    order = torch.randperm(50, generator=torch.Generator().manual_seed(page)).tolist()
    n = 20
    src, dst = order[:n], order[n:2 * n]
    src[3] = -1
    src[4] = src[5]                                  # one page to two
    rows = [random.Random(i).randint(1, page) for i in range(n)]
    rows[0], rows[1], rows[2], rows[6] = page, 0, -3, page + 9
    want = layer.raw.clone()
    for s, d, r in zip(src, dst, rows):
        if s >= 0:
            r = min(max(r, 0), page)
            want[:, d, :, :r] = layer.raw[:, s, :, :r]
    kda.kda_attn_copy_pages(layer.attn, n, i32(src), i32(dst), i32(rows))
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
    assert torch.equal(layer.raw, want)
    layer.done()


@pytest.mark.parametrize("bad", [-2, 50, 2 ** 31 - 1, -2 ** 31])
def test_copy_outside_the_cache(bad):
    layer = Layer(50)
    want = layer.raw.clone()
    want[:, 7, :, :5] = layer.raw[:, 3, :, :5]
    kda.kda_attn_copy_pages(layer.attn, 3, i32([bad, 3, 4]), i32([1, 7, bad]), i32([16, 5, 16]))
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(layer.raw, want)
    kda.kda_attn_copy_pages(layer.attn, 1, i32([4]), i32([-1]), i32([16]))
    assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_ERR_INVALID_ARG
    layer.done()


def test_captured():
    """Two forks and their copies in graphs over one workspace, replayed in turn."""
    page, B = 16, 3
    layers, graphs, outs = [], [], []
    ws = None
    for seed in (0, 1):
        layer = Layer(30, page=page, seed=seed)
        before = layer.raw.clone()
        table, lens, rows = [[0, 1], [2, 3], [4, 5]], [20 + seed, 17, 32], [0, 0, 2 - seed]
        args = [i32(rows), i32(lens), i32(table), i32([0] * 30), i32([10, 11, 12] + [-1] * 27), i32([3])]
        new = torch.full((B, 2), -77, dtype=torch.int32, device=DEV)
        small = [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(4)] + [i32([0] * 4)]
        if ws is None:
            ws = torch.empty(kda.kda_attn_fork_workspace_bytes(layer.attn, B, 2), dtype=torch.uint8, device=DEV)
        zero = torch.zeros_like(args[3])
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            args[3].copy_(zero)
            kda.kda_attn_fork(layer.attn, B, *args, new, *small, ws)
            kda.kda_attn_copy_pages(layer.attn, B, *small[1:4])
        layers.append((layer, before))
        graphs.append(g)
        outs.append((new, small, args, rows, lens, table))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (layer, before), (new, small, args, rows, lens, table) in zip(layers, outs):
        refs, free, want = [0] * 30, [10, 11, 12] + [-1] * 27, [[-77] * 2 for _ in range(B)]
        new_lens, copies, info = fork_ref.fork(rows, lens, table, refs, free, 3, want, page)
        assert new.tolist() == want and small[0].tolist() == new_lens and small[4].tolist() == info and args[3].tolist() == refs
        for s, d, r in copies:
            if s >= 0:
                before[:, d, :, :r] = before[:, s, :, :r]
        assert torch.equal(before, layer.raw)
        assert kda.kda_attn_sync_status(layer.attn) == kda.KDA_OK
        layer.done()


def test_refusals():
    layer = Layer(8)
    B = 2
    args = dict(rows=i32([0, 1]), kv_lens=i32([1, 1]), block_table=i32([[0], [1]]), page_refs=i32([0] * 8), free_pages=i32([2, 3]),
                free_count=i32([2]), new_table=i32([[7], [7]]), new_lens=i32([7, 7]), copy_src=i32([7, 7]), copy_dst=i32([7, 7]),
                copy_rows=i32([7, 7]), info=i32([7] * 4), workspace=torch.empty(1 << 12, dtype=torch.uint8, device=DEV))

    def refused(status, B=2, **change):
        before = kda.kda_launch_count()
        with pytest.raises(kda.KDAError) as e:
            kda.kda_attn_fork(layer.attn, B, **{**args, **change})
        assert e.value.status == status and kda.kda_launch_count() == before

    bad, align = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_ALIGNMENT
    refused(bad, B=-1)
    refused(bad, new_table=args["block_table"])
    refused(bad, new_lens=args["kv_lens"])
    refused(bad, workspace=args["workspace"][:32])
    refused(bad, max_pages=0)
    refused(bad, max_pages=2 ** 28)
    refused(align, workspace=args["workspace"][4:])
    odd = torch.zeros(64, dtype=torch.uint8, device=DEV)
    refused(align, free_count=odd[2:].data_ptr())
    many = 16385
    wide = dict(rows=i32([0] * many), kv_lens=i32([0] * many), block_table=i32([[0]] * many), new_table=i32([[0]] * many),
                new_lens=i32([0] * many), copy_src=i32([0] * many), copy_dst=i32([0] * many), copy_rows=i32([0] * many))
    refused(kda.KDA_ERR_UNSUPPORTED, B=many, **wide)
    kda.kda_attn_fork(layer.attn, 0, **args)
    with pytest.raises(ValueError):
        kda.kda_attn_fork(layer.attn, B, **{**args, "new_table": i32([[7, 7], [7, 7]])})
    with pytest.raises(ValueError):
        kda.kda_attn_fork(layer.attn, B, **{**args, "rows": torch.zeros(2, dtype=torch.int64, device=DEV)})
    for n, change in ((-1, {}), (1, dict(src=odd[2:].data_ptr()))):
        with pytest.raises(kda.KDAError):
            kda.kda_attn_copy_pages(layer.attn, n, **{**dict(src=i32([0]), dst=i32([1]), rows=i32([1])), **change})
    kda.kda_attn_copy_pages(layer.attn, 0, i32([0]), i32([1]), i32([1]))
    fresh = kda.kda_attn_create(1, 1, page_size=16, rotary_dim=0)   # no cache bound
    with pytest.raises(kda.KDAError):
        kda.kda_attn_fork(fresh, B, **args)
    with pytest.raises(kda.KDAError):
        kda.kda_attn_copy_pages(fresh, 1, i32([0]), i32([1]), i32([1]))
    kda.kda_attn_destroy(fresh)
    layer.done()


@pytest.mark.parametrize("name", ["attn_fork", "attn_copy_pages", "all"])
def test_injected_launch_failure(name, monkeypatch):
    monkeypatch.setenv("KDA_FAULT_INJECT", name)
    layer = Layer(8)
    monkeypatch.delenv("KDA_FAULT_INJECT")
    before = layer.raw.clone()
    small = [i32([7]) for _ in range(4)] + [i32([7] * 4)]
    ws = torch.empty(1 << 12, dtype=torch.uint8, device=DEV)
    calls = {"attn_fork": lambda: kda.kda_attn_fork(layer.attn, 1, i32([0]), i32([3]), i32([[0]]), i32([0] * 8), i32([1]), i32([1]), i32([[7]]), *small, ws),
             "attn_copy_pages": lambda: kda.kda_attn_copy_pages(layer.attn, 1, i32([0]), i32([1]), i32([16]))}
    for which, fn in calls.items():
        launches = kda.kda_launch_count()
        if name in (which, "all"):
            with pytest.raises(kda.KDAError) as e:
                fn()
            assert e.value.status == kda.KDA_ERR_CUDA and "injected" in kda.kda_last_error_detail()
            assert kda.kda_launch_count() == launches
            torch.cuda.synchronize()
            assert which != "attn_fork" or all(bool((t == 7).all()) for t in small)
            assert which != "attn_copy_pages" or torch.equal(before, layer.raw)
    layer.done()
