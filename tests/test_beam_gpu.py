"""Beam selection and the reordering of states on a GB300, against the formulas in 64 bits."""
import math

import pytest
import torch

import beam_ref
import kda_delta_rule_token_gb300 as kda

pytestmark = pytest.mark.gpu

DEV = "cuda"
D = 128
# A row's lse: terms in fp32 are off by their exponent's two roundings (2^-24 of it, which
# counts for terms within 2^-20 of the largest: exponents to 29), ex2's 2^-22, and the sum's.
SLACK = (29 * 2 + 4 + 4) * 2.0 ** -24


class Ctx:
    def __init__(self, heads=1):
        self.params = (torch.zeros(3, heads * D, 4, device=DEV), torch.zeros(heads, D, device=DEV),
                       torch.zeros(heads, D, device=DEV), torch.ones(heads, D, device=DEV))
        self.ctx = kda.kda_create(heads, *self.params)

    def __enter__(self):
        return self.ctx

    def __exit__(self, *_):
        kda.kda_destroy(self.ctx)


def select(ctx, logits, scores, num, done=None, end=0, keep=False, stream=None, ws=None):
    G, K = scores.shape
    if ws is None:
        ws = torch.full((kda.kda_beam_select_workspace_bytes(ctx, G, K, logits.shape[1], num),), 0xff, dtype=torch.uint8, device=DEV)
    guard = 37
    out = [torch.full((G * num + 2 * guard,), 77, dtype=t, device=DEV) for t in (torch.float32, torch.int32, torch.int32)]
    inner = [t[guard:guard + G * num].view(G, num) for t in out]
    kda.kda_beam_select(ctx, G, K, logits, scores, num, *inner, ws, done=done, end_token=end, keep_places=keep, stream=stream)
    torch.cuda.synchronize()
    for t in out:
        assert bool((t[:guard] == 77).all()) and bool((t[-guard:] == 77).all())
    return inner


def run(logits, scores, num, done=None, end=0, keep=False, slack=SLACK):
    with Ctx() as ctx:
        got = select(ctx, logits, scores, num, done, end, keep)
        assert kda.kda_sync_status(ctx) == kda.KDA_OK
    beam_ref.check([t.cpu() for t in got], beam_ref.scores64(logits, scores, done, end).cpu(), num, keep, slack)
    return got


def make(G, K, V, bf16=False, seed=0, scale=3.0, pad=0, shift=0):
    """Logits in rows V + pad apart, `shift` elements behind an aligned address."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.full((G * K * (V + pad) + shift + 64,), math.nan, device=DEV)
    if bf16:
        buf = buf.to(torch.bfloat16)
    x = buf[shift:shift + G * K * (V + pad)].view(G * K, V + pad)[:, :V]
    x.copy_(scale * torch.randn(G * K, V, generator=gen, device=DEV))
    scores = -10 * torch.rand(G, K, generator=gen, device=DEV)
    return x, scores


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("G,K,V,num", [
    (1, 1, 1, 1), (1, 1, 2, 2), (2, 3, 1, 3), (3, 1, 5, 5), (1, 4, 17, 4), (5, 2, 63, 64), (2, 4, 255, 8), (1, 64, 64, 64),
    (3, 5, 1000, 5), (1, 4, 4095, 8), (2, 3, 4096, 7), (2, 2, 4097, 4), (1, 8, 8193, 16), (2, 7, 32000, 7),
    (1, 32, 50001, 64), (1, 1, 262143, 64), (9, 8, 131071, 8), (1, 64, 20000, 1), (70, 4, 700, 4), (300, 3, 4100, 3)])
def test_sizes(G, K, V, num, bf16):
    x, scores = make(G, K, V, bf16, seed=V + num)
    run(x, scores, num, keep=num == K)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 2), (5, 7), (8, 4), (13, 3)])
@pytest.mark.parametrize("V", [3, 4099, 9001])
def test_strides_and_alignment(V, pad, shift, bf16):
    x, scores = make(2, 3, V, bf16, seed=pad + shift, pad=pad, shift=shift)
    run(x, scores, 6)


@pytest.mark.parametrize("keep", [False, True])
def test_done_beams(keep):
    x, scores = make(6, 4, 5000, seed=3)
    done = torch.tensor([[0, 0, 0, 0], [1, 0, 0, 0], [0, 1, 1, 0], [1, 1, 1, 1], [0, 0, 0, 1], [1, 0, 1, 1]], dtype=torch.uint8, device=DEV)
    scores[2, 1] = 5.0   # stays ahead of all others
    scores[4, 3] = -math.inf
    x[4:8] = math.nan    # of beams, one of which is done: not read there
    run(x, scores, 4, done, 17, keep)
    run(x, scores, 4, done.bool(), 4999, keep)
    if not keep:
        run(x, scores, 9, done, 0)


def test_first_step():
    """Beams that are still alike: all of one row."""
    x, scores = make(3, 4, 3001, seed=5)
    x[:] = x[::4].repeat_interleave(4, 0)
    scores[:] = -math.inf
    scores[:, 0] = 0
    _, tokens, rows = run(x, scores, 4, keep=True)
    assert bool((rows == torch.arange(0, 12, 4, device=DEV)[:, None]).all())
    assert torch.equal(tokens[:, 0].long(), x[::4].argmax(1))


@pytest.mark.parametrize("V", [300, 4096, 30000])
@pytest.mark.parametrize("kind", ["same", "few", "rising", "falling", "steps", "open", "lowest", "zeros"])
def test_orders_and_ties(kind, V):
    """Equal logits in number, and orders in which every logit passes the ones before it."""
    x, scores = make(2, 4, V, seed=8)
    i = torch.arange(V, device=DEV, dtype=torch.float32)
    if kind == "same":
        x[:] = 0.5
    elif kind == "few":
        x[:] = (x / 3).round()
    elif kind == "rising":
        x[:] = i / 64
    elif kind == "falling":
        x[:] = -i / 64
    elif kind == "steps":
        x[:] = (i / 97).floor()
    elif kind == "open":     # a grammar leaves six tokens open, another row none
        x.masked_fill_(torch.rand(x.shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV) * V > 6, -math.inf)
        x[3] = -math.inf
    elif kind == "lowest":
        x[:, 5:] = torch.finfo(torch.float32).min
    else:
        x[:] = torch.where(i.long() % 2 == 0, 0.0, -0.0)
    run(x, scores, 8)
    run(x, scores, 4, keep=True)
    scores[:] = -3.0         # equal beams as well
    if kind != "lowest":
        run(x[:1].expand(8, V).contiguous(), scores, 8)


@pytest.mark.parametrize("V", [40, 6000])
def test_nan_and_infinities(V):
    x, scores = make(5, 2, V, seed=9)
    x[0, V // 2] = math.nan            # the row offers nothing
    x[2, 1] = math.inf
    x[3] = -math.inf
    x[4:6] = math.nan                  # nor does the group
    scores[3] = torch.tensor([math.nan, -math.inf], device=DEV)
    scores[4, 0] = math.inf
    s, t, r = run(x, scores, 3)
    assert s[2].tolist() == [-math.inf] * 3 and t[2].tolist() == [0, 1, 2] and r[2].tolist() == [4] * 3
    assert s[3].tolist() == [-math.inf] * 3


def test_wide_ranges():
    """Logits of 1e4 and more beside small ones, whole tiles of masked ones first."""
    x, scores = make(2, 3, 20000, seed=11)
    x[:, :9000] = -1e4
    x[1, 15000] = 3e4
    x[2] *= 1e4
    x[3] += 1e6
    x[4, :8192] = -math.inf
    # Logits up to 1e6 and distances of up to 1e5 from a row's largest, which are exact or rounded once.
    run(x, scores, 6, slack=SLACK)


def test_large_vocabulary_of_many_rows():
    x, scores = make(64, 8, 131072, seed=12)
    run(x, scores, 8, keep=True)


@pytest.mark.parametrize("kind", ["random", "ascending", "descending"])
def test_long_segments(kind):
    """Rows of which a CTA has 44 tiles, 64 candidates and more from every look: its list is brought down in between."""
    G, K, V, num = 80, 8, 41 * 4096 + 7, 64
    x, scores = make(G, K, V, seed=3, scale=2.0)
    if kind != "random":
        ramp = torch.arange(V, device=DEV) * 2e-4
        x.copy_(ramp if kind == "ascending" else ramp.flip(0))
        x.add_(torch.arange(G * K, device=DEV)[:, None] * 7e-5)
    with Ctx() as ctx:
        got = select(ctx, x, scores, num)
        assert kda.kda_sync_status(ctx) == kda.KDA_OK
    for g in range(G):
        y = beam_ref.scores64(x[g * K:(g + 1) * K], scores[g:g + 1], None, 0)
        s, k, v = (t[0] for t in beam_ref.best(y, num + 1))
        assert bool(((got[0][g].double() - s[:num]).abs() <= SLACK + 2.0 ** -23 * s[:num].abs()).all()), g
        apart = torch.cat([torch.ones(1, dtype=torch.bool, device=DEV), s[:-1] - s[1:] > 2 * SLACK])
        sure = apart[:-1] & apart[1:]
        assert bool(((got[1][g] == v[:num]) & (got[2][g] == k[:num] + g * K))[sure].all()), g


@pytest.mark.parametrize("bf16", [False, True])
def test_many_small_groups(bf16):
    """More rows than CTAs by far."""
    G, K, V, num = 20011, 2, 5, 3
    x, scores = make(G, K, V, bf16, seed=5)
    with Ctx() as ctx:
        got = select(ctx, x, scores, num)
    y = beam_ref.scores64(x, scores, None, 0)
    s, k, v = beam_ref.best(y, num)
    assert bool(((got[0].double() - s).abs() <= SLACK + 2.0 ** -23 * s.abs()).all())
    # Neighbours of different beams that are further apart than their scores may be off have the formula's place.
    s4 = beam_ref.best(y, num + 1)[0]
    apart = torch.cat([torch.ones_like(s4[:, :1], dtype=torch.bool), (s4[:, :-1] - s4[:, 1:]) > 2 * SLACK], 1)
    sure = apart[:, :-1] & apart[:, 1:]
    rows = k + torch.arange(G, device=DEV)[:, None] * K
    assert bool(((got[1] == v) & (got[2] == rows))[sure].all()) and float(sure.float().mean()) > 0.9


def test_result_does_not_depend_on_the_run():
    x, scores = make(3, 8, 70001, bf16=True, seed=13)
    with Ctx() as ctx:
        one = select(ctx, x, scores, 16)
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(one, select(ctx, x, scores, 16)))


def test_captured_and_on_another_stream():
    """Two graphs over one workspace, replayed in turn, on a stream of their own."""
    xs = [make(2, 4, 9000, seed=s) for s in (20, 21)]
    stream = torch.cuda.Stream()
    with Ctx() as ctx:
        ws = torch.empty(kda.kda_beam_select_workspace_bytes(ctx, 2, 4, 9000, 4), dtype=torch.uint8, device=DEV)
        outs, graphs = [], []
        for x, scores in xs:
            out = [torch.zeros(2, 4, dtype=t, device=DEV) for t in (torch.float32, torch.int32, torch.int32)]
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=stream):
                kda.kda_beam_select(ctx, 2, 4, x, scores, 4, *out, ws, keep_places=True)
            outs.append(out)
            graphs.append(g)
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for (x, scores), out in zip(xs, outs):
            beam_ref.check([t.cpu() for t in out], beam_ref.scores64(x, scores, None, 0).cpu(), 4, True, SLACK)


def test_select_refusals():
    x, scores = make(2, 4, 100)
    with Ctx() as ctx:
        out = lambda n: [torch.full((2, n), 7, dtype=t, device=DEV) for t in (torch.float32, torch.int32, torch.int32)]  # noqa: E731
        ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

        def refused(status, o, *args, **more):
            before = kda.kda_launch_count()
            with pytest.raises(kda.KDAError) as e:
                kda.kda_beam_select(ctx, *args, *o, **{"workspace": ws, **more})
            assert e.value.status == status and kda.kda_launch_count() == before
            assert all(bool((t == 7).all()) for t in o)

        bad, align, unsupported = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_ALIGNMENT, kda.KDA_ERR_UNSUPPORTED
        refused(bad, out(4), -1, 4, x, scores, 4)
        refused(bad, out(4), 2, 0, x, scores, 4)
        refused(bad, out(0), 2, 4, x, scores, 0)
        refused(bad, out(3), 2, 4, x, scores, 3, keep_places=True)
        done = torch.zeros(2, 4, dtype=torch.uint8, device=DEV)
        refused(bad, out(4), 2, 4, x, scores, 4, done=done, end_token=100)
        refused(bad, out(4), 2, 4, x, scores, 4, done=done, end_token=-1)
        refused(bad, out(9), 2, 4, x[:, :2], scores, 9)
        refused(bad, out(4), 2, 4, x, scores, 4, workspace=ws[:16])
        refused(align, out(4), 2, 4, x, scores, 4, workspace=ws[8:])
        refused(unsupported, out(65), 2, 4, x, scores, 65)
        refused(unsupported, out(4), 1, 65, x.repeat(9, 1), scores.repeat(9, 1), 4)
        assert kda.kda_beam_select_workspace_bytes(ctx, 2, 65, 100, 4) == 0
        assert kda.kda_beam_select_workspace_bytes(ctx, 0, 4, 100, 4) == 0
        # Parts of rows are numbered in 32 bits, up to two for each row.
        for groups, beams in ((2 ** 30 + 1, 1), (2 ** 24 + 1, 64), (2 ** 31 - 1, 1)):
            assert kda.kda_beam_select_workspace_bytes(ctx, groups, beams, 8, 1) == 0
            assert kda.load().kda_beam_select(ctx, groups, beams, 8, x.data_ptr(), 0, 8, scores.data_ptr(), None, 0, 1, 0, 16, 16, 16,
                                              ws.data_ptr(), 1 << 62, None) == bad
        assert kda.kda_beam_select_workspace_bytes(ctx, 2 ** 30, 1, 8, 1) > 2 ** 34
        kda.kda_beam_select(ctx, 0, 4, x, scores, 4, *out(4), ws)
        for wrong in (dict(scores=scores.double()), dict(done=done.int()), dict(logits=x.t()), dict(scores=scores[:1])):
            args = {"logits": x, "scores": scores, **wrong}
            with pytest.raises(ValueError):
                kda.kda_beam_select(ctx, 2, 4, args["logits"], args["scores"], 4, *out(4), ws, done=args.get("done"))


# ---------------------------------------------------------------- reordering


def states(B, H, bf16=False, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    guard = 1024
    S = torch.randint(-2 ** 31, 2 ** 31 - 1, (B * H * D * D // (2 if bf16 else 1) + 2 * guard,), generator=gen, device=DEV, dtype=torch.int32)
    conv = torch.randint(-2 ** 31, 2 ** 31 - 1, (B * 9 * H * D + 2 * guard,), generator=gen, device=DEV, dtype=torch.int32)
    inner = S[guard:-guard].view(torch.int16 if bf16 else torch.int32).view(B, H, D, D), conv[guard:-guard].view(B, 3, 3 * H * D)
    return (S, conv), inner


def reordered(buffers, inner, rows, keep=()):
    """What a call has to leave, guards included: in place, sequences in `keep` and -1 as they are."""
    out = [b.clone() for b in buffers]
    for o, b, t in zip(out, buffers, inner):
        v = o[1024:-1024].view(t.dtype).view(t.shape)
        for i, r in enumerate(rows):
            if r >= 0 and i not in keep:
                v[i] = t[r]
    return out


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,H,rows", [
    (1, 1, [0]), (1, 2, [-1]), (2, 1, [0, 0]), (2, 3, [1, 1]), (4, 2, [0, 0, 2, 2]), (5, 1, [0, 1, 2, 3, 4]),
    (7, 2, [0, -1, 2, 0, 4, 2, 0]), (12, 5, [0, 0, 0, 0, 5, 5, 6, 5, 11, 11, 11, 11])])
def test_reorder_in_place(B, H, rows, bf16):
    buffers, inner = states(B, H, bf16, seed=B)
    want = reordered(buffers, inner, rows)
    with Ctx(H) as ctx:
        kda.kda_beam_reorder(ctx, B, torch.tensor(rows, dtype=torch.int32, device=DEV), *inner)
        assert kda.kda_sync_status(ctx) == kda.KDA_OK
    assert all(torch.equal(a, b) for a, b in zip(want, buffers))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 2), (6, 1), (16, 4), (33, 1)])
def test_reorder_into_other_buffers(B, H, bf16):
    buffers, inner = states(B, H, bf16, seed=B)
    other, other_inner = states(B, H, bf16, seed=B + 100)
    rows = torch.randint(-1, B, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    before = [b.clone() for b in buffers]
    want = [b.clone() for b in other]
    for o, t in zip(want, inner):
        v = o[1024:-1024].view(t.dtype).view(t.shape)
        for i, r in enumerate(rows):
            if r >= 0:
                v[i] = t[r]
    with Ctx(H) as ctx:
        kda.kda_beam_reorder(ctx, B, torch.tensor(rows, dtype=torch.int32, device=DEV), *inner, S_out=other_inner[0], conv_out=other_inner[1])
        assert kda.kda_sync_status(ctx) == kda.KDA_OK
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    assert all(torch.equal(a, b) for a, b in zip(before, buffers))


@pytest.mark.parametrize("rows,left", [
    ([0, 4, 2, 3], {1}), ([0, -2, 2, 3], {1}), ([0, 2 ** 31 - 1, 0, 3], {1}),
    ([1, 0, 2, 2], {0, 1}),            # two that change places
    ([1, 1, 0, 3], {2}),               # from one that moves away itself
    ([-1, 0, 2, 2], {1})])             # from one that is left as it is, not as its own
def test_reorder_errors_in_place(rows, left):
    buffers, inner = states(4, 2)
    want = reordered(buffers, inner, rows, left)
    with Ctx(2) as ctx:
        kda.kda_beam_reorder(ctx, 4, torch.tensor(rows, dtype=torch.int32, device=DEV), *inner)
        assert kda.kda_sync_status(ctx) == kda.KDA_ERR_INVALID_ARG
        assert kda.kda_sync_status(ctx) == kda.KDA_OK
    assert all(torch.equal(a, b) for a, b in zip(want, buffers))


def test_reorder_errors_into_other_buffers():
    buffers, inner = states(3, 1)
    other, other_inner = states(3, 1, seed=1)
    left = other_inner[0][1].clone()
    with Ctx(1) as ctx:
        kda.kda_beam_reorder(ctx, 3, torch.tensor([2, 3, 0], dtype=torch.int32, device=DEV), *inner, S_out=other_inner[0], conv_out=other_inner[1])
        assert kda.kda_sync_status(ctx) == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(other_inner[0][0], inner[0][2]) and torch.equal(other_inner[0][2], inner[0][0])
    assert torch.equal(other_inner[0][1], left)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_reorder_many_sequences(in_place, bf16):
    """More than are listed at a time, with an error among them."""
    B = 5001
    S = torch.randint(0, 2 ** 15, (B, 1, D, D), device=DEV, dtype=torch.int16 if bf16 else torch.int32)
    conv = torch.randn(B, 3, 3 * D, device=DEV)
    rows = [b - 1 if b % 7 == 1 else -1 if b % 7 == 3 else b for b in range(B)]
    rows[4500] = B
    if not in_place:
        rows[2], rows[5000] = 4999, 0
    S_out, conv_out = (S, conv) if in_place else (torch.zeros_like(S), torch.zeros_like(conv))
    old, old_conv = S_out.clone(), conv_out.clone()
    stays = torch.tensor([r in (-1, B) for r in rows], device=DEV)
    at = torch.tensor([0 if r in (-1, B) else r for r in rows], device=DEV)
    want = torch.where(stays[:, None, None, None], old, S[at])
    want_conv = torch.where(stays[:, None, None], old_conv, conv[at])
    with Ctx() as ctx:
        kda.kda_beam_reorder(ctx, B, torch.tensor(rows, dtype=torch.int32, device=DEV), S, conv, S_out=S_out, conv_out=conv_out)
        assert kda.kda_sync_status(ctx) == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(S_out, want) and torch.equal(conv_out, want_conv)


def test_reorder_beyond_4_gib():
    B, H = 300, 256
    S = torch.zeros(B, H, D, D, device=DEV)
    conv = torch.zeros(B, 3, 3 * H * D, device=DEV)
    for b in (0, 7, 299):
        S[b], conv[b] = b + 1, -b - 1
    rows = list(range(B))
    rows[298], rows[1], rows[150] = 299, 7, 299
    with Ctx(H) as ctx:
        kda.kda_beam_reorder(ctx, B, torch.tensor(rows, dtype=torch.int32, device=DEV), S, conv)
        assert kda.kda_sync_status(ctx) == kda.KDA_OK
    want = torch.zeros(B, device=DEV)
    for b in (0, 7, 299):
        want[b] = b + 1
    want[298], want[1], want[150] = 300, 8, 300
    assert bool((S.view(B, -1) == want[:, None]).all()) and bool((conv.view(B, -1) == -want[:, None]).all())


def test_reorder_refusals():
    buffers, inner = states(3, 1)
    other, other_inner = states(3, 1, seed=1)
    rows = torch.zeros(3, dtype=torch.int32, device=DEV)
    with Ctx(1) as ctx:
        before = kda.kda_launch_count()
        for status, S, conv, more in (
                (kda.KDA_ERR_INVALID_ARG, *inner, dict(S_out=other_inner[0])),
                (kda.KDA_ERR_INVALID_ARG, *inner, dict(conv_out=other_inner[1])),
                (kda.KDA_ERR_INVALID_ARG, inner[0][:2], inner[1][:2], dict(S_out=inner[0][1:], conv_out=other_inner[1])),
                (kda.KDA_ERR_ALIGNMENT, buffers[0][1:], inner[1], {})):
            with pytest.raises(kda.KDAError) as e:
                kda.kda_beam_reorder(ctx, 2, rows, S, conv, **more)
            assert e.value.status == status
        with pytest.raises(kda.KDAError):
            kda.kda_beam_reorder(ctx, -1, rows, *inner)
        kda.kda_beam_reorder(ctx, 0, rows, *inner)
        assert kda.kda_launch_count() == before
        with pytest.raises(ValueError):
            kda.kda_beam_reorder(ctx, 3, rows.long(), *inner)
        with pytest.raises(ValueError):
            kda.kda_beam_reorder(ctx, 3, rows[:2], *inner)


@pytest.mark.parametrize("name", ["beam_select", "beam_reorder", "all"])
def test_injected_launch_failure(name, monkeypatch):
    monkeypatch.setenv("KDA_FAULT_INJECT", name)
    with Ctx() as ctx:
        monkeypatch.delenv("KDA_FAULT_INJECT")
        x, scores = make(1, 2, 50)
        buffers, inner = states(2, 1)
        before = [b.clone() for b in buffers]
        out = [torch.full((1, 2), 7, dtype=t, device=DEV) for t in (torch.float32, torch.int32, torch.int32)]
        ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
        rows = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
        calls = {"beam_select": lambda: kda.kda_beam_select(ctx, 1, 2, x, scores, 2, *out, ws),
                 "beam_reorder": lambda: kda.kda_beam_reorder(ctx, 2, rows, *inner)}
        for which, call in calls.items():
            if name in (which, "all"):
                launches = kda.kda_launch_count()
                with pytest.raises(kda.KDAError) as e:
                    call()
                assert e.value.status == kda.KDA_ERR_CUDA and "injected" in kda.kda_last_error_detail()
                assert kda.kda_launch_count() == launches
                torch.cuda.synchronize()
                assert all(bool((t == 7).all()) for t in out) and all(torch.equal(a, b) for a, b in zip(before, buffers))
