"""Beam search over a hybrid model of one KDA layer and one softmax-attention layer, with random weights.

    python examples/beam_decode.py          # needs a GB300 and the built library

Every prompt is read once, by the first of its beams, and taken over by the others; a step then is one token
of every beam: the layers, the choice of the best continuations (kda_beam_select), and the beams'
recurrent states (kda_beam_reorder) and cache pages (kda_attn_fork, kda_attn_copy_pages) after them.
Attention reads a prompt's keys once for all of its beams (kda_attn_decode_shared).  Nothing comes back
to the host before the end.  The scores found are compared with those of the same tokens in requests that
share nothing.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import kda_delta_rule_token_gb300 as kda  # noqa: E402
from hybrid_decode import DEV, AttentionLayer, KDALayer, Server, Step, _randn  # noqa: E402


class SharedAttentionLayer(AttentionLayer):
    """The attention layer whose single tokens know which requests go on from the same prompt."""

    def share(self, groups, cu, prefix):
        self.shared = (groups, cu, prefix)
        size = kda.kda_attn_shared_workspace_bytes(self.attn, cu.numel() and int(cu[-1]))
        self.shared_workspace = torch.empty(size, dtype=torch.uint8, device=DEV)

    def __call__(self, x, step):
        if not step.single or not hasattr(self, "shared"):
            return super().__call__(x, step)
        n = x.shape[0]
        q, k, v, gate = self.qkvg(x, f32=False)
        kda.kda_attn_append(self.attn, n, q, k, v, step.positions, step.slots, q)
        o = torch.empty(n, self.heads, kda.HEAD_DIM, device=DEV)
        kda.kda_attn_decode_shared(self.attn, n, q, step.table, step.kv_lens, *self.shared, o, self.shared_workspace, gate_logit=gate)
        return x + self.out(o)


class Model:
    def __init__(self, requests, pages, width, heads, hidden, vocab, page_size, cache_type, seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.first = KDALayer(heads, hidden, requests, gen)
        self.second = SharedAttentionLayer(heads, hidden, pages, page_size, gen, cache_type)
        self.embed = _randn(vocab, hidden, gen=gen)
        self.head = _randn(vocab, hidden, gen=gen, scale=hidden ** -0.5)
        self.server = Server(requests, pages, width)

    def step(self, tokens, new):
        """The logits after each of the packed tokens."""
        step = Step(self.second.attn, self.server, new)
        return self.second(self.first(self.embed[tokens], step), step) @ self.head.t()

    def done(self):
        for layer in (self.first, self.second):
            assert kda.kda_sync_status(layer.ctx) == kda.KDA_OK
        assert kda.kda_attn_sync_status(self.second.attn) == kda.KDA_OK
        kda.kda_attn_destroy(self.second.attn)
        for layer in (self.first, self.second):
            kda.kda_destroy(layer.ctx)


class Beams:
    """What a search keeps beside the model: scores and tokens of the beams, and whose pages are whose."""

    def __init__(self, model, groups, beams, vocab, steps, end):
        self.model, self.groups, self.beams, self.end = model, groups, beams, end
        n = groups * beams
        self.scores = torch.full((groups, beams), -float("inf"), device=DEV)
        self.scores[:, 0] = 0      # the beams of a prompt are alike at first
        self.done = torch.zeros(groups, beams, dtype=torch.uint8, device=DEV)
        self.tokens = torch.zeros(n, steps, dtype=torch.int64, device=DEV)
        self.out = [torch.empty(groups, beams, dtype=t, device=DEV) for t in (torch.float32, torch.int32, torch.int32)]
        ctx, attn = model.first.ctx, model.second.attn
        self.workspace = torch.empty(kda.kda_beam_select_workspace_bytes(ctx, groups, beams, vocab, beams), dtype=torch.uint8, device=DEV)
        pages, width = model.server.free.numel(), model.server.table.shape[1]
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.spare = torch.full_like(model.server.table, -1)
        self.copies = [torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(3)]
        self.fork_workspace = torch.empty(kda.kda_attn_fork_workspace_bytes(attn, n, width), dtype=torch.uint8, device=DEV)

    def take_over(self, rows):
        """Every beam goes on from beam rows[b]: pages and states."""
        m, s, n = self.model, self.model.server, rows.numel()
        lens, info = torch.empty_like(s.lens), torch.empty(4, dtype=torch.int32, device=DEV)
        kda.kda_attn_fork(m.second.attn, n, rows, s.lens, s.table, self.refs, s.free, s.free_count, self.spare, lens,
                          *self.copies, info, self.fork_workspace)
        kda.kda_attn_copy_pages(m.second.attn, n, *self.copies)
        s.table, self.spare = self.spare, s.table
        s.lens, s.free_count = lens, info[2:3]
        kda.kda_beam_reorder(m.first.ctx, n, rows, m.first.state, m.first.conv)

    def go_on(self, logits, t):
        """The best continuations become the beams."""
        scores, tokens, rows = self.out
        kda.kda_beam_select(self.model.first.ctx, self.groups, self.beams, logits, self.scores, self.beams, scores, tokens, rows,
                            self.workspace, done=self.done, end_token=self.end, keep_places=True)
        self.scores = scores.clone()
        flat = rows.view(-1)
        self.take_over(flat)
        self.tokens = self.tokens[flat.long()]
        self.tokens[:, t] = tokens.view(-1)
        self.done = (self.done.view(-1)[flat.long()].view_as(self.done) | (tokens == self.end)).to(torch.uint8)
        return self.tokens[:, t]


def search(prompts, beams, steps, heads, hidden, vocab, page_size, cache_type, seed, end):
    """Scores [prompts, beams] and tokens [prompts * beams, steps] of the best beams."""
    groups, longest = len(prompts), max(len(p) for p in prompts)
    n, width = groups * beams, -(-(longest + steps) // page_size)
    pages = groups * width + n * (-(-steps // page_size) + 2)
    model = Model(n, pages, width, heads, hidden, vocab, page_size, cache_type, seed)
    search = Beams(model, groups, beams, vocab, steps, end)
    new = [len(prompts[b // beams]) if b % beams == 0 else 0 for b in range(n)]
    ends = (torch.tensor([len(p) for p in prompts], device=DEV).cumsum(0) - 1).repeat_interleave(beams)
    logits = model.step(torch.cat(prompts), new)[ends]       # all of a prompt's beams after its last token
    model.second.share(groups, torch.arange(0, n + 1, beams, dtype=torch.int32, device=DEV),
                       torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=DEV))
    tokens = search.go_on(logits, 0)
    for t in range(1, steps):
        tokens = search.go_on(model.step(tokens, [1] * n), t)
    search.take_over(torch.full((n,), -1, dtype=torch.int32, device=DEV))   # the end: all pages are free again
    left = int(model.server.free_count)
    model.done()
    assert left == pages and not bool(search.refs.any()), f"{left} of {pages} pages came back"
    return search.scores, search.tokens


def score(prompts, tokens, beams, heads, hidden, vocab, page_size, cache_type, seed, end):
    """The same tokens in as many requests that share nothing: their scores [prompts, beams]."""
    n, steps = tokens.shape
    longest = max(len(p) for p in prompts)
    width = -(-(longest + steps) // page_size)
    model = Model(n, n * width, width, heads, hidden, vocab, page_size, cache_type, seed)
    each = [prompts[b // beams] for b in range(n)]
    ends = torch.tensor([len(p) for p in each], device=DEV).cumsum(0) - 1
    logits = model.step(torch.cat(each), [len(p) for p in each])[ends]
    total, live = torch.zeros(n, dtype=torch.float64, device=DEV), torch.ones(n, dtype=torch.bool, device=DEV)
    for t in range(steps):
        gain = torch.log_softmax(logits.double(), 1).gather(1, tokens[:, t, None])[:, 0]
        total += torch.where(live, gain, 0)
        live &= tokens[:, t] != end
        if t + 1 < steps:
            logits = model.step(tokens[:, t], [1] * n)
    model.done()
    return total.view(len(prompts), beams)


def main(lengths=(200, 37, 1000), beams=4, steps=12, heads=8, hidden=512, vocab=1000, page_size=16,
         cache_type=kda.KDA_CACHE_BF16, seed=0, end=7):
    """How far the search's scores are from those of requests that share nothing, at most."""
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    prompts = [torch.randint(0, vocab, (n,), generator=gen, device=DEV) for n in lengths]
    args = (heads, hidden, vocab, page_size, cache_type, seed, end)
    found, tokens = search(prompts, beams, steps, *args)
    alone = score(prompts, tokens, beams, *args)
    off = (found.double() - alone).abs().max().item()
    print(f"{len(prompts)} prompts of {', '.join(map(str, lengths))} tokens, {beams} beams, {steps} steps: best scores "
          f"{', '.join('%.2f' % s for s in found.amax(1).tolist())}, off by {off:.1e} at most from requests that share nothing")
    return off


if __name__ == "__main__":
    kda.load()
    main()
    main(cache_type=kda.KDA_CACHE_E4M3, page_size=64, beams=16, lengths=(700, 90))
