"""Two layers of a hybrid model, prompts and then single tokens: one KDA layer
(recurrent state) and one softmax-attention layer (paged key/value cache), with
random weights.

    python examples/hybrid_decode.py          # needs a GB300 and the built library

Each layer reads the residual stream x [tokens, hidden], projects it, runs its
token mixing and adds W_o of the result.  The same tokens run once as whole
prompts and once as prompts without their last tokens, followed by single-token
steps; the two ways have to agree on the last token's x.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_delta_rule_token_gb300 as kda  # noqa: E402

D = kda.HEAD_DIM
DEV = "cuda"


def _randn(*shape, gen, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)


class Projections:
    """q, k, v, gate and output projections of one layer of `heads` heads."""

    def __init__(self, heads, hidden, gen):
        self.heads, self.hidden = heads, hidden
        hd = heads * D
        self.params = (_randn(3, hd, 4, gen=gen, scale=0.4), torch.zeros(heads, D, device=DEV),
                       torch.full((heads, D), -2.0, device=DEV), torch.ones(heads, D, device=DEV))
        self.ctx = kda.kda_create(heads, *self.params)
        self.w = (_randn(4 * hd, hidden, gen=gen, scale=hidden ** -0.5, dtype=torch.bfloat16),
                  _randn(hidden, hd, gen=gen, scale=hd ** -0.5, dtype=torch.bfloat16))
        kda.kda_bind_projections(self.ctx, hidden, *self.w)

    def qkvg(self, x, f32):
        n = x.shape[0]
        q, k, v = (torch.empty(n, self.heads, D, device=DEV, dtype=torch.float32 if f32 else torch.bfloat16) for _ in range(3))
        gate = torch.empty(n, self.heads, D, device=DEV)
        kda.kda_project_qkvg(self.ctx, n, x.to(torch.bfloat16), q, k, v, gate, qkv_f32=f32)
        return q, k, v, gate

    def out(self, o):
        n = o.shape[0]
        y = torch.empty(n, self.hidden, device=DEV)
        ws = torch.empty(kda.kda_project_o_workspace_bytes(self.ctx, n), dtype=torch.uint8, device=DEV)
        kda.kda_project_o(self.ctx, n, o, y, ws)
        return y


class KDALayer(Projections):
    def __init__(self, heads, hidden, requests, gen, rank=64):
        super().__init__(heads, hidden, gen)
        self.low = (_randn(rank, hidden, gen=gen, scale=hidden ** -0.5), _randn(heads * D, rank, gen=gen, scale=rank ** -0.5),
                    _randn(heads, hidden, gen=gen, scale=hidden ** -0.5))
        kda.kda_bind_lowrank(self.ctx, hidden, rank, *self.low)
        self.state = torch.zeros(requests, heads, D, D, device=DEV)
        self.conv = torch.zeros(requests, 3, 3 * heads * D, device=DEV)

    def __call__(self, x, step):
        n = x.shape[0]
        z, beta = torch.empty(n, self.heads, D, device=DEV), torch.empty(n, self.heads, device=DEV)
        ws = torch.empty(kda.kda_lowrank_workspace_bytes(self.ctx, n), dtype=torch.uint8, device=DEV)
        kda.kda_lowrank(self.ctx, n, x, z, beta, ws)
        o = torch.empty(n, self.heads, D, device=DEV)
        q, k, v, gate = self.qkvg(x, f32=step.single)
        if step.single:
            kda.kda_decode_step(self.ctx, n, q, k, v, z, beta, gate, self.conv, self.state, o)
        else:
            kda.kda_prefill_varlen(self.ctx, step.requests, step.cu, n, q, k, v, z, beta, gate, self.conv, self.state, o)
        return x + self.out(o)


class AttentionLayer(Projections):
    """Gated softmax attention with normalised, rotated queries and keys."""

    def __init__(self, heads, hidden, pages, page_size, gen, cache_type):
        super().__init__(heads, hidden, gen)
        e4m3 = cache_type == kda.KDA_CACHE_E4M3
        self.gammas = torch.ones(2, D, device=DEV)
        self.scales = torch.full((2, heads), 1 / 16, device=DEV)
        self.attn = kda.kda_attn_create(
            heads, heads, page_size=page_size, cache_type=cache_type, rotary_dim=64,
            inv_freq=[10000.0 ** (-i / 32) for i in range(32)], q_gamma=self.gammas[0], k_gamma=self.gammas[1],
            k_scale=self.scales[0] if e4m3 else None, v_scale=self.scales[1] if e4m3 else None)
        self.cache = torch.empty(2, pages, heads, page_size, D, device=DEV, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        kda.kda_attn_bind_cache(self.attn, pages, self.cache[0], self.cache[1])
        self.workspace = torch.empty(kda.kda_attn_workspace_bytes(self.attn), dtype=torch.uint8, device=DEV)

    def __call__(self, x, step):
        n = x.shape[0]
        q, k, v, gate = self.qkvg(x, f32=False)
        kda.kda_attn_append(self.attn, n, q, k, v, step.positions, step.slots, q)
        o = torch.empty(n, self.heads, D, device=DEV)
        if step.single:
            kda.kda_attn_decode(self.attn, n, q, step.table, step.kv_lens, o, self.workspace, gate_logit=gate)
        else:
            kda.kda_attn_prefill(self.attn, step.requests, n, step.cu, q, step.table, step.kv_lens, o, self.workspace,
                                 gate_logit=gate)
        return x + self.out(o)


class Step:
    """What one step's layers share: planned once, whatever the number of layers."""

    def __init__(self, attn, server, new):
        b, n = len(new), sum(new)
        self.requests, self.single = b, all(c == 1 for c in new)
        self.table = server.table
        self.cu, self.kv_lens = torch.empty(b + 1, dtype=torch.int32, device=DEV), torch.empty(b, dtype=torch.int32, device=DEV)
        self.positions, self.slots = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, dtype=torch.int64, device=DEV)
        info = torch.empty(4, dtype=torch.int32, device=DEV)
        kda.kda_attn_plan(attn, b, n, server.lens, torch.tensor(new, dtype=torch.int32, device=DEV), server.free,
                          server.free_count, server.table, self.cu, self.kv_lens, self.positions, self.slots, info)
        server.lens, server.free_count = self.kv_lens, info[2:3]   # nothing of this comes back to the host


class Server:
    """The requests' cached lengths, the block table and the stack of unused pages."""

    def __init__(self, requests, pages, width):
        self.lens = torch.zeros(requests, dtype=torch.int32, device=DEV)
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(pages, device=DEV).to(torch.int32)
        self.free_count = torch.tensor([pages], dtype=torch.int32, device=DEV)


def run(x, chunks, heads, hidden, page_size, cache_type, seed):
    """x [requests][length, hidden] through both layers, in steps of chunks[step][request]
    tokens; the last step's outputs."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    requests, longest = len(x), max(t.shape[0] for t in x)
    width = -(-longest // page_size)
    pages = requests * width
    first = KDALayer(heads, hidden, requests, gen)
    second = AttentionLayer(heads, hidden, pages, page_size, gen, cache_type)
    server, done = Server(requests, pages, width), [0] * requests
    for new in chunks:
        step = Step(second.attn, server, new)
        y = torch.cat([t[d:d + n] for t, d, n in zip(x, done, new)])
        y = second(first(y, step), step)
        done = [d + n for d, n in zip(done, new)]
    for layer in (first, second):
        assert kda.kda_sync_status(layer.ctx) == kda.KDA_OK
    assert kda.kda_attn_sync_status(second.attn) == kda.KDA_OK
    kda.kda_attn_destroy(second.attn)
    for layer in (first, second):
        kda.kda_destroy(layer.ctx)
    return y


def main(lengths=(200, 37, 1000), singles=4, heads=8, hidden=1024, page_size=16, cache_type=kda.KDA_CACHE_BF16, seed=0):
    """Largest difference of the last tokens' x between the two ways, relative to the largest x."""
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    x = [_randn(n, hidden, gen=gen) for n in lengths]
    args = (heads, hidden, page_size, cache_type, seed)
    whole = run(x, [list(lengths)], *args)
    ends = torch.tensor(lengths, device=DEV).cumsum(0) - 1
    steps = run(x, [[n - singles for n in lengths]] + [[1] * len(lengths)] * singles, *args)
    off = ((whole[ends] - steps).abs().max() / whole[ends].abs().max()).item()
    print(f"{len(lengths)} requests of {', '.join(map(str, lengths))} tokens, the last {singles} one by one: "
          f"off by {off:.1e} of the whole prompts' values")
    return off


if __name__ == "__main__":
    kda.load()
    main()
    main(cache_type=kda.KDA_CACHE_E4M3, page_size=64)
