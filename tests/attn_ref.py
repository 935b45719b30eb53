"""Plain 64-bit forms of the paged softmax-attention operators, one request
and one head at a time, and the error bounds their GPU tests use.

Bounds count roundings: a value rounded to a type is off by at most half a
step, eps / 2 relative (bf16 2^-8, e4m3 2^-4, fp32 2^-24).
"""
from __future__ import annotations

import math

import torch

D = 128
U32 = 2.0 ** -24
UBF = 2.0 ** -8
F64 = torch.float64


def plan(cache_lens, new_lens, free_pages, free_count, table, page, N):
    """The plan's outputs, request by request; `table` is a list of lists (changed in place)."""
    free_count = min(max(free_count, 0), len(free_pages))
    max_pages = len(table[0])
    cu, kv, info = [0], [], [0, 0, 0, 0]
    positions, slots = [0] * N, [-1] * N
    rows = upto = 0
    for b, (c, n) in enumerate(zip(cache_lens, new_lens)):
        first, rows = rows, rows + max(n, 0)
        cu.append(min(rows, 2 ** 31 - 1))
        before, after = -(-c // page), -(-(c + n) // page)
        fits = c >= 0 and n >= 0 and after <= max_pages and rows <= N
        need = after - before if fits else 0
        excl, upto = upto, upto + need
        ok = fits and (need == 0 or upto <= free_count)
        if ok:
            for i in range(need):
                table[b][before + i] = free_pages[free_count - 1 - (excl + i)]
            if need:
                info[1] = upto
        else:
            info[3] += 1
        kv.append(c + n if ok else 0)
        for i in range(max(n, 0)):
            if first + i < N:
                positions[first + i] = c + i
                if ok:
                    p = c + i
                    slots[first + i] = table[b][p // page] * page + p % page
    info[0], info[2] = min(rows, 2 ** 31 - 1), free_count - info[1]
    return cu, kv, positions, slots, info


def norm_rotate(x, gamma, positions, inv_freq, rotary, interleaved, eps):
    """x [N, H, 128] (any type) in 64 bits, and per value a bound on the fp32 form's error."""
    x = x.to(F64)
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.to(F64)
    mag = x.abs()
    if rotary:
        half = rotary // 2
        th = positions.to(F64)[:, None] * torch.tensor(list(inv_freq), dtype=F64, device=x.device)
        c, s = th.cos()[:, None], th.sin()[:, None]
        i = torch.arange(half, device=x.device)
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[..., first], x[..., second]
        y = x.clone()
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        both = a.abs() + b.abs()
        mag = mag.clone()
        mag[..., first], mag[..., second] = both, both
        x = y
    # fp32: the sum of 128 squares in a tree and its root, two products, and
    # a rotation whose angle is off by 2^-25 half turns: below 16 roundings.
    return x, 16 * U32 * mag


def attend(q, k_cache, v_cache, table, kv_lens, cu_new, page, scale, k_scale=None, v_scale=None, gate=None):
    """o [N, Hq, 128], lse [N, Hq], and bounds on both for bf16 rounding of
    the softmax weights (2^-8 relative) and fp32 everywhere else.  cu_new
    None: one token per request."""
    N, Hq, _ = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    dev = q.device
    o = torch.zeros(N, Hq, D, dtype=F64, device=dev)
    lse = torch.full((N, Hq), -math.inf, dtype=F64, device=dev)
    bound, lbound = torch.zeros_like(o), torch.zeros(N, Hq, dtype=F64, device=dev)
    for b, L in enumerate(kv_lens):
        r0, r1 = (b, b + 1) if cu_new is None else (cu_new[b], cu_new[b + 1])
        n = r1 - r0
        if L <= 0 or n <= 0:
            continue
        pages = torch.tensor(table[b][: -(-L // page)], device=dev)
        sees = torch.arange(L, device=dev)[None] <= (L - n + torch.arange(n, device=dev))[:, None]
        for h in range(Hkv):
            k = k_cache[pages, h].to(F64).reshape(-1, D)[:L]
            v = v_cache[pages, h].to(F64).reshape(-1, D)[:L]
            if k_scale is not None:
                k, v = k * k_scale[h].to(F64), v * v_scale[h].to(F64)
            for g in range(G):
                x = q[r0:r1, h * G + g].to(F64)
                z = x @ k.T * scale
                zmax = (x.abs() @ k.abs().T * scale).masked_fill(~sees, 0).amax(1, keepdim=True)
                z = z.masked_fill(~sees, -math.inf)
                m = z.amax(1, keepdim=True)
                e = torch.exp(z - m.masked_fill(m == -math.inf, 0))
                e = e.masked_fill(~sees, 0)
                total = e.sum(1, keepdim=True)
                safe = total.masked_fill(total == 0, 1)
                oo, mean = e @ v / safe, e @ v.abs() / safe
                # A logit is off by up to 132 roundings of the sum of |q k|
                # (relative error of its weight), the exponential by 2^-21,
                # sums over L keys by L roundings, each counted for weight
                # and sum; the weights themselves round to bf16.
                rel = 2 * (132 * U32 * zmax + 2.0 ** -21 + (L + 64) * U32)
                bb = (UBF + rel) * mean
                if gate is not None:
                    s = torch.sigmoid(gate[r0:r1, h * G + g].to(F64))
                    oo, bb = oo * s, bb * s + 2.0 ** -20 * (oo * s).abs()
                o[r0:r1, h * G + g], bound[r0:r1, h * G + g] = oo, bb
                l = (m + torch.log(safe)).squeeze(1)
                lse[r0:r1, h * G + g] = torch.where(total.squeeze(1) == 0, -math.inf, l)
                lbound[r0:r1, h * G + g] = rel.squeeze(1) + 4 * U32 * l.abs().nan_to_num(posinf=0.0)
    return o, lse, bound, lbound
