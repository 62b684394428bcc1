"""Plain forms of the paged KV-cache operators in 64 bits, for the tests: a
scheduler's bookkeeping with Python lists, rotary positions as complex
numbers, and attention row by row over gathered keys; with the error bounds
that the kernels' number formats imply."""
from __future__ import annotations

import math

import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2      # one rounding to bf16, relative
FP32_HALF = torch.finfo(torch.float32).eps / 2


def pages_of(n, page):
    return -(-n // page)


def plan(cached, new, table, ring, state, page, width, row_cap):
    """(table, ring, cu, kv, positions, slots, state_out) as lists; table a
    list of lists.  positions and slots hold the written rows only."""
    table, ring = [list(r) for r in table], list(ring)
    n_pages, (head, n_free) = len(ring), state[:2]
    reasons = 0
    for c, n in zip(cached, new):
        if c < 0 or c + n < 0:
            reasons |= 1
        elif max(pages_of(c, page), pages_of(c + n, page)) > width:
            reasons |= 2
    ok = [not (c < 0 or c + n < 0) for c, n in zip(cached, new)]
    held = [pages_of(c, page) if o else 0 for c, o in zip(cached, ok)]
    need = [pages_of(c + n, page) if o else 0 for c, n, o in zip(cached, new, ok)]
    grow = sum(max(0, b - a) for a, b in zip(held, need))
    back = sum(max(0, a - b) for a, b in zip(held, need))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + max(0, n))
    if cu[-1] > row_cap:
        reasons |= 4
    if not 0 <= head < n_pages or n_free < 0 or n_free + back > n_pages:
        reasons |= 8
    fits = reasons == 0 and grow <= n_free
    taken = put = 0
    positions, slots = [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        if fits:
            for q in range(held[b], need[b]):
                table[b][q] = ring[(head + taken) % n_pages]
                taken += 1
            for q in range(need[b], held[b]):
                ring[(head + n_free + put) % n_pages] = table[b][q]
                put += 1
        for i in range(max(0, n)):
            pos = max(c, 0) + i
            positions.append(pos)
            slots.append(table[b][pos // page] * page + pos % page if fits else -1)
    kv = [c + n if fits else c for c, n in zip(cached, new)]
    out = [(head + taken) % n_pages if fits else head, n_free - taken + put, max(0, grow - n_free), reasons]
    return table, ring, cu, kv, positions[:row_cap], slots[:row_cap], out


def rotate(x, cos, sin):
    """x [..., D] float64 rotated by cos, sin [..., D/2], and the sum of the
    magnitudes of the products (for the error bound)."""
    half = x.shape[-1] // 2
    lo, hi = x[..., :half], x[..., half:]
    y = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    mag = torch.cat([(lo * cos).abs() + (hi * sin).abs(), (hi * cos).abs() + (lo * sin).abs()], -1)
    return y, mag


def rotate_bound(y, mag):
    """two fp32 products and a sum (three roundings), then one rounding to bf16"""
    return BF16_HALF * y.abs() + 4 * FP32_HALF * mag


def attention(q, k_pages, v_pages, table, kv_lens, cu, causal, scale=None):
    """Float64 attention of packed rows q [T, Hq, D] over the pages.  Returns
    out, lse, and elementwise bounds of their errors.

    Error of a kernel that multiplies bf16 operands into fp32 sums, keeps p in
    bf16 for the second product and the row sum in fp32:
      score: |s' - s| <= eps_s = D * 2^-24 * scale * sum_d |q_d k_d| (largest over the keys), and the
             scaled score enters 2^x with an argument rounded to fp32: 2^-23 |s| more;
      p:     relative 2 (eps_s) + 2^-21 (2^x approximation), and 2^-8 for its bf16 rounding;
      sums over n keys: n * 2^-24 relative each (numerator, denominator), joined partials included;
      out:   one rounding to bf16.
    """
    T, hq, d = q.shape
    hkv, page = k_pages.shape[1], k_pages.shape[2]
    n_pages, width = k_pages.shape[0], table.shape[1]
    g = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(T, hq, d, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    tol_o = torch.zeros_like(out)
    tol_l = torch.zeros_like(lse)
    for b in range(len(kv_lens)):
        t0, t1, kv = cu[b], cu[b + 1], min(max(kv_lens[b], 0), width * page)
        if t0 == t1:
            continue
        ids = table[b, : pages_of(kv, page)].long()
        good = (ids >= 0) & (ids < n_pages)
        seen = good.repeat_interleave(page)[:kv]
        at = ids.clamp(0, n_pages - 1)
        k = k_pages[at].double().permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :kv]
        v = v_pages[at].double().permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :kv]
        see = seen[None, :].expand(t1 - t0, kv).clone()
        if causal:
            last = kv_lens[b] - (t1 - t0) + torch.arange(t1 - t0)
            see &= torch.arange(kv)[None, :] <= last[:, None]
        # masked keys and values may hold anything
        k = torch.where(seen[None, :, None], k, 0.0)
        v = torch.where(seen[None, :, None], v, 0.0)
        for h in range(hq):
            qq = q[t0:t1, h].double()
            s = (qq @ k[h // g].t()) * scale
            eps_s = d * FP32_HALF * scale * (qq.abs() @ k[h // g].abs().t())
            eps_s = torch.where(see, eps_s + 2 * FP32_HALF * s.abs(), 0.0).amax(-1, keepdim=True) if kv else s[:, :0]
            s = torch.where(see, s, -math.inf)
            some = see.any(-1)
            if not bool(some.any()):
                continue
            r = some.nonzero().flatten()
            p = torch.softmax(s[r], -1)
            o = p @ v[h // g]
            a = p @ v[h // g].abs()
            n = kv + 1
            rel = 2 * eps_s[r] + 2.0 ** -21 + 2 * n * FP32_HALF
            out[t0 + r, h] = o
            lse[t0 + r, h] = torch.logsumexp(s[r], -1)
            tol_o[t0 + r, h] = BF16_HALF * o.abs() + (1 + BF16_HALF) * (BF16_HALF + rel) * a
            tol_l[t0 + r, h] = rel.squeeze(-1) + 4 * FP32_HALF * (1 + lse[t0 + r, h].abs())
    return out, lse, tol_o, tol_l
