"""Cases of the paged KV-cache operators: what they compute in plain torch and how they are called.

Requests of different lengths share one pool of key/value pages.  Three operators serve them:

  plan       request lengths -> block tables, slots and positions of the new rows, and the pool's free list
  append     rotary positions on q and k of the new rows, k and v written to their slots in the pages
  attention  the new rows' queries over their requests' pages (one row each, whole canvases, causal chunks)

With `own` false `run` computes them from elementary torch operations in 32 bits; with `own` true it makes the
calls of block_discrete_diffusion_denoise_b200 that a user makes.
"""
import math
import random

import torch

own = False

# (query heads, kv heads, head_dim) of the repository's workloads: tiny, small and the 26B-A4B shapes
TINY, SMALL, A4B = (4, 2, 64), (8, 2, 128), (16, 8, 176)
ROPE_BASE = 10000.0


def _case(name, op, batch, past, rows, heads=A4B, page=64, causal=False, mix=0):
    """past and rows: (lowest, highest) cached length and new rows of a request, drawn for each from `mix`."""
    return dict(name=name, op=op, batch=batch, past_lo=past[0], past_hi=past[1], rows_lo=rows[0], rows_hi=rows[1],
                hq=heads[0], hkv=heads[1], hd=heads[2], page=page, causal=causal, mix=mix)


def listed():
    return [
        # one request starts a 256-token canvas behind a 2048-token prompt: a call of pure latency
        _case("plan_one", "plan", 1, (2048, 2048), (256, 256)),
        # a scheduler's turn over 200 requests: some grow by up to two canvases, some give pages back
        _case("plan_mixed", "plan", 200, (0, 8191), (-700, 512), page=16, mix=1),
        # the canvas of one request enters the cache, every layer of every step
        _case("append_canvas", "append", 1, (2048, 2048), (256, 256)),
        # one new row for each of 61 requests, odd count, small pages
        _case("append_tokens", "append", 61, (0, 1500), (1, 1), SMALL, 16, mix=2),
        # a prefill of eight long prompts in one call
        _case("append_prefill", "append", 8, (0, 300), (1500, 2500), mix=3),
        # one new token of one request: latency
        _case("token_one", "attention", 1, (2047, 2047), (1, 1)),
        # one new token each for 33 short requests, odd lengths, pages of 16
        _case("token_small", "attention", 33, (0, 1500), (1, 1), SMALL, 16, mix=4),
        # one new token each for 64 requests of ragged lengths: the cache is streamed once
        _case("token_batch", "attention", 64, (256, 8190), (1, 1), mix=5),
        # the denoising step's attention: a 256-token canvas over itself and a 2048-token prompt
        _case("canvas_2k", "attention", 1, (2048, 2048), (256, 256)),
        # eight canvases behind prompts of different lengths
        _case("canvas_batch", "attention", 8, (1500, 6500), (256, 256), mix=6),
        # a canvas behind a 32768-token prompt
        _case("canvas_32k", "attention", 1, (32768, 32768), (256, 256)),
        # causal chunks of five prompts, ragged, over what is already cached
        _case("prefill_ragged", "attention", 5, (0, 2000), (100, 1100), SMALL, 32, causal=True, mix=7),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = rng.choice([TINY, SMALL, A4B, A4B])
    page = rng.choice([16, 32, 64, 64, 128])
    mix = rng.randrange(1, 1 << 30)
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "attention"])
    if op == "plan":
        hi = _log(rng, 1, 512)
        case = _case("", op, _log(rng, 1, 256), (0, _log(rng, 16, 16384)), (-rng.randrange(0, 800), hi), heads, page, mix=mix)
    elif op == "append":
        batch = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, 16000 // batch))
        case = _case("", op, batch, (0, 500), (max(1, hi // 2), hi), heads, page, mix=mix)
    else:
        kind = rng.choice(["token", "token", "canvas", "canvas", "prefill"])
        if kind == "token":  # up to 260,000 cached tokens in all
            batch = _log(rng, 1, 128)
            hi = _log(rng, 40, min(32768, 260000 // batch))
            rows, causal = (1, rng.choice([1, 1, 1, 4])), True
        elif kind == "canvas":
            batch = _log(rng, 1, 8)
            hi = _log(rng, 100, 32768 // batch)
            n = rng.choice([16, 64, 250, 256])
            rows, causal = (n, n), False
        else:
            batch = _log(rng, 1, 8)
            top = _log(rng, 50, 4000 // batch)
            hi = _log(rng, 20, 4000)
            rows, causal = (max(1, top // 4), top), True
        case = _case("", op, batch, (rng.choice([0, hi // 8, hi // 2]), hi), rows, heads, page, causal, mix)
    del case["name"]
    return case


def _lengths(case):
    """(cached length, new rows) of every request: plain numbers, from the case alone."""
    rng = random.Random(case["mix"])
    out = []
    for _ in range(case["batch"]):
        past = rng.randint(case["past_lo"], case["past_hi"])
        out.append((past, max(-past, rng.randint(case["rows_lo"], case["rows_hi"]))))
    return out


def _pages(n, page):
    return -(-n // page)


def _rope_table(n, hd, device):
    """cos and sin of position * base^(-2j/hd), angles in 64 bits, stored in 32: [n, hd/2, 2]."""
    j = torch.arange(hd // 2, dtype=torch.float64, device=device)
    a = torch.arange(n, dtype=torch.float64, device=device)[:, None] * ROPE_BASE ** (-2.0 * j / hd)
    return torch.stack([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    dev = "cuda"
    lens = _lengths(case)
    page, B = case["page"], case["batch"]
    past = [p for p, _ in lens]
    new = [n for _, n in lens]
    g = torch.Generator(device=dev).manual_seed(seed)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    held = [_pages(p, page) for p in past]                   # pages before the call
    need = [_pages(p + n, page) for p, n in lens]            # pages after it
    width = max(1, max(max(held), max(need)))
    used = held if case["op"] == "plan" else need
    total = sum(used) + sum(max(0, b - a) for a, b in zip(held, need))
    n_pages = total + total // 8 + 8
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    col = torch.arange(width, dtype=torch.int32, device=dev)
    n_used = i32(used)
    first = torch.cumsum(n_used, 0) - n_used
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    table = torch.where(col < n_used[:, None], order[at.long()], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
    cu = [0]
    for n in new:
        cu.append(cu[-1] + max(0, n))
    T = cu[-1]
    s = dict(case=case, B=B, T=T, page=page, n_pages=n_pages, table=table, width=width, max_rows=max(max(0, n) for n in new))
    if case["op"] == "plan":
        # the free pages stand in a ring from a place of their own, wrapping around its end
        n_free = n_pages - sum(held)
        head = n_pages - 1 - n_free // 3
        ring = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        place = (head + torch.arange(n_free, device=dev)) % n_pages
        ring[place] = order[sum(held):]
        s.update(cached=i32(past), new=i32(new), ring=ring, state=i32([head, n_free, 0, 0]),
                 cu=torch.full((B + 1,), -1, dtype=torch.int32, device=dev),
                 kv=torch.full((B,), -1, dtype=torch.int32, device=dev),
                 positions=torch.full((T + 64,), -2, dtype=torch.int32, device=dev),
                 slots=torch.full((T + 64,), -2, dtype=torch.int32, device=dev),
                 state_out=i32([-1, -1, -1, -1]))
        return s
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    bf = torch.bfloat16
    s.update(cu=i32(cu), kv=i32([p + n for p, n in lens]))

    def pool():
        return torch.randn(n_pages, hkv, page, hd, generator=g, device=dev, dtype=bf)

    if case["op"] == "append":
        row = torch.arange(T, device=dev)
        req = torch.searchsorted(s["cu"].long(), row, right=True) - 1
        pos = i32(past).long()[req] + row - s["cu"].long()[req]
        slot = table.long()[req, pos // page] * page + pos % page
        s.update(qkv=torch.randn(T, (hq + 2 * hkv) * hd, generator=g, device=dev, dtype=bf),
                 positions=pos.to(torch.int32), slots=slot.to(torch.int32),
                 rope=_rope_table(max(p + n for p, n in lens), hd, dev), k=pool(), v=pool(),
                 q=torch.empty(T, hq, hd, dtype=bf, device=dev))
        return s
    s.update(q=torch.randn(T, hq, hd, generator=g, device=dev, dtype=bf), k=pool(), v=pool(),
             out=torch.empty(T, hq, hd, dtype=bf, device=dev), lse=torch.empty(T, hq, dtype=torch.float32, device=dev))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_plan(s):
    page, n, W = s["page"], s["n_pages"], s["width"]
    cached, new = s["cached"].long(), s["new"].long()
    head, n_free = s["state"][0].long(), s["state"][1].long()
    total = cached + new
    held, need = (cached + page - 1) // page, (total + page - 1) // page
    grow, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    rows = new.clamp(min=0)
    zero = rows.new_zeros(1)
    cu = torch.cat([zero, rows.cumsum(0)])
    fits = grow.sum() <= n_free
    # pages taken from the head of the ring, in order of request and page
    col = torch.arange(W, device=cached.device)
    take = head + (grow.cumsum(0) - grow)[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < need[:, None]) & fits
    table = torch.where(fresh, s["ring"][take % n], s["table"])
    # pages given back, put behind the tail
    put = head + n_free + (back.cumsum(0) - back)[:, None] + col - need[:, None]
    given = (col >= need[:, None]) & (col < held[:, None]) & fits
    ring = torch.cat([s["ring"], s["ring"].new_zeros(1)])
    ring[torch.where(given, put % n, n).flatten()] = s["table"].flatten()
    # rows
    row = torch.arange(s["positions"].numel(), device=cached.device)
    req = (torch.searchsorted(cu, row, right=True) - 1).clamp(max=s["B"] - 1)
    live = row < cu[-1]
    pos = cached[req] + row - cu[req]
    slot = table.long()[req, (pos // page).clamp(min=0, max=W - 1)] * page + pos % page
    slot = torch.where(fits, slot, -1)
    positions = torch.where(live, pos, s["positions"].long())
    slots = torch.where(live, slot, s["slots"].long())
    kv = torch.where(fits, total, cached)
    popped, pushed = torch.where(fits, grow.sum(), 0), torch.where(fits, back.sum(), 0)
    state = torch.stack([(head + popped) % n, n_free - popped + pushed, (grow.sum() - n_free).clamp(min=0), torch.zeros_like(head)])
    i32 = torch.int32
    return [table, ring[:n], cu.to(i32), kv.to(i32), positions.to(i32), slots.to(i32), state.to(i32)]


def _plain_append(s):
    c = s["case"]
    hq, hkv, hd, page = c["hq"], c["hkv"], c["hd"], s["page"]
    x = s["qkv"].float().view(s["T"], hq + 2 * hkv, hd)
    cs = s["rope"][s["positions"].long()][:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    lo, hi = x[..., : hd // 2], x[..., hd // 2:]
    r = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    at, off = s["slots"].long() // page, s["slots"].long() % page
    s["k"][at, :, off] = r[:, hq:hq + hkv].to(torch.bfloat16)
    s["v"][at, :, off] = x[:, hq + hkv:].to(torch.bfloat16)
    return [r[:, :hq].to(torch.bfloat16), s["k"], s["v"]]


def _plain_attention(s):
    c = s["case"]
    hq, hkv, hd, B, T, R = c["hq"], c["hkv"], c["hd"], s["B"], s["T"], s["max_rows"]
    G = hq // hkv
    S = s["width"] * s["page"]
    cu, kv = s["cu"].long(), s["kv"].long()
    at = s["table"].long().clamp(min=0)

    def gather(pool):                                        # [B, hkv, S, hd]
        return pool[at].float().permute(0, 2, 1, 3, 4).reshape(B, hkv, S, hd)

    i = torch.arange(R, device=cu.device)
    q = s["q"][(cu[:-1, None] + i).clamp(max=T - 1)].float()           # [B, R, hq, hd]
    q = q.view(B, R, hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, hkv, R * G, hd)
    x = torch.matmul(q, gather(s["k"]).transpose(2, 3)) / math.sqrt(hd)  # [B, hkv, R*G, S]
    rows = cu[1:] - cu[:-1]
    limit = kv[:, None] + torch.zeros_like(i)
    if c["causal"]:
        limit = (kv - rows)[:, None] + i + 1
    see = torch.arange(S, device=cu.device) < torch.minimum(limit, kv[:, None])[:, :, None]
    see = see[:, None, :, None, :].expand(B, 1, R, G, S).reshape(B, 1, R * G, S)
    x = torch.where(see, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, gather(s["v"])) / z
    lse = (m + torch.log(z)).view(B, hkv, R, G).permute(0, 2, 1, 3).reshape(B, R, hq)
    o = o.view(B, hkv, R, G, hd).permute(0, 2, 1, 3, 4).reshape(B, R, hq, hd)
    row = torch.arange(T, device=cu.device)
    req = torch.searchsorted(cu, row, right=True) - 1
    return [o[req, row - cu[req]].to(torch.bfloat16), lse[req, row - cu[req]]]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention}[op](s)
    import block_discrete_diffusion_denoise_b200 as dg

    if op == "plan":
        dg.paged_plan(s["cached"], s["new"], s["table"], s["ring"], s["state"], s["page"], s["cu"], s["kv"],
                      s["positions"], s["slots"], s["state_out"])
        return [s["table"], s["ring"], s["cu"], s["kv"], s["positions"], s["slots"], s["state_out"]]
    if op == "append":
        dg.paged_append(s["qkv"], s["positions"], s["slots"], s["rope"], s["k"], s["v"], s["q"])
        return [s["q"], s["k"], s["v"]]
    dg.paged_attention(s["q"], s["k"], s["v"], s["table"], s["kv"], s["cu"], s["out"], lse=s["lse"],
                       causal=s["case"]["causal"], max_rows=s["max_rows"])
    return [s["out"], s["lse"]]


def work(case):
    lens = _lengths(case)
    page, B = case["page"], case["batch"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    T = sum(max(0, n) for _, n in lens)
    if case["op"] == "plan":
        moved = sum(abs(_pages(p + n, page) - _pages(p, page)) for p, n in lens)
        # the page ids that the new rows' slots are made of are read once each
        seen = sum(_pages(p + n, page) - p // page for p, n in lens if n > 0)
        return {"bytes": 4 * (2 * B + 4 + seen + 2 * moved + 2 * B + 1 + 2 * T + 4), "flops": 0}
    if case["op"] == "append":
        far = max(p + n for p, n in lens)
        return {"bytes": T * ((hq + 2 * hkv) * hd * 4 + 8) + min(T, far) * hd * 4, "flops": T * (hq + hkv) * hd * 3}
    keys = sum(p + n for p, n in lens)
    if case["causal"]:
        seen = sum(n * p + n * (n + 1) // 2 for p, n in lens)
    else:
        seen = sum(n * (p + n) for p, n in lens)
    table = sum(_pages(p + n, page) for p, n in lens)
    return {"bytes": keys * hkv * hd * 4 + T * hq * (hd * 4 + 4) + 4 * (table + 2 * B + 1), "flops": 4 * seen * hq * hd}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None                                           # whole numbers only
    s = prepare(case, seed)
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    lens = _lengths(case)
    if case["op"] == "append":
        x = s["qkv"].double().view(-1, hq + 2 * hkv, hd)
        # the table's own cos and sin are the operator's input: a pair (j, j + hd/2) is one complex number turned
        turn = torch.view_as_complex(s["rope"].double())[s["positions"].long()]
        k, v = s["k"].double(), s["v"].double()

        def rotated(h):
            z = torch.complex(x[:, h, : hd // 2], x[:, h, hd // 2:]) * turn
            return torch.cat([z.real, z.imag], -1)

        k_rows, v_rows = k.transpose(1, 2).reshape(-1, hkv, hd), v.transpose(1, 2).reshape(-1, hkv, hd)
        for h in range(hkv):
            k_rows[s["slots"].long(), h] = rotated(hq + h)
            v_rows[s["slots"].long(), h] = x[:, hq + hkv + h]
        back = [t.view(-1, page, hkv, hd).transpose(1, 2) for t in (k_rows, v_rows)]
        return [torch.stack([rotated(h) for h in range(hq)], 1), back[0], back[1]]
    out = torch.zeros(s["T"], hq, hd, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], hq, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (past, n) in enumerate(lens):
        keys = past + n
        ids = s["table"][b, : _pages(keys, page)].long()
        hidden = None
        if case["causal"]:
            hidden = torch.arange(keys, device="cuda")[None] > past + torch.arange(n, device="cuda")[:, None]
        for h in range(hkv):
            k = s["k"][ids, h].reshape(-1, hd)[:keys].double()
            v = s["v"][ids, h].reshape(-1, hd)[:keys].double()
            for a in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][t0:t0 + n, a].double() @ k.t() * hd ** -0.5
                if hidden is not None:
                    x.masked_fill_(hidden, -math.inf)
                lse[t0:t0 + n, a] = torch.logsumexp(x, 1)
                out[t0:t0 + n, a] = torch.softmax(x, 1) @ v
        t0 += n
    return [out, lse]
