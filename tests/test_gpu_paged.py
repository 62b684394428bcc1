"""The paged KV cache on the GPU: plan, append and attention against the plain
64-bit forms of paged_reference, at the sizes and masks where they can go
wrong, alone and as they are used together."""
import math
import random

import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg
import paged_reference as ref

pytestmark = pytest.mark.gpu

TINY, SMALL, A4B = (4, 2, 64), (8, 2, 128), (16, 8, 176)
BF = torch.bfloat16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def run_plan(cached, new, table, ring, state, page, cap, pad_cols=0):
    B, W = len(cached), len(table[0])
    wide = i32([r + [-9] * pad_cols for r in table])
    t = {"table": wide[:, :W], "ring": i32(ring), "state": i32(state), "cu": i32([-7] * (B + 1)),
         "kv": i32([-7] * B), "pos": i32([-7] * cap), "slot": i32([-7] * cap), "out": i32([-7] * 4)}
    dg.paged_plan(i32(cached), i32(new), t["table"], t["ring"], t["state"], page, t["cu"], t["kv"], t["pos"], t["slot"],
                  t["out"])
    torch.cuda.synchronize()
    assert (wide[:, W:] == -9).all()
    return {k: v.tolist() for k, v in t.items()}


def check_plan(cached, new, table, ring, state, page, cap, pad_cols=0):
    got = run_plan(cached, new, table, ring, state, page, cap, pad_cols)
    want = ref.plan(cached, new, table, ring, state, page, len(table[0]), cap)
    w_table, w_ring, w_cu, w_kv, w_pos, w_slot, w_out = want
    assert got["out"] == w_out
    assert got["cu"] == w_cu and got["kv"] == w_kv
    assert got["table"] == w_table and got["ring"] == w_ring
    n = len(w_pos)
    assert got["pos"][:n] == w_pos and got["slot"][:n] == w_slot
    assert all(x == -7 for x in got["pos"][n:] + got["slot"][n:])      # behind the last row
    assert got["state"] == state
    return got


def pool_state(rng, cached, page, spare, width=None):
    """tables over random pages and a ring holding the free ones, wrapped around its end"""
    held = [ref.pages_of(c, page) for c in cached]
    n_pages = sum(held) + spare
    ids = list(range(n_pages))
    rng.shuffle(ids)
    W = width or max(held + [1])
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (W - h))
        at += h
    free = ids[at:]
    head = rng.randrange(n_pages)
    ring = [-1] * n_pages
    for i, f in enumerate(free):
        ring[(head + i) % n_pages] = f
    return table, ring, [head, len(free)]


@pytest.mark.parametrize("batch,page,most,grow", [(1, 64, 2048, 256), (1, 16, 0, 1), (2, 32, 65, 40), (37, 16, 300, 33),
                                                  (149, 128, 1000, 300), (300, 64, 500, 70), (3, 16, 40, 9000)])
def test_plan_matches_the_bookkeeping(batch, page, most, grow):
    rng = random.Random(batch * 1000 + page)
    cached = [rng.randint(0, most) for _ in range(batch)]
    new = [max(-c, rng.randint(-grow // 2, grow)) for c in cached]
    new[0] = grow
    W = max(ref.pages_of(c + max(n, 0), page) for c, n in zip(cached, new)) + 2
    spare = sum(ref.pages_of(c + max(n, 0), page) - ref.pages_of(c, page) for c, n in zip(cached, new))
    table, ring, state = pool_state(rng, cached, page, spare + 3, W)
    rows = sum(max(0, n) for n in new)
    got = check_plan(cached, new, table, ring, state, page, rows + 5, pad_cols=3)
    assert got["out"][2:] == [0, 0]
    check_plan(cached, new, table, ring, state, page, rows)             # no row to spare


def test_plan_takes_the_last_free_page_and_not_one_more():
    rng = random.Random(5)
    cached = [10, 64, 0]
    table, ring, state = pool_state(rng, cached, 64, 3, 4)
    assert check_plan(cached, [55, 1, 64], table, ring, state, 64, 200)["out"][1:] == [0, 0, 0]
    assert check_plan(cached, [55, 1, 65], table, ring, state, 64, 200)["out"][1:] == [3, 1, 0]


def test_plan_releases_everything_and_counts_idle_requests():
    rng = random.Random(6)
    cached = [130, 1, 64, 0, 17]
    table, ring, state = pool_state(rng, cached, 16, 0, 9)
    got = check_plan(cached, [-130, -1, 0, 0, -1], table, ring, state, 16, 0)
    assert got["out"] == [state[0], 9 + 1 + 1, 0, 0] and got["kv"] == [0, 0, 64, 0, 16] and got["cu"] == [0] * 6


@pytest.mark.parametrize("what", ["length", "release", "width", "rows", "state", "huge"])
def test_plan_refuses_as_a_whole(what):
    rng = random.Random(7)
    cached, new = [20, 40, 5], [10, -20, 30]
    table, ring, state = pool_state(rng, cached, 16, 8, 5)
    cap = 100
    reason = {"length": 1, "release": 1, "width": 2, "rows": 4, "state": 8, "huge": 1}[what]
    if what == "length":
        cached[1] = -3
        new[1] = 5
    elif what == "release":
        new[1] = -41
    elif what == "width":
        new[2] = 16 * 5 - 5 + 1
    elif what == "rows":
        cap = 39
    elif what == "state":
        state = [len(ring), 2]
    else:
        cached[2], new[2] = 2 ** 31 - 5, 20
    if what == "huge":                      # the sum passes 32 bits: nothing is followed
        got = run_plan(cached, new, table, ring, state, 16, cap)
        assert got["out"][3] & 1 and got["table"] == table and got["ring"] == ring and got["kv"] == cached
        assert got["slot"][:30] == [-1] * 30
        return
    got = check_plan(cached, new, table, ring, state, 16, cap)
    assert got["out"][3] == reason


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("heads", [TINY, SMALL, A4B])
@pytest.mark.parametrize("page,rows,pad", [(16, 1, 0), (64, 77, 8), (128, 300, 64)])
def test_append_rotates_and_writes_only_its_slots(heads, page, rows, pad):
    hq, hkv, d = heads
    g = torch.Generator().manual_seed(rows)
    n_pages, n_pos = ref.pages_of(rows, page) + 3, 4000
    width = (hq + 2 * hkv) * d
    wide = torch.randn(rows, width + pad, generator=g).to(BF).cuda()
    qkv = wide[:, :width]
    pos = torch.randint(0, n_pos, (rows,), generator=g)
    slots = torch.randperm(n_pages * page, generator=g)[:rows]
    if rows > 8:
        slots[3], slots[5], slots[6] = -1, n_pages * page, 2 ** 31 - 1       # outside the pool
        pos[7] = n_pos                                                    # outside the table
        pos[8] = n_pos - 1
    rope = dg.rope_table(n_pos, d)
    k0 = torch.randn(n_pages, hkv, page, d, generator=g).to(BF)
    v0 = torch.randn(n_pages, hkv, page, d, generator=g).to(BF)
    k, v = k0.cuda(), v0.cuda()
    q = torch.full((rows, hq, d), 7.0, dtype=BF, device="cuda")
    extra = torch.full((4,), 5, dtype=torch.int32)
    dg.paged_append(qkv, torch.cat([pos.int(), extra]).cuda(), torch.cat([slots.int(), extra]).cuda(), rope, k, v, q)
    torch.cuda.synchronize()
    x = qkv.cpu().double().view(rows, hq + 2 * hkv, d)
    known = (pos >= 0) & (pos < n_pos)
    cs = rope.cpu().double()[pos.clamp(0, n_pos - 1)][:, None]
    y, mag = ref.rotate(x[:, : hq + hkv], cs[..., 0], cs[..., 1])
    tol = ref.rotate_bound(y, mag)
    qq = q.cpu().double()
    assert ((qq - y[:, :hq]).abs() <= tol[:, :hq])[known].all()
    assert torch.isnan(qq[~known]).all()
    kept = known & (slots >= 0) & (slots < n_pages * page)
    at, off = slots[kept] // page, slots[kept] % page
    kk, vv = k.cpu(), v.cpu()
    assert ((kk[at, :, off].double() - y[kept, hq:]).abs() <= tol[kept, hq:]).all()
    assert torch.equal(vv[at, :, off], x[kept, hq + hkv:].to(BF))
    kk[at, :, off] = k0[at, :, off]
    vv[at, :, off] = v0[at, :, off]
    assert torch.equal(kk, k0) and torch.equal(vv, v0)                   # nothing else moved


def test_append_reaches_pages_beyond_32_bit_offsets():
    hq, hkv, d = A4B
    page, rows = 64, 70
    n_pages = 2 ** 32 // (hkv * page * d) + 40                     # more than 2^32 elements in a pool
    g = torch.Generator().manual_seed(24)
    qkv = torch.randn(rows, (hq + 2 * hkv) * d, generator=g).to(BF).cuda()
    slots = (n_pages - 1 - torch.arange(rows)) * page + torch.arange(rows) % page
    small = [torch.empty(rows, hkv, page, d, dtype=BF, device="cuda") for _ in range(2)]
    big = [torch.empty(n_pages, hkv, page, d, dtype=BF, device="cuda") for _ in range(2)]
    q = [torch.empty(rows, hq, d, dtype=BF, device="cuda") for _ in range(2)]
    pos, rope = i32(list(range(rows))), dg.rope_table(rows, d)
    dg.paged_append(qkv, pos, slots.int().cuda(), rope, *big, q[0])
    near = torch.arange(rows) * page + torch.arange(rows) % page
    dg.paged_append(qkv, pos, near.int().cuda(), rope, *small, q[1])
    assert torch.equal(*q)
    r = torch.arange(rows, device="cuda")
    for b, s in zip(big, small):
        assert torch.equal(b[n_pages - 1 - r, :, r % page], s[r, :, r % page])


def test_rope_table_has_the_angles_of_far_positions():
    t = dg.rope_table(40000, 176).cpu().double()
    for p, j in [(0, 0), (1, 0), (39999, 0), (39999, 1), (12345, 87), (33023, 3)]:
        a = p * 10000.0 ** (-2.0 * j / 176)
        # cos and sin are rounded to fp32 once
        assert abs(t[p, j, 0] - math.cos(a)) <= ref.FP32_HALF and abs(t[p, j, 1] - math.sin(a)) <= ref.FP32_HALF


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def paged_cache(g, heads, page, kv_lens, rows, width_pad=0, spare=3, loud=0.0):
    """Pools with NaN wherever no request has a key (unused pages, the rest of
    last pages), a table with other ids behind the last pages, and packed
    queries; on the CPU."""
    hq, hkv, d = heads
    held = [ref.pages_of(max(n, 0), page) for n in kv_lens]
    n_pages = sum(held) + spare
    W = max(held + [1]) + width_pad
    ids = torch.randperm(n_pages, generator=g).int()
    k = torch.full((n_pages, hkv, page, d), math.nan, dtype=BF)
    v = k.clone()
    table = torch.full((len(kv_lens), W), -1, dtype=torch.int32)
    at = 0
    for b, (n, h) in enumerate(zip(kv_lens, held)):
        table[b, :h] = ids[at:at + h]
        table[b, h:] = torch.randint(-5, n_pages + 5, (W - h,), generator=g).int()
        for i in range(h):
            m = min(page, n - i * page)
            k[ids[at + i], :, :m] = torch.randn(hkv, m, d, generator=g).to(BF)
            v[ids[at + i], :, :m] = torch.randn(hkv, m, d, generator=g).to(BF) + loud
        at += h
    q = torch.randn(sum(rows), hq, d, generator=g).to(BF)
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return q, k, v, table, cu


def check_attention(q, k, v, table, kv_lens, cu, causal, max_rows=0, scale=None, dev=None):
    T, hq, d = q.shape
    out = torch.full((T, hq, d), 9.0, dtype=BF, device="cuda")
    lse = torch.full((T, hq), 9.0, device="cuda")
    qd, kd, vd, td = dev if dev else (q.cuda(), k.cuda(), v.cuda(), table.cuda())
    dg.paged_attention(qd, kd, vd, td, i32(kv_lens), i32(cu), out, lse=lse, causal=causal, max_rows=max_rows, scale=scale)
    torch.cuda.synchronize()
    w_out, w_lse, tol_o, tol_l = ref.attention(q, k, v, table, kv_lens, cu, causal, scale)
    o, l = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(o).all()
    worst = ((o - w_out).abs() - tol_o).max().item()
    assert worst <= 0, f"out beyond its bound by {worst}"
    empty = torch.isinf(w_lse)
    assert torch.equal(torch.isinf(l) & (l < 0), empty)
    assert (o[empty] == 0).all()
    assert ((l - w_lse).abs()[~empty] <= tol_l[~empty]).all()
    return out, lse


CASES = {
    "one token, one key": ([1], [1], True),
    "one token, lengths around a page": ([15, 16, 17, 63, 64, 65, 127, 128, 129], [1] * 9, True),
    "one token, long and short": ([1500, 1, 700, 2], [1] * 4, True),
    "one token, no keys for some": ([0, 5, 0, 70], [1] * 4, True),
    "no rows for some": ([40, 40, 0, 100], [0, 1, 0, 1], True),
    "a few rows, causal": ([9, 130, 5], [3, 5, 5], True),
    "a few rows, all keys": ([9, 130, 5], [3, 5, 5], False),
    "a canvas": ([300], [256], False),
    "canvases of 16 and none": ([16, 90, 700], [16, 0, 16], False),
    "causal chunks": ([129, 200, 70], [129, 100, 1], True),
    "causal, first rows see nothing": ([3, 150], [7, 200], True),
    "rows around a tile": ([140, 300, 260], [63, 129, 257], False),
    "single token among prompts": ([400, 65, 333], [1, 65, 333], True),
}


@pytest.mark.parametrize("heads", [TINY, SMALL, A4B])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("name", list(CASES))
def test_attention_matches_the_formula(name, page, heads):
    kv, rows, causal = CASES[name]
    g = torch.Generator().manual_seed(len(name) + page)
    q, k, v, table, cu = paged_cache(g, heads, page, kv, rows, width_pad=2)
    out, lse = check_attention(q, k, v, table, kv, cu, causal)
    # a bound of the rows picks the kernel, not the result
    check_attention(q, k, v, table, kv, cu, causal, max_rows=max(rows))


@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("kv,rows,causal", [([1000, 77, 4097], [1, 1, 1], True), ([1000, 4097], [256, 256], False),
                                            ([513, 1025], [500, 30], True)])
def test_attention_on_the_other_page_sizes(page, kv, rows, causal):
    g = torch.Generator().manual_seed(page)
    q, k, v, table, cu = paged_cache(g, A4B, page, kv, rows)
    check_attention(q, k, v, table, kv, cu, causal, max_rows=max(rows))


@pytest.mark.parametrize("heads", [(2, 2, 64), (32, 1, 128), (64, 4, 64), (128, 1, 64), (6, 6, 176)])
@pytest.mark.parametrize("rows", [1, 40])
def test_attention_on_other_head_groups(heads, rows):
    g = torch.Generator().manual_seed(heads[0])
    kv = [200, 31]
    q, k, v, table, cu = paged_cache(g, heads, 32, kv, [rows, min(rows, 31)])
    check_attention(q, k, v, table, kv, cu, True, max_rows=rows)


@pytest.mark.parametrize("rows", [1, 32])
def test_attention_over_many_requests(rows):
    rng = random.Random(3)
    kv = [rng.choice([rows, 33, 64, 100 + rng.randrange(60)]) + rows for _ in range(700 if rows == 1 else 90)]
    g = torch.Generator().manual_seed(4)
    q, k, v, table, cu = paged_cache(g, TINY, 16, kv, [rows] * len(kv))
    check_attention(q, k, v, table, kv, cu, True, max_rows=rows)


@pytest.mark.parametrize("batch", [31, 32, 33, 64, 65, 96, 97, 127, 128, 129, 257])
@pytest.mark.parametrize("most", [1, 70])
def test_stretches_start_in_the_right_request(batch, most):
    """batches around the sizes at which the search for a stretch's start changes, requests without rows among them"""
    rng = random.Random(batch)
    rows = [rng.choice([0, 1, most, rng.randint(1, most)]) for _ in range(batch)]
    rows[0], rows[-1] = 0, most
    kv = [n + rng.choice([0, 0, 15, 64, 130]) for n in rows]
    g = torch.Generator().manual_seed(batch)
    q, k, v, table, cu = paged_cache(g, TINY, 16, kv, rows)
    for causal in (True, False):
        check_attention(q, k, v, table, kv, cu, causal, max_rows=most)


def test_causal_prompts_of_more_than_32_row_tiles():
    g = torch.Generator().manual_seed(23)
    kv, rows = [4300, 90, 8400], [4250, 3, 8400]
    q, k, v, table, cu = paged_cache(g, (2, 1, 64), 64, kv, rows)
    check_attention(q, k, v, table, kv, cu, True)


@pytest.mark.parametrize("rows", [1, 64])
def test_attention_masks_pages_outside_the_pool(rows):
    g = torch.Generator().manual_seed(8)
    kv = [640, 200, 100]
    q, k, v, table, cu = paged_cache(g, SMALL, 16, kv, [rows] * 3)
    table[0, 0], table[0, 7], table[0, 39] = -1, k.shape[0], 2 ** 31 - 1
    table[1, 3:9] = -2 ** 31
    table[2] = -1                                                # a request without one good page
    check_attention(q, k, v, table, kv, cu, False, max_rows=rows)


@pytest.mark.parametrize("rows", [1, 64])
def test_attention_clamps_lengths_to_the_table(rows):
    g = torch.Generator().manual_seed(9)
    q, k, v, table, cu = paged_cache(g, SMALL, 16, [160, 96], [rows] * 2)
    kv = [2 ** 31 - 1, -4]
    w = [160, 0]
    k2 = k.clone()
    k2[torch.isnan(k2)] = 1.0
    out, lse = check_attention(q, k2, torch.nan_to_num(v, nan=2.0), table, w, cu, False, max_rows=rows)
    o2 = torch.empty_like(out)
    dg.paged_attention(q.cuda(), k2.cuda(), torch.nan_to_num(v, nan=2.0).cuda(), table.cuda(), i32(kv), i32(cu), o2,
                       max_rows=rows)
    assert torch.equal(o2, out)


@pytest.mark.parametrize("rows", [1, 3, 64])
def test_causal_rows_keep_their_places_beyond_the_table(rows):
    """a row's last key goes by the request's own length, where the table holds fewer pages too"""
    g = torch.Generator().manual_seed(22)
    q, k, v, table, cu = paged_cache(g, SMALL, 16, [160, 96], [rows] * 2)
    k, v = torch.nan_to_num(k, nan=1.0), torch.nan_to_num(v, nan=2.0)
    table = table.clamp(0, k.shape[0] - 1)
    check_attention(q, k, v, table, [table.shape[1] * 16 + 30, 96 + 2], cu, True, max_rows=rows)
    check_attention(q, k, v, table, [table.shape[1] * 16 + 3, 90], cu, True, max_rows=rows)


@pytest.mark.parametrize("rows", [1, 40])
def test_attention_takes_strided_queries_and_tables(rows):
    hq, hkv, d = A4B
    g = torch.Generator().manual_seed(10)
    kv, n = [300, 75], [rows, rows]
    q, k, v, table, cu = paged_cache(g, A4B, 64, kv, n)
    T = q.shape[0]
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g).to(BF)
    qkv[:, : hq * d] = q.view(T, -1)
    wide = torch.full((2, table.shape[1] + 5), -3, dtype=torch.int32)
    wide[:, : table.shape[1]] = table
    qd, td = qkv.cuda()[:, : hq * d].view(T, hq, d), wide.cuda()[:, : table.shape[1]]
    assert not qd.is_contiguous() and not td.is_contiguous()
    check_attention(q, k, v, table, kv, cu, True, max_rows=rows, dev=(qd, k.cuda(), v.cuda(), td))


@pytest.mark.parametrize("rows", [1, 40])
def test_attention_leaves_rows_outside_the_requests(rows):
    g = torch.Generator().manual_seed(11)
    kv = [100, 90]
    q, k, v, table, cu = paged_cache(g, SMALL, 16, kv, [rows] * 2)
    pad = torch.full((5, *q.shape[1:]), math.nan, dtype=BF)
    q2 = torch.cat([pad, q, pad])
    out = torch.full_like(q2, 4.0, device="cuda")
    lse = torch.full(q2.shape[:2], 4.0, device="cuda")
    dg.paged_attention(q2.cuda(), k.cuda(), v.cuda(), table.cuda(), i32(kv), i32([5 + c for c in cu]), out, lse=lse,
                       max_rows=rows)
    plain, l = check_attention(q, k, v, table, kv, cu, False, max_rows=rows)
    assert torch.equal(out[5:-5], plain) and torch.equal(lse[5:-5], l)
    for edge in (slice(0, 5), slice(-5, None)):
        assert (out[edge] == 4).all() and (lse[edge] == 4).all()


@pytest.mark.parametrize("batch", [1, 300])
@pytest.mark.parametrize("rows", [1, 600])
def test_attention_of_rows_that_belong_to_no_request(batch, rows):
    """no request has a row: nothing is written, whatever the workspace held"""
    g = torch.Generator().manual_seed(20)
    q, k, v, table, cu = paged_cache(g, TINY, 16, [40] * batch, [0] * batch)
    q = torch.randn(rows, 4, 64, generator=g).to(BF).cuda()
    out = torch.full_like(q, 4.0)
    lse = torch.full((rows, 4), 4.0, device="cuda")
    for fill in (0x7f, 0x01):
        torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")          # freed: the workspace's next memory
        dg.paged_attention(q, k.cuda(), v.cuda(), table.cuda(), i32([40] * batch), i32(cu), out, lse=lse)
    assert (out == 4).all() and (lse == 4).all()


def test_attention_refuses_memory_that_it_would_overwrite():
    g = torch.Generator().manual_seed(21)
    q, k, v, table, cu = paged_cache(g, SMALL, 16, [40], [20])
    a = [t.cuda() for t in (q, k, v, table)]
    for out in (a[0], a[1].view(-1)[:20 * 8 * 128].view(20, 8, 128)):
        with pytest.raises(dg.DGError) as e:
            dg.paged_attention(*a, i32([40]), i32(cu), out)
        assert e.value.status == dg.DG_ERR_INVALID_ARG


@pytest.mark.parametrize("rows", [1, 40])
def test_attention_with_large_scores_and_values(rows):
    """scores far from zero in both directions, and one key that takes all the weight"""
    g = torch.Generator().manual_seed(12)
    kv = [333, 128]
    q, k, v, table, cu = paged_cache(g, SMALL, 64, kv, [rows] * 2, loud=30.0)
    k[table[0, 2], :, 5] *= 40.0
    check_attention(q * 6, k, v, table, kv, cu, False, max_rows=rows)
    check_attention(q, k, v, table, kv, cu, False, max_rows=rows, scale=1e-6)
    check_attention(q, k, v, table, kv, cu, False, max_rows=rows, scale=3.0)


@pytest.mark.parametrize("rows", [1, 40])
def test_attention_with_infinite_and_nan_operands(rows):
    """-inf scores take no weight; a NaN key makes its rows NaN and no others"""
    g = torch.Generator().manual_seed(13)
    kv = [200, 200]
    q, k, v, table, cu = paged_cache(g, TINY, 16, kv, [rows] * 2)
    q = q.abs() + 0.1
    k[table[0, 3], :, 2] = -3e38                                   # its scores overflow to -inf or nearly
    k[table[1, 1], :, 4] = math.nan
    out = torch.empty_like(q, device="cuda")
    dg.paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), i32(kv), i32(cu), out, max_rows=rows)
    o = out.cpu()
    assert torch.isnan(o[cu[1]:]).all()
    k[table[0, 3], :, 2] = -100.0                                  # weightless in 32 bits all the same
    w, _, tol, _ = ref.attention(q, k, torch.nan_to_num(v), table, kv, cu, False)
    assert ((o[: cu[1]].double() - w[: cu[1]]).abs() <= tol[: cu[1]]).all()


@pytest.mark.parametrize("rows", [1, 300])
def test_attention_reaches_pages_beyond_32_bit_offsets(rows):
    hq, hkv, d = A4B
    page = 64
    n_pages = 2 ** 32 // (hkv * page * d) + 40                     # more than 2^32 elements in a pool
    g = torch.Generator().manual_seed(14)
    kv = [rows + 500]
    q, k, v, table, cu = paged_cache(g, A4B, page, kv, [rows])
    big = [torch.empty(n_pages, hkv, page, d, dtype=BF, device="cuda") for _ in range(2)]
    shift = n_pages - k.shape[0]
    for b, s in zip(big, (k, v)):
        b[shift:] = s.cuda()
    check_attention(q, k, v, table, kv, cu, True, max_rows=rows, dev=(q.cuda(), *big, (table + shift).cuda()))


@pytest.mark.parametrize("rows", [1, 256])
def test_attention_is_the_same_every_time(rows):
    g = torch.Generator().manual_seed(15)
    kv = [1000 + rows, 77 + rows, 3000 + rows]
    q, k, v, table, cu = paged_cache(g, A4B, 64, kv, [rows] * 3)
    a = [t.cuda() for t in (q, k, v, table)]
    outs = []
    for _ in range(4):
        out, lse = torch.empty_like(a[0]), torch.empty(q.shape[:2], device="cuda")
        dg.paged_attention(*a, i32(kv), i32(cu), out, lse=lse, causal=True, max_rows=rows)
        outs.append((out, lse))
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])


# ---------------------------------------------------------------------------
# what the binding refuses
# ---------------------------------------------------------------------------
def refusals(fn, good, bad):
    """fn takes the good arguments; each of the bad ones in an argument's place is refused, with its name said"""
    fn(**good)
    for name, values in bad.items():
        for v in values:
            with pytest.raises(dg.DGError) as e:
                fn(**{**good, name: v})
            assert e.value.status == dg.DG_ERR_INVALID_ARG and (name in str(e.value) or "q" in str(e.value)), (name, e.value)
    torch.cuda.synchronize()


def misfits(t, shorter=True):
    """t on the host, of another type, strided, and one element short"""
    wide = torch.stack([t, t], -1)[..., 0]
    return [t.cpu(), t.double(), wide if t.numel() > 1 else t.cpu(), None] + \
        ([t[:-1]] if shorter and t.dim() == 1 else [])


def test_plan_refuses_misfits():
    good = dict(cached_lens=i32([5, 70]), new_rows=i32([3, 1]), block_table=i32([[0, -1], [1, 2]]),
                free_pages=i32(range(9)), free_state=i32([3, 6]), page_size=64, cu_rows=i32([0] * 3), kv_lens=i32([0] * 2),
                positions=i32([0] * 8), slots=i32([0] * 8), free_state_out=i32([0] * 4))
    bad = {k: misfits(v, k not in ("free_pages", "slots")) for k, v in good.items() if k not in ("page_size", "block_table")}
    bad["block_table"] = [good["block_table"].cpu(), good["block_table"].long(), i32([0, 1]), i32([[0, 1], [2, 3]]).t(),
                          None, i32([[], []])]
    refusals(dg.paged_plan, good, bad)
    for page in (2 ** 32 + 64, None, "64", 64.0):
        with pytest.raises(dg.DGError) as e:
            dg.paged_plan(**{**good, "page_size": page})
        assert e.value.status == dg.DG_ERR_INVALID_ARG and "page_size" in str(e.value)
    with pytest.raises(dg.DGError) as e:
        dg.paged_plan(**{**good, "page_size": 48})
    assert e.value.status == dg.DG_ERR_UNSUPPORTED


def test_append_refuses_misfits():
    good = dict(qkv=torch.zeros(4, 512, dtype=BF, device="cuda"), positions=i32([0] * 4), slots=i32(range(4)),
                rope=dg.rope_table(10, 64), k_pages=torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda"),
                v_pages=torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda"),
                q_out=torch.zeros(4, 4, 64, dtype=BF, device="cuda"))
    bad = {k: misfits(v) for k, v in good.items()}
    bad["qkv"] += [good["qkv"][:3], torch.zeros(4, 448, dtype=BF, device="cuda")]
    bad["rope"] += [dg.rope_table(10, 128)]
    bad["v_pages"] += [torch.zeros(3, 2, 16, 64, dtype=BF, device="cuda")]
    refusals(dg.paged_append, good, bad)


def test_attention_refuses_misfits():
    good = dict(q=torch.zeros(4, 4, 64, dtype=BF, device="cuda"), k_pages=torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda"),
                v_pages=torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda"), block_table=i32([[0, 1], [1, 0]]),
                kv_lens=i32([20, 3]), cu_rows=i32([0, 2, 4]), out=torch.zeros(4, 4, 64, dtype=BF, device="cuda"),
                lse=torch.zeros(4, 4, device="cuda"))
    bad = {k: misfits(v) for k, v in good.items() if k != "block_table"}
    bad["lse"] = [x for x in bad["lse"] if x is not None] + [torch.zeros(4, 5, device="cuda")]
    bad["out"] += [good["out"][:3]]
    bad["q"] += [torch.zeros(4, 4, 128, dtype=BF, device="cuda")]
    bad["block_table"] = [good["block_table"].cpu(), good["block_table"].long(), i32([0, 1]), i32([[0, 1], [2, 3]]).t(), None]
    refusals(dg.paged_attention, good, bad)
    for kw in (dict(max_rows=1.5), dict(max_rows=None), dict(scale=1e39), dict(scale="1"), dict(scale=0.0),
               dict(scale=math.nan)):
        with pytest.raises(dg.DGError) as e:
            dg.paged_attention(**good, **kw)
        assert e.value.status == dg.DG_ERR_INVALID_ARG, kw
    dg.paged_attention(**good, max_rows=2 ** 40)                 # a bound above the rows says nothing
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Server:
    """A small serving loop: lengths on the host, everything else in the pages."""

    def __init__(self, heads, page, batch, n_pages, cap):
        hq, hkv, d = heads
        self.heads, self.page, self.cap = heads, page, cap
        self.k = torch.full((n_pages, hkv, page, d), math.nan, dtype=BF, device="cuda")
        self.v = self.k.clone()
        self.table = torch.full((batch, n_pages), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.randperm(n_pages).int().cuda()
        self.state = [i32([0, n_pages, 0, 0]), i32([0] * 4)]
        self.cached = i32([0] * batch)
        self.kv, self.cu = i32([0] * batch), i32([0] * (batch + 1))
        self.pos, self.slot = i32([0] * cap), i32([0] * cap)
        self.rope = dg.rope_table(n_pages * page, d)

    def turn(self, new, qkv, causal, max_rows=0, commit=True):
        hq, hkv, d = self.heads
        dg.paged_plan(self.cached, new, self.table, self.ring, self.state[0], self.page, self.cu, self.kv, self.pos,
                      self.slot, self.state[1])
        self.state.reverse()
        self.q = q = torch.empty(qkv.shape[0], hq, d, dtype=BF, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        dg.paged_append(qkv, self.pos, self.slot, self.rope, self.k, self.v, q)
        dg.paged_attention(q, self.k, self.v, self.table, self.kv, self.cu, out, lse=lse, causal=causal,
                           max_rows=max_rows)
        self.cached.copy_(self.kv)
        return out, lse


def rotated(heads, history):
    """(rows, bound) of the q and k heads of one request's whole history of qkv rows, in 64 bits"""
    hq, hkv, d = heads
    x = history.double().view(-1, hq + 2 * hkv, d)
    j = torch.arange(d // 2, dtype=torch.float64)
    a = torch.arange(x.shape[0], dtype=torch.float64)[:, None] * 10000.0 ** (-2 * j / d)
    y, mag = ref.rotate(x[:, : hq + hkv], a.cos()[:, None], a.sin()[:, None])
    # the table's cos and sin are rounded to fp32 (2^-24 of each product) on top of the kernel's own arithmetic
    return y, ref.rotate_bound(y, mag) + ref.FP32_HALF * mag


@pytest.mark.parametrize("heads,page", [(TINY, 16), (A4B, 64)])
def test_a_serving_loop_of_plan_append_attention(heads, page):
    """Every turn's q and every key and value of every request stand in the pages as its history says, and the
    attention is that of these operands."""
    hq, hkv, d = heads
    width = (hq + 2 * hkv) * d
    g = torch.Generator().manual_seed(16)
    s = Server(heads, page, 4, 64, 400)
    history = [torch.empty(0, width, dtype=BF) for _ in range(4)]
    turns = [([100, 1, 37, 0], True), ([1, 1, 1, 60], True), ([16, 16, 16, 16], False), ([-16, -16, 0, -76], None),
             ([1, 1, 1, 1], True), ([64, 0, -54, 2], False), ([3, 3, 3, 3], True)]
    for new, causal in turns:
        rows = [max(0, n) for n in new]
        qkv = torch.randn(sum(rows), width, generator=g).to(BF)
        out, lse = s.turn(i32(new), qkv.cuda(), bool(causal))
        q, k, v, table = s.q.cpu(), s.k.cpu(), s.v.cpu(), s.table.cpu()
        cu = [0]
        for b, n in enumerate(new):
            cu.append(cu[-1] + max(0, n))
            history[b] = torch.cat([history[b][: len(history[b]) + min(0, n)], qkv[cu[b]:cu[b + 1]]])
            if not len(history[b]):
                continue
            y, tol = rotated(heads, history[b])
            t = torch.arange(len(history[b]))
            at, off = table[b, t // page].long(), t % page
            assert ((k[at, :, off].double() - y[:, hq:]).abs() <= tol[:, hq:]).all()
            assert torch.equal(v[at, :, off], history[b].view(-1, hq + 2 * hkv, d)[:, hq + hkv:])
            if n > 0:
                assert ((q[cu[b]:cu[b + 1]].double() - y[-n:, :hq]).abs() <= tol[-n:, :hq]).all()
        lens = [len(h) for h in history]
        assert s.kv.tolist() == lens
        w, w_lse, tol, tol_l = ref.attention(q, k, v, table, lens, cu, bool(causal))
        assert ((out.cpu().double() - w).abs() <= tol).all()
        assert ((lse.cpu().double() - w_lse).abs() <= tol_l).all()
    state = s.state[0].tolist()
    held = sum(ref.pages_of(len(h), page) for h in history)
    assert state[1] == 64 - held and state[2:] == [0, 0]
    free = [s.ring[(state[0] + i) % 64].item() for i in range(state[1])]
    used = [s.table[b, i].item() for b in range(4) for i in range(ref.pages_of(len(history[b]), page))]
    assert sorted(free + used) == list(range(64))                   # every page once


@pytest.mark.parametrize("rows", [1, 48])
def test_captured_calls_replay_with_other_lengths(rows):
    """The three calls captured once and replayed with other lengths and rows
    give what eager calls give; two captures replayed on two streams do not
    meet in a workspace."""
    heads, page, B = SMALL, 16, 3
    hq, hkv, d = heads
    width = (hq + 2 * hkv) * d
    g = torch.Generator().manual_seed(17)
    T = rows * B

    def server():
        torch.manual_seed(0)
        return Server(heads, page, B, 200, T)

    fill = torch.randn(3, T, width, generator=g).to(BF).cuda()
    new_rows = i32([rows] * B)
    eager = server()
    want = [tuple(t.clone() for t in eager.turn(new_rows, fill[i], True, rows)) for i in range(3)]

    graphs = []
    for _ in range(2):
        s = server()
        qkv = fill[0].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):                              # warm-up off the current stream
            server().turn(new_rows, qkv, True, rows)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = s.turn(new_rows, qkv, True, rows)
            s.state[1].copy_(s.state[0])                           # the next replay reads what this one wrote
        graphs.append((graph, s, qkv, got, torch.cuda.Stream()))
    for graph, s, qkv, got, st in graphs:                           # state as before the capture
        f = server()
        for a in ("k", "v", "table", "ring", "cached"):
            getattr(s, a).copy_(getattr(f, a))
        for t in s.state:
            t.copy_(f.state[0])
    torch.cuda.synchronize()
    for i in range(3):
        for graph, s, qkv, got, st in graphs:
            with torch.cuda.stream(st):
                qkv.copy_(fill[i])
                graph.replay()
        torch.cuda.synchronize()
        for graph, s, qkv, got, st in graphs:
            assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])


@pytest.mark.parametrize("rows", [1, 64])
def test_calls_on_a_side_stream_wait_for_it(rows):
    g = torch.Generator().manual_seed(18)
    kv = [500 + rows, 64 + rows]
    q, k, v, table, cu = paged_cache(g, A4B, 64, kv, [rows] * 2)
    want, _ = check_attention(q, k, v, table, kv, cu, True, max_rows=rows)
    side = torch.cuda.Stream()
    kd, vd, td, kvd, cud = k.cuda(), v.cuda(), table.cuda(), i32(kv), i32(cu)
    src = q.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        qd = torch.zeros_like(src)
        out = torch.empty_like(src)
        torch.cuda._sleep(20_000_000)
        qd.copy_(src)                                              # ready late, on the side stream
        dg.paged_attention(qd, kd, vd, td, kvd, cud, out, causal=True, max_rows=rows)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [1, 64])
def test_two_streams_at_once(rows):
    g = torch.Generator().manual_seed(19)
    sets = []
    for i in range(2):
        kv = [2000 + 100 * i + rows, 64 + rows, 900 + rows]
        q, k, v, table, cu = paged_cache(g, A4B, 64, kv, [rows] * 3)
        want, _ = check_attention(q, k, v, table, kv, cu, True, max_rows=rows)
        sets.append(([t.cuda() for t in (q, k, v, table)], i32(kv), i32(cu), want, torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, kv, cu, want, st, outs in sets:
            with torch.cuda.stream(st):
                out = torch.empty_like(a[0])
                dg.paged_attention(*a, kv, cu, out, causal=True, max_rows=rows)
                outs.append(out)
    torch.cuda.synchronize()
    for a, kv, cu, want, st, outs in sets:
        assert all(torch.equal(o, want) for o in outs)
