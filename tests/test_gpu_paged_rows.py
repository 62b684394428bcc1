"""Entries of cu_rows that lie outside the call's rows, or decrease: a request
gets the rows of them that exist, and no other memory is touched."""
import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg

from test_gpu_paged import BF, SMALL, i32, paged_cache

pytestmark = pytest.mark.gpu

LO, HI = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_attention_with_row_sums_outside_the_call(rows, causal):
    g = torch.Generator().manual_seed(31)
    kv = [400, 330]
    q, k, v, table, _ = paged_cache(g, SMALL, 16, kv, [rows, rows])
    T = 2 * rows
    q, k, v, table = q.cuda(), k.cuda(), v.cuda(), table.cuda()

    def run(cu):
        guard = 64
        buf = torch.full((T + 2 * guard, *q.shape[1:]), 4.0, dtype=BF, device="cuda")
        lse = torch.full((T + 2 * guard, q.shape[1]), 4.0, device="cuda")
        dg.paged_attention(q, k, v, table, i32(kv), i32(cu), buf[guard:-guard], lse=lse[guard:-guard], causal=causal,
                           max_rows=rows)
        for edge in (slice(0, guard), slice(-guard, None)):
            assert (buf[edge] == 4).all() and (lse[edge] == 4).all()
        return buf, lse

    for bad, same in (([0, rows, LO], [0, rows, rows]), ([0, rows, rows - 1], [0, rows, rows]),
                      ([LO, rows, HI], [0, rows, T]), ([-1, rows, T + 1], [0, rows, T]), ([HI, LO, LO], [T, T, T]),
                      ([T + 1, T, T], [T, T, T])):
        for a, b in zip(run(bad), run(same)):
            assert torch.equal(a, b), bad
