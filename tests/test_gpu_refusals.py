"""Calls that a context refuses before it launches anything."""
import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg
import synth_inputs as si

from gpu_helpers import make_context

pytestmark = pytest.mark.gpu


def refused(status, fn, *a, **kw):
    with pytest.raises(dg.DGError) as e:
        fn(*a, **kw)
    assert e.value.status == status


def test_a_prefix_near_the_end_of_32_bits_is_beyond_capacity():
    w = si.workload("tiny")
    ctx, _ = make_context(w, max_seq=400)
    t = torch.zeros(64, dtype=torch.int32, device="cuda")
    for n in (145, 2 ** 31 - 256, 2 ** 31 - 1):                  # 145 + 256 > 400
        assert ctx.lib.dg_prefill(ctx.ctx, t.data_ptr(), 1, n) == 3
        refused(3, ctx._check, ctx.lib.dg_prefill(ctx.ctx, t.data_ptr(), 1, n))
    ctx.close()
