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


def test_sampler_hooks_of_a_ragged_batch_take_its_sequences_only():
    w = si.workload("tiny").with_(batch=4)
    ctx, _ = make_context(w, max_seq=400)
    am = torch.zeros(5, 256, dtype=torch.int32, device="cuda")
    conf, ent = torch.ones(5, 256, device="cuda"), torch.zeros(5, 256, device="cuda")
    out = torch.full((5, 256), -7, dtype=torch.int32, device="cuda")
    ctx.prefill_ragged(torch.zeros(30, dtype=torch.int32, device="cuda"), [20, 10])
    for n in (3, 4, 5):
        refused(1, ctx.debug_sample, am, conf, n, 0, 1, 0.5, out)
        refused(1, ctx.debug_entropy_sample, am, ent, None, n, 0, 1, 1.0, 0.1, out)
    ctx.sync()
    assert (out == -7).all()
    ctx.debug_sample(am, conf, 2, 0, 1, 0.5, out)
    ctx.sync()
    assert (out[:2] == 0).all() and (out[2:] == -7).all()
    # one length for all: any batch
    ctx.prefill(torch.zeros(2, 20, dtype=torch.int32, device="cuda"))
    ctx.debug_sample(am, conf, 5, 0, 1, 0.5, out)
    ctx.debug_entropy_sample(am, ent, None, 4, 0, 1, 1.0, 0.1, out)
    ctx.sync()
    ctx.close()
