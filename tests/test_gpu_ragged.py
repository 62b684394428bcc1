"""Ragged batches of a context (dg_prefill_ragged): prompts of different
lengths whose keys and values lie in pages of the context's cache.  Every
sequence is compared with the oracle run on it alone, at its own positions;
the threshold and the entropy sampler draw at those positions; graph and eager
steps agree; and the regular batches before and after it are unaffected."""
import numpy as np
import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg
import oracle
import synth_inputs as si
from oracle import model as om

from gpu_helpers import compare_step, device_weights_oracle, gpu_step, make_context, oracle_step

pytestmark = pytest.mark.gpu


def prompts(w, lens):
    """token rows of the prefix generator, cut to the lengths"""
    t = si.uniform_tokens(w, "prefix", len(lens), max(lens))
    return [t[b, :n].contiguous() for b, n in enumerate(lens)]


def packed(parts):
    return torch.cat(parts).cuda()


def of_sequence(g, b):
    """sequence b of a recorded GPU step"""
    one = slice(b, b + 1)
    return {k: [x[one] for x in v] if isinstance(v, list) else v[one] for k, v in g.items()}


def canvas_of(w, block=0):
    return si.uniform_tokens(w, "canvas", w.batch, w.canvas, block=block).numpy()


@pytest.mark.parametrize("name,layers,lens,blocks", [("tiny", 2, [130, 37, 1], 2), ("small", 1, [200, 64], 1)])
def test_every_sequence_matches_the_oracle_on_it_alone(name, layers, lens, blocks):
    w = si.workload(name).with_layers(layers).with_(batch=len(lens))
    ctx, weights = make_context(w, max_seq=max(lens) + 2 * w.canvas)
    parts = prompts(w, lens)
    ctx.prefill_ragged(packed(parts), lens)
    assert ctx.cached_lens == lens and ctx.cached_len == max(lens)
    steps = []
    for k in range(blocks):
        if k:
            ctx.commit_block(torch.as_tensor(canvas_of(w, k - 1)).cuda())
            assert ctx.cached_lens == [n + k * w.canvas for n in lens]
        steps.append(gpu_step(ctx, w, canvas_of(w, k), k, 7, 0.9, capture=True))
    ctx.close()
    orc = device_weights_oracle(w, weights, keep_layers=True, seqs=[0])
    for b, t in enumerate(parts):
        orc.seq_ids = np.array([b])
        orc.prefill(t.numpy()[None])
        for k, g in enumerate(steps):
            if k:
                orc.commit_block(canvas_of(w, k - 1)[b:b + 1])
            gb = of_sequence(g, b)
            compare_step(gb, oracle_step(orc, canvas_of(w, k)[b:b + 1], k, 7, 0.9, 1.0, gb), 0.9, orc=orc)


def test_prompts_longer_than_a_prefill_chunk():
    """1500 packed tokens go in chunks of 1280, the first of which ends inside the fourth prompt"""
    lens = [500, 3, 700, 256, 41]
    w = si.workload("tiny").with_(batch=5)
    ctx, weights = make_context(w, max_seq=960, prefill_rows=1)         # R = batch * canvas = 1280
    parts = prompts(w, lens)
    ctx.prefill_ragged(packed(parts), lens)
    assert ctx.cached_lens == lens
    g = gpu_step(ctx, w, canvas_of(w), 0, 3, 0.9, capture=True)
    ctx.close()
    orc = device_weights_oracle(w, weights, keep_layers=True, seqs=[0])
    for b in (3, 4):
        orc.seq_ids = np.array([b])
        orc.prefill(parts[b].numpy()[None])
        gb = of_sequence(g, b)
        compare_step(gb, oracle_step(orc, canvas_of(w)[b:b + 1], 0, 3, 0.9, 1.0, gb), 0.9, orc=orc)


def test_graph_and_eager_steps_agree_over_blocks():
    lens = [100, 1, 333]
    w = si.workload("tiny").with_(batch=3)
    results = []
    for graph in (False, True):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            ctx, weights = make_context(w, max_seq=333 + 3 * 256, stream=st.cuda_stream if graph else None)
            got = []
            if not graph:
                torch.cuda.synchronize()
            ctx.prefill_ragged(packed(prompts(w, lens)), lens)
            for block in range(2):
                cur = torch.as_tensor(canvas_of(w, block)).cuda()
                if not graph:
                    torch.cuda.synchronize()
                for step in range(2):
                    out = torch.empty_like(cur)
                    conf = torch.empty(3, 256, device="cuda")
                    settled = torch.empty(3, dtype=torch.int32, device="cuda")
                    ctx.denoise_step(cur, step, 11, 0.4, out, conf, settled)
                    ctx.sync()
                    got += [out.clone(), conf.clone(), settled.clone()]
                    cur = out
                ctx.commit_block(cur)
            ctx.sync()
            results.append(got)
            ctx.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_entropy_steps_with_self_conditioning_and_host_steps():
    """graph and eager agree there too, with a regular batch in between (its graphs are others), and a step on host
    buffers gives what one on the device does"""
    lens = [100, 1, 333]
    w = si.workload("tiny").with_(batch=3)
    results = []
    for graph in (False, True):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            weights = {**si.model_weights(w, "cuda"), **si.self_cond_weights(w, "cuda")}
            ctx, _ = make_context(w, max_seq=333 + 3 * 256, weights=weights, stream=st.cuda_stream if graph else None)
            got = []
            regular = si.uniform_tokens(w, "prefix", 3, 90).cuda()
            tokens = packed(prompts(w, lens))
            canvas = torch.as_tensor(canvas_of(w)).cuda()
            ctx.set_self_conditioning(True)
            for ragged in (True, False, True):
                torch.cuda.synchronize()
                ctx.prefill_ragged(tokens, lens) if ragged else ctx.prefill(regular)
                cur, prev = canvas, None
                for step in range(2):
                    out, am = torch.empty_like(cur), torch.empty_like(cur)
                    ent = torch.empty(3, 256, device="cuda")
                    if not graph:
                        torch.cuda.synchronize()
                    ctx.denoise_step_entropy(cur, step, 11, 0.8, 20.0, 0.005, out, prev_argmax=prev, argmax_out=am,
                                             entropy=ent)
                    ctx.sync()
                    got += [out.clone(), am.clone(), ent.clone()]
                    cur, prev = out, am
                ctx.commit_block(cur)
                ctx.sync()
            ctx.set_self_conditioning(False)
            out, conf = torch.empty_like(canvas), torch.empty(3, 256, device="cuda")
            if not graph:
                torch.cuda.synchronize()
            ctx.denoise_step(canvas, 1, 5, 0.4, out, conf)
            ctx.sync()
            h_out, h_conf = np.zeros((3, 256), np.int32), np.zeros((3, 256), np.float32)
            ctx.denoise_step_host(canvas_of(w).astype(np.int32), 1, 5, 0.4, h_out, h_conf)
            np.testing.assert_array_equal(h_out, out.cpu().numpy())
            np.testing.assert_array_equal(h_conf, conf.cpu().numpy())
            results.append(got)
            ctx.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    for a, b in zip(results[0][:6], results[0][12:]):              # the second ragged batch gives what the first did
        assert torch.equal(a, b)


def test_samplers_draw_at_each_sequences_own_positions():
    lens = [16, 200, 77]
    w = si.workload("tiny").with_(batch=3)
    ctx, _ = make_context(w, max_seq=600)
    ctx.prefill_ragged(packed(prompts(w, lens)), lens)
    C, V, seed = w.canvas, w.shape.vocab, 0x0123456789ABCDEF
    g = torch.Generator().manual_seed(3)
    am = torch.randint(0, V, (3, C), generator=g, dtype=torch.int32)
    conf = torch.rand(3, C, generator=g)
    ent = torch.rand(3, C, generator=g) * 2.0
    out = torch.empty(3, C, dtype=torch.int32, device="cuda")
    ctx.debug_sample(am.cuda(), conf.cuda(), 3, 5, seed, 0.5, out)
    ent_out = torch.empty_like(out)
    ctx.debug_entropy_sample(am.cuda(), ent.cuda(), None, 3, 5, seed, 3.0, 0.01, ent_out)
    ctx.sync()
    for b in range(3):
        noise = om.renoise_tokens(np.arange(lens[b], lens[b] + C), 5, b, seed, V)
        np.testing.assert_array_equal(out[b].cpu().numpy(), om.sample(am[b].numpy(), conf[b].numpy(), 0.5, noise))
        ref, _ = om.entropy_sample(am[b].numpy(), ent[b].numpy(), None, 3.0, 0.01, noise)
        np.testing.assert_array_equal(ent_out[b].cpu().numpy(), ref)
    ctx.close()


def test_regular_batches_before_and_after_a_ragged_one():
    w = si.workload("tiny").with_(batch=2)
    ctx, _ = make_context(w, max_seq=700)
    tokens = si.uniform_tokens(w, "prefix", 2, 90).cuda()
    canvas = canvas_of(w)
    ctx.prefill(tokens)
    before = gpu_step(ctx, w, canvas, 0, 1, 0.9)
    ctx.prefill_ragged(packed(prompts(w, [90, 90])), [90, 90])
    ragged = gpu_step(ctx, w, canvas, 0, 1, 0.9)
    ctx.prefill(tokens)
    assert ctx.cached_lens == [90, 90]
    after = gpu_step(ctx, w, canvas, 0, 1, 0.9)
    for k in ("canvas_out", "conf", "argmax", "lse"):
        np.testing.assert_array_equal(before[k], after[k])
    # equal lengths: the same model on the same tokens
    assert np.abs(before["lse"] - ragged["lse"]).max() < 5e-2
    ctx.close()


def test_capacity_is_checked_before_anything_runs():
    w = si.workload("tiny").with_(batch=2)
    ctx, _ = make_context(w, max_seq=400)              # 800 positions: 12 pages of 64
    t = torch.zeros(2000, dtype=torch.int32, device="cuda")
    with pytest.raises(dg.DGError) as e:
        ctx.prefill_ragged(t, [145, 10])               # 145 + 256 > 400
    assert e.value.status == 3
    with pytest.raises(dg.DGError) as e:
        ctx.prefill_ragged(t, [144, 144])              # 7 + 7 pages of 12
    assert e.value.status == 3
    with pytest.raises(dg.DGError) as e:
        ctx.prefill_ragged(t, [10, 10, 10])
    assert e.value.status == 3
    ctx.prefill_ragged(t, [100, 10])                   # 6 + 5 pages
    canvas = torch.zeros(2, 256, dtype=torch.int32, device="cuda")
    with pytest.raises(dg.DGError) as e:
        ctx.commit_block(canvas)                       # 100 + 512 > 400
    assert e.value.status == 3
    ctx.close()


def test_generate_blocks_over_prompts_of_different_lengths():
    lens = [60, 7]
    w = si.workload("tiny").with_(batch=2)
    ctx, _ = make_context(w, max_seq=14 * 64, temperature=0.05)   # whole pages for every sequence
    res = dg.generate_blocks(ctx, [p.cuda() for p in prompts(w, lens)],
                             lambda k: torch.as_tensor(canvas_of(w, k)).cuda(), 2, 3, 0.9, 5, commit_last=True)
    assert len(res["blocks"]) == 2 and ctx.cached_lens == [n + 512 for n in lens]
    assert all(b.shape == (2, 256) and bool(((b >= 0) & (b < w.shape.vocab)).all()) for b in res["blocks"])
    ctx.close()
