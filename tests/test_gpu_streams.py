"""generate_blocks on a context whose stream is not torch's current one: the
blocks are those of the same calls made by hand on the context's own stream,
whatever the current stream is still busy with, and whatever it does with the
memory afterwards."""
import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg
import synth_inputs as si

from gpu_helpers import make_context

pytestmark = pytest.mark.gpu

LENS, BLOCKS, STEPS, TAU, SEED = [60, 7], 2, 3, 0.9, 5
BUSY = 100_000_000        # cycles: longer than the host needs for all the calls that follow


def workload():
    return si.workload("tiny").with_(batch=2)


def context(w, stream):
    with torch.cuda.stream(stream):
        ctx, _ = make_context(w, max_seq=20 * 64, temperature=0.05, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    return ctx


def prompts(w, ragged):
    t = si.uniform_tokens(w, "prefix", 2, max(LENS))
    return [t[b, :n].contiguous() for b, n in enumerate(LENS)] if ragged else t


def canvas(w, k):
    return torch.as_tensor(si.uniform_tokens(w, "canvas", 2, 256, block=k))


def step(ctx, cur, s):
    out, conf = torch.empty_like(cur), torch.empty(2, 256, device="cuda")
    settled = torch.empty(2, dtype=torch.int32, device="cuda")
    ctx.denoise_step(cur, s, SEED, TAU, out, conf, settled)
    ctx.sync()
    return out, bool((settled != 0).all())


def by_hand(w, ragged):
    """the final canvases, and a step behind the last commit"""
    st = torch.cuda.Stream()
    ctx = context(w, st)
    blocks = []
    with torch.cuda.stream(st):
        p = prompts(w, ragged)
        if ragged:
            ctx.prefill_ragged(torch.cat(p).cuda(), LENS)
        else:
            ctx.prefill(p.cuda())
        for k in range(BLOCKS):
            cur = canvas(w, k).cuda()
            for s in range(STEPS):
                cur, done = step(ctx, cur, s)
                if done:
                    break
            blocks.append(cur.cpu())
            ctx.commit_block(cur)
            ctx.sync()
        after = step(ctx, canvas(w, BLOCKS).cuda(), 0)[0].cpu()
    ctx.close()
    return blocks, after


@pytest.mark.parametrize("ragged", [True, False])
def test_blocks_do_not_depend_on_what_the_current_stream_is_busy_with(ragged):
    w = workload()
    want, want_after = by_hand(w, ragged)
    ctx = context(w, torch.cuda.Stream())
    p, canvases = prompts(w, ragged), [canvas(w, k).cuda() for k in range(BLOCKS)]
    p = [x.cuda() for x in p] if ragged else p.cuda()
    for x in (p if ragged else [p]):
        assert bool((x < w.shape.vocab).all())
    current = torch.cuda.Stream()
    current.wait_stream(torch.cuda.default_stream())
    with torch.cuda.stream(current):
        # the prefix and the canvases are written only after the wait; until then their memory holds other tokens
        late = [torch.zeros_like(x) for x in p] if ragged else torch.zeros_like(p)
        current.synchronize()
        torch.cuda._sleep(BUSY)
        for a, b in zip(late, p):
            a.copy_(b)

        def init(k):
            t = torch.zeros_like(canvases[k])
            torch.cuda._sleep(BUSY)
            return t.copy_(canvases[k])
        out = dg.generate_blocks(ctx, late, init, BLOCKS, STEPS, TAU, SEED, commit_last=True)
        # memory that the call gave back, overwritten while the last commit may still run
        for _ in range(8):
            torch.zeros_like(canvases[0])
        for a, b in zip(out["blocks"], want):
            assert torch.equal(a.cpu(), b)
        fresh = canvas(w, BLOCKS).cuda()
        current.synchronize()
        assert torch.equal(step(ctx, fresh, 0)[0].cpu(), want_after)
    ctx.close()
