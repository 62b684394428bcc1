"""The timeline of a ragged batch's step: its kernels start while the ones
before them run, and their records must still follow one another (in a child
process, as the binding loads one library per process)."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, os, sys
sys.path.insert(0, os.environ["DG_ROOT"]); sys.path.insert(0, os.path.join(os.environ["DG_ROOT"], "tests"))
import torch
import block_discrete_diffusion_denoise_b200 as dgp
import synth_inputs as si
from gpu_helpers import make_context
w = si.workload("tiny").with_(batch=2)
s = torch.cuda.Stream()
with torch.cuda.stream(s):
    ctx, _ = make_context(w, max_seq=1280, stream=s.cuda_stream)
    tokens = torch.cat([si.uniform_tokens(w, "prefix", 1, n, device="cuda").reshape(-1) for n in (130, 40)])
    cur = si.uniform_tokens(w, "canvas", 2, 256, device="cuda")
    out = torch.empty_like(cur); conf = torch.empty(2, 256, device="cuda")
    res = {}

    def record(name, call):
        ctx.debug_timeline_reset()
        call()
        rec, n = ctx.debug_timeline()
        launches = dgp.timeline_launches(rec)
        overlap = max(a["t1_ns"] - b["t0_ns"] for a, b in zip(launches, launches[1:]))
        res[name] = {"names": [l["name"] for l in launches], "overlap_ns": overlap,
                     "spans_us": sum(k["total_us"] for k in dgp.timeline_summary(launches)["kernels"].values()),
                     "wall_us": dgp.timeline_summary(launches)["wall_us"]}
    record("prefill", lambda: ctx.prefill_ragged(tokens, [130, 40]))
    for st in range(3):                       # warm-up (the graph is captured)
        ctx.denoise_step(cur, st, 1, 0.9, out, conf)
    record("step", lambda: ctx.denoise_step(cur, 3, 1, 0.9, out, conf))
    print(json.dumps(res))
    ctx.close()
"""

TICK_NS = 1024       # the global timer's coarsest step


def test_launches_of_a_ragged_batch_do_not_overlap():
    lib = os.path.join(ROOT, "block_discrete_diffusion_denoise_b200", "libdg_timeline.so")
    assert os.path.exists(lib), "libdg_timeline.so is not built"
    env = dict(os.environ, DG_LIBRARY=lib, DG_ROOT=ROOT)
    res = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]
    d = json.loads(res.stdout.strip().splitlines()[-1])
    assert d["step"]["names"] == ["embed_norm"] + 2 * [
        "gemm_dense", "paged_append", "attention", "attn_merge", "gemm_dense", "residual_norm", "gemm_dense",
        "route_dispatch", "gemm_moe", "combine_norm"] + ["gemm_lmhead", "lmhead_merge_sample"]
    names = d["prefill"]["names"]
    # the stretch's plan, its forward up to the last layer's keys and values, and the canvases' plan
    assert names[:2] == ["paged_plan", "embed_norm"] and names[-2:] == ["paged_append", "paged_plan"]
    for x in d.values():
        assert x["overlap_ns"] <= TICK_NS, x
        assert x["spans_us"] <= x["wall_us"] + 1e-3 * TICK_NS * len(x["names"])
