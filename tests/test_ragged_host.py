"""Ragged batches without a device: what the binding refuses, and what it
passes to the library."""
import ctypes

import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg

from test_binding_checks import _host_context, _i32, _refused


def test_prompts_and_lengths_go_to_the_library_as_they_are():
    ctx = _host_context()
    seen = []

    class Lib:
        def dg_prefill_ragged(self, c, tokens, batch, lens):
            seen.append((tokens, batch, [lens[b] for b in range(batch)]))
            return 0
    ctx.lib = Lib()
    t = _i32(47)
    ctx.prefill_ragged(t, [40, 7])
    ctx.prefill_ragged(t, torch.tensor([3]))           # more tokens than lengths: the first ones
    assert seen == [(t.data_ptr(), 2, [40, 7]), (t.data_ptr(), 1, [3])] and ctx._batch == 1


def test_malformed_prompts_never_reach_the_library():
    ctx = _host_context()
    for tokens, lens in [(_i32(2, 40), [40, 40]), (_i32(40), []), (_i32(40), [40, 0]), (_i32(40), [41]),
                         (_i32(40), [20, 21]), (_i32(40), [-1, 5]), (torch.zeros(40), [40]),
                         (_i32(80)[::2], [40])]:
        _refused(ctx.prefill_ragged, tokens, lens)
    assert ctx.lib.calls == [] and ctx._batch is None
    assert ctx.cached_lens == []


def test_null_arguments_are_refused():
    lib = dg.load_library()
    assert lib.dg_prefill_ragged(None, None, 0, None) == 1
    assert lib.dg_cached_lens(None, ctypes.byref(ctypes.c_int32())) == 1


@pytest.mark.parametrize("prefix,call", [(_i32(2, 5), "dg_prefill"), ([_i32(5), _i32(1, 9)], "dg_prefill_ragged")])
def test_generate_blocks_takes_either_kind_of_prompts(prefix, call):
    ctx = _host_context()
    dg.generate_blocks(ctx, prefix, lambda k: _i32(2, 256), 0, 1, 0.9, 0)
    assert ctx.lib.calls == [call] and ctx._batch == 2
