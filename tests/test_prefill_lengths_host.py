"""Prompts too long for the 32 bits of a length are refused, not cut off (the
library itself compares lengths without wrapping around)."""
import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg

from test_binding_checks import _host_context, _i32, _refused


class Prompt(torch.Tensor):
    """a tensor that says it is longer than it is"""
    size_ = ()

    @property
    def shape(self):
        return torch.Size(self.size_)

    def numel(self):
        return 1 << 40


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5])
def test_lengths_beyond_32_bits_never_reach_the_library(n):
    ctx = _host_context()
    _refused(ctx.prefill_ragged, _i32(5).as_subclass(Prompt), [n])
    _refused(ctx.prefill_ragged, _i32(5).as_subclass(Prompt), [1, n, 1])
    t = _i32(1, 5).as_subclass(Prompt)
    t.size_ = (1, n)
    _refused(ctx.prefill, t)
    assert ctx.lib.calls == [] and ctx._batch is None


def test_the_longest_length_still_goes_through():
    ctx = _host_context()
    ctx.prefill_ragged(_i32(5).as_subclass(Prompt), [2 ** 31 - 1])
    assert ctx.lib.calls == ["dg_prefill_ragged"]
