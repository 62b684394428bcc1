"""The order of torch's streams and a context's, without a device: what
generate_blocks makes on torch's current stream is waited for before the
context's next call, and its memory is kept until the context is done with it."""
import ctypes

import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg

from test_binding_checks import _host_context, _i32


class Ordered(dg.Context):
    """A context on the host that writes down what it is told to wait for, between the library's calls."""

    def _behind_torch(self, *tensors):
        self.lib.calls.append(("wait", tensors))


def ordered():
    ctx = _host_context()
    ctx.__class__ = Ordered
    return ctx


@pytest.mark.parametrize("entropy", [None, {"gamma": 1.0, "stop_entropy": 0.1}])
@pytest.mark.parametrize("prefix", [_i32(2, 5), [_i32(5), _i32(1, 9)]])
def test_every_call_of_generate_blocks_follows_the_tensors_it_works_on(prefix, entropy):
    ctx = ordered()
    given = {}

    def watch(name, *at):
        inner = getattr(ctx, name)

        def call(*a, **kw):
            last = ctx.lib.calls[-1]
            assert last[0] == "wait", name
            tensors = [x for x in list(a) + list(kw.values()) if isinstance(x, torch.Tensor)]
            given.setdefault(name, []).append((tensors, last[1]))
            return inner(*a, **kw)
        setattr(ctx, name, call)
    for name in ("prefill", "prefill_ragged", "denoise_step", "denoise_step_entropy"):
        watch(name)
    dg.generate_blocks(ctx, prefix, lambda k: _i32(2, 256), 2, 2, 0.9, 0, entropy=entropy)
    for name, calls in given.items():
        for used, kept in calls:
            if name != "prefill":                 # the caller keeps its own prefix
                assert all(any(t is k for k in kept) for t in used), name
    assert set(given) == {"prefill_ragged" if isinstance(prefix, list) else "prefill",
                          "denoise_step" if entropy is None else "denoise_step_entropy"}


@pytest.mark.parametrize("entropy", [None, {"gamma": 1.0, "stop_entropy": 0.1}])
def test_a_step_is_finished_when_its_hook_runs(entropy):
    ctx = _host_context()
    seen = []
    dg.generate_blocks(ctx, _i32(2, 5), lambda k: _i32(2, 256), 1, 2, 0.9, 0, entropy=entropy,
                       after_step=lambda *a: seen.append(list(ctx.lib.calls)))
    name = "dg_denoise_step" if entropy is None else "dg_denoise_step_entropy"
    assert len(seen) >= 1 and all(calls[-2:] == [name, "dg_sync"] for calls in seen)


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.waited = handle, []

    def wait_stream(self, other):
        self.waited.append(other)


class Tensor:
    is_cuda = True

    def __init__(self):
        self.kept = []

    def record_stream(self, s):
        self.kept.append(s)


@pytest.mark.parametrize("handle", [0, 77])
def test_the_contexts_stream_waits_for_the_current_one_and_keeps_the_memory(handle, monkeypatch):
    ctx = _host_context()
    ctx._device_type, ctx._stream, ctx._weights = "cuda", handle, {"embed": torch.zeros(1)}
    mine, current = Stream(handle), Stream(42)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, dev: mine if h == handle else None)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev: mine if handle == 0 else None)
    t, host = Tensor(), torch.zeros(1)
    ctx._behind_torch(t, host)
    assert mine.waited == [current] and t.kept == [mine]
    # on its own stream there is nothing to order
    current.cuda_stream = handle
    ctx._behind_torch(t)
    assert mine.waited == [current] and t.kept == [mine]


class TorchStream:
    _as_parameter_ = ctypes.c_void_p(88)      # what torch.cuda.Stream offers to ctypes


@pytest.mark.parametrize("stream,handle", [(None, 0), (0, 0), (77, 77), (ctypes.c_void_p(78), 78),
                                           (ctypes.c_void_p(None), 0), (TorchStream(), 88)])
def test_a_context_knows_its_stream_in_every_form_that_it_takes(stream, handle, monkeypatch):
    given = []

    class Lib:
        def dg_create(self, cfg, weights, stream, out):
            given.append(stream)
            return 7
    monkeypatch.setattr(dg, "load_library", Lib)
    monkeypatch.setattr(dg, "check_weights", lambda *a: None)
    cfg = {n: 1 for n, _ in dg.dg_config._fields_}
    weights = dict(embed=_i32(1), final_norm=_i32(1), layers=[{f: _i32(1) for f in dg.LAYER_FIELDS}])
    ctx = dg.Context.__new__(dg.Context)
    with pytest.raises(dg.DGError):
        ctx.__init__(cfg, weights, stream=stream)
    assert ctx._stream == handle and given == [stream]
