"""Where a call that is given a stream allocates and copies, seen on the CPU:
tensors that say they are CUDA ones, a library that records what it is given,
and a note of the stream that is current at every allocation and copy."""
import contextlib

import pytest
import torch

import qlora_bit_frozen_b200 as q



class Side:
    cuda_stream = 77


SIDE = Side()


class Cuda(torch.Tensor):
    """A CPU tensor that says it is a CUDA one, and notes where it is copied."""
    is_cuda = True

    def contiguous(self):
        if not self.is_contiguous():
            Cuda.seen.append(("copy", Cuda.stream))
        return super().contiguous()

    def new_empty(self, *a, **kw):
        Cuda.seen.append(("new", Cuda.stream))
        return super().new_empty(*a, **kw)


def cuda(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Cuda)


class Library:
    """Every status is OK, every size 512 bytes; notes the calls' last argument, the stream."""
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 512
            self.streams.append(args[-1])
            return 0
        return call


@pytest.fixture
def here(monkeypatch):
    Cuda.seen, Cuda.stream = [], None
    lib = Library()
    empty = torch.empty

    def noted(*a, **kw):
        Cuda.seen.append(("empty", Cuda.stream))
        return empty(*a, **kw).as_subclass(Cuda)

    @contextlib.contextmanager
    def on_stream(s):
        before, Cuda.stream = Cuda.stream, s
        yield
        Cuda.stream = before

    monkeypatch.setattr(q._ffi, "load", lambda: lib)
    monkeypatch.setattr(torch, "empty", noted)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: {77: SIDE}[raw])
    monkeypatch.setattr(q, "_on", lambda dev: contextlib.nullcontext())
    return lib


@pytest.mark.parametrize("call", [
    lambda W: q.qlora_quantize_int8(W, stream=SIDE),
    lambda W: q.qlora_quantize_nf4(W, 16, 4, stream=SIDE),
    lambda W: q.qlora_quantize_nf4_noalloc(W, 16, 4, stream=SIDE),
    lambda W: q.qlora_quantize_nf4_fp32scale(W, 16, stream=SIDE),
    lambda W: q.qlora_quantize_affine(W, 4, 16, stream=SIDE)],
    ids=["int8", "nf4", "nf4_noalloc", "nf4_fp32scale", "affine"])
def test_quantizers_copy_and_allocate_on_their_stream(here, call):
    call(cuda(32, 48).t())
    assert ("copy", SIDE) in Cuda.seen and len(Cuda.seen) >= 3
    assert {s for _, s in Cuda.seen} == {SIDE} and here.streams == [77]


def weight(O=32, I=48):
    return q.QuantizedWeight(q.FMT_INT8, O, I, I, 0, 8, cuda(O, I, dtype=torch.int8), scale=cuda(O))


@pytest.mark.parametrize("call", [
    lambda w, X, A, B: q.qlora_linear_fwd(w, X, A, B, 1.0, stream=SIDE),
    lambda w, X, A, B: q.qlora_linear_bwd(w, X, cuda(4, 32), A, B, 1.0, stream=SIDE),
    lambda w, X, A, B: q.qlora_dequantize(w, stream=SIDE),
    lambda w, X, A, B: q.qlora_merge(w, A, B, 1.0, stream=SIDE)],
    ids=["forward", "backward", "dequantize", "merge"])
def test_outputs_are_allocated_on_the_stream_of_the_call(here, call):
    call(weight(), cuda(4, 48), cuda(8, 48), cuda(32, 8))
    assert Cuda.seen and {s for _, s in Cuda.seen} == {SIDE} and here.streams == [77]


@pytest.mark.parametrize("stream", [SIDE, 77])
def test_no_switch_of_streams_where_all_buffers_are_given(here, monkeypatch, stream):
    """Any stream that says its handle does, and the switch is left out."""
    monkeypatch.setattr(torch.cuda, "stream", None)
    w, X, A, B, ws = weight(), cuda(4, 48), cuda(8, 48), cuda(32, 8), cuda(512)
    q.qlora_linear_fwd(w, X, A, B, 1.0, Y=cuda(4, 32), U_out=cuda(4, 8), ws=ws, stream=stream)
    q.qlora_linear_fwd(w, X, A, B, 1.0, Y=cuda(4, 32), want_u=False, ws=ws, stream=stream)
    q.qlora_linear_bwd(w, X, cuda(4, 32), A, B, 1.0, dX=cuda(4, 48), dA=cuda(8, 48), dB=cuda(32, 8), ws=ws, stream=stream)
    q.qlora_linear_bwd(w, X, cuda(4, 32), A, B, 1.0, dX=cuda(4, 48), want_da=False, want_db=False, ws=ws, stream=stream)
    assert here.streams == [77] * 4


@pytest.mark.parametrize("call", [
    lambda w, W, A, B: q.qlora_quantize_int8(W),
    lambda w, W, A, B: q.qlora_quantize_nf4(W, 16, 4),
    lambda w, W, A, B: q.qlora_quantize_nf4_noalloc(W, 16, 4),
    lambda w, W, A, B: q.qlora_quantize_nf4_fp32scale(W, 16),
    lambda w, W, A, B: q.qlora_quantize_affine(W, 4, 16),
    lambda w, W, A, B: q.qlora_dequantize(w),
    lambda w, W, A, B: q.qlora_merge(w, A, B, 1.0),
    lambda w, W, A, B: q.qlora_adam_step(A, A, A, A, 1, 1e-3),
    lambda w, W, A, B: q.qlora_workspace_status(A),
    lambda w, W, A, B: q.qlora_linear_fwd(w, cuda(4, 48), A, B, 1.0),
    lambda w, W, A, B: q.qlora_linear_bwd(w, cuda(4, 48), cuda(4, 32), A, B, 1.0)],
    ids=["int8", "nf4", "nf4_noalloc", "nf4_fp32scale", "affine", "dequantize", "merge", "adam", "status", "forward",
         "backward"])
def test_calls_run_on_the_device_of_their_tensors(here, call, monkeypatch):
    """Also where another device is the current one: its current stream, and the launch there."""
    at = []

    @contextlib.contextmanager
    def on(dev):
        at.append(dev)
        yield
        at.pop()

    monkeypatch.setattr(q, "_on", on)
    monkeypatch.setattr(q, "_stream", lambda s, dev: at + [dev])
    call(weight(), cuda(32, 48), cuda(8, 48), cuda(32, 8))
    assert here.streams == [2 * [torch.device("cpu")]]


def listed(n, state_bits=32):
    params, grads = [cuda(300) for _ in range(n)], [cuda(300) for _ in range(n)]
    return params, grads, q.OptimTensors.with_states(params, grads, state_bits)


@pytest.fixture
def steps(here, monkeypatch):
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: zeros(*a, **kw).as_subclass(Cuda))
    control = zeros(4, dtype=torch.int32).as_subclass(Cuda)

    def norm(T):
        q.qlora_grad_norm(T, 1.0, control, stream=SIDE)

    def adamw(T):
        q.qlora_adamw_step(T, t=1, stream=SIDE)

    return norm, adamw


@pytest.mark.parametrize("state_bits", [8, 32])
def test_listed_tensors_that_move_are_refused(here, steps, state_bits):
    norm, adamw = steps
    for step, lists in ((norm, ("grads",)), (adamw, ("params", "grads"))):
        for name in lists:
            params, grads, T = listed(5, state_bits)
            for _ in range(7):
                step(T)
            every = getattr(T, name)
            for x in every:  # as module.to() and the like do
                x.data = x.data.clone()
            launched = len(here.streams)
            with pytest.raises(ValueError, match=name):
                step(T)
            assert len(here.streams) == launched
            params, grads, T = listed(5, state_bits)
            one = getattr(T, name)[3]
            one.data = one.data.clone()
            with pytest.raises(ValueError, match=name):
                for _ in range(5):
                    step(T)
            with pytest.raises(ValueError, match=name):  # and so is every call after that
                step(T)
    for k in range(4):  # both calls a step, as they are used
        params, grads, T = listed(4, state_bits)
        params[k].data = params[k].data.clone()
        with pytest.raises(ValueError, match="params"):
            for _ in range(4):
                norm(T)
                adamw(T)


def test_storage_of_listed_tensors_is_held(here, steps):
    """What the calls point at stays valid when a tensor is given other storage."""
    import gc
    import weakref

    import numpy as np

    array = np.zeros(300, np.float32)
    alive = weakref.ref(array)
    p = torch.Tensor._make_subclass(Cuda, torch.from_numpy(array))  # (no view, which would hold it too)
    T = q.OptimTensors.with_states([p], [cuda(300)])
    p.data = torch.zeros(300)
    del array
    gc.collect()
    assert alive() is not None
    del T
    gc.collect()
    assert alive() is None
