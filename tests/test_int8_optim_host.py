"""Refusals and host logic of the 8-bit integer weight and of the many-tensor
optimizer calls: every bad argument is turned down on the host, before any
launch.  No call here reaches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import qlora_bit_frozen_b200 as q
from qlora_bit_frozen_b200 import _ffi, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _ffi.load()


@pytest.fixture
def d():
    buf = ctypes.create_string_buffer(8192)
    p = ctypes.c_void_p((ctypes.addressof(buf) + 255) // 256 * 256)
    p.keep = buf
    return p


def off(p, n):
    return ctypes.c_void_p(p.value + n)


@pytest.mark.parametrize("I,p", [(0, 0), (1, 16), (16, 16), (17, 32), (4096, 4096), (131071, 131072)])
def test_pitch(lib, I, p):
    assert lib.qlora_int8_pitch(I) == p == q.qlora_int8_pitch(I)
    assert lib.qlora_int8_pitch(-1) == 0


def test_quantizer_refusals(lib, d):
    f = lib.qlora_quantize_int8
    assert f(d, -1, 4, d, d, d, 256, None) == _ffi.ERR_SHAPE
    assert f(d, 4, -1, d, d, d, 256, None) == _ffi.ERR_SHAPE
    assert f(d, 1 << 31, 1 << 31, d, d, d, 256, None) == _ffi.ERR_SHAPE
    assert f(d, 1 << 31, 1, d, d, d, 256, None) == _ffi.ERR_SHAPE
    assert f(None, 4, 4, d, d, d, 256, None) == _ffi.ERR_INVALID_ARG
    assert f(d, 4, 4, None, d, d, 256, None) == _ffi.ERR_INVALID_ARG
    assert f(d, 4, 4, d, None, d, 256, None) == _ffi.ERR_INVALID_ARG
    assert f(d, 4, 4, d, d, None, 256, None) == _ffi.ERR_INVALID_ARG
    assert f(d, 4, 4, d, d, off(d, 8), 256, None) == _ffi.ERR_ALIGNMENT
    assert f(off(d, 2), 4, 4, d, d, d, 256, None) == _ffi.ERR_ALIGNMENT
    assert f(d, 4, 4, d, off(d, 1), d, 256, None) == _ffi.ERR_ALIGNMENT
    assert f(d, 4, 4, d, d, d, 255, None) == _ffi.ERR_WORKSPACE
    assert lib.qlora_quantize_int8_workspace_bytes(4, 4) >= 256
    assert lib.qlora_quantize_int8_workspace_bytes(1 << 31, 1 << 31) == 0


def weight(d, O=64, I=128, **kw):
    w = _ffi.qlora_weight(_ffi.FMT_INT8, O, I, I or 1, 0, 8, d.value, None, None, None, d.value, None)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def test_linear_refusals(lib, d):
    big = 1 << 40

    def fwd(w, X=d, R=4, A=d, B=d, r=8, comp=1, Y=d, U=None, ws=d, n=big):
        return lib.qlora_linear_fwd(ctypes.byref(w), X, R, A, B, r, 1.0, comp, Y, U, ws, n, None)

    def bwd(w, X=d, dY=d, R=4, A=d, B=d, r=8, comp=1, U=None, dX=d, dA=d, dB=d, ws=d, n=big):
        return lib.qlora_linear_bwd(ctypes.byref(w), X, dY, R, A, B, r, 1.0, U, comp, dX, dA, dB, ws, n, None)

    for f in (fwd, bwd):
        assert f(weight(d, bits=4)) == _ffi.ERR_SHAPE
        assert f(weight(d, block=0)) == _ffi.ERR_SHAPE
        assert f(weight(d, codes=None)) == _ffi.ERR_INVALID_ARG
        assert f(weight(d, scale=None)) == _ffi.ERR_INVALID_ARG
        assert f(weight(d, codes=d.value + 8)) == _ffi.ERR_ALIGNMENT
        assert f(weight(d, scale=d.value + 2)) == _ffi.ERR_ALIGNMENT
        assert f(weight(d, O=0)) == _ffi.ERR_SHAPE
        assert f(weight(d, I=0)) == _ffi.ERR_SHAPE
        assert f(weight(d, O=131073)) == _ffi.ERR_UNSUPPORTED
        assert f(weight(d, I=131073)) == _ffi.ERR_UNSUPPORTED
        assert f(weight(d), r=0) == _ffi.ERR_SHAPE
        assert f(weight(d), r=65) == _ffi.ERR_UNSUPPORTED
        assert f(weight(d), R=-1) == _ffi.ERR_SHAPE
        assert f(weight(d), R=1 << 31) == _ffi.ERR_SHAPE
        assert f(weight(d), comp=2) == _ffi.ERR_INVALID_ARG
        assert f(weight(d), A=None) == _ffi.ERR_INVALID_ARG
        assert f(weight(d), ws=None) == _ffi.ERR_INVALID_ARG
        assert f(weight(d), ws=off(d, 64)) == _ffi.ERR_ALIGNMENT
        assert f(weight(d), n=4096) == _ffi.ERR_WORKSPACE
    assert fwd(weight(d), X=off(d, 1)) == _ffi.ERR_ALIGNMENT
    assert fwd(weight(d), X=off(d, 2), comp=0) == _ffi.ERR_ALIGNMENT
    assert bwd(weight(d), dY=None) == _ffi.ERR_INVALID_ARG
    assert bwd(weight(d), X=None) == _ffi.ERR_INVALID_ARG


@pytest.mark.parametrize("R", [0, 1, 16, 300, 16384])
@pytest.mark.parametrize("O,I", [(1, 1), (70, 33), (12288, 4096)])
def test_workspace_sizes(lib, R, O, I):
    w = _ffi.qlora_weight(_ffi.FMT_INT8, O, I, I, 0, 8, None, None, None, None, None, None)
    for op, K in ((0, I), (1, O)):
        for comp in (0, 1):
            n = lib.qlora_linear_workspace_bytes(ctypes.byref(w), R, 8, op, comp)
            assert n % 256 == 0 and n >= 256 + R * K  # the quantized rows are in it
    w.I = 0
    assert lib.qlora_linear_workspace_bytes(ctypes.byref(w), R, 8, 0, 1) == 0


def test_token_limit(lib, d):
    """More tokens than the counts of CTAs hold are refused, and have no workspace."""
    w, n = weight(d, O=16, I=16), 1 << 62
    for R, ok in ((1 << 28, True), ((1 << 28) + 1, False)):
        for op in (0, 1):
            assert (lib.qlora_linear_workspace_bytes(ctypes.byref(w), R, 64, op, 1) > 0) == ok
        fwd = lib.qlora_linear_fwd(ctypes.byref(w), d, R, d, d, 64, 1.0, 1, d, None, d, 256 if ok else n, None)
        bwd = lib.qlora_linear_bwd(ctypes.byref(w), d, d, R, d, d, 64, 1.0, None, 1, d, d, d, d, 256 if ok else n, None)
        assert fwd == bwd == (_ffi.ERR_WORKSPACE if ok else _ffi.ERR_SHAPE)


def tensors(d, n=(16,), **kw):
    a = (_ffi.qlora_tensor * len(n))()
    for t, k in zip(a, n):
        t.param = t.grad = t.m = t.v = t.m_scale = t.v_scale = d.value
        t.n = k
        for key, v in kw.items():
            setattr(t, key, v)
    return a


def test_norm_refusals(lib, d):
    def f(t, count=1, most=1.0, c=d, ws=d, n=1 << 30):
        return lib.qlora_grad_norm(t, count, most, c, ws, n, None)

    assert f(tensors(d), -1) == _ffi.ERR_SHAPE
    assert f(None, 1) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d, n=(-1,))) == _ffi.ERR_SHAPE
    assert f(tensors(d, n=((1 << 38) + 1,))) == _ffi.ERR_SHAPE
    assert f(tensors(d, grad_type=2)) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d, grad=None)) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d, grad=d.value + 2)) == _ffi.ERR_ALIGNMENT
    assert f(tensors(d, grad=d.value + 1, grad_type=1)) == _ffi.ERR_ALIGNMENT
    for bad in (float("nan"), float("inf")):
        assert f(tensors(d), most=bad) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d), c=None) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d), ws=None) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d), c=off(d, 2)) == _ffi.ERR_ALIGNMENT
    assert f(tensors(d), ws=off(d, 16)) == _ffi.ERR_ALIGNMENT
    assert f(tensors(d), n=8) == _ffi.ERR_WORKSPACE
    size = lib.qlora_grad_norm_workspace_bytes
    assert size(tensors(d), 1) >= 256 and size(None, 0) >= 256 and size(tensors(d), -1) == 0
    assert size(tensors(d, n=(16,) * 2000), 2000) > size(tensors(d), 1)


def test_step_refusals(lib, d):
    def f(t, count=1, bits=32, step=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, c=None):
        return lib.qlora_adamw_step(t, count, bits, step, lr, b1, b2, eps, wd, c, None)

    for bits in (4, 16, 0):
        assert f(tensors(d), bits=bits) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d), step=0) == _ffi.ERR_SHAPE
    assert f(tensors(d), -1) == _ffi.ERR_SHAPE
    nan, inf = float("nan"), float("inf")
    for kw in ({"b1": 1.0}, {"b1": -0.1}, {"b2": 1.0}, {"b2": nan}, {"eps": 0.0}, {"eps": inf}, {"lr": inf},
               {"lr": nan}, {"wd": -0.1}, {"wd": inf}, {"wd": nan}):
        assert f(tensors(d), **kw) == _ffi.ERR_INVALID_ARG, kw
    for k in ("param", "grad", "m", "v"):
        assert f(tensors(d, **{k: None})) == _ffi.ERR_INVALID_ARG
        assert f(tensors(d, **{k: d.value + 2})) == _ffi.ERR_ALIGNMENT
    for k in ("m_scale", "v_scale"):
        assert f(tensors(d, **{k: None}), bits=8) == _ffi.ERR_INVALID_ARG
        assert f(tensors(d, **{k: d.value + 2}), bits=8) == _ffi.ERR_ALIGNMENT
    assert f(tensors(d, param_type=2)) == _ffi.ERR_INVALID_ARG
    assert f(tensors(d), c=off(d, 2)) == _ffi.ERR_ALIGNMENT


def test_binding_refusals():
    z = lambda n=256, dt=torch.float32: torch.zeros(n, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        q.OptimTensors([z()])
    with pytest.raises(ValueError, match="one for each"):
        q.OptimTensors([z()], [z(), z()], [z()], [z()])
    with pytest.raises(ValueError, match="states"):
        q.OptimTensors([z()], [z()])
    with pytest.raises(ValueError, match="both"):
        q.OptimTensors([z()], [z()], [z()], [z()], m_scale=[z(1)])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        q.OptimTensors([z(dt=torch.float16)])
    with pytest.raises(ValueError, match="8 or 32"):
        q.OptimTensors.with_states([z()], [z()], 16)
    with pytest.raises(ValueError, match="CUDA"):
        q.qlora_quantize_int8(z(64).reshape(8, 8))
    # an empty list holds nothing to step
    q.qlora_adamw_step(q.OptimTensors([], [], [], []), t=1)
    with pytest.raises(ValueError, match="gradients only"):
        q.qlora_adamw_step(q.OptimTensors([]), t=1)


def test_overlap_is_refused():
    a = torch.zeros(100)
    t = q.OptimTensors([])
    t.params, t.m, t.v = [a, a[50:]], [torch.zeros(100)], [torch.zeros(100)]
    with pytest.raises(ValueError, match="overlap"):
        t._refuse_overlap()
    t.params = [a[:50], a[50:]]
    t._refuse_overlap()
    t.m = [a[10:20]]
    with pytest.raises(ValueError, match="overlap"):
        t._refuse_overlap()


def test_checkpoint_round_trip_of_an_int8_weight(tmp_path):
    O, I = 6, 19
    codes = torch.randint(-127, 128, (O, q.qlora_int8_pitch(I)), dtype=torch.int8)
    codes[:, I:] = 0
    w = q.QuantizedWeight(q.FMT_INT8, O, I, I, 0, 8, codes, scale=torch.rand(O))
    np.savez(tmp_path / "w.npz", **w.state_dict())
    with np.load(tmp_path / "w.npz") as f:
        state = {k: f[k] for k in f.files}
    back = q.QuantizedWeight.from_state_dict(state, device="cpu")
    assert torch.equal(back.codes.reshape(-1), codes.reshape(-1)) and torch.equal(back.scale, w.scale)
    assert back.payload_bytes() == w.payload_bytes() == O * q.qlora_int8_pitch(I) + 4 * O
    for bad in ({"bits": 4}, {"codes": state["codes"].reshape(-1)[:-1]}, {"codes": state["codes"].view(np.uint8)},
                {"scale": None}):
        with pytest.raises(ValueError):
            q.QuantizedWeight.from_state_dict({**state, **bad}, device="cpu")
