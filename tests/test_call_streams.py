"""Calls on a stream of their own beside a busy current stream: they wait for
nothing of it, and it overwrites nothing of theirs."""
import pytest
import torch

import qlora_bit_frozen_b200 as q

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def normal(seed, *shape, dtype=F32):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)


def busy():
    """Keeps the current stream at work for some 50 ms."""
    torch.cuda._sleep(100_000_000)


def buffers(w):
    return [t for t in (w.codes, w.scale_codes, w.group_absmax, w.mean, w.scale, w.bias) if t is not None]


@pytest.mark.parametrize("call", [q.qlora_quantize_int8, q.qlora_quantize_nf4, q.qlora_quantize_nf4_noalloc,
                                  q.qlora_quantize_nf4_fp32scale, q.qlora_quantize_affine])
@pytest.mark.parametrize("raw", [False, True])
def test_a_transposed_weight_beside_a_busy_stream(call, raw):
    """The dense copy of a strided weight is made on the call's stream."""
    W = normal(1, 768, 512)
    want = call(W.t().contiguous())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    got = call(W.t(), stream=side.cuda_stream if raw else side)
    assert all(torch.equal(a, b) for a, b in zip(buffers(got), buffers(want)))


@pytest.mark.parametrize("fmt", ["int8", "nf4"])
@pytest.mark.parametrize("R", [3, 700])
def test_outputs_beside_a_busy_stream(fmt, R):
    """Outputs that a call allocates are not memory that the current stream has yet to write."""
    O, I, r = 640, 512, 8
    W, X, dY, A, B = (normal(1, O, I), normal(2, R, I, dtype=BF), normal(3, R, O, dtype=BF), normal(4, r, I),
                      normal(5, O, r))
    w = q.qlora_quantize_int8(W) if fmt == "int8" else q.qlora_quantize_nf4(W)
    calls = [lambda s: q.qlora_linear_fwd(w, X, A, B, 16.0, stream=s),
             lambda s: q.qlora_linear_bwd(w, X, dY, A, B, 16.0, stream=s),
             lambda s: (q.qlora_dequantize(w, stream=s),), lambda s: (q.qlora_merge(w, A, B, 16.0, stream=s),)]
    for call in calls:
        want = call(None)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        busy()
        for x in want:  # written after the work above, and given back at once
            torch.full_like(x, 7)
        got = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
