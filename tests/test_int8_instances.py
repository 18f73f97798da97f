"""The 8-bit linear layer where an instance of its kernels is met on purpose:
output edges inside a warp, every kernel that quantizes rows, long sums.
Definitions in 64 bits; what is exact there is compared bit for bit."""
import pytest
import torch

import qlora_bit_frozen_b200 as q
from test_int8_linear import BF, F32, make, rows64, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [17, 40, 64, 90, 129])
@pytest.mark.parametrize("O,I", [(33, 97), (127, 161), (225, 31), (1000, 1025)])
def test_outputs_that_end_inside_a_warp(R, O, I, dtype):
    """Widths off 32, over several runs of eight tokens: every value, and none beside them."""
    W, X, dY, A, B = make(R, O, I, 4, dtype)
    w, nw, s = weight(W)

    def fenced(m):
        buf = torch.full((R * m + 64,), 7.0, dtype=dtype, device="cuda")
        return buf[R * m:], buf[:R * m].view(R, m)

    after, Y = fenced(O)
    q.qlora_linear_fwd(w, X, A, torch.zeros_like(B), 8.0, Y=Y)
    n, sx = rows64(X.float())
    assert torch.equal(Y, (((n @ nw.T).float() * sx[:, None]) * s[None, :]).to(dtype)) and bool((after == 7).all())
    after, dX = fenced(I)
    q.qlora_linear_bwd(w, X, dY, torch.zeros_like(A), B, 8.0, dX=dX)
    n, sg = rows64(dY.float() * s[None, :])
    assert torch.equal(dX, ((n @ nw).float() * sg[:, None]).to(dtype)) and bool((after == 7).all())


def half_steps(seed, R, K, dtype):
    """Rows whose quotients by their scale lie on halves and beside them (fp32), some scaled."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = (torch.randint(-254, 255, (R, K), device="cuda", generator=g).float() / 2).to(dtype)
    X[:, K // 3] = 127
    X[::2] *= 0.3
    if dtype == F32:
        X *= 1 + torch.randint(-2, 3, X.shape, device="cuda", generator=g) * 2.0 ** -23
    return X


def unit(K):
    """A weight of unit rows: what is multiplied by it are the rows' own codes."""
    w = q.QuantizedWeight(q.FMT_INT8, K, K, K, 0, 8, torch.zeros(K, q.qlora_int8_pitch(K), dtype=torch.int8, device="cuda"),
                          scale=torch.ones(K, device="cuda"))
    w.codes[:, :K].fill_diagonal_(1)
    return w, torch.zeros(1, K, device="cuda"), torch.zeros(K, 1, device="cuda")


# 2500 rows of these widths are more than one launch with the dot products takes, and more than the CTAs of any grid
@pytest.mark.parametrize("dtype,K", [(BF, 1024), (BF, 2048), (BF, 2064), (BF, 4096), (BF, 4112), (BF, 12288), (BF, 20480),
                                     (BF, 1003), (F32, 1024), (F32, 1040), (F32, 2048), (F32, 2064), (F32, 10240),
                                     (F32, 16384), (F32, 16400), (F32, 1001)])
def test_rows_of_the_forward(dtype, K):
    """One, two and four vectors a thread, and one value at a time: every code and scale, near ties too."""
    w, A, B = unit(K)
    ties = half_steps(K, 1250, K, dtype)
    X = torch.cat([ties, torch.randn(1250, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(K)).to(dtype)])
    Y, _ = q.qlora_linear_fwd(w, X, A, B, 1.0)
    n, s = rows64(X.float())
    assert torch.equal(Y, (n.float() * s[:, None]).to(dtype))


@pytest.mark.parametrize("dtype,K", [(BF, 1024), (BF, 2048), (BF, 2064), (BF, 4096), (BF, 12288), (BF, 12304), (BF, 17408),
                                     (BF, 20480), (BF, 20496), (BF, 1003), (F32, 1024), (F32, 1040), (F32, 6144), (F32, 6160),
                                     (F32, 10240), (F32, 10256), (F32, 1001)])
def test_rows_of_the_input_gradient(dtype, K):
    """The same of rows times the channels' scales: powers of two, which keep the ties, and any others."""
    w, A, B = unit(K)
    g = torch.Generator(device="cuda").manual_seed(K)
    two = 2.0 ** torch.randint(-3, 4, (K,), device="cuda", generator=g).float()
    any_ = torch.rand(K, device="cuda", generator=g) + 0.5
    for scale, dY in ((two, half_steps(K, 2500, K, dtype) / two.to(dtype)),
                      (any_, torch.randn(2500, K, device="cuda", generator=g).to(dtype))):
        w.scale = scale
        dX, _, _ = q.qlora_linear_bwd(w, None, dY, A, B, 1.0, want_da=False, want_db=False)
        n, s = rows64(dY.float() * scale)
        assert torch.equal(dX, (n.float() * s[:, None]).to(dtype))


def sum_error(terms):
    """How far a long sum of random terms may be from its value, in the norm of many sums.  A sum is taken in
    runs of 256 terms, 16 at a time: the tensor core cuts at most 2^-23 of the running sum at each of a run's
    16 steps, and that sum has grown to sqrt(j / 16) of the run's by step j.  The runs are then added in
    fp32: half a step, 2^-24, of a sum that has grown to sqrt(i / runs), errors of either sign.  The factor's
    three parts, and fp32 values' too, leave less than 2^-24 of each term.  (One running sum over all terms
    would be cut at each of its steps: 15 times as much over 4096 terms.)"""
    cut = 2.0 ** -23 * sum((j / 16) ** 0.5 for j in range(1, 17))
    runs = -(-terms // 256)
    return cut + 2.0 ** -24 * ((runs + 1) / 2) ** 0.5 + 2.0 ** -24


def close_in_norm(got, ref, tol):
    assert float((got.double() - ref).norm() / ref.norm()) <= tol


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r", [16, 64])
def test_long_sums_over_columns(r, dtype):
    """U and V of 16384 columns (V read through dA, of tokens that hold a single one)."""
    R, K = 2048, 16384
    g = torch.Generator(device="cuda").manual_seed(r)
    X = torch.randn(R, K, device="cuda", generator=g).to(dtype)
    A, B = torch.randn(r, K, device="cuda", generator=g), torch.randn(K, r, device="cuda", generator=g)
    w = q.QuantizedWeight(q.FMT_INT8, 16, K, K, 0, 8, torch.zeros(16, K, dtype=torch.int8, device="cuda"),
                          scale=torch.ones(16, device="cuda"))
    _, U = q.qlora_linear_fwd(w, X, A, torch.zeros(16, r, device="cuda"), 1.0)
    close_in_norm(U, X.double() @ A.double().T, sum_error(K))
    w = q.QuantizedWeight(q.FMT_INT8, K, R, R, 0, 8, torch.zeros(K, R, dtype=torch.int8, device="cuda"),
                          scale=torch.ones(K, device="cuda"))
    one = torch.eye(R, device="cuda").to(dtype)
    _, dA, _ = q.qlora_linear_bwd(w, one, X, torch.zeros(r, R, device="cuda"), B, float(r), want_dx=False, want_db=False)
    close_in_norm(dA, (X.double() @ B.double()).T, sum_error(K) + 2.0 ** -23)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r", [16, 64])
def test_long_sums_over_tokens(r, dtype):
    """dA and dB of 16384 tokens (V of single terms)."""
    R, O, I = 16384, 2064, 2048
    g = torch.Generator(device="cuda").manual_seed(r)
    X, dY = (torch.randn(R, n, device="cuda", generator=g).to(dtype) for n in (I, O))
    A, B, U = torch.zeros(r, I, device="cuda"), torch.zeros(O, r, device="cuda"), torch.randn(R, r, device="cuda", generator=g)
    B[torch.arange(r), torch.arange(r)] = 1 + torch.rand(r, device="cuda", generator=g)  # V: column j of dY, times that
    w = q.QuantizedWeight(q.FMT_INT8, O, I, I, 0, 8, torch.zeros(O, I, dtype=torch.int8, device="cuda"),
                          scale=torch.ones(O, device="cuda"))
    _, dA, dB = q.qlora_linear_bwd(w, X, dY, A, B, float(r), U=U, want_dx=False)
    close_in_norm(dA, (dY.double() @ B.double()).T @ X.double(), sum_error(R) + 2.0 ** -23)
    close_in_norm(dB, dY.double().T @ U.double(), sum_error(R))


@pytest.mark.parametrize("R,O,I,r", [(1, 64, 48, 1), (12, 96, 112, 8), (50, 96, 112, 8), (700, 272, 256, 24),
                                     (8192, 1024, 1024, 64)])
def test_gradients_of_the_adapter_against_differences(R, O, I, r):
    """<Y, dY> is linear in A, in B and, with a zero weight, in X: a difference over a whole step is the
    derivative along it.  On small whole numbers every sum stays below 2^24, so nothing is rounded in fp32 and
    the two are equal."""
    g = torch.Generator(device="cuda").manual_seed(r)
    X, A, B, dY, EX, EA, EB = (torch.randint(-1, 2, s, device="cuda", generator=g).float()
                               for s in ((R, I), (r, I), (O, r), (R, O), (R, I), (r, I), (O, r)))
    w, _, _ = weight(torch.zeros(O, I, device="cuda"))
    f = lambda X, A, B: q.qlora_linear_fwd(w, X, A, B, float(r))[0].double()  # noqa: E731
    grads = q.qlora_linear_bwd(w, X, dY, A, B, float(r))
    for grad, E, plus, minus in zip(grads, (EX, EA, EB), (f(X + EX, A, B), f(X, A + EA, B), f(X, A, B + EB)),
                                    (f(X - EX, A, B), f(X, A - EA, B), f(X, A, B - EB))):
        assert float(grad.abs().max()) < 2 ** 24
        assert float(((plus - minus) / 2 * dY.double()).sum()) == float((grad.double() * E.double()).sum())
