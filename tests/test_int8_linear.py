"""The linear layer on a symmetric 8-bit base, against its definition in 64
bits (plain torch operations).

Tolerances, derived from the operation counts (u = 2^-24, fp32's half step):
- With a zero adapter and fp32 activations nothing is inexact but the
  definition's own roundings (integer sum to fp32, times the row's scale,
  times the channel's): the output is compared bit for bit.
- U = X A^T: the factors enter as two bf16 halves (relative error 2^-16 at
  most) and K products are added in fp32: |dU| <= (2^-16 + K u) |X| |A|^T in
  every element; V, dA and dB alike over their own sums.
- The epilogue adds r terms in fp32: (r + 3) u |U| |B|^T.
- One rounding to the output's type: eps / 2 of the result.
"""
import pytest
import torch

import qlora_bit_frozen_b200 as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32

# rows, outputs, inputs: one to many, odd and even, below and above every tile
SHAPES = [(1, 1, 1), (1, 5, 3), (2, 64, 64), (3, 130, 70), (1, 4096, 512), (7, 257, 1000), (16, 1000, 257),
          (17, 384, 640), (33, 100, 4096), (64, 2048, 128), (100, 129, 31), (129, 256, 256), (300, 700, 144),
          (513, 513, 513), (777, 2048, 1024), (1500, 1300, 272), (2050, 1024, 656), (3000, 2304, 640),
          (4100, 4352, 384)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, *shape, std=1.0):
    return torch.randn(*shape, device="cuda", generator=gen(seed)) * std


def rows64(x):
    """Codes and scale of each row by the definition, in 64 bits but for its own fp32 roundings."""
    s = (x.abs().amax(1).double() / 127).float()
    n = torch.round((x.double() / s.double()[:, None]).float())
    return torch.where(s[:, None] > 0, n, 0.0).clamp(-127, 127).double(), s


def make(R, O, I, r, dtype, seed=1):
    W = normal(seed, O, I, std=0.02)
    X = (normal(seed + 1, R, I) * torch.exp(normal(seed + 2, R, 1))).to(dtype)
    dY = (normal(seed + 3, R, O, std=1e-3) * torch.exp(normal(seed + 4, R, 1))).to(dtype)
    return W, X, dY, normal(seed + 5, r, I, std=0.02), normal(seed + 6, O, r, std=0.02)


def weight(W):
    w = q.qlora_quantize_int8(W)
    return w, w.codes[:, :W.shape[1]].double(), w.scale


def close(got, ref, tol):
    """Elementwise |got - ref| <= tol."""
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - ref).abs() / tol.clamp(min=1e-300)).max()))


def products(X, A):
    """X A^T and how far the kernels may be from it."""
    X, A = X.double(), A.double()
    return X @ A.T, (2.0 ** -16 + X.shape[1] * U) * (X.abs() @ A.abs().T)


@pytest.mark.parametrize("O,I", [(1, 1), (1, 17), (5, 3), (64, 64), (33, 1000), (1024, 1024), (3, 20000), (700, 4100),
                                 (1300, 4112), (900, 13312), (700, 20000), (1500, 8192)])
def test_quantize_is_exact(O, I):
    W = normal(3, O, I, std=0.02)
    if O > 2:
        W[1] = 0
        W[2] *= 1e-42 / W[2].abs().max()  # subnormal numbers
    w, n, s = weight(W)
    rn, rs = rows64(W)
    assert torch.equal(w.scale, rs)
    assert torch.equal(n, rn)
    assert w.codes.shape == (O, q.qlora_int8_pitch(I)) and not bool(w.codes[:, I:].any())
    assert torch.equal(q.qlora_dequantize(w), (n.float() * s[:, None]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_refuses_nonfinite_weights(bad):
    W = normal(4, 8, 40)
    W[7, 39] = bad
    with pytest.raises(q.QLoraError) as e:
        q.qlora_quantize_int8(W)
    assert e.value.status == 4


@pytest.mark.parametrize("I", [16, 4096, 4112, 8192, 16384, 16400, 40000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_near_ties(I, dtype):
    """Quotients on and beside halves, where the rounding decides, for every way a row is read."""
    X = (torch.randint(-254, 255, (64, I), device="cuda", generator=gen(7)).float() / 2).to(dtype)
    X[:, 0] = 127
    X[::2] *= 0.3
    if dtype == F32:
        X *= 1 + torch.randint(-2, 3, X.shape, device="cuda", generator=gen(8)) * 2.0 ** -23
    w = q.QuantizedWeight(q.FMT_INT8, 16, I, I, 0, 8, torch.zeros(16, I, dtype=torch.int8, device="cuda"),
                          scale=torch.ones(16, device="cuda"))
    w.codes.fill_diagonal_(1)
    for k in (0, I - 16):  # 16 columns of codes at either end, read through a unit weight
        w.codes.zero_()
        w.codes[torch.arange(16), torch.arange(k, k + 16)] = 1
        Y, _ = q.qlora_linear_fwd(w, X, torch.zeros(1, I, device="cuda"), torch.zeros(16, 1, device="cuda"), 1.0)
        n, s = rows64(X.float())
        assert torch.equal(Y, (n[:, k:k + 16].float() * s[:, None]).to(dtype))


def test_quantize_of_nothing():
    assert q.qlora_quantize_int8(torch.empty(0, 5, device="cuda")).scale.numel() == 0
    assert torch.equal(q.qlora_quantize_int8(torch.empty(3, 0, device="cuda")).scale, torch.zeros(3, device="cuda"))


@pytest.mark.parametrize("R,O,I", SHAPES)
def test_zero_adapter_forward_and_gradient_are_exact(R, O, I):
    """fp32 activations, B = 0 (forward) and A = 0 (gradient): bit for bit."""
    W, X, dY, A, B = make(R, O, I, 4, F32)
    w, nw, s = weight(W)
    Y, _ = q.qlora_linear_fwd(w, X, A, torch.zeros_like(B), 8.0)
    n, sx = rows64(X)
    assert torch.equal(Y, ((n @ nw.T).float() * sx[:, None]) * s[None, :])
    dX, _, _ = q.qlora_linear_bwd(w, X, dY, torch.zeros_like(A), B, 8.0)
    n, sg = rows64(dY * s[None, :])
    assert torch.equal(dX, (n @ nw).float() * sg[:, None])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r", [1, 8, 13, 16, 32, 64])
@pytest.mark.parametrize("R,O,I", [(1, 300, 200), (19, 256, 512), (200, 520, 264), (1400, 1030, 300), (2300, 2048, 512),
                                   (1201, 640, 9216), (3001, 1024, 1003), (3001, 1003, 1024)])
def test_forward_and_backward(R, O, I, r, dtype):
    W, X, dY, A, B = make(R, O, I, r, dtype, seed=10 + r)
    w, nw, s = weight(W)
    c, half = 24.0 / r, HALF[dtype]
    B64, A64, X64, dY64 = B.double(), A.double(), X.double(), dY.double()

    Y, Ug = q.qlora_linear_fwd(w, X, A, B, 24.0)
    assert Y.dtype == dtype and Ug.dtype == F32
    u, du = products(X, A)
    close(Ug, u, du)
    n, sx = rows64(X.float())
    base = (n @ nw.T) * sx.double()[:, None] * s.double()[None, :]
    off = 4 * U * base.abs() + c * (du @ B64.abs().T + (r + 3) * U * (u.abs() @ B64.abs().T))
    ref = base + c * (u @ B64.T)
    close(Y, ref, half * (ref.abs() + off) + off)

    for Uin in (Ug, None):
        dX, dA, dB = q.qlora_linear_bwd(w, X, dY, A, B, 24.0, U=Uin)
        assert dX.dtype == dtype and dA.dtype == dB.dtype == F32
        v, dv = products(dY, B.T)
        n, sg = rows64(dY.float() * s[None, :])
        base = (n @ nw) * sg.double()[:, None]
        off = 4 * U * base.abs() + c * (dv @ A64.abs() + (r + 3) * U * (v.abs() @ A64.abs()))
        ref = base + c * (v @ A64)
        close(dX, ref, half * (ref.abs() + off) + off)
        rel = 2.0 ** -16 + (R + 3) * U
        close(dA, c * v.T @ X64, c * (rel * v.abs().T @ X64.abs() + dv.T @ X64.abs()) * 1.001)
        close(dB, c * dY64.T @ u, c * (rel * dY64.abs().T @ u.abs() + dY64.abs().T @ du) * 1.001)


@pytest.mark.parametrize("R", [1, 40, 2000])
@pytest.mark.parametrize("r", [8, 20])
def test_parts_of_the_gradient_alone(R, r):
    W, X, dY, A, B = make(R, 1096, 1080, r, BF)
    w, _, _ = weight(W)
    full = q.qlora_linear_bwd(w, X, dY, A, B, 16.0)
    for k in range(3):
        want = [j == k for j in range(3)]
        part = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, want_dx=want[0], want_da=want[1], want_db=want[2])
        assert [x is not None for x in part] == want
        assert torch.equal(part[k], full[k])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r", [1, 5, 16, 33, 64])
@pytest.mark.parametrize("R,O,I", [(65, 1500, 136), (100, 4100, 520), (129, 272, 2064), (257, 264, 130), (2600, 777, 1100)])
def test_ranks_over_token_counts(R, O, I, r, dtype):
    test_forward_and_backward(R, O, I, r, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r", [1, 8, 16, 40, 64])
@pytest.mark.parametrize("R,O,I", [(2, 512, 384), (14, 512, 384), (90, 1024, 640), (640, 1024, 512), (2500, 1536, 1024)])
def test_adapter_keeps_all_bits(R, O, I, r, dtype):
    """Sums of one term each, a factor's value times a power of two: the 24 bits of the factor come
    through, but for the tensor core's last bit (one truncated addition: 2^-23)."""
    W, _, _, A, B = make(R, O, I, r, dtype)
    w, _, _ = weight(torch.zeros_like(W))
    rows = torch.arange(R, device="cuda")
    at = rows * 37 % I
    X = torch.zeros(R, I, dtype=dtype, device="cuda")
    X[rows, at] = 2.0 ** (rows % 9 - 4).float().to(dtype)
    _, Ug = q.qlora_linear_fwd(w, X, A, torch.zeros_like(B), float(r))
    u = 2.0 ** (rows % 9 - 4).double()[:, None] * A.double()[:, at].T
    close(Ug, u, 2 * U * u.abs())
    # U has one power of two a token, so that Y = U B^T holds the values of B
    j = rows % r
    one = torch.zeros(r, I, device="cuda")
    k = torch.arange(r, device="cuda") * (I // r)
    one[torch.arange(r), k] = 0.25
    X.zero_()
    X[rows, k[j]] = 2.0
    Y, _ = q.qlora_linear_fwd(w, X, one, B, float(r))
    y = 0.5 * B.double()[:, j].T
    close(Y, y, (HALF[dtype] + 2 * U) * 1.01 * y.abs())
    # and the same of V, dX = V A, dA = V^T X and dB = dY^T U with one token that counts
    dY = torch.zeros(R, O, dtype=dtype, device="cuda")
    o = rows * 29 % O
    dY[rows, o] = 0.5
    dX, _, _ = q.qlora_linear_bwd(w, X, dY, A, torch.zeros_like(B).index_fill_(1, torch.tensor([r - 1], device="cuda"), 4.0),
                                  float(r))
    close(dX, 2 * A.double()[r - 1].expand(R, I), (HALF[dtype] + 2 * U) * 1.01 * 2 * A.double()[r - 1].abs())
    t = R // 2
    X.zero_()
    X[t] = 2.0 ** (torch.arange(I, device="cuda") % 7 - 3).float().to(dtype)
    dY.zero_()
    dY[t] = 2.0 ** (torch.arange(O, device="cuda") % 5 - 2).float().to(dtype)
    Uin = normal(5, R, r)
    one = torch.zeros_like(B)
    one[3] = B[3]
    _, dA, dB = q.qlora_linear_bwd(w, X, dY, A, one, float(r), U=Uin)
    v = dY.double()[t, 3] * B.double()[3]
    ref = v[:, None] * X.double()[t][None, :]
    close(dA, ref, 4 * U * ref.abs())
    ref = dY.double()[t][:, None] * Uin.double()[t][None, :]
    close(dB, ref, 2 * U * ref.abs())


@pytest.mark.parametrize("R,r", [(90, 64), (700, 8), (3000, 16)])
def test_nonfinite_values_keep_to_their_rows_and_columns(R, r):
    """A bad token changes its own row only, a bad row of a factor its own output only."""
    O, I = 1100, 1030
    W, X, dY, A, B = make(R, O, I, r, BF)
    w, _, _ = weight(W)
    bad = torch.tensor([0, R // 2, R - 1], device="cuda")
    X[bad] = 0
    Y, Ug = q.qlora_linear_fwd(w, X, A, B, 16.0)
    X2, B2 = X.clone(), B.clone()
    X2[bad, 7] = torch.tensor([float("nan"), float("inf"), float("-inf")], dtype=BF, device="cuda")
    B2[5, 0] = float("inf")
    B2[O - 1, r - 1] = float("nan")
    Y2, U2 = q.qlora_linear_fwd(w, X2, A, B2, 16.0)
    rows = torch.ones(R, dtype=torch.bool, device="cuda")
    rows[bad] = False
    cols = torch.ones(O, dtype=torch.bool, device="cuda")
    cols[[5, O - 1]] = False
    assert torch.equal(Y2[rows][:, cols], Y[rows][:, cols]) and torch.equal(U2[rows], Ug[rows])
    assert bool(torch.isnan(Y2[bad]).all()) and not bool(torch.isfinite(Y2[:, ~cols]).any())


@pytest.mark.parametrize("R", [3, 300, 2000])
def test_a_call_on_a_stream_of_its_own_keeps_its_workspace(R):
    """The workspace that a call allocates is not handed out while its stream still uses it."""
    W, X, dY, A, B = make(R, 1024, 1024, 16, BF)
    w, _, _ = weight(W)
    Y, Ug = q.qlora_linear_fwd(w, X, A, B, 16.0)
    g = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, U=Ug)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        outs = [(torch.empty_like(Y), torch.empty_like(Ug), [torch.empty_like(x) for x in g]) for _ in range(4)]
        torch.cuda.synchronize()
        for y, u, (dx, da, db) in outs:
            q.qlora_linear_fwd(w, X, A, B, 16.0, Y=y, U_out=u, stream=stream)
            q.qlora_linear_bwd(w, X, dY, A, B, 16.0, U=u, dX=dx, dA=da, dB=db, stream=stream)
            n = max(q.qlora_linear_workspace_bytes(w, R, 16, op, q.COMPUTE_BF16) for op in (0, 1))
            for _ in range(3):  # takes what the current stream's pool has to give
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for y, u, grads in outs:
            assert torch.equal(y, Y) and torch.equal(u, Ug) and all(torch.equal(a, b) for a, b in zip(grads, g))


def test_no_rows():
    W, X, dY, A, B = make(1, 48, 32, 8, BF)
    w, _, _ = weight(W)
    Y, Ug = q.qlora_linear_fwd(w, X[:0], A, B, 16.0)
    assert Y.shape == (0, 48) and Ug.shape == (0, 8)
    dX, dA, dB = q.qlora_linear_bwd(w, X[:0], dY[:0], A, B, 16.0)
    assert dX.shape == (0, 32) and not bool(dA.any()) and not bool(dB.any())


@pytest.mark.parametrize("R", [5, 600])
def test_special_tokens_and_channels(R):
    """Zero tokens, subnormal and huge ones, NaN and Inf: each keeps to its own row."""
    O, I, r = 384, 272, 8
    W, X, dY, A, B = make(R, O, I, r, F32)
    W[0] = 0
    w, nw, s = weight(W)
    B0 = torch.zeros_like(B)
    X[0] = 0
    X[1] *= 1e-43 / X[1].abs().max()
    X[2] *= 1e35 / X[2].abs().max()
    Y, _ = q.qlora_linear_fwd(w, X, A, B0, 16.0)
    n, sx = rows64(X)
    ref = ((n @ nw.T).float() * sx[:, None]) * s[None, :]
    assert torch.equal(Y, ref)
    assert not bool(Y[0].any()) and not bool(Y[:, 0].any())
    X[3, 5] = float("nan")
    X[4, I - 1] = float("inf")
    Y2, _ = q.qlora_linear_fwd(w, X, A, B0, 16.0)
    assert bool(torch.isnan(Y2[3:5]).all())
    keep = [i for i in range(R) if i not in (3, 4)]
    assert torch.equal(Y2[keep], ref[keep])
    dY[0] = 0
    dY[3, O - 1] = float("-inf")
    dX, _, _ = q.qlora_linear_bwd(w, X, dY, torch.zeros_like(A), B, 16.0, want_da=False, want_db=False)
    assert not bool(dX[0].any()) and bool(torch.isnan(dX[3]).all()) and bool(torch.isfinite(dX[4:]).all())


@pytest.mark.parametrize("R,O,I", [(1, 256, 256), (9, 384, 512), (300, 512, 256), (1500, 1024, 512)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned_arrays_and_untouched_surroundings(R, O, I, dtype):
    """Activations and outputs one element off any wide alignment; nothing beside the outputs is written."""
    W, X, dY, A, B = make(R, O, I, 8, dtype)
    w, _, _ = weight(W)

    def shifted(x):
        buf = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        buf[1:] = x.reshape(-1)
        return buf[1:].view(x.shape)

    def fenced(n, m):
        buf = torch.full((n * m + 129,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[1:1 + n * m].view(n, m)

    Y, Ug = q.qlora_linear_fwd(w, X, A, B, 16.0)
    dX, _, _ = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, U=Ug)
    buf, Y2 = fenced(R, O)
    q.qlora_linear_fwd(w, shifted(X), A, B, 16.0, Y=Y2)
    assert float(buf[0]) == 7 and bool((buf[1 + R * O:] == 7).all())
    # U may be summed in another order there
    tol = HALF[dtype] * 2 * Y.double().abs() + 1e-4 * Y.double().abs().max()
    close(Y2, Y.double(), tol)
    buf, dX2 = fenced(R, I)
    q.qlora_linear_bwd(w, shifted(X), shifted(dY), A, B, 16.0, U=Ug, dX=dX2)
    assert float(buf[0]) == 7 and bool((buf[1 + R * I:] == 7).all())
    close(dX2, dX.double(), HALF[dtype] * 2 * dX.double().abs() + 1e-4 * dX.double().abs().max())


def test_workspace_of_the_stated_size_is_enough_and_fenced():
    for R, O, I in ((1, 300, 272), (20, 512, 512), (700, 640, 300), (1500, 1024, 512)):
        W, X, dY, A, B = make(R, O, I, 16, BF)
        w, _, _ = weight(W)
        for op in (0, 1):
            n = q.qlora_linear_workspace_bytes(w, R, 16, op, q.COMPUTE_BF16)
            buf = torch.full((n + 512,), 113, dtype=torch.uint8, device="cuda")
            ws = buf[:n]
            if op == 0:
                a = q.qlora_linear_fwd(w, X, A, B, 16.0, ws=ws)
                b = q.qlora_linear_fwd(w, X, A, B, 16.0)
            else:
                a = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, ws=ws)
                b = q.qlora_linear_bwd(w, X, dY, A, B, 16.0)
            assert all(torch.equal(x, y) for x, y in zip(a, b))
            assert bool((buf[n:] == 113).all())
            assert q.qlora_workspace_status(ws) == 0
            with pytest.raises(q.QLoraError):
                q.qlora_linear_fwd(w, X, A, B, 16.0, ws=buf[:256])


@pytest.mark.parametrize("R", [1, 12, 300, 2100])
def test_same_bits_on_every_call_and_stream_and_in_a_graph(R):
    O, I = 1024, 768
    W, X, dY, A, B = make(R, O, I, 16, BF)
    w, _, _ = weight(W)
    Y, Ug = q.qlora_linear_fwd(w, X, A, B, 16.0)
    g = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, U=Ug)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y2, U2 = q.qlora_linear_fwd(w, X, A, B, 16.0)
        g2 = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, U=U2)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, Y2) and all(torch.equal(a, b) for a, b in zip(g, g2))
    ws = [q.workspace(q.qlora_linear_workspace_bytes(w, R, 16, op, q.COMPUTE_BF16)) for op in (0, 1)]
    Y3, U3 = torch.zeros_like(Y), torch.zeros_like(Ug)
    g3 = [torch.zeros_like(x) for x in g]
    Xs = torch.zeros_like(X)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlora_linear_fwd(w, Xs, A, B, 16.0, Y=Y3, U_out=U3, ws=ws[0])
        q.qlora_linear_bwd(w, Xs, dY, A, B, 16.0, U=U3, dX=g3[0], dA=g3[1], dB=g3[2], ws=ws[1])
    for x in (torch.zeros_like(X), X):
        Xs.copy_(x)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, Y3) and all(torch.equal(a, b) for a, b in zip(g, g3))


def test_two_streams_at_once():
    a = make(1024, 1024, 1024, 16, BF)
    b = make(3, 2048, 512, 8, BF, seed=40)
    wa, wb = weight(a[0])[0], weight(b[0])[0]
    ra = q.qlora_linear_fwd(wa, a[1], a[3], a[4], 16.0)[0]
    rb = q.qlora_linear_fwd(wb, b[1], b[3], b[4], 16.0)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    out = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            ya = q.qlora_linear_fwd(wa, a[1], a[3], a[4], 16.0)[0]
        with torch.cuda.stream(s2):
            yb = q.qlora_linear_fwd(wb, b[1], b[3], b[4], 16.0)[0]
        out.append((ya, yb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) and torch.equal(y, rb) for x, y in out)


def test_gradients_against_differences():
    """<Y, dY> is linear in A and in B, and in X where the weight is zero: a
    difference over a whole step gives the derivative along it but for
    rounding (Y's error above, summed against dY)."""
    R, O, I, r = 50, 96, 112, 8
    W, X, dY, A, B = make(R, O, I, r, F32)
    w, _, _ = weight(W)
    f = lambda w, X, A, B: q.qlora_linear_fwd(w, X, A, B, 16.0)[0].double()  # noqa: E731
    dX, dA, dB = q.qlora_linear_bwd(w, X, dY, A, B, 16.0)
    EA, EB, EX = normal(90, r, I, std=0.02), normal(91, O, r, std=0.02), normal(92, R, I)
    y = f(w, X, A, B)
    size = (y.abs() + f(w, X, A + EA, B).abs() + f(w, X, A, B + EB).abs()) * dY.double().abs()
    # every Y is within (2^-15 + (I + r + 8) u) of terms no larger than 64 |Y|max
    tol = float((2.0 ** -15 + (I + r + 8) * U) * 64 * size.max() * R * O) ** 1.0
    for g, E, plus, minus in ((dA, EA, f(w, X, A + EA, B), f(w, X, A - EA, B)),
                              (dB, EB, f(w, X, A, B + EB), f(w, X, A, B - EB))):
        diff = float(((plus - minus) / 2 * dY.double()).sum())
        want = float((g.double() * E.double()).sum())
        assert abs(diff - want) <= tol
        assert abs(diff - want) <= 0.01 * float((g.double() * E.double()).abs().sum())
    w0, _, _ = weight(torch.zeros_like(W))
    dX0, _, _ = q.qlora_linear_bwd(w0, X, dY, A, B, 16.0)
    diff = float(((f(w0, X + EX, A, B) - f(w0, X - EX, A, B)) / 2 * dY.double()).sum())
    terms = dX0.double() * EX.double()
    assert abs(diff - float(terms.sum())) <= 0.01 * float(terms.abs().sum())


@pytest.mark.parametrize("r", [1, 8, 40])
def test_merge(r):
    O, I = 70, 83
    W, _, _, A, B = make(1, O, I, r, F32)
    w, n, s = weight(W)
    got = q.qlora_merge(w, A, B, 12.0)
    base = (n.float() * s[:, None]).double()
    delta = (12.0 / r) * (B.double() @ A.double())
    close(got, base + delta, 2 * U * (base.abs() + delta.abs()) + (r + 3) * U * (12.0 / r) * (B.double().abs() @ A.double().abs()))
    assert torch.equal(q.qlora_merge(w, A, B, 0.0), q.qlora_dequantize(w))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_another_device_than_the_current_one():
    with torch.cuda.device(1):
        W = torch.randn(256, 128, device="cuda:1")
        X = torch.randn(20, 128, device="cuda:1", dtype=BF)
        A, B = torch.randn(8, 128, device="cuda:1"), torch.randn(256, 8, device="cuda:1")
        ref = q.qlora_linear_fwd(q.qlora_quantize_int8(W), X, A, B, 8.0)[0]
    got = q.qlora_linear_fwd(q.qlora_quantize_int8(W), X, A, B, 8.0)[0]
    assert torch.equal(got, ref)


@pytest.mark.parametrize("R,O,I", [(2, 131072, 16400), (130, 131072, 16400), (1_100_000, 2048, 1000), (1_100_000, 1000, 2048)])
def test_offsets_past_32_bits(R, O, I):
    """More than 2^31 weight codes, activations or outputs: the first and last rows and columns."""
    r, c = 8, 2.0
    W, A, B = (normal(k, *s, std=0.02) for k, s in enumerate(((O, I), (r, I), (O, r))))
    w = q.qlora_quantize_int8(W)
    X, dY = (normal(k, R, n).to(BF) for k, n in ((5, I), (6, O)))
    Y, Ug = q.qlora_linear_fwd(w, X, A, B, c * r)
    dX, dA, dB = q.qlora_linear_bwd(w, X, dY, A, B, c * r, U=Ug)
    rows = sorted({0, 1, R // 2, R - 2, R - 1})
    outs = torch.tensor([0, 1, O // 2, O - 2, O - 1], device="cuda")
    nw, s = rows64(W[outs])
    n, sx = rows64(X[rows].float())
    u, du = products(X[rows], A)
    base = (n @ nw.T) * sx.double()[:, None] * s.double()[None, :]
    b = B[outs].double()
    off = 4 * U * base.abs() + c * (du @ b.abs().T + (r + 3) * U * (u.abs() @ b.abs().T))
    ref = base + c * (u @ b.T)
    close(Y[rows][:, outs], ref, HALF[BF] * (ref.abs() + off) + off)
    cols = torch.tensor([0, 1, I // 2, I - 2, I - 1], device="cuda")
    n, sg = rows64(dY[rows].float() * w.scale[None, :])
    v, dv = products(dY[rows], B.T)
    a = A[:, cols].double()
    base = (n @ w.codes[:, cols].double()) * sg.double()[:, None]
    off = 4 * U * base.abs() + c * (dv @ a.abs() + (r + 3) * U * (v.abs() @ a.abs()))
    ref = base + c * (v @ a)
    close(dX[rows][:, cols], ref, HALF[BF] * (ref.abs() + off) + off)
    # the gradients' last columns, over all tokens
    v, dv = products(dY, B.T)
    x = X[:, cols].double()
    rel = 2.0 ** -16 + (R + 3) * U
    close(dA[:, cols], c * v.T @ x, c * (rel * v.abs().T @ x.abs() + dv.T @ x.abs()) * 1.001)
    u, du = products(X, A)
    g = dY[:, outs].double()
    close(dB[outs], c * g.T @ u, c * (rel * g.abs().T @ u.abs() + g.abs().T @ du) * 1.001)


@pytest.mark.parametrize("O,I", [(3, 7), (5, 8), (700, 4100), (4096, 1028), (131072, 32771), (131072, 32772)])
@pytest.mark.parametrize("shift", [0, 1])
def test_dequantize_is_exact(O, I, shift):
    """One product a weight, also past 2^32 weights and into an unaligned output (the rows at either end)."""
    codes = torch.randint(-127, 128, (O, q.qlora_int8_pitch(I)), dtype=torch.int8, device="cuda", generator=gen(1))
    scale = torch.rand(O, device="cuda", generator=gen(2))
    w = q.QuantizedWeight(q.FMT_INT8, O, I, I, 0, 8, codes, scale=scale)
    buf = torch.full((O * I + 9,), 7.0, device="cuda")
    q.qlora_dequantize(w, out=buf[shift:shift + O * I].view(O, I))
    got = buf[shift:shift + O * I].view(O, I)
    rows = torch.unique(torch.cat([torch.arange(min(O, 700)), torch.arange(max(0, O - 700), O)])).cuda()
    assert torch.equal(got[rows], codes[rows, :I].float() * scale[rows, None])
    assert bool((buf[:shift] == 7).all()) and bool((buf[shift + O * I:] == 7).all())


# fp32 activations, and bf16 rows that do not start on 16 bytes, in numbers that go to the tensor cores in parts
COPIES = [(2200, 4096, 4100, 64, F32), (2200, 264, 4100, 64, F32), (2200, 4100, 264, 64, F32), (9000, 4100, 1030, 16, F32),
          (1200, 2047, 2050, 64, BF), (1200, 2048, 2047, 64, BF), (1200, 2047, 2048, 64, BF), (9001, 1001, 1003, 16, BF)]


@pytest.mark.parametrize("R,O,I,r,dtype", COPIES)
def test_activations_in_parts(R, O, I, r, dtype):
    test_forward_and_backward(R, O, I, r, dtype)


@pytest.mark.parametrize("R,O,I,r,dtype", COPIES)
def test_activations_in_parts_keep_to_the_workspace_and_to_each_other(R, O, I, r, dtype):
    """The stated workspace is enough, on any content; each gradient has the same bits alone."""
    W, X, dY, A, B = make(R, O, I, r, dtype)
    w, _, _ = weight(W)
    Y, Ug = q.qlora_linear_fwd(w, X, A, B, 16.0)
    full = q.qlora_linear_bwd(w, X, dY, A, B, 16.0)
    compute = q.COMPUTE_BF16 if dtype == BF else q.COMPUTE_FP32
    for fill in (0, 255):
        for op in (0, 1):
            n = q.qlora_linear_workspace_bytes(w, R, r, op, compute)
            buf = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")
            if op == 0:
                got = q.qlora_linear_fwd(w, X, A, B, 16.0, ws=buf[:n])
                assert torch.equal(got[0], Y) and torch.equal(got[1], Ug)
            else:
                got = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, ws=buf[:n])
                assert all(torch.equal(a, b) for a, b in zip(got, full))
            assert bool((buf[n:] == fill).all())
    for k in range(3):
        part = q.qlora_linear_bwd(w, X, dY, A, B, 16.0, want_dx=k == 0, want_da=k == 1, want_db=k == 2)
        assert torch.equal(part[k], full[k])


@pytest.mark.parametrize("R,O,I,r,dtype", COPIES)
def test_activations_in_parts_keep_all_bits(R, O, I, r, dtype):
    """Sums of one term each: the activation's bits times a power of two come through (as in
    test_adapter_keeps_all_bits)."""
    W, X, dY, A, B = make(R, O, I, r, dtype)
    w, _, _ = weight(torch.zeros_like(W))
    rows = torch.arange(R, device="cuda")
    at = rows * 37 % I
    one = torch.zeros_like(X)
    one[rows, at] = X[rows, at]
    A = 2.0 ** (torch.arange(r * I, device="cuda") % 11 - 5).float().view(r, I)
    _, Ug = q.qlora_linear_fwd(w, one, A, torch.zeros_like(B), float(r))
    u = X[rows, at].double()[:, None] * A.double()[:, at].T
    close(Ug, u, 2 * U * u.abs())
    t = R - 1
    one = torch.zeros_like(dY)
    one[t] = dY[t]
    Uin = 2.0 ** (torch.arange(R * r, device="cuda") % 7 - 3).float().view(R, r)
    _, _, dB = q.qlora_linear_bwd(w, X, one, A, B, float(r), U=Uin)
    ref = dY[t].double()[:, None] * Uin[t].double()[None, :]
    close(dB, ref, 2 * U * ref.abs())


def test_two_graphs_share_a_workspace():
    """Each captured call leaves nothing in the workspace that the other's replay could meet."""
    cases, ws = [], q.workspace(1 << 27)
    for R, O, I, r, dtype in ((300, 1024, 768, 16, BF), (2100, 640, 520, 40, BF), (5, 1024, 1030, 8, F32)):
        W, X, dY, A, B = make(R, O, I, r, dtype)
        w, _, _ = weight(W)
        want = q.qlora_linear_fwd(w, X, A, B, 16.0) + q.qlora_linear_bwd(w, X, dY, A, B, 16.0)
        got = [torch.zeros_like(x) for x in want]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q.qlora_linear_fwd(w, X, A, B, 16.0, Y=got[0], U_out=got[1], ws=ws)
            q.qlora_linear_bwd(w, X, dY, A, B, 16.0, dX=got[2], dA=got[3], dB=got[4], ws=ws)
        cases.append((graph, got, want, (w, X, dY, A, B)))
    for k in (0, 1, 2, 1, 0, 2, 2, 0):
        graph, got, want, _ = cases[k]
        for x in got:
            x.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
