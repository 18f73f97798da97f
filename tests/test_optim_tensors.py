"""The gradient norm and the AdamW step over many tensors.

The step is compared bit for bit with the definition's fp32 operations, one
rounding each (numpy), and with the formula in 64 bits: the roundings are 2
on m, 4 on v, 6 on the step and 2 on the parameter, each at most u = 2^-24 of
a term."""
import math

import numpy as np
import pytest
import torch

import qlora_bit_frozen_b200 as q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
f32 = np.float32
BF, F32 = torch.bfloat16, torch.float32
HP = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
SIZES = [1, 255, 256, 257, 5, 0, 4096, 10007, 64 * 80]


def to_np(t):
    t = t.reshape(-1)
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def blocks(x):
    n = -(-x.size // 256) * 256
    out = np.zeros(n, x.dtype)
    out[:x.size] = x
    return out.reshape(-1, 256)


def decode(m, ms, v, vs, n):
    """m and v of 8-bit states, in the definition's fp32 steps."""
    k = blocks(m).astype(f32) * f32(1 / 127)
    mm = (k * np.abs(k)) * ms[:, None]
    k = blocks(v).astype(f32) * f32(1 / 255)
    r = (k * k) * vs[:, None]
    return mm.reshape(-1)[:n], (r * r).reshape(-1)[:n]


def encode(m, r):
    bm, br = blocks(m), blocks(r)
    ms, vs = np.abs(bm).max(1), br.max(1)
    tiny = np.finfo(f32).tiny

    def inv(s):
        return np.where(s >= tiny, f32(1) / np.where(s >= tiny, s, 1), 0).astype(f32)[:, None]

    km = np.rint(np.sqrt(np.abs(bm) * inv(ms)) * f32(127))
    kv = np.rint(np.sqrt(br * inv(vs)) * f32(255))
    kv = np.where((br > 0) & (vs >= tiny)[:, None], np.maximum(kv, 1), kv)
    km = np.where(bm < 0, -km, km).astype(np.int8).reshape(-1)[:m.size]
    return km, ms, kv.astype(np.uint8).reshape(-1)[:m.size], vs


def step32(p, g, m, v, t, scale=1.0, lr=0, beta1=0, beta2=0, eps=0, weight_decay=0):
    lr, b1, b2, eps, wd = (float(f32(x)) for x in (lr, beta1, beta2, eps, weight_decay))
    g = g * f32(scale)
    m = m * f32(b1) + g * f32(1 - b1)
    v = v * f32(b2) + (g * g) * f32(1 - b2)
    r = np.sqrt(v)
    d = (m * f32(lr / (1 - b1 ** t))) / (r * f32(1 / math.sqrt(1 - b2 ** t)) + f32(eps))
    return p * f32(1 - lr * wd) - d, m, v, r


def step64(p, g, m, v, t, scale=1.0, lr=0, beta1=0, beta2=0, eps=0, weight_decay=0):
    lr, b1, b2, eps, wd = (float(f32(x)) for x in (lr, beta1, beta2, eps, weight_decay))
    p, g, m, v = (x.astype(np.float64) for x in (p, g, m, v))
    g = g * scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    d = lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p * (1 - lr * wd) - d, m, v, d


def arrays(sizes, bits, pt=F32, gt=F32, seed=0, shift=0):
    """Parameters, gradients and mid-training states; shift: that many elements off a 256-byte boundary."""
    rng = np.random.default_rng(seed)

    def put(x, dt):
        buf = torch.empty(x.size + shift, dtype=dt, device="cuda")
        buf[shift:] = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt)
        return buf[shift:]

    P, G, M, V, MS, VS = [], [], [], [], [], []
    for n in sizes:
        size = np.exp(rng.normal(size=n)) * 1e-3
        P.append(put(rng.normal(size=n) * 0.02, pt))
        G.append(put(rng.normal(size=n) * size, gt))
        m, v = (rng.normal(size=n) * size * 0.3).astype(f32), ((np.exp(0.3 * rng.normal(size=n)) * size) ** 2).astype(f32)
        if bits == 32:
            M.append(put(m, F32))
            V.append(put(v, F32))
        else:
            km, ms, kv, vs = encode(m, np.sqrt(v))
            M.append(put(km, torch.int8))
            V.append(put(kv, torch.uint8))
            MS.append(put(ms, F32))
            VS.append(put(vs, F32))
    return q.OptimTensors(G, P, M, V, *((MS, VS) if bits == 8 else ()))


def bits_of(x):
    return x.view(np.uint32) if x.dtype == f32 else x


def check_step(T, before, t, scale=1.0, hp=HP):
    for i, n in enumerate(p.numel() for p in T.params):
        p, g, m, v, ms, vs = before[i]
        if T.state_bits == 8:
            m0, v0 = decode(m, ms, v, vs, n)
        else:
            m0, v0 = m, v
        pn, mn, vn, rn = step32(p, g, m0, v0, t, scale, **hp)
        got = to_np(T.params[i])
        if T.params[i].dtype == BF:
            pn = torch.from_numpy(pn).to(BF).float().numpy()
        assert np.array_equal(bits_of(got), bits_of(pn)), i
        if T.state_bits == 32:
            assert np.array_equal(bits_of(to_np(T.m[i])), bits_of(mn)), i
            assert np.array_equal(bits_of(to_np(T.v[i])), bits_of(vn)), i
        else:
            km, sm, kv, sv = encode(mn, rn)
            for a, b in ((T.m, km), (T.m_scale, sm), (T.v, kv), (T.v_scale, sv)):
                assert np.array_equal(bits_of(to_np(a[i])), bits_of(b)), i
        # the formula in 64 bits, from the same states
        p64, m64, v64, d64 = step64(p, g, m0, v0, t, scale, **hp)
        half = 2.0 ** -8 if T.params[i].dtype == BF else 0.0
        # m's cancellation: its two terms each carry 2 roundings, and the step follows m
        terms = 3 * U * (np.abs(m0) + np.abs(scale * g))
        root = np.sqrt(v64 / (1 - float(f32(hp["beta2"])) ** t)) + float(f32(hp["eps"]))
        off = 8 * U * np.abs(d64) + float(f32(hp["lr"])) / (1 - float(f32(hp["beta1"])) ** t) * terms / root
        off = off + 4 * U * np.abs(p) + half * np.abs(p64)
        assert np.all(np.abs(got - p64) <= off * (1 + half)), i


def snapshot(T):
    none = [None] * len(T.params)
    return [tuple(None if x is None else to_np(x).copy() for x in row) for row in
            zip(T.params, T.grads, T.m, T.v, T.m_scale or none, T.v_scale or none)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt", [F32, BF])
@pytest.mark.parametrize("gt", [F32, BF])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_step_is_exact(bits, pt, gt, shift):
    T = arrays(SIZES, bits, pt, gt, seed=bits + shift, shift=shift)
    for t in (1, 2, 1000):
        before = snapshot(T)
        q.qlora_adamw_step(T, t=t, **HP)
        check_step(T, before, t)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [1, 60, 61, 500, 501, 1203])
def test_many_tensors(bits, count):
    """Either form of the launch, its limits, and several launches."""
    sizes = [1 + (37 * i) % 700 for i in range(count)]
    T = arrays(sizes, bits, seed=count)
    before = snapshot(T)
    q.qlora_adamw_step(T, t=3, **HP)
    check_step(T, before, 3)
    c = q.step_control()
    q.qlora_grad_norm(T, 0.0, c)
    want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in T.grads))
    assert abs(float(c[:1].view(F32)) - want) <= 2 * U * want


@pytest.mark.parametrize("bits", [32, 8])
def test_one_large_tensor(bits):
    T = arrays([3_000_001], bits, seed=5)
    before = snapshot(T)
    q.qlora_adamw_step(T, t=9, **HP)
    check_step(T, before, 9)


def test_without_decay_and_states_from_zero():
    for bits in (32, 8):
        P = [torch.full((300,), 0.5, device="cuda"), torch.zeros(7, 9, device="cuda")]
        G = [torch.full((300,), -2.0, device="cuda"), torch.zeros(7, 9, device="cuda")]
        T = q.OptimTensors.with_states(P, G, bits)
        q.qlora_adamw_step(T, t=1, lr=0.1)
        # the first step of a constant gradient is lr sign(g); a zero gradient moves nothing
        assert np.allclose(to_np(P[0]), 0.6, rtol=0, atol=1e-6)
        assert not bool(P[1].any()) and not bool(T.m[1].any()) and not bool(T.v[1].any())


def test_eight_bit_states_hold_what_they_stand_for():
    """Decoded states are within half a step of the square-root code, and nothing that moved keeps a zero v."""
    n = 256 * 40
    rng = np.random.default_rng(3)
    g = (np.exp(3 * rng.normal(size=n)) * rng.choice([-1, 1], size=n)).astype(f32)
    T = q.OptimTensors.with_states([torch.zeros(n, device="cuda")], [torch.from_numpy(g).cuda()], 8)
    q.qlora_adamw_step(T, t=1, lr=1e-3)
    km, kv = to_np(T.m[0]), to_np(T.v[0])
    assert kv.min() >= 1
    m = (f32(1) - f32(0.9)) * g
    dec, dv = decode(km, to_np(T.m_scale[0]), kv, to_np(T.v_scale[0]), n)
    top = np.repeat(to_np(T.m_scale[0]), 256)
    root = np.sqrt(np.abs(m) / top)
    assert np.all(np.abs(np.sqrt(np.abs(dec) / top) - root) <= 0.5 / 127 + 1e-5)
    r, topv = np.sqrt((1 - float(f32(0.999))) * g.astype(np.float64) ** 2), np.repeat(to_np(T.v_scale[0]), 256)
    low = kv == 1  # may have been raised from 0
    err = np.abs(np.sqrt(np.sqrt(dv) / topv) - np.sqrt(r / topv))
    assert np.all(err[~low] <= 0.5 / 255 + 1e-5) and np.all(err <= 1 / 255 + 1e-5)


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradients_are_skipped_or_stay_in_their_block(bits):
    T = arrays([700, 300], bits, seed=8)
    T.grads[0][300] = float("nan")
    before = snapshot(T)
    c = q.step_control()
    q.qlora_grad_norm(T, 1.0, c)
    assert int(c[2]) == 1 and int(c[3]) == 0 and math.isnan(float(c[:1].view(F32))) and float(c[1:2].view(F32)) == 1.0
    q.qlora_adamw_step(T, control=c, **HP)
    for a, b in zip(before, snapshot(T)):
        assert all(x is None or np.array_equal(x, y, equal_nan=x.dtype == f32) for x, y in zip(a, b))
    q.qlora_adamw_step(T, t=1, **HP)  # without control: the value, or its block of 8-bit states, is lost
    assert math.isnan(float(T.params[0][300])) and bool(torch.isfinite(T.params[0][:300]).all())
    T.grads[0][300] = 0.0
    q.qlora_adamw_step(T, t=2, **HP)
    lost = torch.isnan(T.params[0])
    if bits == 8:
        assert bool(lost[256:512].all()) and not bool(lost[:256].any()) and not bool(lost[512:].any())
    else:
        assert int(lost.sum()) == 1
    assert bool(torch.isfinite(T.params[1]).all())


@pytest.mark.parametrize("gt", [F32, BF])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes", [[], [0], [1], SIZES, [3_000_001], [5] * 700])
def test_norm(gt, shift, sizes):
    """64-bit squares and sums (n 2^-53), one square root, one rounding to fp32."""
    T = arrays(sizes, 32, gt=gt, seed=len(sizes), shift=shift)
    G = q.OptimTensors(T.grads)
    c = q.step_control()
    for k, most in enumerate((0.0, 1e-3, 1e9)):
        q.qlora_grad_norm(G, most, c)
        want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in T.grads))
        got, scale = float(c[:1].view(F32)), float(c[1:2].view(F32))
        assert abs(got - want) <= U * (1 + 1e-6) * want
        assert scale == (float(f32(most) / f32(got)) if 0 < most < got else 1.0)
        assert int(c[2]) == 0 and int(c[3]) == k + 1
    again = q.step_control()
    q.qlora_grad_norm(G, 1e9, again)
    assert torch.equal(again[:2], c[:2])


@pytest.mark.parametrize("bad,nan", [(float("nan"), True), (float("inf"), False), (-float("inf"), False)])
def test_norm_of_nonfinite_gradients(bad, nan):
    g = torch.ones(100_000, device="cuda")
    g[77_777] = bad
    c = q.step_control()
    q.qlora_grad_norm(q.OptimTensors([torch.ones(3, device="cuda"), g]), 1.0, c)
    x = float(c[:1].view(F32))
    assert (math.isnan(x) if nan else x == math.inf) and int(c[2]) == 1 and int(c[3]) == 0


def test_norm_where_squares_leave_fp32():
    c = q.step_control()
    q.qlora_grad_norm(q.OptimTensors([torch.full((4,), 1e30, device="cuda")]), 1.0, c)
    assert abs(float(c[:1].view(F32)) - 2e30) <= 1e24 and int(c[2]) == 0
    q.qlora_grad_norm(q.OptimTensors([torch.full((4,), 1e-30, device="cuda")]), 1.0, c)
    assert abs(float(c[:1].view(F32)) - 2e-30) <= 1e-36 and float(c[1:2].view(F32)) == 1.0
    q.qlora_grad_norm(q.OptimTensors([torch.full((64,), 3e38, device="cuda")]), 1.0, c)
    assert int(c[2]) == 1 and int(c[3]) == 2  # the norm itself is above FLT_MAX


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_steps_eager_and_captured(bits):
    """A captured norm and step, replayed, counts its steps and gives the same bits as eager ones."""
    A, B = arrays(SIZES, bits, seed=21), arrays(SIZES, bits, seed=21)
    ca, cb = q.step_control(), q.step_control()
    ws = q.workspace(q.qlora_grad_norm_workspace_bytes(B))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q.qlora_grad_norm(B, 0.05, cb, ws=ws)
        q.qlora_adamw_step(B, control=cb, **HP)
    for k in range(4):
        for i, (x, y) in enumerate(zip(A.grads, B.grads)):
            new = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(100 * k + i))
            x.copy_(new)
            y.copy_(new)
        before = snapshot(A)
        q.qlora_grad_norm(A, 0.05, ca)
        q.qlora_adamw_step(A, control=ca, **HP)
        check_step(A, before, k + 1, scale=float(ca[1:2].view(F32)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ca, cb) and int(ca[3]) == k + 1
        for a, b in zip(snapshot(A), snapshot(B)):
            assert all(x is None or np.array_equal(x, y) for x, y in zip(a, b))


def test_another_stream():
    A, B = arrays(SIZES, 8, seed=31), arrays(SIZES, 8, seed=31)
    q.qlora_adamw_step(A, t=5, **HP)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q.qlora_adamw_step(B, t=5, **HP)
    torch.cuda.synchronize()
    for a, b in zip(snapshot(A), snapshot(B)):
        assert all(x is None or np.array_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
def test_values_around_the_tensors_stay(bits):
    buf = torch.full((4096,), 3.0, device="cuda")
    p, g = buf[100:100 + 777], torch.randn(777, device="cuda")
    st = torch.full((2000,), 9, dtype=torch.int8 if bits == 8 else F32, device="cuda")
    st2 = torch.full((2000,), 9, dtype=torch.uint8 if bits == 8 else F32, device="cuda")
    st[50:827] = 0
    st2[50:827] = 0
    extra = ([torch.zeros(4, device="cuda")], [torch.zeros(4, device="cuda")]) if bits == 8 else ()
    T = q.OptimTensors([g], [p], [st[50:827]], [st2[50:827]], *extra)
    q.qlora_adamw_step(T, t=1, **HP)
    assert bool((buf[:100] == 3).all()) and bool((buf[877:] == 3).all())
    for x in (st, st2):
        assert bool((x[:50] == 9).all()) and bool((x[827:] == 9).all())


def test_a_training_step_on_an_int8_base():
    """Forward, backward, clipping and the 8-bit AdamW step as they are used
    together, three times, against the same step in 64 bits: the adapters
    follow it, and the frozen weight keeps every byte."""
    torch.manual_seed(0)
    R, O, I, r, alpha = 200, 320, 256, 8, 16.0
    layers = []
    for k in range(2):
        w = q.qlora_quantize_int8(torch.randn(O if k == 0 else I, I if k == 0 else O, device="cuda") * 0.05)
        layers.append((w, torch.randn(r, w.I, device="cuda") * 0.05, torch.randn(w.O, r, device="cuda") * 0.05))
    params = [x for _, A, B in layers for x in (A, B)]
    grads = [torch.zeros_like(p) for p in params]
    T = q.OptimTensors.with_states(params, grads, 8)
    c = q.step_control()
    codes = [w.codes.clone() for w, _, _ in layers]
    X = torch.randn(R, I, device="cuda")
    target = torch.randn(R, I, device="cuda")
    for k in range(3):
        H, U0 = q.qlora_linear_fwd(layers[0][0], X, layers[0][1], layers[0][2], alpha)
        Y, U1 = q.qlora_linear_fwd(layers[1][0], H, layers[1][1], layers[1][2], alpha)
        dY = Y - target
        dH, _, _ = q.qlora_linear_bwd(layers[1][0], H, dY, layers[1][1], layers[1][2], alpha, U=U1,
                                      dA=grads[2], dB=grads[3])
        q.qlora_linear_bwd(layers[0][0], X, dH, layers[0][1], layers[0][2], alpha, U=U0, want_dx=False,
                           dA=grads[0], dB=grads[1])
        s = alpha / r
        want = [s * (dH.double() @ params[1].double()).T @ X.double(), s * dH.double().T @ (X.double() @ params[0].double().T),
                s * (dY.double() @ params[3].double()).T @ H.double(), s * dY.double().T @ (H.double() @ params[2].double().T)]
        for g, x in zip(grads, want):  # fp32 sums of R and I terms: well within 1e-5 of their norm
            assert float((g.double() - x).norm() / x.norm()) < 1e-5
        before = snapshot(T)
        q.qlora_grad_norm(T, 1.0, c)
        q.qlora_adamw_step(T, control=c, lr=1e-3, weight_decay=0.01)
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
        assert abs(float(c[:1].view(F32)) - norm) <= 2 * U * norm and int(c[3]) == k + 1
        check_step(T, before, k + 1, scale=float(c[1:2].view(F32)),
                   hp=dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01))
    assert all(torch.equal(a, w.codes) for a, (w, _, _) in zip(codes, layers))
    out = q.qlora_merge(*layers[0], alpha)
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_a_control_block_without_a_step_changes_nothing(bits):
    T = arrays(SIZES, bits, seed=41)
    before = snapshot(T)
    q.qlora_adamw_step(T, control=q.step_control(), **HP)
    for a, b in zip(before, snapshot(T)):
        assert all(x is None or np.array_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_norm_on_a_stream_of_its_own_keeps_its_workspace(bits):
    """The workspace that a call allocates is not handed out while its stream still uses it."""
    T = arrays([300_000] * 40, bits, seed=43)
    want = q.qlora_grad_norm(T, 1.0, q.step_control()).clone()
    side = torch.cuda.Stream()
    out = [q.step_control() for _ in range(6)]
    torch.cuda.synchronize()
    for c in out:
        q.qlora_grad_norm(T, 1.0, c, stream=side)
        for _ in range(4):
            torch.full((q.qlora_grad_norm_workspace_bytes(T),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c in out)


def test_what_is_written_overlaps_nothing():
    buf = torch.zeros(4096, device="cuda")
    z = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    for p, g in ((buf[:512], buf[256:768]), (buf[256:768], buf[:512]), (buf[:512], buf[:512]), (buf[100:200], buf[:512])):
        with pytest.raises(ValueError):
            q.OptimTensors([g], [p], [z(p.numel())], [z(p.numel())])
    # beside each other, and one gradient for two parameters, are fine
    q.OptimTensors([buf[512:1024]] * 2, [buf[:512], buf[1024:1536]], [z(512), z(512)], [z(512), z(512)])
