"""Measured cases of the 8-bit integer linear layer and of the optimizer step over many tensors.

Operators (plain form: elementary torch operations; own form: the library's calls):
  quant  per-channel 8-bit quantization of a weight matrix
  fwd    Y  = X_q W_q^T with a scale for each token and channel, + s (X A^T) B^T
  bwd    dX = (dY sw)_q W_q with a scale for each token, + s (dY B) A;  dA, dB
  norm   global gradient norm of many tensors, clip factor, finite check, step count
  adamw  AdamW over many tensors, states in 32 or in 8 bits
"""
import math

import torch

own = False

DEV = "cuda"
T = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 256  # values of an 8-bit state that share a scale


def listed():
    return [
        # one token of generation through the widest projection: weight bytes and launch latency
        {"name": "fwd one token 12288x4096", "op": "fwd", "R": 1, "O": 12288, "I": 4096, "r": 8, "dtype": "bf16"},
        # a short, ragged prompt through a small attention projection
        {"name": "fwd 777 tokens 2048x1024", "op": "fwd", "R": 777, "O": 2048, "I": 1024, "r": 8, "dtype": "bf16"},
        # a training batch through the 14B-class gate projection
        {"name": "fwd 16384 tokens 17408x5120", "op": "fwd", "R": 16384, "O": 17408, "I": 5120, "r": 16, "dtype": "bf16"},
        # gradients of a few tokens
        {"name": "bwd 16 tokens 4096x4096", "op": "bwd", "R": 16, "O": 4096, "I": 4096, "r": 8, "dtype": "bf16"},
        # a training batch back through the 8B-class gate projection
        {"name": "bwd 8192 tokens 12288x4096", "op": "bwd", "R": 8192, "O": 12288, "I": 4096, "r": 32, "dtype": "bf16"},
        # a small attention projection at load time
        {"name": "quant 1024x1024", "op": "quant", "O": 1024, "I": 1024},
        # the largest weight at load time
        {"name": "quant 17408x5120", "op": "quant", "O": 17408, "I": 5120},
        # the adapters of the q and v projections of a small model, states in 32 bits
        {"name": "adamw 32 bits 112 tensors", "op": "adamw", "bits": 32, "layers": 28, "r": 8,
         "shapes": "2048x1024,1024x1024", "ptype": "fp32", "gtype": "fp32", "shift": 0, "t": 100},
        # the same, states in 8 bits, gradients in bf16, at an address that no wide load fits
        {"name": "adamw 8 bits 112 tensors", "op": "adamw", "bits": 8, "layers": 28, "r": 8,
         "shapes": "2048x1024,1024x1024", "ptype": "fp32", "gtype": "bf16", "shift": 1, "t": 7},
        # every linear of a 14B-class model, states in 8 bits
        {"name": "adamw 8 bits 560 tensors", "op": "adamw", "bits": 8, "layers": 40, "r": 16,
         "shapes": "5120x5120,1024x5120,1024x5120,5120x5120,17408x5120,17408x5120,5120x17408",
         "ptype": "fp32", "gtype": "fp32", "shift": 0, "t": 1000},
        # gradient clipping of the two sets
        {"name": "norm 112 tensors", "op": "norm", "layers": 28, "r": 8, "shapes": "2048x1024,1024x1024",
         "gtype": "fp32", "shift": 0},
        {"name": "norm 560 tensors", "op": "norm", "layers": 40, "r": 16,
         "shapes": "5120x5120,1024x5120,1024x5120,5120x5120,17408x5120,17408x5120,5120x17408",
         "gtype": "fp32", "shift": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _side(rng, lo, hi):
    """A matrix extent: a multiple of 128, of 16, or any number."""
    n = _log(rng, lo, hi)
    step = rng.choice((128, 16, 16, 1))
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "adamw", "adamw", "norm", "quant"))
    if op in ("fwd", "bwd"):
        O, I = _side(rng, 64, 17408), _side(rng, 64, 17408)
        most = 16384 * 17408 * 5120 // (2 if op == "bwd" else 1)
        R = _log(rng, 1, max(1, min(16384, most // (O * I))))
        return {"op": op, "R": R, "O": O, "I": I, "r": rng.choice((1, 4, 8, 16, 32, 64)),
                "dtype": rng.choice(("bf16", "bf16", "bf16", "fp32"))}
    if op == "quant":
        O = _side(rng, 64, 17408)
        return {"op": op, "O": O, "I": _side(rng, 64, min(17408, 17408 * 5120 // O))}
    c = {"op": op, "layers": rng.randint(1, 40), "r": rng.choice((4, 8, 16, 32, 64)),
         "shapes": ",".join("%dx%d" % (_side(rng, 64, 8192), _side(rng, 64, 8192)) for _ in range(rng.randint(1, 7))),
         "gtype": rng.choice(("fp32", "fp32", "bf16")), "shift": rng.choice((0, 0, 0, 1))}
    while _total(c) > 60_000_000:
        c["layers"] = max(1, c["layers"] // 2)
        c["r"] = max(4, c["r"] // 2)
    if op == "adamw":
        c |= {"bits": rng.choice((8, 32)), "ptype": rng.choice(("fp32", "fp32", "bf16")), "t": _log(rng, 1, 20000)}
    return c


# ------------------------------------------------------------------ inputs

def _sizes(case):
    """Element counts of the adapter factors, A [r x I] and B [O x r] of each linear of each layer."""
    r, one = case["r"], []
    for s in case["shapes"].split(","):
        O, I = (int(v) for v in s.split("x"))
        one += [r * I, O * r]
    return one * case["layers"]


def _total(case):
    return sum(_sizes(case))


def _places(case):
    """Where each tensor lies in the arena that holds them all: from a multiple of 256 on, zeros between."""
    at, total = [], 0
    for n in _sizes(case):
        at.append((total, n))
        total += (n + BLOCK - 1) // BLOCK * BLOCK
    return at, total


def _shifted(n, dtype, shift):
    return torch.zeros(n + shift, dtype=dtype, device=DEV)[shift:]


def pitch(I):
    return (I + 15) // 16 * 16


def _weight(case, gen):
    """Normal weights, one in a thousand twenty times as large."""
    O, I = case["O"], case["I"]
    W = torch.randn(O, I, device=DEV, generator=gen) * 0.02
    return torch.where(torch.rand(O, I, device=DEV, generator=gen) < 0.001, W * 20, W)


def _activations(R, n, gen, dtype, size):
    """Tokens of differing size, a few strong channels, one padded (all-zero) token in about 32."""
    x = torch.randn(R, n, device=DEV, generator=gen)
    x *= size * torch.exp(0.5 * torch.randn(R, 1, device=DEV, generator=gen))
    x *= torch.where(torch.rand(1, n, device=DEV, generator=gen) < 0.005, 10.0, 1.0)
    if R > 1:
        x *= torch.rand(R, 1, device=DEV, generator=gen) >= 0.03
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "quant":
        s["W"] = _weight(case, gen)
        return s
    if op in ("fwd", "bwd"):
        R, O, I, r = case["R"], case["O"], case["I"], case["r"]
        W = _weight(case, gen)
        s["scale"] = W.abs().amax(1) / 127
        s["codes"] = torch.zeros(O, pitch(I), dtype=torch.int8, device=DEV)
        s["codes"][:, :I] = torch.round(W / s["scale"][:, None]).to(torch.int8)
        del W
        s["A"] = torch.randn(r, I, device=DEV, generator=gen) * 0.02
        s["B"] = torch.randn(O, r, device=DEV, generator=gen) * 0.02
        s["alpha"] = 2.0 * r
        s["X"] = _activations(R, I, gen, T[case["dtype"]], 1.0)
        if op == "bwd":
            s["dY"] = _activations(R, O, gen, T[case["dtype"]], 1e-3)
            s["U"] = (s["X"].double() @ s["A"].double().T).float()
        return s
    at, total = _places(case)
    live = torch.zeros(total, device=DEV)
    for a, n in at:
        live[a:a + n] = 1
    rand = lambda: torch.randn(total, device=DEV, generator=gen)  # noqa: E731
    size = torch.exp(rand()) * 1e-3
    s["g"] = _shifted(total, T[case["gtype"]], case["shift"])
    s["g"].copy_(rand() * size * live)
    s["control"] = torch.zeros(4, dtype=torch.int32, device=DEV)  # norm, scale, skip, step
    if op == "norm":
        s["max_norm"] = 0.3
        return s
    s["control"][1:2].view(torch.float32).fill_(0.5)
    s["control"][3] = case["t"]
    s["p"] = _shifted(total, T[case["ptype"]], case["shift"])
    s["p"].copy_(rand() * 0.02 * live)
    m, v = rand() * size * 0.3 * live, (torch.exp(0.3 * rand()) * size) ** 2 * live
    if case["bits"] == 32:
        s["m"], s["v"] = _shifted(total, torch.float32, case["shift"]), _shifted(total, torch.float32, case["shift"])
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        s["m"], s["m_scale"] = _code_m(m)
        s["v"], s["v_scale"] = _code_r(v.sqrt())
    return s


# ------------------------------------------------------------- plain forms

def _over_127(a):
    return a / torch.full((1,), 127.0, device=DEV)  # a true division


def _quant_rows(x):
    """Codes and scale of each row: scale = max |x| / 127, code = round(x / scale), half to even."""
    scale = _over_127(x.abs().amax(1))
    q = torch.round(x / scale[:, None])
    return torch.where(scale[:, None] > 0, q, 0.0).clamp(-127, 127), scale


def _lora_scale(s):
    return s["alpha"] / s["r"]


def _plain_quant(s):
    q, scale = _quant_rows(s["W"])
    codes = torch.zeros(s["O"], pitch(s["I"]), dtype=torch.int8, device=DEV)
    codes[:, :s["I"]] = q.to(torch.int8)
    return {"codes": codes, "scale": scale}


def _plain_fwd(s):
    X = s["X"].float()
    q, sx = _quant_rows(X)
    U = X @ s["A"].T
    Y = q @ s["codes"][:, :s["I"]].float().T
    Y = Y * sx[:, None] * s["scale"][None, :]
    Y += _lora_scale(s) * (U @ s["B"].T)
    return {"Y": Y.to(s["X"].dtype), "U": U}


def _plain_bwd(s):
    X, dY, c = s["X"].float(), s["dY"].float(), _lora_scale(s)
    V = dY @ s["B"]
    dA, dB = c * (V.T @ X), c * (dY.T @ s["U"])
    q, sg = _quant_rows(dY * s["scale"][None, :])
    dX = q @ s["codes"][:, :s["I"]].float()
    dX = dX * sg[:, None] + c * (V @ s["A"])
    return {"dX": dX.to(s["X"].dtype), "dA": dA, "dB": dB}


def _control(s):
    c = s["control"]
    return {"norm": c[0:1].view(torch.float32), "scale": c[1:2].view(torch.float32), "skip": c[2:3], "step": c[3:4]}


def _plain_norm(s):
    c = _control(s)
    norm = s["g"].double().square().sum().sqrt().float()
    most = torch.full_like(norm, s["max_norm"])
    c["norm"].copy_(norm)
    c["scale"].copy_(torch.where(norm > most, most / norm, torch.ones_like(norm)))
    c["skip"].copy_(~torch.isfinite(norm))
    c["step"].add_(torch.isfinite(norm))
    return c


LR, B1, B2, EPS, WD = (float(torch.tensor(x, dtype=torch.float32)) for x in (2e-4, 0.9, 0.999, 1e-8, 0.01))


def _inverse(scale):
    return torch.where(scale >= 2.0 ** -126, 1 / scale, 0.0)[:, None]


def _code_m(m):
    """Signed 8-bit codes of blocks of 256: the square root of |m| over the block's largest, in 127 steps."""
    m = m.view(-1, BLOCK)
    scale = m.abs().amax(1)
    q = torch.round(torch.sqrt(m.abs() * _inverse(scale)) * 127.0)
    return torch.where(m < 0, -q, q).to(torch.int8).view(-1), scale


def _code_r(r):
    """Unsigned 8-bit codes of r = sqrt(v), in 255 steps of its square root; what is not zero keeps a code of 1 at least."""
    r = r.view(-1, BLOCK)
    scale = r.amax(1)
    q = torch.round(torch.sqrt(r * _inverse(scale)) * 255.0)
    q = torch.where((r > 0) & (scale[:, None] >= 2.0 ** -126), q.clamp(min=1), q)
    return q.to(torch.uint8).view(-1), scale


def _plain_adamw(s):
    c = _control(s)
    bc1, bc2 = 1.0 - B1 ** s["t"], 1.0 - B2 ** s["t"]
    g = s["g"].float() * c["scale"]
    if s["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        u = s["m"].view(-1, BLOCK).float() * (1.0 / 127.0)
        m = ((u * u.abs()) * s["m_scale"][:, None]).view(-1)
        u = s["v"].view(-1, BLOCK).float() * (1.0 / 255.0)
        v = ((u * u) * s["v_scale"][:, None]).view(-1)
        v = v * v
    m = m * B1 + g * (1.0 - B1)
    v = v * B2 + (g * g) * (1.0 - B2)
    r = torch.sqrt(v)
    step = (m * (LR / bc1)) / (r * (1.0 / math.sqrt(bc2)) + EPS)
    s["p"].copy_(s["p"].float() * (1.0 - LR * WD) - step)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    q, scale = _code_m(m)
    s["m"].copy_(q)
    s["m_scale"].copy_(scale)
    q, scale = _code_r(r)
    s["v"].copy_(q)
    s["v_scale"].copy_(scale)
    return {"p": s["p"], "m": s["m"], "m_scale": s["m_scale"], "v": s["v"], "v_scale": s["v_scale"]}


# ------------------------------------------------------- the library's calls

def _own_weight(q, s):
    """The weight, as a program keeps it once it has quantized or loaded it."""
    if "weight" not in s:
        s["weight"] = q.QuantizedWeight(q.FMT_INT8, s["O"], s["I"], s["I"], 0, 8, s["codes"], scale=s["scale"])
    return s["weight"]


def _own_tensors(q, s):
    """The tensors of the arena, as a training program keeps them."""
    if "tensors" not in s:
        at, _ = _places(s)
        cut = lambda x: [x[a:a + n] for a, n in at]  # noqa: E731
        scales = lambda x: [x[a // BLOCK:-(-(a + n) // BLOCK)] for a, n in at]  # noqa: E731
        kw = {}
        if s["op"] == "adamw":
            kw = {"params": cut(s["p"]), "m": cut(s["m"]), "v": cut(s["v"])}
            if s["bits"] == 8:
                kw |= {"m_scale": scales(s["m_scale"]), "v_scale": scales(s["v_scale"])}
        s["tensors"] = q.OptimTensors(grads=cut(s["g"]), **kw)
    return s["tensors"]


def _own_run(s):
    import qlora_bit_frozen_b200 as q

    op = s["op"]
    if op == "quant":
        w = q.qlora_quantize_int8(s["W"])
        return {"codes": w.codes, "scale": w.scale}
    if op == "fwd":
        Y, U = q.qlora_linear_fwd(_own_weight(q, s), s["X"], s["A"], s["B"], s["alpha"])
        return {"Y": Y, "U": U}
    if op == "bwd":
        dX, dA, dB = q.qlora_linear_bwd(_own_weight(q, s), s["X"], s["dY"], s["A"], s["B"], s["alpha"], U=s["U"])
        return {"dX": dX, "dA": dA, "dB": dB}
    if op == "norm":
        q.qlora_grad_norm(_own_tensors(q, s), s["max_norm"], s["control"])
        return _control(s)
    q.qlora_adamw_step(_own_tensors(q, s), lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, control=s["control"])
    names = ("p", "m", "v") if s["bits"] == 32 else ("p", "m", "m_scale", "v", "v_scale")
    return {k: s[k] for k in names}


def run(s):
    if own:
        return _own_run(s)
    return {"quant": _plain_quant, "fwd": _plain_fwd, "bwd": _plain_bwd, "norm": _plain_norm, "adamw": _plain_adamw}[s["op"]](s)


# --------------------------------------------------------------------- cost

def work(case):
    op = case["op"]
    if op == "quant":
        O, I = case["O"], case["I"]
        return {"bytes": 4 * O * I + O * pitch(I) + 4 * O, "flops": 3 * O * I}
    if op in ("fwd", "bwd"):
        R, O, I, r = case["R"], case["O"], case["I"], case["r"]
        e = 2 if case["dtype"] == "bf16" else 4
        b = O * I + 4 * O + 4 * r * (O + I) + e * R * (O + I) + 4 * R * r
        f = 2 * R * O * I + 2 * R * r * (O + I)
        if op == "bwd":
            b += 4 * r * (O + I) + e * R * I
            f += 2 * R * r * (O + I)
        return {"bytes": b, "flops": f}
    n, e = _total(case), {"fp32": 4, "bf16": 2}
    if op == "norm":
        return {"bytes": e[case["gtype"]] * n, "flops": 2 * n}
    state = 4 * 4 if case["bits"] == 32 else 4 * 1 + 4 * 4 / BLOCK
    return {"bytes": (2 * e[case["ptype"]] + e[case["gtype"]] + state) * n, "flops": 15 * n}


# ------------------------------------------------- from the definition, 64 bits

def _f32(x):
    """A value that the definition holds in 32 bits, in 64."""
    return x.float().double()


def _exact_rows(x):
    """A row's 8-bit integers n and step d, n the whole number nearest to x / d; both are part of the definition."""
    top = torch.maximum(x.max(1).values, -x.min(1).values)
    d = _f32(top / 127.0).unsqueeze(1)
    n = torch.round(_f32(x / torch.where(d > 0, d, 1.0)))
    return torch.clamp(n, -127, 127) * (d > 0), d


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        n, d = _exact_rows(s["W"].double())
        return {"codes": None, "scale": d.squeeze(1)}
    if op in ("fwd", "bwd"):
        W = s["codes"].narrow(1, 0, case["I"]).double()
        A, B, d = s["A"].double(), s["B"].double(), s["scale"].double()
        c, X = 2.0, s["X"].double()
        if op == "fwd":
            n, dx = _exact_rows(X)
            U = X @ A.T
            Y = torch.mm(n, W.T).mul_(dx).mul_(d)
            return {"Y": Y.addmm_(U, B.T, alpha=c), "U": U}
        dY = s["dY"].double()
        V = dY @ B
        n, dg = _exact_rows(_f32(dY * d))
        dX = torch.mm(n, W).mul_(dg)
        return {"dX": dX.addmm_(V, A, alpha=c), "dA": c * torch.mm(V.T, X), "dB": c * torch.mm(dY.T, s["U"].double())}
    g = s["g"].double()
    if op == "norm":
        n = torch.linalg.vector_norm(g).reshape(1)
        return {"norm": n, "scale": torch.clamp(s["max_norm"] / n, max=1.0), "skip": None, "step": None}
    lr, b1, b2, eps, wd, t = LR, B1, B2, EPS, WD, case["t"]
    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        k = s["m"].double().reshape(-1, BLOCK) / 127
        m = (s["m_scale"].double().unsqueeze(1) * k * abs(k)).flatten()
        k = s["v"].double().reshape(-1, BLOCK) / 255
        v = ((s["v_scale"].double().unsqueeze(1) * k ** 2) ** 2).flatten()
    g = 0.5 * g
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    mh, vh = m / (1 - b1 ** t), v / (1 - b2 ** t)
    p = s["p"].double() * (1 - lr * wd) - lr * mh / (vh ** 0.5 + eps)
    if case["bits"] == 32:
        return {"p": p, "m": m, "v": v}
    top = lambda x: x.reshape(-1, BLOCK).max(1).values  # noqa: E731
    return {"p": p, "m": None, "m_scale": top(abs(m)), "v": None, "v_scale": top(v ** 0.5)}
