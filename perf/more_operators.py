"""Cases of the feed-forward block's operators:

  quant                      rows to 8-bit codes with a scale for each row
  i8                         product of 8-bit codes with scales for each token and channel,
                             plain or gated
  gated                      act(x G^T) * (x U^T): both projections and the gate
  gated_grad                 its gradients, from saved or recomputed pre-activations

With `own` false `run` computes each in plain torch operations in 32 bits (codes
and sums of codes in 64 bits, where 32 would lose whole numbers), rounded once;
with `own` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CODE = {"f32": 0, "f16": 1, "bf16": 2}  # the library's dtype numbers
NONE, SILU, GELU = 0, 1, 2              # the library's gates
TINY = 2.0 ** -126                      # smallest scale


def listed():
    return [
        # One token's activations before an 8-bit projection: latency alone counts.
        dict(name="quant_token", op="quant", m=1, k=4096, dtype="bf16"),
        # A long prompt's activations before the down projection; odd token count.
        dict(name="quant_prompt", op="quant", m=8191, k=11008, dtype="bf16"),
        # One token through the gate and up projections of a served layer.
        dict(name="i8_token", op="i8", m=1, n=11008, k=4096, dtype="bf16", gate=SILU),
        # Thirteen sequences decoding together, down projection; odd output count.
        dict(name="i8_batch", op="i8", m=13, n=4099, k=11008, dtype="f16", gate=NONE),
        # A 512-token prefill through one expert-sized gated block.
        dict(name="i8_prompt", op="i8", m=512, n=1408, k=2048, dtype="bf16", gate=SILU),
        # The largest product: a long prompt through a square projection.
        dict(name="i8_large", op="i8", m=8192, n=8192, k=8192, dtype="f16", gate=NONE),
        # One token through a gated block with plain weights.
        dict(name="gated_token", op="gated", m=1, n=11008, k=4096, dtype="f16", gate=SILU, saved=0),
        # Forty-eight sequences decoding together.
        dict(name="gated_batch", op="gated", m=48, n=11008, k=4096, dtype="bf16", gate=GELU, saved=0),
        # Forward of a training step: the pre-activations are kept for the backward pass.
        dict(name="gated_train", op="gated", m=4096, n=11008, k=4096, dtype="bf16", gate=SILU, saved=1),
        # A small layer trained in 32 bits; odd token count.
        dict(name="gated_f32", op="gated", m=509, n=1408, k=2048, dtype="f32", gate=SILU, saved=1),
        # Backward of that training step.
        dict(name="grad_train", op="gated_grad", m=4096, n=11008, k=4096, dtype="bf16", gate=SILU, saved=1),
        # Backward with activation checkpointing: pre-activations computed again; odd token count.
        dict(name="grad_again", op="gated_grad", m=3001, n=1408, k=2048, dtype="f16", gate=GELU, saved=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _stepped(rng, lo, hi, step):
    return step * _log_int(rng, max(1, lo // step), hi // step)


def draw(rng):
    op = rng.choice(["quant", "i8", "i8", "gated", "gated", "gated_grad", "gated_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "quant":
        k = _stepped(rng, 64, 16384, 64) if rng.random() < 0.7 else _log_int(rng, 16, 16384)
        return dict(op=op, m=min(_log_int(rng, 1, 16384), (1 << 25) // k), k=k, dtype=dtype)
    n = _stepped(rng, 64, 16384, 64) if rng.random() < 0.7 else _log_int(rng, 16, 16384)
    if op == "i8":
        gate = rng.choice([NONE, SILU, GELU])
        k = _stepped(rng, 128, 16384, rng.choice([16, 64, 128]))
        n = min(n, (1 << 28) // ((1 + (gate > 0)) * k))
        return dict(op=op, m=min(_log_int(rng, 1, 8192), (1 << 38) // (n * k)), n=n, k=k, dtype=dtype, gate=gate)
    k = _stepped(rng, 64, 8192, 64) if rng.random() < 0.7 else _log_int(rng, 16, 8192)
    n = min(n, (1 << 26) // k)
    # products of at most 2^35 multiplications, 2^33 in 32 bits
    m = max(1, min(_log_int(rng, 1, 8192), (1 << (33 if dtype == "f32" else 35)) // (n * k)))
    return dict(op=op, m=m, n=n, k=k, dtype=dtype, gate=rng.choice([SILU, GELU]), saved=rng.randint(0, 1))


# ---- what a program holds before the call ------------------------------------


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _activations(g, m, k, dtype):
    """Normal values; one channel in 64 is ten times as large, as activations have them."""
    x = torch.randn(m, k, generator=g, device=DEV)
    x *= torch.where(torch.rand(k, generator=g, device=DEV) < 1 / 64, 10.0, 1.0)
    return x.to(dtype)


def _codes(x):
    """Codes of the rows of x and their scales."""
    top = x.abs().amax(1).double()
    scale = (top / 127).clamp_min(TINY).float()
    return torch.round(x.double() / scale.double()[:, None]).to(torch.int8), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    op, m, k, t = c["op"], c["m"], c["k"], DTYPES[c["dtype"]]
    empty = lambda *shape, d=t: torch.empty(*shape, dtype=d, device=DEV)  # noqa: E731
    if op == "quant":
        s["x"] = _activations(g, m, k, t)
        s["q"], s["scale"] = empty(m, k, d=torch.int8), empty(m, d=torch.float32)
        return s
    n = c["n"]
    if op == "i8":
        s["q"], s["scale"] = _codes(_activations(g, m, k, torch.float32))
        s["w"], s["wscale"] = _codes(_randn(g, n * (1 + (c["gate"] > 0)), k, scale=1 / math.sqrt(k)))
        s["y"] = empty(m, n)
        return s
    s["x"] = _randn(g, m, k, dtype=t)
    s["w"] = _randn(g, 2 * n, k, scale=1.2 / math.sqrt(k), dtype=t)
    if op == "gated":
        s["h"] = empty(m, n)
        s["pre"] = empty(m, 2 * n) if c["saved"] else None
        return s
    s["pre"] = (s["x"].float() @ s["w"].float().t()).to(t) if c["saved"] else None
    s["dh"] = _randn(g, m, n, dtype=t)
    s["dpre"], s["dx"], s["dw"] = empty(m, 2 * n), empty(m, k), empty(2 * n, k)
    return s


# ---- the plain forms -----------------------------------------------------------


def _plain_quant(s):
    q, scale = _codes(s["x"])
    return {"q": q, "scale": scale}


def _sigmoid_part(a, gate):
    """sigmoid(z(a)) with act(a) = a * sigmoid(z(a)), and z'(a)."""
    if gate == SILU:
        return 1 / (1 + torch.exp(-a)), 1.0
    c = 2 * math.sqrt(2 / math.pi)
    return 1 / (1 + torch.exp(-c * (a + 0.044715 * a * a * a))), c * (1 + 3 * 0.044715 * a * a)


def _plain_i8(s):
    c = s["case"]
    q, w = s["q"].float(), s["w"].float()
    total = torch.zeros(q.shape[0], w.shape[0], dtype=torch.float64, device=q.device)
    for at in range(0, c["k"], 1024):  # sums of 1024 products stay whole numbers in 32 bits
        total += q[:, at:at + 1024] @ w[:, at:at + 1024].t()
    y = total.float() * s["wscale"] * s["scale"][:, None]
    if c["gate"]:
        a, b = y[:, : c["n"]], y[:, c["n"]:]
        y = a * _sigmoid_part(a, c["gate"])[0] * b
    return {"y": y.to(s["y"].dtype)}


def _plain_gated(s):
    c, t = s["case"], s["x"].dtype
    pre = s["x"].float() @ s["w"].float().t()
    a, b = pre[:, : c["n"]], pre[:, c["n"]:]
    out = {"h": (a * _sigmoid_part(a, c["gate"])[0] * b).to(t)}
    if c["saved"]:
        out["pre"] = pre.to(t)
    return out


def _plain_gated_grad(s):
    c, t = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    pre = s["pre"].float() if c["saved"] else x @ w.t()
    a, b, d = pre[:, : c["n"]], pre[:, c["n"]:], s["dh"].float()
    sig, slope = _sigmoid_part(a, c["gate"])
    dpre = torch.cat((d * b * (sig + a * sig * (1 - sig) * slope), d * a * sig), 1)
    return {"dpre": dpre.to(t), "dx": (dpre @ w).to(t), "dw": (dpre.t() @ x).to(t)}


PLAIN = {"quant": _plain_quant, "i8": _plain_i8, "gated": _plain_gated, "gated_grad": _plain_gated_grad}


# ---- the library's calls ---------------------------------------------------------


def _call(s):
    """The library entry point, the descriptor and the buffers of a state, as a serving or training loop keeps
    them, and the outputs."""
    import gemv_expert_id_amd as mm

    c = s["case"]
    op, dt, m, k = c["op"], CODE[c["dtype"]], c["m"], c["k"]
    buf = lambda *names: [mm.buf(s[n]) for n in names]  # noqa: E731
    if op == "quant":
        return mm.mm_i8_quant, mm.quant_params(dt, m, k), buf("x", "q", "scale"), {n: s[n] for n in ("q", "scale")}
    if op == "i8":
        p = mm.i8_params(dt, m, c["n"], k, gate=c["gate"])
        return mm.mm_i8_gemm, p, buf("q", "scale", "w", "wscale", "y"), {"y": s["y"]}
    p = mm.gated_params(dt, m, c["n"], k, gate=c["gate"])
    pre = mm.buf(s["pre"]) if c["saved"] else None
    if op == "gated":
        names = ("h", "pre") if c["saved"] else ("h",)
        return mm.mm_gated, p, buf("x", "w", "h") + [pre], {n: s[n] for n in names}
    return (mm.mm_gated_grad, p, buf("x", "w") + [pre] + buf("dh", "dpre", "dx", "dw"),
            {n: s[n] for n in ("dpre", "dx", "dw")})


def run(state):
    if own:
        if "call" not in state:
            state["call"] = _call(state)
        entry, params, bufs, outputs = state["call"]
        entry(params, *bufs, stream=torch.cuda.current_stream())
        return outputs
    return PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------


def work(case):
    c = case
    op, m, k, z = c["op"], c["m"], c["k"], SIZE[c["dtype"]]
    if op == "quant":
        return {"bytes": m * k * (z + 1) + 4 * m, "flops": 3 * m * k}
    n = c["n"]
    if op == "i8":
        rows = n * (1 + (c["gate"] > 0))
        return {"bytes": (m + rows) * (k + 4) + m * n * z, "flops": 2 * m * rows * k}
    if op == "gated":
        return {"bytes": (m * k + 2 * n * k + m * n * (1 + 2 * c["saved"])) * z, "flops": 4 * m * n * k}
    return {"bytes": (2 * m * k + 4 * n * k + m * n * (3 + 2 * c["saved"])) * z,
            "flops": (8 if c["saved"] else 12) * m * n * k}


# ---- the definitions in 64 bits ------------------------------------------------------


def _exact_quant(s):
    """Codes by counting the borders that each magnitude passes: border j lies at (j - 1/2) scale, ties to even."""
    x = s["x"].double()
    scale = torch.maximum(x.amax(1), -x.amin(1)).div(127).to(torch.float32)
    scale = torch.where(scale < TINY, torch.full_like(scale, TINY), scale)
    mag, half = x.abs(), scale.double()[:, None] * 0.5
    j = torch.floor(mag / scale.double()[:, None])
    rest = mag - j * scale.double()[:, None]  # exact: 24 bits and 7
    up = (rest > half) | ((rest == half) & (j % 2 == 1))
    return {"q": ((j + up) * torch.sign(x)).to(torch.int8), "scale": scale}


def _act64(a, gate):
    """act and its derivative, through tanh."""
    if gate == SILU:
        t = torch.tanh(a / 2)
        return a * (1 + t) / 2, (1 + t) / 2 + a * (1 - t * t) / 4
    r = math.sqrt(2 / math.pi)
    t = torch.tanh(r * (a + 0.044715 * a ** 3))
    return a * (1 + t) / 2, (1 + t) / 2 + a * (1 - t * t) / 2 * r * (1 + 0.134145 * a ** 2)


def _exact_i8(s):
    c = s["case"]
    n = c["n"]
    x = s["q"].double() * s["scale"].double()[:, None]
    w = s["w"].double() * s["wscale"].double()[:, None]
    if not c["gate"]:
        return {"y": x @ w.t()}
    return {"y": _act64(x @ w[:n].t(), c["gate"])[0] * (x @ w[n:].t())}


def _exact_gated(s):
    n, x, w = s["case"]["n"], s["x"].double(), s["w"].double()
    a, b = x @ w[:n].t(), x @ w[n:].t()
    out = {"h": _act64(a, s["case"]["gate"])[0] * b}
    if s["case"]["saved"]:
        out["pre"] = torch.cat((a, b), 1)
    return out


def _exact_gated_grad(s):
    """The two halves apart, each with its own products."""
    c = s["case"]
    n, x, w, d = c["n"], s["x"].double(), s["w"].double(), s["dh"].double()
    if c["saved"]:
        a, b = s["pre"][:, :n].double(), s["pre"][:, n:].double()
    else:
        a, b = x @ w[:n].t(), x @ w[n:].t()
    f, df = _act64(a, c["gate"])
    da, db = d * b * df, d * f
    return {"dpre": torch.cat((da, db), 1), "dx": da @ w[:n] + db @ w[n:],
            "dw": torch.cat((da.t() @ x, db.t() @ x), 0)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"quant": _exact_quant, "i8": _exact_i8, "gated": _exact_gated, "gated_grad": _exact_gated_grad}[case["op"]](s)
