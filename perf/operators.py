"""Cases of the mixture-of-experts operators around the expert-ID products:

  topk, topk_grad            router: softmax over the experts, the top_k of each token
  sort, sort_grad            token rows in expert order, and the gradient back to the tokens
  combine, combine_grad      expert rows back to tokens with weights, and both gradients
  q4_gemv, q4_direct,        products with 4-bit weights and group scales: one matrix; one expert
  q4_sorted                  for each routed row; rows sorted by expert

With `own` false `run` computes each in plain torch operations in 32 bits,
rounded once; with `own` true it calls the library. Expert ids are int32, -1
for a slot without an expert (0xFFFFFFFF in the library).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CODE = {"f32": 0, "f16": 1, "bf16": 2}  # the library's dtype numbers


def listed():
    return [
        # One token's router at decode: latency alone counts.
        dict(name="topk_token", op="topk", m=1, experts=64, top_k=8, dtype="f32", renormalize=1, masked=0.0),
        # A long prompt through a wide router; a few experts are switched off with -inf.
        dict(name="topk_prompt", op="topk", m=16384, experts=256, top_k=8, dtype="bf16", renormalize=1, masked=0.05),
        # Training step of a router whose weights keep the softmax's own scale; odd expert count.
        dict(name="topk_grad", op="topk_grad", m=8191, experts=97, top_k=6, dtype="f32", renormalize=0, masked=0.0),
        # Four sequences decoding together: eight experts each.
        dict(name="sort_decode", op="sort", m=4, experts=64, top_k=8, width=2048, dtype="bf16", dropped=0.0),
        # The 512-token prefill of the 64-expert layer, f32 activations.
        dict(name="sort_prompt", op="sort", m=512, experts=64, top_k=8, width=2048, dtype="f32", dropped=0.0),
        # Backward of the sort on a ragged batch with slots dropped at capacity.
        dict(name="sort_grad", op="sort_grad", m=3001, experts=60, top_k=4, width=1408, dtype="f16", dropped=0.05),
        # Expert outputs back to a long prompt's tokens, onto the residual stream.
        dict(name="combine_prompt", op="combine", m=8192, experts=64, top_k=8, width=2048, dtype="bf16", dropped=0.0),
        # Training: gradients to the expert rows and to the router's weights; rows of odd length.
        dict(name="combine_grad", op="combine_grad", m=2048, experts=32, top_k=8, width=4095, dtype="bf16", dropped=0.02),
        # One token through one large projection.
        dict(name="q4_token", op="q4_gemv", m=1, n=11008, k=4096, group=128, dtype="f16", scales="f16", gated=0),
        # Thirteen sequences decoding together; odd output count.
        dict(name="q4_batch", op="q4_gemv", m=13, n=4099, k=4096, group=64, dtype="bf16", scales="bf16", gated=0),
        # Gate and up projections of one token's eight experts, gated in the epilogue.
        dict(name="q4_experts_token", op="q4_direct", m=1, experts=64, top_k=8, n=1408, k=2048, group=32, dtype="bf16", scales="bf16", gated=1),
        # Down projection of 64 decoding sequences' rows, sorted by expert; f32 as in the expert-ID matmul.
        dict(name="q4_experts_batch", op="q4_sorted", m=64, experts=64, top_k=8, n=2048, k=1408, group=64, dtype="f32", scales="f16", gated=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["topk", "topk_grad", "sort", "sort_grad", "combine", "combine_grad", "q4_gemv", "q4_direct", "q4_sorted"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("topk", "topk_grad"):
        experts = _log_int(rng, 8, 512)
        m = min(_log_int(rng, 1, 16384), (1 << 22) // experts)
        return dict(op=op, m=m, experts=experts, top_k=rng.randint(1, 8), dtype=dtype,
                    renormalize=rng.randint(0, 1), masked=rng.choice([0.0, 0.0, 0.05, 0.5]))
    experts = _log_int(rng, 8, 256)
    top_k = rng.randint(1, 8)
    if op in ("sort", "sort_grad", "combine", "combine_grad"):
        width = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            width = -(-width // 64) * 64
        # rows of at most 32 M elements, so no drawn case costs more than the listed ones
        m = min(_log_int(rng, 1, 8192), (1 << 25) // (width * top_k))
        return dict(op=op, m=m, experts=experts, top_k=top_k, width=width, dtype=dtype,
                    dropped=rng.choice([0.0, 0.0, 0.05, 0.5]))
    group = rng.choice([32, 64, 128])
    k = group * _log_int(rng, 512 // group, 8192 // group)
    scales = rng.choice(["f16", "bf16"])
    gated = rng.randint(0, 1)
    if op == "q4_gemv":
        n = min(_log_int(rng, 64, 16384), (48 << 20) // ((1 + gated) * k))
        return dict(op=op, m=_log_int(rng, 1, 64), n=n, k=k, group=group, dtype=dtype, scales=scales, gated=gated)
    experts = _log_int(rng, 8, 128)
    n = max(1, min(_log_int(rng, 64, 4096), (160 << 20) // ((1 + gated) * k * experts)))
    m = _log_int(rng, 1, 8) if op == "q4_direct" else _log_int(rng, 2, 64)
    return dict(op=op, m=m, experts=experts, top_k=top_k, n=n, k=k, group=group, dtype=dtype, scales=scales, gated=gated)


# ---- what a program holds before the call ------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _ids(g, m, experts, top_k, dropped):
    """Distinct experts for each token, some more popular than others; `dropped` of the slots hold none."""
    popular = torch.randn(experts, generator=g, device=DEV) * 0.5
    score = torch.randn(m, experts, generator=g, device=DEV) + popular
    ids = torch.sort(score, dim=1, descending=True).indices[:, :top_k].to(torch.int32)
    gone = torch.rand(m, top_k, generator=g, device=DEV) < dropped
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous()


def _plan(ids, experts):
    """Expert order of the routed rows: segment offsets, row at each place, place of each row."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), torch.full_like(flat, experts), flat)
    sorted_key, order = torch.sort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.searchsorted(sorted_key, torch.arange(experts + 1, device=order.device))
    return offsets.to(torch.int32), order.to(torch.int32), position.to(torch.int32)


def _quantised(g, experts, rows, k, group, scales):
    """Normal weights in 4-bit codes with a scale and a bias for each group: two codes a byte, the even one low."""
    w = torch.randn(experts, rows, k // group, group, generator=g, device=DEV) * 0.02
    lo, hi = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).to(DTYPES[scales])
    b = lo.to(DTYPES[scales])
    q = ((w - b.float()) / s.float()).round_().clamp_(0, 15).to(torch.uint8).reshape(experts, rows, k // 2, 2)
    return (q[..., 0] | (q[..., 1] << 4)).contiguous(), s[..., 0].contiguous(), b[..., 0].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    op, m, t = c["op"], c["m"], DTYPES[c["dtype"]]
    if op in ("topk", "topk_grad"):
        e, k = c["experts"], c["top_k"]
        logits = _randn(g, m, e, scale=1.5)
        logits[torch.rand(m, e, generator=g, device=DEV) < c["masked"]] = float("-inf")
        s["logits"] = logits.to(t)
        if op == "topk":
            s["ids"] = torch.empty(m, k, dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty(m, k, device=DEV)
        else:
            top = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
            ids = top.indices[:, :k].to(torch.int32)
            s["ids"] = torch.where(torch.isinf(top.values[:, :k]), torch.full_like(ids, -1), ids).contiguous()
            s["dweights"] = _randn(g, m, k)
            s["dlogits"] = torch.empty(m, e, dtype=t, device=DEV)
        return s
    if op in ("sort", "sort_grad", "combine", "combine_grad"):
        e, k, h = c["experts"], c["top_k"], c["width"]
        s["ids"] = _ids(g, m, e, k, c["dropped"])
        s["offsets"], s["order"], s["position"] = _plan(s["ids"], e)
        if op == "sort":
            s["x"] = _randn(g, m, h, dtype=t)
            s["xs"] = torch.empty(m * k, h, dtype=t, device=DEV)
            s["offsets"], s["order"], s["position"] = (torch.empty_like(v) for v in (s["offsets"], s["order"], s["position"]))
        elif op == "sort_grad":
            s["dxs"] = _randn(g, m * k, h, dtype=t)
            s["dx"] = torch.empty(m, h, dtype=t, device=DEV)
        else:
            s["y"] = _randn(g, m * k, h, dtype=t)
            s["weights"] = torch.softmax(torch.randn(m, k, generator=g, device=DEV), dim=1)
            if op == "combine":
                s["residual"] = _randn(g, m, h, dtype=t)
                s["out"] = torch.empty(m, h, dtype=t, device=DEV)
            else:
                s["dout"] = _randn(g, m, h, dtype=t)
                s["dy"] = torch.empty(m * k, h, dtype=t, device=DEV)
                s["dweights"] = torch.empty(m, k, device=DEV)
        return s
    e, k = c.get("experts", 1), c.get("top_k", 1)
    s["codes"], s["scales"], s["biases"] = _quantised(g, e, c["n"] * (1 + c["gated"]), c["k"], c["group"], c["scales"])
    rows = m * k
    if op != "q4_gemv":
        s["ids"] = _ids(g, m, e, k, 0.0)
    s["x"] = _randn(g, rows if op == "q4_sorted" else m, c["k"], dtype=t)
    if op == "q4_sorted":
        s["offsets"] = _plan(s["ids"], e)[0]
    s["y"] = torch.empty(rows, c["n"], dtype=t, device=DEV)
    return s


# ---- the plain forms -----------------------------------------------------------


def _plain_topk(s):
    c, l = s["case"], s["logits"].float()
    top = torch.sort(l, dim=1, descending=True, stable=True)
    values, ids = top.values[:, : c["top_k"]], top.indices[:, : c["top_k"]].to(torch.int32)
    gone = torch.isneginf(values)
    peak = values[:, :1].masked_fill(gone[:, :1], 0.0)
    w = torch.exp(values - peak)
    total = w.sum(1, keepdim=True) if c["renormalize"] else torch.exp(l - peak).sum(1, keepdim=True)
    w = torch.where(gone, torch.zeros_like(w), w / total)
    return {"ids": ids.masked_fill(gone, -1), "weights": w}


def _plain_topk_grad(s):
    c, l, g = s["case"], s["logits"].float(), s["dweights"]
    gone = s["ids"] < 0
    at = s["ids"].masked_fill(gone, 0).long()
    g = g.masked_fill(gone, 0.0)
    full = torch.zeros_like(l).scatter_add_(1, at, g)
    if c["renormalize"]:
        picked = torch.zeros_like(l).scatter_add_(1, at, (~gone).float()) > 0
        l = l.masked_fill(~picked, float("-inf"))
    peak = l.amax(1, keepdim=True)
    e = torch.exp(l - peak.masked_fill(torch.isneginf(peak), 0.0))
    p = e / e.sum(1, keepdim=True).clamp_min(1e-30)
    return {"dlogits": (p * (full - (p * full).sum(1, keepdim=True))).to(s["logits"].dtype)}


def _plain_sort(s):
    c = s["case"]
    offsets, order, position = _plan(s["ids"], c["experts"])
    rows = s["x"][(order // c["top_k"]).long()]
    live = torch.arange(rows.shape[0], device=rows.device) < offsets[-1]
    xs = torch.where(live[:, None], rows, torch.zeros_like(rows))
    return {"xs": xs, "offsets": offsets, "order": order, "position": position}


def _token_rows(rows, s):
    """[m, top_k, width] rows of each token in 32 bits, zeros where a slot has no expert; and which slots have one."""
    c = s["case"]
    live = (s["position"] < s["offsets"][-1]).reshape(c["m"], c["top_k"])
    got = rows[s["position"].long()].float().reshape(c["m"], c["top_k"], -1)
    return torch.where(live[..., None], got, torch.zeros_like(got)), live


def _plain_sort_grad(s):
    return {"dx": _token_rows(s["dxs"], s)[0].sum(1).to(s["dxs"].dtype)}


def _plain_combine(s):
    rows, live = _token_rows(s["y"], s)
    out = (rows * s["weights"].masked_fill(~live, 0.0)[..., None]).sum(1) + s["residual"].float()
    return {"out": out.to(s["y"].dtype)}


def _plain_combine_grad(s):
    rows, live = _token_rows(s["y"], s)
    d = s["dout"].float()[:, None, :]
    dy = (d * s["weights"].masked_fill(~live, 0.0)[..., None]).to(s["y"].dtype).reshape(s["y"].shape)
    return {"dy": dy[s["order"].long()], "dweights": (d * rows).sum(-1)}


def _dequantised(codes, scales, biases, group):
    q = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*codes.shape[:-1], -1, group)
    w = q.float() * scales.float()[..., None] + biases.float()[..., None]
    return w.reshape(*codes.shape[:-1], -1)


def _gate(y, c):
    if not c["gated"]:
        return y
    a, b = y[..., : c["n"]], y[..., c["n"]:]
    return a / (1 + torch.exp(-a)) * b


def _plain_q4_gemv(s):
    c = s["case"]
    w = _dequantised(s["codes"][0], s["scales"][0], s["biases"][0], c["group"])
    return {"y": _gate(s["x"].float() @ w.t(), c).to(s["x"].dtype)}


def _plain_q4_direct(s):
    c = s["case"]
    at = s["ids"].reshape(-1).long()
    w = _dequantised(s["codes"][at], s["scales"][at], s["biases"][at], c["group"])
    x = s["x"].float().repeat_interleave(c["top_k"], 0)
    return {"y": _gate(torch.bmm(w, x[:, :, None])[..., 0], c).to(s["x"].dtype)}


def _plain_q4_sorted(s):
    c = s["case"]
    rows = torch.arange(s["x"].shape[0], device=DEV)
    off = s["offsets"].long()
    e = torch.searchsorted(off[1:], rows, right=True)
    at = rows - off[e]
    x = torch.zeros(c["experts"], c["m"], c["k"], device=DEV)
    x[e, at] = s["x"].float()
    w = _dequantised(s["codes"], s["scales"], s["biases"], c["group"])
    return {"y": _gate(torch.bmm(x, w.transpose(1, 2))[e, at], c).to(s["x"].dtype)}


PLAIN = {"topk": _plain_topk, "topk_grad": _plain_topk_grad, "sort": _plain_sort, "sort_grad": _plain_sort_grad,
         "combine": _plain_combine, "combine_grad": _plain_combine_grad, "q4_gemv": _plain_q4_gemv,
         "q4_direct": _plain_q4_direct, "q4_sorted": _plain_q4_sorted}


# ---- the library's calls ---------------------------------------------------------


def _call(s):
    """The library entry point, the descriptor and the buffers of a state, as a serving loop keeps them, and the outputs."""
    import gemv_expert_id_amd as mm

    c = s["case"]
    op, dt = c["op"], CODE[c["dtype"]]
    buf = lambda *names: [mm.buf(s[n]) for n in names]  # noqa: E731
    if op in ("topk", "topk_grad"):
        p = mm.topk_params(dt, c["m"], c["experts"], c["top_k"], renormalize=c["renormalize"])
        if op == "topk":
            return mm.mm_topk, p, buf("logits", "ids", "weights"), {n: s[n] for n in ("ids", "weights")}
        return mm.mm_topk_grad, p, buf("logits", "ids", "dweights", "dlogits"), {"dlogits": s["dlogits"]}
    if op in ("sort", "sort_grad", "combine", "combine_grad"):
        p = mm.sort_params(dt, c["m"], c["top_k"], c["experts"], c["width"])
        if op == "sort":
            return (mm.mm_id_sort, p, buf("x", "ids", "xs", "offsets", "order", "position"),
                    {n: s[n] for n in ("xs", "offsets", "order", "position")})
        if op == "sort_grad":
            return mm.mm_id_sort_grad, p, buf("dxs", "offsets", "position", "dx"), {"dx": s["dx"]}
        if op == "combine":
            return (mm.mm_id_combine, p, buf("y", "offsets", "position", "weights", "residual", "out"),
                    {"out": s["out"]})
        return (mm.mm_id_combine_grad, p, buf("dout", "y", "offsets", "position", "weights", "dy", "dweights"),
                {n: s[n] for n in ("dy", "dweights")})
    p = mm.q4_params(dt, CODE[c["scales"]], c["m"], c["n"], c["k"], c["group"], n_experts=c.get("experts", 1),
                     top_k=c.get("top_k", 1), gated=c["gated"])
    if op == "q4_gemv":
        return mm.mm_q4_gemv, p, buf("codes", "scales", "biases", "x", "y"), {"y": s["y"]}
    if op == "q4_direct":
        return mm.mm_q4_id_direct, p, buf("codes", "scales", "biases", "x", "ids", "y"), {"y": s["y"]}
    return mm.mm_q4_id_sorted, p, buf("codes", "scales", "biases", "x", "offsets", "y"), {"y": s["y"]}


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
    op, m, z = c["op"], c["m"], SIZE[c["dtype"]]
    if op in ("topk", "topk_grad"):
        cells, slots = m * c["experts"], m * c["top_k"]
        if op == "topk":
            return {"bytes": cells * z + slots * 8, "flops": 4 * cells}
        return {"bytes": 2 * cells * z + slots * 8, "flops": 6 * cells}
    if op in ("sort", "sort_grad", "combine", "combine_grad"):
        h, rows = c["width"], m * c["top_k"]
        live = rows * (1 - c["dropped"])
        plan = rows * 4 + (c["experts"] + 1) * 4
        if op == "sort":
            return {"bytes": (m + rows) * h * z + plan + rows * 8, "flops": 0}
        if op == "sort_grad":
            return {"bytes": (m + live) * h * z + plan, "flops": live * h}
        if op == "combine":
            return {"bytes": (2 * m + live) * h * z + plan + rows * 4, "flops": 2 * live * h}
        return {"bytes": (m + live + rows) * h * z + plan + rows * 8, "flops": 3 * live * h}
    e, t = c.get("experts", 1), c.get("top_k", 1)
    matrices = 1.0 if e == 1 else e * (1 - (1 - t / e) ** m)  # experts that a pass meets
    n = c["n"] * (1 + c["gated"])
    rows = m * t
    weights = matrices * n * (c["k"] // 2 + c["k"] // c["group"] * 4)
    x = (rows if op == "q4_sorted" else m) * c["k"] * z
    return {"bytes": weights + x + rows * c["n"] * z, "flops": 2 * rows * n * c["k"]}


# ---- the definitions in 64 bits ------------------------------------------------------


def _exact_topk(s):
    c, l = s["case"], s["logits"].double().cpu()
    ids = torch.full((c["m"], c["top_k"]), -1, dtype=torch.int32)
    w = torch.zeros(c["m"], c["top_k"], dtype=torch.float64)
    rest, rows = l.clone(), torch.arange(c["m"])
    for k in range(c["top_k"]):  # the largest left, the lowest index of equal ones
        best = rest.max(1).values
        at = (rest == best[:, None]).to(torch.uint8).argmax(1)
        ok = best > float("-inf")
        ids[ok, k] = at[ok].to(torch.int32)
        w[ok, k] = best[ok]
        rest[rows, at] = float("-inf")
    live = ids >= 0
    base = torch.logsumexp(l, 1)
    if c["renormalize"]:
        base = torch.logsumexp(torch.where(live, w, torch.full_like(w, float("-inf"))), 1)
    return {"ids": ids, "weights": torch.where(live, torch.exp(w - base[:, None]), torch.zeros_like(w))}


def _exact_topk_grad(s):
    """Through the derivative of log-sum-exp: dl = dw . w (delta - w')."""
    c, l = s["case"], s["logits"].double()
    ids, g = s["ids"].long(), s["dweights"].double()
    out = torch.zeros_like(l)
    live = ids >= 0
    at = ids.clamp_min(0)
    z = torch.gather(l, 1, at).masked_fill(~live, float("-inf"))
    some = live.any(1)
    base = torch.logsumexp(z if c["renormalize"] else l, 1, keepdim=True)
    w = torch.where(live, torch.exp(z - base), torch.zeros_like(z))
    gw = torch.where(live, g * w, torch.zeros_like(w))
    total = gw.sum(1, keepdim=True)
    if c["renormalize"]:
        out.scatter_add_(1, at, torch.where(live, -w * total, torch.zeros_like(w)))
    else:
        out = torch.where(some[:, None], -torch.exp(l - base) * total, out)
    return {"dlogits": out.scatter_add_(1, at, gw)}


def _exact_plan(s):
    c = s["case"]
    flat = s["ids"].reshape(-1).long().cpu()
    parts = [torch.nonzero(flat == e).reshape(-1) for e in range(c["experts"])]
    parts.append(torch.nonzero((flat < 0) | (flat >= c["experts"])).reshape(-1))
    order = torch.cat(parts)
    offsets = torch.tensor([0] + [len(p) for p in parts[:-1]]).cumsum(0)
    position = torch.empty_like(order)
    for i, r in enumerate(order.tolist()):
        position[r] = i
    return offsets, order, position, order[: int(offsets[-1])].to(DEV)


def _exact_rows(s):
    """sort, combine and their gradients: through the list of live rows, in expert order."""
    c = s["case"]
    op, k = c["op"], c["top_k"]
    offsets, order, position, live = _exact_plan(s)
    n, token = live.numel(), live // k
    if op == "sort":
        xs = torch.zeros(c["m"] * k, c["width"], dtype=torch.float64, device=DEV)
        xs[:n] = s["x"].double()[token]
        return {"xs": xs, "offsets": offsets.to(torch.int32), "order": order.to(torch.int32), "position": position.to(torch.int32)}
    if op == "sort_grad":
        dx = torch.zeros(c["m"], c["width"], dtype=torch.float64, device=DEV)
        return {"dx": dx.index_add_(0, token, s["dxs"][:n].double())}
    w = s["weights"].reshape(-1)[live].double()[:, None]
    if op == "combine":
        return {"out": s["residual"].double().index_add_(0, token, s["y"][:n].double() * w)}
    d = s["dout"].double()[token]
    dy = torch.zeros(c["m"] * k, c["width"], dtype=torch.float64, device=DEV)
    dy[:n] = d * w
    dw = torch.zeros(c["m"] * k, dtype=torch.float64, device=DEV)
    dw[live] = (d * s["y"][:n].double()).sum(1)
    return {"dy": dy, "dweights": dw.reshape(c["m"], k)}


def _exact_q4(s):
    """One expert after another: x . (s q + b) as s (x . q) + b sum(x), group by group."""
    c = s["case"]
    op, e, k, g = c["op"], c.get("experts", 1), c["k"], c["group"]
    rows = c["m"] * c.get("top_k", 1)
    if op == "q4_gemv":
        of = torch.zeros(rows, dtype=torch.long, device=DEV)
        x = s["x"].double()
    elif op == "q4_direct":
        of = s["ids"].reshape(-1).long()
        x = s["x"].double()[torch.arange(rows, device=DEV) // c["top_k"]]
    else:
        of = torch.repeat_interleave(torch.arange(e, device=DEV), torch.diff(s["offsets"].long()))
        x = s["x"].double()
    y = torch.zeros(rows, c["n"], dtype=torch.float64, device=DEV)
    for i in range(e):
        at = torch.nonzero(of == i).reshape(-1)
        if not at.numel():
            continue
        q = torch.empty(s["codes"].shape[1], k, dtype=torch.float64, device=DEV)
        q[:, 0::2] = (s["codes"][i] % 16).double()
        q[:, 1::2] = (s["codes"][i] // 16).double()
        xi = x[at].reshape(len(at), k // g, g)
        dot = torch.bmm(xi.transpose(0, 1).contiguous(), q.reshape(-1, k // g, g).permute(1, 2, 0).contiguous())
        z = (dot * s["scales"][i].double().t()[:, None, :]).sum(0) + xi.sum(-1) @ s["biases"][i].double().t()
        if c["gated"]:
            z = z[:, : c["n"]] * torch.sigmoid(z[:, : c["n"]]) * z[:, c["n"]:]
        y[at] = z
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "topk":
        return _exact_topk(s)
    if op == "topk_grad":
        return _exact_topk_grad(s)
    return _exact_q4(s) if op.startswith("q4") else _exact_rows(s)
