"""Plain definitions in 64 bits of the router, the sorted rows and the 4-bit
products, for the tests: loops over tokens and experts on the CPU, written from
the formulas in include/mm.h."""
from __future__ import annotations

import numpy as np
import torch

NONE = 0xFFFFFFFF
TORCH = {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}
U = 2.0 ** -24  # half a step of f32, relative


def half_step(dtype: int) -> float:
    return torch.finfo(TORCH[dtype]).eps / 2


def rounding(dtype: int, value):
    """Half a step of `value` in the type; a value below the smallest normal
    number has the step of that number."""
    return half_step(dtype) * np.maximum(np.abs(value), torch.finfo(TORCH[dtype]).tiny)


def topk(logits: np.ndarray, k: int, renormalize: bool):
    """ids u32 [m, k], weights f64 [m, k] of f64 logits."""
    m, _ = logits.shape
    ids = np.full((m, k), NONE, dtype=np.uint32)
    w = np.zeros((m, k))
    with np.errstate(invalid="ignore"):
        for t in range(m):
            row = logits[t]
            can = [e for e in range(row.size) if row[e] > -np.inf]
            pick = sorted(can, key=lambda e: (-row[e], e))[:k]
            ids[t, :len(pick)] = pick
            if not pick:
                continue
            peak = row[pick[0]]
            over = row[pick] if renormalize else row[~(row == -np.inf)]
            total = np.exp(over - peak).sum()
            w[t, :len(pick)] = np.exp(row[pick] - peak) / total
            if np.isnan(row).any():
                w[t, :len(pick)] = np.nan
    return ids, w


def topk_grad(logits: np.ndarray, ids: np.ndarray, g: np.ndarray, renormalize: bool):
    m, E = logits.shape
    out = np.zeros((m, E))
    for t in range(m):
        live = [s for s in range(ids.shape[1]) if ids[t, s] < E]
        if not live:
            continue
        chosen = ids[t, live]
        z = np.full(E, -np.inf)
        if renormalize:
            z[chosen] = logits[t, chosen]
        else:
            z = logits[t].copy()
        p = np.exp(z - z.max())
        p /= p.sum()
        full = np.zeros(E)
        full[chosen] = g[t, live]
        out[t] = p * (full - (full * p).sum())
    return out


def plan(ids: np.ndarray, E: int):
    """offsets, order, position of the stable sort by expert."""
    flat = ids.reshape(-1).astype(np.int64)
    key = [int(v) if v < E else E for v in flat]
    order = sorted(range(len(key)), key=lambda r: (key[r], r))
    offsets = [sum(1 for v in key if v < e) for e in range(E + 1)]
    position = np.zeros(len(key), dtype=np.uint32)
    for i, r in enumerate(order):
        position[r] = i
    return (np.array(offsets, dtype=np.uint32), np.array(order, dtype=np.uint32), position)


def combine(y: np.ndarray, live: int, position: np.ndarray, w: np.ndarray, residual):
    """f64 out [m, h], and the sum of the magnitudes added."""
    m, k = w.shape
    out = np.zeros((m, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    mag = np.abs(out)
    for t in range(m):
        for s in range(k):
            i = int(position[t * k + s])
            if i < live:
                out[t] += w[t, s] * y[i]
                mag[t] += np.abs(w[t, s] * y[i])
    return out, mag


def combine_grad(dout: np.ndarray, y: np.ndarray, live: int, position: np.ndarray, w: np.ndarray):
    """dy, dweights, and the magnitudes added into dweights."""
    m, k = w.shape
    dy = np.zeros_like(y, dtype=np.float64)
    dw, mag = np.zeros((m, k)), np.zeros((m, k))
    for t in range(m):
        for s in range(k):
            i = int(position[t * k + s])
            if i < live:
                dy[i] = w[t, s] * dout[t]
                dw[t, s] = (dout[t] * y[i]).sum()
                mag[t, s] = np.abs(dout[t] * y[i]).sum()
    return dy, dw, mag


def q4_weights(codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, group: int):
    """f64 [.., N, k] of codes u8 [.., N, k/2]."""
    c = codes.cpu().to(torch.int64)
    q = torch.stack((c % 16, c // 16), dim=-1).reshape(*c.shape[:-1], -1).double()
    s = scales.cpu().double().repeat_interleave(group, -1)
    b = biases.cpu().double().repeat_interleave(group, -1)
    return q * s + b


def q4_product(codes, scales, biases, group: int, x: torch.Tensor, gated: bool, f32_parts: bool):
    """f64 y [rows, n] of one expert, and a bound on the error of its sums in
    32 bits. The kernel forms, group by group, (16 + q) . x and 16 . x and adds
    their scaled values: each magnitude below is what is added, and each
    addition of the chain (a matrix instruction adds 32 products, counted as 32
    additions; f32 activations are three parts, so three times as many) rounds
    by at most 2^-24 of it."""
    w = q4_weights(codes, scales, biases, group)
    xd = x.cpu().double()
    y = xd @ w.t()
    s = scales.cpu().double().abs().repeat_interleave(group, -1)
    b = biases.cpu().double().abs().repeat_interleave(group, -1)
    mag = xd.abs() @ (47 * s + b).t()
    k = xd.shape[1]
    err = mag * (2.0 ** -24) * ((2 * group + 8) * (3 if f32_parts else 1) + 2 * (k // group) + 8)
    if not gated:
        return y, err
    n = y.shape[1] // 2
    g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    silu = g * torch.sigmoid(g)
    # |silu'| < 1.1; exp, the division and two products: a few steps of the result
    return silu * u, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 16 * 2.0 ** -24 * (silu * u).abs()
