"""The layer operators from their definitions, in 64 bits on the CPU: token by token
for the gated delta rule, row by row for the norms.  Shares no code with the CUDA
library or with the solver's oracle."""
from __future__ import annotations

import numpy as np


def delta_rule(q, k, v, g, beta, S, scale):
    """One sequence.  q, k [T, Hk, K]; v [T, H, V]; g [T, H, K] or [T, H]; beta [T, H];
    S [H, K, V].  Returns (o [T, H, V], the final states); S is not written."""
    H = v.shape[1]
    of = np.arange(H) // (H // q.shape[1])
    S = np.array(S, np.float64)
    o = np.zeros(v.shape, np.float64)
    for t in range(v.shape[0]):
        gt = g[t] if g.ndim == 3 else g[t][:, None]
        S = S * np.exp(gt)[:, :, None]
        kt, qt = k[t][of], q[t][of]
        u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, kt))
        S = S + kt[:, :, None] * u[:, None, :]
        o[t] = scale * np.einsum("hkv,hk->hv", S, qt)
    return o, S


def add_norm(x, residual, weight, alpha, eps):
    r = alpha * x + (0.0 if residual is None else residual)
    return r / np.sqrt(np.mean(r * r, -1, keepdims=True) + eps) * weight, r


def gated_norm(x, gate, weight, eps, activation):
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * weight / (1 + np.exp(-gate))
    return y * gate if activation == "silu" else y
