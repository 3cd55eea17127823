"""Plain 64-bit forms of the prompt and decay-rule operators (test code)."""
from __future__ import annotations

import numpy as np
import torch

import oracle as O

EPS32 = 2.0 ** -24          # half a step of FP32, relative
EPS_BF16 = 2.0 ** -8        # half a step of bf16, relative


def recurrence(rule, q, k, v, alpha, beta, S0):
    """One request and all its heads, token by token in float64.  q, k
    [L][Hqk][dk], v [L][H][dv], alpha, beta [L][H], S0 [H][dk][dv].  Returns
    (out [L][H][dv], S, the largest Frobenius norm a head's state (or one
    token's k v^T) reached [H])."""
    f8 = torch.float64
    L, H = v.shape[0], v.shape[1]
    rep = lambda x: x.to(f8).repeat_interleave(H // x.shape[1], dim=1)  # noqa: E731
    q, k, v, alpha = rep(q), rep(k), v.to(f8), alpha.to(f8)
    S = S0.to(f8).clone()
    out = torch.zeros(L, H, v.shape[2], dtype=f8, device=v.device)
    top = S.flatten(1).norm(dim=1)
    for t in range(L):
        S = alpha[t][:, None, None] * S
        d = v[t]
        if rule == "delta":
            d = beta[t].to(f8)[:, None] * (d - torch.einsum("hk,hkv->hv", k[t], S))
        add = k[t][:, :, None] * d[:, None, :]
        S = S + add
        out[t] = torch.einsum("hk,hkv->hv", q[t], S)
        top = torch.maximum(top, torch.maximum(S.flatten(1).norm(dim=1), add.flatten(1).norm(dim=1)))
    return out, S, top


def inputs(g, T, H, Hqk, dk, dv, dtype, device="cuda", unit=True):
    """Seeded prompt tensors (CPU generator, so that every device sees the same)."""
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = r(T, Hqk, dk), r(T, Hqk, dk), r(T, H, dv)
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    half = torch.exp(torch.rand(H, generator=g) * np.log(512.0))
    alpha = torch.exp(-torch.nn.functional.softplus(r(T, H)) / half)
    beta = torch.sigmoid(r(T, H))
    cv = lambda x: x.to(dtype).to(device)  # noqa: E731
    return dict(q=cv(q), k=cv(k), v=cv(v), alpha=alpha.to(device), beta=beta.to(device))


def decay_step(fmt, is_fp16, st: O.State, q, k, v, alpha):
    """The decay rule on unpacked oracle states, with its FP32 roundings; all
    arrays for one batch: st over [n][H], q, k [n][H][dk], v [n][H][dv], alpha
    [n][H].  Returns (out float64 [n][H][dv], requantized State)."""
    S = O.unpack(st, is_fp16).astype(np.float32)
    Sp = (alpha[..., None, None].astype(np.float32) * S).astype(np.float32)
    # fl(k v + S'): the product of two float32 values is exact in float64
    X = (k[..., None].astype(np.float64) * v[..., None, :].astype(np.float64)
         + Sp.astype(np.float64)).astype(np.float32)
    out = (q[..., None].astype(np.float64) * X.astype(np.float64)).sum(axis=-2)
    return out, O.pack(fmt, is_fp16, X), X
