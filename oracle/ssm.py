"""Plain 64-bit form of the state space layer's operators (convolution, selective scan, gated norm),
token by token on the CPU, and how far a 32-bit evaluation may be from it.

It shares no code with the CUDA path.  ``scan`` also returns bounds on the error of y and S that follow
from the roundings of one token's update: with u = 2^-24 (half a step of fp32),
  - d = softplus(v), v = dt + bias: rounding v moves d by up to u |v| softplus'(v) = u |v| sigmoid(v) (for v far below zero,
    where softplus is the exponential, that is |v| u of d itself), and max, exp, log1p and the sum after them are each off
    by a few u: e = u (|v| sigmoid(v) + 8 d); without the softplus u |v|; where a limit is taken instead, u of that
    limit, which is a 32-bit number;
  - a = exp(d A): |A| e from d and u |d A| from the product, 2 u of the exp: (|A| e + u (2 + |d A|)) a;
  - S' = a S + (d B) x: three more roundings of products and one of the sum.
So E' = a E + (|A| e + u (4 + |d A|)) a |S| + (e + 4 u d) |B||x| + u |S'| bounds the state's error, where |S| is the
state made of absolute values; y adds |C| E, N + 2 roundings of the sum over n, and 2 of D x.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24


def _d(t):
    return None if t is None else t.detach().cpu().double()


def step_sizes(dt, bias, softplus=True, lo=0.0, hi=float("inf")):
    v = _d(dt) + (0 if bias is None else _d(bias))
    if softplus:
        v = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    return torch.clamp(v, lo, hi)


def step_errors(dt, bias, softplus=True, lo=0.0, hi=float("inf")):
    """The bound e of above on the error of a step size in 32 bits."""
    v = _d(dt) + (0 if bias is None else _d(bias))
    if softplus:
        d = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
        e = U32 * (v.abs() * torch.sigmoid(v) + 8 * d)
    else:
        d, e = v, U32 * v.abs()
    limited = torch.clamp(d, lo, hi)
    return torch.where((d < lo - e) | (d > hi + e), U32 * limited.abs(), torch.maximum(e, U32 * limited.abs()))


def scan(x, dt, A, Bm, Cm, D=None, dt_bias=None, lengths=None, S_in=None, softplus=True, dt_min=0.0, dt_max=float("inf")):
    """y [B,T,H,P] (zeros behind a sequence), S [B,H,N,P], the sums of absolute values behind y, and the bounds
    (y, S) of the 32-bit errors described above."""
    x, Bm, Cm, A = _d(x), _d(Bm), _d(Cm), _d(A)
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    d = step_sizes(dt, dt_bias, softplus, dt_min, dt_max)
    e = step_errors(dt, dt_bias, softplus, dt_min, dt_max)
    D = torch.zeros(H, dtype=torch.float64) if D is None else _d(D)
    Bm, Cm = Bm.repeat_interleave(H // G, 2), Cm.repeat_interleave(H // G, 2)
    y, ya, ye = (torch.zeros((B, T, H, P), dtype=torch.float64) for _ in range(3))
    S = torch.zeros((B, H, N, P), dtype=torch.float64) if S_in is None else _d(S_in).clone()
    Sa, E = S.abs(), torch.zeros_like(S)
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for t in range(n):
            dA = (d[b, t] * A)[:, None, None]
            a = torch.exp(dA)
            bx = Bm[b, t][:, :, None] * x[b, t, :, None, :]
            w, ed = d[b, t][:, None, None] * bx, e[b, t][:, None, None]
            # (a decay of 0 has no error, however large |A|)
            E[b] = a * E[b] + torch.where(a > 0, A.abs()[:, None, None] * ed + U32 * (4 + dA.abs()), 0.0) * a * Sa[b]
            E[b] += (ed + 4 * U32 * d[b, t][:, None, None]) * bx.abs()
            S[b] = a * S[b] + w
            Sa[b] = a * Sa[b] + w.abs()
            E[b] += U32 * Sa[b]
            c = Cm[b, t, :, :, None]
            skip = D[:, None] * x[b, t]
            y[b, t] = (c * S[b]).sum(1) + skip
            ya[b, t] = (c.abs() * Sa[b]).sum(1) + skip.abs()
            ye[b, t] = (c.abs() * E[b]).sum(1) + U32 * (N + 4) * ya[b, t]
    return y, S, ya, ye, E


def conv(x, w, bias=None, silu=True, lengths=None, state_in=None):
    """y [B,T,C] (zeros behind a sequence), the kept inputs [B,W-1,C], and the sums of absolute values."""
    x, w = _d(x), _d(w)
    B, T, C = x.shape
    W = w.shape[1]
    bias = torch.zeros(C, dtype=torch.float64) if bias is None else _d(bias)
    state = torch.zeros((B, W - 1, C), dtype=torch.float64) if state_in is None else _d(state_in)
    y, ya = torch.zeros_like(x), torch.zeros_like(x)
    kept = torch.zeros_like(state)
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        full = torch.cat([state[b], x[b, :n]])
        kept[b] = full[n:]
        for t in range(n):
            v = bias + sum(w[:, k] * full[t + k] for k in range(W))
            ya[b, t] = bias.abs() + sum((w[:, k] * full[t + k]).abs() for k in range(W))
            y[b, t] = v * torch.sigmoid(v) if silu else v
    return y, kept, ya


def norm_gate(x, z=None, w=None, groups=1, eps=1e-6, gate_first=True):
    x, z, w = _d(x), _d(z), _d(w)
    gate = 1.0 if z is None else z * torch.sigmoid(z)
    u = x * gate if gate_first else x
    v = u.reshape(x.shape[0], groups, -1)
    v = (v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + eps)).reshape(x.shape)
    v = v if w is None else v * w
    return v if gate_first else v * gate
