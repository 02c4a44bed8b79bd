"""The error bounds of oracle/ssm.py against 32-bit evaluations on the CPU (numpy, one rounding per operation)."""
import numpy as np
import pytest
import torch

from oracle import ssm as plain

U32 = 2.0 ** -24


def _step_sizes32(dt, bias, softplus, lo, hi):
    """The step sizes as the kernels take them: sum, exp and log1p in 32 bits."""
    v = dt + bias
    if softplus:
        v = np.maximum(v, np.float32(0)) + np.log1p(np.exp(-np.abs(v)))
    return np.clip(v, np.float32(lo), np.float32(hi))


@pytest.mark.parametrize("softplus,lo,hi", [(True, 0.0, np.inf), (True, 0.001, 0.1), (False, 0.0, np.inf), (False, -1.0, 0.5)])
def test_bound_on_step_sizes_holds(softplus, lo, hi):
    rng = np.random.default_rng(0)
    bias = rng.uniform(-24, 8, 400000).astype(np.float32)
    dt = rng.normal(0, 1.5, bias.size).astype(np.float32)
    d32 = _step_sizes32(dt, bias, softplus, lo, hi).astype(np.float64)
    args = (torch.from_numpy(dt), torch.from_numpy(bias), softplus, lo, hi)
    d = plain.step_sizes(*args).numpy()
    e = plain.step_errors(*args).numpy()
    assert np.all(np.abs(d32 - d) <= e)
    # and is no wider than the step size's own conditioning: 24 u of the value within 16 of zero
    near = np.abs(dt + bias) < 16
    assert np.all(e[near] <= 24 * U32 * np.maximum(np.abs(d[near]), np.abs(dt + bias)[near] if not softplus else 0) + 1e-30)


def _scan32(x, dt, A, Bm, Cm, D, bias, n_tokens):
    S = np.zeros((Bm.shape[-1], x.shape[-1]), np.float32)
    ys = []
    for t in range(n_tokens):
        d = _step_sizes32(dt[t], bias, True, 0.0, np.inf)
        a = np.exp(np.float32(d * A))
        S = a * S + (d * Bm[t])[:, None] * x[t][None, :]
        y = np.zeros(x.shape[-1], np.float32)
        for k in range(S.shape[0]):
            y = y + Cm[t, k] * S[k]
        ys.append(y + D * x[t])
    return np.stack(ys), S


@pytest.mark.parametrize("bias", [-14.0, -9.0, -4.0, 1.0])
def test_bounds_on_scan_hold(bias):
    rng = np.random.default_rng(1)
    T, N, P = 200, 16, 8
    f = lambda *s: rng.normal(0, 1, s).astype(np.float32)  # noqa: E731
    x, dt, Bm, Cm = f(T, P), f(T), f(T, N), f(T, N)
    A, D, bias = np.float32(-3.0), np.float32(0.7), np.float32(bias)
    y32, S32 = _scan32(x, dt, A, Bm, Cm, D, bias, T)
    t = lambda v: torch.from_numpy(np.asarray(v, np.float32))  # noqa: E731
    y, S, _, ye, E = plain.scan(t(x)[None, :, None], t(dt)[None, :, None], t([A]), t(Bm)[None, :, None], t(Cm)[None, :, None], t([D]), t([bias]))
    assert np.all(np.abs(S32 - S[0, 0].numpy()) <= E[0, 0].numpy())
    assert np.all(np.abs(y32 - y[0, :, 0].numpy()) <= ye[0, :, 0].numpy())
