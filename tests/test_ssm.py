"""State space layer on the GPU (through the C ABI) against the plain 64-bit form in oracle/ssm.py.

Tolerances are bounds, element by element:
  - fp32 roundings of the scan: the bound the oracle carries along with the recurrence;
  - prompts with bf16 inputs and output meet the state and the token-to-token weights as two bf16 pieces each (2^-16),
    and sum up to 64 tokens at once (64 u, 2^-18): together at most 2^-15 of the sum of absolute values;
  - one rounding to the output's type: half a step, eps / 2 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import ssm as plain
from sparse_slot_recurrent_b200 import ramnet

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ramnet.load()
    yield
    ramnet.sync_status()


def _half_step(v, dtype):
    return v.abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).tiny


def _near(got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    assert bool(torch.isfinite(got).all())
    off = (got - want).abs() - tol
    assert float(off.max()) <= 0, f"off by up to {float((got - want).abs().max()):.3g}, {float(off.max()):.3g} over the bound"


def _layer(B, T, H, G, N, P, dtype, seed=0, dt_hi=0.1):
    """A layer's operands as a user has them: x, B and C are slices of one convolution output."""
    g = torch.Generator().manual_seed(seed)
    xbc = torch.nn.functional.silu(torch.randn((B, T, H * P + 2 * G * N), generator=g)).to(dtype).cuda()
    x = xbc[..., :H * P].unflatten(-1, (H, P))
    Bm = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    Cm = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
    base = torch.exp(torch.rand((H,), generator=g) * float(np.log(dt_hi / 1e-3)) + float(np.log(1e-3)))
    return dict(x=x, dt=(0.5 * torch.randn((B, T, H), generator=g)).to(dtype).cuda(),
                A=-(1 + 15 * torch.rand((H,), generator=g)).cuda(), Bm=Bm, Cm=Cm,
                D=(torch.rand((H,), generator=g) + 0.5).cuda(), dt_bias=torch.log(torch.expm1(base)).cuda())


def _scan_tols(y, ya, ye, E, S, out_dtype, split, Sa_bound=None):
    ty = ye + _half_step(y, out_dtype) + (2.0 ** -15 * ya if split else 0)
    # blocks of 64 tokens are summed at once: 64 more roundings than token by token
    tS = E + (64 * U32 * S.abs().amax(dim=(2, 3), keepdim=True) if split else 0) + 1e-30
    return ty, tS


def _check_scan(cfg, L, lengths=None, S_in=None, out_dtype=None, **kw):
    y, S = ramnet.ssm_forward(cfg, **L, lengths=lengths, S_in=S_in, out_dtype=out_dtype, **kw)
    ramnet.sync_status()
    wy, wS, ya, ye, E = plain.scan(**L, lengths=lengths, S_in=S_in, softplus=cfg.dt_softplus, dt_min=cfg.dt_min,
                                   dt_max=cfg.dt_max)
    split = L["x"].dtype == BF and y.dtype == BF
    ty, tS = _scan_tols(wy, ya, ye, E, wS, y.dtype, split)
    for b in range(y.shape[0]):
        n = y.shape[1] if lengths is None else min(max(int(lengths[b]), 0), y.shape[1])
        if n:
            _near(y[b, :n], wy[b, :n], ty[b, :n])
    _near(S, wS, tS)
    return y, S


SHAPES = [
    # B, T, H, G, N, P
    (1, 1, 1, 1, 16, 16),
    (2, 63, 2, 1, 64, 64),
    (1, 64, 4, 2, 128, 64),
    (1, 65, 2, 1, 128, 128),
    (2, 129, 3, 3, 32, 32),
    (1, 200, 5, 1, 64, 32),
    (1, 97, 3, 1, 128, 16),
    (1, 70, 2, 2, 256, 64),
    (1, 130, 2, 1, 16, 256),
    (3, 33, 9, 3, 64, 64),
    (1, 257, 1, 1, 128, 128),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (BF, F32)], ids=["f32", "bf16", "bf16-f32"])
def test_scan_matches_plain_form(shape, dtype, out):
    B, T, H, G, N, P = shape
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(*shape, dtype)
    _check_scan(cfg, L, out_dtype=out)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_scan_ragged_batch_leaves_rows_behind_a_sequence(dtype):
    B, T, H, G, N, P = 6, 150, 4, 2, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, T, H, G, N, P, dtype)
    lengths = torch.tensor([0, 1, 64, 150, 999, -3], dtype=torch.int32).cuda()
    S_in = torch.randn((B, H, N, P), generator=torch.Generator().manual_seed(5)).cuda()
    # whatever lies in the padding must not reach any output
    for k, name in enumerate(("x", "dt", "Bm", "Cm")):
        for b, n in enumerate((0, 1, 64, 150, 150, 0)):
            L[name][b, n:] = (float("nan"), float("inf"), -float("inf"), float("nan"))[k]
    y = torch.full((B, T, H, P), 7.0, dtype=dtype, device="cuda")
    _, S = _check_scan(cfg, L, lengths=lengths, S_in=S_in, y=y)
    for b, n in enumerate((0, 1, 64, 150, 150, 0)):
        assert bool((y[b, n:] == 7.0).all())
    assert torch.equal(S[0], S_in[0]) and torch.equal(S[5], S_in[5])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_scan_state_in_place_and_carried(dtype):
    """A prompt in two calls over one state array, then single tokens, against the whole prompt at once."""
    B, T, H, G, N, P = 2, 150, 4, 1, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, T, H, G, N, P, dtype)
    part = lambda a, b: {k: (v[:, a:b] if v.dim() > 1 else v) for k, v in L.items()}  # noqa: E731
    S = torch.zeros((B, H, N, P), device="cuda")
    ys = [ramnet.ssm_forward(cfg, **part(0, 71), S_in=S, S_out=S)[0], ramnet.ssm_forward(cfg, **part(71, 147), S_in=S, S_out=S)[0]]
    for t in range(147, 150):
        one = {k: (v[:, t] if v.dim() > 1 else v) for k, v in L.items()}
        ys.append(ramnet.ssm_step(cfg, **one, S=S)[:, None])
    ramnet.sync_status()
    wy, wS, ya, ye, E = plain.scan(**L)
    ty, tS = _scan_tols(wy, ya, ye, E, wS, dtype, dtype == BF)
    _near(torch.cat(ys, 1), wy, ty)
    _near(S, wS, tS)


def test_scan_strong_decay_weak_decay_and_clamped_steps():
    """Decays from none to far below the smallest float, step sizes clamped, no softplus, no D."""
    B, T, H, G, N, P = 1, 140, 4, 1, 64, 64
    for dtype in (F32, BF):
        L = _layer(B, T, H, G, N, P, dtype)
        L["A"] = torch.tensor([0.0, -1e-4, -300.0, -2.0], device="cuda")
        cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P, dt_softplus=False, dt_min=0.01, dt_max=1.5)
        L["dt_bias"], L["D"] = None, None
        _check_scan(cfg, L)
        # a step size of nothing changes nothing
        zero = dict(L, dt=torch.zeros_like(L["dt"]))
        S_in = torch.randn((B, H, N, P), device="cuda")
        cfg0 = ramnet.SsmConfig(H=H, G=G, N=N, P=P, dt_softplus=False)
        _, S = ramnet.ssm_forward(cfg0, **zero, S_in=S_in)
        assert torch.equal(S, S_in)


def test_scan_long_prompt_keeps_its_precision():
    """4096 tokens of slow decay: the state's error stays within the recurrence's own bound."""
    B, T, H, G, N, P = 1, 4096, 2, 1, 64, 64
    for dtype in (F32, BF):
        L = _layer(B, T, H, G, N, P, dtype)
        L["A"] = torch.tensor([-0.01, -1.0], device="cuda")
        _, S = _check_scan(ramnet.SsmConfig(H=H, G=G, N=N, P=P), L)
        wS = plain.scan(**L)[1]
        assert float((S.cpu().double() - wS).norm() / wS.norm()) < 1e-5


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_scan_odd_strides_and_alignment(dtype):
    """Operands whose rows start on odd elements, permuted heads, and step sizes with a stride between heads."""
    B, T, H, G, N, P = 2, 77, 3, 1, 32, 32
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, T, H, G, N, P, dtype)
    odd = torch.empty((B, T, 1 + H * P + 2 * N), dtype=dtype, device="cuda")
    odd[..., 1:1 + H * P] = L["x"].flatten(2)
    odd[..., 1 + H * P:1 + H * P + N] = L["Bm"][:, :, 0]
    odd[..., 1 + H * P + N:] = L["Cm"][:, :, 0]
    M = dict(L, x=odd[..., 1:1 + H * P].unflatten(-1, (H, P)), Bm=odd[..., 1 + H * P:1 + H * P + N].unflatten(-1, (1, N)),
             Cm=odd[..., 1 + H * P + N:].unflatten(-1, (1, N)))
    wide = torch.zeros((B, T, H, 3), dtype=dtype, device="cuda")
    wide[..., 1] = L["dt"]
    M["dt"] = wide[..., 1]
    _check_scan(cfg, M)
    M["x"] = L["x"].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    _check_scan(cfg, M)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_scan_overlapping_and_repeated_views(dtype):
    """Views whose rows overlap (a sliding window) or repeat (one B and C for all of a batch or a sequence)."""
    B, T, H, G, N, P = 2, 150, 4, 2, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, T, H, G, N, P, dtype)
    g = torch.Generator().manual_seed(9)
    flat = torch.randn((B, (T + H) * P), generator=g).to(dtype).cuda()
    L["x"] = flat.as_strided((B, T, H, P), ((T + H) * P, P, P, 1))
    _check_scan(cfg, L)
    one = torch.randn((1, T, G, N), generator=g).to(dtype).cuda()
    L["Bm"] = one.expand(B, T, G, N)
    _check_scan(cfg, L)
    L["Cm"] = one[:, :1].expand(B, T, G, N)
    L["dt"] = L["dt"][:, :, :1].expand(B, T, H)
    _check_scan(cfg, L)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,P", [(64, 64), (128, 32), (256, 16)], ids=str)
def test_scan_cut_into_segments(dtype, N, P):
    """A prompt long enough to be cut into segments, with sequences that end in the first, that are not there at all,
    and that end with a token in a chunk; the state carried in place; and a workspace that starts as NaN."""
    B, T, H, G = 4, 1500, 3, 1
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, T, H, G, N, P, dtype)
    L["A"] = torch.tensor([-1.0, -0.02, -16.0], device="cuda")
    n = (1500, 0, 1, 1089)
    lengths = torch.tensor(n, dtype=torch.int32).cuda()
    S0 = torch.randn((B, H, N, P), generator=torch.Generator().manual_seed(2)).cuda()
    for k in ("x", "dt", "Bm", "Cm"):
        for b in range(B):
            L[k][b, n[b]:] = float("nan")
    ws = torch.full((ramnet.ssm_workspace_bytes(cfg, B, T),), 255, dtype=torch.uint8, device="cuda")
    assert ws.numel() > B * H * (N * P * 4)  # pieces' states are among it
    y = torch.full((B, T, H, P), 3.0, dtype=dtype, device="cuda")
    S = S0.clone()
    ramnet.ssm_forward(cfg, **L, lengths=lengths, S_in=S, S_out=S, y=y, workspace=ws)
    ramnet.sync_status()
    wy, wS, ya, ye, E = plain.scan(**L, lengths=lengths, S_in=S0)
    ty, tS = _scan_tols(wy, ya, ye, E, wS, dtype, dtype == BF)
    for b in range(B):
        if n[b]:
            _near(y[b, :n[b]], wy[b, :n[b]], ty[b, :n[b]])
        assert bool((y[b, n[b]:] == 3.0).all())
    _near(S, wS, tS)
    assert torch.equal(S[1], S0[1])


@pytest.mark.parametrize("T", [300, 1300], ids=["whole", "cut"])
def test_scan_is_deterministic_and_captured(T):
    B, H, G, N, P = 2, 4, 1, 128, 64
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, T, H, G, N, P, BF)
    need = ramnet.ssm_workspace_bytes(cfg, B, T)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    y0, S0 = ramnet.ssm_forward(cfg, **L)
    y, S = torch.zeros_like(y0), torch.zeros_like(S0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ramnet.ssm_forward(cfg, **L, y=y, S_out=S, workspace=ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ramnet.ssm_forward(cfg, **L, y=y, S_out=S, workspace=ws)
    for _ in range(3):
        y.zero_(), S.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(S, S0)


STEP = [(1, 1, 1, 16, 16), (3, 4, 2, 32, 64), (2, 6, 3, 128, 32), (2, 2, 1, 64, 256), (2, 2, 1, 256, 128), (40, 5, 5, 128, 128)]


@pytest.mark.parametrize("shape", STEP, ids=str)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (BF, F32)], ids=["f32", "bf16", "bf16-f32"])
def test_step_matches_plain_form(shape, dtype, out):
    B, H, G, N, P = shape
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, 3, H, G, N, P, dtype)
    S0 = torch.randn((B, H, N, P), generator=torch.Generator().manual_seed(1)).cuda()
    S = S0.clone()
    ys = [ramnet.ssm_step(cfg, **{k: (v[:, t] if v.dim() > 1 else v) for k, v in L.items()}, S=S, out_dtype=out) for t in range(3)]
    ramnet.sync_status()
    wy, wS, ya, ye, E = plain.scan(**L, S_in=S0)
    _near(torch.stack(ys, 1), wy, ye + _half_step(wy, out))
    _near(S, wS, E + 1e-30)


def test_thousands_of_single_tokens_keep_their_precision():
    """A slowly decaying state stepped token by token: a bias of the decay's exponential would add up."""
    T, H, N, P = 3000, 2, 16, 32
    cfg = ramnet.SsmConfig(H=H, G=1, N=N, P=P)
    L = _layer(1, T, H, 1, N, P, F32)
    L["A"] = torch.tensor([-0.01, -0.3], device="cuda")
    S = torch.zeros((1, H, N, P), device="cuda")
    for t in range(T):
        y = ramnet.ssm_step(cfg, **{k: (v[:, t] if v.dim() > 1 else v) for k, v in L.items()}, S=S)
    wy, wS, _, ye, E = plain.scan(**L)
    _near(S, wS, E)
    _near(y, wy[:, -1], ye[:, -1])
    assert float((S.cpu().double() - wS).norm() / wS.norm()) < 1e-5


@pytest.mark.parametrize("softplus", [True, False], ids=["softplus", "plain"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_a_step_size_that_is_no_number_shows(dtype, softplus):
    B, T, H, N, P = 2, 100, 3, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=1, N=N, P=P, dt_softplus=softplus)
    L = _layer(B, T, H, 1, N, P, dtype)
    clean = ramnet.ssm_forward(cfg, **L)
    L["dt"][1, 70, 2] = float("nan")
    y, S = ramnet.ssm_forward(cfg, **L)
    assert bool(torch.isnan(y[1, 70:, 2]).all()) and bool(torch.isnan(S[1, 2]).all())
    for b, h in ((0, 0), (0, 2), (1, 0), (1, 1)):
        assert torch.equal(y[b, :, h], clean[0][b, :, h]) and torch.equal(S[b, h], clean[1][b, h])
    assert torch.equal(y[1, :64, 2], clean[0][1, :64, 2])
    S = torch.zeros((B, H, N, P), device="cuda")
    y = ramnet.ssm_step(cfg, **{k: (v[:, 70] if v.dim() > 1 else v) for k, v in L.items()}, S=S)
    assert bool(torch.isnan(y[1, 2]).all()) and bool(torch.isnan(S[1, 2]).all())
    assert bool(torch.isfinite(S[0]).all()) and bool(torch.isfinite(S[1, :2]).all())


CONV = [(1, 1, 1, 2), (2, 70, 6, 3), (1, 40, 12, 4), (1, 2, 8, 4), (2, 3, 16, 4), (3, 33, 24, 3), (2, 65, 17, 4), (2, 130, 520, 2), (1, 31, 7, 3)]


def _conv_tol(wy, ya, W, silu, out):
    # W + 1 roundings of the sum; SiLU's slope is below 1.1, its own error 2^-20 (hardware exp2, bf16 results: the
    # exponent's argument adds its size) or 8 u of the value; then the output's rounding
    t = 1.1 * (W + 2) * U32 * ya + _half_step(wy, out)
    if silu:
        t = t + (wy.abs() * (2.0 ** -20 * (1 + ya)) if out == BF else wy.abs() * U32 * (8 + 2 * ya))
    return t + 1e-30


@pytest.mark.parametrize("shape", CONV, ids=str)
@pytest.mark.parametrize("silu", [True, False], ids=["silu", "linear"])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)], ids=["f32", "bf16", "bf16-f32", "f32-bf16"])
def test_conv_matches_plain_form(shape, silu, dtype, out):
    B, T, C, W = shape
    g = torch.Generator().manual_seed(3)
    wide = torch.randn((B, T, 2 * C + 1), generator=g).to(dtype).cuda()
    x = wide[..., C + 1:] if C % 2 else wide[..., 1:C + 1]
    w, bias = torch.randn((C, W), generator=g).cuda(), torch.randn((C,), generator=g).cuda()
    state = torch.randn((B, W - 1, C), generator=g).to(dtype).cuda()
    for xx in (x, x.contiguous()):
        for st, bi in ((None, None), (state, bias)):
            y, kept = ramnet.conv_forward(xx, w, bias=bi, silu=silu, state_in=st, out_dtype=out)
            wy, wk, ya = plain.conv(xx, w, bi, silu, None, st)
            _near(y, wy, _conv_tol(wy, ya, W, silu, out))
            assert torch.equal(kept.cpu().double(), wk)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_conv_ragged_in_place_and_single_tokens(dtype):
    B, T, C, W = 6, 70, 40, 4
    g = torch.Generator().manual_seed(4)
    x = torch.randn((B, T, C), generator=g).to(dtype).cuda()
    w, bias = torch.randn((C, W), generator=g).cuda(), torch.randn((C,), generator=g).cuda()
    state = torch.randn((B, W - 1, C), generator=g).to(dtype).cuda()
    n = (0, 1, 2, 3, 70, 33)
    lengths = torch.tensor([-1, 1, 2, 3, 99, 33], dtype=torch.int32).cuda()
    wy, wk, ya = plain.conv(x, w, bias, True, lengths, state)
    for b in range(B):
        x[b, n[b]:] = float("nan")
    y = torch.full_like(x, 5.0)
    s = state.clone()
    ramnet.conv_forward(x, w, bias=bias, lengths=lengths, state_in=s, y=y, state_out=s)  # the state in place
    for b in range(B):
        if n[b]:
            _near(y[b, :n[b]], wy[b, :n[b]], _conv_tol(wy, ya, W, True, dtype)[b, :n[b]])
        assert bool((y[b, n[b]:] == 5.0).all())
    assert torch.equal(s.cpu().double(), wk)
    more = torch.randn((B, 5, C), generator=g).to(dtype).cuda()
    wy2, wk2, ya2 = plain.conv(more, w, bias, True, None, s)
    for t in range(5):
        yt = ramnet.conv_step(more[:, t], w, s, bias=bias)
        _near(yt, wy2[:, t], _conv_tol(wy2, ya2, W, True, dtype)[:, t])
    assert torch.equal(s.cpu().double(), wk2)


NORM = [(1, 1, 1), (3, 8, 1), (5, 24, 3), (2, 2048, 1), (7, 1536, 2), (2, 17, 1), (2, 9000, 1), (1, 20000, 1), (3, 18000, 2),
        (300, 64, 4), (1000, 100, 1), (3, 1918, 1), (2, 348, 4), (2, 700, 2), (1, 3001, 1), (2, 6784, 4)]


@pytest.mark.parametrize("shape", NORM, ids=str)
@pytest.mark.parametrize("first", [True, False], ids=["gate-first", "norm-first"])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (BF, F32)], ids=["f32", "bf16", "bf16-f32"])
def test_norm_gate_matches_plain_form(shape, first, dtype, out):
    R, D, groups = shape
    g = torch.Generator().manual_seed(6)
    x = torch.randn((R, D), generator=g).to(dtype).cuda()
    z = (3 * torch.randn((R, 2 * D + 1), generator=g)).to(dtype).cuda()[:, 1:D + 1]
    w = torch.randn((D,), generator=g).cuda()
    x[0] = 0  # a row of nothing: eps alone
    for zz, ww in ((z, w), (z.contiguous(), None), (None, w)):  # (the first on odd elements: single values)
        y = ramnet.norm_gate(x, z=zz, w=ww, groups=groups, eps=1e-5, gate_first=first, out_dtype=out)
        want = plain.norm_gate(x, zz, ww, groups, 1e-5, first)
        # a sum of squares off by (adds) u is half that in its root: at most D/groups/256 adds per thread and 13 more,
        # twice an SiLU error (8 u, bf16 results 2^-19 with the exponent's argument) and 10 u for the rest
        gate = 0.0 if zz is None else (2.0 ** -19 * 12 if out == BF else U32 * 40)
        rel = U32 * (0.5 * (D / groups / 256 + 45) + 10) + 2 * gate
        _near(y, want, want.abs() * rel + _half_step(want, out) + 1e-30)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_layer_prompt_then_tokens_equals_one_prompt(dtype):
    """The whole run as a layer makes it: convolution, scan, norm over a prompt, then token by token on the
    states it left, against the prompt and the tokens in one go (same inputs, same states)."""
    B, T, H, G, N, P, W = 2, 90, 4, 2, 64, 64, 4
    C, extra = H * P + 2 * G * N, 4
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    g = torch.Generator().manual_seed(8)
    proj = torch.randn((B, T + extra, H * P + C + H), generator=g).to(dtype).cuda()  # z, convolution input, dt
    w, bias = (torch.randn((C, W), generator=g) / 2).cuda(), torch.randn((C,), generator=g).cuda()
    par = dict(A=-(1 + torch.rand((H,), generator=g)).cuda(), D=torch.ones(H).cuda(), dt_bias=torch.full((H,), -3.0).cuda())
    nw = torch.randn((H * P,), generator=g).cuda()

    def split(v):
        return (v[..., :H * P].unflatten(-1, (H, P)), v[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
                v[..., H * P + G * N:].unflatten(-1, (G, N)))

    def prompt(p, S=None, cs=None):
        v, cs = ramnet.conv_forward(p[..., H * P:H * P + C], w, bias=bias, state_in=cs)
        x, Bm, Cm = split(v)
        y, S = ramnet.ssm_forward(cfg, x, p[..., H * P + C:], par["A"], Bm, Cm, D=par["D"], dt_bias=par["dt_bias"], S_in=S)
        flat = p.reshape(-1, p.shape[-1]) if p.is_contiguous() else p.contiguous().reshape(-1, p.shape[-1])
        return ramnet.norm_gate(y.reshape(-1, H * P), z=flat[:, :H * P], w=nw, groups=G).unflatten(0, p.shape[:2]), S, cs

    whole, S_all, cs_all = prompt(proj)
    y, S, cs = prompt(proj[:, :T].contiguous())
    outs = [y]
    for t in range(T, T + extra):
        p = proj[:, t]
        v = ramnet.conv_step(p[:, H * P:H * P + C], w, cs, bias=bias)
        x, Bm, Cm = split(v)
        yt = ramnet.ssm_step(cfg, x, p[:, H * P + C:], par["A"], Bm, Cm, S, D=par["D"], dt_bias=par["dt_bias"])
        outs.append(ramnet.norm_gate(yt.flatten(1), z=p[:, :H * P], w=nw, groups=G)[:, None])
    ramnet.sync_status()
    got = torch.cat(outs, 1).cpu().double()
    want = whole.cpu().double()
    # the convolution is the same arithmetic; the scan's outputs differ by fp32 roundings before they are rounded,
    # so by at most a step of the type, which the norm hands on (twice: the value and the row's root)
    step = torch.finfo(dtype).eps
    lim = 3 * step * want.abs().amax() if dtype == BF else 1e-4 * want.abs().amax()
    assert float((got - want).abs().max()) <= float(lim)
    assert float((S - S_all).norm() / S_all.norm()) < 1e-5
    assert torch.equal(cs, cs_all)


def test_two_calls_at_once_on_streams_of_their_own():
    """Two prompts on two streams, without workspaces of the caller's, interleaved with each other and with
    allocations on the current stream; and a norm and a convolution on a stream that is passed in."""
    B, T, H, G, N, P = 2, 700, 4, 2, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    Ls = [_layer(B, T, H, G, N, P, BF, seed=s) for s in (1, 2)]
    refs = [ramnet.ssm_forward(cfg, **L) for L in Ls]
    flat = Ls[0]["x"].flatten(2).contiguous()
    w = torch.ones((H * P, 4), device="cuda")
    cref, nref = ramnet.conv_forward(flat, w), ramnet.norm_gate(flat.flatten(0, 1))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ls]
    outs = []
    for rep in range(4):
        for L, s in zip(Ls, streams):
            outs.append(ramnet.ssm_forward(cfg, **L, stream=s))
            torch.full((1 << 20,), float("nan"), device="cuda")
    outs += [ramnet.ssm_forward(cfg, **L, stream=torch.cuda.current_stream().cuda_stream) for L in Ls]  # a raw handle
    c, n = ramnet.conv_forward(flat, w, stream=streams[0]), ramnet.norm_gate(flat.flatten(0, 1), stream=streams[1])
    torch.cuda.synchronize()
    for i, (y, S) in enumerate(outs):
        assert torch.equal(y, refs[i % 2][0]) and torch.equal(S, refs[i % 2][1])
    assert torch.equal(c[0], cref[0]) and torch.equal(c[1], cref[1]) and torch.equal(n, nref)


def test_a_call_on_another_stream_leaves_memory_in_use_alone():
    """Memory that was let go on the current stream, while work there still reads it, is not taken by a call that
    runs on another stream."""
    B, T, H, N, P = 2, 256, 4, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=1, N=N, P=P)
    L = _layer(B, T, H, 1, N, P, BF)
    flat = L["x"].flatten(2).contiguous()
    w = torch.ones((H * P, 4), device="cuda")
    ref = ramnet.ssm_forward(cfg, **L)
    other = torch.cuda.Stream()
    sizes = (ramnet.ssm_workspace_bytes(cfg, B, T), B * T * H * P * 2, B * H * N * P * 4, B * 3 * H * P * 2)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes]
    copies = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for c, t in zip(copies, held):
        c.copy_(t)
    del held, t
    y, S = ramnet.ssm_forward(cfg, **L, stream=other)
    ramnet.conv_forward(flat, w, stream=other)
    ramnet.norm_gate(flat.flatten(0, 1), stream=other.cuda_stream)
    torch.cuda.synchronize()
    assert all(bool((c == 77).all()) for c in copies)
    assert torch.equal(y, ref[0]) and torch.equal(S, ref[1])


def test_steps_captured_and_replayed():
    """A layer's step (convolution, scan, norm) as one graph over fixed buffers, replayed on new tokens."""
    B, H, G, N, P, W = 3, 4, 2, 64, 64, 4
    C = H * P + 2 * G * N
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    g = torch.Generator().manual_seed(11)
    w, A = torch.randn((C, W), generator=g).cuda(), -(1 + torch.rand((H,), generator=g)).cuda()
    toks = torch.randn((5, B, C + H), generator=g).to(BF).cuda()

    def step(tok, cs, S):
        v = ramnet.conv_step(tok[:, :C], w, cs)
        x, Bm, Cm = v[:, :H * P].unflatten(-1, (H, P)), v[:, H * P:H * P + G * N].unflatten(-1, (G, N)), v[:, H * P + G * N:].unflatten(-1, (G, N))
        return ramnet.norm_gate(ramnet.ssm_step(cfg, x, tok[:, C:], A, Bm, Cm, S).flatten(1))

    cs, S = torch.zeros((B, W - 1, C), dtype=BF, device="cuda"), torch.zeros((B, H, N, P), device="cuda")
    want = [step(t, cs, S).clone() for t in toks]
    end = (cs.clone(), S.clone())
    tok = toks[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(tok, cs, S)
    cs.zero_(), S.zero_()
    for t, y in zip(toks, want):
        tok.copy_(t)
        graph.replay()
        assert torch.equal(out, y)
    assert torch.equal(cs, end[0]) and torch.equal(S, end[1])


def test_other_stream_and_offsets_past_32_bits():
    """A call on a stream of its own, and operands whose last sequence starts beyond 2^31 elements."""
    H, G, N, P, T = 2, 1, 16, 16, 5
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(2, T, H, G, N, P, BF)
    far = (1 << 31) + 64
    big = torch.empty(far + T * H * P, dtype=BF, device="cuda")
    x = big.as_strided((2, T, H, P), (far, H * P, P, 1))
    x.copy_(L["x"])
    ref = ramnet.ssm_forward(cfg, **L)
    cref = ramnet.conv_forward(L["x"].flatten(2), torch.ones((H * P, 4), device="cuda"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = ramnet.ssm_forward(cfg, **dict(L, x=x))
        cgot = ramnet.conv_forward(x.flatten(2), torch.ones((H * P, 4), device="cuda"))
    s.synchronize()
    for a, b in zip(ref + cref, got + cgot):
        assert torch.equal(a, b)
