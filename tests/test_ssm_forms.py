"""State space layer on the GPU: the forms, sizes and types between those of test_ssm.py, against the plain 64-bit forms in
oracle/ssm.py, with that file's tolerances."""
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


def _within(got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape and bool(torch.isfinite(got).all())
    over = (got - want).abs() - tol
    assert float(over.max()) <= 0, f"off by up to {float((got - want).abs().max()):.3g}, {float(over.max()):.3g} over the bound"


def _half_step(v, dtype):
    return v.abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).tiny


def _layer(B, T, H, G, N, P, dtype, seed=0):
    """x, B and C as slices of one convolution output; decays from fast to slow, so that segments carry state."""
    g = torch.Generator().manual_seed(seed)
    xbc = torch.nn.functional.silu(torch.randn((B, T, H * P + 2 * G * N), generator=g)).to(dtype).cuda()
    return dict(x=xbc[..., :H * P].unflatten(-1, (H, P)), dt=(0.5 * torch.randn((B, T, H), generator=g) - 4).to(dtype).cuda(),
                A=-torch.exp(torch.linspace(-4, 3, H)).cuda(), Bm=xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
                Cm=xbc[..., H * P + G * N:].unflatten(-1, (G, N)), D=(torch.rand((H,), generator=g) + 0.5).cuda())


def _check(cfg, L, n, S_in, out=None):
    """A ragged batch with a carried state, a workspace that starts as NaN and padding that holds none."""
    x = L["x"]
    B, T, H, P = x.shape
    lengths = torch.tensor(n, dtype=torch.int32).cuda()
    for k in ("x", "dt", "Bm", "Cm"):
        for b in range(B):
            L[k][b, n[b]:] = float("nan")
    out = x.dtype if out is None else out
    ws = torch.full((ramnet.ssm_workspace_bytes(cfg, B, T),), 255, dtype=torch.uint8, device="cuda")
    y, S = torch.full((B, T, H, P), 3.0, dtype=out, device="cuda"), S_in.clone()
    ramnet.ssm_forward(cfg, **L, lengths=lengths, S_in=S, S_out=S, y=y, workspace=ws)
    ramnet.sync_status()
    wy, wS, ya, ye, E = plain.scan(**L, lengths=lengths, S_in=S_in)
    pieces = x.dtype == BF and out == BF
    ty = ye + _half_step(wy, out) + (2.0 ** -15 * ya if pieces else 0)
    tS = E + (64 * U32 * wS.abs().amax(dim=(2, 3), keepdim=True) if pieces else 0) + 1e-30
    for b in range(B):
        if n[b]:
            _within(y[b, :n[b]], wy[b, :n[b]], ty[b, :n[b]])
        assert bool((y[b, n[b]:] == 3.0).all())
        if n[b] == 0:
            assert torch.equal(S[b], S_in[b])
    _within(S, wS, tS)


CUT = [
    # B, T, H, G, N, P, lengths
    (6, 1021, 24, 2, 64, 64, (1021, 0, 511, 256, 1, 513)),     # two segments, the first in two pieces
    (8, 1280, 8, 1, 128, 128, (1280, 0, 577, 640, 641, 1, 64, 1279)),  # the same, one head per 128 channels
    (2, 768, 9, 1, 32, 128, (768, 449)),                       # three segments in four pieces each
    (1, 2048, 2, 1, 64, 256, (1999,)),                         # heads of two blocks, eight segments in two pieces each
    (2, 1100, 3, 1, 128, 128, (1100, 700)),
    (1, 1300, 3, 1, 16, 64, (1300,)),
    (1, 1600, 5, 1, 32, 32, (1333,)),                          # four heads per 128 channels, the last block with one
]


@pytest.mark.parametrize("shape", CUT, ids=lambda s: str(s[:6]))
def test_prompts_cut_on_the_tensor_cores(shape):
    B, T, H, G, N, P, n = shape
    S_in = torch.randn((B, H, N, P), generator=torch.Generator().manual_seed(2)).cuda()
    _check(ramnet.SsmConfig(H=H, G=G, N=N, P=P), _layer(B, T, H, G, N, P, BF), n, S_in)


PLAIN_CUT = [(2, 333, 5, 5, 16, 32, (333, 200)), (2, 400, 3, 1, 32, 16, (400, 81)), (1, 700, 2, 1, 64, 16, (700,)), (1, 900, 3, 1, 16, 64, (895,)),
             (2, 500, 2, 2, 16, 16, (500, 0)), (1, 500, 2, 1, 32, 32, (500,)), (1, 700, 2, 1, 16, 128, (700,)), (1, 600, 1, 1, 256, 64, (600,)),
             (1, 400, 2, 1, 16, 256, (399,)), (1, 400, 2, 1, 128, 16, (400,))]


@pytest.mark.parametrize("shape", PLAIN_CUT, ids=lambda s: str(s[:6]))
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F32, BF), (BF, F32)], ids=["f32", "f32-bf16", "bf16-f32"])
def test_prompts_cut_token_by_token(shape, dtype, out):
    B, T, H, G, N, P, n = shape
    S_in = torch.randn((B, H, N, P), generator=torch.Generator().manual_seed(2)).cuda()
    _check(ramnet.SsmConfig(H=H, G=G, N=N, P=P), _layer(B, T, H, G, N, P, dtype), n, S_in, out)


@pytest.mark.parametrize("shape", [(3, 4, 2, 32, 64), (2, 2, 1, 256, 128), (1, 3, 1, 16, 16)], ids=str)
def test_step_fp32_in_bf16_out(shape):
    B, H, G, N, P = shape
    L = {k: (v[:, 0] if v.dim() > 1 else v) for k, v in _layer(B, 1, H, G, N, P, F32).items()}
    S0 = torch.randn((B, H, N, P), generator=torch.Generator().manual_seed(1)).cuda()
    S = S0.clone()
    y = ramnet.ssm_step(ramnet.SsmConfig(H=H, G=G, N=N, P=P), **L, S=S, out_dtype=BF)
    wy, wS, _, ye, E = plain.scan(**{k: (v[:, None] if v.dim() > 1 else v) for k, v in L.items()}, S_in=S0)
    _within(y, wy[:, 0], ye[:, 0] + _half_step(wy[:, 0], BF))
    _within(S, wS, E + 1e-30)


@pytest.mark.parametrize("dims", [(3, 24, 1), (2, 2048, 1), (5, 700, 2), (2, 17, 1), (1, 9000, 1)], ids=str)
@pytest.mark.parametrize("first", [True, False], ids=["gate-first", "norm-first"])
def test_norm_gate_fp32_in_bf16_out(dims, first):
    R, D, groups = dims
    g = torch.Generator().manual_seed(6)
    x, z, w = torch.randn((R, D), generator=g).cuda(), 3 * torch.randn((R, D), generator=g).cuda(), torch.randn((D,), generator=g).cuda()
    y = ramnet.norm_gate(x, z=z, w=w, groups=groups, eps=1e-5, gate_first=first, out_dtype=BF)
    want = plain.norm_gate(x, z, w, groups, 1e-5, first)
    rel = U32 * (0.5 * (D / groups / 256 + 45) + 10) + 2 * 2.0 ** -19 * 12  # as test_ssm.py's bound for bf16 results
    _within(y, want, want.abs() * rel + _half_step(want, BF) + 1e-30)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [1, 7, 12, 40, 1043])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)], ids=["f32", "bf16", "bf16-f32", "f32-bf16"])
def test_conv_step_of_every_width(W, C, dtype, out):
    """... with channel counts that take every vector width, rows on odd elements and dense ones, with and without a bias and SiLU."""
    B = 3
    g = torch.Generator().manual_seed(W * C)
    wide = torch.randn((B, 2 * C + 1), generator=g).to(dtype).cuda()
    w, bias = torch.randn((C, W), generator=g).cuda(), torch.randn((C,), generator=g).cuda()
    state = torch.randn((B, W - 1, C), generator=g).to(dtype).cuda()
    for x in (wide[:, 1:C + 1], wide[:, C + 1:].contiguous()):
        for bi, silu in ((None, True), (bias, False), (bias, True)):
            s = state.clone()
            y = ramnet.conv_step(x, w, s, bias=bi, silu=silu, out_dtype=out)
            wy, wk, ya = plain.conv(x[:, None], w, bi, silu, None, state)
            tol = 1.1 * (W + 2) * U32 * ya + _half_step(wy, out) + 1e-30  # W + 1 roundings of the sum, SiLU's slope below 1.1
            if silu:  # its own error: hardware exp2 for bf16 results, 8 u of the value, the exponent's argument adds its size
                tol = tol + wy.abs() * (2.0 ** -20 * (1 + ya) if out == BF else U32 * (8 + 2 * ya))
            _within(y, wy[:, 0], tol[:, 0])
            assert torch.equal(s.cpu().double(), wk)


def test_operands_past_32_bits_on_the_tensor_cores():
    """The last sequence of x and dt, and the last row of a norm, begin beyond 2^31 elements."""
    B, T, H, G, N, P = 2, 200, 2, 1, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _layer(B, T, H, G, N, P, BF)
    ref = ramnet.ssm_forward(cfg, **L)
    far = (1 << 31) + 64
    big = torch.empty(far + T * H * P, dtype=BF, device="cuda")
    x = big.as_strided((B, T, H, P), (far, H * P, P, 1))
    x.copy_(L["x"])
    got = ramnet.ssm_forward(cfg, **dict(L, x=x))
    ramnet.sync_status()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    one = {k: (v[:, 3] if v.dim() > 1 else v) for k, v in L.items()}
    S, S2 = (torch.zeros((B, H, N, P), device="cuda") for _ in range(2))
    assert torch.equal(ramnet.ssm_step(cfg, **one, S=S), ramnet.ssm_step(cfg, **dict(one, x=x[:, 3]), S=S2)) and torch.equal(S, S2)
    rows = x[:, 0].flatten(1)
    assert torch.equal(ramnet.norm_gate(rows, z=rows), ramnet.norm_gate(rows.contiguous(), z=rows.contiguous()))
    w, s, s2 = torch.ones((H * P, 4), device="cuda"), *(torch.zeros((B, 3, H * P), dtype=BF, device="cuda") for _ in range(2))
    assert torch.equal(ramnet.conv_step(rows, w, s), ramnet.conv_step(rows.contiguous(), w, s2)) and torch.equal(s, s2)
    dt = big.as_strided((B, T, H), (far, H, 1))
    dt.copy_(L["dt"])
    got = ramnet.ssm_forward(cfg, **dict(L, dt=dt))
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
