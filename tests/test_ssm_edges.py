"""State space layer on the GPU at the edges of its definition, against the plain 64-bit form in oracle/ssm.py or a closed
form.  Tolerances are those of test_ssm.py: the oracle's bound on fp32 roundings, 2^-15 of the sum of absolute values where
bf16 prompts meet the state and the token-to-token weights as two bf16 pieces, half a step of the output's type."""
import time

import pytest
import torch

from oracle import ssm as plain
from sparse_slot_recurrent_b200 import ramnet

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U32 = 2.0 ** -24


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


def _operands(B, T, H, G, N, P, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=r(B, T, H, P).to(dtype).cuda(), dt=r(B, T, H).mul(0.5).to(dtype).cuda(), A=-(1 + 15 * torch.rand((H,), generator=g)).cuda(),
                Bm=r(B, T, G, N).to(dtype).cuda(), Cm=r(B, T, G, N).to(dtype).cuda(), D=(torch.rand((H,), generator=g) + 0.5).cuda())


def _token(L, t):
    return {k: (v[:, t] if v is not None and v.dim() > 1 else v) for k, v in L.items()}


def _check(cfg, L, S_in=None, lengths=None, **kw):
    y, S = ramnet.ssm_forward(cfg, **L, S_in=S_in, lengths=lengths, **kw)
    ramnet.sync_status()
    wy, wS, ya, ye, E = plain.scan(**L, S_in=S_in, lengths=lengths, softplus=cfg.dt_softplus, dt_min=cfg.dt_min, dt_max=cfg.dt_max)
    pieces = L["x"].dtype == BF and y.dtype == BF
    ty = ye + wy.abs() * torch.finfo(y.dtype).eps / 2 + torch.finfo(y.dtype).tiny + (2.0 ** -15 * ya if pieces else 0)
    # sums of 64 tokens at once: 64 more roundings than token by token
    tS = E + (64 * U32 * wS.abs().amax(dim=(2, 3), keepdim=True) if pieces else 0) + 1e-30
    for b in range(y.shape[0]):
        n = y.shape[1] if lengths is None else min(max(int(lengths[b]), 0), y.shape[1])
        if n:
            _within(y[b, :n], wy[b, :n], ty[b, :n])
    _within(S, wS, tS)
    return y, S


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [70, 1100], ids=["whole", "cut"])
def test_a_state_that_forgets_everything_at_every_token(dtype, T):
    """d A from -1e30 to below fp32's lowest number, over a chunk and from one token on: the decay is 0, so that a token
    sees itself alone, in the prompt as in single tokens."""
    B, H, N, P = 1, 4, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=1, N=N, P=P)
    L = _operands(B, T, H, 1, N, P, dtype)
    L["A"] = torch.tensor([-1e32, -1e37, torch.finfo(F32).min, -float("inf")], device="cuda")
    S_in = torch.randn((B, H, N, P), generator=torch.Generator().manual_seed(3)).cuda()
    y, S = ramnet.ssm_forward(cfg, **L, S_in=S_in)
    ramnet.sync_status()
    x, Bm, Cm = (L[k].cpu().double() for k in ("x", "Bm", "Cm"))
    d = plain.step_sizes(L["dt"], None)
    g = (Bm * Cm).sum(-1)  # [B,T,1]
    skip = L["D"].cpu().double()[:, None] * x
    wy = (d * g)[..., None] * x + skip
    ya = (d * (Bm * Cm).abs().sum(-1))[..., None] * x.abs() + skip.abs()
    wS = d[:, -1, :, None, None] * Bm[:, -1, 0, None, :, None] * x[:, -1, :, None, :]
    # a step size good to 16 u, then products and a sum over n
    u = U32 * (N + 24)
    _within(y, wy, ya * (u + (2.0 ** -15 if dtype == BF else 0)) + wy.abs() * torch.finfo(dtype).eps / 2 + 1e-30)
    _within(S, wS, wS.abs() * U32 * 24 + 1e-30)
    one = S_in.clone()
    _within(ramnet.ssm_step(cfg, **_token(L, 5), S=one), wy[:, 5], ya[:, 5] * u + wy[:, 5].abs() * torch.finfo(dtype).eps / 2 + 1e-30)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_a_token_that_resets_the_state_leaves_its_chunk_precise(dtype):
    """Slow decay but for a few tokens with d A = -1e12: what follows them in the same chunk decays by their own step sizes."""
    B, T, H, N, P = 2, 150, 2, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=1, N=N, P=P, dt_softplus=False)
    L = _operands(B, T, H, 1, N, P, dtype)
    L["A"] = torch.tensor([-1e12, -3e12], device="cuda")
    L["dt"] = (torch.rand((B, T, H), generator=torch.Generator().manual_seed(1)) * 1e-13 + 1e-14).to(dtype).cuda()
    for t in (0, 20, 37, 64, 127):
        L["dt"][:, t] = 1.0
    L["D"] = None
    _check(cfg, L)


CAUSAL = [
    # T, H, G, N, P
    (100, 4, 2, 64, 64),
    (150, 3, 1, 128, 128),
    (90, 5, 1, 16, 32),
    (70, 2, 1, 32, 256),
    (900, 2, 1, 64, 64),  # in segments
    (40, 2, 1, 64, 16),
]


@pytest.mark.parametrize("shape", CAUSAL, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("what", ["x", "Bm", "Cm", "dt"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_what_is_no_number_reaches_no_earlier_token(shape, dtype, what, bad):
    T, H, G, N, P = shape
    B, at = 2, T - 27
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _operands(B, T, H, G, N, P, dtype)
    y0, S0 = ramnet.ssm_forward(cfg, **L)
    M = dict(L, **{what: L[what].clone()})
    hit = torch.zeros((B, H, P), dtype=torch.bool, device="cuda")  # what the value may reach, from its token on
    if what == "x":
        M["x"][1, at, H - 1, 5] = bad
        hit[1, H - 1, 5] = True
    elif what == "dt":
        M["dt"][1, at, H - 1] = bad
        hit[1, H - 1] = True
    else:
        M[what][1, at, G - 1, 3] = bad
        hit[1, H - H // G:] = True
    y, S = ramnet.ssm_forward(cfg, **M)
    ramnet.sync_status()
    assert torch.equal(y[:, :at], y0[:, :at])
    keep = ~hit[:, None].expand(y.shape)
    assert torch.equal(y[keep], y0[keep])
    keepS = ~hit[:, :, None].expand(S.shape)
    assert torch.equal(S[keepS], S0[keepS])
    if what == "Cm":  # a token's C reaches that token's output alone
        assert torch.equal(S, S0)
        assert not bool(torch.isfinite(y[:, at][hit]).any())
        after = torch.ones_like(y, dtype=torch.bool)
        after[:, at] = False
        assert torch.equal(y[after], y0[after])
    else:
        assert not bool(torch.isfinite(y[:, at:][hit[:, None].expand(y[:, at:].shape)]).any()) or what == "dt"
        assert not bool(torch.isfinite(S.movedim(2, 3)[hit]).all(-1).any())


@pytest.mark.parametrize("what", ["x", "Bm", "Cm", "dt"])
def test_numbers_that_are_none_in_a_ragged_batch(what):
    """... in the last token of each of some sequences that end within a chunk; rows behind them stay as they were."""
    B, T, H, G, N, P = 4, 200, 4, 2, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=G, N=N, P=P)
    L = _operands(B, T, H, G, N, P, BF)
    n = (1, 64, 97, 200)
    lengths = torch.tensor(n, dtype=torch.int32).cuda()
    y0, _ = ramnet.ssm_forward(cfg, **L, lengths=lengths, y=torch.full((B, T, H, P), 7.0, dtype=BF, device="cuda"))
    for b in range(B):
        L[what][b, n[b] - 1] = float("nan")
    y, S = ramnet.ssm_forward(cfg, **L, lengths=lengths, y=torch.full((B, T, H, P), 7.0, dtype=BF, device="cuda"))
    for b in range(B):
        assert torch.equal(y[b, :n[b] - 1], y0[b, :n[b] - 1])
        assert bool(torch.isnan(y[b, n[b] - 1]).all())
        assert bool((y[b, n[b]:] == 7.0).all())
        assert bool(torch.isnan(S[b]).all()) == (what != "Cm")


def _owner(t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]


def test_memory_of_a_call_on_the_default_stream_by_its_handle():
    """stream=0, while another stream is current: outputs and workspace lie in the default stream's memory."""
    B, T, H, N, P = 2, 100, 4, 64, 64
    cfg = ramnet.SsmConfig(H=H, G=1, N=N, P=P)
    L = _operands(B, T, H, 1, N, P, BF)
    flat, w = L["x"].flatten(2), torch.ones((H * P, 4), device="cuda")
    ref = ramnet.ssm_forward(cfg, **L)
    S = torch.zeros((B, H, N, P), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        outs = [*ramnet.ssm_forward(cfg, **L, stream=0), ramnet.ssm_step(cfg, **_token(L, 0), S=S, stream=0),
                *ramnet.conv_forward(flat, w, stream=0), ramnet.norm_gate(flat.flatten(0, 1), stream=torch.cuda.default_stream().cuda_stream)]
        for t in outs:
            assert _owner(t) == [0]
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])


def test_memory_of_a_call_on_a_stream_by_its_handle_or_as_an_object():
    class Wrapped:  # what the slot layer's calls take as a stream too
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    s = torch.cuda.Stream()
    x = torch.randn((5, 64), device="cuda")
    want = ramnet.norm_gate(x)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream, Wrapped(s)):
        y = ramnet.norm_gate(x, stream=stream)
        assert _owner(y) == [s.cuda_stream]
        s.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("shape", [(4, 2048, 16, 128, 128), (2, 300, 4, 64, 64), (2, 1500, 6, 32, 16), (3, 130, 5, 128, 32),
                                   (8, 256, 32, 32, 128)], ids=str)
def test_waits_that_run_out_are_reported_and_the_context_survives(shape):
    """A prompt on the tensor cores with limits on its waits that its hand-overs outlast (on purpose; nothing is lost on the
    device).  Below 4 us every wait gives up at once; at one to three polls of 4 us those do that take longer, with copies and
    products in flight, or none.  The kernels end by themselves, with RAMNET_ERR_TIMEOUT recorded if any gave up and the
    usual bits if none did; nothing outside the outputs is written, and a call with the default limit then gives its usual bits."""
    B, T, H, P, N = shape
    cfg = ramnet.SsmConfig(H=H, G=1, N=N, P=P)
    L = _operands(B, T, H, 1, N, P, BF)
    lengths = torch.tensor(([T, T - 37, 70, T] * 2)[:B], dtype=torch.int32).cuda()
    y0, S0 = (torch.full((B, T, H, P), 5.0, dtype=BF, device="cuda"), torch.zeros((B, H, N, P), device="cuda"))
    ramnet.ssm_forward(cfg, **L, lengths=lengths, y=y0, S_out=S0)
    ramnet.sync_status()
    guard = torch.full((3, B, T, H, P), 5.0, dtype=BF, device="cuda")  # y lies between values that are nobody's to write
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for limit in (1, 3, 4, 8, 12, 4, 1):
        other.zero_()  # inputs come from memory, not from L2
        guard[1] = 5.0
        t0 = time.perf_counter()
        ramnet.set_scan_wait_limit(limit)
        try:
            _, S = ramnet.ssm_forward(cfg, **L, lengths=lengths, y=guard[1])
            if limit < 4:
                with pytest.raises(ramnet.RamnetError) as e:
                    ramnet.sync_status()
                assert e.value.status == ramnet.RAMNET_ERR_TIMEOUT
            else:
                try:
                    ramnet.sync_status()
                    assert torch.equal(guard[1], y0) and torch.equal(S, S0)
                except ramnet.RamnetError as e:
                    assert e.status == ramnet.RAMNET_ERR_TIMEOUT
                    print("gave up at", limit, "us")
        finally:
            ramnet.set_scan_wait_limit(0)
        assert time.perf_counter() - t0 < 5.0
        ramnet.sync_status()  # cleared
        assert bool((guard[0] == 5.0).all()) and bool((guard[2] == 5.0).all())
        for b in range(B):
            assert bool((guard[1, b, int(lengths[b]):] == 5.0).all())
        y, S = torch.full_like(y0, 5.0), torch.zeros_like(S0)
        ramnet.ssm_forward(cfg, **L, lengths=lengths, y=y, S_out=S)
        ramnet.sync_status()
        assert torch.equal(y, y0) and torch.equal(S, S0)
