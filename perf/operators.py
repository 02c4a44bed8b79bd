"""Workloads of the state space layer's operators: the short causal convolution and the selective scan, each for prompts and for
single tokens, and the gated row norm behind them.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, through the
framework's entry points.  Shapes follow the framework's workloads: B8 H8 T4096 and B4 H16 T16384 prompts and 256 sequences of 16
heads for single tokens, 128 channels per head.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a long-context prompt of the larger layer (4 sequences x 16384 tokens x 16 heads of 128)
        {"name": "scan long prompt", "op": "scan", "B": 4, "T": 16384, "H": 16, "P": 128, "N": 128, "G": 1, "dtype": "bf16",
         "ragged": False, "carry": False},
        # a batch of prompts of the smaller layer
        {"name": "scan prompts", "op": "scan", "B": 8, "T": 4096, "H": 8, "P": 128, "N": 128, "G": 1, "dtype": "bf16",
         "ragged": False, "carry": False},
        # turns of a conversation: ragged lengths behind a carried state, narrow heads in two groups
        {"name": "scan ragged turns", "op": "scan", "B": 6, "T": 1021, "H": 24, "P": 64, "N": 64, "G": 2, "dtype": "bf16",
         "ragged": True, "carry": True},
        # a short fp32 prompt, as used to check a layer
        {"name": "scan fp32", "op": "scan", "B": 2, "T": 333, "H": 5, "P": 32, "N": 16, "G": 5, "dtype": "f32",
         "ragged": False, "carry": True},
        # one token of each of 256 sequences
        {"name": "scan tokens", "op": "scan_step", "B": 256, "H": 16, "P": 128, "N": 128, "G": 1, "dtype": "bf16"},
        # one token of one sequence: latency
        {"name": "scan one token", "op": "scan_step", "B": 1, "H": 24, "P": 64, "N": 64, "G": 2, "dtype": "f32"},
        # the convolution in front of the long prompt's scan: x, B and C of all heads
        {"name": "conv long prompt", "op": "conv", "B": 4, "T": 16384, "C": 2304, "W": 4, "dtype": "bf16", "ragged": False,
         "carry": False},
        # ragged fp32 turns with an odd channel count
        {"name": "conv ragged turns", "op": "conv", "B": 5, "T": 777, "C": 1043, "W": 3, "dtype": "f32", "ragged": True,
         "carry": True},
        # the convolution for one token of each of 256 sequences, and of one
        {"name": "conv tokens", "op": "conv_step", "B": 256, "C": 2304, "W": 4, "dtype": "bf16"},
        {"name": "conv one token", "op": "conv_step", "B": 1, "C": 1043, "W": 4, "dtype": "f32"},
        # the gated norm behind the long prompt's scan, all 16 heads in one norm
        {"name": "norm long prompt", "op": "norm", "R": 65536, "D": 2048, "groups": 1, "gate": True, "first": True, "dtype": "bf16"},
        # the gated norm of 256 single tokens, one norm per group of heads, gate behind the norm
        {"name": "norm tokens", "op": "norm", "R": 256, "D": 1536, "groups": 2, "gate": True, "first": False, "dtype": "f32"},
    ]


def _size(rng, lo, hi):
    """A size from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_step", "conv", "conv_step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "scan_step"):
        P = rng.choice([16, 32, 64, 64, 128, 128])
        N = rng.choice([16, 32, 64, 128, 128, 256])
        G = rng.choice([1, 1, 2, 3])
        H = G * _size(rng, 1, 24)
        if op == "scan_step":
            B = max(1, min(_size(rng, 1, 512), (256 * 16 * 128 * 128) // (H * P * N)))
            return {"op": op, "B": B, "H": H, "P": P, "N": N, "G": G, "dtype": dtype}
        B = rng.randint(1, 8)
        most = (4 * 16384 * 16 * 128 * 128) // (B * H * P * N)
        T = _size(rng, 1, max(1, min(16384, most)))
        return {"op": op, "B": B, "T": T, "H": H, "P": P, "N": N, "G": G, "dtype": dtype, "ragged": rng.random() < 0.5,
                "carry": rng.random() < 0.5}
    if op == "conv":
        B, C = rng.randint(1, 8), _size(rng, 16, 4600)
        T = _size(rng, 1, max(1, min(16384, (4 * 16384 * 2304) // (2 * B * C))))
        return {"op": op, "B": B, "T": T, "C": C, "W": rng.choice([2, 3, 4, 4]), "dtype": dtype, "ragged": rng.random() < 0.5,
                "carry": rng.random() < 0.5}
    if op == "conv_step":
        return {"op": op, "B": _size(rng, 1, 512), "C": _size(rng, 16, 4600), "W": rng.choice([2, 3, 4, 4]), "dtype": dtype}
    groups = rng.choice([1, 1, 2, 4])
    D = groups * _size(rng, 16, 2048)
    return {"op": op, "R": _size(rng, 1, max(1, min(65536, (65536 * 2048) // (2 * D)))), "D": D, "groups": groups,
            "gate": rng.random() < 0.8, "first": rng.random() < 0.5, "dtype": dtype}


def _layer(case, gen, shape):
    """Inputs and parameters of a scan: x, B and C lie side by side, as the convolution writes them."""
    H, P, N, G, t = case["H"], case["P"], case["N"], case["G"], DTYPES[case["dtype"]]
    f = dict(generator=gen, device="cuda", dtype=torch.float32)
    xbc = torch.nn.functional.silu(torch.randn((*shape, H * P + 2 * G * N), **f)).to(t)
    x = xbc[..., :H * P].unflatten(-1, (H, P))
    Bm = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    Cm = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
    # step sizes log-uniform over 0.001 to 0.1 through the softplus, decay rates from 1 to 16
    base = torch.exp(torch.rand((H,), **f) * 4.6 - 6.9)
    s = {"x": x, "Bm": Bm, "Cm": Cm, "dt": (torch.randn((*shape, H), **f) * 0.5).to(t), "A": -(1 + 15 * torch.rand((H,), **f)),
         "D": torch.rand((H,), **f) + 0.5, "dt_bias": torch.log(torch.expm1(base))}
    return s


def _lengths(case, gen):
    """Lengths from none to all of T, the first sequence whole, or None."""
    if not case["ragged"]:
        return None
    n = torch.randint(0, case["T"] + 1, (case["B"],), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = case["T"]
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, t = case["op"], DTYPES[case["dtype"]]
    f = dict(generator=gen, device="cuda", dtype=torch.float32)
    if op == "scan":
        B, T, H, P, N = (case[k] for k in "BTHPN")
        s = _layer(case, gen, (B, T))
        s["S_in"] = torch.randn((B, H, N, P), **f) if case["carry"] else None
        s["lengths"] = _lengths(case, gen)
        s["y"] = torch.zeros((B, T, H, P), dtype=t, device="cuda")  # rows behind a sequence stay as they are
        s["S_out"] = torch.empty((B, H, N, P), dtype=torch.float32, device="cuda")
    elif op == "scan_step":
        s = _layer(case, gen, (case["B"],))
        s["S"] = torch.randn((case["B"], case["H"], case["N"], case["P"]), **f)
    elif op == "conv":
        B, T, C, W = (case[k] for k in "BTCW")
        # one projection writes the gate, the convolution's input and the step sizes side by side
        wide = torch.randn((B, T, 2 * C), **f).to(t)
        s = {"x": wide[..., C:], "w": torch.randn((C, W), **f) / W ** 0.5, "bias": 0.1 * torch.randn((C,), **f)}
        s["state_in"] = torch.randn((B, W - 1, C), **f).to(t) if case["carry"] else None
        s["lengths"] = _lengths(case, gen)
        s["y"] = torch.zeros((B, T, C), dtype=t, device="cuda")
        s["state_out"] = torch.empty((B, W - 1, C), dtype=t, device="cuda")
    elif op == "conv_step":
        B, C, W = (case[k] for k in "BCW")
        wide = torch.randn((B, 2 * C), **f).to(t)
        s = {"x": wide[:, C:], "w": torch.randn((C, W), **f) / W ** 0.5, "bias": 0.1 * torch.randn((C,), **f),
             "state": torch.randn((B, W - 1, C), **f).to(t)}
    else:
        R, D = case["R"], case["D"]
        s = {"x": torch.randn((R, D), **f).to(t), "w": 1 + 0.1 * torch.randn((D,), **f),
             "z": torch.randn((R, 2 * D), **f).to(t)[:, :D] if case["gate"] else None}
    s["case"] = case
    if own:
        from sparse_slot_recurrent_b200 import ramnet
        s["ramnet"] = ramnet
        if op in ("scan", "scan_step"):
            s["cfg"] = ramnet.SsmConfig(H=case["H"], G=case["G"], N=case["N"], P=case["P"])
        if op == "scan":
            need = ramnet.ssm_workspace_bytes(s["cfg"], case["B"], case["T"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


def _silu(v):
    return v / (1 + torch.exp(-v))


def _step_sizes(dt, bias):
    """softplus(dt + bias) in 64 bits."""
    v = dt.double() + bias.double()
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _valid(lengths, B, T, device):
    """[B,T] truth values: the tokens that a sequence has."""
    t = torch.arange(T, device=device)
    return (t < lengths[:, None]) if lengths is not None else (t >= 0).expand(B, T)


def _decay_between(total):
    """exp of the sums of total[..., k] over j <= k < i, for i >= j, else 0: [..., n] -> [..., n+1, n+1]."""
    c = torch.cat([torch.zeros_like(total[..., :1]), torch.cumsum(total, -1)], -1)
    n = c.shape[-1]
    low = torch.ones((n, n), dtype=torch.bool, device=c.device).tril()
    return torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~low, -torch.inf))


def _plain_scan(x, dt, A, Bm, Cm, D, dt_bias, S_in, lengths, y, S_out):
    """The scan by blocks of 64 tokens: products within a block, the state between blocks; 32 bits, the decays' sums in 64."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    Q, R = 64, H // G
    n = (T + Q - 1) // Q
    ok = _valid(lengths, B, T, x.device)
    pad = lambda v: torch.cat([v, v.new_zeros((B, n * Q - T, *v.shape[2:]))], 1).unflatten(1, (n, Q))  # noqa: E731
    d = torch.where(ok[..., None], _step_sizes(dt, dt_bias), 0)  # a token that is not there neither decays nor writes
    xf = torch.where(ok[..., None, None], x, 0).float()
    d, xq = pad(d), pad(xf).unflatten(3, (G, R))  # [B,n,Q,H], [B,n,Q,G,R,P]
    bq = pad(torch.where(ok[..., None, None], Bm, 0).float())
    cq = pad(torch.where(ok[..., None, None], Cm, 0).float())  # [B,n,Q,G,N]
    cum = torch.cumsum(d * A.double(), 2).movedim(2, 3)  # [B,n,H,Q]
    low = torch.ones((Q, Q), dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -torch.inf)).float()  # [B,n,H,Q,Q]
    df = d.float()
    scores = torch.matmul(cq.movedim(3, 2), bq.movedim(3, 2).transpose(-1, -2))  # [B,n,G,Q,Q]
    w = scores[:, :, :, None] * decay.unflatten(2, (G, R)) * df.movedim(2, 3).unflatten(2, (G, R))[..., None, :]
    inside = torch.matmul(w, xq.movedim(2, 4))  # [B,n,G,R,Q,P]
    left = (torch.exp(cum[..., -1:] - cum) * d.movedim(2, 3)).float().unflatten(2, (G, R))  # [B,n,G,R,Q]
    wrote = torch.matmul(bq.movedim(3, 2).transpose(-1, -2)[:, :, :, None], left[..., None] * xq.movedim(2, 4))  # [B,n,G,R,N,P]
    first = torch.zeros((B, H, N, P), device=x.device) if S_in is None else S_in
    states = torch.cat([first.unflatten(1, (G, R))[:, None], wrote], 1)  # [B,n+1,G,R,N,P]
    between = _decay_between(cum[..., -1].movedim(1, 2)).float()  # [B,H,n+1,n+1]
    carried = torch.matmul(between, states.movedim(1, 3).flatten(4).flatten(1, 2))  # [B,H,n+1,N*P]
    carried = carried.unflatten(-1, (N, P)).unflatten(1, (G, R)).movedim(3, 1)  # [B,n+1,G,R,N,P]
    before = torch.matmul(cq.movedim(3, 2)[:, :, :, None], carried[:, :-1])  # [B,n,G,R,Q,P]
    out = inside + before * torch.exp(cum).float().unflatten(2, (G, R))[..., None]
    out = out.movedim(4, 2).flatten(3, 4).flatten(1, 2)[:, :T] + D[:, None] * xf
    y.copy_(torch.where(ok[..., None, None], out.to(y.dtype), y))
    S_out.copy_(carried[:, -1].flatten(1, 2))
    return y, S_out


def _plain_scan_step(x, dt, A, Bm, Cm, D, dt_bias, S):
    R = x.shape[1] // Bm.shape[1]
    d = _step_sizes(dt, dt_bias)
    b, c = (v.float().repeat_interleave(R, 1) for v in (Bm, Cm))  # [B,H,N]
    xf = x.float()
    S.mul_(torch.exp(d * A.double()).float()[..., None, None]).add_((d.float()[..., None] * b)[..., None] * xf[:, :, None, :])
    out = (c[..., None] * S).sum(2) + D[:, None] * xf
    return out.to(x.dtype), S


def _plain_conv(x, w, bias, state_in, lengths, y, state_out):
    B, T, C = x.shape
    W = w.shape[1]
    ok = _valid(lengths, B, T, x.device)
    head = x.new_zeros((B, W - 1, C)) if state_in is None else state_in
    full = torch.cat([head, x], 1)  # [B,T+W-1,C]
    acc = sum(full[:, k:k + T].float() * w[:, k] for k in range(W)) + bias
    y.copy_(torch.where(ok[..., None], _silu(acc).to(y.dtype), y))
    n = lengths.long() if lengths is not None else torch.full((B,), T, device=x.device)
    at = n[:, None] + torch.arange(W - 1, device=x.device)
    state_out.copy_(torch.gather(full, 1, at[..., None].expand(-1, -1, C)))
    return y, state_out


def _plain_conv_step(x, w, bias, state):
    full = torch.cat([state, x[:, None]], 1)  # [B,W,C]
    y = _silu((full.float() * w.t()).sum(1) + bias).to(x.dtype)
    state.copy_(full[:, 1:])
    return y, state


def _plain_norm(x, z, w, groups, first, eps):
    u = x.float()
    gate = None if z is None else _silu(z.float())
    if first and gate is not None:
        u = u * gate
    v = u.unflatten(-1, (groups, -1))
    v = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)).flatten(-2) * w
    if not first and gate is not None:
        v = v * gate
    return v.to(x.dtype)


EPS = 1e-6


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        r = s["ramnet"]
        if op == "scan":
            return r.ssm_forward(s["cfg"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], dt_bias=s["dt_bias"],
                                 lengths=s["lengths"], S_in=s["S_in"], y=s["y"], S_out=s["S_out"], workspace=s["workspace"])
        if op == "scan_step":
            y = r.ssm_step(s["cfg"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["S"], D=s["D"], dt_bias=s["dt_bias"],
                           out_dtype=s["x"].dtype)
            return y, s["S"]
        if op == "conv":
            return r.conv_forward(s["x"], s["w"], bias=s["bias"], silu=True, lengths=s["lengths"], state_in=s["state_in"],
                                  y=s["y"], state_out=s["state_out"])
        if op == "conv_step":
            return r.conv_step(s["x"], s["w"], s["state"], bias=s["bias"], silu=True, out_dtype=s["x"].dtype), s["state"]
        return r.norm_gate(s["x"], z=s["z"], w=s["w"], groups=case["groups"], eps=EPS, gate_first=case["first"],
                           out_dtype=s["x"].dtype)
    if op == "scan":
        return _plain_scan(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["dt_bias"], s["S_in"], s["lengths"], s["y"],
                           s["S_out"])
    if op == "scan_step":
        return _plain_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["dt_bias"], s["S"])
    if op == "conv":
        return _plain_conv(s["x"], s["w"], s["bias"], s["state_in"], s["lengths"], s["y"], s["state_out"])
    if op == "conv_step":
        return _plain_conv_step(s["x"], s["w"], s["bias"], s["state"])
    return _plain_norm(s["x"], s["z"], s["w"], case["groups"], case["first"], EPS)


def exact(case, seed):
    """The definitions, token by token, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "scan_step"):
        one = op == "scan_step"
        lift = (lambda v: v[:, None]) if one else (lambda v: v)
        x, dt, Bm, Cm = (lift(s[k]).double() for k in ("x", "dt", "Bm", "Cm"))
        A, D, bias = (s[k].double() for k in ("A", "D", "dt_bias"))
        B, T, H, P = x.shape
        G, N = Bm.shape[2:]
        S0 = s["S"] if one else s["S_in"]
        S = torch.zeros((B, G, H // G, N, P), dtype=torch.float64, device="cuda") if S0 is None else \
            S0.double().reshape(B, G, H // G, N, P).clone()
        step = torch.log(1 + torch.exp(dt + bias))
        a = torch.exp(step * A).reshape(B, T, G, H // G)
        u = (step[..., None] * x).reshape(B, T, G, H // G, P)
        n = None if one or s["lengths"] is None else s["lengths"].tolist()
        y = torch.zeros((B, T, G, H // G, P), dtype=torch.float64, device="cuda")
        if n is None:
            for t in range(T):
                S.mul_(a[:, t, :, :, None, None]).addcmul_(Bm[:, t, :, None, :, None], u[:, t, :, :, None, :])
                torch.matmul(Cm[:, t, :, None, None, :], S, out=(o := torch.empty((B, G, H // G, 1, P), dtype=torch.float64,
                                                                                  device="cuda")))
                y[:, t] = o[..., 0, :]
        else:
            for b in range(B):
                for t in range(n[b]):
                    S[b].mul_(a[b, t, :, :, None, None]).addcmul_(Bm[b, t, :, None, :, None], u[b, t, :, :, None, :])
                    y[b, t] = torch.matmul(Cm[b, t, :, None, None, :], S[b])[..., 0, :]
        y = y.reshape(B, T, H, P) + D[:, None] * x
        if n is not None:
            for b in range(B):
                y[b, n[b]:] = 0
        return (y[:, 0] if one else y), S.reshape(B, H, N, P)
    if op in ("conv", "conv_step"):
        one = op == "conv_step"
        x = s["x"][:, None] if one else s["x"]
        W, (B, T, C) = case["W"], x.shape
        old = s["state"] if one else s["state_in"]
        n = [T] * B if one or s["lengths"] is None else s["lengths"].tolist()
        y = torch.zeros((B, T, C), dtype=torch.float64, device="cuda")
        kept = torch.zeros((B, W - 1, C), dtype=torch.float64, device="cuda")
        for b in range(B):
            before = torch.zeros((W - 1, C), dtype=torch.float64, device="cuda") if old is None else old[b].double()
            full = torch.cat([before, x[b, :n[b]].double()])
            kept[b] = full[n[b]:]
            v = (full.unfold(0, W, 1) * s["w"].double()).sum(-1) + s["bias"].double()
            y[b, :n[b]] = v * torch.sigmoid(v)
        return (y[:, 0] if one else y), kept
    x, w = s["x"].double(), s["w"].double()
    g = 1.0 if s["z"] is None else s["z"].double() * torch.sigmoid(s["z"].double())
    u = (x * g if case["first"] else x).reshape(case["R"], case["groups"], -1)
    u = (u * torch.rsqrt(u.pow(2).mean(-1, keepdim=True) + EPS)).reshape(case["R"], -1) * w
    return u if case["first"] else u * g


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("scan", "scan_step"):
        B, H, P, N, G = (case[k] for k in "BHPNG")
        T = case.get("T", 1)
        state = B * H * N * P * 4
        moved = B * T * (2 * H * P + 2 * G * N + H) * es + state * (2 if op == "scan_step" or case["carry"] else 1) + 12 * H
        return {"bytes": moved, "flops": 5 * B * T * H * N * P}  # per state value: decay, write (2), read (2)
    if op in ("conv", "conv_step"):
        B, C, W = case["B"], case["C"], case["W"]
        T = case.get("T", 1)
        state = B * (W - 1) * C * es
        return {"bytes": 2 * B * T * C * es + state * (2 if op == "conv_step" or case["carry"] else 1) + C * (W + 1) * 4,
                "flops": B * T * C * (2 * W + 4)}
    R, D = case["R"], case["D"]
    return {"bytes": R * D * es * (3 if case["gate"] else 2) + 4 * D, "flops": R * D * (9 if case["gate"] else 4)}
