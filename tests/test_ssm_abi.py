"""Host-side refusals of the state space layer's entry points, and of their Python binding (no GPU needed)."""
import copy
import ctypes
import dataclasses
import io
import pickle

import pytest
import torch

from sparse_slot_recurrent_b200 import build as build_mod
from sparse_slot_recurrent_b200 import ramnet

FAKE = 1 << 40  # 16-byte aligned, never dereferenced: every call below fails host-side
BF, F = ramnet.RAMNET_BF16, ramnet.RAMNET_F32
BAD = ramnet.RAMNET_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return ramnet.load()


def _cfg(**kw):
    return ramnet.SsmConfig(**{**dict(H=4, G=2, N=64, P=64), **kw})


def _strides(*v):
    return None if v[0] is None else ctypes.pointer(ramnet._Strides(*v))


def _fwd(lib, cfg=None, B=2, T=100, dt=BF, x=FAKE, xs=None, dt_ptr=FAKE, A=FAKE, Bm=FAKE, Cm=FAKE, D=None, bias=None,
         lengths=None, S_in=None, y=FAKE, od=BF, S_out=FAKE, ws=FAKE, nbytes=1 << 40):
    ref = (cfg or _cfg())._ref
    return lib.ramnet_ssm_forward(ref, B, T, dt, x, xs, dt_ptr, None, A, Bm, None, Cm, None, D, bias, lengths, S_in, y, od,
                                  S_out, ws, nbytes, None)


@pytest.mark.parametrize("kw", [dict(N=48), dict(N=0), dict(P=8), dict(P=512), dict(G=3), dict(G=0), dict(H=0),
                                dict(dt_min=1.0, dt_max=0.5), dict(dt_min=float("nan"))], ids=str)
def test_bad_layers_refused(lib, kw):
    assert _fwd(lib, _cfg(**kw)) == BAD
    assert ramnet.last_error() != ""
    assert ramnet.ssm_workspace_bytes(_cfg(**kw), 2, 100) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(B=0), "B"), (dict(T=0), "T"), (dict(B=1 << 30, T=1 << 30), "large"), (dict(cfg=_cfg(H=1, G=1), B=1, T=(1 << 30) + 1), "large"),
    (dict(dt=7), "dtype"), (dict(od=9), "dtype"),
    (dict(x=None), "x"), (dict(x=FAKE + 1), "aligned"), (dict(dt_ptr=None), "dt"), (dict(A=None), "A"), (dict(A=FAKE + 2), "A"),
    (dict(Bm=None), "Bm"), (dict(Cm=None), "Cm"), (dict(Cm=FAKE + 3), "Cm"), (dict(D=FAKE + 2), "D"), (dict(bias=FAKE + 1), "bias"),
    (dict(lengths=FAKE + 2), "lengths"), (dict(S_in=FAKE + 4), "S_in"), (dict(y=None), "y"), (dict(y=FAKE + 8), "y"),
    (dict(S_out=None), "S_out"), (dict(S_out=FAKE + 4), "S_out"), (dict(xs=_strides(100, -1, 64)), "strides"),
    (dict(xs=_strides(1 << 62, 1, 64)), "strides")], ids=str)
def test_bad_scan_arguments_refused(lib, kw, word):
    assert _fwd(lib, **kw) == BAD
    assert word in ramnet.last_error()


def test_null_layer_refused(lib):
    assert lib.ramnet_ssm_forward(None, 1, 1, BF, *([FAKE, None] * 2), FAKE, *([FAKE, None] * 2), None, None, None, None, FAKE, BF,
                                  FAKE, FAKE, 1 << 40, None) == BAD
    assert "cfg" in ramnet.last_error()


def _step(lib, cfg=None, B=2, dt=BF, x=FAKE, S=FAKE, y=FAKE, od=BF, A=FAKE):
    return lib.ramnet_ssm_step((cfg or _cfg())._ref, B, dt, x, None, FAKE, None, A, FAKE, None, FAKE, None, None, None, S, y, od,
                               None)


def test_bad_step_arguments_refused(lib):
    for kw in (dict(cfg=_cfg(N=3)), dict(B=0), dict(dt=5), dict(od=5), dict(x=None), dict(x=FAKE + 1), dict(S=None), dict(S=FAKE + 8),
               dict(y=FAKE + 2), dict(y=None), dict(A=None)):
        assert _step(lib, **kw) == BAD, kw


def _conv(lib, B=2, T=9, C=8, W=4, dt=BF, x=FAKE, xb=72, xt=8, w=FAKE, bias=None, lengths=None, si=None, y=FAKE, od=BF, so=None):
    return lib.ramnet_conv_forward(B, T, C, W, dt, x, xb, xt, w, bias, 1, lengths, si, y, od, so, None)


def test_bad_conv_arguments_refused(lib):
    for kw in (dict(B=0), dict(T=0), dict(C=0), dict(W=1), dict(W=5), dict(dt=3), dict(od=3), dict(x=None), dict(x=FAKE + 1),
               dict(xb=-1), dict(xt=-8), dict(w=None), dict(w=FAKE + 2), dict(bias=FAKE + 1), dict(lengths=FAKE + 1),
               dict(si=FAKE + 2), dict(so=FAKE + 4), dict(y=None), dict(y=FAKE + 4), dict(B=1 << 20, C=1 << 20),
               dict(B=1 << 16, T=1 << 16), dict(B=1 << 10, T=1 << 20, C=1 << 20),
               dict(B=1, T=(1 << 30) + 1, C=1)):
        assert _conv(lib, **kw) == BAD, kw
    step = lambda B=2, C=8, W=4, dt=BF, x=FAKE, xb=8, w=FAKE, st=FAKE, y=FAKE, od=BF: lib.ramnet_conv_step(  # noqa: E731
        B, C, W, dt, x, xb, w, None, 1, st, y, od, None)
    for kw in (dict(B=0), dict(C=0), dict(W=1), dict(W=5), dict(dt=3), dict(od=3), dict(x=None), dict(xb=-1), dict(w=None),
               dict(st=None), dict(st=FAKE + 2), dict(y=None), dict(y=FAKE + 2)):
        assert step(**kw) == BAD, kw


def test_bad_norm_arguments_refused(lib):
    norm = lambda R=4, D=64, groups=2, dt=BF, x=FAKE, xr=64, z=FAKE, zr=64, w=FAKE, eps=1e-6, y=FAKE, od=BF: lib.ramnet_norm_gate(  # noqa: E731
        R, D, groups, dt, x, xr, z, zr, w, eps, 1, y, od, None)
    for kw in (dict(R=0), dict(D=0), dict(groups=0), dict(groups=3), dict(dt=4), dict(od=4), dict(x=None), dict(x=FAKE + 1), dict(xr=-1),
               dict(z=FAKE + 1), dict(zr=-4), dict(w=FAKE + 4), dict(eps=-1.0), dict(eps=float("nan")), dict(y=None), dict(y=FAKE + 2),
               dict(R=1 << 31), dict(R=1, D=(1 << 30) + 2)):
        assert norm(**kw) == BAD, kw


def test_binding_refuses_what_the_kernels_would_misread():
    cfg = _cfg()
    x, dt, A = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 4), torch.zeros(4)
    Bm = torch.zeros(2, 5, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ramnet.ssm_forward(cfg, x, dt, A, Bm, Bm)
    with pytest.raises(TypeError, match="dtype"):
        ramnet.ssm_forward(cfg, x.half(), dt, A, Bm, Bm)
    with pytest.raises(ValueError, match="CUDA"):
        ramnet.conv_forward(torch.zeros(1, 2, 3), torch.zeros(3, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ramnet.norm_gate(torch.zeros(2, 8))


@pytest.mark.gpu
def test_binding_checks_shapes_types_and_devices():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    cfg = _cfg()
    f = dict(device="cuda")
    x, dt, A, Bm = torch.zeros(2, 5, 4, 64, **f), torch.zeros(2, 5, 4, **f), torch.zeros(4, **f), torch.zeros(2, 5, 2, 64, **f)
    for args, err in (((x[:, :, :3], dt, A, Bm, Bm), ValueError), ((x, dt[:, :4], A, Bm, Bm), ValueError),
                      ((x, dt, A.double(), Bm, Bm), TypeError), ((x, dt, A.cpu(), Bm, Bm), ValueError),
                      ((x, dt, A, Bm[:, :, :1], Bm), ValueError), ((x, dt, A, Bm.bfloat16(), Bm), TypeError),
                      ((x.transpose(2, 3), dt, A, Bm, Bm), ValueError), ((x, dt, A[::2], Bm, Bm), ValueError)):
        with pytest.raises(err):
            ramnet.ssm_forward(cfg, *args)
    with pytest.raises(TypeError):
        ramnet.ssm_forward(cfg, x, dt, A, Bm, Bm, lengths=torch.zeros(2, dtype=torch.int64, **f))
    with pytest.raises(ValueError):
        ramnet.ssm_forward(cfg, x, dt, A, Bm, Bm, S_in=torch.zeros(2, 4, 64, 65, **f))
    with pytest.raises(ValueError):
        ramnet.conv_step(torch.zeros(2, 8, **f), torch.zeros(8, 4, **f), torch.zeros(2, 4, 8, **f))
    with pytest.raises(ramnet.RamnetError):
        ramnet.conv_step(torch.zeros(2, 8, **f), torch.zeros(8, 5, **f), torch.zeros(2, 4, 8, **f))
    with pytest.raises(ramnet.RamnetError):
        ramnet.norm_gate(torch.zeros(2, 8, **f), groups=3)


# ------------------------------------------------------------------ sizes that the library's 32-bit arguments do not hold

HUGE = (1 << 32) + 5  # 5 in 32 bits


def _wide(*shape, dtype=torch.bfloat16):
    return torch.zeros((1,) * len(shape), dtype=dtype).expand(shape)


@pytest.mark.parametrize("name,call", [
    ("T", lambda: ramnet.conv_forward(_wide(1, HUGE, 1), torch.zeros(1, 4))),
    ("B", lambda: ramnet.conv_forward(_wide(HUGE, 1, 1), torch.zeros(1, 4))),
    ("C", lambda: ramnet.conv_forward(_wide(1, 1, HUGE), _wide(HUGE, 4, dtype=torch.float32))),
    ("W", lambda: ramnet.conv_forward(_wide(1, 3, 1), _wide(1, HUGE, dtype=torch.float32))),
    ("B", lambda: ramnet.conv_step(_wide(HUGE, 1), torch.zeros(1, 4), _wide(HUGE, 3, 1))),
    ("C", lambda: ramnet.conv_step(_wide(1, HUGE), _wide(HUGE, 4, dtype=torch.float32), _wide(1, 3, HUGE))),
    ("W", lambda: ramnet.conv_step(_wide(1, 1), _wide(1, HUGE, dtype=torch.float32), _wide(1, HUGE - 1, 1))),
    ("D", lambda: ramnet.norm_gate(_wide(1, HUGE))),
    ("groups", lambda: ramnet.norm_gate(_wide(1, 5), groups=HUGE)),
    ("groups", lambda: ramnet.norm_gate(_wide(1, 5), groups=1 - (1 << 32))),
    ("T", lambda: ramnet.ssm_forward(_cfg(), _wide(1, HUGE, 4, 64), _wide(1, HUGE, 4), torch.zeros(4), _wide(1, HUGE, 2, 64), _wide(1, HUGE, 2, 64))),
    ("B", lambda: ramnet.ssm_forward(_cfg(), _wide(HUGE, 2, 4, 64), _wide(HUGE, 2, 4), torch.zeros(4), _wide(HUGE, 2, 2, 64), _wide(HUGE, 2, 2, 64))),
    ("B", lambda: ramnet.ssm_step(_cfg(), _wide(HUGE, 4, 64), _wide(HUGE, 4), torch.zeros(4), _wide(HUGE, 2, 64), _wide(HUGE, 2, 64),
                                  _wide(HUGE, 4, 64, 64, dtype=torch.float32))),
    ("T", lambda: ramnet.ssm_workspace_bytes(_cfg(), 1, (1 << 32) + 64)),
    ("B", lambda: ramnet.ssm_workspace_bytes(_cfg(), HUGE, 64)),
    ("H", lambda: _cfg(H=(1 << 32) + 4)),
    ("N", lambda: _cfg(N=64 - (1 << 32))),
    ("d_p", lambda: ramnet.Config(d_p=(1 << 32) + 4, U=2, K=4, d_v=64)),
    ("K", lambda: ramnet.Config(d_p=4, U=2, K=(1 << 32) + 4, d_v=64)),
    ("T", lambda: ramnet.scan_workspace_bytes(_SLOTS, 1, HUGE, 1)),
    ("T", lambda: ramnet.decode_addresses(_SLOTS, _wide(1, HUGE, 1, 8), idx_out=torch.zeros(1), w_out=torch.zeros(1))),
    ("T", lambda: ramnet.scan_forward_host_scratch_bytes(_SLOTS, 1, HUGE, 1, torch.bfloat16, torch.float32, 2)),
    ("limit_us", lambda: ramnet.set_scan_wait_limit((1 << 32) + 5)),
    ("limit_us", lambda: ramnet.selftest_wait_timeout((1 << 32) + 5)),
], ids=lambda v: v if isinstance(v, str) else "")
def test_sizes_past_32_bits_refused_by_the_binding(lib, name, call):
    """... and not cut to their low 32 bits: the library would see a small size that passes its checks."""
    with pytest.raises(ramnet.RamnetError, match=f"{name}=") as e:
        call()
    assert e.value.status == BAD
    assert ramnet.set_scan_wait_limit(0) is None


_SLOTS = ramnet.Config(d_p=4, U=2, K=4, d_v=64)


@pytest.mark.parametrize("cfg", [ramnet.SsmConfig(H=6, G=3, N=32, P=128, dt_softplus=False, dt_min=0.001, dt_max=0.5),
                                 ramnet.Config(d_p=4, U=2, K=4, d_v=64)], ids=["ssm", "slots"])
def test_configurations_are_copied_and_pickled(lib, cfg):
    """A layer that holds one is deep-copied, saved and sent to worker processes."""
    for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), dataclasses.replace(cfg)):
        assert other == cfg and hash(other) == hash(cfg) and repr(other) == repr(cfg)
        if isinstance(cfg, ramnet.SsmConfig):
            a, b = other._ref.contents, cfg._ref.contents
            assert ctypes.addressof(a) != ctypes.addressof(b)
            assert [getattr(a, f[0]) for f in a._fields_] == [getattr(b, f[0]) for f in b._fields_] == [6, 3, 32, 128, 0, b.dt_min, 0.5]
            assert ramnet.ssm_workspace_bytes(other, 2, 100) == ramnet.ssm_workspace_bytes(cfg, 2, 100) > 0
    saved = io.BytesIO()
    torch.save({"cfg": cfg}, saved)
    saved.seek(0)
    assert torch.load(saved, weights_only=False)["cfg"] == cfg


@pytest.mark.parametrize("H,G,P", [((1 << 22) + 1, 1, 256), (1 << 23, 1 << 20, 256), ((1 << 26) + 3, 1, 16), (1 << 27, 2, 16)])
def test_tokens_of_too_many_channels_refused(lib, H, G, P):
    """Channels of a token are counted in 32 bits, up to a block past their end."""
    cfg = _cfg(H=H, G=G, N=16, P=P)
    assert _fwd(lib, cfg, B=1, T=1) == BAD
    assert "large" in ramnet.last_error()
    assert ramnet.ssm_workspace_bytes(cfg, 1, 1) == 0
    assert ramnet.ssm_workspace_bytes(_cfg(H=(1 << 30) // P, G=1, N=16, P=P), 1, 1) > 0
