"""Thin Python binding of the RAM-Net C ABI (``include/ramnet.h``).

Argument marshalling only: torch supplies device memory and the current CUDA stream;
every step of the layer runs in the library's kernels.  The library is loaded from the
package directory (``libramnet.so``, built by ``build.py``; with the environment variable
RAMNET_DEBUG=1 the range-checking build ``libramnet_debug.so``); if it is missing or fails
to load, every call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass, fields

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
DEBUG = os.environ.get("RAMNET_DEBUG", "0") not in ("", "0")
LIB_PATH = os.path.join(_PKG, "libramnet_debug.so" if DEBUG else "libramnet.so")

RAMNET_OK, RAMNET_ERR_INVALID_ARG, RAMNET_ERR_UNSUPPORTED, RAMNET_ERR_CUDA, RAMNET_ERR_TIMEOUT, \
    RAMNET_ERR_DEVICE_CHECK = range(6)
RAMNET_F32, RAMNET_BF16 = 0, 1

# every symbol include/ramnet.h declares
EXPORTED = ("ramnet_decode_addresses", "ramnet_scan_workspace_bytes", "ramnet_scan_layout", "ramnet_scan_forward",
            "ramnet_scan_route", "ramnet_scan_recur", "ramnet_scan_forward_noalloc", "ramnet_decode_step",
            "ramnet_scan_forward_host_scratch_bytes", "ramnet_scan_forward_host",
            "ramnet_ssm_workspace_bytes", "ramnet_ssm_forward", "ramnet_ssm_step", "ramnet_conv_forward",
            "ramnet_conv_step", "ramnet_norm_gate",
            "ramnet_selftest_wait_timeout", "ramnet_set_scan_wait_limit", "ramnet_sync_status", "ramnet_last_error")
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # RAMNET_NOALLOC_SCRATCH_BYTES


class RamnetError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"ramnet status {status}: {msg}")
        self.status = status


_MAX = 2 ** 31 - 1


def _fits(**sizes):
    """Raises for a size that the library's 32-bit arguments do not hold (ctypes would cut it to its low bits, and the
    library would see a small size that passes its checks)."""
    for name, v in sizes.items():
        if not -_MAX <= v <= _MAX:
            raise RamnetError(RAMNET_ERR_INVALID_ARG, f"{name}={v} too large (32 bits)")


class _Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64), ("h", ctypes.c_int64)]


class _Cfg(ctypes.Structure):
    _fields_ = [("d_p", ctypes.c_int32), ("U", ctypes.c_int32), ("K", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("eps_gsu", ctypes.c_float),
                ("eps_norm", ctypes.c_float), ("renorm", ctypes.c_int32)]


@dataclass(frozen=True)
class Config:
    d_p: int
    U: int
    K: int
    d_v: int
    eps_gsu: float = 1e-6
    eps_norm: float = 1e-6
    renorm: int = 1

    def __post_init__(self):
        _fits(d_p=self.d_p, U=self.U, K=self.K, d_v=self.d_v, renorm=self.renorm)

    @property
    def M(self) -> int:
        return self.d_p ** self.U

    @property
    def L(self) -> int:
        return self.d_p * self.U

    def _c(self) -> _Cfg:
        return _Cfg(self.d_p, self.U, self.K, self.d_v, self.eps_gsu, self.eps_norm, self.renorm)


class _SsmCfg(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("G", ctypes.c_int32), ("N", ctypes.c_int32), ("P", ctypes.c_int32),
                ("dt_softplus", ctypes.c_int32), ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


@dataclass(frozen=True)
class SsmConfig:
    """A state space layer: H heads of P channels with N state values per channel, B and C
    vectors shared by the H/G heads of a group; step size clamp(softplus(dt + bias), dt_min, dt_max)."""
    H: int
    G: int
    N: int
    P: int
    dt_softplus: bool = True
    dt_min: float = 0.0
    dt_max: float = float("inf")

    def __post_init__(self):
        _fits(H=self.H, G=self.G, N=self.N, P=self.P)
        c = _SsmCfg(self.H, self.G, self.N, self.P, int(self.dt_softplus), self.dt_min, self.dt_max)
        object.__setattr__(self, "_ref", ctypes.pointer(c))

    def __reduce__(self):  # by its fields: the pointer is this object's own
        return type(self), tuple(getattr(self, f.name) for f in fields(self))


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32


def load() -> ctypes.CDLL:
    """Load libramnet.so (raises if it is absent or lacks a declared symbol)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with sparse_slot_recurrent_b200/build.py"
                           + (" --debug" if DEBUG else ""))
    lib = ctypes.CDLL(LIB_PATH)
    for name in EXPORTED:
        if not hasattr(lib, name):
            raise RuntimeError(f"{LIB_PATH} does not export {name}")
    C = ctypes.POINTER(_Cfg)
    lib.ramnet_decode_addresses.restype = ctypes.c_int
    lib.ramnet_decode_addresses.argtypes = [C, _I, _I, _I, _P, ctypes.c_int, ctypes.POINTER(_Strides), _P, _P, _P,
                                            _P, _P]
    lib.ramnet_scan_workspace_bytes.restype = ctypes.c_size_t
    lib.ramnet_scan_workspace_bytes.argtypes = [C, _I, _I, _I]
    lib.ramnet_scan_layout.restype = ctypes.c_int
    lib.ramnet_scan_layout.argtypes = [C, ctypes.c_int, _P, _P, _P, _P]
    lib.ramnet_scan_forward.restype = ctypes.c_int
    lib.ramnet_scan_forward.argtypes = [C, _I, _I, _I, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                        _P, ctypes.c_int, _P, _P, _P, ctypes.c_size_t, _P]
    lib.ramnet_scan_route.restype = ctypes.c_int
    lib.ramnet_scan_route.argtypes = [C, _I, _I, _I, ctypes.c_int, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    lib.ramnet_scan_recur.restype = ctypes.c_int
    lib.ramnet_scan_recur.argtypes = [C, _I, _I, _I, ctypes.c_int, _P, _P, _P, _P, _P, _P, ctypes.c_int, _P, _P,
                                      _P, ctypes.c_size_t, _P]
    lib.ramnet_scan_forward_noalloc.restype = ctypes.c_int
    lib.ramnet_scan_forward_noalloc.argtypes = [C, _I, _I, _I, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                                _P, _P, ctypes.c_int, _P, _P, _P]
    lib.ramnet_decode_step.restype = ctypes.c_int
    lib.ramnet_decode_step.argtypes = [C, _I, _I, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                       ctypes.c_int, _P]
    lib.ramnet_selftest_wait_timeout.restype = ctypes.c_int
    lib.ramnet_selftest_wait_timeout.argtypes = [ctypes.c_uint32, _P]
    lib.ramnet_scan_forward_host_scratch_bytes.restype = ctypes.c_size_t
    lib.ramnet_scan_forward_host_scratch_bytes.argtypes = [_P, _I, _I, _I, _I, _I, _I]
    lib.ramnet_scan_forward_host.restype = ctypes.c_int
    lib.ramnet_scan_forward_host.argtypes = ([_P, _I, _I, _I, _I] + [_P] * 11 + [_I] + [_P] * 2 +
                                             [_I, _P, ctypes.c_size_t, _P])
    SC, ST, L, D = ctypes.POINTER(_SsmCfg), ctypes.POINTER(_Strides), ctypes.c_int64, ctypes.c_int
    lib.ramnet_ssm_workspace_bytes.restype = ctypes.c_size_t
    lib.ramnet_ssm_workspace_bytes.argtypes = [SC, _I, _I]
    lib.ramnet_ssm_forward.restype = ctypes.c_int
    lib.ramnet_ssm_forward.argtypes = [SC, _I, _I, D, _P, ST, _P, ST, _P, _P, ST, _P, ST, _P, _P, _P, _P, _P, D, _P,
                                       _P, ctypes.c_size_t, _P]
    lib.ramnet_ssm_step.restype = ctypes.c_int
    lib.ramnet_ssm_step.argtypes = [SC, _I, D, _P, ST, _P, ST, _P, _P, ST, _P, ST, _P, _P, _P, _P, D, _P]
    lib.ramnet_conv_forward.restype = ctypes.c_int
    lib.ramnet_conv_forward.argtypes = [_I, _I, _I, _I, D, _P, L, L, _P, _P, _I, _P, _P, _P, D, _P, _P]
    lib.ramnet_conv_step.restype = ctypes.c_int
    lib.ramnet_conv_step.argtypes = [_I, _I, _I, D, _P, L, _P, _P, _I, _P, _P, D, _P]
    lib.ramnet_norm_gate.restype = ctypes.c_int
    lib.ramnet_norm_gate.argtypes = [L, _I, _I, D, _P, L, _P, L, _P, ctypes.c_float, _I, _P, D, _P]
    lib.ramnet_set_scan_wait_limit.restype = ctypes.c_int
    lib.ramnet_set_scan_wait_limit.argtypes = [ctypes.c_uint32]
    lib.ramnet_sync_status.restype = ctypes.c_int
    lib.ramnet_sync_status.argtypes = [_P]
    lib.ramnet_last_error.restype = ctypes.c_char_p
    lib.ramnet_last_error.argtypes = []
    _lib = lib
    return lib


def last_error() -> str:
    return load().ramnet_last_error().decode()


def _check(status: int):
    if status != RAMNET_OK:
        raise RamnetError(status, last_error())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dt(t) -> int:
    if t.dtype == torch.bfloat16:
        return RAMNET_BF16
    if t.dtype == torch.float32:
        return RAMNET_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dense(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def decode_addresses(cfg: Config, logits: torch.Tensor, pos0=None, cape_mask=None, idx_out=None, w_out=None,
                     stream=None):
    """logits [B,T,H,U*d_p] (fp32 or bf16; any strides with the last dimension contiguous)
    -> (idx int32 [B,T,H,K], w fp32 [B,T,H,K])."""
    B, T, H, L = logits.shape
    _fits(B=B, T=T, H=H)
    if logits.stride(-1) != 1:
        raise ValueError("the last dimension of logits must be contiguous")
    _dense(pos0, cape_mask)
    if idx_out is None:
        idx_out = torch.empty((B, T, H, cfg.K), dtype=torch.int32, device=logits.device)
    if w_out is None:
        w_out = torch.empty((B, T, H, cfg.K), dtype=torch.float32, device=logits.device)
    c = cfg._c()
    st = _Strides(*logits.stride()[:3])
    _check(load().ramnet_decode_addresses(ctypes.byref(c), B, T, H, _ptr(logits), _dt(logits), ctypes.byref(st),
                                          _ptr(pos0), _ptr(cape_mask), _ptr(idx_out), _ptr(w_out), _stream(stream)))
    return idx_out, w_out


def scan_workspace_bytes(cfg: Config, B: int, T: int, H: int) -> int:
    _fits(B=B, T=T, H=H)
    c = cfg._c()
    return int(load().ramnet_scan_workspace_bytes(ctypes.byref(c), B, T, H))


@dataclass(frozen=True)
class ScanLayout:
    chunk: int
    ncta: int
    scan_warps: int
    hdr_words: int


def scan_layout(cfg: Config, in_dtype=torch.bfloat16) -> ScanLayout:
    """The prefill's work split for this config and input dtype (see ramnet_scan_layout)."""
    vals = [ctypes.c_int32() for _ in range(4)]
    c = cfg._c()
    dt = RAMNET_BF16 if in_dtype == torch.bfloat16 else RAMNET_F32
    _check(load().ramnet_scan_layout(ctypes.byref(c), dt, *(ctypes.byref(v) for v in vals)))
    return ScanLayout(*(v.value for v in vals))


def scan_forward(cfg: Config, k_logits, q_logits, v, g, z, norm_w=None, cape_mask=None, pos0=None, S_in=None,
                 m_in=None, out_dtype=torch.float32, y=None, S_out=None, m_out=None, workspace=None, stream=None):
    """Prefill scan.  Returns (y [B,T,H,d_v], S_out [B,H,M,d_v], m_out [B,H,M])."""
    B, T, H, L = k_logits.shape
    _fits(B=B, T=T, H=H)
    dev = k_logits.device
    _dense(k_logits, q_logits, v, g, z, norm_w, cape_mask, pos0, S_in, m_in)
    if y is None:
        y = torch.empty((B, T, H, cfg.d_v), dtype=out_dtype, device=dev)
    if S_out is None:
        S_out = torch.empty((B, H, cfg.M, cfg.d_v), dtype=torch.float32, device=dev)
    if m_out is None:
        m_out = torch.empty((B, H, cfg.M), dtype=torch.float32, device=dev)
    need = scan_workspace_bytes(cfg, B, T, H)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    c = cfg._c()
    _check(load().ramnet_scan_forward(
        ctypes.byref(c), B, T, H, _dt(k_logits), _ptr(k_logits), _ptr(q_logits), _ptr(v), _ptr(g), _ptr(z),
        _ptr(norm_w), _ptr(cape_mask), _ptr(pos0), _ptr(S_in), _ptr(m_in), _ptr(y), _dt(y), _ptr(S_out),
        _ptr(m_out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return y, S_out, m_out


def scan_forward_host_scratch_bytes(cfg: Config, B: int, T: int, H: int, in_dtype, out_dtype, pieces: int) -> int:
    _fits(B=B, T=T, H=H, pieces=pieces)
    c = cfg._c()
    codes = {torch.bfloat16: RAMNET_BF16, torch.float32: RAMNET_F32}
    n = load().ramnet_scan_forward_host_scratch_bytes(ctypes.byref(c), B, T, H, codes[in_dtype], codes[out_dtype],
                                                      pieces)
    if n == 0:
        raise RamnetError(RAMNET_ERR_INVALID_ARG, last_error() or "bad sizes")
    return n


def scan_forward_host(cfg: Config, k_logits, q_logits, v, g, z, y, S_out, m_out, scratch, pieces=4, norm_w=None,
                      cape_mask=None, pos0=None, S_in=None, m_in=None, stream=None):
    """Prefill scan with k_logits, q_logits, v, g, z and y in host memory (CPU tensors, page-locked
    for overlap) and the rest on the device; run in ``pieces`` runs along T whose copies overlap
    the kernels.  ``scratch`` is a uint8 device tensor of scan_forward_host_scratch_bytes()."""
    B, T, H, L = k_logits.shape
    _fits(B=B, T=T, H=H, pieces=pieces)
    for t in (k_logits, q_logits, v, g, z, y):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host tensors must be contiguous CPU tensors")
    _dense(norm_w, cape_mask, pos0, S_in, m_in, S_out, m_out, scratch)
    c = cfg._c()
    _check(load().ramnet_scan_forward_host(
        ctypes.byref(c), B, T, H, _dt(k_logits), k_logits.data_ptr(), q_logits.data_ptr(), v.data_ptr(), g.data_ptr(),
        z.data_ptr(), _ptr(norm_w), _ptr(cape_mask), _ptr(pos0), _ptr(S_in), _ptr(m_in), y.data_ptr(), _dt(y),
        _ptr(S_out), _ptr(m_out), pieces, _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream)))
    return y, S_out, m_out


def scan_route(cfg: Config, k_logits, q_logits, g, workspace, cape_mask=None, pos0=None, stream=None):
    """First launch of scan_forward: address decode, CAPE, write retentions, event grouping
    into ``workspace`` (uint8 device tensor of at least scan_workspace_bytes())."""
    B, T, H, L = k_logits.shape
    _fits(B=B, T=T, H=H)
    _dense(k_logits, q_logits, g, cape_mask, pos0, workspace)
    c = cfg._c()
    _check(load().ramnet_scan_route(ctypes.byref(c), B, T, H, _dt(k_logits), _ptr(k_logits), _ptr(q_logits), _ptr(g),
                                    _ptr(cape_mask), _ptr(pos0), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))


def scan_recur(cfg: Config, v, z, y, S_out, m_out, workspace, norm_w=None, S_in=None, m_in=None, stream=None):
    """Second launch of scan_forward: the recurrence over the events scan_route wrote."""
    B, T, H, dv = v.shape
    _fits(B=B, T=T, H=H)
    _dense(v, z, y, S_out, m_out, workspace, norm_w, S_in, m_in)
    c = cfg._c()
    _check(load().ramnet_scan_recur(ctypes.byref(c), B, T, H, _dt(v), _ptr(v), _ptr(z), _ptr(norm_w), _ptr(S_in),
                                    _ptr(m_in), _ptr(y), _dt(y), _ptr(S_out), _ptr(m_out), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))
    return y, S_out, m_out


def scan_forward_noalloc(cfg: Config, k_logits, q_logits, v, g, z, y, S_out, m_out, norm_w=None, cape_mask=None,
                         pos0=None, S_in=None, m_in=None, stream=None):
    """Prefill scan on the library's built-in scratch (no workspace argument).  All outputs
    are passed in; nothing is allocated.  Returns (y, S_out, m_out)."""
    B, T, H, L = k_logits.shape
    _fits(B=B, T=T, H=H)
    _dense(k_logits, q_logits, v, g, z, norm_w, cape_mask, pos0, S_in, m_in, y, S_out, m_out)
    c = cfg._c()
    _check(load().ramnet_scan_forward_noalloc(
        ctypes.byref(c), B, T, H, _dt(k_logits), _ptr(k_logits), _ptr(q_logits), _ptr(v), _ptr(g), _ptr(z),
        _ptr(norm_w), _ptr(cape_mask), _ptr(pos0), _ptr(S_in), _ptr(m_in), _ptr(y), _dt(y), _ptr(S_out),
        _ptr(m_out), _stream(stream)))
    return y, S_out, m_out


def decode_step(cfg: Config, k_logits, q_logits, v, g, z, S, m, pos=None, norm_w=None, cape_mask=None,
                out_dtype=torch.float32, y=None, stream=None):
    """One decode token per (b,h); S [B,H,M,d_v] and m [B,H,M] fp32 are updated in place.
    Returns y [B,H,d_v]."""
    B, H, L = k_logits.shape
    if B > _MAX or H > _MAX:
        _fits(B=B, H=H)
    _dense(k_logits, q_logits, v, g, z, S, m, pos, norm_w, cape_mask)
    if y is None:
        y = torch.empty((B, H, cfg.d_v), dtype=out_dtype, device=k_logits.device)
    c = cfg._c()
    _check(load().ramnet_decode_step(ctypes.byref(c), B, H, _dt(k_logits), _ptr(k_logits), _ptr(q_logits), _ptr(v),
                                     _ptr(g), _ptr(z), _ptr(norm_w), _ptr(cape_mask), _ptr(pos), _ptr(S), _ptr(m),
                                     _ptr(y), _dt(y), _stream(stream)))
    return y


def selftest_wait_timeout(limit_us: int, stream=None):
    """Launch the failure-detection self-test (a bounded wait that must run out)."""
    _fits(limit_us=limit_us)
    _check(load().ramnet_selftest_wait_timeout(limit_us, _stream(stream)))


def set_scan_wait_limit(limit_us: int):
    """Limit of the bounded waits of the prefill recurrence and the selective scan for later launches (0: 2 s default)."""
    _fits(limit_us=limit_us)
    _check(load().ramnet_set_scan_wait_limit(limit_us))


def sync_status(stream=None):
    """Wait for the stream and raise if a kernel recorded a timeout or failed check."""
    _check(load().ramnet_sync_status(_stream(stream)))


# ------------------------------------------------------------------ state space layer

_DTYPES = {torch.bfloat16: RAMNET_BF16, torch.float32: RAMNET_F32}


@functools.lru_cache(maxsize=1024)
def _strides_of(b: int, t: int, h: int):
    return ctypes.pointer(_Strides(b, t, h))


def _refuse(t, name, shape, dtype, dev, dense):
    """Raises for the first thing that is wrong with an operand."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} expected")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, {dtype} expected")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, cuda:{dev} expected")
    if dense:
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"the last dimension of {name} must be contiguous")


def _dense_ptr(t, name, shape, dtype, dev):
    """Pointer of a contiguous operand after its checks (None stays None)."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, shape, dtype, dev, True)


def _rows_ptr(t, name, shape, dtype, dev):
    """Pointer of an operand that only needs its last dimension contiguous."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev and (t.stride(-1) == 1 or t.shape[-1] == 1):
        return t.data_ptr()
    _refuse(t, name, shape, dtype, dev, False)


def _input(x, name):
    """Dtype code and device index of the operand that the others go by."""
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return code, x.get_device()


def _empty(shape, dtype, device, stream):
    """A new tensor, in memory that is ordered on the stream that will write it: memory of the current stream may
    still be in use there by work that came before."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)  # (an ExternalStream of handle 0 would be some new stream, not the default one)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _output(y, name, shape, out_dtype, x, dev, stream):
    """The output tensor (allocated if not given) and its dtype code."""
    if y is None:
        y = _empty(shape, x.dtype if out_dtype is None else out_dtype, x.device, stream)
    elif out_dtype is not None and y.dtype is not out_dtype:
        raise TypeError(f"{name} is {y.dtype}, out_dtype is {out_dtype}")
    else:
        _dense_ptr(y, name, shape, y.dtype, dev)
    code = _DTYPES.get(y.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {y.dtype}")
    return y, code


def _launch(dev, stream, call, *args):
    """Calls the library with dev current and the stream (dev's current one if None) as the last argument.  The two
    lookups are the ones behind torch.cuda.current_device and current_stream, whose wrappers cost more than a launch."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _launch(dev, stream, call, *args)
    status = call(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status != RAMNET_OK:
        raise RamnetError(status, last_error())


def ssm_workspace_bytes(cfg: SsmConfig, B: int, T: int) -> int:
    _fits(B=B, T=T)
    return int(load().ramnet_ssm_workspace_bytes(cfg._ref, B, T))


def _ssm_operands(cfg, x, dt, A, Bm, Cm, D, dt_bias):
    """Checked operands shared by the two forms: lead is [B] or [B, T]."""
    code, dev = _input(x, "x")
    lead, H, t, f32 = x.shape[:-2], cfg.H, x.dtype, torch.float32
    bc = (*lead, cfg.G, cfg.N)
    px = _rows_ptr(x, "x", (*lead, H, cfg.P), t, dev)
    if dt.shape != (*lead, H) or dt.dtype is not t or dt.get_device() != dev:
        _refuse(dt, "dt", (*lead, H), t, dev, False)
    return code, dev, (px, dt.data_ptr(), _dense_ptr(A, "A", (H,), f32, dev), _rows_ptr(Bm, "Bm", bc, t, dev),
                       _rows_ptr(Cm, "Cm", bc, t, dev), _dense_ptr(D, "D", (H,), f32, dev),
                       _dense_ptr(dt_bias, "dt_bias", (H,), f32, dev))


def ssm_forward(cfg: SsmConfig, x, dt, A, Bm, Cm, D=None, dt_bias=None, lengths=None, S_in=None, out_dtype=None, y=None,
                S_out=None, workspace=None, stream=None):
    """Selective scan over a prompt: x [B,T,H,P], dt [B,T,H], Bm and Cm [B,T,G,N] (bf16 or fp32, any strides
    with the last dimension of x, Bm and Cm contiguous), A, D, dt_bias [H] fp32, lengths [B] int32.
    Returns (y [B,T,H,P] in out_dtype (x's if None), S_out [B,H,N,P] fp32).  Rows of a y that is passed in
    behind a sequence's last token keep their values; S_out may be S_in."""
    B, T = x.shape[:2]
    if B > _MAX or T > _MAX:
        _fits(B=B, T=T)
    code, dev, (px, pdt, pA, pB, pC, pD, pbias) = _ssm_operands(cfg, x, dt, A, Bm, Cm, D, dt_bias)
    state = (B, cfg.H, cfg.N, cfg.P)
    plen = _dense_ptr(lengths, "lengths", (B,), torch.int32, dev)
    pin = _dense_ptr(S_in, "S_in", state, torch.float32, dev)
    y, ycode = _output(y, "y", x.shape, out_dtype, x, dev, stream)
    if S_out is None:
        S_out = _empty(state, torch.float32, x.device, stream)
    pout = _dense_ptr(S_out, "S_out", state, torch.float32, dev)
    if workspace is None:
        workspace = _empty(ssm_workspace_bytes(cfg, B, T), torch.uint8, x.device, stream)
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be contiguous and on the device of x")
    _launch(dev, stream, load().ramnet_ssm_forward, cfg._ref, B, T, code, px, _strides_of(*x.stride()[:3]), pdt,
            _strides_of(*dt.stride()), pA, pB, _strides_of(*Bm.stride()[:3]), pC, _strides_of(*Cm.stride()[:3]), pD, pbias,
            plen, pin, y.data_ptr(), ycode, pout, workspace.data_ptr(), workspace.nbytes)
    return y, S_out


def ssm_step(cfg: SsmConfig, x, dt, A, Bm, Cm, S, D=None, dt_bias=None, out_dtype=None, y=None, stream=None):
    """Selective scan for one token per sequence: x [B,H,P], dt [B,H], Bm and Cm [B,G,N]; S [B,H,N,P] fp32 is
    updated in place.  Returns y [B,H,P]."""
    B = x.shape[0]
    if B > _MAX:
        _fits(B=B)
    code, dev, (px, pdt, pA, pB, pC, pD, pbias) = _ssm_operands(cfg, x, dt, A, Bm, Cm, D, dt_bias)
    pS = _dense_ptr(S, "S", (B, cfg.H, cfg.N, cfg.P), torch.float32, dev)
    y, ycode = _output(y, "y", x.shape, out_dtype, x, dev, stream)
    (xb, xh, _), (db, dh), (bb, bg, _), (cb, cg, _) = x.stride(), dt.stride(), Bm.stride(), Cm.stride()
    _launch(dev, stream, load().ramnet_ssm_step, cfg._ref, B, code, px, _strides_of(xb, 0, xh), pdt, _strides_of(db, 0, dh), pA,
            pB, _strides_of(bb, 0, bg), pC, _strides_of(cb, 0, cg), pD, pbias, pS, y.data_ptr(), ycode)
    return y


def conv_forward(x, w, bias=None, silu=True, lengths=None, state_in=None, out_dtype=None, y=None, state_out=None,
                 stream=None):
    """Short causal convolution over a prompt: x [B,T,C] (bf16 or fp32, channels contiguous), w [C,W] and
    bias [C] fp32, state_in [B,W-1,C] in x's dtype (the inputs before the first token; zeros if None).
    Returns (y [B,T,C], state_out [B,W-1,C]); state_out may be state_in."""
    (B, T, C), W, t, f32 = x.shape, w.shape[1], x.dtype, torch.float32
    if B > _MAX or T > _MAX or C > _MAX or W > _MAX:
        _fits(B=B, T=T, C=C, W=W)
    code, dev = _input(x, "x")
    px, pw, pb = _rows_ptr(x, "x", x.shape, t, dev), _dense_ptr(w, "w", (C, W), f32, dev), _dense_ptr(bias, "bias", (C,), f32, dev)
    plen = _dense_ptr(lengths, "lengths", (B,), torch.int32, dev)
    pin = _dense_ptr(state_in, "state_in", (B, W - 1, C), t, dev)
    y, ycode = _output(y, "y", x.shape, out_dtype, x, dev, stream)
    if state_out is None:
        state_out = _empty((B, W - 1, C), t, x.device, stream)
    pout = _dense_ptr(state_out, "state_out", (B, W - 1, C), t, dev)
    _launch(dev, stream, load().ramnet_conv_forward, B, T, C, W, code, px, x.stride(0), x.stride(1), pw, pb, bool(silu), plen, pin,
            y.data_ptr(), ycode, pout)
    return y, state_out


def conv_step(x, w, state, bias=None, silu=True, out_dtype=None, y=None, stream=None):
    """The convolution for one token per sequence: x [B,C]; state [B,W-1,C] in x's dtype takes the token in
    and drops its oldest.  Returns y [B,C]."""
    (B, C), W, t, f32 = x.shape, w.shape[1], x.dtype, torch.float32
    if B > _MAX or C > _MAX or W > _MAX:
        _fits(B=B, C=C, W=W)
    code, dev = _input(x, "x")
    px, pw, pb = _rows_ptr(x, "x", x.shape, t, dev), _dense_ptr(w, "w", (C, W), f32, dev), _dense_ptr(bias, "bias", (C,), f32, dev)
    ps = _dense_ptr(state, "state", (B, W - 1, C), t, dev)
    y, ycode = _output(y, "y", x.shape, out_dtype, x, dev, stream)
    _launch(dev, stream, load().ramnet_conv_step, B, C, W, code, px, x.stride(0), pw, pb, bool(silu), ps, y.data_ptr(), ycode)
    return y


def norm_gate(x, z=None, w=None, groups=1, eps=1e-6, gate_first=True, out_dtype=None, y=None, stream=None):
    """RMSNorm of the rows of x [R,D] over ``groups`` groups of channels, times w [D] fp32 (starting on 16 bytes),
    gated by silu(z) (z [R,D], None: no gate) before the norm or behind it.  Returns y [R,D]."""
    R, D = x.shape
    if D > _MAX or not -_MAX <= groups <= _MAX:
        _fits(D=D, groups=groups)
    code, dev = _input(x, "x")
    px = _rows_ptr(x, "x", x.shape, x.dtype, dev)
    pz, zs = (None, 0) if z is None else (_rows_ptr(z, "z", x.shape, x.dtype, dev), z.stride(0))
    pw = _dense_ptr(w, "w", (D,), torch.float32, dev)
    y, ycode = _output(y, "y", x.shape, out_dtype, x, dev, stream)
    _launch(dev, stream, load().ramnet_norm_gate, R, D, groups, code, px, x.stride(0), pz, zs, pw, eps, bool(gate_first),
            y.data_ptr(), ycode)
    return y
