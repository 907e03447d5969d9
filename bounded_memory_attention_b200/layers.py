"""Binding of the layers around RMA attention: the query/key norm with the position rotation, and
the gated-delta-rule layers (short convolution, single token, block of tokens).

Argument marshalling only, as in the package itself; see include/rma.h for the semantics.  Tensors
must be on the state's device; a call runs on the given stream, or on that device's current one,
whichever device is current.  As with every asynchronous call, a tensor that is freed while a call
on another stream than its own is in flight must be kept alive by the caller.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import RmaError, _check, _GdnConfig, _GdnLayout, lib  # noqa: F401

_BF16, _F32, _F64, _I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _int32(value: int, name: str) -> int:
    """`value`, which ctypes would otherwise cut to its low 32 bits."""
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError(f"{name} is beyond 32 bits: {value}")
    return value


def _call(function, name: str, index: int, stream, handle, layer, *args) -> None:
    """`function(handle, layer, *args, stream)` with device `index` current; its error raised."""
    args = (handle, _int32(layer, "layer"), *args)
    if _current_device() == index:
        code = function(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(index):
            code = function(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if code != 0:
        raise RmaError(code, name)


def _wrong(t, dtype, name: str, index: int, otherwise: str):
    """What is wrong with `t` as a tensor of `dtype` on CUDA device `index`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        return TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        return ValueError(f"{name} is on {t.device}, the state on device {index}")
    return ValueError(otherwise)


def _dense(t, dtype, numel: int, name: str, index: int) -> int:
    """The address of a contiguous tensor."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.numel() == numel
            and t.is_contiguous()):
        return t.data_ptr()
    raise _wrong(t, dtype, name, index, f"{name} must be contiguous, of {numel} elements: got {list(getattr(t, 'shape', []))}")


def _rows(t, dtype, batch: int, n: int, inner: tuple, name: str, index: int):
    """(address, elements from one token to the next) of a [batch, n, *inner] tensor (or
    [batch, *inner] for n == 1) whose tokens are contiguous rows, evenly spaced over the batch too."""
    row = inner[0] if len(inner) == 1 else inner[0] * inner[1]
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index
            and (t.shape == (batch, n, *inner) or n == 1 and t.shape == (batch, *inner))):
        raise _wrong(t, dtype, name, index, f"{name} must be {[batch, n, *inner]}: got {list(getattr(t, 'shape', []))}")
    if t.is_contiguous():
        return t.data_ptr(), row
    strides = t.stride()
    step = 1
    for size, stride in zip(reversed(inner), reversed(strides)):
        if size != 1 and stride != step:
            raise ValueError(f"{name}: the values of a token must be contiguous")
        step *= size
    if n == 1:
        return t.data_ptr(), strides[0] if batch > 1 else row
    if batch > 1 and strides[0] != n * strides[1]:
        raise ValueError(f"{name}: the tokens must be evenly spaced over the whole batch")
    return t.data_ptr(), strides[1]


def _tokens(t, batch: int, dims: int, name: str) -> int:
    """n of a [batch, n, ...] tensor with `dims` dimensions, 1 for one with a dimension less."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() == dims:
        return t.shape[1]
    if t.dim() == dims - 1:
        return 1
    raise ValueError(f"{name} has shape {list(t.shape)}, expected [{batch}, tokens, ...]")


def qk_norm_rope(state, layer: int, q, k, w_q, w_k, inv_freq, q_out, k_out, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, stream=None):
    """rma_qk_norm_rope: RMS-normed and rotated queries and keys, as decode_step and prefill_block of this
    state take them; returns (q_out, k_out).

    q [B, n, HQ, 256] and k [B, n, G, 256] bf16 ([B, HQ, 256] and [B, G, 256] for one token) may be views of
    wider rows; w_q, w_k [256] f32; inv_freq [pairs] f64 (None: no rotation); positions [B, n] i32, or None
    for the places that the layer's counters give the next tokens."""
    c = state.cfg
    device = state.buffer.get_device()
    B, G, D = c.batch, c.n_groups, c.head_dim
    HQ = G * c.q_per_group
    n = _tokens(q, B, 4, "q")
    qp, qs = _rows(q, _BF16, B, n, (HQ, D), "q", device)
    kp, ks = _rows(k, _BF16, B, n, (G, D), "k", device)
    pairs = 0 if inv_freq is None else inv_freq.numel()
    args = (_dense(w_q, _F32, D, "w_q", device), _dense(w_k, _F32, D, "w_k", device), float(eps),
            _dense(inv_freq, _F64, pairs, "inv_freq", device) if pairs else None, 2 * pairs, 1 if interleaved else 0,
            None if positions is None else _dense(positions, _I32, B * n, "positions", device),
            _dense(q_out, _BF16, B * n * HQ * D, "q_out", device), _dense(k_out, _BF16, B * n * G * D, "k_out", device))
    _call(lib.rma_qk_norm_rope, "rma_qk_norm_rope", device, stream, state._h, layer, n, qp, qs, kp, ks, *args)
    return q_out, k_out


@dataclass
class GdnConfig:
    """Dimensions of the gated-delta-rule layers; the defaults are the pages' model's (16 key heads, 32 value
    heads of 128, four taps)."""
    batch: int = 1
    n_layers: int = 1
    n_k_heads: int = 16
    n_v_heads: int = 32
    head_dim: int = 128
    conv_width: int = 4
    qk_l2norm: bool = True
    l2_eps: float = 1e-6
    scale: float = 128 ** -0.5

    def _c(self) -> _GdnConfig:
        sizes = (_int32(getattr(self, f), f) for f in ("batch", "n_layers", "n_k_heads", "n_v_heads", "head_dim", "conv_width"))
        return _GdnConfig(*sizes, _int32(int(self.qk_l2norm), "qk_l2norm"), self.l2_eps, self.scale)

    @property
    def channels(self) -> int:
        return (2 * self.n_k_heads + self.n_v_heads) * self.head_dim


def gdn_state_bytes(cfg: GdnConfig) -> int:
    c = cfg._c()
    return int(lib.rma_gdn_state_bytes(ctypes.byref(c)))


class GdnState:
    """A device state buffer (a torch uint8 tensor owned here) laid out by rma_gdn_state_alloc, all zeros.

    Attributes conv [L, B, 3, C] bf16 and delta [L, B, HV, 128, 128] f32 (key, value) are torch views into the
    buffer; a batch slot starts a new sequence when both are zeroed there."""

    def __init__(self, cfg: GdnConfig, device=None, stream=None, buffer: torch.Tensor = None):
        """Lay a state out over `buffer` (a CUDA uint8 tensor, 256-byte aligned, at least gdn_state_bytes(cfg)
        bytes), or over a fresh one."""
        self.cfg = cfg
        self._h = ctypes.c_void_p()
        n = gdn_state_bytes(cfg)
        if n == 0:
            raise ValueError(f"invalid GDN config: {lib.rma_last_error().decode()}")
        if buffer is not None:
            if buffer.dtype != torch.uint8 or not buffer.is_cuda or not buffer.is_contiguous():
                raise TypeError("buffer must be a contiguous CUDA uint8 tensor")
            if buffer.numel() < n:
                raise ValueError(f"buffer holds {buffer.numel()} bytes, the state needs {n}")
            self.buffer = buffer.view(-1)[:n]
        else:
            raw = torch.empty(n + 256, dtype=torch.uint8, device=torch.device("cuda" if device is None else device))
            off = (-raw.data_ptr()) % 256
            self.buffer = raw[off:off + n]
        c = cfg._c()
        lay = _GdnLayout()
        device = self.buffer.get_device()
        with torch.cuda.device(device):
            _check(lib.rma_gdn_state_alloc(ctypes.byref(c), self.buffer.data_ptr(), n,
                                           _raw_stream(device) if stream is None else stream.cuda_stream,
                                           ctypes.byref(self._h)), "rma_gdn_state_alloc")
        _check(lib.rma_gdn_state_layout(self._h, ctypes.byref(lay)), "rma_gdn_state_layout")
        self.layout = {f: int(getattr(lay, f)) for f, _ in _GdnLayout._fields_}

        def view(name, dtype, *shape):
            numel = 1
            for s in shape:
                numel *= s
            o = self.layout[name]
            return self.buffer[o:o + numel * dtype.itemsize].view(dtype).view(*shape)

        L, B, D = cfg.n_layers, cfg.batch, cfg.head_dim
        self.conv = view("conv", _BF16, L, B, cfg.conv_width - 1, cfg.channels)
        self.delta = view("delta", _F32, L, B, cfg.n_v_heads, D, D)

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def workspace_bytes(self, n_tok: int) -> int:
        out = ctypes.c_size_t()
        _check(lib.rma_gdn_workspace_bytes(self._h, _int32(int(n_tok), "n_tok"), ctypes.byref(out)), "rma_gdn_workspace_bytes")
        return int(out.value)

    def workspace(self, n_tok: int) -> torch.Tensor:
        """A fresh device workspace for gdn_prefill of n_tok tokens per sequence."""
        n = self.workspace_bytes(n_tok)
        w = torch.empty(n + 256, dtype=torch.uint8, device=self.buffer.device)
        off = (-w.data_ptr()) % 256
        return w[off:off + n]

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib.rma_gdn_state_free(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _lens(lens, batch: int, device):
    return None if lens is None else _dense(lens, _I32, batch, "lens", device)


def gdn_conv(state: GdnState, layer: int, x, w, out, bias=None, lens=None, stream=None):
    """rma_gdn_conv: the short convolution with SiLU over x [B, n, C] ([B, C] for one token; may be a view of
    wider rows), w [C, 4] f32, bias [C] f32 or None, lens [B] i32 or None; returns ``out``."""
    c = state.cfg
    device = state.buffer.get_device()
    B, C = c.batch, c.channels
    n = _tokens(x, B, 3, "x")
    xp, xs = _rows(x, _BF16, B, n, (C,), "x", device)
    wp = _dense(w, _F32, C * c.conv_width, "w", device)
    bp = None if bias is None else _dense(bias, _F32, C, "bias", device)
    op = _dense(out, _BF16, B * n * C, "out", device)
    _call(lib.rma_gdn_conv, "rma_gdn_conv", device, stream, state._h, layer, n, xp, xs, wp, bp,
          _lens(lens, B, device), op)
    return out


def _gate_rows(a, b, batch: int, n: int, heads: int, device):
    ap, stride = _rows(a, _BF16, batch, n, (heads,), "a", device)
    bp, bs = _rows(b, _BF16, batch, n, (heads,), "b", device)
    if bs != stride:
        raise ValueError("a and b must have the same spacing of tokens")
    return ap, bp, stride


def gdn_decode_step(state: GdnState, layer: int, qkv, a, b, a_log, dt_bias, out, stream=None):
    """rma_gdn_decode_step: one token of the gated delta rule; qkv [B, C] as gdn_conv writes it, a and b [B, HV]
    (may be views of wider rows), a_log and dt_bias [HV] f32, out [B, HV, 128]; returns ``out``."""
    c = state.cfg
    device = state.buffer.get_device()
    B, HV = c.batch, c.n_v_heads
    ap, bp, stride = _gate_rows(a, b, B, 1, HV, device)
    args = (_dense(qkv, _BF16, B * c.channels, "qkv", device), ap, bp, stride,
            _dense(a_log, _F32, HV, "a_log", device), _dense(dt_bias, _F32, HV, "dt_bias", device),
            _dense(out, _BF16, B * HV * c.head_dim, "out", device))
    _call(lib.rma_gdn_decode_step, "rma_gdn_decode_step", device, stream, state._h, layer, *args)
    return out


def gdn_prefill(state: GdnState, layer: int, qkv, a, b, a_log, dt_bias, out, ws, lens=None, stream=None):
    """rma_gdn_prefill: the gated delta rule over qkv [B, n, C], a and b [B, n, HV], out [B, n, HV, 128]; `ws`
    from state.workspace(n); lens [B] i32 or None; returns ``out``."""
    c = state.cfg
    device = state.buffer.get_device()
    B, HV = c.batch, c.n_v_heads
    n = _tokens(qkv, B, 3, "qkv")
    ap, bp, stride = _gate_rows(a, b, B, n, HV, device)
    args = (_dense(qkv, _BF16, B * n * c.channels, "qkv", device), ap, bp, stride,
            _dense(a_log, _F32, HV, "a_log", device), _dense(dt_bias, _F32, HV, "dt_bias", device),
            _lens(lens, B, device), _dense(out, _BF16, B * n * HV * c.head_dim, "out", device),
            _dense(ws, torch.uint8, ws.numel(), "ws", device), ws.numel())
    _call(lib.rma_gdn_prefill, "rma_gdn_prefill", device, stream, state._h, layer, n, *args)
    return out


def gdn_get_status(state: GdnState, stream=None) -> int:
    """Wait for the stream, then read and clear the GDN state's status word (STATUS_* bits)."""
    flags = ctypes.c_uint32()
    device = state.buffer.get_device()
    with torch.cuda.device(device):
        _check(lib.rma_gdn_get_status(state._h, _raw_stream(device) if stream is None else stream.cuda_stream,
                                      ctypes.byref(flags)), "rma_gdn_get_status")
    return int(flags.value)
