"""What a step does between its products and before it samples:

    rope = Rope(*rope_frequencies(head_dim))
    qkv = rope.rotate(qkv, positions, heads=n_q_heads + n_kv_heads, dtype=torch.bfloat16)
    x, h = residual_norm(x, y, weight)             # x + y, and its norm for the next product
    scores = adjust_scores(scores, tokens, parents, counts=counts, repetition=r, mask=grammar)
    accept, path = verify_sample(scores, ...)
    count_tokens(counts, tokens, path, accept)

The arithmetic runs in libqmm.so's kernels (qmm_rotate, qmm_residual_norm,
qmm_adjust_scores, qmm_count_tokens of include/qmm.h).
"""
from __future__ import annotations

import ctypes
import math
import struct
from fractions import Fraction

from ._lib import (QMM_ERR_DEVICE, QMM_NORM_CENTERED, QMM_ROPE_HALF, QMM_ROPE_INTERLEAVED, load, qmm_adjust_args, qmm_norm_args,
                   qmm_rope, qmm_rotate_args)
from .paged import _check, _dtype, _flat, _rows, _strided, _stream_ptr

_ROTATE = struct.Struct("@IIIiiiiiPP6qPIIifP")
_NORM = struct.Struct("@IIqqIIIfPqPqPqPqPPPPPqf0q")
_ADJUST = struct.Struct("@IIiiqPqqPqqPPPPqPqPPPPqPqq")
assert _ROTATE.size == ctypes.sizeof(qmm_rotate_args) and _NORM.size == ctypes.sizeof(qmm_norm_args)
assert _ADJUST.size == ctypes.sizeof(qmm_adjust_args)
_LAYOUTS = {"half": QMM_ROPE_HALF, "interleaved": QMM_ROPE_INTERLEAVED}
# 2 pi to 40 digits, so that a frequency's turns are as exact as the frequency
_TWO_PI = 2 * Fraction(31415926535897932384626433832795028841972, 10 ** 40)


def _current(func, at):
    import torch
    if torch._C._cuda_getDevice() != at:
        _check(func, QMM_ERR_DEVICE)


def _at(t):
    return 0 if t is None else t.data_ptr()


# ------------------------------------------------------------------ rotary positions
def rope_frequencies(dims: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_length: int = 8192, slow: float = 1.0, fast: float = 32.0):
    """(frequencies, amplitude): radians a position of the dims / 2 pairs, float64,
    base^(-2 i / dims), for a context `factor` times the trained `original_length`
    positions:

    None        as trained;
    "linear"    all divided by factor (position interpolation);
    "base"      base times factor^(dims / (dims - 2)): the slowest is divided by
                factor, the fastest kept;
    "by parts"  divided by factor where a pair makes fewer than `slow` turns in
                original_length, kept from `fast` turns on, blended linearly in turns
                between; the amplitude is 0.1 ln(factor) + 1.
    """
    import torch
    if dims < 2 or dims % 2:
        raise ValueError(f"dims must be even and at least 2, not {dims}")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "by parts"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'by parts', not {scaling!r}")
    if scaling == "base":
        if dims == 2:
            raise ValueError("scaling 'base' needs more than one pair")
        base = base * factor ** (dims / (dims - 2))
    freq = torch.tensor([base ** (-2 * i / dims) for i in range(dims // 2)], dtype=torch.float64)
    if scaling == "linear":
        return freq / factor, 1.0
    if scaling == "by parts":
        if not fast > slow:
            raise ValueError("fast must be more turns than slow")
        turns = original_length * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        return freq * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return freq, 1.0


class Rope:
    """Rotary positions: frequencies in radians a position (one a pair, float64; the
    turned dimensions are twice as many), a layout and an amplitude."""

    def __init__(self, frequencies, amplitude: float = 1.0, layout: str = "half", device="cuda"):
        import torch
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
        values = [float(f) for f in (frequencies.tolist() if hasattr(frequencies, "tolist") else frequencies)]
        if not values:
            raise ValueError("at least one frequency")
        if not all(map(math.isfinite, values)) or not math.isfinite(amplitude):
            raise ValueError("frequencies and amplitude must be finite")
        turns = [round(Fraction(f) / _TWO_PI * (1 << 64)) % (1 << 64) for f in values]
        signed = [t - (1 << 64) if t >> 63 else t for t in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64).to(device)
        self.dims, self.layout, self.amplitude = 2 * len(values), layout, float(amplitude)
        self.device_index = self.turns.get_device()
        self._c = qmm_rope(ctypes.sizeof(qmm_rope), _LAYOUTS[layout], self.dims, self.amplitude, self.turns.data_ptr())
        self._fields = (self._c.struct_size, self._c.layout, self.dims, self.amplitude, self.turns.data_ptr())
        self.address = ctypes.addressof(self._c)

    def rotate(self, x, positions, heads=None, dtype=None, out=None, stream=None):
        """x [B, T, H, D] (or [T, H, D]) turned by positions int32 [B, T] ([T]): its
        first `heads` heads (None: all), the others converted to `dtype` (None: x's)
        as they are.  out may be x.  See qmm_rotate."""
        import torch
        if stream is not None:  # the result is allocated on the stream that writes it
            with torch.cuda.stream(stream):
                return self.rotate(x, positions, heads, dtype, out)
        if x.dim() not in (3, 4):
            raise ValueError("x must be [B, T, heads, head_dim] or [T, heads, head_dim]")
        if not x.is_cuda:
            raise TypeError(f"x must be a CUDA tensor, not on {x.device}")
        at = x.get_device()
        dtype = (x.dtype if dtype is None else dtype) if out is None else out.dtype if dtype is None else dtype
        if at != self.device_index:
            raise ValueError(f"x must be on cuda:{self.device_index}, not cuda:{at}")
        shape = x.shape
        _rows("x", x)
        _flat("positions", positions, torch.int32, shape[:-2], at)
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=x.device)
        else:
            _strided("out", out, dtype, shape, at)
        if x.numel() == 0:
            return out
        _current("rotate", at)
        qmm_rotate(x, out, positions, self, shape[-2] if heads is None else heads)
        return out


def qmm_rotate(x, out, positions, rope, heads, stream=None) -> None:
    """x, out CUDA [B, T, H, D] or [T, H, D]; positions int32; rope: a Rope;
    asynchronous."""
    xs, os = x.stride(), out.stride()
    if len(xs) == 3:
        B, (T, H, D), xs, os = 1, x.shape, (0, *xs), (0, *os)
    else:
        B, T, H, D = x.shape
    rc = load().qmm_rotate(_ROTATE.pack(
        _ROTATE.size, _dtype(x.dtype), _dtype(out.dtype), B, T, H, heads, D, x.data_ptr(), out.data_ptr(), xs[0], xs[1], xs[2],
        os[0], os[1], os[2], positions.data_ptr(), *rope._fields), _stream_ptr(stream, x.get_device()))
    if rc:
        _check("qmm_rotate", rc)


# ------------------------------------------------------------------ residual sums and norms
def _row_stride(name, t, shape, at):
    """The distance of the rows of t [..., N]."""
    if t.shape == shape and t.get_device() == at and t.is_contiguous():
        return shape[-1]
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor, not on {t.device}")
    if t.get_device() != at:
        raise ValueError(f"{name} must be on cuda:{at}, not {t.device}")
    if t.numel() == 0:
        return shape[-1]
    if t.dim() != 2:
        try:
            t = t.view(-1, shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: its rows must lie a fixed distance apart") from None
    if t.stride(1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.stride(0)


def residual_norm(residual, y=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None,
                  scale: float = 1.0, eps: float = 1e-6, centered: bool = False, dtype=None, out=None, residual_out=None,
                  stream=None):
    """(r', h): r' = residual + scale gate z with z = y or its norm with post_weight
    and post_bias, and h = norm(r') weight + bias in `dtype` (None: bf16).  Without y
    r' is the residual, without weight h is None.  Tensors are [..., N], weights and
    biases fp32 [N], gate fp32 [N] or [..., N]; residual_out and out may each be residual,
    y or a gate [..., N] where types and strides agree.  See qmm_residual_norm."""
    import torch
    if stream is not None:  # the results are allocated on the stream that writes them
        with torch.cuda.stream(stream):
            return residual_norm(residual, y, weight, bias, post_weight, post_bias, gate, scale, eps, centered, dtype, out,
                                 residual_out)
    if residual.dim() < 1 or not residual.is_cuda:
        raise ValueError("residual must be a CUDA tensor [..., N]")
    if y is None and weight is None:
        raise ValueError("neither y nor weight: nothing to do")
    if y is None and not (post_weight is post_bias is gate is residual_out is None):
        raise ValueError("post_weight, post_bias, gate and residual_out are for y")
    if post_bias is not None and post_weight is None:
        raise ValueError("post_bias without post_weight")
    if weight is None and not (bias is out is dtype is None):
        raise ValueError("bias, dtype and out are for weight")
    shape, at, f32 = residual.shape, residual.get_device(), torch.float32
    N, vector = shape[-1], shape[-1:]
    ld = _row_stride("residual", residual, shape, at)
    if weight is not None:
        _flat("weight", weight, f32, vector, at)
        if bias is not None:
            _flat("bias", bias, f32, vector, at)
    if post_weight is not None:
        _flat("post_weight", post_weight, f32, vector, at)
        if post_bias is not None:
            _flat("post_bias", post_bias, f32, vector, at)
    ld_y = ld_gate = ld_sums = ld_out = 0
    if gate is not None:
        if gate.dtype is not f32:
            raise TypeError(f"gate must be float32, not {gate.dtype}")
        if gate.shape == vector:
            _flat("gate", gate, f32, vector, at)
        else:
            ld_gate = _row_stride("gate", gate, shape, at)
    sums = residual
    if y is not None:
        ld_y = _row_stride("y", y, shape, at)
        if residual_out is None:
            sums, ld_sums = torch.empty(shape, dtype=residual.dtype, device=residual.device), N
        else:
            if residual_out.dtype is not residual.dtype:
                raise TypeError(f"residual_out must be {residual.dtype}, not {residual_out.dtype}")
            sums, ld_sums = residual_out, _row_stride("residual_out", residual_out, shape, at)
    if weight is not None:
        if out is None:
            out, ld_out = torch.empty(shape, dtype=torch.bfloat16 if dtype is None else dtype, device=residual.device), N
        else:
            if dtype is not None and out.dtype is not dtype:
                raise TypeError(f"out must be {dtype}, not {out.dtype}")
            ld_out = _row_stride("out", out, shape, at)
    numel = residual.numel()
    if numel == 0:
        return sums, out
    _current("residual_norm", at)
    _residual_norm(numel // N, N, residual, ld, y, ld_y, None if y is None else sums, ld_sums, out, ld_out, weight, bias,
                   post_weight, post_bias, gate, ld_gate, scale, eps, centered, _stream_ptr(None, at))
    return sums, out


def qmm_residual_norm(residual, y, residual_out, out, weight=None, bias=None, post_weight=None, post_bias=None, gate=None,
                      ld_gate: int = 0, scale: float = 1.0, eps: float = 1e-6, centered: bool = False, stream=None) -> None:
    """residual, y, residual_out, out CUDA [M, N]; the others as in qmm_norm_args;
    asynchronous."""
    M, N = residual.shape

    def ld(t):
        return 0 if t is None else t.stride(0)

    _residual_norm(M, N, residual, ld(residual), y, ld(y), residual_out, ld(residual_out), out, ld(out), weight, bias,
                   post_weight, post_bias, gate, ld_gate, scale, eps, centered, _stream_ptr(stream, residual.get_device()))


def _residual_norm(M, N, residual, ld, y, ld_y, sums, ld_sums, out, ld_out, weight, bias, post_weight, post_bias, gate, ld_gate,
                   scale, eps, centered, stream):
    dt = _dtype(residual.dtype)
    rc = load().qmm_residual_norm(_NORM.pack(
        _NORM.size, QMM_NORM_CENTERED if centered else 0, M, N, dt, dt if y is None else _dtype(y.dtype),
        dt if out is None else _dtype(out.dtype), eps, residual.data_ptr(), ld, 0 if y is None else y.data_ptr(), ld_y,
        0 if sums is None else sums.data_ptr(), ld_sums, 0 if out is None else out.data_ptr(), ld_out,
        0 if weight is None else weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
        0 if post_weight is None else post_weight.data_ptr(), 0 if post_bias is None else post_bias.data_ptr(),
        0 if gate is None else gate.data_ptr(), ld_gate, scale), stream)
    if rc:
        _check("qmm_residual_norm", rc)


# ------------------------------------------------------------------ scores
def adjust_scores(scores, tokens=None, parents=None, counts=None, prompt=None, repetition=None, frequency=None,
                  presence=None, bias=None, mask=None, n_tokens=None, out=None, stream=None):
    """scores [B, T, V] (or [B, V]: one node a sequence) with penalties, biases and
    grammar masks, ahead of verify_sample; out may be scores.  See qmm_adjust_scores."""
    import torch
    if stream is not None:  # the result is allocated on the stream that writes it
        with torch.cuda.stream(stream):
            return adjust_scores(scores, tokens, parents, counts, prompt, repetition, frequency, presence, bias, mask,
                                 n_tokens, out)
    if scores.dim() == 2:
        if tokens is not None or parents is not None or n_tokens is not None:
            raise ValueError("tokens, parents and n_tokens are for scores [B, T, V]")
        if mask is not None:
            if mask.dim() != 2:
                raise ValueError("mask must be [B, ceil(V / 32)]")
            mask = mask[:, None]
        if out is not None and out.dim() != 2:
            raise ValueError("out must be [B, V]")
        return adjust_scores(scores[:, None], None, None, counts, prompt, repetition, frequency, presence, bias, mask, None,
                             None if out is None else out[:, None])[:, 0]
    if scores.dim() != 3 or not scores.is_cuda:
        raise ValueError("scores must be a CUDA tensor [B, T, V]")
    B, T, V = scores.shape
    words, at, i32, f32 = (V + 31) // 32, scores.get_device(), torch.int32, torch.float32
    _rows("scores", scores)
    if tokens is not None:
        _flat("tokens", tokens, i32, (B, T), at)
    if parents is not None:
        _flat("parents", parents, i32, (B, T), at)
    if n_tokens is not None:
        _flat("n_tokens", n_tokens, i32, (B,), at)
    if repetition is not None:
        _flat("repetition", repetition, f32, (B,), at)
    if frequency is not None:
        _flat("frequency", frequency, f32, (B,), at)
    if presence is not None:
        _flat("presence", presence, f32, (B,), at)
    if counts is not None:
        _strided("counts", counts, i32, (B, V), at)
    if prompt is not None:
        _strided("prompt", prompt, i32, (B, words), at)
    if mask is not None:
        _strided("mask", mask, i32, (B, T, words), at)
    if bias is not None:
        _strided("bias", bias, f32, (V,) if bias.dim() == 1 else (B, V), at)
    if out is None:
        out = torch.empty(scores.shape, dtype=scores.dtype, device=scores.device)
    else:
        _strided("out", out, scores.dtype, (B, T, V), at)
    if scores.numel() == 0:
        return out
    _current("adjust_scores", at)
    qmm_adjust_scores(scores, out, tokens, parents, counts, prompt, repetition, frequency, presence, bias, mask, n_tokens)
    return out


def qmm_adjust_scores(scores, out, tokens=None, parents=None, counts=None, prompt=None, repetition=None, frequency=None,
                      presence=None, bias=None, mask=None, n_tokens=None, stream=None) -> None:
    """scores, out CUDA [B, T, V] in fp32, bf16 or f16; the other arguments as in
    qmm_adjust_args; asynchronous."""
    B, T, V = scores.shape
    ss, os = scores.stride(), out.stride()
    ms = (0, 0) if mask is None else mask.stride()
    rc = load().qmm_adjust_scores(_ADJUST.pack(
        _ADJUST.size, _dtype(scores.dtype), B, T, V, scores.data_ptr(), ss[0], ss[1], out.data_ptr(), os[0], os[1],
        _at(tokens), _at(parents), _at(n_tokens), _at(counts), 0 if counts is None else counts.stride(0), _at(prompt),
        0 if prompt is None else prompt.stride(0), _at(repetition), _at(frequency), _at(presence), _at(bias),
        0 if bias is None or bias.dim() == 1 else bias.stride(0), _at(mask), ms[0], ms[1]),
        _stream_ptr(stream, scores.get_device()))
    if rc:
        _check("qmm_adjust_scores", rc)


def count_tokens(counts, tokens, path, accept, stream=None) -> None:
    """counts int32 [B, V] += 1 for every token that a step emitted: the accepted nodes'
    and the next one, as verify_sample gives them.  See qmm_count_tokens."""
    import torch
    if counts.dim() != 2 or not counts.is_cuda:
        raise ValueError("counts must be a CUDA tensor [B, V]")
    at, i32 = counts.get_device(), torch.int32
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, T]")
    B, T = counts.shape[0], tokens.shape[1]
    _strided("counts", counts, i32, counts.shape, at)
    _flat("tokens", tokens, i32, (B, T), at)
    _flat("path", path, i32, (B, T), at)
    _flat("accept", accept, i32, (B, 2), at)
    if B == 0:
        return
    _current("count_tokens", at)
    qmm_count_tokens(counts, tokens, path, accept, stream)


def qmm_count_tokens(counts, tokens, path, accept, stream=None) -> None:
    """counts CUDA int32 [B, V], tokens, path int32 [B, T], accept int32 [B, 2];
    asynchronous."""
    B, T = tokens.shape
    rc = load().qmm_count_tokens(counts.data_ptr(), counts.stride(0), B, T, counts.shape[1], tokens.data_ptr(),
                                 path.data_ptr(), accept.data_ptr(), _stream_ptr(stream, counts.device.index))
    if rc:
        _check("qmm_count_tokens", rc)
