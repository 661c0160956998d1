"""The serving operators between the all-reduced message and the attention of
the next layer.

``qr_rms_norm`` adds the residual and normalises, with an output in 16 bits or
(``qr_rms_norm_q8``) as rows in 8 bits with a scale each, which
``qr_q8_quantize`` makes of any activations; ``qr_w8_matmul`` multiplies such
rows by 8-bit weights with a scale for each output channel; ``qr_rope`` turns
queries and keys by their positions.  ``include/qr.h`` has the arithmetic,
layouts and contracts; checks, streams and errors are as in ``serving.py``.

Each call first offers its arguments to the compiled module ``_qr_fast``
(``csrc/qr_fast.cpp``), which does the common form of it, with outputs of its
own, in a third of the interpreter's time or less, and declines everything else:
what the functions here then check, serve or refuse.
Where that module is missing, they do it all, after a warning.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import warnings

import numpy as np
import torch

from . import _check, _cuda_contig, _dtype_code, _same_device, lib
from .build import FAST_PATH
from .serving import KVPlan, _as_current, _current, _int_tensor, _matrix, _on

_L = None  # the library, these calls' signatures set
_F = None  # the compiled module, bound to the library


def _lib():
    global _L
    if _L is None:
        L = lib()
        vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        norm = [i32, i64, i32, vp, i64, vp, i64, vp, i64, vp, i32, f32, vp, i64]
        sigs = {
            "qr_q8_quantize": (i32, [i32, i64, i32, vp, i64, vp, i64, vp, vp]),
            "qr_rms_norm": (i32, norm + [vp]),
            "qr_rms_norm_q8": (i32, norm + [vp, vp]),
            "qr_w8_bytes": (sz, [i32, i32]),
            "qr_w8_pack": (i32, [i32, i32, vp, i64, vp, vp, vp]),
            "qr_w8_quantize": (i32, [i32, i32, i32, vp, i64, vp, vp]),
            "qr_w8_matmul_workspace_bytes": (sz, [i64, i32]),
            "qr_w8_matmul": (i32, [i32, i64, vp, i64, vp, i32, i32, vp, vp, i64, vp, sz, vp]),
            "qr_rope": (i32, [i32, i64, i32, i32, i32, vp, f32, vp, i32, vp, vp]
                        + 2 * [vp, i64, i64, i32, vp, i64, i64] + [vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _L = L
    return _L


class _Interpreted:
    """Stands for the compiled module where there is none: it declines every call."""

    @staticmethod
    def _declines(*args):
        return None

    quantize = norm = rope = matmul = _declines


def _fast():
    global _F
    if _F is None:
        L = _lib()
        try:
            spec = importlib.util.spec_from_file_location(__package__ + "._qr_fast", FAST_PATH)
            _qr_fast = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(_qr_fast)
        except ImportError as e:
            warnings.warn(f"the calls of layer.py run without the compiled module _qr_fast, their host time some three "
                          f"times as long ({e})", RuntimeWarning, stacklevel=3)
            _F = _Interpreted()
            return _F
        _qr_fast.bind(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value
                        for name in ("qr_q8_quantize", "qr_rms_norm", "qr_rms_norm_q8", "qr_rope", "qr_w8_matmul",
                                     "qr_w8_matmul_workspace_bytes")))
        _F = _qr_fast
    return _F


_MOST = 2 ** 31 - 1  # of a size that the C ABI takes as an int: ctypes would pass a larger one's low bits


def _sizes(what: str, *sizes: int) -> None:
    if max(sizes) > _MOST:
        raise ValueError(f"{what}: a size of {max(sizes)} is beyond {_MOST}")


def _rows_of(t, what: str, shape, dtype, device: torch.device) -> tuple[int, int]:
    """(address, row stride) of a matrix of this shape and dtype on ``device``."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device.index:
        stride, inner = t.stride()
        if inner == 1 or shape[1] < 2:
            return t.data_ptr(), stride
    _matrix(t, what, shape[1])
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must match x's shape and dtype")
    raise ValueError(f"{what} must be on {device}")


# ---------------------------------------------------------------------------
# rows in 8 bits
# ---------------------------------------------------------------------------
class Q8Rows:
    """Rows in 8 bits: row t is ``codes[t] * scales[t]``.

    ``codes``: int8 ``[tokens, cols]``, its rows 16-byte aligned and contiguous;
    ``scales``: contiguous fp32 ``[tokens]``."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        _matrix(codes, "codes")
        if codes.dtype != torch.int8:
            raise TypeError(f"codes must be torch.int8, got {codes.dtype}")
        if codes.numel() and (codes.data_ptr() % 16 or (codes.shape[0] > 1 and codes.stride(0) % 16)):
            raise ValueError("codes: every row must begin on a 16-byte boundary")
        _int_tensor(scales, "scales", torch.float32, (codes.shape[0],))
        _same_device([codes, scales], "Q8Rows")
        self.codes, self.scales = codes, scales
        self.pitch = codes.stride(0)  # between rows

    tokens = property(lambda self: self.codes.shape[0])
    cols = property(lambda self: self.codes.shape[1])
    device = property(lambda self: self.codes.device)

    @classmethod
    def empty(cls, tokens: int, cols: int, device="cuda") -> "Q8Rows":
        codes = torch.empty((tokens, (cols + 15) // 16 * 16), dtype=torch.int8, device=device)
        return cls(codes[:, :cols], torch.empty(tokens, dtype=torch.float32, device=device))

    def __getitem__(self, rows: slice) -> "Q8Rows":
        return Q8Rows(self.codes[rows], self.scales[rows])

    def float(self) -> torch.Tensor:
        """The values that the rows stand for, in fp32."""
        return self.codes.float() * self.scales[:, None]


def _made(got, what: str) -> Q8Rows:
    """A Q8Rows of (codes, scales, pitch), without its checks; or the error of a status."""
    if type(got) is int:
        _check(got, what)
    out = Q8Rows.__new__(Q8Rows)
    out.codes, out.scales, out.pitch = got
    return out


def _rows8_out(out, tokens: int, cols: int, device, what: str) -> Q8Rows:
    if out is None:
        return Q8Rows.empty(tokens, cols, device)
    if not isinstance(out, Q8Rows):
        raise TypeError(f"{what}: out must be a Q8Rows")
    if out.tokens != tokens or out.cols != cols:
        raise ValueError(f"{what}: out is [{out.tokens}, {out.cols}], expected [{tokens}, {cols}]")
    if out.device != device:
        raise ValueError(f"{what}: every tensor must be on {device}")
    return out


def qr_q8_quantize(x: torch.Tensor, out: Q8Rows | None = None, stream=None) -> Q8Rows:
    """Rows of fp16/bf16 x [tokens, cols] in 8 bits."""
    if out is None and stream is None:
        got = (_F or _fast()).quantize(x)
        if got is not None:
            return _made(got, "qr_q8_quantize")
    if stream is not None:
        _matrix(x, "x")
        with _as_current(x.device, stream):
            return qr_q8_quantize(x, out)
    _matrix(x, "x")
    dt = _dtype_code(x, "x")
    tokens, cols = x.shape
    _sizes("qr_q8_quantize", cols)
    dev = x.device
    out = _rows8_out(out, tokens, cols, dev, "qr_q8_quantize")
    if tokens and cols:
        status = (_L or _lib()).qr_q8_quantize(dt, tokens, cols, x.data_ptr(), x.stride(0), out.codes.data_ptr(),
                                               out.pitch, out.scales.data_ptr(), _current(dev))
        if status:
            _check(status, "qr_q8_quantize")
    elif tokens:
        out.scales.zero_()
    return out


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def _norm(what, x, weight, eps, residual, residual_out, out, eight):
    _matrix(x, "x")
    dt = _dtype_code(x, "x")
    shape, dtype, dev = x.shape, x.dtype, x.device
    tokens, cols = shape
    _sizes(what, cols)
    wide = isinstance(weight, torch.Tensor) and weight.dtype is torch.float32
    if not ((wide or isinstance(weight, torch.Tensor) and weight.dtype is dtype) and weight.shape == (cols,)
            and weight.get_device() == dev.index and weight.is_contiguous()):
        _int_tensor(weight, "weight", torch.float32 if wide else dtype, (cols,))
        _on(dev, what, weight)
    if not 0.0 < eps < math.inf:
        raise ValueError(f"eps must be finite and above 0, got {eps}")
    if residual is None:
        if residual_out is not None:
            raise ValueError(f"{what}: residual_out without residual")
        at = stride = out_at = out_stride = 0
    else:
        at, stride = _rows_of(residual, "residual", shape, dtype, dev)
        if residual_out is None or residual_out is residual:
            out_at, out_stride = at, stride
        else:
            out_at, out_stride = _rows_of(residual_out, "residual_out", shape, dtype, dev)
    if eight:
        out = _rows8_out(out, tokens, cols, dev, what)
        if tokens and cols:
            status = (_L or _lib()).qr_rms_norm_q8(
                dt, tokens, cols, x.data_ptr(), x.stride(0), at, stride, out_at, out_stride, weight.data_ptr(), wide, eps,
                out.codes.data_ptr(), out.pitch, out.scales.data_ptr(), _current(dev))
            if status:
                _check(status, what)
        elif tokens:
            out.scales.zero_()
        return out
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
        y, y_stride = out.data_ptr(), cols
    else:
        y, y_stride = _rows_of(out, "out", shape, dtype, dev)
    if tokens and cols:
        status = (_L or _lib()).qr_rms_norm(dt, tokens, cols, x.data_ptr(), x.stride(0), at, stride, out_at, out_stride,
                                            weight.data_ptr(), wide, eps, y, y_stride, _current(dev))
        if status:
            _check(status, what)
    return out


def qr_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h = x + residual (x without one), y = h / sqrt(mean(h^2) + eps) * weight
    for each row of fp16/bf16 x [tokens, cols].  ``residual_out`` (by default
    ``residual`` itself) gets h; ``weight`` is x's type or fp32."""
    if out is None and stream is None:
        got = (_F or _fast()).norm(x, weight, eps, residual, residual_out, False)
        if got is not None:
            if type(got) is int:
                _check(got, "qr_rms_norm")
            return got
    if stream is not None:
        _matrix(x, "x")
        with _as_current(x.device, stream):
            return qr_rms_norm(x, weight, eps, residual, residual_out, out)
    return _norm("qr_rms_norm", x, weight, eps, residual, residual_out, out, False)


def qr_rms_norm_q8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                   residual_out: torch.Tensor | None = None, out: Q8Rows | None = None, stream=None) -> Q8Rows:
    """qr_rms_norm with its output as rows in 8 bits."""
    if out is None and stream is None:
        got = (_F or _fast()).norm(x, weight, eps, residual, residual_out, True)
        if got is not None:
            return _made(got, "qr_rms_norm_q8")
    if stream is not None:
        _matrix(x, "x")
        with _as_current(x.device, stream):
            return qr_rms_norm_q8(x, weight, eps, residual, residual_out, out)
    return _norm("qr_rms_norm_q8", x, weight, eps, residual, residual_out, out, True)


# ---------------------------------------------------------------------------
# 8-bit weights
# ---------------------------------------------------------------------------
class W8Weight:
    """8-bit weights [rows, cols] packed for qr_w8_matmul."""

    def __init__(self, packed: torch.Tensor, rows: int, cols: int):
        _cuda_contig(packed, "packed")
        need = qr_w8_bytes(rows, cols)
        if need == 0:
            raise ValueError(f"unsupported 8-bit weights: rows={rows} cols={cols}")
        if packed.dtype != torch.uint8 or packed.numel() < need:
            raise ValueError(f"packed must be torch.uint8 of at least {need} bytes")
        self.packed, self.rows, self.cols = packed, rows, cols


def qr_w8_bytes(rows: int, cols: int) -> int:
    return int(_lib().qr_w8_bytes(rows, cols)) if max(rows, cols) <= _MOST else 0


def _new_w8(rows: int, cols: int, device) -> W8Weight:
    return W8Weight(torch.empty(qr_w8_bytes(rows, cols), dtype=torch.uint8, device=device), rows, cols)


def qr_w8_pack(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> W8Weight:
    """Packs int8 codes [rows, cols] and fp32 scales [rows]: w = code * scale."""
    _matrix(codes, "codes")
    if stream is not None:
        with _as_current(codes.device, stream):
            return qr_w8_pack(codes, scales)
    if codes.dtype != torch.int8:
        raise TypeError(f"codes must be torch.int8, got {codes.dtype}")
    rows, cols = codes.shape
    _int_tensor(scales, "scales", torch.float32, (rows,))
    dev = _same_device([codes, scales], "qr_w8_pack")
    w = _new_w8(rows, cols, dev)
    _check(_lib().qr_w8_pack(rows, cols, codes.data_ptr(), codes.stride(0), scales.data_ptr(), w.packed.data_ptr(),
                             _current(dev)), "qr_w8_pack")
    return w


def qr_w8_quantize(w: torch.Tensor, stream=None) -> W8Weight:
    """Quantizes fp16/bf16 weights [rows, cols], a scale for each row."""
    _matrix(w, "w")
    if stream is not None:
        with _as_current(w.device, stream):
            return qr_w8_quantize(w)
    dt = _dtype_code(w, "w")
    out = _new_w8(w.shape[0], w.shape[1], w.device)
    _check(_lib().qr_w8_quantize(dt, w.shape[0], w.shape[1], w.data_ptr(), w.stride(0), out.packed.data_ptr(),
                                 _current(w.device)), "qr_w8_quantize")
    return out


def qr_w8_matmul_workspace_bytes(tokens: int, cols: int) -> int:
    return int(_lib().qr_w8_matmul_workspace_bytes(tokens, cols)) if max(tokens, cols) <= _MOST else 0


def qr_w8_matmul_workspace(tokens: int, weight: W8Weight) -> torch.Tensor:
    """A workspace for products of up to ``tokens`` rows with ``weight``; it
    serves every later call of at most these sizes on one stream."""
    return torch.empty(qr_w8_matmul_workspace_bytes(max(1, tokens), weight.cols), dtype=torch.uint8,
                       device=weight.packed.device)


_OUT_CODES = {torch.float16: 0, torch.bfloat16: 1}


def qr_w8_matmul(x: Q8Rows, weight: W8Weight, dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x @ w.T for rows in 8 bits and 8-bit weights, in ``dtype`` (fp16 or
    bf16; y's where that is given).  More than 16 tokens use ``workspace``
    (uint8, qr_w8_matmul_workspace); without one it is allocated."""
    if y is None and stream is None and isinstance(x, Q8Rows) and isinstance(weight, W8Weight) and dtype in _OUT_CODES:
        got = (_F or _fast()).matmul(x.codes, x.scales, weight.packed, weight.rows, weight.cols,
                                     dtype is torch.bfloat16, workspace)
        if got is not None:
            if type(got) is int:
                _check(got, "qr_w8_matmul")
            return got
    if stream is not None:
        with _as_current(weight.packed.device, stream):
            return qr_w8_matmul(x, weight, dtype, y, workspace)
    if not isinstance(x, Q8Rows):
        raise TypeError("x must be a Q8Rows")
    tokens, cols, rows = x.tokens, weight.cols, weight.rows
    if x.cols != cols:
        raise ValueError(f"x has {x.cols} columns, expected {cols}")
    dev = weight.packed.device
    if y is None:
        y = torch.empty((tokens, rows), dtype=dtype, device=dev)
    else:
        _matrix(y, "y", rows)
        if y.shape[0] != tokens:
            raise ValueError("y must be [tokens, rows]")
    dt = _OUT_CODES.get(y.dtype)
    if dt is None:
        raise TypeError(f"the product is torch.float16 or torch.bfloat16, got {y.dtype}")
    if x.device != dev or y.device != dev:
        _on(dev, "qr_w8_matmul", x.codes, y)
    if tokens:
        if workspace is not None:
            _cuda_contig(workspace, "workspace")
            if workspace.dtype != torch.uint8:
                raise TypeError(f"workspace must be torch.uint8, got {workspace.dtype}")
            _on(dev, "qr_w8_matmul", workspace)
        elif tokens > 16:
            workspace = torch.empty(qr_w8_matmul_workspace_bytes(tokens, cols), dtype=torch.uint8, device=dev)
        status = (_L or _lib()).qr_w8_matmul(
            dt, tokens, x.codes.data_ptr(), x.pitch, x.scales.data_ptr(), rows, cols, weight.packed.data_ptr(),
            y.data_ptr(), y.stride(0), 0 if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), _current(dev))
        if status:
            _check(status, "qr_w8_matmul")
    return y


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 0, fast_turns: float = 32.0, slow_turns: float = 1.0):
    """(radians a position of each pair in float64, the rotated values' factor).

    ``scaling``: "none"; "linear", every frequency over ``factor``; "ntk", the
    base times factor ** (rot_dim / (rot_dim - 2)); "yarn", frequencies that
    turn more than ``fast_turns`` times in ``original_len`` positions kept,
    those that turn less than ``slow_turns`` times over ``factor``, a ramp
    between, and the values times 0.1 ln(factor) + 1."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not base > 1 or not factor >= 1:
        raise ValueError(f"base must be above 1 and factor at least 1, got {base} and {factor}")
    pair = np.arange(0, rot_dim, 2, dtype=np.float64)
    plain = float(base) ** (-pair / rot_dim)
    if scaling == "none":
        return plain, 1.0
    if scaling == "linear":
        return plain / factor, 1.0
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs a rot_dim of at least 4")
        return (base * factor ** (rot_dim / (rot_dim - 2.0))) ** (-pair / rot_dim), 1.0
    if scaling != "yarn":
        raise ValueError(f'scaling must be "none", "linear", "ntk" or "yarn", got {scaling!r}')
    if original_len < 1:
        raise ValueError("yarn scaling needs original_len")

    def pair_that_turns(times):
        return rot_dim * math.log(original_len / (times * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(pair_that_turns(fast_turns)), 0), min(math.ceil(pair_that_turns(slow_turns)), rot_dim - 1)
    ramp = np.clip((np.arange(rot_dim // 2) - low) / max(high - low, 0.001), 0.0, 1.0)
    return plain / factor * ramp + plain * (1.0 - ramp), 0.1 * math.log(factor) + 1.0


class Rope:
    """A table of rotary positions: the frequencies of the ``2 * len`` rotated
    values of a head (radians a position, at most 3), which of a head's values
    are a pair (``layout``: "half", j and j + len; "interleaved", 2j and
    2j + 1), and a factor of the rotated values."""

    def __init__(self, frequencies, layout: str = "half", factor: float = 1.0, device="cuda"):
        f = np.asarray(frequencies, dtype=np.float64)
        if f.ndim != 1 or f.size < 1 or not np.isfinite(f).all() or (np.abs(f) > 3.0).any():
            raise ValueError("frequencies must be a list of numbers of magnitude up to 3")
        if layout not in ("half", "interleaved"):
            raise ValueError(f'layout must be "half" or "interleaved", got {layout!r}')
        if not math.isfinite(factor):
            raise ValueError(f"factor must be finite, got {factor}")
        # turns a position times 2^64: below 2^63 in magnitude, exact but for the division's rounding
        turns = [int(t) for t in np.rint(f / (2 * math.pi) * 2.0 ** 64)]
        self.turns = torch.tensor(turns, dtype=torch.int64).to(device)
        self.layout, self.factor, self.rot_dim, self.interleaved = layout, float(factor), 2 * f.size, layout == "interleaved"

    # (of the tensor: a copy of the table has another one)
    address = property(lambda self: self.turns.data_ptr())
    device = property(lambda self: self.turns.device)

    @classmethod
    def make(cls, rot_dim: int, base: float = 10000.0, layout: str = "half", device="cuda", **scaling) -> "Rope":
        """The table of ``rope_frequencies(rot_dim, base, **scaling)``."""
        frequencies, factor = rope_frequencies(rot_dim, base, **scaling)
        return cls(frequencies, layout, factor, device)


def _heads(t: torch.Tensor, what: str, shape=None, dtype=None, device=None) -> tuple[int, int, int]:
    """(address, token stride, head stride) of [tokens, heads, head_dim], of this
    shape and dtype on ``device`` where they are given."""
    if isinstance(t, torch.Tensor) and t.dim() == 3:
        token, head, inner = t.stride()
        if (inner == 1 or t.shape[2] < 2) and t.is_cuda:
            if shape is None:
                return t.data_ptr(), token, head
            if t.dtype is dtype and t.shape == shape and t.get_device() == device.index:
                return t.data_ptr(), token, head
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{what} must be a tensor [tokens, heads, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (there is no CPU path)")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{what}: the values of a head must be contiguous")
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)}")
    raise ValueError(f"{what} must be on {device}")


def qr_rope(q: torch.Tensor, k: torch.Tensor | None, rope: Rope, positions: torch.Tensor | None = None,
            plan: KVPlan | None = None, out=None, stream=None):
    """Queries and keys (fp16/bf16 [tokens, heads, head_dim]; k may be None)
    turned by their positions: ``positions`` (int32 [tokens]), or those of a
    step's ``plan`` (tokens past its last one are left alone in ``out``).
    Returns (q, k), new or ``out``; ``out=(q, k)`` turns them in place.  New
    outputs of a plan, in which the tokens left out are zeros, may share an
    allocation."""
    in_place = out is not None and out[0] is q and out[1] is k
    if stream is None and (out is None or in_place) and (positions is None) != (plan is None):
        got = (_F or _fast()).rope(q, k, rope.turns, rope.rot_dim, rope.interleaved, rope.factor, positions,
                                   None if plan is None else plan.q_offsets, None if plan is None else plan.kv_lens, in_place)
        if got is not None:
            if type(got) is int:
                _check(got, "qr_rope")
            return got
    if stream is not None:
        _heads(q, "q")
        with _as_current(q.device, stream):
            return qr_rope(q, k, rope, positions, plan, out)
    q_in = _heads(q, "q")
    dt = _dtype_code(q, "q")
    shape, dtype, dev = q.shape, q.dtype, q.device
    tokens, q_heads, dim = shape
    _sizes("qr_rope", q_heads, dim)
    k_in, k_heads = (0, 0, 0), 0
    if k is not None:
        k_heads = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
        k_in = _heads(k, "k", (tokens, k_heads, dim), dtype, dev)
        _sizes("qr_rope", k_heads)
    if rope.rot_dim > dim:
        raise ValueError(f"the table rotates {rope.rot_dim} values of a head, which has {dim}")
    if rope.device != dev:
        _on(dev, "qr_rope", rope.turns)
    if (positions is None) == (plan is None):
        raise ValueError("either positions or plan")
    if plan is None:
        _int_tensor(positions, "positions", torch.int32, (tokens,))
        if positions.get_device() != dev.index:
            _on(dev, "qr_rope", positions)
        at, requests, offsets, lens = positions.data_ptr(), 0, 0, 0
        new = torch.empty
    else:
        requests = plan.kv_lens.numel()
        _sizes("qr_rope", requests)
        _int_tensor(plan.kv_lens, "plan.kv_lens", torch.int32)
        _int_tensor(plan.q_offsets, "plan.q_offsets", torch.int32, (requests + 1,))
        _on(dev, "qr_rope", plan.kv_lens, plan.q_offsets)
        at, offsets, lens = 0, plan.q_offsets.data_ptr(), plan.kv_lens.data_ptr()
        new = torch.zeros  # (tokens that the plan leaves out: not what the memory held)
    k_at, k_out = (0, 0, 0), None
    if out is None:
        q_out = new(shape, dtype=dtype, device=dev)
        q_at = q_out.data_ptr(), q_heads * dim, dim
        if k is not None:
            k_out = new((tokens, k_heads, dim), dtype=dtype, device=dev)
            k_at = k_out.data_ptr(), k_heads * dim, dim
    else:
        q_out, k_out = out
        if (k is None) != (k_out is None):
            raise ValueError("out must be (q, k), None where k is")
        q_at = q_in if q_out is q else _heads(q_out, "out's q", shape, dtype, dev)
        if k is not None:
            k_at = k_in if k_out is k else _heads(k_out, "out's k", (tokens, k_heads, dim), dtype, dev)
    if not q_heads:  # (the keys alone)
        q_in, q_heads, q_at, k_heads = k_in, k_heads, k_at, 0
    if tokens and q_heads:
        if not k_heads:
            k_in = k_at = (0, 0, 0)
        status = (_L or _lib()).qr_rope(dt, tokens, dim, rope.rot_dim, rope.interleaved, rope.address, rope.factor, at,
                                        requests, offsets, lens, *q_in, q_heads, *q_at, *k_in, k_heads, *k_at, _current(dev))
        if status:
            _check(status, "qr_rope")
    return q_out, k_out


__all__ = ["Q8Rows", "Rope", "W8Weight", "qr_q8_quantize", "qr_rms_norm", "qr_rms_norm_q8", "qr_rope", "qr_w8_bytes",
           "qr_w8_matmul", "qr_w8_matmul_workspace", "qr_w8_matmul_workspace_bytes", "qr_w8_pack", "qr_w8_quantize",
           "rope_frequencies"]
