"""The serving operators of ``libqr.so``: what a tensor-parallel rank runs
before its message is all-reduced.

``qr_kv_plan`` builds a step's block tables and slots on the GPU from the
requests' lengths, ``qr_kv_append`` writes keys and values into a paged cache
held in 8 bits (one scale for each block of tokens and head),
``qr_kv_attention`` attends over it (single tokens, drafts, prompt chunks),
and ``qr_w4_matvec`` multiplies by 4-bit weights with group scales.
``include/qr.h`` has the arithmetic, layouts and contracts.

As the rest of the binding, these functions check the tensors, pick the
caller's current stream and call the C ABI; they raise if ``libqr.so`` is
missing, and there is no CPU path.  A call given ``stream`` (a
``torch.cuda.Stream`` or a raw handle) runs as it would with that stream
current: outputs and workspaces that it makes for itself are allocated and
zeroed there, and belong to that stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _cuda_contig, _dtype_code, _check, _same_device, _stream, lib

KV_BLOCK_SIZES = (16, 32, 64, 128, 256)
W4_GROUPS = (32, 64, 128)


class KVCacheStruct(ctypes.Structure):
    """qr_kv_cache_t."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("k_block_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_block_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("blocks", ctypes.c_int), ("heads", ctypes.c_int),
                ("block_size", ctypes.c_int), ("head_dim", ctypes.c_int)]


_L = None  # the library, its serving signatures set


def _lib():
    global _L
    if _L is None:
        L = lib()
        vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        # qr_kv_cache_t by address (KVCache keeps the structure alive)
        sigs = {
            "qr_kv_plan": (i32, [i32, vp, vp, i32, vp, i32, vp, i32, vp, vp, vp, i64, vp, vp]),
            "qr_kv_append": (i32, [i32, i64, vp, vp, i64, i64, i64, i64, vp, vp, vp]),
            "qr_kv_attention_workspace_bytes": (sz, [i32, i64, i32, i32, i32]),
            "qr_kv_attention": (i32, [i32, i32, i64, i32, vp, i64, i64, vp, vp, vp, i32, vp, f32, i32, i32, i32,
                                      vp, i64, i64, vp, vp, sz, vp]),
            "qr_w4_bytes": (sz, [i32, i32, i32, i32]),
            "qr_w4_pack": (i32, [i32, i32, i32, vp, vp, vp, vp, vp]),
            "qr_w4_quantize": (i32, [i32, i32, i32, i32, vp, i64, vp, vp]),
            "qr_w4_matvec_workspace_bytes": (sz, [i64, i32]),
            "qr_w4_matvec": (i32, [i32, i64, vp, i64, i32, i32, i32, i32, vp, vp, i64, vp, sz, vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _L = L
    return _L


# The handle of a device's current stream without building a Stream object
# around it: these calls are made thousands of times a second.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(device: torch.device) -> int:
    return _raw_stream(device.index) if _raw_stream is not None else _stream(device, None)


def _as_current(device: torch.device, stream):
    """A context in which ``stream`` is the current one.  What a call allocates
    on another stream than its own could still be in use by work queued there,
    be zeroed after the call has read it, and be handed on while the call
    runs."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(device, stream)
        # (0 and 1 are the runtime's names of the default stream)
        stream = torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _int_tensor(t, what: str, dtype, shape=None) -> None:
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    _cuda_contig(t, what)
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _on(device: torch.device, what: str, *tensors) -> None:
    for t in tensors:
        if t.device != device:
            raise ValueError(f"{what}: every tensor must be on {device}")


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
class KVCache:
    """A paged key/value cache held in 8 bits.

    ``k_codes`` / ``v_codes``: int8 ``[blocks, heads, block_size, head_dim]``,
    each head's ``[block_size, head_dim]`` contiguous (blocks and heads may
    be strided, so the two may be slices of one buffer); ``k_scales`` /
    ``v_scales``: contiguous fp32 ``[blocks, heads]``."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        for t, what in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                raise ValueError(f"{what} must be a tensor [blocks, heads, block_size, head_dim]")
            if not t.is_cuda:
                raise ValueError(f"{what} must be a CUDA tensor (there is no CPU path)")
            if t.dtype != torch.int8:
                raise TypeError(f"{what} must be torch.int8, got {t.dtype}")
            if t.stride(3) != 1 or t.stride(2) != t.shape[3]:
                raise ValueError(f"{what}: each head's [block_size, head_dim] must be contiguous")
        if v_codes.shape != k_codes.shape:
            raise ValueError("k_codes and v_codes must have the same shape")
        blocks, heads, block_size, head_dim = k_codes.shape
        for t, what in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _int_tensor(t, what, torch.float32, (blocks, heads))
        self.device = _same_device([k_codes, v_codes, k_scales, v_scales], "KVCache")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.blocks, self.heads, self.block_size, self.head_dim = blocks, heads, block_size, head_dim
        self._struct = KVCacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                     k_codes.stride(0), k_codes.stride(1), v_codes.stride(0), v_codes.stride(1),
                                     blocks, heads, block_size, head_dim)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, blocks: int, heads: int, block_size: int, head_dim: int, device="cuda") -> "KVCache":
        """A new cache; nothing in it is read before it is written."""
        if block_size not in KV_BLOCK_SIZES:
            raise ValueError(f"block_size must be one of {KV_BLOCK_SIZES}, got {block_size}")
        shape = (blocks, heads, block_size, head_dim)
        return cls(torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros((blocks, heads), device=device), torch.zeros((blocks, heads), device=device))


class KVPlan(NamedTuple):
    """What qr_kv_plan writes (``block_table`` is the caller's, updated)."""
    block_table: torch.Tensor  # int32 [requests, width]
    q_offsets: torch.Tensor    # int32 [requests + 1]
    kv_lens: torch.Tensor      # int32 [requests]
    slots: torch.Tensor        # int64 [max_tokens]
    counts: torch.Tensor       # int32 [4]: blocks taken, new tokens, blocks short, table entries short


def qr_kv_plan(cached_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
               free_blocks: torch.Tensor, block_size: int, max_tokens: int, plan: KVPlan | None = None,
               stream=None) -> KVPlan:
    """Block tables, offsets and slots of a step on the GPU from the requests'
    cached and new lengths (int32 [requests]); new blocks are taken from
    ``free_blocks`` (int32) in request order and entered in ``block_table``
    (int32 [requests, width], in place).  ``plan`` reuses an earlier result's
    buffers."""
    _int_tensor(cached_lens, "cached_lens", torch.int32)
    if stream is not None:
        with _as_current(cached_lens.device, stream):
            return qr_kv_plan(cached_lens, new_lens, block_table, free_blocks, block_size, max_tokens, plan)
    requests = cached_lens.numel()
    _int_tensor(new_lens, "new_lens", torch.int32, cached_lens.shape)
    _int_tensor(block_table, "block_table", torch.int32)
    _int_tensor(free_blocks, "free_blocks", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != requests:
        raise ValueError(f"block_table must be [{requests}, width]")
    dev = cached_lens.device
    _on(dev, "qr_kv_plan", new_lens, block_table, free_blocks)
    if plan is None:
        slots = torch.empty(max_tokens, dtype=torch.int64, device=dev)
        q_offsets = torch.empty(requests + 1, dtype=torch.int32, device=dev)
        kv_lens = torch.empty_like(cached_lens)
        counts = torch.empty(4, dtype=torch.int32, device=dev)
        plan = KVPlan(block_table, q_offsets, kv_lens, slots, counts)
    else:
        _, q_offsets, kv_lens, slots, counts = plan
        _int_tensor(q_offsets, "plan.q_offsets", torch.int32, (requests + 1,))
        _int_tensor(kv_lens, "plan.kv_lens", torch.int32, (requests,))
        _int_tensor(slots, "plan.slots", torch.int64, (max_tokens,))
        _int_tensor(counts, "plan.counts", torch.int32, (4,))
        _on(dev, "qr_kv_plan", q_offsets, kv_lens, slots, counts)
        plan = plan._replace(block_table=block_table)
    status = (_L or _lib()).qr_kv_plan(
        requests, cached_lens.data_ptr(), new_lens.data_ptr(), block_size, free_blocks.data_ptr(), free_blocks.numel(),
        block_table.data_ptr(), block_table.shape[1], q_offsets.data_ptr(), kv_lens.data_ptr(), slots.data_ptr(),
        max_tokens, counts.data_ptr(), _current(dev))
    if status:
        _check(status, "qr_kv_plan")
    return plan


def _rows(t: torch.Tensor, what: str, heads: int | None, dim: int) -> None:
    """A [tokens, heads, head_dim] operand, its last dimension contiguous."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 3:
        n = t.shape
        if n[2] == dim and (heads is None or n[1] == heads) and t.stride(2) == 1:
            return
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{what} must be a tensor [tokens, heads, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (there is no CPU path)")
    if t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected [tokens, {heads or 'heads'}, {dim}]")
    if t.stride(2) != 1:
        raise ValueError(f"{what}: the values of a head must be contiguous")


def qr_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> KVCache:
    """Quantizes fp16/bf16 keys and values ([tokens, heads, head_dim]) into
    the cache at ``slots`` (int64 [tokens], as qr_kv_plan gives them)."""
    if stream is not None:
        with _as_current(cache.device, stream):
            return qr_kv_append(cache, k, v, slots)
    _rows(k, "k", cache.heads, cache.head_dim)
    _rows(v, "v", cache.heads, cache.head_dim)
    tokens = k.shape[0]
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have the same shape and dtype")
    dt = _dtype_code(k, "k")
    _int_tensor(slots, "slots", torch.int64, (tokens,))
    dev = cache.device
    _on(dev, "qr_kv_append", k, v, slots)
    if tokens:
        kt, kh, _ = k.stride()
        vt, vh, _ = v.stride()
        status = (_L or _lib()).qr_kv_append(dt, tokens, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(),
                                             cache._ref, _current(dev))
        if status:
            _check(status, "qr_kv_append")
    return cache


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def qr_kv_attention_workspace_bytes(requests: int, tokens: int, q_heads: int, heads: int, head_dim: int) -> int:
    return int(_lib().qr_kv_attention_workspace_bytes(requests, tokens, q_heads, heads, head_dim))


def qr_kv_attention_workspace(q: torch.Tensor, cache: KVCache, requests: int,
                              max_q: int | None = None) -> torch.Tensor:
    """A zeroed workspace for attention of queries shaped like ``q`` by up to
    ``requests`` requests; one serves every later call of at most these sizes
    on one stream, with any ``max_q`` (which need not be given)."""
    need = qr_kv_attention_workspace_bytes(requests, q.shape[0], q.shape[1], cache.heads, cache.head_dim)
    if need == 0:
        raise ValueError(f"unsupported attention shape: requests={requests} q={tuple(q.shape)} heads={cache.heads}")
    return torch.zeros(need, dtype=torch.uint8, device=q.device)


def qr_kv_attention(q: torch.Tensor, cache: KVCache, q_offsets: torch.Tensor, kv_lens: torch.Tensor,
                    block_table: torch.Tensor, scale: float | None = None, causal: bool = True, window: int = 0,
                    max_q: int | None = None, out: torch.Tensor | None = None, return_lse: bool = False,
                    workspace: torch.Tensor | None = None, stream=None):
    """Attention of ragged fp16/bf16 queries ([tokens, q_heads, head_dim],
    request r's at ``q_offsets[r]:q_offsets[r+1]``) over the cache; ``scale``
    defaults to head_dim ** -0.5, ``max_q`` (a bound on the queries of one
    request, which picks the kernel) to the number of tokens: a decode batch
    that does not give it runs the kernel for prompts, right and slower.
    Returns ``out``, or ``(out, lse)``.  Without ``workspace`` each call
    allocates and zeroes one (up to 42 MB)."""
    if stream is not None:
        with _as_current(cache.device, stream):
            return qr_kv_attention(q, cache, q_offsets, kv_lens, block_table, scale, causal, window, max_q, out,
                                   return_lse, workspace)
    _rows(q, "q", None, cache.head_dim)
    tokens, q_heads = q.shape[0], q.shape[1]
    dt = _dtype_code(q, "q")
    _int_tensor(kv_lens, "kv_lens", torch.int32)
    requests = kv_lens.numel()
    _int_tensor(q_offsets, "q_offsets", torch.int32, (requests + 1,))
    _int_tensor(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != requests:
        raise ValueError(f"block_table must be [{requests}, width]")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _rows(out, "out", q_heads, cache.head_dim)
        if out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("out must match q's shape and dtype")
    lse = torch.empty((tokens, q_heads), dtype=torch.float32, device=q.device) if return_lse else None
    if tokens:
        if workspace is None:
            workspace = qr_kv_attention_workspace(q, cache, requests)
        else:
            _cuda_contig(workspace, "workspace")
            if workspace.dtype != torch.uint8:
                raise TypeError(f"workspace must be torch.uint8, got {workspace.dtype}")
        dev = cache.device
        _on(dev, "qr_kv_attention", q, kv_lens, q_offsets, block_table, out, workspace)
        qt, qh, _ = q.stride()
        ot, oh, _ = out.stride()
        status = (_L or _lib()).qr_kv_attention(
            dt, requests, tokens, q_heads, q.data_ptr(), qt, qh, q_offsets.data_ptr(), kv_lens.data_ptr(),
            block_table.data_ptr(), block_table.shape[1], cache._ref, cache.head_dim ** -0.5 if scale is None else scale,
            1 if causal else 0, window, tokens if max_q is None else max_q, out.data_ptr(), ot, oh,
            lse.data_ptr() if return_lse else None, workspace.data_ptr(), workspace.numel(), _current(dev))
        if status:
            _check(status, "qr_kv_attention")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
class W4Weight:
    """4-bit weights [rows, cols] packed for qr_w4_matvec."""

    def __init__(self, packed: torch.Tensor, rows: int, cols: int, group: int, has_zeros: bool):
        _cuda_contig(packed, "packed")
        need = qr_w4_bytes(rows, cols, group, has_zeros)
        if need == 0:
            raise ValueError(f"unsupported 4-bit weights: rows={rows} cols={cols} group={group}")
        if packed.dtype != torch.uint8 or packed.numel() < need:
            raise ValueError(f"packed must be torch.uint8 of at least {need} bytes")
        self.packed, self.rows, self.cols, self.group, self.has_zeros = packed, rows, cols, group, bool(has_zeros)


def qr_w4_bytes(rows: int, cols: int, group: int, has_zeros: bool = False) -> int:
    return int(_lib().qr_w4_bytes(rows, cols, group, 1 if has_zeros else 0))


def _new_w4(rows: int, cols: int, group: int, has_zeros: bool, device) -> W4Weight:
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, got {group}")
    packed = torch.empty(qr_w4_bytes(rows, cols, group, has_zeros), dtype=torch.uint8, device=device)
    return W4Weight(packed, rows, cols, group, has_zeros)


def qr_w4_pack(codes: torch.Tensor, scales: torch.Tensor, cols: int, group: int,
               zeros: torch.Tensor | None = None, stream=None) -> W4Weight:
    """Packs row-major codes (uint8 [rows, ceil(cols/2)], the even column in
    the low nibble), fp16 scales and optional uint8 zero points (both
    [rows, ceil(cols/group)]): w = (code - zero) * scale, zero 8 if None."""
    _cuda_contig(codes, "codes")
    if stream is not None:
        with _as_current(codes.device, stream):
            return qr_w4_pack(codes, scales, cols, group, zeros)
    if codes.dtype != torch.uint8 or codes.dim() != 2 or codes.shape[1] != (cols + 1) // 2:
        raise ValueError(f"codes must be torch.uint8 [rows, {(cols + 1) // 2}]")
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, got {group}")
    rows, groups = codes.shape[0], -(-cols // group)
    _int_tensor(scales, "scales", torch.float16, (rows, groups))
    if zeros is not None:
        _int_tensor(zeros, "zeros", torch.uint8, (rows, groups))
    dev = _same_device([codes, scales] + ([] if zeros is None else [zeros]), "qr_w4_pack")
    w = _new_w4(rows, cols, group, zeros is not None, dev)
    _check(_lib().qr_w4_pack(rows, cols, group, codes.data_ptr(), scales.data_ptr(),
                             None if zeros is None else zeros.data_ptr(), w.packed.data_ptr(), _current(dev)),
           "qr_w4_pack")
    return w


def _matrix(t: torch.Tensor, what: str, cols: int | None = None) -> None:
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2:
        n = t.shape[1]
        if (cols is None or n == cols) and (n < 2 or t.stride(1) == 1):
            return
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{what} must be a matrix")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (there is no CPU path)")
    if cols is not None and t.shape[1] != cols:
        raise ValueError(f"{what} has {t.shape[1]} columns, expected {cols}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the values of a row must be contiguous")


def qr_w4_quantize(w: torch.Tensor, group: int = 32, stream=None) -> W4Weight:
    """Quantizes fp16/bf16 weights [rows, cols] with the INT4 codec's
    arithmetic on groups of 32, 64 or 128 columns."""
    _matrix(w, "w")
    if stream is not None:
        with _as_current(w.device, stream):
            return qr_w4_quantize(w, group)
    dt = _dtype_code(w, "w")
    out = _new_w4(w.shape[0], w.shape[1], group, False, w.device)
    _check(_lib().qr_w4_quantize(dt, w.shape[0], w.shape[1], group, w.data_ptr(), w.stride(0), out.packed.data_ptr(),
                                 _current(w.device)), "qr_w4_quantize")
    return out


def qr_w4_matvec_workspace_bytes(tokens: int, cols: int) -> int:
    return int(_lib().qr_w4_matvec_workspace_bytes(tokens, cols))


def qr_w4_matvec(x: torch.Tensor, weight: W4Weight, y: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x @ w.T for fp16/bf16 x [tokens, cols] and 4-bit weights.  More than
    16 tokens whose rows are not 16-byte aligned are copied into ``workspace``
    (uint8, qr_w4_matvec_workspace_bytes) first; without one it is allocated."""
    if stream is not None:
        with _as_current(weight.packed.device, stream):
            return qr_w4_matvec(x, weight, y, workspace)
    _matrix(x, "x", weight.cols)
    dt = _dtype_code(x, "x")
    tokens = x.shape[0]
    if y is None:
        y = torch.empty((tokens, weight.rows), dtype=x.dtype, device=x.device)
    else:
        _matrix(y, "y", weight.rows)
        if y.dtype != x.dtype or y.shape[0] != tokens:
            raise ValueError("y must be [tokens, rows] of x's dtype")
    dev = weight.packed.device
    _on(dev, "qr_w4_matvec", x, y)
    if tokens:
        at, stride, cols = x.data_ptr(), x.stride(0), weight.cols
        if workspace is not None:
            _cuda_contig(workspace, "workspace")
            if workspace.dtype != torch.uint8:
                raise TypeError(f"workspace must be torch.uint8, got {workspace.dtype}")
            _on(dev, "qr_w4_matvec", workspace)
        elif tokens > 16 and (at | 2 * stride) & 15:
            workspace = torch.empty(qr_w4_matvec_workspace_bytes(tokens, cols), dtype=torch.uint8, device=dev)
        status = (_L or _lib()).qr_w4_matvec(
            dt, tokens, at, stride, weight.rows, cols, weight.group, weight.has_zeros, weight.packed.data_ptr(),
            y.data_ptr(), y.stride(0), None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), _current(dev))
        if status:
            _check(status, "qr_w4_matvec")
    return y


__all__ = ["KVCache", "KVPlan", "W4Weight", "qr_kv_plan", "qr_kv_append", "qr_kv_attention",
           "qr_kv_attention_workspace", "qr_kv_attention_workspace_bytes", "qr_w4_bytes", "qr_w4_pack",
           "qr_w4_quantize", "qr_w4_matvec",
           "qr_w4_matvec_workspace_bytes"]
