"""One tensor-parallel attention layer step on one GPU: the serving operators
as they are used, ending in the quantized all-reduce.

R ranks each hold a share of the heads, a key/value cache of those heads in 8
bits and a slice of the output projection in 4 bits.  A step plans its tokens'
places once, and then every rank appends its keys and values, attends, and
multiplies by its slice; the partial outputs are summed by ``qr_allreduce``.
``TPAttentionBlock`` begins where the last all-reduce ended: it adds the message
to the residual, normalises into rows in 8 bits, and every rank makes its
queries, keys and values from them with its 8-bit projection and turns them by
their positions.  On one GPU the ranks are R sets of buffers, run in turn on one
stream.

A step reads its plan's counts back before it writes anything, so it waits once
for the GPU and cannot be captured in a graph (the calls it makes can); requests
only grow, and their blocks are not given back.
"""
from __future__ import annotations

import torch

from . import (KVCache, KVPlan, Rope, W4Weight, W8Weight, qr_allreduce, qr_kv_append, qr_kv_attention,
               qr_kv_attention_workspace, qr_kv_attention_workspace_bytes, qr_kv_plan, qr_rms_norm_q8, qr_rope,
               qr_w4_matvec, qr_w8_matmul, qr_w8_matmul_workspace)


class TPAttentionLayer:
    """Caches and projections of R ranks, and the block tables they share.

    ``weights``: each rank's ``W4Weight`` of [hidden, heads_of_rank * head_dim].
    """

    def __init__(self, weights: list[W4Weight], kv_heads: int, head_dim: int, requests: int, max_len: int,
                 blocks: int, block_size: int = 16, bits: int = 4, device="cuda"):
        self.weights, self.bits, self.block_size, self.head_dim = weights, bits, block_size, head_dim
        self.caches = [KVCache.empty(blocks, kv_heads, block_size, head_dim, device) for _ in weights]
        self.block_table = torch.full((requests, -(-max_len // block_size)), -1, dtype=torch.int32, device=device)
        self.free_blocks = torch.arange(blocks, dtype=torch.int32, device=device)
        self.cached = torch.zeros(requests, dtype=torch.int32, device=device)
        self.workspace, self.workspace_tokens = None, 0
        self.counts = None  # of a step whose blocks are still on the free list (on the host)

    def step(self, q: list[torch.Tensor], k: list[torch.Tensor], v: list[torch.Tensor], new_lens: torch.Tensor,
             max_q: int) -> torch.Tensor:
        """The layer's attention output [tokens, hidden] for ``new_lens`` new
        tokens of each request (int32, on the device), from every rank's
        queries, keys and values ([tokens, heads, head_dim]); ``max_q`` bounds
        the new tokens of one request.  Blocks that the step before took and
        that are still on the free list are dropped first (release_taken).
        Raises RuntimeError where the tokens do not fit the free blocks or the
        table, ValueError where ``new_lens`` are not the queries' tokens; the
        layer is then as it was, but for table entries past its requests' ends."""
        plan, counts = self._plan(new_lens, q[0].shape[0])
        return self._attend(plan, counts, ((q[r], k[r], v[r]) for r in range(len(self.caches))), max_q)

    def _plan(self, new_lens: torch.Tensor, tokens: int) -> tuple[KVPlan, torch.Tensor]:
        """The step's plan and its counts, read back; raises as ``step`` does."""
        if self.counts is not None:
            self.release_taken()
        plan = qr_kv_plan(self.cached, new_lens, self.block_table, self.free_blocks, self.block_size, tokens)
        counts = plan.counts.cpu()
        _, new, short, beyond = counts.tolist()
        if short or beyond:
            raise RuntimeError(f"the step needs {short} blocks and {beyond} table entries more than there are")
        if new != tokens:
            raise ValueError(f"new_lens bring {new} tokens, the queries are {tokens}")
        return plan, counts

    def _attend(self, plan: KVPlan, counts: torch.Tensor, ranks, max_q: int) -> torch.Tensor:
        """The rest of a step, from every rank's (queries, keys, values) in turn."""
        partial = []
        for cache, weight, (q, k, v) in zip(self.caches, self.weights, ranks):
            tokens = q.shape[0]
            if tokens > self.workspace_tokens:
                self.workspace = qr_kv_attention_workspace(q, cache, plan.kv_lens.numel())
                self.workspace_tokens = tokens
            qr_kv_append(cache, k, v, plan.slots)
            out = qr_kv_attention(q, cache, plan.q_offsets, plan.kv_lens, plan.block_table, max_q=max_q,
                                  workspace=self.workspace)
            partial.append(qr_w4_matvec(out.view(tokens, -1), weight))
        y = qr_allreduce(self.bits, partial)
        self.cached = plan.kv_lens
        self.counts = counts
        return y

    def release_taken(self) -> None:
        """Drops the blocks that the last step took from the free list; the
        next step does it otherwise."""
        if self.counts is None:
            return
        taken, _, short, beyond = self.counts.tolist()
        if short or beyond:
            raise RuntimeError(f"the last step needed {short} blocks and {beyond} table entries more than there are")
        self.free_blocks = self.free_blocks[taken:]
        self.counts = None


class TPAttentionBlock:
    """A ``TPAttentionLayer`` with what stands before it: the norm of the residual
    stream, every rank's query, key and value projection and the positions.

    ``norm_weight``: [hidden], the activations' type or fp32; ``qkv``: each
    rank's ``W8Weight`` of [(q_heads + 2 * kv_heads) * head_dim, hidden], its
    queries' heads, then its keys', then its values'."""

    def __init__(self, norm_weight: torch.Tensor, qkv: list[W8Weight], rope: Rope, layer: TPAttentionLayer,
                 eps: float = 1e-6):
        kv_heads, dim = layer.caches[0].heads, layer.head_dim
        rows, hidden = qkv[0].rows, norm_weight.shape[0]
        if len(qkv) != len(layer.caches):
            raise ValueError(f"{len(qkv)} projections for {len(layer.caches)} ranks")
        if any(w.rows != rows or w.cols != hidden for w in qkv):
            raise ValueError(f"every rank's projection must be [{rows}, {hidden}]")
        self.q_heads = rows // dim - 2 * kv_heads
        if rows % dim or self.q_heads < kv_heads or self.q_heads % kv_heads:
            raise ValueError(f"a projection of {rows} rows holds no heads of {dim} for {kv_heads} key heads")
        if any(w.cols != self.q_heads * dim for w in layer.weights):
            raise ValueError(f"the layer's weights must have {self.q_heads * dim} columns")
        if any(w.rows != layer.weights[0].rows for w in layer.weights):
            raise ValueError("the layer's weights must have the same rows")
        # what a step would refuse only after it has written the residual
        if qr_kv_attention_workspace_bytes(1, 1, self.q_heads, kv_heads, dim) == 0:
            raise ValueError(f"no attention of {self.q_heads} heads of {dim} over {kv_heads} key heads")
        if rope.rot_dim > dim:
            raise ValueError(f"the table rotates {rope.rot_dim} values of a head, which has {dim}")
        dev = layer.caches[0].device
        if any(d != dev for d in (norm_weight.device, rope.device, *(w.packed.device for w in (*qkv, *layer.weights)))):
            raise ValueError(f"every tensor must be on {dev}")
        self.norm_weight, self.qkv, self.rope, self.layer, self.eps = norm_weight, qkv, rope, layer, eps
        self.workspace, self.workspace_tokens = None, 0

    def step(self, x: torch.Tensor, residual: torch.Tensor, new_lens: torch.Tensor, max_q: int) -> torch.Tensor:
        """The block's attention output [tokens, hidden], the next message, from
        the last one, ``x`` [tokens, hidden], which is added to ``residual`` in
        place.  ``new_lens``, ``max_q`` and what is raised (before ``residual``
        or a cache is written) as ``TPAttentionLayer.step``."""
        if max_q is not None and max_q < 1:
            raise ValueError(f"max_q must be at least 1, got {max_q}")
        tokens = x.shape[0]
        plan, counts = self.layer._plan(new_lens, tokens)
        rows = qr_rms_norm_q8(x, self.norm_weight, self.eps, residual)
        if tokens > self.workspace_tokens:
            self.workspace, self.workspace_tokens = qr_w8_matmul_workspace(tokens, self.qkv[0]), tokens
        return self.layer._attend(plan, counts, (self._heads(rows, w, plan, x.dtype) for w in self.qkv), max_q)

    def _heads(self, rows, weight: W8Weight, plan: KVPlan, dtype):
        """A rank's queries, keys and values, slices of its projection."""
        y = qr_w8_matmul(rows, weight, dtype, workspace=self.workspace)
        y = y.view(rows.tokens, -1, self.layer.head_dim)
        q, rest = y[:, :self.q_heads], y[:, self.q_heads:]
        kv_heads = rest.shape[1] // 2
        k, v = rest[:, :kv_heads], rest[:, kv_heads:]
        qr_rope(q, k, self.rope, plan=plan, out=(q, k))
        return q, k, v


__all__ = ["TPAttentionBlock", "TPAttentionLayer"]
