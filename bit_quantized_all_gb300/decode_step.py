"""One tensor-parallel attention layer step on one GPU: the serving operators
as they are used, ending in the quantized all-reduce.

R ranks each hold a share of the heads, a key/value cache of those heads in 8
bits and a slice of the output projection in 4 bits.  A step plans its tokens'
places once, and then every rank appends its keys and values, attends, and
multiplies by its slice; the partial outputs are summed by ``qr_allreduce``.
On one GPU the ranks are R sets of buffers, run in turn on one stream.

A step reads its plan's counts back before it writes anything, so it waits once
for the GPU and cannot be captured in a graph (the calls it makes can); requests
only grow, and their blocks are not given back.
"""
from __future__ import annotations

import torch

from . import (KVCache, W4Weight, qr_allreduce, qr_kv_append, qr_kv_attention, qr_kv_attention_workspace, qr_kv_plan,
               qr_w4_matvec)


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
        if self.counts is not None:
            self.release_taken()
        tokens = q[0].shape[0]
        plan = qr_kv_plan(self.cached, new_lens, self.block_table, self.free_blocks, self.block_size, tokens)
        counts = plan.counts.cpu()
        _, new, short, beyond = counts.tolist()
        if short or beyond:
            raise RuntimeError(f"the step needs {short} blocks and {beyond} table entries more than there are")
        if new != tokens:
            raise ValueError(f"new_lens bring {new} tokens, the queries are {tokens}")
        if tokens > self.workspace_tokens:
            self.workspace = qr_kv_attention_workspace(q[0], self.caches[0], new_lens.numel())
            self.workspace_tokens = tokens
        partial = []
        for rank, cache in enumerate(self.caches):
            qr_kv_append(cache, k[rank], v[rank], plan.slots)
            out = qr_kv_attention(q[rank], cache, plan.q_offsets, plan.kv_lens, plan.block_table, max_q=max_q,
                                  workspace=self.workspace)
            partial.append(qr_w4_matvec(out.view(tokens, -1), self.weights[rank]))
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


__all__ = ["TPAttentionLayer"]
