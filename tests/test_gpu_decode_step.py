"""The serving operators together, as TPAttentionLayer runs them: a prompt step
and decode steps of four ranks against the same layer in 64 bits over the
values that the caches and weights hold."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import serving_testlib as ref
from bit_quantized_all_gb300.decode_step import TPAttentionLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def test_prompt_then_decode():
    rng = np.random.default_rng(0)
    R, heads, kv_heads, dim, hidden, bs = 4, 4, 1, 128, 1024, 16
    dense, weights = [], []
    for _ in range(R):
        codes = rng.integers(0, 256, (hidden, heads * dim // 2)).astype(np.uint8)
        scales = (rng.random((hidden, heads * dim // 128)) * 0.01 + 0.002).astype(np.float16)
        weights.append(qr.qr_w4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), heads * dim, 128))
        dense.append(ref.w4_dense(codes, scales, None, heads * dim, 128))
    layer = TPAttentionLayer(weights, kv_heads, dim, requests=3, max_len=200, blocks=48, block_size=bs)
    lens = np.zeros(3, np.int64)
    for step, new in enumerate(([37, 5, 90], [1, 1, 1], [1, 0, 3], [1, 1, 1])):
        T = sum(new)
        q, k, v = ([torch.from_numpy(rng.standard_normal((T, n, dim)).astype(np.float32)).bfloat16().cuda() for _ in range(R)]
                   for n in (heads, kv_heads, kv_heads))
        y = layer.step(q, k, v, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
        if step % 2:  # otherwise the next step does it
            layer.release_taken()
        lens += new
        assert layer.cached.tolist() == lens.tolist()
        offsets = np.concatenate([[0], np.cumsum(new)])
        table = layer.block_table.cpu().numpy()
        partial, bound = [], np.zeros((T, hidden))
        for r in range(R):
            c = layer.caches[r]
            out, _, b_out, _ = ref.attention(q[r].float().cpu().numpy(), offsets, lens, table, c.k_codes.cpu().numpy(),
                                             c.k_scales.cpu().numpy(), c.v_codes.cpu().numpy(), c.v_scales.cpu().numpy(),
                                             dim ** -0.5, dtype=1)
            x, bx = out.reshape(T, -1), b_out.reshape(T, -1)
            p, bp = ref.matvec(x, dense[r], 1)
            partial.append(p)
            bound += bp + bx @ np.abs(dense[r]).T
        # the all-reduce: each rank's blocks of 32 lose half a step of the
        # largest magnitude / 8 (and up to a whole one at the clipped end), the
        # sum's blocks once more, and the output rounds to bf16
        blocks = [np.abs(p).reshape(-1, 32).max(1) for p in partial]
        total = sum(partial)
        err = sum(np.repeat(b, 32).reshape(T, hidden) for b in blocks) / 8
        top = np.repeat((np.abs(total) + err + bound).reshape(-1, 32).max(1), 32).reshape(T, hidden)
        limit = 1.01 * (err + top / 8) + 2 * bound + 2.0 ** -8 * np.abs(total)
        assert (np.abs(y.float().cpu().numpy() - total) <= limit).all(), step
    layer.counts = torch.tensor([0, 0, 1, 0])
    with pytest.raises(RuntimeError):
        layer.release_taken()
