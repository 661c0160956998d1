"""TPAttentionLayer at other head sizes, and steps that do not fit."""
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


def _layer(rng, dim, blocks, ranks=2, heads=4, kv_heads=2, hidden=64, requests=2, max_len=100):
    dense, weights = [], []
    for _ in range(ranks):
        codes = rng.integers(0, 256, (hidden, heads * dim // 2)).astype(np.uint8)
        scales = (rng.random((hidden, -(-heads * dim // 64))) * 0.01 + 0.002).astype(np.float16)
        weights.append(qr.qr_w4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), heads * dim, 64))
        dense.append(ref.w4_dense(codes, scales, None, heads * dim, 64))
    layer = TPAttentionLayer(weights, kv_heads, dim, requests=requests, max_len=max_len, blocks=blocks, block_size=16)

    def inputs(tokens):
        return [[torch.from_numpy(rng.standard_normal((tokens, n, dim)).astype(np.float32)).bfloat16().cuda()
                 for _ in range(ranks)] for n in (heads, kv_heads, kv_heads)]

    def check(q, new, y, lens):
        """y against the layer in 64 bits over what its caches hold (as in
        test_gpu_decode_step)."""
        T = sum(new)
        offsets, table = np.concatenate([[0], np.cumsum(new)]), layer.block_table.cpu().numpy()
        partial, bound = [], np.zeros((T, hidden))
        for r, c in enumerate(layer.caches):
            out, _, b_out, _ = ref.attention(q[r].float().cpu().numpy(), offsets, lens, table, c.k_codes.cpu().numpy(),
                                             c.k_scales.cpu().numpy(), c.v_codes.cpu().numpy(), c.v_scales.cpu().numpy(),
                                             dim ** -0.5, dtype=1)
            p, bp = ref.matvec(out.reshape(T, -1), dense[r], 1)
            partial.append(p)
            bound += bp + b_out.reshape(T, -1) @ np.abs(dense[r]).T
        total = sum(partial)
        err = sum(np.repeat(np.abs(p).reshape(-1, 32).max(1), 32).reshape(T, hidden) for p in partial) / 8
        top = np.repeat((np.abs(total) + err + bound).reshape(-1, 32).max(1), 32).reshape(T, hidden)
        limit = 1.01 * (err + top / 8) + 2 * bound + 2.0 ** -8 * np.abs(total)
        assert (np.abs(y.float().cpu().numpy() - total) <= limit).all()
    return layer, inputs, check


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dim", [64, 80, 256])
def test_layer_of_other_head_sizes(dim):
    layer, inputs, check = _layer(np.random.default_rng(dim), dim, blocks=20)
    lens = np.zeros(2, np.int64)
    for new in ([50, 3], [1, 1], [2, 0]):
        q, k, v = inputs(sum(new))
        y = layer.step(q, k, v, _i32(new), max(new))
        lens += new
        check(q, new, y, lens)


@pytest.mark.parametrize("blocks,max_len", [(3, 100), (20, 32)])
def test_a_step_that_does_not_fit_raises_and_changes_nothing(blocks, max_len):
    """Too few blocks, too narrow a table: the step says so itself, and a
    smaller one goes on from where the layer was."""
    layer, inputs, check = _layer(np.random.default_rng(3), 64, blocks=blocks, max_len=max_len)
    q, k, v = inputs(21)
    check(q, [20, 1], layer.step(q, k, v, _i32([20, 1]), 20), np.array([20, 1]))
    held = [(c.k_codes.clone(), c.v_codes.clone(), c.k_scales.clone(), c.v_scales.clone()) for c in layer.caches]
    q, k, v = inputs(60)
    with pytest.raises(RuntimeError):
        layer.step(q, k, v, _i32([40, 20]), 40)
    assert layer.cached.tolist() == [20, 1]
    for c, h in zip(layer.caches, held):
        for now, was in zip((c.k_codes, c.v_codes, c.k_scales, c.v_scales), h):
            assert torch.equal(now, was)
    q, k, v = inputs(3)
    y = layer.step(q, k, v, _i32([1, 2]), 2)
    assert layer.cached.tolist() == [21, 3]
    check(q, [1, 2], y, np.array([21, 3]))


@pytest.mark.parametrize("new", [[3, 1], [1, 0]])
def test_a_step_whose_lengths_are_not_its_tokens_raises(new):
    layer, inputs, _ = _layer(np.random.default_rng(4), 64, blocks=20)
    q, k, v = inputs(2)
    with pytest.raises(ValueError):
        layer.step(q, k, v, _i32(new), 3)
    assert layer.cached.tolist() == [0, 0]
