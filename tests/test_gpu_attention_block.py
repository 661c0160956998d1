"""The operators before the attention together, as TPAttentionBlock runs them:
prompt and decode steps of two ranks, bit for bit the calls one by one with the
positions given, and the queries and keys against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import layer_testlib as ref
from bit_quantized_all_gb300.decode_step import TPAttentionBlock, TPAttentionLayer

pytestmark = pytest.mark.gpu
R, HEADS, KV, DIM, HIDDEN, EPS = 2, 4, 2, 64, 512, 1e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _weights(rng):
    rows = (HEADS + 2 * KV) * DIM
    qkv = [torch.from_numpy(rng.standard_normal((rows, HIDDEN)).astype(np.float32) * 0.05).bfloat16().cuda() for _ in range(R)]
    out = [torch.from_numpy(rng.standard_normal((HIDDEN, HEADS * DIM)).astype(np.float32) * 0.05).bfloat16().cuda() for _ in range(R)]
    return qkv, out


def _layer(out):
    return TPAttentionLayer([qr.qr_w4_quantize(w) for w in out], KV, DIM, requests=3, max_len=300, blocks=64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_prompt_then_decode(layout):
    rng = np.random.default_rng(1)
    dense, out = _weights(rng)
    qkv = [qr.qr_w8_quantize(w) for w in dense]
    norm = torch.from_numpy(rng.random(HIDDEN).astype(np.float32) + 0.5).cuda()
    freq, factor = qr.rope_frequencies(DIM)
    rope = qr.Rope(freq, layout)
    block, other = TPAttentionBlock(norm, qkv, rope, _layer(out), EPS), _layer(out)
    lens = np.zeros(3, np.int64)
    for new in ([60, 3, 130], [1, 1, 1], [1, 0, 5], [1, 1, 1], [2, 1, 0]):
        new = np.array(new)
        T = int(new.sum())
        x, residual = (torch.from_numpy(rng.standard_normal((T, HIDDEN)).astype(np.float32)).bfloat16().cuda() for _ in range(2))
        h = x.float().cpu().numpy() + residual.float().cpu().numpy()
        new_lens = torch.from_numpy(new.astype(np.int32)).cuda()
        # the calls one by one
        kept = torch.empty_like(residual)
        rows = qr.qr_rms_norm_q8(x, norm, EPS, residual, kept)
        request = np.repeat(np.arange(3), new)
        pos = lens[request] + np.arange(T) - (np.cumsum(new) - new)[request]
        at = torch.from_numpy(pos.astype(np.int32)).cuda()
        codes, step = ref.rows8(h * norm.cpu().numpy())
        assert np.array_equal(rows.codes.cpu().numpy(), codes)
        scale = step / np.sqrt((h.astype(np.float64) ** 2).mean(1) + EPS)
        heads = ([], [], [])
        for r in range(R):
            y = qr.qr_w8_matmul(rows, qkv[r], torch.bfloat16).view(T, -1, DIM)
            q, k = qr.qr_rope(y[:, :HEADS], y[:, HEADS:HEADS + KV], rope, at)
            wc, ws = ref.rows8(dense[r].float().cpu().numpy())
            plain = (codes.astype(np.float64) @ wc.astype(np.float64).T * scale[:, None] * ws.astype(np.float64)).reshape(T, -1, DIM)
            want, size = ref.rope(plain[:, :HEADS + KV], pos[:, None] * freq, layout, DIM, factor)
            # the projection's rounding and the scale's slack turn with it; then the rotation's own
            bound = (2.0 ** -8 * 1.01 + ref.norm_slack(HIDDEN) + 2.0 ** -20) * size + 2.0 ** -8 * 1.01 * np.abs(want)
            assert (np.abs(torch.cat((q, k), 1).float().cpu().numpy() - want) <= bound).all()
            for got, t in zip(heads, (q, k, y[:, HEADS + KV:])):
                got.append(t)
        want = other.step(*heads, new_lens, int(new.max()))
        got = block.step(x, residual, new_lens, int(new.max()))
        assert torch.equal(got, want) and torch.equal(residual, kept)
        lens += new
        assert block.layer.cached.tolist() == lens.tolist()
    for a, b in zip(block.layer.caches, other.caches):
        assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)


def test_a_step_that_does_not_fit_writes_nothing():
    rng = np.random.default_rng(2)
    dense, out = _weights(rng)
    block = TPAttentionBlock(torch.ones(HIDDEN, device="cuda"), [qr.qr_w8_quantize(w) for w in dense], qr.Rope.make(DIM), _layer(out))
    x = torch.randn((900, HIDDEN), device="cuda").bfloat16()
    residual = torch.randn((900, HIDDEN), device="cuda").bfloat16()
    kept = residual.clone()
    with pytest.raises(RuntimeError):
        block.step(x, residual, torch.tensor([300, 300, 300], dtype=torch.int32, device="cuda") + 100, 400)
    with pytest.raises(ValueError):
        block.step(x, residual, torch.tensor([3, 3, 3], dtype=torch.int32, device="cuda"), 3)
    assert torch.equal(residual, kept) and not block.layer.caches[0].k_codes.any()


def test_refusals():
    rng = np.random.default_rng(3)
    dense, out = _weights(rng)
    qkv, norm, rope = [qr.qr_w8_quantize(w) for w in dense], torch.ones(HIDDEN, device="cuda"), qr.Rope.make(DIM)
    for bad in (dict(qkv=qkv[:1]), dict(norm_weight=norm[:256]), dict(qkv=[qkv[0], qr.qr_w8_quantize(dense[1][:-DIM])]),
                dict(qkv=[qr.qr_w8_quantize(w[:-DIM]) for w in dense]), dict(qkv=[qr.qr_w8_quantize(w[:-1]) for w in dense])):
        with pytest.raises(ValueError):
            TPAttentionBlock(**{"norm_weight": norm, "qkv": qkv, "rope": rope, "layer": _layer(out), **bad})


def test_a_step_without_every_rank_is_refused():
    _, out = _weights(np.random.default_rng(4))
    layer = _layer(out)
    q = [torch.zeros(2, HEADS, DIM, dtype=torch.bfloat16, device="cuda")]
    k = [torch.zeros(2, KV, DIM, dtype=torch.bfloat16, device="cuda")]
    with pytest.raises(IndexError):
        layer.step(q, k, k, torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda"), 1)
