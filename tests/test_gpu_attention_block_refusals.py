"""A TPAttentionBlock refuses what a step could not finish before a step writes the residual or a cache."""
import pytest
import torch

import bit_quantized_all_gb300 as qr
from bit_quantized_all_gb300.decode_step import TPAttentionBlock, TPAttentionLayer

pytestmark = pytest.mark.gpu
HEADS, KV, HIDDEN = 4, 2, 512


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _parts(dim=64, hidden=(HIDDEN, HIDDEN)):
    half = dict(dtype=torch.float16, device="cuda")
    out = [qr.qr_w4_quantize(torch.ones((n, HEADS * dim), **half)) for n in hidden]
    layer = TPAttentionLayer(out, KV, dim, requests=2, max_len=64, blocks=16)
    qkv = [qr.qr_w8_quantize(torch.ones(((HEADS + 2 * KV) * dim, HIDDEN), **half)) for _ in out]
    return dict(norm_weight=torch.ones(HIDDEN, device="cuda"), qkv=qkv, rope=qr.Rope.make(8), layer=layer)


def _refused(**bad):
    ok = _parts(**{name: bad.pop(name) for name in ("dim", "hidden") if name in bad})
    layer = ok["layer"]
    x, residual = (torch.randn((4, HIDDEN), device="cuda").half() for _ in range(2))
    kept, max_q = residual.clone(), bad.pop("max_q", 2)
    with pytest.raises(ValueError):
        TPAttentionBlock(**{**ok, **bad}).step(x, residual, torch.tensor([2, 2], dtype=torch.int32, device="cuda"), max_q)
    assert torch.equal(residual, kept) and not layer.caches[0].k_codes.any()


def test_a_table_wider_than_the_heads():
    _refused(rope=qr.Rope.make(66))


def test_tables_and_weights_elsewhere():
    _refused(rope=qr.Rope.make(64, device="cpu"))
    _refused(norm_weight=torch.ones(HIDDEN))


def test_heads_that_the_attention_does_not_serve():
    _refused(dim=8)
    _refused(dim=72)
    _refused(dim=272)


def test_unlike_outputs():
    _refused(hidden=(HIDDEN, HIDDEN + 32))


@pytest.mark.parametrize("max_q", [0, -1])
def test_no_queries(max_q):
    _refused(max_q=max_q)


def test_no_bound_on_the_queries():
    """max_q None: all of the step's tokens, as qr_kv_attention takes it."""
    x, residual = (torch.randn((4, HIDDEN), device="cuda").half() for _ in range(2))
    new = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    a, b = (TPAttentionBlock(**_parts()).step(x, residual.clone(), new, max_q) for max_q in (None, 4))
    assert torch.equal(a, b)
