"""qr_rope on queries and keys whose heads alternate in one projection ([tokens, heads, 3, head_dim])."""
import pytest
import torch

import bit_quantized_all_gb300 as qr
from bit_quantized_all_gb300 import layer

A, B, C = (0x7F0000000000 + (i << 36) for i in range(3))  # 16-byte aligned, far apart


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses are only passed where no GPU can be reached")
@pytest.mark.parametrize("tokens", [1, 5])
def test_heads_that_overlap_are_refused(tokens):
    """In place, 8 heads of 64: apart where the keys begin 64 values on and 64 are left, not otherwise."""
    for begin, head, token, fits in ((64, 192, 1536, True), (128, 192, 1536, True), (64, 128, 1024, True), (63, 192, 1536, False),
                                     (129, 192, 1536, False), (32, 96, 768, False), (192, 192, 1536, False),
                                     (64, 192, 1537, tokens == 1)):
        args = dict(dtype=1, tokens=tokens, dim=64, rot=64, inter=0, turns=A, factor=1.0, pos=B, requests=0, off=None, kv=None,
                    q=C, qt=token, qh=head, hq=8, qo=C, qot=token, qoh=head, k=C + 2 * begin, kt=token, kh=head, hk=8,
                    ko=C + 2 * begin, kot=token, koh=head, stream=None)
        got = layer._lib().qr_rope(*args.values())
        # (what passes the checks finds no GPU)
        assert got == (qr.QR_ERR_CUDA if fits else qr.QR_ERR_INVALID_ARG), (begin, head, token)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 4, 64, 64), (7, 8, 128, 64), (300, 3, 64, 64), (5, 2, 6, 4)])
def test_in_place(layout, tokens, heads, dim, rot):
    qkv = torch.randn((tokens, heads, 3, dim), device="cuda").bfloat16()
    kept = qkv.clone()
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    rope, at = qr.Rope.make(rot, layout=layout), torch.arange(tokens, dtype=torch.int32, device="cuda")
    want = qr.qr_rope(q.contiguous(), k.contiguous(), rope, at)
    got = qr.qr_rope(q, k, rope, at, out=(q, k))
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 2], kept[:, :, 2])
    # from one place of the projection into another
    a, b = kept[:, :, 0], kept[:, :, 2]
    qr.qr_rope(a, None, rope, at, out=(b, None))
    assert torch.equal(b, want[0])
