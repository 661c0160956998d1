"""Sizes beyond the C ABI's ints are refused, not cut to their low bits."""
import pytest
import torch

import bit_quantized_all_gb300 as qr

FAR = 2 ** 32


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def test_bytes():
    for rows, cols in ((FAR + 16, 64), (16, FAR + 64), (2 ** 63 + 16, 64)):
        assert qr.qr_w8_bytes(rows, cols) == 0
    for tokens, cols in ((17, FAR + 64), (2 ** 64 + 17, 64)):
        assert qr.qr_w8_matmul_workspace_bytes(tokens, cols) == 0


@pytest.mark.gpu
def test_rows():
    x = torch.zeros((1, FAR + 64), dtype=torch.float16, device="cuda")
    for call in (lambda: qr.qr_q8_quantize(x), lambda: qr.qr_rms_norm(x, x[0]), lambda: qr.qr_rms_norm_q8(x, x[0]),
                 lambda: qr.qr_w8_quantize(x),
                 lambda: qr.qr_w8_pack(x.view(torch.int8), torch.ones(1, device="cuda"))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_heads():
    rope, at = qr.Rope.make(64), torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda")
    many, long = q.expand(1, FAR + 1, 64), torch.zeros((1, 1, FAR + 64), dtype=torch.float16, device="cuda")
    for args, out in (((many, None), (many, None)), ((q, many), (q, many)), ((long, None), None)):
        with pytest.raises(ValueError):
            qr.qr_rope(*args, rope, at, out=out)
