"""The calls before the attention with an empty dimension."""
import pytest
import torch

import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu
DT = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens", [0, 1, 4])
def test_rows_without_values(dtype, tokens):
    x = torch.zeros((tokens, 0), dtype=dtype, device="cuda")
    w = torch.zeros(0, dtype=dtype, device="cuda")
    for y in (qr.qr_q8_quantize(x), qr.qr_rms_norm_q8(x, w), qr.qr_rms_norm_q8(x, w, 1e-5, x.clone())):
        assert y.codes.shape == (tokens, 0) and torch.equal(y.scales, torch.zeros(tokens, device="cuda"))
    assert qr.qr_rms_norm(x, w).shape == (tokens, 0)
    y = qr.Q8Rows.empty(tokens, 0)
    assert qr.qr_q8_quantize(x, out=y) is y and (y.tokens, y.cols) == (tokens, 0)
