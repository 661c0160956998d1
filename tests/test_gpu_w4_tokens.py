"""qr_w4_matvec of more tokens than tiles of them fit a grid's second dimension."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


@pytest.mark.parametrize("shift", [0, 1])
def test_more_tokens_than_a_grid_s_second_dimension_holds(shift):
    """65535 tiles of 64 tokens and some: the tail has to be what it is alone."""
    rng = np.random.default_rng(9)
    rows, cols, tokens = 40, 32 + shift, 65535 * 64 + 131
    weight = qr.qr_w4_quantize(torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).half().cuda(), 32)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((tokens, cols), generator=gen, device="cuda", dtype=torch.float16)
    y = torch.full((tokens, rows), 7.0, dtype=torch.float16, device="cuda")
    qr.qr_w4_matvec(x, weight, y)
    for at in (0, 1 << 21, 65535 * 64 - 64, 65535 * 64, tokens - 67):
        part = x[at:at + 67].clone()
        assert torch.equal(y[at:at + 67], qr.qr_w4_matvec(part, weight)), at
    assert not (y == 7).all(1).any()
