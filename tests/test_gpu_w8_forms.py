"""qr_w8_matmul at the sizes whose forms smaller ones do not reach: tiles of up to
192 and 256 tokens, several tiles (and token tiles) a CTA, each whole or in parts;
up to 16 tokens several row tiles a CTA, evenly and with a remainder.

Codes are small, so that every sum stays below 2^24 and is exact, and the two
products with the scales and the output's rounding are fixed: held to equality
against an fp64 product."""
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


def _codes(gen, rows, cols, most):
    raw = torch.randint(-most, most + 1, (rows, (cols + 15) // 16 * 16), generator=gen, device="cuda", dtype=torch.int8)
    return raw[:, :cols]


def _check(tokens, rows, cols, dtype, wide=0):
    most = min(127, int((2 ** 24 / cols) ** 0.5) - 1)
    assert most * most * cols < 2 ** 24
    gen = torch.Generator(device="cuda").manual_seed(tokens + rows + cols)
    x, w = _codes(gen, tokens, cols, most), _codes(gen, rows, cols, most)
    sx, sw = (torch.rand(n, generator=gen, device="cuda") * 0.02 + 0.001 for n in (tokens, rows))
    out = torch.full((tokens, rows + wide), 3.0, dtype=DT[dtype], device="cuda")
    got = qr.qr_w8_matmul(qr.Q8Rows(x, sx), qr.qr_w8_pack(w, sw), DT[dtype], out[:, :rows])
    total = (x.double() @ w.double().t()).float()
    assert torch.equal(got, (total * sx[:, None] * sw).to(DT[dtype]))
    assert (out[:, rows:] == 3).all() and qr.qr_wait_timeouts() == 0


# 152 SMs: tiles of (144, 192, 176, 208, 240, 256) tokens, whole and shared by CTAs, one to seven a CTA
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens,rows,cols", [
    (129, 10240, 2050), (190, 10239, 2050), (500, 5000, 2050), (129, 5000, 8192), (190, 5000, 8190), (380, 10240, 8192),
    (129, 20481, 5123), (300, 10240, 8192), (513, 10240, 4100), (257, 20481, 4100), (190, 40000, 2050),
    (200, 10240, 2050), (700, 5000, 4100), (200, 5000, 8192), (250, 10240, 8192), (500, 5001, 8192), (200, 20481, 4100),
    (700, 10240, 4100), (1500, 5000, 4100), (250, 40000, 4100), (2000, 5000, 4100), (1024, 10240, 8192)])
def test_tiles_of_many_tokens(tokens, rows, cols, dtype):
    _check(tokens, rows, cols, dtype)


# up to 128 tokens a tile, with three and more tiles a CTA: both accumulators in turn
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1024, 10240, 512), (4096, 2050, 1000), (4096, 1000, 2050), (4000, 20480, 64), (40, 40000, 200), (20, 40001, 130),
    (100, 40000, 128), (180, 41000, 70), (5000, 1024, 200), (1024, 1280, 8192), (64, 10240, 8192)])
def test_many_tiles(tokens, rows, cols, dtype):
    _check(tokens, rows, cols, dtype)


@pytest.mark.parametrize("tokens,rows,cols", [(129, 20481, 2050), (200, 10242, 2050), (700, 5000, 4100), (40, 40001, 200)])
@pytest.mark.parametrize("wide", [1, 2, 4, 8])
def test_outputs_on_other_boundaries(tokens, rows, cols, wide):
    _check(tokens, rows, cols, 1, wide)


# 457 to 1793 row tiles, both sides of 608, 912 and 1368 (four, six and nine for each of 152 SMs)
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows", [7297, 7313, 9728, 9729, 9745, 14592, 14609, 20481, 21888, 21889, 28673])
@pytest.mark.parametrize("tokens", [1, 8, 9, 16])
@pytest.mark.parametrize("cols", [64, 330, 2049])
def test_many_rows(tokens, rows, cols, dtype):
    _check(tokens, rows, cols, dtype)
