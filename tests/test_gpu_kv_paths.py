"""Paths of qr_kv_attention that only unusual shapes reach: the second level of
the tcgen05 kernel's join, windows above 128 dimensions."""
import pytest
import torch

import bit_quantized_all_gb300 as qr
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kv,nq,heads,dim", [(20000, 40, 1, 128), (9000, 300, 1, 64), (12011, 33, 2, 80)])
def test_items_of_more_parts_than_one_group(dtype, kv, nq, heads, dim):
    """Above 32 rows, one or a few items in all: each is divided among more than
    16 CTAs, whose parts are joined in groups and then the groups."""
    c = Case([kv], [nq], heads, 1, dim=dim, bs=64, dtype=dtype, seed=kv)
    out, lse = c.check()
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dim", [144, 192, 256])
@pytest.mark.parametrize("window", [1, 33, 100])
def test_window_above_128_dimensions(dim, window):
    Case([40, 200, 333], [8, 70, 1], 2, 4, dim=dim, bs=32, seed=window).check(window=window)
