"""Queries that are not finite: a row that sees a key becomes NaN whatever the
signs, one that sees nothing stays empty, and no other row changes."""
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
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kv", [1, 2, 300])
@pytest.mark.parametrize("codes", [100, -100])
@pytest.mark.parametrize("nq,heads", [(1, 1), (40, 1), (1, 2)])
def test_an_infinite_query_makes_its_row_nan(dtype, sign, kv, codes, nq, heads):
    """All keys of one sign: every score is an infinity of the same sign."""
    c = Case([kv], [nq], heads, 4, dtype=dtype, seed=43)
    c.kc[:] = codes
    c.cache.k_codes.copy_(torch.from_numpy(c.kc))
    row = nq - 1  # the last query sees every key
    clean, clean_lse = c.run()
    c.q_dev = c.q_dev.clone()
    c.q_dev[row, 1, 7] = sign * float("inf")
    out, lse = c.run()
    assert torch.isnan(out[row, 1].float()).all() and torch.isnan(lse[row, 1])
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[row, 1] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("nq", [3, 40])
def test_a_query_that_is_not_finite_and_sees_nothing_is_empty(value, nq):
    c = Case([0, 2], [nq, nq], 1, 4, seed=44)
    c.q_dev = c.q_dev.clone()
    c.q_dev[0, 0, 3] = c.q_dev[nq, 2, 3] = value  # nothing cached; before position 0
    out, lse = c.run()
    for t, h in ((0, 0), (nq, 2)):
        assert (out[t, h] == 0).all() and torch.isneginf(lse[t, h])
    assert torch.isfinite(out.float()).all()


def test_a_non_finite_query_leaves_the_other_rows_bits():
    """Long enough for tiles that every row sees whole."""
    c = Case([900], [40], 1, 4, seed=45)
    clean, clean_lse = c.run()
    for value in (float("inf"), float("nan")):
        c.q_dev = c.q.cuda()
        c.q_dev[5, 2, 9] = value
        out, lse = c.run()
        keep = torch.ones_like(lse, dtype=torch.bool)
        keep[5, 2] = False
        assert torch.isnan(out[5, 2].float()).all() and torch.isnan(lse[5, 2])
        assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
