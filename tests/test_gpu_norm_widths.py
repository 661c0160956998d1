"""Norm and rows in 8 bits on both sides of the widths at which another kernel takes over (layer_testlib has the bounds)."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import layer_testlib as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


@pytest.mark.parametrize("dtype,code", [(torch.float16, 0), (torch.bfloat16, 1)])
@pytest.mark.parametrize("tokens", [2, 310])
@pytest.mark.parametrize("cols", [5120, 5128, 5121, 7936, 8185, 15863, 15865, 16375, 16377, 16384, 16392, 20480, 20488,
                                  31735, 31737, 32768, 32776])
def test_both_sides(cols, tokens, dtype, code):
    rng = np.random.default_rng(cols + tokens)
    x, res = (torch.from_numpy(rng.standard_normal((tokens, cols)).astype(np.float32)).to(dtype) for _ in range(2))
    w = torch.from_numpy(rng.random(cols).astype(np.float32) + 0.5)
    h = x.float().numpy() + res.float().numpy()
    rs = 1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(1) + EPS)
    slack = ref.norm_slack(cols)
    xd, resd, wd = x.cuda(), res.cuda(), w.cuda()
    rows = qr.qr_rms_norm_q8(xd, wd, EPS, resd)
    assert torch.equal(resd.cpu(), torch.from_numpy(h).to(dtype))
    codes, step = ref.rows8(h * w.numpy())
    assert np.array_equal(rows.codes.cpu().numpy(), codes)
    want = step.astype(np.float64) * rs
    assert (np.abs(rows.scales.cpu().numpy() - want) <= (slack + 2.0 ** -23) * want).all()
    got = qr.qr_rms_norm(xd, wd, EPS, res.cuda()).float().cpu().numpy()
    want = h.astype(np.float64) * rs[:, None] * w.numpy().astype(np.float64)
    assert (np.abs(got - want) <= (slack + ref.U_OUT[code] * 1.001) * np.abs(want) + ref.TINY[code]).all()
    codes, step = ref.rows8(x.float().numpy())
    rows = qr.qr_q8_quantize(xd)
    assert np.array_equal(rows.codes.cpu().numpy(), codes) and np.array_equal(rows.scales.cpu().numpy(), step)
