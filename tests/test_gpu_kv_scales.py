"""qr_kv_attention where value scales lie far apart, as the header accepts any
that are finite and not negative (bounds: serving_testlib)."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import serving_testlib as ref
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _set_v_scales(c, of_block):
    """The value scale of each request's i-th block."""
    for r in range(len(c.kv)):
        for i in range(-(-int(c.kv[r]) // c.bs)):
            c.vs[c.table[r, i]] = np.float32(of_block(i))
    c.cache.v_scales.copy_(torch.from_numpy(c.vs))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("nq", [1, 40, 130])
@pytest.mark.parametrize("low,high", [(-30, 0), (-95, 0), (-99, 25), (-60, 60), (-20, 100), (0, 100)])
@pytest.mark.parametrize("order", [0, 1])
def test_value_scales_far_apart(dtype, nq, low, high, order):
    """Every second group of 16 keys has one scale, the others the other: the
    softmax sum may lose neither.  fp16 outputs that pass the type's range are
    infinite in both."""
    c = Case([700, 384], [nq, nq], 1, 4, bs=16, dtype=dtype, seed=41)
    _set_v_scales(c, lambda i: 2.0 ** (high if (i + order) % 2 else low))
    out, lse = c.run(causal=False)
    want, want_lse, b_out, b_lse = ref.attention(c.q.float().numpy(), c.offsets, c.kv, c.table, c.kc, c.ks, c.vc, c.vs,
                                                 128 ** -0.5, False, 0, dtype)
    assert (np.abs(lse.cpu().numpy() - want_lse) <= b_lse).all()
    got = out.float().cpu().numpy().astype(np.float64)
    most = [65504.0, 3.3895e38][dtype]
    sure = np.abs(want) + b_out < most  # neither can have passed the type's range
    assert (np.abs(got - want)[sure] <= b_out[sure]).all()
    past = np.abs(want) - b_out > 1.001 * most
    assert np.isinf(got[past]).all()


@pytest.mark.parametrize("nq", [1, 40, 130])
def test_one_scale_then_another_far_below_it(nq):
    """A row that has seen a large scale, then tiles of small ones alone."""
    c = Case([900], [nq], 2, 4, bs=32, seed=42)
    _set_v_scales(c, lambda i: 2.0 ** 60 if i < 4 else 2.0 ** -70)
    c.check(causal=False)
    _set_v_scales(c, lambda i: 2.0 ** -70 if i < 4 else 2.0 ** 60)
    c.check()
