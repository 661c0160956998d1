"""Small angles of qr_rope in relative terms: with one value of a pair 0, the
other one's product with the sine is all there is.

Bound, for angles up to a quarter turn, whose sine errs by no larger a part than
they do: the angle's half turns are off by at most two roundings to fp32, the sine
by an ulp, the factor's and the value's products by a rounding each, 6 * 2^-24 in
all; the table's frequency in turns is a whole number of 2^-64, off by half of
one, and of a double.  2^-21 covers them; then the output's half step."""
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


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,u,tiny", [(torch.float16, 2.0 ** -11, 2.0 ** -25), (torch.bfloat16, 2.0 ** -8, 2.0 ** -134)])
@pytest.mark.parametrize("kw", [dict(base=500000.0, scaling="yarn", factor=8.0, original_len=8192),
                                dict(base=1e8, scaling="linear", factor=32.0)])
def test_the_sine_alone(layout, dtype, u, tiny, kw):
    dim = 128
    freq, factor = qr.rope_frequencies(dim, **kw)
    rope = qr.Rope(freq, layout, factor)
    pos = np.array([1, 2, -1, 3, -7, 12, 100, -1000, 0])
    b = np.random.default_rng(1).uniform(8192, 32768, (len(pos), dim // 2)).astype(np.float32)
    x = torch.zeros((len(pos), 1, dim), dtype=dtype, device="cuda")
    first, second = (slice(0, dim // 2), slice(dim // 2, dim)) if layout == "half" else (slice(0, dim, 2), slice(1, dim, 2))
    x[:, 0, second] = torch.from_numpy(b).to(dtype).cuda()
    got, _ = qr.qr_rope(x, None, rope, torch.from_numpy(pos.astype(np.int32)).cuda())
    got = got[:, 0, first].double().cpu().numpy()
    want = -factor * np.sin(pos[:, None] * freq) * x[:, 0, second].double().cpu().numpy()
    over = np.abs(got - want) - ((2.0 ** -21 + u * 1.001) * np.abs(want) + tiny)
    over = np.where(np.abs(pos[:, None] * freq) <= np.pi / 2, over, 0.0)
    assert (over <= 0).all(), (over.max(), np.unravel_index(over.argmax(), over.shape))
