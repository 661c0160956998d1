"""qr_kv_attention's second product against the definition in 64 bits, with the
softmax weights held to two fp16 numbers.

The bound, derived: a weight that enters as hi + lo, both fp16, is off by at
most 2^-11 * 2^-11 = 2^-22 of itself, and by 2^-25 of the row's largest where
lo falls below fp16's range.  With d = 2^-19 |scale| max_i sum |q k_i| + 2^-20
for the scores (serving_testlib), B = sum_i P_i |v_i| and fp32 sums,
    |d out| <= (2^-22 + 2 d + 2^-18) B + 2^-25 sum_i |v_i| / l + u_out |out|.
The inputs make B large and out small: the values of a dimension are half +127
and half -127 and the scores nearly equal, so the output's own rounding hides
nothing.  One fp16 number per weight is off by up to 2^-12 of it.
"""
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


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("keys", [2, 4, 16, 128, 256])
@pytest.mark.parametrize("nq", [4, 40])
def test_weights_keep_what_one_fp16_number_loses(dtype, dim, keys, nq):
    c = Case([keys], [nq], 1, 4, dim=dim, bs=16, dtype=dtype, seed=keys + dim)
    rng = np.random.default_rng(keys)
    signs = np.stack([rng.permutation(np.repeat([127, -127], keys // 2)) for _ in range(dim)], 1)
    blocks = c.table[0, :-(-keys // 16)]
    flat = np.zeros((len(blocks) * 16, dim), np.int8)
    flat[:keys] = signs
    c.vc[blocks, 0] = flat.reshape(len(blocks), 16, dim)
    c.ks[blocks], c.vs[blocks] = np.float32(1e-4), np.float32(0.02)
    c.cache.v_codes.copy_(torch.from_numpy(c.vc))
    c.cache.k_scales.copy_(torch.from_numpy(c.ks))
    c.cache.v_scales.copy_(torch.from_numpy(c.vs))
    out, _ = c.run(causal=False)
    k = (c.kc[blocks, 0].astype(np.float64) * c.ks[blocks, 0].astype(np.float64)[:, None, None]).reshape(-1, dim)[:keys]
    v = flat[:keys].astype(np.float64) * np.float64(np.float32(0.02))
    q = c.q.float().numpy().astype(np.float64)
    s = np.einsum("thd,kd->thk", q, k) * dim ** -0.5
    mag = np.einsum("thd,kd->thk", np.abs(q), np.abs(k)).max(-1) * dim ** -0.5
    e = np.exp(s - s.max(-1, keepdims=True))
    l = e.sum(-1, keepdims=True)
    want, B = (e / l) @ v, (e / l) @ np.abs(v)
    d = (2.0 ** -19 * mag + 2.0 ** -20)[..., None]
    bound = ((2.0 ** -22 + 2 * d + 2.0 ** -18) * B + 2.0 ** -25 * np.abs(v).sum(0) / l
             + ref.U_OUT[dtype] * np.abs(want) + ref.TINY[dtype])
    over = np.abs(out.float().cpu().numpy() - want) / bound
    assert over.max() <= 1, over.max()
