"""qr_kv_append of magnitudes so small that the inverse of their scale is beyond
fp32: codes are 0 there, and equal to the definition everywhere."""
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


def _append(x, codes, scales, slots, bs):
    """serving_testlib.append with 1 / s taken as 0 where fp32 does not hold it."""
    codes, scales = codes.copy(), scales.copy()
    x, t = x.astype(np.float32), 0
    while t < len(slots):
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t] + n and (slots[t] + n) % bs:
            n += 1
        b, o = divmod(int(slots[t]), bs)
        for h in range(codes.shape[1]):
            run = x[t:t + n, h]
            old = scales[b, h] if o else np.float32(0)
            new = np.maximum(old, np.float32(np.abs(run).max()) * np.float32(2.0 ** -7))
            with np.errstate(all="ignore"):
                r = np.float32(1) / new
            if not np.isfinite(r):
                r = np.float32(0)
            if o and new > old:
                codes[b, h, :o] = np.rint(np.clip(codes[b, h, :o].astype(np.float32) * old * r, -128, 127))
            codes[b, h, o:o + n] = np.rint(np.clip(run * r, -128, 127))
            scales[b, h] = new
        t += n
    return codes, scales


@pytest.mark.parametrize("exponent", [-133, -130, -122, -121, -120, -118, -100])
def test_append_of_magnitudes_whose_inverse_scale_overflows(exponent):
    """A whole block around 2^exponent, with zeros and negatives; then a second
    run into the same block, as large and larger."""
    rng = np.random.default_rng(-exponent)
    bs, heads, dim = 16, 2, 32
    cache = qr.KVCache.empty(3, heads, bs, dim)
    codes, scales = np.zeros((3, heads, bs, dim), np.int8), np.zeros((3, heads), np.float32)
    for first, n, up in ((16, 5, 0), (21, 3, 0), (24, 2, 3), (26, 1, 40)):
        x = rng.uniform(-1, 1, (n, heads, dim)) * 2.0 ** min(exponent + up, 0)
        x[:, :, :8] = 0
        x[0, :, 9], x[0, :, 10] = 2.0 ** (exponent + up), -2.0 ** (exponent + up)
        x = torch.from_numpy(x.astype(np.float32)).bfloat16()
        slots = np.arange(first, first + n)
        codes, scales = _append(x.float().numpy(), codes, scales, slots, bs)
        qr.qr_kv_append(cache, x.cuda(), x.cuda(), torch.from_numpy(slots).cuda())
        for got_c, got_s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
            assert np.array_equal(got_s.cpu().numpy(), scales)
            assert np.array_equal(got_c.cpu().numpy(), codes)
