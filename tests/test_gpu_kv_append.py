"""qr_kv_append against a run-by-run numpy form.  Every rounding of the
definition is one in fp32, so codes and scales have to be equal."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import serving_testlib as ref

pytestmark = pytest.mark.gpu
DT = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _values(rng, shape, dtype, spread=1.0):
    x = rng.standard_normal(shape).astype(np.float32) * np.exp(spread * rng.standard_normal(shape[:1] + (1, 1))).astype(np.float32)
    return torch.from_numpy(x).to(DT[dtype])


def _cache(rng, blocks, heads, bs, dim):
    codes = [rng.integers(-128, 128, (blocks, heads, bs, dim)).astype(np.int8) for _ in range(2)]
    scales = [np.float32(2.0 ** -7) * np.abs(torch.from_numpy(rng.standard_normal((blocks, heads))).bfloat16().float().numpy()) for _ in range(2)]
    return codes, scales


def _check(codes, scales, cache, k, v, slots, bs):
    want = [ref.append(x.float().cpu().numpy(), c, s, slots, bs) for x, c, s in zip((k, v), codes, scales)]
    qr.qr_kv_append(cache, k, v, torch.from_numpy(slots).cuda())
    for got_c, got_s, (c, s) in zip((cache.k_codes, cache.v_codes), (cache.k_scales, cache.v_scales), want):
        assert np.array_equal(got_s.cpu().numpy(), s)
        assert np.array_equal(got_c.cpu().numpy(), c)
    return [c for c, _ in want], [s for _, s in want]


def _upload(codes, scales):
    d = [torch.from_numpy(x).cuda() for x in (*codes, *scales)]
    return qr.KVCache(*d)


def _slots(rng, lens, new, bs, blocks):
    """Slots of requests with `lens` cached and `new` new tokens in random blocks."""
    ids, at, out = rng.permutation(blocks), 0, []
    for c, n in zip(lens, new):
        row = ids[at:at + -(-(c + n) // bs)]
        at += len(row)
        out += [int(row[p // bs]) * bs + p % bs for p in range(c, c + n)]
    return np.array(out, dtype=np.int64)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("bs", [16, 64])
def test_runs(dtype, dim, bs):
    rng = np.random.default_rng(dim + bs + dtype)
    lens, new = [0, 0, 5, bs - 1, bs, 3 * bs + 2, 7], [1, 2 * bs + 3, 1, 1, bs, 4, 0]
    blocks, heads = 24, 3
    codes, scales = _cache(rng, blocks, heads, bs, dim)
    slots = _slots(rng, lens, new, bs, blocks)
    _check(codes, scales, _upload(codes, scales), _values(rng, (len(slots), heads, dim), dtype).cuda(),
           _values(rng, (len(slots), heads, dim), dtype).cuda(), slots, bs)


@pytest.mark.parametrize("bs", [32, 128, 256])
def test_token_by_token(bs):
    """A block filled one token at a time: its scale grows and its codes follow."""
    rng = np.random.default_rng(bs)
    heads, dim = 2, 64
    codes, scales = _cache(rng, 3, heads, bs, dim)
    cache = _upload(codes, scales)
    for p in range(0, bs + 3):
        slots = np.array([(1 if p < bs else 0) * bs + p % bs], dtype=np.int64)
        k, v = (_values(rng, (1, heads, dim), 1, 1.5).cuda() for _ in range(2))
        codes, scales = _check(codes, scales, cache, k, v, slots, bs)


def test_decode_batch_and_prompts():
    rng = np.random.default_rng(9)
    for lens, new, bs in (([int(x) for x in rng.integers(0, 300, 300)], [1] * 300, 16), ([0, 40], [2000, 700], 32)):
        blocks = sum(-(-(c + n) // bs) for c, n in zip(lens, new)) + 2
        codes, scales = _cache(rng, blocks, 2, bs, 128)
        slots = _slots(rng, lens, new, bs, blocks)
        _check(codes, scales, _upload(codes, scales), _values(rng, (len(slots), 2, 128), 1).cuda(),
               _values(rng, (len(slots), 2, 128), 1).cuda(), slots, bs)


def test_skipped_tokens_zeros_extremes_and_ties():
    rng = np.random.default_rng(3)
    bs, heads, dim = 16, 2, 64
    codes, scales = _cache(rng, 6, heads, bs, dim)
    slots = np.array([-1, 0, 1, 2, -1, -1, 6 * 16, 40, 41, 5 * 16 + 15, 1 << 40], dtype=np.int64)
    k, v = (_values(rng, (len(slots), heads, dim), 1) for _ in range(2))
    k[1:4] = 0                                     # a fresh block of zeros
    v[1, 0, :] = torch.tensor([2.0 ** -133, 3e38] * 32).bfloat16()
    k[7, 0] = torch.arange(dim).float() / 2        # halves of a power-of-two scale: ties
    k[7, 0, 0] = 128.0
    k[7:9, 1] = -0.0
    _check(codes, scales, _upload(codes, scales), k.cuda(), v.cuda(), slots, bs)


def test_strided_operands_and_cache():
    """k and v as slices of one projection, the cache's halves as slices of one buffer."""
    rng = np.random.default_rng(5)
    bs, heads, dim, blocks = 32, 3, 80, 9
    codes, scales = _cache(rng, blocks, heads, bs, dim)
    both = torch.full((blocks, heads + 1, 2, bs, dim), 77, dtype=torch.int8, device="cuda")
    both[:, :heads, 0] = torch.from_numpy(codes[0]).cuda()
    both[:, :heads, 1] = torch.from_numpy(codes[1]).cuda()
    cache = qr.KVCache(both[:, :heads, 0], both[:, :heads, 1], *(torch.from_numpy(s).cuda() for s in scales))
    slots = _slots(rng, [4, 0, 31], [40, 33, 2], bs, blocks)
    qkv = _values(rng, (len(slots), 3 * heads + 1, dim), 0).cuda()
    _check(codes, scales, cache, qkv[:, heads:2 * heads], qkv[:, 2 * heads:3 * heads], slots, bs)
    assert (both[:, heads] == 77).all()


def test_non_finite_values_stay_in_their_block_and_head():
    rng = np.random.default_rng(6)
    bs, heads, dim = 16, 2, 64
    codes, scales = _cache(rng, 4, heads, bs, dim)
    cache = _upload(codes, scales)
    slots = np.array([16, 17, 35], dtype=np.int64)
    k, v = (_values(rng, (3, heads, dim), 1) for _ in range(2))
    clean = [ref.append(x.float().numpy(), c, s, slots, bs) for x, c, s in zip((k, v), codes, scales)]
    k[0, 0, 3], k[1, 0, 5] = float("nan"), float("inf")
    qr.qr_kv_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    got_c, got_s = cache.k_codes.cpu().numpy(), cache.k_scales.cpu().numpy()
    got_c[1, 0], got_s[1, 0] = clean[0][0][1, 0], clean[0][1][1, 0]
    assert np.array_equal(got_c, clean[0][0]) and np.array_equal(got_s, clean[0][1])
    assert np.array_equal(cache.v_codes.cpu().numpy(), clean[1][0])


def test_codes_are_the_int8_codec_s():
    """On blocks of 32 values whose scale fp16 holds, the codes are qr_encode(8)'s."""
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.integers(-127, 128, (1, 1, 32)).astype(np.float32) / 16).half()
    x[0, 0, 0] = -8.0
    cache = qr.KVCache.empty(1, 1, 16, 32)
    qr.qr_kv_append(cache, x.cuda(), x.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"))
    wire = qr.qr_encode(8, x.reshape(-1).cuda()).cpu().numpy()
    assert np.array_equal(cache.k_codes.cpu().numpy()[0, 0, 0].astype(np.int64) + 128, wire[:32].astype(np.int64))


def test_no_tokens_and_refusals():
    cache = qr.KVCache.empty(2, 2, 16, 64)
    k = torch.zeros((0, 2, 64), dtype=torch.float16, device="cuda")
    qr.qr_kv_append(cache, k, k, torch.zeros(0, dtype=torch.int64, device="cuda"))
    k = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        qr.qr_kv_append(cache, k.float(), k.float(), slots)
    with pytest.raises(ValueError):
        qr.qr_kv_append(cache, k, k[:2], slots)
    with pytest.raises(ValueError):
        qr.qr_kv_append(cache, k[..., :48], k[..., :48], slots)
    with pytest.raises(TypeError):
        qr.qr_kv_append(cache, k, k, slots.int())
    wide = torch.zeros((3, 2, 68), dtype=torch.float16, device="cuda")
    with pytest.raises(qr.QRError) as e:
        qr.qr_kv_append(cache, wide[..., :64], k, slots)
    assert e.value.status == qr.QR_ERR_MISALIGNED
    with pytest.raises(qr.QRError) as e:
        qr.qr_kv_append(cache, wide.view(-1)[1:385].view(3, 2, 64), k, slots)
    assert e.value.status == qr.QR_ERR_MISALIGNED
    with pytest.raises(ValueError):
        qr.KVCache.empty(2, 2, 24, 64)
    with pytest.raises(qr.QRError) as e:
        qr.qr_kv_append(qr.KVCache.empty(2, 2, 16, 72), torch.zeros((3, 2, 72), dtype=torch.float16, device="cuda"),
                        torch.zeros((3, 2, 72), dtype=torch.float16, device="cuda"), slots)
    assert e.value.status == qr.QR_ERR_UNSUPPORTED
