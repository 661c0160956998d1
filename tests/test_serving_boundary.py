"""The serving operators' C ABI without a GPU: sizes and refusals.

Every call fails validation, which runs on the host before any CUDA call, so
the made-up addresses are never used; the tests run only where no GPU can be
reached.
"""
import ctypes

import pytest

import bit_quantized_all_gb300 as qr
from bit_quantized_all_gb300 import serving

A, B, C, D, E, F, G, W = (0x7F0000000000 + (i << 36) for i in range(8))  # 16-byte aligned, far apart

no_gpu_only = pytest.mark.skipif(
    __import__("torch").cuda.is_available(),
    reason="made-up device addresses are only passed where no GPU can be reached")


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_quantized_all_gb300 import build
    build.build()
    serving._lib()


def _cache(**kw):
    v = dict(k_codes=A, v_codes=B, k_scales=C, v_scales=D, k_block_stride=2 * 2048, k_head_stride=2048,
             v_block_stride=2 * 2048, v_head_stride=2048, blocks=10, heads=2, block_size=16, head_dim=128)
    v.update(kw)
    return serving.KVCacheStruct(*(v[n] for n, _ in serving.KVCacheStruct._fields_))


@no_gpu_only
def test_plan_refusals():
    ok = dict(requests=4, cached=A, new=B, bs=16, free=C, num_free=8, table=D, width=5, off=E, kv=F, slots=G, most=9,
              counts=W, stream=None)

    def call(**kw):
        return serving._lib().qr_kv_plan(*{**ok, **kw}.values())

    for kw in (dict(requests=0), dict(cached=None), dict(new=None), dict(table=None), dict(off=None), dict(kv=None),
               dict(counts=None), dict(width=0), dict(num_free=-1), dict(most=-1), dict(free=None), dict(slots=None),
               dict(kv=E + 4), dict(off=A), dict(table=B - 8), dict(slots=C + 16), dict(counts=D + 76)):
        assert call(**kw) == qr.QR_ERR_INVALID_ARG, kw
    for kw in (dict(bs=0), dict(bs=24), dict(bs=512), dict(requests=65537)):
        assert call(**kw) == qr.QR_ERR_UNSUPPORTED, kw
    assert call(most=1 << 31) == qr.QR_ERR_SIZE
    for kw in (dict(cached=A + 2), dict(slots=G + 4), dict(table=D + 1)):
        assert call(**kw) == qr.QR_ERR_MISALIGNED, kw


@no_gpu_only
def test_append_refusals():
    ok = dict(dtype=1, tokens=7, k=E, v=F, kt=512, kh=128, vt=512, vh=128, slots=G, cache=_cache(), stream=None)

    def call(**kw):
        v = {**ok, **kw}
        v["cache"] = ctypes.addressof(v["cache"]) if v["cache"] is not None else None
        return serving._lib().qr_kv_append(*v.values())

    for kw in (dict(tokens=0), dict(k=None), dict(v=None), dict(slots=None), dict(cache=None),
               dict(cache=_cache(k_codes=None)), dict(cache=_cache(blocks=0)), dict(cache=_cache(heads=0)),
               dict(k=A), dict(v=C), dict(slots=B + 8)):
        assert call(**kw) == qr.QR_ERR_INVALID_ARG, kw
    for kw in (dict(dtype=2), dict(cache=_cache(head_dim=72)), dict(cache=_cache(head_dim=272)),
               dict(cache=_cache(block_size=48))):
        assert call(**kw) == qr.QR_ERR_UNSUPPORTED, kw
    for kw in (dict(tokens=1 << 31), dict(kt=64), dict(vh=64), dict(kt=1 << 60), dict(cache=_cache(k_head_stride=1024)),
               dict(cache=_cache(v_block_stride=2048)), dict(cache=_cache(k_block_stride=1 << 60))):
        assert call(**kw) == qr.QR_ERR_SIZE, kw
    for kw in (dict(k=E + 2), dict(kt=516), dict(vh=132), dict(slots=G + 4), dict(cache=_cache(k_codes=A + 8)),
               dict(cache=_cache(k_head_stride=2056, k_block_stride=5000)), dict(cache=_cache(v_scales=D + 2))):
        assert call(**kw) == qr.QR_ERR_MISALIGNED, kw


@no_gpu_only
def test_attention_refusals():
    ok = dict(dtype=0, requests=3, tokens=9, q_heads=8, q=E, qt=1024, qh=128, off=F, kv=F + 4096, table=F + 8192,
              width=6, cache=_cache(), scale=0.1, causal=1, window=0, max_q=9, out=G, ot=1024, oh=128, lse=None,
              ws=W, ws_bytes=1 << 34, stream=None)

    def call(**kw):
        v = {**ok, **kw}
        v["cache"] = ctypes.addressof(v["cache"]) if v["cache"] is not None else None
        return serving._lib().qr_kv_attention(*v.values())

    for kw in (dict(requests=0), dict(tokens=0), dict(q_heads=0), dict(q=None), dict(off=None), dict(kv=None),
               dict(table=None), dict(cache=None), dict(out=None), dict(ws=None), dict(width=0), dict(max_q=0),
               dict(window=-1), dict(window=3, causal=0), dict(scale=float("nan")), dict(scale=float("-inf")),
               dict(out=E), dict(out=A), dict(lse=G + 16), dict(ws=E)):
        assert call(**kw) == qr.QR_ERR_INVALID_ARG, kw
    for kw in (dict(dtype=3), dict(q_heads=9), dict(requests=65537), dict(q_heads=65536),
               dict(cache=_cache(head_dim=8))):
        assert call(**kw) == qr.QR_ERR_UNSUPPORTED, kw
    for kw in (dict(width=1 << 27), dict(tokens=1 << 31), dict(qt=100), dict(oh=1 << 58), dict(ws_bytes=8),
               dict(ot=128, oh=128)):
        assert call(**kw) == qr.QR_ERR_SIZE, kw
    for kw in (dict(q=E + 4), dict(out=G + 8), dict(qt=1028), dict(oh=132, ot=1056), dict(lse=B + 2), dict(ws=W + 8),
               dict(off=F + 2)):
        assert call(**kw) == qr.QR_ERR_MISALIGNED, kw


def test_w4_sizes():
    assert qr.qr_w4_bytes(16, 64, 32) == 512 + 64 and qr.qr_w4_bytes(16, 64, 64, True) == 512 + 32 + 16
    assert qr.qr_w4_bytes(17, 65, 128) == 2 * (2 * 512 + 32)
    assert qr.qr_w4_bytes(1, 1, 32, True) == 512 + 64 + 32
    for bad in ((0, 64, 32), (16, 0, 32), (16, 64, 16), (16, 64, 0), (-1, 64, 32), (2 ** 31 - 1, 64, 32)):
        assert qr.qr_w4_bytes(*bad) == 0
    assert qr.qr_w4_matvec_workspace_bytes(17, 65) == 17 * 2 * 128 and qr.qr_w4_matvec_workspace_bytes(0, 65) == 0
    assert qr.qr_kv_attention_workspace_bytes(4, 4, 8, 2, 128) > 0
    for bad in ((0, 4, 8, 2, 128), (4, 0, 8, 2, 128), (4, 4, 8, 3, 128), (4, 4, 1, 2, 128), (4, 4, 8, 2, 100)):
        assert qr.qr_kv_attention_workspace_bytes(*bad) == 0


@no_gpu_only
def test_w4_refusals():
    L = serving._lib()
    pack = dict(rows=8, cols=64, group=32, codes=A, scales=B, zeros=None, packed=C, stream=None)
    quant = dict(dtype=1, rows=8, cols=64, group=32, w=A, stride=64, packed=C, stream=None)
    mul = dict(dtype=1, tokens=2, x=A, xs=64, rows=8, cols=64, group=32, zeros=0, packed=B, y=C, ys=8, ws=None,
               ws_bytes=0, stream=None)

    def call(fn, base, **kw):
        return getattr(L, fn)(*{**base, **kw}.values())

    for fn, base, kw, want in (
            ("qr_w4_pack", pack, dict(codes=None), 1), ("qr_w4_pack", pack, dict(rows=0), 1),
            ("qr_w4_pack", pack, dict(group=48), 2), ("qr_w4_pack", pack, dict(cols=2 ** 31 - 1), 4),
            ("qr_w4_pack", pack, dict(packed=C + 8), 3), ("qr_w4_pack", pack, dict(scales=B + 1), 3),
            ("qr_w4_pack", pack, dict(packed=A), 1), ("qr_w4_pack", pack, dict(zeros=C + 16), 1),
            ("qr_w4_quantize", quant, dict(w=None), 1), ("qr_w4_quantize", quant, dict(dtype=7), 2),
            ("qr_w4_quantize", quant, dict(stride=63), 4), ("qr_w4_quantize", quant, dict(w=A + 1), 3),
            ("qr_w4_quantize", quant, dict(packed=A), 1),
            ("qr_w4_matvec", mul, dict(tokens=0), 1), ("qr_w4_matvec", mul, dict(x=None), 1),
            ("qr_w4_matvec", mul, dict(dtype=-1), 2), ("qr_w4_matvec", mul, dict(group=16), 2),
            ("qr_w4_matvec", mul, dict(xs=63), 4), ("qr_w4_matvec", mul, dict(ys=7), 4),
            ("qr_w4_matvec", mul, dict(tokens=1 << 31), 4), ("qr_w4_matvec", mul, dict(y=C + 1), 3),
            ("qr_w4_matvec", mul, dict(packed=B + 4), 3), ("qr_w4_matvec", mul, dict(y=A), 1),
            ("qr_w4_matvec", mul, dict(y=B), 1),
            # 17 unaligned rows need a workspace of their size
            ("qr_w4_matvec", mul, dict(tokens=17, x=A + 2, ws=D, ws_bytes=17 * 128 - 1), 4),
            ("qr_w4_matvec", mul, dict(tokens=17, xs=65), 4),
            ("qr_w4_matvec", mul, dict(tokens=17, xs=65, ws=D + 8, ws_bytes=1 << 20), 3),
            ("qr_w4_matvec", mul, dict(tokens=17, xs=65, ws=B, ws_bytes=1 << 20), 1)):
        assert call(fn, base, **kw) == want, (fn, kw)


def test_tensors_must_be_on_a_gpu():
    import torch
    with pytest.raises(ValueError):
        qr.KVCache(torch.zeros((1, 1, 16, 64), dtype=torch.int8), torch.zeros((1, 1, 16, 64), dtype=torch.int8),
                   torch.zeros((1, 1)), torch.zeros((1, 1)))
    with pytest.raises(ValueError):
        qr.qr_w4_pack(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.float16), 64, 32)
    with pytest.raises(ValueError):
        qr.qr_w4_quantize(torch.zeros((4, 64), dtype=torch.float16))
