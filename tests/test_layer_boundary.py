"""The C ABI of the norm, the rotary positions and the 8-bit product without a
GPU: sizes and refusals (made-up addresses, never used: validation runs before
any CUDA call), and the frequencies of scaled positions."""
import math

import numpy as np
import pytest

import bit_quantized_all_gb300 as qr
from bit_quantized_all_gb300 import layer

A, B, C, D, E, F, G, W = (0x7F0000000000 + (i << 36) for i in range(8))  # 16-byte aligned, far apart

no_gpu_only = pytest.mark.skipif(
    __import__("torch").cuda.is_available(),
    reason="made-up device addresses are only passed where no GPU can be reached")

INVALID, UNSUPPORTED, MISALIGNED, SIZE = (qr.QR_ERR_INVALID_ARG, qr.QR_ERR_UNSUPPORTED, qr.QR_ERR_MISALIGNED,
                                          qr.QR_ERR_SIZE)


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_quantized_all_gb300 import build
    build.build()
    layer._lib()


def _refused(name, ok, cases):
    for kw, want in cases:
        assert set(kw) <= set(ok), kw
        assert getattr(layer._lib(), name)(*{**ok, **kw}.values()) == want, (name, kw)


@no_gpu_only
def test_quantize_refusals():
    ok = dict(dtype=1, tokens=4, cols=100, x=A, xs=100, codes=B, cs=112, scales=C, stream=None)
    _refused("qr_q8_quantize", ok, [
        (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(tokens=0), INVALID),
        (dict(cols=0), INVALID), (dict(codes=A), INVALID), (dict(scales=A + 700), INVALID), (dict(scales=B + 16), INVALID),
        (dict(dtype=2), UNSUPPORTED), (dict(xs=99), SIZE), (dict(cs=96), SIZE), (dict(tokens=1 << 31), SIZE),
        (dict(xs=1 << 60), SIZE), (dict(tokens=1, cols=(1 << 30) + 1), SIZE), (dict(x=A + 1), MISALIGNED), (dict(codes=B + 8), MISALIGNED), (dict(cs=120), MISALIGNED),
        (dict(scales=C + 2), MISALIGNED)])


@no_gpu_only
@pytest.mark.parametrize("eight", [False, True])
def test_norm_refusals(eight):
    ok = dict(dtype=0, tokens=4, cols=100, x=A, xs=112, res=B, rs=100, out=C, os=100, w=D, w32=0, eps=1e-6, y=E, ys=112)
    if eight:
        ok["scales"] = F
    ok["stream"] = None
    cases = [
        (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(res=None), INVALID),
        (dict(tokens=0), INVALID), (dict(cols=-1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
        (dict(eps=float("inf")), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(xs=90), SIZE), (dict(rs=99), SIZE),
        (dict(os=1 << 60), SIZE), (dict(ys=64), SIZE), (dict(tokens=1 << 31), SIZE), (dict(x=A + 1), MISALIGNED),
        (dict(w=D + 2, w32=1), MISALIGNED), (dict(out=C + 1), MISALIGNED),
        (dict(out=A), INVALID),  # x's strides are others
        (dict(out=B + 2), INVALID), (dict(out=D), INVALID), (dict(y=D + 160), INVALID), (dict(y=C), INVALID),
        (dict(out=E), INVALID), (dict(y=A + 16), INVALID)]
    if eight:
        cases += [(dict(y=A), INVALID), (dict(scales=None), INVALID), (dict(scales=A), INVALID), (dict(scales=E), INVALID),
                  (dict(y=E + 8), MISALIGNED), (dict(ys=104), MISALIGNED), (dict(scales=F + 1), MISALIGNED)]
    _refused("qr_rms_norm_q8" if eight else "qr_rms_norm", ok, cases)


def test_w8_sizes():
    assert qr.qr_w8_bytes(16, 64) == 1024 + 64 and qr.qr_w8_bytes(17, 65) == 2 * (2 * 1024 + 64)
    for bad in ((0, 64), (16, 0), (-1, 64), (2 ** 31 - 1, 64), (16, 2 ** 31 - 1)):
        assert qr.qr_w8_bytes(*bad) == 0
    assert qr.qr_w8_matmul_workspace_bytes(17, 65) >= 17 * 128 * 2
    assert qr.qr_w8_matmul_workspace_bytes(0, 65) == 0 and qr.qr_w8_matmul_workspace_bytes(5, 0) == 0
    # a workspace of more tokens serves fewer
    sizes = [qr.qr_w8_matmul_workspace_bytes(t, 640) for t in range(1, 1200)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@no_gpu_only
def test_w8_refusals():
    pack = dict(rows=20, cols=100, codes=A, stride=100, scales=B, packed=C, stream=None)
    _refused("qr_w8_pack", pack, [
        (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(packed=None), INVALID), (dict(rows=0), INVALID),
        (dict(cols=2 ** 31 - 1), SIZE), (dict(stride=99), SIZE), (dict(packed=C + 8), MISALIGNED),
        (dict(scales=B + 2), MISALIGNED), (dict(packed=A), INVALID), (dict(packed=B), INVALID)])
    quant = dict(dtype=1, rows=20, cols=100, w=A, stride=100, packed=C, stream=None)
    _refused("qr_w8_quantize", quant, [
        (dict(w=None), INVALID), (dict(packed=None), INVALID), (dict(cols=0), INVALID), (dict(dtype=9), UNSUPPORTED),
        (dict(stride=9), SIZE), (dict(w=A + 1), MISALIGNED), (dict(packed=C + 4), MISALIGNED), (dict(packed=A), INVALID)])
    need = qr.qr_w8_matmul_workspace_bytes(17, 100)
    mul = dict(dtype=1, tokens=17, x=A, xs=112, xsc=B, rows=20, cols=100, packed=C, y=D, ys=20, ws=E, ws_bytes=need,
               stream=None)
    _refused("qr_w8_matmul", mul, [
        (dict(x=None), INVALID), (dict(xsc=None), INVALID), (dict(packed=None), INVALID), (dict(y=None), INVALID),
        (dict(tokens=0), INVALID), (dict(rows=0), INVALID), (dict(dtype=-1), UNSUPPORTED), (dict(xs=96), SIZE),
        (dict(ys=19), SIZE), (dict(tokens=1 << 31), SIZE), (dict(ws=None), SIZE), (dict(ws_bytes=need - 1), SIZE),
        (dict(x=A + 8), MISALIGNED), (dict(xs=120), MISALIGNED), (dict(packed=C + 8), MISALIGNED), (dict(y=D + 1), MISALIGNED),
        (dict(ws=E + 8), MISALIGNED), (dict(y=A), INVALID), (dict(y=B), INVALID), (dict(y=C), INVALID),
        (dict(ws=A), INVALID), (dict(ws=C), INVALID), (dict(ws=D), INVALID)])


@no_gpu_only
def test_rope_refusals():
    ok = dict(dtype=1, tokens=5, dim=64, rot=64, inter=0, turns=A, factor=1.0, pos=B, requests=0, off=None, kv=None,
              q=C, qt=640, qh=64, hq=8, qo=D, qot=512, qoh=64, k=C + 1024, kt=640, kh=64, hk=2, ko=E, kot=128, koh=64,
              stream=None)
    plan = dict(pos=None, requests=3, off=F, kv=G)
    _refused("qr_rope", ok, [
        (dict(turns=None), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(tokens=0), INVALID),
        (dict(hq=0), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID), (dict(hk=0), INVALID), (dict(rot=0), INVALID),
        (dict(pos=None), INVALID), (dict(plan, requests=0), INVALID), (dict(plan, off=None), INVALID),
        (dict(plan, kv=None), INVALID), (dict(factor=float("inf")), INVALID), (dict(dtype=2), UNSUPPORTED),
        (dict(rot=63), UNSUPPORTED), (dict(rot=66), UNSUPPORTED), (dict(dim=1026, rot=2), UNSUPPORTED),
        (dict(dim=63, rot=62), UNSUPPORTED), (dict(hq=70000), UNSUPPORTED), (dict(plan, requests=65537), UNSUPPORTED),
        (dict(qt=63), SIZE), (dict(koh=63), SIZE), (dict(tokens=1 << 31), SIZE), (dict(qot=64, qoh=64), SIZE),
        (dict(q=C + 1), MISALIGNED), (dict(ko=E + 1), MISALIGNED), (dict(turns=A + 4), MISALIGNED), (dict(pos=B + 2), MISALIGNED),
        (dict(plan, kv=G + 2), MISALIGNED),
        (dict(qo=C), INVALID),   # q in place with other strides
        (dict(qo=C + 2, qot=640), INVALID), (dict(qo=E), INVALID), (dict(ko=C, kot=640), INVALID), (dict(qo=A), INVALID),
        (dict(qo=B), INVALID), (dict(plan, ko=F), INVALID)])


def test_frequencies():
    f, factor = qr.rope_frequencies(8, 10000.0)
    assert np.allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-14) and factor == 1.0
    assert np.allclose(qr.rope_frequencies(8, scaling="linear", factor=4.0)[0], f / 4, rtol=1e-14)
    ntk = qr.rope_frequencies(8, scaling="ntk", factor=4.0)[0]
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], f[-1] / 4, rtol=1e-12)  # the slowest pair is stretched by the factor
    g, factor = qr.rope_frequencies(128, scaling="yarn", factor=16.0, original_len=4096)
    plain = qr.rope_frequencies(128)[0]
    assert np.allclose(g[:16], plain[:16]) and np.allclose(g[-8:], plain[-8:] / 16) and (np.diff(g / plain) <= 1e-12).all()
    assert math.isclose(factor, 0.1 * math.log(16) + 1)
    for kw in (dict(rot_dim=7), dict(rot_dim=0), dict(base=1.0), dict(factor=0.5, scaling="linear"), dict(scaling="other"),
               dict(scaling="yarn", factor=2.0), dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            qr.rope_frequencies(**{"rot_dim": 64, **kw})


def test_tables_and_tensors():
    import torch
    rope = qr.Rope([1.0, 0.5], device="cpu")
    assert rope.rot_dim == 4 and rope.turns.tolist() == [round(2 ** 64 / (2 * math.pi)), round(2 ** 63 / (2 * math.pi))]
    for kw in (dict(frequencies=[]), dict(frequencies=[4.0]), dict(frequencies=[float("nan")]), dict(layout="other"),
               dict(factor=float("inf"))):
        with pytest.raises(ValueError):
            qr.Rope(**{"frequencies": [1.0], "device": "cpu", **kw})
    x = torch.zeros((4, 64), dtype=torch.float16)
    for call in (lambda: qr.qr_q8_quantize(x), lambda: qr.qr_rms_norm(x, x[0]), lambda: qr.qr_w8_quantize(x),
                 lambda: qr.Q8Rows(x.to(torch.int8), x[:, 0].float()),
                 lambda: qr.qr_rope(x[:, None], None, rope, torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
