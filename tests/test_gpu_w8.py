"""8-bit weights: packing, quantizing and the product of rows in 8 bits
(layer_testlib has the bounds)."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import layer_testlib as ref

pytestmark = pytest.mark.gpu
DT = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _codes(rng, rows, cols, most=127, low=None):
    """int8 codes whose rows begin on 16-byte boundaries, other bytes 99."""
    raw = torch.full((rows, (cols + 15) // 16 * 16), 99, dtype=torch.int8)
    raw[:, :cols] = torch.from_numpy(rng.integers(-most if low is None else low, most + 1, (rows, cols)).astype(np.int8))
    return raw.cuda()[:, :cols]


def _scales(rng, n):
    return torch.from_numpy((rng.random(n) * 0.02 + 0.001).astype(np.float32)).cuda()


def _want(x, sx, w, sw, dtype):
    """The product as every rounding is fixed, for sums below 2^24; and the sums."""
    total = x.cpu().numpy().astype(np.float64) @ w.cpu().numpy().astype(np.float64).T
    y = (total.astype(np.float32) * sx.cpu().numpy()[:, None]) * sw.cpu().numpy()
    return torch.from_numpy(y).to(DT[dtype]), total


def _check_equal(x, sx, w, sw, dtype, y=None, weight=None):
    got = qr.qr_w8_matmul(qr.Q8Rows(x, sx), weight or qr.qr_w8_pack(w, sw), DT[dtype], y)
    want, total = _want(x, sx, w, sw, dtype)
    mag = np.abs(x.cpu().numpy().astype(np.float64)) @ np.abs(w.cpu().numpy().astype(np.float64)).T
    assert mag.max() < 2 ** 24
    assert torch.equal(got.cpu(), want), (got.cpu().float() - want.float()).abs().max()
    return got


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 410, 520, 769, 1100])
def test_tokens(dtype, tokens):
    rng = np.random.default_rng(tokens)
    rows, cols = 272, 960
    _check_equal(_codes(rng, tokens, cols), _scales(rng, tokens), _codes(rng, rows, cols), _scales(rng, rows), dtype)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (16, 64), (17, 65), (33, 31), (5, 127), (15, 129), (100, 1000),
                                       (257, 1024), (64, 1000), (2000, 72), (128, 960), (129, 960), (640, 64), (31, 200)])
@pytest.mark.parametrize("tokens", [1, 5, 16, 23, 48, 100, 140, 270])
def test_shapes(rows, cols, tokens):
    rng = np.random.default_rng(rows * 7 + cols + tokens)
    _check_equal(_codes(rng, tokens, cols), _scales(rng, tokens), _codes(rng, rows, cols), _scales(rng, rows), 1)


@pytest.mark.parametrize("tokens", [1, 12, 16, 20, 40, 90, 300])
@pytest.mark.parametrize("cols", [4095, 8192, 20000])
def test_long_rows(tokens, cols):
    rng = np.random.default_rng(cols + tokens)
    rows = 150
    x, w = _codes(rng, tokens, cols, 7), _codes(rng, rows, cols, 7)
    _check_equal(x, _scales(rng, tokens), w, _scales(rng, rows), 0)


@pytest.mark.parametrize("tokens", [1, 16, 64, 257])
def test_large_sums(tokens):
    """Sums past 2^24: the largest codes, of one sign and of both."""
    rng = np.random.default_rng(tokens)
    rows, cols = 140, 9000
    sx, sw = _scales(rng, tokens), _scales(rng, rows)
    for x, w in ((_codes(rng, tokens, cols, 127, 100), _codes(rng, rows, cols, 127, 90)),
                 (_codes(rng, tokens, cols, 127, -128), _codes(rng, rows, cols, 127, -128)),
                 (_codes(rng, tokens, cols, -128, -128), _codes(rng, rows, cols, -128, -128))):
        got = qr.qr_w8_matmul(qr.Q8Rows(x, sx), qr.qr_w8_pack(w, sw), torch.bfloat16).float().cpu().numpy()
        xs, ws = x.cpu().numpy().astype(np.float64), w.cpu().numpy().astype(np.float64)
        scale = np.outer(sx.cpu().numpy().astype(np.float64), sw.cpu().numpy().astype(np.float64))
        want, mag = (xs @ ws.T) * scale, (np.abs(xs) @ np.abs(ws).T) * scale
        bound = ((cols / 8 + 64) * 2.0 ** -23) * mag + 2.0 ** -8 * 1.001 * np.abs(want)
        assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("tokens", [1, 9, 30, 70, 200])
def test_strides_and_surroundings(tokens):
    rng = np.random.default_rng(tokens)
    rows, cols = 209, 500
    raw = torch.from_numpy(rng.integers(-128, 128, (tokens, 640)).astype(np.int8)).cuda()
    x = raw[:, 16:16 + cols]  # what surrounds a row are codes too
    wide = torch.from_numpy(rng.integers(-128, 128, (rows, 3 * cols + 1)).astype(np.int8)).cuda()
    w = wide[:, 7:7 + cols]
    sx, sw = _scales(rng, tokens), _scales(rng, rows)
    out = torch.full((tokens, rows + 9), 3.0, dtype=torch.float16, device="cuda")
    _check_equal(x, sx, w, sw, 0, y=out[:, 5:5 + rows])
    assert (out[:, :5] == 3).all() and (out[:, 5 + rows:] == 3).all()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,cols", [(1, 1), (20, 100), (130, 1000), (64, 4096)])
def test_quantize(dtype, rows, cols):
    rng = np.random.default_rng(rows)
    w = torch.from_numpy(rng.standard_normal((rows, cols + 3)).astype(np.float32)).to(DT[dtype]).cuda()[:, 1:1 + cols]
    w[0] = 0
    codes, step = ref.rows8(w.float().cpu().numpy())
    a = qr.qr_w8_quantize(w)
    b = qr.qr_w8_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(step).cuda())
    assert torch.equal(a.packed, b.packed)


def test_scales_that_are_not_finite_stay_in_their_row():
    rng = np.random.default_rng(0)
    for tokens in (4, 40, 150):
        x, w = _codes(rng, tokens, 200), _codes(rng, 300, 200)
        sx, sw = _scales(rng, tokens), _scales(rng, 300)
        weight = qr.qr_w8_pack(w, sw)
        good = qr.qr_w8_matmul(qr.Q8Rows(x, sx), weight)
        bad = sx.clone()
        bad[2] = float("nan")
        got = qr.qr_w8_matmul(qr.Q8Rows(x, bad), weight)
        keep = torch.arange(tokens) != 2
        assert torch.equal(got[keep], good[keep]) and torch.isnan(got[2]).all()


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_captured_and_replayed(tokens):
    rng = np.random.default_rng(tokens)
    rows, cols = 400, 700
    w = qr.qr_w8_quantize(torch.randn((rows, cols), device="cuda").half())
    x = torch.randn((tokens, cols), device="cuda").half()
    norm = torch.rand(cols, device="cuda")
    def chain():
        return qr.qr_w8_matmul(qr.qr_rms_norm_q8(x, norm), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = chain()
    for _ in range(3):
        x.normal_()
        graph.replay()
        assert torch.equal(y, chain())


def test_no_tokens_and_refusals():
    rng = np.random.default_rng(1)
    weight = qr.qr_w8_pack(_codes(rng, 40, 64), _scales(rng, 40))
    x = qr.Q8Rows(_codes(rng, 40, 64), _scales(rng, 40))
    assert qr.qr_w8_matmul(x[:0], weight).shape == (0, 40)
    y = torch.zeros((40, 40), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=x.codes), dict(x=qr.Q8Rows.empty(4, 65)), dict(dtype=torch.float32), dict(y=y[:, :39]), dict(y=y[:3]),
                dict(y=y.t()[:, :40].float()), dict(workspace=torch.zeros(9, device="cuda")),
                dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises((TypeError, ValueError)):
            qr.qr_w8_matmul(**{"x": x, "weight": weight, **bad})
    with pytest.raises(qr.QRError):
        qr.qr_w8_matmul(x, weight, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    for args in ((x.codes, x.scales[:3]), (x.codes.float(), x.scales), (x.codes, x.scales.half())):
        with pytest.raises((TypeError, ValueError)):
            qr.qr_w8_pack(*args)
    with pytest.raises((TypeError, ValueError)):
        qr.W8Weight(torch.zeros(10, dtype=torch.uint8, device="cuda"), 40, 64)
