"""Rows in 8 bits and the root-mean-square norm against their definitions
(layer_testlib has the bounds)."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import layer_testlib as ref

pytestmark = pytest.mark.gpu
DT = [torch.float16, torch.bfloat16]
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _x(rng, shape, dtype, big=8.0):
    x = rng.standard_normal(shape).astype(np.float32)
    x[..., rng.integers(0, shape[-1])] *= big
    return torch.from_numpy(x).to(DT[dtype])


def _f32(t):
    return t.float().cpu().numpy()


def _sum(x, res):
    return _f32(x) if res is None else _f32(x) + _f32(res)


def _check(x, w, res, eight, dtype, out=None, residual_out=None):
    """Device tensors in; compares outputs and the residual's sum."""
    h = _sum(x, res)
    cols = h.shape[1]
    rs = 1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(1) + EPS)
    slack = ref.norm_slack(cols)
    call = qr.qr_rms_norm_q8 if eight else qr.qr_rms_norm
    if res is not None and residual_out is None:
        residual_out = torch.empty_like(res)
    got = call(x, w, EPS, res, residual_out, out)
    if res is not None:
        assert torch.equal(residual_out.cpu(), torch.from_numpy(h).to(DT[dtype])), "residual"
    if eight:
        codes, step = ref.rows8(h * _f32(w))
        assert np.array_equal(got.codes.cpu().numpy(), codes)
        want = step.astype(np.float64) * rs
        assert (np.abs(got.scales.cpu().numpy() - want) <= (slack + 2.0 ** -23) * want).all()
    else:
        want = h.astype(np.float64) * rs[:, None] * _f32(w).astype(np.float64)
        bound = (slack + ref.U_OUT[dtype] * 1.001) * np.abs(want) + ref.TINY[dtype]
        over = np.abs(_f32(got) - want) - bound
        assert (over <= 0).all(), over.max()
    return got


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("tokens,cols", [(1, 1), (3, 7), (2, 8), (5, 64), (7, 129), (4, 1000), (33, 1024), (9, 1032),
                                         (3, 2047), (2, 5123), (17, 8192), (3, 16384), (2, 24575), (2, 40000), (1, 70001)])
def test_shapes(dtype, eight, residual, tokens, cols):
    rng = np.random.default_rng(tokens * 1000 + cols)
    x = _x(rng, (tokens, cols), dtype).cuda()
    res = _x(rng, (tokens, cols), dtype, 3.0).cuda() if residual else None
    for w in (torch.from_numpy(rng.random(cols).astype(np.float32) + 0.5).cuda(), _x(rng, (cols,), dtype).cuda()):
        _check(x, w, res, eight, dtype)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens,cols", [(1, 1), (4, 63), (6, 512), (300, 768), (2, 5121), (19, 8192), (2, 30001)])
def test_quantize(dtype, tokens, cols):
    rng = np.random.default_rng(cols)
    x = _x(rng, (tokens, cols), dtype)
    x[0] = 0
    y = qr.qr_q8_quantize(x.cuda())
    codes, step = ref.rows8(_f32(x))
    assert np.array_equal(y.codes.cpu().numpy(), codes)
    assert np.abs(y.scales.cpu().numpy() - step).max() <= 2.0 ** -24 * step.max()
    assert np.array_equal(y.scales.cpu().numpy(), step)  # (division is correctly rounded on both sides)


@pytest.mark.parametrize("tokens,cols", [(2000, 96), (1500, 200), (700, 3000), (400, 8192), (300, 20480), (513, 5123)])
@pytest.mark.parametrize("eight", [False, True])
def test_many_rows(tokens, cols, eight):
    rng = np.random.default_rng(tokens)
    x, res = _x(rng, (tokens, cols), 1).cuda(), _x(rng, (tokens, cols), 1).cuda()
    w = _x(rng, (cols,), 1).cuda()
    _check(x, w, res, eight, 1)
    _check(x, w, None, eight, 1)


@pytest.mark.parametrize("cols", [96, 1000, 1001, 4096])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strided_rows_leave_their_surroundings(cols, off):
    rng = np.random.default_rng(cols + off)
    wide = [_x(rng, (9, cols + 24 + (off & 1)), 0).cuda() for _ in range(4)]
    kept = [t.clone() for t in wide]
    x, res, res_out, y = (t[:, off:off + cols] for t in wide)
    w = _x(rng, (cols,), 0).cuda()
    _check(x, w, res, False, 0, out=y, residual_out=res_out)
    for t, k in zip(wide, kept):
        assert torch.equal(t[:, :off], k[:, :off]) and torch.equal(t[:, off + cols:], k[:, off + cols:])
    assert torch.equal(wide[0], kept[0]) and torch.equal(wide[1], kept[1])
    raw = torch.full((9, (cols + 15) // 16 * 16 + 16), 77, dtype=torch.int8, device="cuda")
    q8 = qr.Q8Rows(raw[:, :cols], torch.empty(9, device="cuda"))
    _check(x, w, res, True, 0, out=q8, residual_out=res_out)
    assert (raw[:, cols:] == 77).all()
    qr.qr_q8_quantize(x, out=q8)
    assert (raw[:, cols:] == 77).all()


@pytest.mark.parametrize("tokens", [5, 3000])
@pytest.mark.parametrize("cols", [33, 640, 1003])
def test_rows_on_unlike_boundaries(cols, tokens):
    """Operands that do not lie alike between 16-byte words, one after the other."""
    rng = np.random.default_rng(cols)
    plain = [_x(rng, (tokens, cols), 1).cuda() for _ in range(2)]
    w = _x(rng, (cols,), 1).cuda()
    odd_w = torch.zeros(cols + 3, dtype=torch.bfloat16, device="cuda")[3:].copy_(w)
    for which in range(5):
        wide = torch.full((tokens, cols + 13), 2.0, dtype=torch.bfloat16, device="cuda")
        odd = wide[:, 5:5 + cols]
        x, res = (odd.copy_(t) if which == i else t for i, t in enumerate(plain))
        res_out = odd if which == 2 else torch.empty_like(plain[0])
        y = odd if which == 3 else None
        _check(x, odd_w if which == 4 else w, res, False, 1, out=y, residual_out=res_out)
        assert (wide[:, :5] == 2).all() and (wide[:, 5 + cols:] == 2).all()
        _check(x, odd_w if which == 4 else w, res, True, 1, residual_out=res_out)
        assert (wide[:, :5] == 2).all() and (wide[:, 5 + cols:] == 2).all()


@pytest.mark.parametrize("cols", [512, 1001, 40000])
def test_in_place(cols):
    rng = np.random.default_rng(cols)
    w = _x(rng, (cols,), 1).cuda()
    x, res = _x(rng, (5, cols), 1).cuda(), _x(rng, (5, cols), 1).cuda()
    fresh = torch.empty_like(res)
    want = qr.qr_rms_norm(x, w, EPS, res, fresh)
    x2, res2 = x.clone(), res.clone()
    got = qr.qr_rms_norm(x2, w, EPS, res2, out=x2)  # the residual in place by default, the output over x
    assert got is x2 and torch.equal(x2, want) and torch.equal(res2, fresh)
    x2, res2 = x.clone(), res.clone()
    qr.qr_rms_norm(x2, w, EPS, res2, residual_out=x2, out=res2)  # crosswise
    assert torch.equal(res2, want) and torch.equal(x2, fresh)
    q8 = qr.qr_rms_norm_q8(x, w, EPS, res, torch.empty_like(res))
    x2 = x.clone()
    got = qr.qr_rms_norm_q8(x2, w, EPS, res, residual_out=x2)
    assert torch.equal(got.codes, q8.codes) and torch.equal(got.scales, q8.scales) and torch.equal(x2, fresh)


@pytest.mark.parametrize("tokens", [3, 200, 2500])
@pytest.mark.parametrize("cols", [33, 251, 1001, 5123, 17001])
def test_residual_in_place_at_odd_sizes(cols, tokens):
    """A warp's last lane has a piece of the next warp's, which that one overwrites."""
    rng = np.random.default_rng(cols)
    x, res, w = _x(rng, (tokens, cols), 1).cuda(), _x(rng, (tokens, cols), 1).cuda(), _x(rng, (cols,), 1).cuda()
    fresh = torch.empty_like(res)
    want = qr.qr_rms_norm_q8(x, w, EPS, res, fresh)
    for _ in range(5):
        res2, x2 = res.clone(), x.clone()
        got = qr.qr_rms_norm_q8(x2, w, EPS, res2)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales) and torch.equal(res2, fresh)
        got = qr.qr_rms_norm_q8(x2, w, EPS, res, residual_out=x2)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales) and torch.equal(x2, fresh)


@pytest.mark.parametrize("cols", [64, 8192, 5123])
def test_small_and_large_values(cols):
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((6, cols)).astype(np.float32)
    x *= np.array([1e-38, 1e-30, 1e-3, 1e4, 1e15, 0], dtype=np.float32)[:, None]
    x = torch.from_numpy(x).bfloat16().cuda()
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    _check(x, w, None, False, 1)
    _check(x, w, None, True, 1)
    y = qr.qr_rms_norm(x, w, EPS)
    assert (y[5] == 0).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("cols", [80, 8192, 5123])
def test_a_row_that_is_not_finite_stays_alone(value, cols):
    rng = np.random.default_rng(cols)
    x = _x(rng, (4, cols), 1).cuda()
    w = _x(rng, (cols,), 1).cuda()
    bad = x.clone()
    bad[2, cols // 3] = value
    good, other = qr.qr_rms_norm(x, w, EPS), qr.qr_rms_norm(bad, w, EPS)
    keep = torch.tensor([0, 1, 3])
    assert torch.equal(good[keep], other[keep]) and not torch.isfinite(other[2, cols // 3])
    good, other = qr.qr_rms_norm_q8(x, w, EPS), qr.qr_rms_norm_q8(bad, w, EPS)
    assert torch.equal(good.codes[keep], other.codes[keep]) and torch.equal(good.scales[keep], other.scales[keep])
    assert not torch.isfinite(other.scales[2])
    assert not torch.isfinite(qr.qr_q8_quantize(bad).scales[2])


def test_no_tokens_and_refusals():
    x = torch.zeros((0, 64), dtype=torch.float16, device="cuda")
    w = torch.zeros(64, dtype=torch.float16, device="cuda")
    assert qr.qr_rms_norm(x, w).shape == (0, 64) and qr.qr_rms_norm_q8(x, w).codes.shape == (0, 64)
    assert qr.qr_q8_quantize(x).scales.shape == (0,)
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    for bad in (dict(weight=w[:32]), dict(weight=w.bfloat16()), dict(weight=w.cpu()), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(residual=x[:2]), dict(residual=x.bfloat16()), dict(residual_out=x),
                dict(out=x[:, :32]), dict(out=x.float())):
        with pytest.raises((TypeError, ValueError)):
            qr.qr_rms_norm(**{"x": x, "weight": w, **bad})
    for bad in (x.float(), x.t(), x[0], x.cpu()):
        with pytest.raises((TypeError, ValueError)):
            qr.qr_q8_quantize(bad)
    wide = torch.zeros((4, 100), dtype=torch.float16, device="cuda")
    with pytest.raises(qr.QRError):  # an output over part of an input
        qr.qr_rms_norm(wide[:, :64], w, out=wide[:, 8:72])
    with pytest.raises(ValueError):
        qr.Q8Rows(torch.zeros((4, 60), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda"))
    with pytest.raises(TypeError):
        qr.qr_q8_quantize(x, out=x)
    # slices of the same wider rows are apart
    qr.qr_rms_norm(wide[:, :32], w[:32], out=wide[:, 64:96])
