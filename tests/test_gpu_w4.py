"""4-bit weights: packing, quantizing and the product against the definition
in 64 bits (serving_testlib has the bound)."""
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


def _weights(rng, rows, cols, group, zeros):
    codes = rng.integers(0, 256, (rows, -(-cols // 2))).astype(np.uint8)
    groups = -(-cols // group)
    scales = (rng.random((rows, groups)) * 0.02 + 0.001).astype(np.float16)
    z = rng.integers(0, 16, (rows, groups)).astype(np.uint8) if zeros else None
    return codes, scales, z


def _pack(codes, scales, z, cols, group):
    return qr.qr_w4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), cols, group,
                         None if z is None else torch.from_numpy(z).cuda())


def _check(x, weight, dense, dtype, y=None):
    got = qr.qr_w4_matvec(x.cuda() if not x.is_cuda else x, weight, y)
    want, bound = ref.matvec(x.float().cpu().numpy(), dense, dtype)
    over = np.abs(got.float().cpu().numpy() - want) - bound
    assert (over <= 0).all(), (over.max(), np.unravel_index(over.argmax(), over.shape))
    return got


def _x(rng, tokens, cols, dtype):
    x = rng.standard_normal((tokens, cols)).astype(np.float32)
    x[:, rng.integers(0, cols)] *= 20
    return torch.from_numpy(x).to(DT[dtype])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tokens", [1, 3, 8, 9, 16, 17, 33, 64, 65, 130])
def test_tokens(dtype, group, zeros, tokens):
    rng = np.random.default_rng(tokens + group)
    rows, cols = 80, 512
    w = _weights(rng, rows, cols, group, zeros)
    _check(_x(rng, tokens, cols, dtype), _pack(*w, cols, group), ref.w4_dense(*w, cols, group), dtype)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (16, 64), (17, 65), (33, 31), (5, 127), (15, 129), (100, 2047),
                                       (257, 1000), (64, 4160), (2000, 72), (31, 8200)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", [1, 2, 21])
def test_odd_sizes(rows, cols, group, tokens):
    rng = np.random.default_rng(rows + cols)
    w = _weights(rng, rows, cols, group, group == 64)
    _check(_x(rng, tokens, cols, tokens % 2), _pack(*w, cols, group), ref.w4_dense(*w, cols, group), tokens % 2)


@pytest.mark.parametrize("dtype,group,zeros", [(0, 128, True), (1, 32, False), (0, 64, True)])
def test_rows_of_a_second_launch(dtype, group, zeros):
    # 153 tiles of 128 rows: on 152 SMs one wave and a launch of its own for
    # the last, of odd height
    rng = np.random.default_rng(group)
    rows, cols, tokens = 19511, 1000, 40
    w = _weights(rng, rows, cols, group, zeros)
    y = torch.full((tokens, rows + 3), 7.0, dtype=DT[dtype], device="cuda")
    _check(_x(rng, tokens, cols, dtype), _pack(*w, cols, group), ref.w4_dense(*w, cols, group), dtype, y[:, :rows])
    assert (y[:, rows:] == 7).all()


@pytest.mark.parametrize("tokens", [1, 12, 40])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (8, 1), (0, 4)])
def test_strides_and_alignment(tokens, pad, shift):
    rng = np.random.default_rng(pad + shift)
    rows, cols = 72, 384
    w = _weights(rng, rows, cols, 32, False)
    buf = torch.full((tokens * (cols + pad) + shift + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = buf[shift:shift + tokens * (cols + pad)].view(tokens, cols + pad)[:, :cols]
    x.copy_(_x(rng, tokens, cols, 1))
    out = torch.full((tokens, rows + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    _check(x, _pack(*w, cols, 32), ref.w4_dense(*w, cols, 32), 1, out[:, 1:rows + 1])
    assert (out[:, 0] == 9).all() and (out[:, rows + 1:] == 9).all()


def test_workspace_for_unaligned_rows():
    rng = np.random.default_rng(7)
    rows, cols, tokens = 150, 333, 40
    w = _weights(rng, rows, cols, 64, True)
    weight, dense = _pack(*w, cols, 64), ref.w4_dense(*w, cols, 64)
    x = _x(rng, tokens, cols, 0).cuda()
    ws = torch.full((qr.qr_w4_matvec_workspace_bytes(tokens, cols),), 255, dtype=torch.uint8, device="cuda")
    got = qr.qr_w4_matvec(x, weight, workspace=ws)
    assert torch.equal(got, _check(x, weight, dense, 0))
    with pytest.raises(qr.QRError) as e:
        qr.qr_w4_matvec(x, weight, workspace=ws[:-16])
    assert e.value.status == qr.QR_ERR_SIZE


def test_every_code_scale_and_zero_is_read_in_its_place():
    """One-hot x: the product returns the weights themselves."""
    rng = np.random.default_rng(1)
    rows, cols, group = 35, 200, 32
    w = _weights(rng, rows, cols, group, True)
    y = qr.qr_w4_matvec(torch.eye(cols, dtype=torch.float16, device="cuda"), _pack(*w, cols, group))
    want = ref.w4_dense(*w, cols, group).astype(np.float16)
    assert np.array_equal(y.t().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(dtype, group):
    """The INT4 codec's codes and scales on each group: read back through one-hot products."""
    rng = np.random.default_rng(group)
    rows, cols = 37, 330
    w = torch.from_numpy(rng.standard_normal((rows, cols + 6)).astype(np.float32)).to(DT[dtype])
    w[3, :40], w[5, 10] = 0, 3000.0
    weight = qr.qr_w4_quantize(w.cuda()[:, :cols], group)
    y = qr.qr_w4_matvec(torch.eye(cols, dtype=torch.float16, device="cuda"), weight).t().cpu().numpy()
    x = w[:, :cols].float().numpy()
    want = np.zeros((rows, cols))
    for g in range(0, cols, group):
        part = x[:, g:g + group]
        s = (np.abs(part).max(1) * np.float32(0.125)).astype(np.float16).astype(np.float32)
        r = np.where(s > 0, np.float32(1) / np.where(s > 0, s, 1), 0).astype(np.float32)
        u = np.rint(np.clip(part * r[:, None], -8, 7))
        want[:, g:g + group] = u * s[:, None].astype(np.float64)
    assert np.array_equal(y, want.astype(np.float16))


def test_quantize_matches_the_int4_wire():
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.standard_normal((8, 2048)).astype(np.float32)).half().cuda()
    y = qr.qr_w4_matvec(torch.eye(2048, dtype=torch.float16, device="cuda"), qr.qr_w4_quantize(w, 32)).t()
    wire = qr.qr_decode(4, qr.qr_encode(4, w), w.numel(), dtype=torch.float16).view(8, 2048)
    assert torch.equal(y, wire)


def test_non_finite_x_stays_in_its_token():
    rng = np.random.default_rng(3)
    w = _weights(rng, 40, 128, 32, False)
    weight = _pack(*w, 128, 32)
    x = _x(rng, 5, 128, 1)
    clean = qr.qr_w4_matvec(x.cuda(), weight)
    x[2, 7] = float("nan")
    got = qr.qr_w4_matvec(x.cuda(), weight)
    keep = [0, 1, 3, 4]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[2]).all()


def test_same_bits_twice_and_on_another_stream():
    rng = np.random.default_rng(4)
    w = _weights(rng, 300, 4096, 128, True)
    weight, x = _pack(*w, 4096, 128), _x(rng, 4, 4096, 0).cuda()
    a = qr.qr_w4_matvec(x, weight)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        b = qr.qr_w4_matvec(x, weight)
    side.synchronize()
    assert torch.equal(a, b)


def test_no_tokens_and_refusals():
    rng = np.random.default_rng(5)
    w = _weights(rng, 40, 128, 32, False)
    weight = _pack(*w, 128, 32)
    assert qr.qr_w4_matvec(torch.zeros((0, 128), dtype=torch.float16, device="cuda"), weight).shape == (0, 40)
    x = torch.zeros((2, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        qr.qr_w4_matvec(x.float(), weight)
    with pytest.raises(ValueError):
        qr.qr_w4_matvec(x[:, :64], weight)
    with pytest.raises(ValueError):
        qr.qr_w4_matvec(x.t(), weight)
    with pytest.raises(ValueError):
        _pack(*w, 128, 48)
    with pytest.raises(ValueError):
        _pack(w[0], w[1][:, :2], None, 128, 32)
    with pytest.raises(ValueError):
        qr.W4Weight(weight.packed[:100], 40, 128, 32, False)
    with pytest.raises(qr.QRError) as e:
        qr.qr_w4_matvec(x, weight, weight.packed.view(torch.float16)[:80].view(2, 40))
    assert e.value.status == qr.QR_ERR_INVALID_ARG
