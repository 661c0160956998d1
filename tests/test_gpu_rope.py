"""Rotary positions against the definition in 64 bits (layer_testlib has the
bound)."""
import math

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


def _x(rng, tokens, heads, dim, dtype):
    return torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32) * 3).to(DT[dtype]).cuda()


def _check(got, x, positions, freq, layout, factor, dtype):
    angle = np.asarray(positions, dtype=np.float64)[:, None] * freq
    want, size = ref.rope(x.float().cpu().numpy(), angle, layout, 2 * len(freq), factor)
    wide = np.concatenate([np.abs(angle), np.abs(angle)], 1) if layout == "half" else np.repeat(np.abs(angle), 2, 1)
    drift = np.zeros(want.shape)
    drift[..., :2 * len(freq)] = wide[:, None] * 2.0 ** -51
    bound = (2.0 ** -20 + drift) * size + ref.U_OUT[dtype] * 1.001 * np.abs(want) + ref.TINY[dtype]
    over = np.abs(got.float().cpu().numpy() - want) - bound
    assert (over <= 0).all(), (over.max(), np.unravel_index(over.argmax(), over.shape))
    rot = 2 * len(freq)
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(2, 2), (6, 4), (16, 16), (64, 64), (80, 20), (80, 40), (96, 96), (128, 128), (128, 32),
                                     (126, 90), (256, 128), (256, 256), (576, 64), (1024, 1024)])
def test_layouts(dtype, layout, dim, rot):
    rng = np.random.default_rng(dim + rot)
    freq, factor = qr.rope_frequencies(rot)
    rope = qr.Rope(freq, layout)
    for tokens, hq, hk in ((1, 1, 1), (5, 8, 2), (37, 3, 1)):
        q, k = _x(rng, tokens, hq, dim, dtype), _x(rng, tokens, hk, dim, dtype)
        pos = rng.integers(0, 5000, tokens)
        gq, gk = qr.qr_rope(q, k, rope, torch.from_numpy(pos.astype(np.int32)).cuda())
        _check(gq, q, pos, freq, layout, factor, dtype)
        _check(gk, k, pos, freq, layout, factor, dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    rng = np.random.default_rng(5)
    freq, factor = qr.rope_frequencies(128, 500000.0, scaling="yarn", factor=32.0, original_len=32768)
    assert abs(factor - (0.1 * math.log(32) + 1)) < 1e-12
    pos = np.array([0, 1, -1, 131071, 1 << 20, (1 << 20) + 1, (1 << 30) + 12345, 2 ** 31 - 1, -2 ** 31, 77])
    q = _x(rng, len(pos), 4, 128, 0)
    got, none = qr.qr_rope(q, None, qr.Rope(freq, layout, factor), torch.from_numpy(pos.astype(np.int32)).cuda())
    assert none is None
    _check(got, q, pos, freq, layout, factor, 0)
    # a position's rotation undone by the opposite one
    plain = qr.Rope(freq, layout)
    at = torch.from_numpy(pos[:-2].astype(np.int32)).cuda()
    q32 = q[:-2].clone()
    there, _ = qr.qr_rope(q32, None, plain, at)
    back, _ = qr.qr_rope(there, None, plain, -at)
    size = q32.float().abs().amax(-1, keepdim=True) * 1.5
    assert ((back.float() - q32.float()).abs() <= 4 * 2.0 ** -11 * size).all()


@pytest.mark.parametrize("tokens", [1, 16, 300, 4097])
@pytest.mark.parametrize("dim", [64, 128])
def test_slices_of_a_projection_in_place(tokens, dim):
    rng = np.random.default_rng(tokens)
    hq, hk = 8, 2
    qkv = _x(rng, tokens, hq + 2 * hk, dim, 1)
    kept = qkv.clone()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    pos = rng.integers(0, 100000, tokens)
    at = torch.from_numpy(pos.astype(np.int32)).cuda()
    freq, factor = qr.rope_frequencies(dim, scaling="linear", factor=4.0)
    rope = qr.Rope(freq)
    want = qr.qr_rope(q, k, rope, at)
    assert torch.equal(qkv, kept)
    got = qr.qr_rope(q, k, rope, at, out=(q, k))
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, hq + hk:], kept[:, hq + hk:])
    _check(want[0], kept[:, :hq], pos, freq, "half", factor, 1)
    # [heads, tokens, dim] in memory
    t = kept[:, :hq].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(qr.qr_rope(t, None, rope, at)[0], want[0])
    # rows that begin on no 16-byte boundary
    odd = torch.zeros((tokens, hq, dim + 3), dtype=torch.bfloat16, device="cuda")
    odd[..., 1:1 + dim] = kept[:, :hq]
    assert torch.equal(qr.qr_rope(odd[..., 1:1 + dim], None, rope, at)[0], want[0])
    out = torch.zeros_like(odd)
    qr.qr_rope(kept[:, :hq], None, rope, at, out=(out[..., 1:1 + dim], None))
    assert torch.equal(out[..., 1:1 + dim], want[0]) and (out[..., 0] == 0).all() and (out[..., 1 + dim:] == 0).all()


@pytest.mark.parametrize("requests,most", [(1, 1), (3, 5), (33, 1), (40, 9), (1100, 3), (5000, 1)])
def test_positions_of_a_plan(requests, most):
    rng = np.random.default_rng(requests)
    new = rng.integers(0, most + 1, requests)
    new[rng.integers(0, requests)] = most
    cached = rng.integers(0, 3000, requests)
    tokens = int(new.sum())
    padded = tokens + 7
    offsets = np.concatenate([[0], np.cumsum(new)])
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    plan = qr.KVPlan(None, i32(offsets), i32(cached + new), None, None)
    request = np.repeat(np.arange(requests), new)
    pos = cached[request] + np.arange(tokens) - offsets[request]
    q, k = _x(rng, padded, 4, 64, 1), _x(rng, padded, 1, 64, 1)
    rope = qr.Rope.make(64)
    gq, gk = qr.qr_rope(q, k, rope, plan=plan)
    want = qr.qr_rope(q[:tokens], k[:tokens], rope, i32(pos))
    assert torch.equal(gq[:tokens], want[0]) and torch.equal(gk[:tokens], want[1])
    assert (gq[tokens:] == 0).all()
    kept = q.clone()
    qr.qr_rope(q, k, rope, plan=plan, out=(q, k))
    assert torch.equal(q[:tokens], want[0]) and torch.equal(q[tokens:], kept[tokens:])


def test_refusals():
    q = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    at = torch.zeros(4, dtype=torch.int32, device="cuda")
    rope = qr.Rope.make(64)
    assert qr.qr_rope(q[:0], None, rope, at[:0])[0].shape == (0, 2, 64)
    for args, kw in (((q.float(), None, rope, at), {}), ((q[..., :32], None, rope, at), {}), ((q, q[:2], rope, at), {}),
                     ((q, q.bfloat16(), rope, at), {}), ((q, None, rope, at.long()), {}), ((q, None, rope, at[:3]), {}),
                     ((q, None, rope), {}), ((q, q, rope, at), dict(out=(q, None))), ((q.cpu(), None, rope, at), {}),
                     ((q.transpose(1, 2), None, rope, at), {}), ((q, None, rope, at), dict(out=(q[:, :1], None)))):
        with pytest.raises((TypeError, ValueError)):
            qr.qr_rope(*args, **kw)
    with pytest.raises(qr.QRError):  # an output over part of an input
        big = torch.zeros((4, 3, 64), dtype=torch.float16, device="cuda")
        qr.qr_rope(big[:, :2], None, rope, at, out=(big[:, 1:], None))
    with pytest.raises(qr.QRError):  # queries and keys that would both be written
        qr.qr_rope(q, q.clone(), rope, at, out=(q, q))
    with pytest.raises(qr.QRError):
        odd = torch.zeros((4, 2, 63), dtype=torch.float16, device="cuda")
        qr.qr_rope(odd, None, qr.Rope.make(62), at)
