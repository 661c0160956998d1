"""qr_kv_plan against a request-by-request numpy form: every output is whole
numbers and has to be equal."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import serving_testlib as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _check(cached, new, bs, width=None, free=None, max_tokens=None, seed=0):
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached), np.asarray(new)
    c, n = np.maximum(cached, 0), np.maximum(new, 0)
    need = -(-(c + n) // bs)
    width = max(1, int(need.max())) if width is None else width
    had = int((-(-c // bs)).sum())
    ids = rng.permutation(had + int(need.sum()) + 3)
    table = np.full((len(c), width), -7)
    at = 0
    for r, k in enumerate(-(-c // bs)):
        table[r, :min(k, width)] = ids[at:at + min(k, width)]
        at += k
    free = ids[had:] if free is None else ids[had:had + free]
    max_tokens = int(n.sum()) if max_tokens is None else max_tokens
    want = ref.plan(cached, new, table, free, bs, max_tokens)
    dev = _i32(table)
    got = qr.qr_kv_plan(_i32(cached), _i32(new), dev, _i32(free), bs, max_tokens)
    for g, w, name in zip(got, want, qr.KVPlan._fields):
        assert np.array_equal(g.cpu().numpy(), w), name
    return got


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_decode_and_mixed(bs):
    rng = np.random.default_rng(bs)
    _check(rng.integers(0, 700, 16), np.ones(16, np.int64), bs)
    _check(rng.integers(0, 700, 37), rng.integers(0, 90, 37), bs)


@pytest.mark.parametrize("cached,new", [([0], [1]), ([0], [0]), ([15], [1]), ([16], [1]), ([17], [16]),
                                        ([0, 0, 0], [0, 5, 0]), ([31, 32, 33], [1, 1, 1]), ([-4, 3], [2, -1]),
                                        ([0], [5000])])
def test_edges(cached, new):
    _check(cached, new, 16)


@pytest.mark.parametrize("requests", [255, 256, 257, 1025, 5000])
def test_many_requests(requests):
    rng = np.random.default_rng(requests)
    new = rng.integers(0, 9, requests)
    new[rng.integers(0, requests, 3)] = 1500
    _check(rng.integers(0, 100, requests), new, 16)


def test_slots_past_the_last_token_are_minus_one():
    got = _check([3, 20], [2, 1], 16, max_tokens=2500)
    assert (got.slots.cpu().numpy()[3:] == -1).all()


def test_more_tokens_than_slots():
    got = _check([0, 0, 0], [30, 30, 30], 16, max_tokens=40)
    assert got.q_offsets.tolist() == [0, 30, 40, 40] and got.counts.tolist() == [6, 90, 0, 0]


@pytest.mark.parametrize("free,width", [(0, None), (3, None), (None, 2), (4, 2)])
def test_exhausted(free, width):
    got = _check([0, 5, 40, 16], [20, 40, 40, 1], 16, free=free, width=width)
    assert got.counts[2].item() > 0 or got.counts[3].item() > 0


def test_reused_buffers_and_another_stream():
    first = _check([0, 9], [4, 8], 16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = qr.qr_kv_plan(_i32([4, 17]), _i32([1, 7]), first.block_table, _i32([90, 91]), 16, 12, plan=first)
    side.synchronize()
    assert again.slots.data_ptr() == first.slots.data_ptr()
    assert again.kv_lens.tolist() == [5, 24] and again.counts.tolist()[:2] == [0, 8]


def test_refusals():
    one = _i32([1])
    table = _i32([[0]])
    with pytest.raises(TypeError):
        qr.qr_kv_plan(one.long(), one, table, one, 16, 1)
    with pytest.raises(ValueError):
        qr.qr_kv_plan(one, _i32([1, 2]), table, one, 16, 1)
    with pytest.raises(ValueError):
        qr.qr_kv_plan(one, one, _i32([0]), one, 16, 1)
    with pytest.raises(ValueError):
        qr.qr_kv_plan(one.cpu(), one, table, one, 16, 1)
    with pytest.raises(qr.QRError):
        qr.qr_kv_plan(one, one, table, one, 24, 1)
