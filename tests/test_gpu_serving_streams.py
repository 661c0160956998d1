"""The serving calls with stream=: what a call allocates for itself (outputs,
workspaces) belongs to the stream that it runs on.

The current stream, or the side stream that the call gets, is held up by a
sleeping kernel, so that the wrong order would show every time."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
from bit_quantized_all_gb300 import serving
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu
HOLD = 100_000_000  # cycles: some 50 ms


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _handles():
    side = torch.cuda.Stream()
    return side, [side, side.cuda_stream]


def _dirty(nbytes):
    """Leaves a block of the current stream's pool full of ones behind."""
    torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()


class _Spy:
    """The library with one call's arguments kept."""

    def __init__(self, name):
        self.name, self.real, self.args = name, serving._lib(), None

    def __getattr__(self, name):
        fn = getattr(self.__dict__["real"], name)
        if name != self.__dict__["name"]:
            return fn

        def call(*args):
            self.args = args
            return fn(*args)
        return call


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("raw", [0, 1])
def test_attention_s_own_workspace_is_zeroed_before_its_use(nq, raw):
    c = Case([3000, 2500], [nq, nq], 1, 8, seed=31)
    want, want_lse = c.check()
    side, handles = _handles()
    _dirty(qr.qr_kv_attention_workspace_bytes(2, 2 * nq, 8, 1, 128))
    off, kv, table = c.i32(c.offsets), c.i32(c.kv), c.i32(c.table)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)  # the current stream is late
    _, lse = qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, max_q=nq, out=out, return_lse=True, stream=handles[raw])
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_s_own_workspace_is_not_handed_on_while_in_use(nq):
    c = Case([3000, 2500], [nq, nq], 1, 8, seed=32)
    want, _ = c.check()
    side, _ = _handles()
    off, kv, table = c.i32(c.offsets), c.i32(c.kv), c.i32(c.table)
    out = torch.zeros_like(want)
    need = qr.qr_kv_attention_workspace_bytes(2, 2 * nq, 8, 1, 128)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)  # the call's stream is late
    qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, max_q=nq, out=out, stream=side)
    _dirty_now = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del _dirty_now


def test_matvec_s_copy_of_x_is_not_handed_on_while_in_use(monkeypatch):
    rng = np.random.default_rng(1)
    tokens, rows, cols = 4000, 64, 1001
    x = torch.from_numpy(rng.standard_normal((tokens, cols)).astype(np.float32)).bfloat16().cuda()
    weight = qr.qr_w4_quantize(torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).bfloat16().cuda(), 32)
    want = qr.qr_w4_matvec(x, weight)
    side, _ = _handles()
    y = torch.zeros_like(want)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    spy = _Spy("qr_w4_matvec")
    monkeypatch.setattr(serving, "_L", spy)
    qr.qr_w4_matvec(x, weight, y, stream=side)
    ws, nbytes = spy.args[-3], spy.args[-2]
    later = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert ws and not (later.data_ptr() < ws + nbytes and ws < later.data_ptr() + nbytes)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def _late_fill(nbytes):
    """A block of the current stream's pool that work still queued there will overwrite."""
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    t.fill_(255)


@pytest.mark.parametrize("raw", [0, 1])
def test_outputs_are_not_overwritten_by_the_current_stream(raw):
    side, handles = _handles()
    s = handles[raw]
    rng = np.random.default_rng(2)
    rows, cols, tokens = 4096, 1024, 300
    w = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).half().cuda()
    x = torch.from_numpy(rng.standard_normal((tokens, cols)).astype(np.float32)).half().cuda()
    codes = torch.from_numpy(rng.integers(0, 256, (rows, cols // 2)).astype(np.uint8)).cuda()
    scales = torch.rand((rows, cols // 32), device="cuda").half()
    weight = qr.qr_w4_quantize(w, 32)
    want, packed, quantized = qr.qr_w4_matvec(x, weight), qr.qr_w4_pack(codes, scales, cols, 32).packed, weight.packed
    torch.cuda.synchronize()
    for call, wanted in ((lambda: qr.qr_w4_matvec(x, weight, stream=s), want),
                         (lambda: qr.qr_w4_quantize(w, 32, stream=s).packed, quantized),
                         (lambda: qr.qr_w4_pack(codes, scales, cols, 32, stream=s).packed, packed)):
        torch.cuda.empty_cache()
        _late_fill(wanted.numel() * wanted.element_size())
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(got, wanted)

    c = Case([700] * 300, [1] * 300, 1, 8, seed=33)
    want, want_lse = c.check()
    off, kv, table = c.i32(c.offsets), c.i32(c.kv), c.i32(c.table)
    ws = qr.qr_kv_attention_workspace(c.q_dev, c.cache, 300)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    _late_fill(want.numel() * 2)
    out, lse = qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, max_q=1, return_lse=True, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)

    n = 1 << 18
    one, table = torch.ones(1, dtype=torch.int32, device="cuda"), torch.full((1, n // 16), -1, dtype=torch.int32, device="cuda")
    free, none, many = torch.arange(n // 16, dtype=torch.int32, device="cuda"), one * 0, one * n
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    _late_fill(n * 8)
    plan = qr.qr_kv_plan(none, many, table, free, 16, n, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(plan.slots, torch.arange(n, device="cuda"))


def test_append_and_the_default_stream_by_handle():
    c = Case([64], [4], 2, 4, seed=34)
    k = torch.randn((64, 2, 128), device="cuda").half()
    slots = torch.arange(64, device="cuda")
    first, second = qr.KVCache.empty(4, 2, 16, 128), qr.KVCache.empty(4, 2, 16, 128)
    torch.cuda.synchronize()
    qr.qr_kv_append(first, k, k, slots)
    qr.qr_kv_append(second, k, k, slots, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(first.k_codes, second.k_codes) and torch.equal(first.v_scales, second.v_scales)
    want, _ = c.check()
    out = qr.qr_kv_attention(c.q_dev, c.cache, c.i32(c.offsets), c.i32(c.kv), c.i32(c.table), max_q=4, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
