"""The compiled form of the calls gives what the interpreted one gives, and
declines what that one has to handle or refuse."""
import pytest
import torch

import bit_quantized_all_gb300 as qr
from bit_quantized_all_gb300 import layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


class _Declines:
    def __getattr__(self, name):
        return lambda *args: None


def _tensors(x):
    return [t for y in (x if isinstance(x, tuple) else (x,)) if y is not None
            for t in ((y.codes, y.scales) if isinstance(y, qr.Q8Rows) else (y,))]


def _calls(tokens, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(tokens + cols)
    x, res = (torch.randn((tokens, cols), generator=gen, device="cuda").to(dtype) for _ in range(2))
    wide = torch.randn((tokens, cols + 5), generator=gen, device="cuda").to(dtype)[:, 3:3 + cols]
    w = torch.rand(cols, generator=gen, device="cuda")
    weight = qr.qr_w8_quantize(torch.randn((70, cols), generator=gen, device="cuda").to(dtype))
    rows = qr.qr_q8_quantize(x)
    qkv = torch.randn((tokens, 10, 96), generator=gen, device="cuda").to(dtype)
    q, k = qkv[:, :8], qkv[:, 8:9]
    rope, at = qr.Rope.make(64, layout="interleaved"), torch.arange(tokens, dtype=torch.int32, device="cuda")
    plan = qr.KVPlan(None, torch.tensor([0, max(1, tokens - 2)], dtype=torch.int32, device="cuda"),
                     torch.tensor([tokens + 9], dtype=torch.int32, device="cuda"), None, None)
    space = qr.qr_w8_matmul_workspace(tokens, weight)

    def in_place():
        r = res.clone()
        return qr.qr_rms_norm_q8(x, w.to(dtype), 1e-5, r), r

    def turned():
        y = qkv.clone()
        got = qr.qr_rope(y[:, :8], y[:, 8:9], rope, plan=plan, out=None)
        a, b = y[:, :8], y[:, 8:9]
        assert qr.qr_rope(a, b, rope, at, out=(a, b))[0] is a
        return (*got, y)

    return [lambda: qr.qr_q8_quantize(x), lambda: qr.qr_q8_quantize(wide), lambda: qr.qr_rms_norm(x, w),
            lambda: qr.qr_rms_norm(wide, w.to(dtype), 1e-5, res, torch.empty_like(res)), in_place,
            lambda: qr.qr_w8_matmul(rows, weight, dtype), lambda: qr.qr_w8_matmul(rows, weight, dtype, workspace=space),
            lambda: qr.qr_rope(q, k, rope, at), lambda: qr.qr_rope(q, None, rope, at), turned]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,cols", [(1, 64), (5, 77), (40, 256)])
def test_the_same_as_the_interpreted_calls(monkeypatch, dtype, tokens, cols):
    calls = _calls(tokens, cols, dtype)
    compiled = [_tensors(c()) for c in calls]
    monkeypatch.setattr(layer, "_F", _Declines())
    for a, c in zip(compiled, calls):
        b = _tensors(c())
        assert len(a) == len(b)
        for s, t in zip(a, b):
            assert s.dtype == t.dtype and s.shape == t.shape and s.stride() == t.stride() and torch.equal(s, t)


def test_declines():
    F = layer._fast()
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    w, at = x[0].clone(), torch.zeros(4, dtype=torch.int32, device="cuda")
    for args in ((x.float(),), (x.cpu(),), (x.t(),), (x[0],), (x[:0],), (None,), (x, x), ([1.0],)):
        assert F.quantize(*args) is None
    for args in ((x, w.float()[:32], 1e-5, None, None, True), (x, w, 0.0, None, None, True), (x, w, 1, None, None, True),
                 (x, w, float("inf"), None, None, False), (x, w, 1e-5, x[:2], None, True), (x, w, 1e-5, None, x, True),
                 (x, w.bfloat16(), 1e-5, None, None, False), (x, w.cpu(), 1e-5, None, None, False), (x, w)):
        assert F.norm(*args) is None
    q, rope = x.view(4, 1, 64), qr.Rope.make(64)
    for args in ((q, q[:2], rope.turns, 64, False, 1.0, at, None, None, False), (q, None, rope.turns, 64, False, 1.0, at[:3], None, None, False),
                 (q, None, rope.turns, 64, False, 1.0, None, at, at, False), (q.float(), None, rope.turns, 64, False, 1.0, at, None, None, False),
                 (q, None, rope.turns, 128, False, 1.0, at, None, None, False), (q.transpose(1, 2), None, rope.turns, 2, False, 1.0, at, None, None, False)):
        assert F.rope(*args) is None
    weight, rows = qr.qr_w8_quantize(x), qr.qr_q8_quantize(x)
    for args in ((rows.codes[:, :32], rows.scales, weight.packed, 4, 64, True, None), (rows.codes, rows.scales[:3], weight.packed, 4, 64, True, None),
                 (rows.codes, rows.scales, weight.packed, 4, 64, True, rows.scales), (x, rows.scales, weight.packed, 4, 64, True, None)):
        assert F.matmul(*args) is None
    # what the C ABI refuses comes back as its status
    with pytest.raises(qr.QRError):
        qr.qr_w8_matmul(qr.Q8Rows.empty(40, 64), weight, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        F.bind(1, 2)


def test_a_plan_that_leaves_tokens_out_captured():
    """Tokens past the plan's last one are zeros in new outputs, in a replay too."""
    q = torch.randn((6, 2, 64), device="cuda").half()
    rope = qr.Rope.make(64)
    plan = qr.KVPlan(None, torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda"),
                     torch.tensor([3, 9], dtype=torch.int32, device="cuda"), None, None)
    want = qr.qr_rope(q[:4], q[:4, :1], rope, torch.tensor([0, 1, 2, 8], dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [qr.qr_rope(q, q[:, :1], rope, plan=plan)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got.append(qr.qr_rope(q, q[:, :1], rope, plan=plan))
    for t in got[1]:
        t.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a in got:
        for t, w in zip(a, want):
            assert torch.equal(t[:4], w) and not t[4:].any()
