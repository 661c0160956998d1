"""The calls before the attention with stream=: they run, and what they allocate
for themselves belongs, there.  The side stream is held up by a sleeping kernel
and only then gets its input, so that the wrong order would show every time."""
import pytest
import torch

import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu
HOLD = 100_000_000  # cycles: some 50 ms


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _calls(tokens):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    norm = torch.rand(640, generator=gen, device="cuda")
    weight = qr.qr_w8_quantize(torch.randn((300, 640), generator=gen, device="cuda").half())
    rope, at = qr.Rope.make(64), torch.arange(tokens, dtype=torch.int32, device="cuda")
    plan = qr.KVPlan(None, torch.tensor([0, tokens - 1], dtype=torch.int32, device="cuda"),
                     torch.tensor([tokens + 5], dtype=torch.int32, device="cuda"), None, None)
    return {
        "quantize": lambda x, **kw: qr.qr_q8_quantize(x, **kw).codes,
        "norm": lambda x, **kw: qr.qr_rms_norm(x, norm, **kw),
        "norm8": lambda x, **kw: qr.qr_rms_norm_q8(x, norm, **kw).codes,
        "rope": lambda x, **kw: qr.qr_rope(x.view(-1, 10, 64), None, rope, at, **kw)[0],
        "rope plan": lambda x, **kw: qr.qr_rope(x.view(-1, 10, 64), None, rope, plan=plan, **kw)[0],
        "product": lambda x, **kw: qr.qr_w8_matmul(qr.qr_q8_quantize(x, **kw), weight, **kw),
        "weights": lambda x, **kw: qr.qr_w8_quantize(x, **kw).packed,
    }


@pytest.mark.parametrize("name", ["quantize", "norm", "norm8", "rope", "rope plan", "product", "weights"])
@pytest.mark.parametrize("tokens", [5, 40, 300])
@pytest.mark.parametrize("raw", [False, True])
def test_runs_on_its_stream(name, tokens, raw):
    call = _calls(tokens)[name]
    first, second = (torch.randn((tokens, 640), device="cuda").half() for _ in range(2))
    want = call(second)
    x = first.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
        x.copy_(second)
    got = call(x, stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert torch.equal(got, want)
    # what the call made on the held stream is not handed out here meanwhile
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    got = call(second, stream=side)
    for _ in range(4):
        torch.full((got.numel() * got.element_size() + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_two_captured_graphs_with_workspaces_of_their_own():
    weight = qr.qr_w8_quantize(torch.randn((3000, 1000), device="cuda").half())
    xs = [qr.qr_q8_quantize(torch.randn((90, 1000), device="cuda").half()) for _ in range(2)]
    want = [qr.qr_w8_matmul(x, weight) for x in xs]
    graphs, got = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(qr.qr_w8_matmul(x, weight))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
