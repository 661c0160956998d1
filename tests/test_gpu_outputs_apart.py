"""The outputs of a call can be saved together, and one can be kept without the other: they own their memory each,
but for the queries and keys that a plan's positions are turned into, which share an allocation."""
import io

import pytest
import torch

import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _outputs(tokens, cols):
    x = torch.randn((tokens, cols), device="cuda").half()
    w = torch.rand(cols, device="cuda")
    for y in (qr.qr_q8_quantize(x), qr.qr_rms_norm_q8(x, w), qr.qr_rms_norm_q8(x, w, 1e-5, x.clone())):
        yield (y.codes, y.scales), y
    q, k = torch.randn((tokens, 4, 64), device="cuda").half(), torch.randn((tokens, 1, 64), device="cuda").half()
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = qr.KVPlan(None, torch.tensor([0, tokens], **i32), torch.tensor([tokens], **i32), None, None)
    rope = qr.Rope.make(64)
    for y in (qr.qr_rope(q, k, rope, torch.arange(tokens, **i32)), qr.qr_rope(q, k, rope, plan=plan)):
        yield y, y


@pytest.mark.parametrize("tokens,cols", [(1, 1), (5, 77), (40, 256)])
def test_saved_and_loaded(tokens, cols):
    for tensors, whole in _outputs(tokens, cols):
        for what in (whole, {"first": tensors[0], "second": tensors[1]}):
            file = io.BytesIO()
            torch.save(what, file)
            file.seek(0)
            got = torch.load(file, weights_only=False)
            got = (got.codes, got.scales) if isinstance(got, qr.Q8Rows) else tuple(got.values()) if isinstance(got, dict) else got
            assert all(torch.equal(a, b) and a.stride() == b.stride() for a, b in zip(got, tensors))


@pytest.mark.parametrize("tokens,cols", [(1, 1), (5, 77), (40, 256)])
def test_memory_of_their_own(tokens, cols):
    for (a, b), _ in list(_outputs(tokens, cols))[:-1]:
        assert a.untyped_storage().data_ptr() != b.untyped_storage().data_ptr()
        assert b.untyped_storage().nbytes() == b.numel() * b.element_size() and b.storage_offset() == 0


def test_one_kept_without_the_other():
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    scales = qr.qr_q8_quantize(torch.zeros((4096, 8192), dtype=torch.float16, device="cuda")).scales
    assert torch.cuda.memory_allocated() - before <= 1 << 20 and scales.shape == (4096,)
