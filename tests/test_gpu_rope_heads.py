"""qr_rope with queries or keys that have no heads."""
import pytest
import torch

import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [64, 32])
@pytest.mark.parametrize("with_plan", [False, True])
def test_keys_alone(layout, rot, with_plan):
    k = torch.randn((5, 3, 64), device="cuda").bfloat16()
    none = k[:, :0]
    rope = qr.Rope.make(rot, layout=layout)
    i32 = dict(dtype=torch.int32, device="cuda")
    at = (dict(plan=qr.KVPlan(None, torch.tensor([0, 4], **i32), torch.tensor([11], **i32), None, None)) if with_plan
          else dict(positions=torch.tensor([7, 8, 9, 10, 0], **i32)))
    want, _ = qr.qr_rope(k, None, rope, **at)
    got = qr.qr_rope(none, k, rope, **at)
    assert got[0].shape == (5, 0, 64) and torch.equal(got[1], want)
    out = torch.zeros_like(k)
    assert qr.qr_rope(none, k, rope, out=(none, out), **at)[1] is out and torch.equal(out, want)
    assert torch.equal(qr.qr_rope(k, none, rope, **at)[0], want)
    kept = k.clone()
    qr.qr_rope(none, k, rope, out=(none, k), **at)
    assert torch.equal(k[:4], want[:4]) and torch.equal(k[4:], kept[4:] if with_plan else want[4:])
    assert [t.shape for t in qr.qr_rope(none, none, rope, **at)] == 2 * [(5, 0, 64)]
