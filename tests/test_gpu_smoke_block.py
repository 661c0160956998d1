"""The smoke test's block compares what it computes: against plain forms that are wrong it fails."""
import numpy as np
import pytest
import torch

import __graft_entry__ as entry
import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


def _run():
    entry._smoke_block(torch, qr, torch.device("cuda", 0))


def test_passes():
    _run()


def test_sees_positions(monkeypatch):
    plain = entry._rotated
    monkeypatch.setattr(entry, "_rotated", lambda x, angle: plain(x, angle * 1.01))
    with pytest.raises(AssertionError, match="positions"):
        _run()


@pytest.mark.parametrize("which", [0, 1])
def test_sees_rows(monkeypatch, which):
    plain = entry._rows8

    def other(v):
        codes, step = plain(v)
        return (np.where(codes == 1, 0, codes), step) if which == 0 else (codes, step * np.float32(1.001))

    monkeypatch.setattr(entry, "_rows8", other)
    with pytest.raises(AssertionError, match="norm"):
        _run()
