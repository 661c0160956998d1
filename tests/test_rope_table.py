"""A Rope's address is that of the table it holds now."""
import copy
import pickle

import pytest

import bit_quantized_all_gb300 as qr


@pytest.mark.parametrize("another", [copy.deepcopy, copy.copy, lambda r: pickle.loads(pickle.dumps(r))])
def test_a_copy_has_its_own_address(another):
    rope = qr.Rope([1.0, 0.5, 0.25], "interleaved", 2.0, device="cpu")
    got = another(rope)
    assert got.turns.tolist() == rope.turns.tolist() and got.address == got.turns.data_ptr()
    assert (got.rot_dim, got.interleaved, got.factor, got.device) == (6, True, 2.0, rope.device)


def test_a_table_that_is_replaced():
    rope = qr.Rope([1.0, 0.5], device="cpu")
    rope.turns = rope.turns.clone()
    assert rope.address == rope.turns.data_ptr()
