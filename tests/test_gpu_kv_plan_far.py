"""qr_kv_plan where the new tokens of one chunk of 2048 requests pass 2^31 - 1,
and more requests follow: those are counted, and get neither block nor slot."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


@pytest.mark.parametrize("far", [2 ** 30, MOST])
def test_requests_past_the_last_token_are_counted_alone(far):
    requests, width, num_free, max_tokens = 4200, 3, 70, 1000
    new = np.full(requests, 5, np.int64)
    new[10] = new[11] = new[2000] = far
    table = torch.full((requests, width), -7, dtype=torch.int32, device="cuda")
    free = torch.arange(100, 100 + num_free, dtype=torch.int32, device="cuda")
    guard = 1 << 16
    buf = torch.full((max_tokens + 2 * guard,), 77, dtype=torch.int64, device="cuda")
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    empty = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = qr.KVPlan(table, empty(requests + 1), empty(requests), buf[guard:guard + max_tokens], empty(4))
    got = qr.qr_kv_plan(i32(np.zeros(requests)), i32(new), table, free, 16, max_tokens, plan=plan)

    need = -(-new // 16)
    start = np.concatenate([[0], np.cumsum(new)])
    first = np.concatenate([[0], np.cumsum(need)])
    assert (buf[:guard] == 77).all() and (buf[guard + max_tokens:] == 77).all()
    assert np.array_equal(got.q_offsets.cpu().numpy(), np.minimum(start, max_tokens))
    assert np.array_equal(got.kv_lens.cpu().numpy(), new)
    assert got.counts.tolist() == [num_free, MOST, int(min(need.sum() - num_free, MOST)), int(min(np.maximum(need - width, 0).sum(), MOST))]
    want = np.full((requests, width), -7)
    for r in range(requests):
        for b in range(min(width, int(need[r]))):
            if start[r] + 16 * b < MOST:  # the block's first token has a number
                want[r, b] = 100 + first[r] + b if first[r] + b < num_free else -1
    assert np.array_equal(table.cpu().numpy(), want)
    slots = np.full(max_tokens, -1)
    for r in range(11):
        for p in range(int(min(new[r], max_tokens - start[r]))):
            if p // 16 < width and want[r, p // 16] >= 0:
                slots[start[r] + p] = want[r, p // 16] * 16 + p % 16
    assert np.array_equal(got.slots.cpu().numpy(), slots)
