"""qr_kv_attention against the definition in 64 bits (serving_testlib has
the bounds and their derivation)."""
import numpy as np
import pytest
import torch

import bit_quantized_all_gb300 as qr
import serving_testlib as ref

pytestmark = pytest.mark.gpu
DT = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


class Case:
    """Requests with given lengths over a cache whose unused blocks and table
    entries hold garbage."""

    def __init__(self, kv, nq, heads=1, group=8, dim=128, bs=16, dtype=1, seed=0, q_gain=1.0, strided=False):
        rng = np.random.default_rng(seed)
        self.dtype, self.bs = dtype, bs
        kv = np.asarray(kv)
        need = -(-np.maximum(kv, 0) // bs)
        width = max(1, int(need.max())) + 2
        blocks = int(need.sum()) + 3
        ids = rng.permutation(blocks)
        table = np.full((len(kv), width), -1)
        table[:, -1] = 1 << 30
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = ids[at:at + n]
            at += n
        self.kc, self.vc = (rng.integers(-128, 128, (blocks, heads, bs, dim)).astype(np.int8) for _ in range(2))
        self.ks, self.vs = ((rng.random((blocks, heads)) * 0.02 + 0.005).astype(np.float32) for _ in range(2))
        for s in (self.ks, self.vs):
            s[ids[at:]] = np.nan
        self.table, self.kv = table, kv
        self.offsets = np.concatenate([[0], np.cumsum(nq)])
        T = max(1, int(self.offsets[-1]))
        q = rng.standard_normal((T, heads * group, dim)).astype(np.float32) * q_gain
        q[..., rng.integers(0, dim)] *= 8
        self.q = torch.from_numpy(q).to(DT[dtype])
        self.max_q = max(1, int(np.max(nq)))
        if strided:
            both = torch.full((blocks, heads + 1, 2, bs, dim), 99, dtype=torch.int8, device="cuda")
            both[:, :heads, 0], both[:, :heads, 1] = torch.from_numpy(self.kc).cuda(), torch.from_numpy(self.vc).cuda()
            kc, vc = both[:, :heads, 0], both[:, :heads, 1]
            wide = torch.full((T, heads * group + 2, dim + 8), float("nan"), dtype=DT[dtype], device="cuda")
            wide[:, 1:-1, :dim] = self.q.cuda()
            self.q_dev = wide[:, 1:-1, :dim]
            self.out_buf = torch.full((T, heads * group + 1, dim + 8), 7.0, dtype=DT[dtype], device="cuda")
            self.out_dev = self.out_buf[:, :-1, :dim]
        else:
            kc, vc = torch.from_numpy(self.kc).cuda(), torch.from_numpy(self.vc).cuda()
            self.q_dev, self.out_dev = self.q.cuda(), None
        self.cache = qr.KVCache(kc, vc, torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda())

    def i32(self, a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def run(self, scale=None, causal=True, window=0, **kw):
        return qr.qr_kv_attention(self.q_dev, self.cache, self.i32(self.offsets), self.i32(self.kv),
                                  self.i32(self.table), scale=scale, causal=causal, window=window,
                                  max_q=kw.pop("max_q", self.max_q), return_lse=True, out=self.out_dev, **kw)

    def check(self, scale=None, causal=True, window=0, **kw):
        out, lse = self.run(scale, causal, window, **kw)
        s = self.q.shape[2] ** -0.5 if scale is None else scale
        want, want_lse, b_out, b_lse = ref.attention(self.q.float().numpy(), self.offsets, self.kv, self.table, self.kc,
                                                     self.ks, self.vc, self.vs, s, causal, window, self.dtype)
        T = int(self.offsets[-1])
        got, got_lse = out.float().cpu().numpy()[:T].astype(np.float64), lse.cpu().numpy()[:T].astype(np.float64)
        want, want_lse, b_out, b_lse = want[:T], want_lse[:T], b_out[:T], b_lse[:T]
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        assert (got[empty] == 0).all()
        over = np.abs(got - want) - b_out
        assert (over <= 0).all(), (over.max(), np.unravel_index(over.argmax(), over.shape))
        over = np.abs(got_lse[~empty] - want_lse[~empty]) - b_lse[~empty]
        assert (over <= 0).all(), over.max()
        return out, lse


EDGE = [0, 1, 15, 16, 17, 31, 33, 64, 127, 300, 0, 129]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("heads,group", [(1, 8), (2, 1), (3, 5), (1, 16), (8, 4)])
def test_single_tokens(dtype, heads, group):
    Case(EDGE, [1] * len(EDGE), heads, group, dtype=dtype, seed=heads + group).check()


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("bs", [16, 64])
def test_head_sizes(dim, bs):
    Case([1, 40, 97, 210], [1, 1, 3, 1], 2, 4, dim=dim, bs=bs, dtype=dim // 16 % 2, seed=dim).check()


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_block_sizes(bs):
    Case([1, bs - 1, bs, bs + 1, 3 * bs + 5], [1] * 5, 2, 4, bs=bs, seed=bs).check()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("heads,group", [(1, 8), (2, 5), (2, 1), (1, 40)])
def test_prompt_chunks(dtype, heads, group):
    Case([40, 130, 33, 257, 7], [40, 60, 1, 129, 0], heads, group, bs=32, dtype=dtype, seed=group).check()


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_prompt_head_sizes(dim):
    Case([70, 300, 200], [70, 150, 33], 1, 4, dim=dim, bs=16, seed=dim).check()


def test_drafts():
    Case([5, 64, 300, 1000], [4, 4, 3, 2], 2, 8, bs=16, seed=1).check()


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 100000])
def test_window(window):
    Case([1, 40, 200, 333], [1, 8, 70, 2], 2, 4, bs=32, seed=window % 97).check(window=window)


def test_not_causal():
    Case([1, 40, 200, 333], [3, 8, 70, 1], 2, 4, bs=32, seed=4).check(causal=False)


def test_rows_that_see_nothing():
    """More queries than keys (the first rows stand before position 0), and
    requests with nothing cached."""
    Case([0, 3, 17, 0, 100], [4, 9, 40, 1, 200], 1, 4, seed=5).check()
    Case([0, 0], [1, 1], 2, 8, seed=6).check()
    Case([0, 2, 20], [4, 9, 40], 1, 4, seed=5).check(causal=False)


def test_bad_block_ids_are_masked():
    c = Case([100, 64], [5, 1], 1, 8, seed=7)
    c.table[0, 1], c.table[0, 3], c.table[1, :4] = -1, c.kc.shape[0], -5
    c.check()


def test_lengths_beyond_the_table_are_cut():
    c = Case([50, 20], [2, 1], 1, 8, seed=8)
    c.table = c.table[:, :2].copy()
    c.kv = np.array([32, 20])
    c.check()
    c.kv = np.array([1 << 30, 20])
    out, lse = c.run(causal=False)
    c.kv = np.array([32, 20])
    same, same_lse = c.run(causal=False)
    assert torch.equal(out, same) and torch.equal(lse, same_lse)


@pytest.mark.parametrize("dtype", [0, 1])
def test_strides(dtype):
    c = Case([1, 40, 97, 210], [1, 30, 3, 1], 2, 4, dim=80, bs=32, dtype=dtype, seed=9, strided=True)
    c.check()
    assert (c.out_buf[:, -1] == 7).all() and (c.out_buf[..., 80:] == 7).all()


@pytest.mark.parametrize("nq", [1, 40])
def test_large_scores_and_scales(nq):
    """Peaked softmax, scores far from zero, scales of very different sizes, zero scales."""
    Case([100, 333], [nq, nq], 1, 4, seed=10, q_gain=100.0).check()
    c = Case([200, 333], [nq, nq], 1, 4, seed=11)
    c.vs *= np.exp(np.linspace(-9, 9, c.vs.size)).astype(np.float32).reshape(c.vs.shape)
    c.cache.v_scales.copy_(torch.from_numpy(c.vs))
    c.check()
    c = Case([200, 333], [nq, nq], 1, 4, seed=12)
    c.ks[:] = np.nan_to_num(c.ks)
    c.ks[::2], c.vs[1::2] = 0, 0
    c.cache.k_scales.copy_(torch.from_numpy(c.ks))
    c.cache.v_scales.copy_(torch.from_numpy(c.vs))
    c.check()
    c = Case([200, 333], [nq, nq], 1, 4, seed=13)
    c.vs[:] = 0
    c.cache.v_scales.copy_(torch.from_numpy(c.vs))
    c.check()


@pytest.mark.parametrize("scale", [0.0, -0.5, 1e-6, 3.0])
def test_scale(scale):
    Case([100, 37], [1, 20], 1, 4, seed=14).check(scale=scale)


def test_zero_queries_and_wide_ranges_of_a_row():
    c = Case([64, 100], [2, 3], 1, 4, seed=16)
    c.q[0] = 0
    c.q[1, 0] = (torch.arange(128).float() % 7 - 3).bfloat16() * 1e30
    c.q[2, 1] = (torch.arange(128).float() % 7 - 3).bfloat16() * 1e-30
    c.q[3, 1, 3:] *= 2.0 ** -20
    c.q_dev = c.q.cuda()
    c.ks[:] = np.nan_to_num(c.ks) * 0 + np.float32(1e-3)
    c.cache.k_scales.copy_(torch.from_numpy(c.ks))
    c.check(scale=1e-3)


@pytest.mark.parametrize("nq", [1, 40])
def test_non_finite_queries_stay_in_their_row(nq):
    c = Case([64, 100, 700], [nq, nq, nq], 2, 4, seed=27)
    clean, clean_lse = c.run()
    c.q_dev = c.q_dev.clone()
    c.q_dev[0, 1, 5], c.q_dev[nq, 6, 0] = float("nan"), float("inf")
    out, lse = c.run()
    bad = torch.zeros_like(lse, dtype=torch.bool)
    bad[0, 1] = bad[nq, 6] = True
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


def test_one_long_context():
    Case([20000], [1], 1, 8, bs=64, seed=17).check()
    Case([9001], [4], 2, 5, bs=16, seed=18).check()


def test_workspace_is_ready_for_the_next_call():
    big = Case([3000, 1, 700], [1, 1, 1], 2, 4, seed=19)
    ws = qr.qr_kv_attention_workspace(torch.empty((64, 16, 128), dtype=torch.bfloat16, device="cuda"), big.cache, 8)
    a, la = big.check(workspace=ws)
    small = Case([5, 2000], [7, 2], 2, 4, seed=20)
    small.check(workspace=ws)
    b, lb = big.run(workspace=ws)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_results_do_not_depend_on_max_q():
    c = Case([40, 130, 257], [1, 3, 100], 1, 8, seed=21)
    want = c.check()
    c.check(max_q=1)
    c.check(max_q=5000)
    assert want[0].shape == c.q.shape


@pytest.mark.parametrize("nq", [1, 4])
def test_max_q_beyond_the_tokens_stays_in_the_workspace(nq):
    c = Case([20000], [nq], 1, 8, seed=22)
    need = qr.qr_kv_attention_workspace_bytes(1, nq, 8, 1, 128)
    buf = torch.full((need + (8 << 20),), 77, dtype=torch.uint8, device="cuda")
    buf[:need] = 0
    want, want_lse = c.check()
    out, lse = c.check(max_q=1 << 20, workspace=buf[:need])
    assert (buf[need:] == 77).all()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_same_bits_twice_and_on_another_stream():
    c = Case([4000, 37, 1], [1, 1, 1], 2, 8, seed=22)
    out, lse = c.check()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again, lse2 = c.run()
    side.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_tokens_past_the_last_request_are_left_alone():
    c = Case([30, 40], [1, 2], 1, 8, seed=23)
    q = torch.cat([c.q_dev, torch.full((5, 8, 128), float("nan"), device="cuda").bfloat16()])
    out = torch.full_like(q, 3.0)
    qr.qr_kv_attention(q, c.cache, c.i32(c.offsets), c.i32(c.kv), c.i32(c.table), out=out)
    assert (out[3:] == 3).all() and torch.isfinite(out[:3].float()).all()


def test_offsets_past_32_bits():
    """Blocks that lie more than 2^32 bytes into the cache."""
    bs, heads, dim = 32, 8, 128
    blocks = (1 << 32) // (bs * heads * dim) + 200
    c = Case([150, 33, 400], [1, 1, 30], heads, 4, dim=dim, bs=bs, seed=24)
    used = c.kc.shape[0]
    kc, vc = (torch.zeros((blocks, heads, bs, dim), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((blocks, heads), float("nan"), device="cuda") for _ in range(2))
    at = blocks - used
    kc[at:], vc[at:] = c.cache.k_codes, c.cache.v_codes
    ks[at:], vs[at:] = c.cache.k_scales, c.cache.v_scales
    small = c.run()
    c.cache = qr.KVCache(kc, vc, ks, vs)
    c.table = np.where((c.table >= 0) & (c.table < used), c.table + at, c.table)
    big = c.run()
    assert torch.equal(small[0], big[0]) and torch.equal(small[1], big[1])


def test_graph_capture():
    c = Case([500, 37], [1, 1], 1, 8, seed=25)
    ws = qr.qr_kv_attention_workspace(c.q_dev, c.cache, 2)
    want, want_lse = c.check(workspace=ws)
    off, kv, table = c.i32(c.offsets), c.i32(c.kv), c.i32(c.table)
    out = torch.zeros_like(c.q_dev)
    qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, max_q=1, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, max_q=1, out=out, workspace=ws)
    out.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_tokens_and_refusals():
    c = Case([30, 40], [1, 2], 1, 8, seed=26)
    off, kv, table = c.i32(c.offsets), c.i32(c.kv), c.i32(c.table)
    none = qr.qr_kv_attention(c.q_dev[:0], c.cache, c.i32([0, 0, 0]), kv, table)
    assert none.shape == (0, 8, 128)
    with pytest.raises(TypeError):
        qr.qr_kv_attention(c.q_dev.float(), c.cache, off, kv, table)
    with pytest.raises(ValueError):
        qr.qr_kv_attention(c.q_dev[..., :64], c.cache, off, kv, table)
    with pytest.raises(ValueError):
        qr.qr_kv_attention(c.q_dev, c.cache, off[:2], kv, table)
    with pytest.raises(TypeError):
        qr.qr_kv_attention(c.q_dev, c.cache, off, kv.long(), table)
    for kw in (dict(window=-1), dict(window=4, causal=False), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(max_q=0)):
        with pytest.raises(qr.QRError) as e:
            qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, **kw)
        assert e.value.status == qr.QR_ERR_INVALID_ARG
    with pytest.raises(qr.QRError) as e:
        qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, out=c.q_dev)
    assert e.value.status == qr.QR_ERR_INVALID_ARG
    with pytest.raises(qr.QRError) as e:
        qr.qr_kv_attention(c.q_dev, c.cache, off, kv, table, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == qr.QR_ERR_SIZE
    two = qr.KVCache.empty(4, 3, 16, 128)
    with pytest.raises((qr.QRError, ValueError)):
        qr.qr_kv_attention(c.q_dev, two, off, kv, table)
