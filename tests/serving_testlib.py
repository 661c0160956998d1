"""Plain 64-bit (numpy) forms of the serving operators and input builders,
shared by their tests.  Nothing here uses the package.

Error bounds (derived, not fitted).  With u_out the output type's unit
roundoff (2^-11 fp16, 2^-8 bf16: half an ulp relative to the value):

attention  scores are fp32 sums of exact products: |dS| <= d :=
           2^-19 * |scale| * max_i sum_d |q_d k_id| + 2^-20 (the log2/exp2
           arithmetic near the running maximum adds at most 2^-20 + 2^-22 |S|,
           which |S| <= |scale| * sum |q k| folds into the same bound).
           A softmax weight is rounded to fp16 (2^-11), so with
           B = sum_i P_i |v_i|:  |d out| <= (2^-11 + 2 d + 2^-18) B
           + u_out |out| + the smallest subnormal of the type; weights below
           fp16's normal range lose at most 2^-25 of the row's largest each,
           i.e. 2^-25 * sum_i |v_i| / l with l >= 1 when scaled by the largest.
           (The weights are held as two fp16 numbers, to 2^-22; test_gpu_kv_weights
           has the bound for that, and inputs on which it tells.)
           |d lse| <= d + 2^-20 + 2^-22 |lse|.
matvec     products are exact in fp32; a sum of K of them in any order of
           tensor-core steps errs by at most (K / 8 + 64) * 2^-23 * sum |x w|.
"""
from __future__ import annotations

import numpy as np

U_OUT = {0: 2.0 ** -11, 1: 2.0 ** -8}
TINY = {0: 2.0 ** -24, 1: 2.0 ** -133}


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def plan(cached, new, table, free, bs, max_tokens):
    """(table, q_offsets, kv_lens, slots, counts), request by request."""
    table = table.copy()
    width = table.shape[1]
    off, kv, slots = [0], [], []
    taken = short = beyond = 0
    for r in range(len(cached)):
        c, n = max(int(cached[r]), 0), max(int(new[r]), 0)
        have, need = -(-c // bs), -(-(c + n) // bs)
        fresh = {}
        for b in range(have, need):
            i = taken + short
            block = int(free[i]) if i < len(free) else -1
            if i < len(free):
                taken += 1
            else:
                short += 1
            fresh[b] = block
            if b < width:
                table[r, b] = block
        beyond += max(0, need - width)
        for p in range(c, c + n):
            b = p // bs
            block = (fresh[b] if b >= have else int(table[r, b])) if b < width else -1
            slots.append(block * bs + p % bs if block >= 0 else -1)
        off.append(off[-1] + n)
        kv.append(c + n)
    total = off[-1]
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return (table, np.minimum(off, max_tokens).astype(np.int64), np.array(kv), np.array(slots, dtype=np.int64),
            np.array([taken, total, short, beyond]))


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _rint_clip(x):
    return np.rint(np.clip(x, np.float32(-128), np.float32(127)))


def append(x, codes, scales, slots, bs):
    """Updated (codes, scales) of one half; float32 step by step, as the
    definition rounds."""
    codes, scales = codes.copy(), scales.copy()
    x = x.astype(np.float32)
    blocks = codes.shape[0]
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if not 0 <= s < blocks * bs:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % bs:
            n += 1
        b, o = divmod(s, bs)
        for h in range(codes.shape[1]):
            run = x[t:t + n, h]
            old = scales[b, h] if o else np.float32(0)
            new = np.maximum(old, np.float32(np.abs(run).max()) * np.float32(2.0 ** -7))
            r = np.float32(1) / new if new > 0 else np.float32(0)
            if o and new > old:
                kept = codes[b, h, :o].astype(np.float32) * old
                codes[b, h, :o] = _rint_clip(kept * r)
            codes[b, h, o:o + n] = _rint_clip(run * r)
            scales[b, h] = new
        t += n
    return codes, scales


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attention(q, q_offsets, kv_lens, table, kc, ks, vc, vs, scale, causal=True, window=0, dtype=1):
    """(out, lse, bound on |d out|, bound on |d lse|) in float64."""
    T, Hq, D = q.shape
    blocks, H, bs, _ = kc.shape
    G = Hq // H
    q = q.astype(np.float64)
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    b_out, b_lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for r in range(len(kv_lens)):
        lo, hi = int(q_offsets[r]), int(q_offsets[r + 1])
        kv = max(0, min(int(kv_lens[r]), table.shape[1] * bs))
        ids = table[r, :-(-kv // bs)] if kv else np.zeros(0, np.int64)
        ok = np.repeat((ids >= 0) & (ids < blocks), bs)[:kv]
        ids = np.where((ids >= 0) & (ids < blocks), ids, 0)
        pos = np.arange(kv)
        for h in range(H):
            k = (kc[ids, h].astype(np.float64) * ks[ids, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:kv]
            v = (vc[ids, h].astype(np.float64) * vs[ids, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:kv]
            k[~ok], v[~ok] = 0, 0
            for t in range(lo, hi):
                p = int(kv_lens[r]) - (hi - lo) + (t - lo)
                see = ok.copy()
                if causal:
                    see &= pos <= p
                if window:
                    see &= pos > p - window
                if not see.any():
                    continue
                for j in range(h * G, (h + 1) * G):
                    s = scale * (k[see] @ q[t, j])
                    mag = abs(scale) * np.abs(k[see]) @ np.abs(q[t, j])
                    top = s.max()
                    e = np.exp(s - top)
                    l = e.sum()
                    out[t, j] = (e @ v[see]) / l
                    lse[t, j] = top + np.log(l)
                    d = 2.0 ** -19 * np.abs(mag).max() + 2.0 ** -20
                    B = (e @ np.abs(v[see])) / l
                    b_out[t, j] = ((2.0 ** -11 + 2 * d + 2.0 ** -18) * B + U_OUT[dtype] * np.abs(out[t, j])
                                   + 2.0 ** -25 * np.abs(v[see]).sum(0) / l + TINY[dtype])
                    b_lse[t, j] = d + 2.0 ** -20 + 2.0 ** -22 * abs(lse[t, j])
    return out, lse, b_out, b_lse


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
def w4_dense(codes, scales, zeros, cols, group):
    """The weights as float64 [rows, cols]."""
    u = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)[:, :cols].astype(np.float64)
    col = np.arange(cols) // group
    z = 8.0 if zeros is None else zeros.astype(np.float64)[:, col]
    return (u - z) * scales.astype(np.float64)[:, col]


def matvec(x, w, dtype):
    """(y, bound on |d y|) in float64."""
    x = x.astype(np.float64)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    return y, (x.shape[1] / 8 + 64) * 2.0 ** -23 * mag + U_OUT[dtype] * np.abs(y) + TINY[dtype]
