"""Cases of the serving operators: the key/value cache held in 8 bits (its
plan, its writer, the attention that reads it) and the matrix-vector product
with 4-bit weights.

Where ``own`` is false, ``run`` computes an operator in plain torch operations
in 32 bits; where it is true, it makes the library's calls.  Lengths are fixed
by the case (a spread between 1 and the largest) and dealt to the requests by
the seed, so that a case's work does not depend on the seed.
"""
import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _qr():
    import bit_quantized_all_gb300 as qr
    return qr


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the step's bookkeeping for 16 decoding requests: pure latency
        dict(name="plan 16 decode", op="plan", requests=16, max_new=1, max_cached=2048, block=16),
        # a large mixed batch: most requests bring long prompts
        dict(name="plan 2048 mixed", op="plan", requests=2048, max_new=1024, max_cached=4096, block=16),
        # 16 decoding requests on one rank of eight (one key/value head each): latency
        dict(name="append 16 decode", op="append", requests=16, max_new=1, max_cached=2048, heads=1, dim=128,
             block=16, dtype="bf16"),
        # a full decode batch on an unsharded layer: single tokens into partly filled blocks
        dict(name="append 256 decode", op="append", requests=256, max_new=1, max_cached=4096, heads=8, dim=128,
             block=64, dtype="fp16"),
        # prompts of a 32 x 1024 batch being written: bandwidth
        dict(name="append 32x1024 prompt", op="append", requests=32, max_new=1024, same_new=True, max_cached=1,
             heads=8, dim=128, block=32, dtype="bf16"),
        # 16 decode slots, hidden 8192 over eight ranks: 8 query heads share one key/value head; two slots idle
        dict(name="attention 16 decode", op="attention", requests=16, idle=2, max_new=1, max_kv=2048, q_heads=8,
             kv_heads=1, dim=128, block=16, dtype="bf16"),
        # a full decode batch with long contexts: bandwidth
        dict(name="attention 128 decode", op="attention", requests=128, idle=0, max_new=1, max_kv=8192, q_heads=32,
             kv_heads=8, dim=128, block=64, dtype="fp16"),
        # one very long context verified four drafted tokens at a time (hidden 5120: 40 heads)
        dict(name="attention 1 long", op="attention", requests=1, idle=0, max_new=4, max_kv=131075, q_heads=40,
             kv_heads=8, dim=128, block=32, dtype="bf16"),
        # prompt chunks of up to 1024 tokens behind what is cached: arithmetic
        dict(name="attention 8 prompts", op="attention", requests=8, idle=0, max_new=1024, max_kv=8192, q_heads=40,
             kv_heads=8, dim=128, block=32, dtype="bf16"),
        # one token through a rank's slice of an 8192 x 8192 projection: latency
        dict(name="matvec 1x8192x1024", op="matvec", tokens=1, rows=8192, cols=1024, group=32, zeros=False,
             dtype="bf16"),
        # a decode batch of 16 through the whole projection, weights with zero points
        dict(name="matvec 16x8192x8192", op="matvec", tokens=16, rows=8192, cols=8192, group=128, zeros=True,
             dtype="fp16"),
        # the largest batch that still counts as few rows, at odd sizes
        dict(name="matvec 64x20481x5123", op="matvec", tokens=64, rows=20481, cols=5123, group=64, zeros=False,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi + 0.5))))))))


def draw(rng):
    op = rng.choice(("plan", "append", "attention", "attention", "matvec"))
    dtype = rng.choice(("fp16", "bf16"))
    block = rng.choice((16, 32, 64, 128))
    if op == "plan":
        return dict(op=op, requests=_log_int(rng, 1, 2048), max_new=_log_int(rng, 1, 1024),
                    max_cached=_log_int(rng, 1, 4096), block=block)
    dim = rng.choice((64, 80, 96, 128, 128, 256))
    if op == "append":
        heads = rng.choice((1, 2, 3, 5, 8, 16))
        requests = _log_int(rng, 1, 512)
        most = max(1, 32 * 1024 * 1024 // (requests * heads * dim))
        max_new = 1 if rng.random() < 0.4 else _log_int(rng, 1, min(1024, most))
        return dict(op=op, requests=requests, max_new=max_new, max_cached=_log_int(rng, 1, 4096), heads=heads,
                    dim=dim, block=block, dtype=dtype)
    if op == "attention":
        kv_heads = rng.choice((1, 2, 3, 8))
        group = rng.choice((1, 4, 5, 8, 16))
        kind = rng.choice(("decode", "decode", "draft", "prompt"))
        requests = _log_int(rng, 1, 128 if kind != "prompt" else 8)
        kv_values = 8 * 128 * 8192 * 128  # the largest listed cache and the largest listed score matrix
        scores = 8 * 40 * 1024 * 8192
        max_kv = min(_log_int(rng, 64, 131072), kv_values // (requests * kv_heads * dim))
        max_new = {"decode": 1, "draft": rng.randint(2, 8), "prompt": _log_int(rng, 16, 1024)}[kind]
        max_new = max(1, min(max_new, max_kv, scores // (requests * kv_heads * group * max_kv)))
        return dict(op=op, requests=requests, idle=1 if requests > 3 and rng.random() < 0.5 else 0, max_new=max_new,
                    max_kv=max_kv, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype)
    rows = _log_int(rng, 64, 20480)
    cols = _log_int(rng, 64, min(16384, 20480 * 5120 // rows))
    return dict(op=op, tokens=_log_int(rng, 1, 64), rows=rows, cols=cols, group=rng.choice((32, 64, 128)),
                zeros=rng.random() < 0.5, dtype=dtype)


# ---------------------------------------------------------------------------
# lengths: a fixed spread for the case, dealt out by the seed
# ---------------------------------------------------------------------------
def _spread(count, most):
    """`count` lengths evenly spread over [1, most], the largest among them."""
    return np.maximum(1, np.ceil(most * (np.arange(count) + 1) / count)).astype(np.int64)


def _lengths(case):
    """(cached, new) lengths of the case's requests, in a fixed order."""
    n = case["requests"]
    if case["op"] == "attention":
        kv = _spread(n, case["max_kv"])
        # the same share of the longest chunk for every request, at least one token
        new = np.minimum(kv, np.maximum(1, case["max_new"] * (n - np.arange(n)) // n))
        kv[:case["idle"]] = 0
        new[:case["idle"]] = 1
        return kv - new, new  # an idle slot: one query, nothing cached (cached = -1)
    new = np.full(n, case["max_new"]) if case.get("same_new") else _spread(n, case["max_new"])[::-1].copy()
    cached = _spread(n, case["max_cached"]) - 1  # from nothing cached on
    return cached, new


def _blocks(lengths, block):
    return -(-np.maximum(lengths, 0) // block)


def _dealt(case, seed):
    cached, new = _lengths(case)
    order = np.random.RandomState(seed % (1 << 31)).permutation(len(cached))
    return cached[order], new[order]


def work(case):
    if case["op"] == "matvec":
        m, n, k, g = case["tokens"], case["rows"], case["cols"], case["group"]
        groups = -(-k // g)
        weights = n * k / 2 + n * groups * (2.5 if case["zeros"] else 2)
        return {"bytes": weights + 2 * m * (n + k), "flops": 2 * m * n * k}
    cached, new = _lengths(case)
    total = cached + new
    tokens, block = int(new.sum()), case["block"]
    if case["op"] == "plan":
        taken = int((_blocks(total, block) - _blocks(cached, block)).sum())
        touched = int((_blocks(total, block) - cached // block).sum())
        return {"bytes": 8 * tokens + 8 * taken + 4 * (touched - taken) + 16 * len(cached), "flops": 0}
    if case["op"] == "append":
        values = tokens * case["heads"] * case["dim"] * 2
        touched = int((_blocks(total, block) - cached // block).sum())
        return {"bytes": 3 * values + 8 * tokens + 2 * 8 * touched * case["heads"], "flops": 0}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    kv = np.maximum(total, 0)
    pairs = int(np.sum(np.where(kv > 0, new * kv - new * (new - 1) // 2, 0)))
    rows = tokens * hq
    return {"bytes": int(kv.sum()) * hk * 2 * d + int(_blocks(kv, block).sum()) * (8 * hk + 4) + rows * (4 * d + 4),
            "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _activations(gen, shape, dtype):
    """Normal values with a few large channels, as projections give them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    big = torch.randint(0, shape[-1], (max(1, shape[-1] // 32),), generator=gen, device="cuda")
    x[..., big] *= 8.0
    return x.to(dtype)


def _ints(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _table(lengths, ids, block, width):
    """Block tables: consecutive entries of `ids` for each request, then -1."""
    need = _blocks(lengths, block)
    at = np.arange(width)[None, :]
    start = np.cumsum(need) - need
    picked = ids[np.minimum(start[:, None] + at, len(ids) - 1)]
    return np.where(at < need[:, None], picked, -1)


def _cache(gen, blocks, heads, block, dim):
    """A filled cache: codes of normal values, a scale for each block and head."""
    shape = (blocks, heads, block, dim)
    out = []
    for _ in range(2):
        codes = torch.empty(shape, dtype=torch.int8, device="cuda")
        step = max(1, (64 << 20) // (heads * block * dim))
        for i in range(0, blocks, step):
            part = codes[i:i + step]
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(36.0).round_().clamp_(-128, 127))
        scales = torch.rand((blocks, heads), generator=gen, device="cuda") * 0.02 + 0.02
        out += [codes, scales]
    return out  # k codes, k scales, v codes, v scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "matvec":
        dtype = DTYPES[case["dtype"]]
        n, k, groups = case["rows"], case["cols"], -(-case["cols"] // case["group"])
        s["x"] = _activations(gen, (case["tokens"], k), dtype)
        s["codes"] = torch.randint(0, 256, (n, -(-k // 2)), generator=gen, device="cuda", dtype=torch.uint8)
        s["scales"] = (torch.rand((n, groups), generator=gen, device="cuda") * 0.004 + 0.001).half()
        s["zero"] = (torch.randint(4, 12, (n, groups), generator=gen, device="cuda", dtype=torch.uint8)
                     if case["zeros"] else None)
        if own:  # a program lays its weights out once
            s["weight"] = _qr().qr_w4_pack(s["codes"], s["scales"], k, group=case["group"], zeros=s["zero"])
        return s
    block = case["block"]
    cached, new = _dealt(case, int(seed))
    total = cached + new
    offsets = np.concatenate([[0], np.cumsum(new)])
    ids_rng = np.random.RandomState((int(seed) + 1) % (1 << 31))
    width = int(_blocks(total, block).max()) if len(total) else 1
    width = max(1, width)
    need = int(_blocks(total, block).sum())
    pool = need + max(4, need // 16)
    ids = ids_rng.permutation(pool)
    s["tokens"], s["max_new"] = int(offsets[-1]), int(new.max())
    if case["op"] == "plan":
        had = int(_blocks(cached, block).sum())
        s["cached"], s["new"] = _ints(cached), _ints(new)
        s["table"] = _ints(_table(cached, ids[:max(1, had)], block, width))
        s["free"] = _ints(ids[had:])
        return s
    table = _table(total, ids, block, width)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "append":
        k_codes, k_scales, v_codes, v_scales = _cache(gen, pool, case["heads"], block, case["dim"])
        # keys and values are slices of one projection's output, as a fused projection leaves them
        kv = _activations(gen, (s["tokens"], 2 * case["heads"], case["dim"]), dtype)
        s["k"], s["v"] = kv[:, :case["heads"]], kv[:, case["heads"]:]
        request = np.repeat(np.arange(len(new)), new)
        at = cached[request] + np.arange(s["tokens"]) - offsets[request]
        held = table[request, at // block]
        s["slots"] = _ints(held.astype(np.int64) * block + at % block, torch.int64)
        touched, place = np.unique(held, return_inverse=True)
        s["touched"], s["place"] = _ints(touched, torch.int64), _ints(place.reshape(-1), torch.int64)
        s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"] = k_codes, k_scales, v_codes, v_scales
        if own:
            s["cache"] = _qr().KVCache(k_codes, v_codes, k_scales, v_scales)
        return s
    s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"] = _cache(gen, pool, case["kv_heads"], block, case["dim"])
    s["q"] = _activations(gen, (s["tokens"], case["q_heads"], case["dim"]), dtype)
    s["offsets"], s["kv_lens"], s["table"] = _ints(offsets), _ints(np.maximum(total, 0)), _ints(table)
    s["max_len"] = max(1, int(total.max()))
    if own:
        qr = _qr()
        s["cache"] = qr.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        s["workspace"] = qr.qr_kv_attention_workspace(s["q"], s["cache"], case["requests"], s["max_new"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"plan": _run_plan, "append": _run_append, "attention": _run_attention, "matvec": _run_matvec}[s["op"]](s)


def _run_plan(s):
    if own:
        plan = _qr().qr_kv_plan(s["cached"], s["new"], s["table"], s["free"], s["block"], s["tokens"])
        return {"table": plan.block_table, "offsets": plan.q_offsets, "kv_lens": plan.kv_lens, "slots": plan.slots}
    cached, new, table, block = s["cached"], s["new"], s["table"], s["block"]
    kv_lens = cached + new
    have, need = (cached + (block - 1)) // block, (kv_lens + (block - 1)) // block
    offsets = torch.cat([new.new_zeros(1), torch.cumsum(new, 0).to(torch.int32)])
    taken = need - have
    start = torch.cumsum(taken, 0) - taken
    at = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (at >= have[:, None]) & (at < need[:, None])
    pick = (start[:, None] + at - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][pick], table))
    token = torch.arange(s["tokens"], device=table.device)
    request = torch.repeat_interleave(torch.arange(new.numel(), device=table.device), new, output_size=s["tokens"])
    pos = cached[request] + token - offsets[request]
    slots = table[request, pos // block].to(torch.int64) * block + pos % block
    return {"table": table, "offsets": offsets, "kv_lens": kv_lens, "slots": slots}


def _append_half(x, codes, scales, s):
    touched, place, offset = s["touched"], s["place"], s["slots"] % s["block"]
    x = x.float()
    most = torch.zeros((touched.numel(), x.shape[1]), device=x.device)
    most.scatter_reduce_(0, place[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    kept = torch.full((touched.numel(),), s["block"], device=x.device, dtype=torch.int64)
    kept.scatter_reduce_(0, place, offset, "amin")
    old = torch.where(kept[:, None] > 0, scales[touched], 0.0)
    scale = torch.maximum(old, most * (1.0 / 128.0))
    factor = torch.where(scale > 0, torch.ones_like(scale) / scale, 0.0)
    held = codes[touched]
    moved = ((held.float() * old[..., None, None]) * factor[..., None, None]).clamp(-128.0, 127.0).round()
    keep = torch.arange(s["block"], device=x.device)[None, :] < kept[:, None]
    codes[touched] = torch.where(keep[:, None, :, None], moved.to(torch.int8), held)
    fresh = (x * factor[place][..., None]).clamp(-128.0, 127.0).round()
    codes[touched[place], :, offset] = fresh.to(torch.int8)
    scales[touched] = scale


def _run_append(s):
    """The updated cache.  A code is a whole number that the definition fixes
    (every rounding of it is one in 32 bits), so codes are held to equality."""
    if own:
        _qr().qr_kv_append(s["cache"], s["k"], s["v"], s["slots"])
    else:
        _append_half(s["k"], s["k_codes"], s["k_scales"], s)
        _append_half(s["v"], s["v_codes"], s["v_scales"], s)
    return {"k_codes": s["k_codes"], "v_codes": s["v_codes"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _run_attention(s):
    scale = s["dim"] ** -0.5
    if own:
        out, lse = _qr().qr_kv_attention(s["q"], s["cache"], s["offsets"], s["kv_lens"], s["table"], scale=scale,
                                         max_q=s["max_new"], return_lse=True, workspace=s["workspace"])
        return {"out": out, "lse": lse}
    q, offsets, kv_lens, table, block = s["q"], s["offsets"].long(), s["kv_lens"].long(), s["table"], s["block"]
    requests, heads, group, dim = s["requests"], s["kv_heads"], s["q_heads"] // s["kv_heads"], s["dim"]
    length, most = s["max_len"], s["max_new"]
    at = torch.arange(length, device=q.device)
    held = table[:, at // block].clamp(min=0).long()
    # [requests, length, heads, dim] -> [requests, heads, length, dim]
    k = (s["k_codes"][held, :, at % block].float() * s["k_scales"][held][..., None]).transpose(1, 2)
    v = (s["v_codes"][held, :, at % block].float() * s["v_scales"][held][..., None]).transpose(1, 2)
    nth = torch.arange(most, device=q.device)
    counts = offsets[1:] - offsets[:-1]
    rows = (offsets[:-1, None] + nth).clamp(max=q.shape[0] - 1)
    qp = q[rows].float().view(requests, most, heads, group, dim).permute(0, 2, 3, 1, 4)
    qp = qp.reshape(requests, heads, group * most, dim)
    scores = torch.matmul(qp, k.transpose(2, 3)).mul_(scale)
    pos = (kv_lens - counts)[:, None] + nth
    seen = (at <= pos[..., None]) & (at < kv_lens[:, None, None])  # [requests, most, length]
    scores = scores.view(requests, heads, group, most, length).masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(requests, heads, group * most, length), v).view(requests, heads, group, most, dim)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log()).squeeze(-1)
    token = torch.arange(q.shape[0], device=q.device)
    request = torch.searchsorted(offsets[1:].contiguous(), token, right=True)
    nth_of = token - offsets[request]
    return {"out": out[request, :, :, nth_of].reshape(-1, heads * group, dim).to(q.dtype),
            "lse": lse[request, :, :, nth_of].reshape(-1, heads * group)}


def _run_matvec(s):
    if own:
        return _qr().qr_w4_matvec(s["x"], s["weight"])
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=-1).flatten(1)[:, :s["cols"]].float()
    column = torch.arange(s["cols"], device=codes.device) // s["group"]
    zero = 8.0 if s["zero"] is None else s["zero"].float()[:, column]
    weight = (codes - zero) * s["scales"].float()[:, column]
    return torch.matmul(s["x"].float(), weight.t()).to(s["x"].dtype)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "matvec":
        x, weight = s["x"].double(), torch.empty((case["rows"], case["cols"]), dtype=torch.float64, device="cuda")
        weight[:, 0::2] = (s["codes"] % 16).double()[:, :weight[:, 0::2].shape[1]]
        weight[:, 1::2] = (s["codes"] // 16).double()[:, :weight[:, 1::2].shape[1]]
        for g in range(s["scales"].shape[1]):
            part = weight[:, g * case["group"]:(g + 1) * case["group"]]
            part -= 8.0 if s["zero"] is None else s["zero"][:, g:g + 1].double()
            part *= s["scales"][:, g:g + 1].double()
        return x @ weight.T
    if case["op"] == "append":
        block, slots = case["block"], s["slots"].cpu().numpy()
        held = slots // block
        runs = np.flatnonzero(np.concatenate([[True], held[1:] != held[:-1]])).tolist() + [len(slots)]
        out = {"k_codes": None, "v_codes": None}
        for name in ("k", "v"):
            scales = s[name + "_scales"].double()
            most = s[name].double().abs().amax(-1).cpu().numpy()
            grown = scales.cpu().numpy()
            for a, b in zip(runs[:-1], runs[1:]):
                at = held[a]
                new = most[a:b].max(0) / 128.0
                grown[at] = np.maximum(grown[at], new) if slots[a] % block else new
            out[name + "_scales"] = torch.from_numpy(grown)
        return out
    cached, new = _dealt(case, int(seed))
    offsets = np.concatenate([[0], np.cumsum(new)])
    hq, hk, d, block = case["q_heads"], case["kv_heads"], case["dim"], case["block"]
    out = torch.zeros((s["tokens"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    for r in range(len(new)):
        kv, n = int(cached[r] + new[r]), int(new[r])
        if kv <= 0:
            continue
        ids = s["table"][r, :-(-kv // block)].long()
        hidden = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda")[:, None]
        for h in range(hk):
            k = (s["k_codes"][ids, h].double() * s["k_scales"][ids, h].double()[:, None, None]).reshape(-1, d)[:kv]
            v = (s["v_codes"][ids, h].double() * s["v_scales"][ids, h].double()[:, None, None]).reshape(-1, d)[:kv]
            for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                at = slice(int(offsets[r]), int(offsets[r]) + n)
                score = (s["q"][at, j].double() @ k.T) * d ** -0.5
                score[hidden] = float("-inf")
                lse[at, j] = torch.logsumexp(score, -1)
                out[at, j] = torch.softmax(score, -1) @ v
    return {"out": out, "lse": lse}
