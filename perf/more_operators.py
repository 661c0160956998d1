"""Cases of the operators between a layer's residual stream and its attention:
root-mean-square norm with the residual's addition and an output in 16 or 8
bits, rows quantized to 8 bits, the 8-bit integer product with a scale for each
token and channel, and rotary positions.

Where ``own`` is false, ``run`` computes an operator in plain torch operations
in 32 bits (the angles of the rotary positions in 64); where it is true, it
makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def _qr():
    import bit_quantized_all_gb300 as qr
    return qr


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # 16 decoding requests of hidden 8192 between two layers: the residual's sum and 8-bit rows, pure latency
        dict(name="norm8 16x8192", op="norm", tokens=16, cols=8192, eight=True, residual=True, fp32_weight=False,
             dtype="bf16"),
        # prompts of a 32 x 1024 batch, residual's sum and 8-bit rows: bandwidth
        dict(name="norm8 32768x8192", op="norm", tokens=32768, cols=8192, eight=True, residual=True,
             fp32_weight=False, dtype="bf16"),
        # the norm before a 16-bit consumer, odd sizes, weights kept in 32 bits, no residual (a stack's last norm)
        dict(name="norm 2049x5123", op="norm", tokens=2049, cols=5123, eight=False, residual=False,
             fp32_weight=True, dtype="fp16"),
        # a decode batch's attention output (hidden 5120) into 8-bit rows
        dict(name="quantize 64x5120", op="quantize", tokens=64, cols=5120, dtype="fp16"),
        # prompts' activations of a 20480 wide layer into 8-bit rows
        dict(name="quantize 8192x20480", op="quantize", tokens=8192, cols=20480, dtype="bf16"),
        # 16 decoding requests on one rank of eight: 8 query heads and one key head
        dict(name="rope 16x9", op="rope", tokens=16, q_heads=8, k_heads=1, dim=128, rot=128, layout="half",
             scaling="none", far=8192, dtype="bf16"),
        # prompts of a 32 x 1024 batch on an unsharded layer of hidden 5120: bandwidth
        dict(name="rope 32768x48", op="rope", tokens=32768, q_heads=40, k_heads=8, dim=128, rot=128,
             layout="interleaved", scaling="none", far=8192, dtype="bf16"),
        # half of each head rotated, in a context stretched to a million tokens
        dict(name="rope 4097x10 far", op="rope", tokens=4097, q_heads=8, k_heads=2, dim=256, rot=128, layout="half",
             scaling="yarn", far=1048576, dtype="fp16"),
        # one token through a rank's share of the query, key and value projection of hidden 8192 (1280 = 10240 / 8)
        dict(name="product 1x1280x8192", op="product", tokens=1, rows=1280, cols=8192, dtype="bf16"),
        # a decode batch of 16 through the whole projection (64 query, 8 key and 8 value heads of 128)
        dict(name="product 16x10240x8192", op="product", tokens=16, rows=10240, cols=8192, dtype="bf16"),
        # a large decode batch at odd sizes
        dict(name="product 129x20481x5123", op="product", tokens=129, rows=20481, cols=5123, dtype="fp16"),
        # prompt chunks: arithmetic
        dict(name="product 4096x10240x8192", op="product", tokens=4096, rows=10240, cols=8192, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "rope", "product", "product"))
    dtype = rng.choice(("fp16", "bf16"))
    if op in ("norm", "quantize"):
        cols = _log_int(rng, 64, 24576)
        if rng.random() < 0.5:
            cols = -(-cols // 128) * 128
        most = (32768 * 8192 if op == "norm" else 8192 * 20480) // cols
        case = dict(op=op, tokens=_log_int(rng, 1, min(65536, most)), cols=cols, dtype=dtype)
        if op == "norm":
            case.update(eight=rng.random() < 0.6, residual=rng.random() < 0.6, fp32_weight=rng.random() < 0.3)
        return case
    if op == "rope":
        dim = rng.choice((64, 80, 96, 128, 128, 256))
        rot = rng.choice((dim, dim, dim // 2, dim // 16 * 4))
        k_heads = rng.choice((1, 2, 3, 8))
        q_heads = k_heads * rng.choice((1, 4, 5, 8))
        most = 32768 * 48 * 128 // (dim * (q_heads + k_heads))
        return dict(op=op, tokens=_log_int(rng, 1, min(65536, most)), q_heads=q_heads, k_heads=k_heads, dim=dim,
                    rot=rot, layout=rng.choice(("half", "interleaved")),
                    scaling=rng.choice(("none", "linear", "ntk", "yarn")), far=_log_int(rng, 1024, 1048576),
                    dtype=dtype)
    rows = _log_int(rng, 64, 20480)
    cols = _log_int(rng, 64, 16384)
    most = min(4096, 4096 * 10240 * 8192 // (rows * cols))
    return dict(op=op, tokens=_log_int(rng, 1, most), rows=rows, cols=cols, dtype=dtype)


def work(case):
    t = case["tokens"]
    if case["op"] == "norm":
        n = t * case["cols"]
        values = 2 * n + (4 * n if case["residual"] else 0) + (n + 4 * t if case["eight"] else 2 * n)
        return {"bytes": values + case["cols"] * (4 if case["fp32_weight"] else 2), "flops": 0}
    if case["op"] == "quantize":
        return {"bytes": 3 * t * case["cols"] + 4 * t, "flops": 0}
    if case["op"] == "rope":
        # the whole of a head's values go to the output, rotated or not
        return {"bytes": 4 * t * (case["q_heads"] + case["k_heads"]) * case["dim"] + 4 * t, "flops": 0}
    n, k = case["rows"], case["cols"]
    return {"bytes": n * k + 4 * n + t * k + 4 * t + 2 * t * n, "flops": 2 * t * n * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _activations(gen, shape, dtype):
    """Normal values with a few large channels, as a layer's activations have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    big = torch.randint(0, shape[-1], (max(1, shape[-1] // 64),), generator=gen, device="cuda")
    x[..., big] *= 8.0
    return x.to(dtype)


def _codes(gen, rows, cols):
    """8-bit codes of normal rows whose largest value is near 127, in rows that begin on 16-byte boundaries."""
    codes = torch.zeros((rows, -(-cols // 16) * 16), dtype=torch.int8, device="cuda")
    step = max(1, (64 << 20) // codes.shape[1])
    for i in range(0, rows, step):
        part = codes[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(32.0).round_().clamp_(-127, 127))
    return codes[:, :cols]


def _frequencies(case):
    """Radians a position for each rotated pair, and the factor of the rotated values, from the published formulas."""
    rot, base, kind = case["rot"], 10000.0, case["scaling"]
    pair = np.arange(0, rot, 2, dtype=np.float64)
    if kind == "linear":
        return base ** (-pair / rot) / 4.0, 1.0
    if kind == "ntk":
        return (base * 4.0 ** (rot / (rot - 2.0))) ** (-pair / rot), 1.0
    plain = base ** (-pair / rot)
    if kind == "none":
        return plain, 1.0
    # "yarn": a ramp over the pairs between those that turn 32 times and once in the original length
    factor, original = 32.0, 32768.0
    at = [rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - low) / max(high - low, 0.001), 0.0, 1.0)
    return plain / factor * ramp + plain * (1.0 - ramp), 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    tokens = case["tokens"]
    if case["op"] in ("norm", "quantize"):
        dtype = DTYPES[case["dtype"]]
        s["x"] = _activations(gen, (tokens, case["cols"]), dtype)
        if case["op"] == "norm":
            weight = torch.rand(case["cols"], generator=gen, device="cuda") + 0.5
            s["weight"] = weight if case["fp32_weight"] else weight.to(dtype)
            s["res"] = _activations(gen, (tokens, case["cols"]), dtype) if case["residual"] else None
            s["res_out"] = torch.empty_like(s["res"]) if case["residual"] else None
        return s
    if case["op"] == "rope":
        dtype, heads = DTYPES[case["dtype"]], case["q_heads"] + 2 * case["k_heads"]
        # queries, keys and values as one projection leaves them
        qkv = _activations(gen, (tokens, heads * case["dim"]), dtype).view(tokens, heads, case["dim"])
        s["q"], s["k"] = qkv[:, :case["q_heads"]], qkv[:, case["q_heads"]:case["q_heads"] + case["k_heads"]]
        # requests of 1024 consecutive tokens that begin anywhere
        begin = torch.randint(0, case["far"], (tokens // 1024 + 1,), generator=gen, device="cuda")
        token = torch.arange(tokens, device="cuda")
        s["positions"] = (begin[token // 1024] + token % 1024).to(torch.int32)
        frequencies, s["factor"] = _frequencies(case)
        s["frequencies"] = torch.from_numpy(frequencies).cuda()
        if own:  # a program makes its table once
            s["table"] = _qr().Rope(frequencies, layout=case["layout"], factor=s["factor"])
        return s
    s["x"], s["x_scales"] = _codes(gen, tokens, case["cols"]), torch.rand(tokens, generator=gen, device="cuda") * 0.02 + 0.02
    s["w"] = _codes(gen, case["rows"], case["cols"])
    s["w_scales"] = torch.rand(case["rows"], generator=gen, device="cuda") * 0.0004 + 0.0004
    if own:  # a program lays its weights out once, and keeps a workspace
        qr = _qr()
        s["weight"] = qr.qr_w8_pack(s["w"], s["w_scales"])
        s["rows8"] = qr.Q8Rows(s["x"], s["x_scales"])
        s["workspace"] = qr.qr_w8_matmul_workspace(tokens, s["weight"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"norm": _run_norm, "quantize": _run_quantize, "rope": _run_rope, "product": _run_product}[s["op"]](s)


def _rows8(v):
    """(codes, step) of each row: whole numbers that the definition fixes, as every rounding is one in 32 bits."""
    most = v.abs().amax(-1, keepdim=True)
    factor = torch.full_like(most, 127.0) / most  # one rounding (a number over a tensor would take two)
    factor = torch.where(torch.isinf(factor), 0.0, factor)
    return (v * factor).round().to(torch.int8), (most / 127.0).squeeze(-1)


def _run_norm(s):
    """The norm's 8-bit codes do not depend on the norm (a factor of the whole row), so they are held to equality."""
    if own:
        if s["eight"]:
            y = _qr().qr_rms_norm_q8(s["x"], s["weight"], EPS, residual=s["res"], residual_out=s["res_out"])
            out = {"codes": y.codes, "scales": y.scales}
        else:
            out = {"y": _qr().qr_rms_norm(s["x"], s["weight"], EPS, residual=s["res"], residual_out=s["res_out"])}
        return {**out, "residual": s["res_out"]} if s["residual"] else out
    h = s["x"].float()
    out = {}
    if s["residual"]:
        h = h + s["res"].float()
        out["residual"] = h.to(s["x"].dtype)
    r = torch.rsqrt(h.square().mean(-1) + EPS)
    if s["eight"]:
        out["codes"], step = _rows8(h * s["weight"].float())
        out["scales"] = step * r
    else:
        out["y"] = (h * r[:, None] * s["weight"].float()).to(s["x"].dtype)
    return out


def _run_quantize(s):
    if own:
        y = _qr().qr_q8_quantize(s["x"])
        return {"codes": y.codes, "scales": y.scales}
    codes, step = _rows8(s["x"].float())
    return {"codes": codes, "scales": step}


def _run_rope(s):
    if own:
        q, k = _qr().qr_rope(s["q"], s["k"], s["table"], s["positions"])
        return {"q": q, "k": k}
    angle = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = (angle.cos().float() * s["factor"])[:, None], (angle.sin().float() * s["factor"])[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        turned = x[..., :s["rot"]]
        if s["layout"] == "half":
            a, b = turned.chunk(2, -1)
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        out[name] = torch.cat((turned, x[..., s["rot"]:]), -1).to(s[name].dtype)
    return out


def _run_product(s):
    if own:
        return _qr().qr_w8_matmul(s["rows8"], s["weight"], DTYPES[s["dtype"]], workspace=s["workspace"])
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    return (y * s["x_scales"][:, None] * s["w_scales"]).to(DTYPES[s["dtype"]])


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        total = s["x"].double() @ s["w"].double().T
        return total * torch.outer(s["x_scales"].double(), s["w_scales"].double())
    if case["op"] == "quantize":
        return {"codes": None, "scales": s["x"].double().abs().max(1).values / 127}
    if case["op"] == "norm":
        out = {}
        h = s["x"].double()
        if case["residual"]:
            h += s["res"].double()
            out["residual"] = h
        root = torch.sqrt(torch.einsum("tc,tc->t", h, h) / case["cols"] + EPS)
        if case["eight"]:
            out["codes"] = None
            out["scales"] = (h * s["weight"].double()).abs().max(1).values / (127 * root)
        else:
            out["y"] = h / root[:, None] * s["weight"].double()
        return out
    # a rotated pair as a complex number times e^(i angle)
    angle = torch.outer(s["positions"].double(), s["frequencies"])
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
    out, rot = {}, case["rot"]
    for name in ("q", "k"):
        y = s[name].double().contiguous()
        first, second = ((y[..., :rot // 2], y[..., rot // 2:rot]) if case["layout"] == "half"
                         else (y[..., 0:rot:2], y[..., 1:rot:2]))
        z = torch.complex(first.contiguous(), second.contiguous()) * turn
        first.copy_(z.real)
        second.copy_(z.imag)
        out[name] = y
    return out
