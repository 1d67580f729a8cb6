"""Calls of the framework's language-model operators, each beside its plain form.

The operators are the ones around the looped einsums in a feed-forward layer: the
root-mean-square norm of the residual stream (with the 8-bit output that the next
product reads, and its backward pass), the quantisation of a matrix into e4m3 blocks
with power-of-two scales, the product of two such matrices, and the products of rows
that are grouped by expert (forward, and both gradients).

`run` is one pass: with `own` false in elementary torch operations in 32 bits, with
`own` true through the framework.  `exact` gives the same outputs from the
definitions in 64 bits.
"""

import functools
import math

import torch

own = False

BLOCK = 128           # columns (and, for weights, rows) that share a scale
TOP = 448.0           # largest finite e4m3 value
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # the norm before a layer's products while a few sequences generate
        dict(name="norm_decode", op="norm", rows=8, cols=4096, x="bf16", out="e4m3", residual=True, pad=0),
        # the same for a prompt, at the hidden size of the GPT-3 feed-forward workload
        dict(name="norm_prefill", op="norm", rows=8192, cols=12288, x="bf16", out="e4m3", residual=True, pad=0),
        # a 32-bit run with an odd width inside wider rows, no residual
        dict(name="norm_odd", op="norm", rows=1537, cols=5005, x="f32", out="f32", residual=False, pad=8),
        # the norm's gradients in a training step, with the residual stream's own gradient added
        dict(name="norm_train", op="norm_backward", rows=8192, cols=12288, x="bf16", residual=True, pad=0),
        # activations after GELU, on their way into the second product
        dict(name="quantize_activations", op="quantize", rows=8192, cols=6144, x="bf16", block_rows=1, pad=0),
        # a weight matrix of odd extents, once per update
        dict(name="quantize_weights", op="quantize", rows=4001, cols=2056, x="f32", block_rows=128, pad=24),
        # the second product of the layer while a few sequences generate: the weights are read once
        dict(name="product_decode", op="product8", m=4, n=12288, k=6144, out="bf16", gelu=False, pad=0),
        # a ragged batch through a small projection, 32-bit result
        dict(name="product_odd", op="product8", m=333, n=1000, k=2064, out="f32", gelu=False, pad=16),
        # the first product with GELU for a prompt, GPT-3 feed-forward sizes
        dict(name="product_prefill", op="product8", m=8192, n=6144, k=12288, out="bf16", gelu=True, pad=0),
        # a few tokens, most experts empty: the weights of the touched ones are read
        dict(name="experts_decode", op="experts", rows=16, experts=32, n=4096, k=2048, out="bf16", skew=2.0, pad=0),
        # a prompt's rows over the experts, unevenly
        dict(name="experts_prefill", op="experts", rows=16384, experts=16, n=4096, k=4096, out="bf16", skew=1.0, pad=0),
        # gradients of the rows and of the experts' weights
        dict(name="experts_train", op="experts_backward", rows=8191, experts=8, n=4096, k=4096, out="f32", skew=1.0, pad=0),
    ]


def _log(rng, low, high, step=1):
    """A size spread over the logarithm of [low, high], a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(low, v // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "quantize", "product8", "product8", "experts",
                     "experts_backward"])
    pad = rng.choice([0, 0, 8, 40])
    if op in ("norm", "norm_backward"):
        cols = _log(rng, 64, 12288)
        case = dict(op=op, rows=_log(rng, 1, 60_000_000 // cols), cols=cols, x=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.6, pad=pad)
        if op == "norm":
            case["out"] = rng.choice(["e4m3", "e4m3", case["x"]])
        return case
    if op == "quantize":
        cols = _log(rng, 32, 16384)
        return dict(op=op, rows=_log(rng, 1, 60_000_000 // cols), cols=cols, x=rng.choice(["bf16", "f32"]),
                    block_rows=rng.choice([1, 128]), pad=pad)
    if op == "product8":
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, 12288), _log(rng, 128, 12288, 16)
        while m * n * k > 300_000_000_000:
            m //= 2
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["bf16", "f32"]), gelu=rng.random() < 0.3, pad=2 * pad)
    rows, n, k = _log(rng, 1, 16384), _log(rng, 64, 4096, 8), _log(rng, 64, 4096, 8)
    if op == "experts_backward":
        rows = max(1, rows // 2)
    return dict(op=op, rows=rows, experts=_log(rng, 1, 64), n=n, k=k, out=rng.choice(["bf16", "f32"]),
                skew=round(rng.uniform(0.0, 2.0), 2), pad=pad)


# ---- sizes ------------------------------------------------------------------
def _up(v, step):
    return -(-v // step) * step


def _matrix(rows, cols, pad, dtype, step=8):
    """An empty [rows, cols] matrix whose rows are `step`-aligned and `pad` longer than they need be."""
    return torch.empty((rows, _up(cols, step) + _up(pad, step)), device="cuda", dtype=dtype)[:, :cols]


def _segments(case):
    """Rows of each expert: uneven with `skew`, some of them none."""
    weights = [(1.0 + (7 * e) % case["experts"]) ** -case["skew"] for e in range(case["experts"])]
    total, counts, left = sum(weights), [], case["rows"]
    for w in weights:
        c = min(left, int(case["rows"] * w / total))
        counts.append(c)
        left -= c
    counts[0] += left
    return counts


def work(case):
    op = case["op"]
    if op == "norm":
        e, s = case["rows"] * case["cols"], SIZE[case["x"]]
        n = e * s * (3 if case["residual"] else 1) + e * SIZE[case["out"]] + case["cols"] * s
        if case["out"] == "e4m3":
            n += case["rows"] * _up(case["cols"], BLOCK) // BLOCK
        return {"bytes": n, "flops": 5 * e}
    if op == "norm_backward":
        e, s = case["rows"] * case["cols"], SIZE[case["x"]]
        return {"bytes": e * s * (4 if case["residual"] else 3) + case["cols"] * (s + 4), "flops": 12 * e}
    if op == "quantize":
        e = case["rows"] * case["cols"]
        blocks = -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // BLOCK)
        return {"bytes": e * (SIZE[case["x"]] + 1) + blocks, "flops": 3 * e}
    if op == "product8":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": (m + n) * k + m * n * SIZE[case["out"]] + m * kb + -(-n // BLOCK) * kb,
                "flops": 2 * m * n * k}
    t, n, k = case["rows"], case["n"], case["k"]
    used = sum(c > 0 for c in _segments(case))
    if op == "experts":
        return {"bytes": 2 * t * k + 2 * used * n * k + t * n * SIZE[case["out"]] + 8 * case["experts"],
                "flops": 2 * t * n * k}
    return {"bytes": 2 * (t * n + t * k + used * n * k) + SIZE[case["out"]] * (t * k + case["experts"] * n * k),
            "flops": 4 * t * n * k}


# ---- inputs -----------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(rows, cols, std, dtype, step=8):
        m = _matrix(rows, cols, case["pad"], dtype, step)
        m.copy_(torch.randn((rows, cols), generator=g, device="cuda").mul_(std))
        return m

    def activations(rows, cols, dtype):
        """Normal values of uneven rows, with a few channels far larger than the others."""
        v = torch.randn((rows, cols), generator=g, device="cuda")
        v *= torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
        v *= torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.004, 30.0, 1.0)
        m = _matrix(rows, cols, case["pad"], dtype)
        m.copy_(v)
        return m

    op, pad, s = case["op"], case["pad"], {"case": case}
    if op in ("norm", "norm_backward"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["x"]]
        s["x"] = activations(rows, cols, dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dt)
        if op == "norm":
            if case["residual"]:
                s["residual"] = activations(rows, cols, dt)
                s["residual_out"] = _matrix(rows, cols, pad, dt)
            s["out"] = _matrix(rows, cols, pad, DTYPES[case["out"]], 16)
            if case["out"] == "e4m3":
                s["scales"] = torch.empty((rows, -(-cols // BLOCK)), device="cuda", dtype=torch.float8_e8m0fnu)
        else:
            s["dout"] = normal(rows, cols, 0.5, dt)
            if case["residual"]:
                s["dresidual"] = normal(rows, cols, 0.5, dt)
            s["dx"] = _matrix(rows, cols, pad, dt)
            s["dweight"] = torch.empty(cols, device="cuda")
    elif op == "quantize":
        rows, cols = case["rows"], case["cols"]
        s["x"] = activations(rows, cols, DTYPES[case["x"]])
        s["q"] = _matrix(rows, cols, pad, torch.float8_e4m3fn, 16)
        s["scales"] = torch.empty((-(-rows // case["block_rows"]), -(-cols // BLOCK)), device="cuda",
                                  dtype=torch.float8_e8m0fnu)
    elif op == "product8":
        m, n, k = case["m"], case["n"], case["k"]
        for name, rows, block_rows, x in (("a", m, 1, activations(m, k, torch.float32)),
                                          ("b", n, BLOCK, normal(n, k, 0.05, torch.float32))):
            q, s[name + "_scales"] = _quantize(x, block_rows)
            s[name] = _matrix(rows, k, pad, torch.float8_e4m3fn, 16)
            s[name].copy_(q)
        s["c"] = _matrix(m, n, pad, DTYPES[case["out"]])
    else:
        t, n, k, experts = case["rows"], case["n"], case["k"], case["experts"]
        s["counts"] = _segments(case)
        s["offsets"] = torch.tensor([0] + s["counts"], device="cuda").cumsum(0)
        s["a"] = normal(t, k, 1.0, torch.bfloat16)
        s["b"] = torch.empty((experts, n, _up(k, 8) + pad), device="cuda", dtype=torch.bfloat16)[:, :, :k]
        for e in range(experts):
            s["b"][e].copy_(torch.randn((n, k), generator=g, device="cuda").mul_(0.05))
        if op == "experts":
            s["c"] = _matrix(t, n, pad, DTYPES[case["out"]])
        else:
            s["dc"] = normal(t, n, 0.5, torch.bfloat16)
            s["da"] = _matrix(t, k, pad, DTYPES[case["out"]])
            s["db"] = torch.empty((experts, n, k), device="cuda", dtype=DTYPES[case["out"]])
    return s


# ---- the framework's calls ----------------------------------------------------
@functools.lru_cache(maxsize=None)
def _context():
    import collective_overlap_amd as cce
    return cce, cce.Context(torch.cuda.current_device())


def _run_own(s):
    cce, ctx = _context()
    case = s["case"]
    op = case["op"]
    if op == "norm":
        cce.cce_rmsnorm(ctx, s["x"], s["weight"], s["out"], EPS, residual=s.get("residual"),
                        residual_out=s.get("residual_out"), scales=s.get("scales"))
        return {k: s[k] for k in ("out", "residual_out", "scales") if k in s}
    if op == "norm_backward":
        cce.cce_rmsnorm_backward(ctx, s["x"], s["weight"], s["dout"], s["dx"], s["dweight"], EPS,
                                 d_residual=s.get("dresidual"))
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "quantize":
        cce.cce_quantize_blocks(ctx, s["x"], s["q"], s["scales"], block_rows=case["block_rows"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "product8":
        cce.cce_block_scaled_gemm(ctx, s["a"], s["a_scales"], s["b"], s["b_scales"], s["c"], gelu=case["gelu"])
        return {"c": s["c"]}
    if op == "experts":
        cce.cce_ragged_gemm(ctx, s["a"], s["b"], s["offsets"], s["c"])
        return {"c": s["c"]}
    cce.cce_ragged_gemm_dgrad(ctx, s["dc"], s["b"], s["offsets"], s["da"])
    cce.cce_ragged_gemm_wgrad(ctx, s["dc"], s["a"], s["offsets"], s["db"])
    return {"da": s["da"], "db": s["db"]}


# ---- the plain forms ------------------------------------------------------------
def _blocks(x, block_rows):
    """x, padded with zeros, as [row blocks, block_rows, column blocks, 128]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % block_rows))
    return x.reshape(x.shape[0] // block_rows, block_rows, -1, BLOCK)


def _quantize(x, block_rows):
    """e4m3 values and power-of-two scales of 32-bit x: the smallest 2^e, e >= -126, that brings a block's
    largest magnitude to 448 or below."""
    rows, cols = x.shape
    b = _blocks(x, block_rows)
    mantissa, exponent = torch.frexp(b.abs().amax((1, 3)))
    e = (exponent - 9 + (mantissa > 0.875)).clamp(min=-126).to(torch.int32)
    q = b * ((127 - e) << 23).view(torch.float32)[:, None, :, None]
    q = q.reshape(b.shape[0] * block_rows, -1)[:rows, :cols].to(torch.float8_e4m3fn)
    return q, ((127 + e) << 23).view(torch.float32).to(torch.float8_e8m0fnu)


def _dequantize(q, scales, block_rows):
    b = _blocks(q.float(), block_rows)
    return (b * scales.float()[:, None, :, None]).reshape(b.shape[0] * block_rows, -1)[: q.shape[0], : q.shape[1]]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        r, got = s["x"], {}
        if case["residual"]:
            r = got["residual_out"] = (s["x"].float() + s["residual"].float()).to(r.dtype)
        r = r.float()
        y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["weight"].float()
        if case["out"] == "e4m3":
            got["out"], got["scales"] = _quantize(y, 1)
        else:
            got["out"] = y.to(DTYPES[case["out"]])
        return got
    if op == "norm_backward":
        r, dy = s["x"].float(), s["dout"].float()
        n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
        dn = dy * s["weight"].float()
        dx = (dn - n * (dn * n).mean(1, keepdim=True)) * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
        if case["residual"]:
            dx = dx + s["dresidual"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0)}
    if op == "quantize":
        q, scales = _quantize(s["x"].float(), case["block_rows"])
        return {"q": q, "scales": scales}
    if op == "product8":
        c = _dequantize(s["a"], s["a_scales"], 1) @ _dequantize(s["b"], s["b_scales"], BLOCK).t()
        if case["gelu"]:
            c = 0.5 * c * (1.0 + torch.erf(c * math.sqrt(0.5)))
        return {"c": c.to(DTYPES[case["out"]])}
    out = DTYPES[case["out"]]
    if op == "experts":
        parts = [a.float() @ w.float().t() for a, w in zip(s["a"].split(s["counts"]), s["b"])]
        return {"c": torch.cat(parts).to(out)}
    rows = list(zip(s["dc"].split(s["counts"]), s["a"].split(s["counts"]), s["b"]))
    return {"da": torch.cat([d.float() @ w.float() for d, a, w in rows]).to(out),
            "db": torch.stack([d.float().t() @ a.float() for d, a, w in rows]).to(out)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definitions in 64 bits ---------------------------------------------------
def _exact_quantize(y, block_rows):
    rows, cols = y.shape
    scales = torch.ones((-(-rows // block_rows), -(-cols // BLOCK)), device=y.device, dtype=torch.float64)
    for j in range(scales.shape[1]):
        top = y[:, j * BLOCK:(j + 1) * BLOCK].abs().amax(1)
        top = torch.nn.functional.pad(top, (0, -rows % block_rows)).reshape(-1, block_rows).amax(1)
        e = torch.ceil(torch.log2(top / TOP)).clamp(min=-126)
        e = torch.where(top > TOP * torch.exp2(e), e + 1, e)           # log2 one step off, either way
        e = torch.where((top <= TOP * torch.exp2(e - 1)) & (e > -126), e - 1, e)
        scales[:, j] = torch.exp2(e)
    wide = scales.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]
    return (y / wide).to(torch.float8_e4m3fn), scales.float().to(torch.float8_e8m0fnu)


def _exact_wide(q, scales, block_rows):
    wide = scales.float().double().repeat_interleave(block_rows, 0)[: q.shape[0]]
    return q.float().double() * wide.repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        x, w, got = s["x"].double(), s["weight"].double(), {}
        if op == "norm":
            if case["residual"]:
                got["residual_out"] = (x + s["residual"].double()).to(s["x"].dtype)
                x = got["residual_out"].double()
            y = x / torch.sqrt(x.square().sum(1, keepdim=True) / case["cols"] + EPS) * w
            if case["out"] == "e4m3":
                got["out"], got["scales"] = _exact_quantize(y, 1)
            else:
                got["out"] = y
            return got
        root = torch.sqrt(x.square().sum(1, keepdim=True) / case["cols"] + EPS)
        d = s["dout"].double()
        inner = (d * w * x).sum(1, keepdim=True) / case["cols"]
        dx = d * w / root - x * inner / root ** 3
        if case["residual"]:
            dx = dx + s["dresidual"].double()
        return {"dx": dx, "dweight": (d * x / root).sum(0)}
    if op == "quantize":
        q, scales = _exact_quantize(s["x"].double(), case["block_rows"])
        return {"q": q, "scales": scales}
    if op == "product8":
        c = _exact_wide(s["a"], s["a_scales"], 1) @ _exact_wide(s["b"], s["b_scales"], BLOCK).t().contiguous()
        return {"c": torch.special.ndtr(c) * c if case["gelu"] else c}
    at, c, da, db = 0, [], [], []
    for e, count in enumerate(s["counts"]):
        a, w = s["a"][at:at + count].double(), s["b"][e].double()
        if op == "experts":
            c.append(a @ w.t().contiguous())
        else:
            d = s["dc"][at:at + count].double()
            da.append(d @ w)
            db.append(d.t().contiguous() @ a)
        at += count
    return {"c": torch.cat(c)} if op == "experts" else {"da": torch.cat(da), "db": torch.stack(db)}
