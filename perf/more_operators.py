"""Cases for measuring the operators of an 8-bit floating-point projection and the layer norm in front
of it: the quantizer to E4M3 with one fp32 scale for each block of 128, the matrix product of two such
operands, and the layer norm with its gradients.

``run`` computes each operator either in a plain form (elementary torch operations in fp32, rounded
once at the end; ``own`` false) or through the library's entry points (``own`` true), on the inputs
that ``prepare`` makes.  ``exact`` is the operators' definition in fp64, written apart from both.

Row and column counts are those of the package's synthetic workloads (hidden 2048 / ffn 5632 and
1408 / hidden 7168; 8192 and 16384 tokens) or generic ones.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128              # elements of a row that share a scale (and rows, of a square block)
QMAX = 448.0             # E4M3's largest value
LEAST = 2.0 ** -126      # least scale
EPS = 1e-5


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the activations of a few tokens before a projection: launch latency
        dict(name="quantize 7x2048", op="quantize", rows=7, cols=2048, x="bf16", block=1, row=True, col=False),
        # an fp32 gradient from a DGRAD product: along its rows for DGRAD, transposed for WGRAD
        dict(name="quantize 8192x5632 f32 both", op="quantize", rows=8192, cols=5632, x="f32", block=1, row=True, col=True),
        # the weights of the large configuration, once a step, for FPROP and DGRAD
        dict(name="quantize 7168x7168 square both", op="quantize", rows=7168, cols=7168, x="bf16", block=128, row=True,
             col=True),
        # FPROP of one token: the weights are read once
        dict(name="product 1x7168x7168", op="product", m=1, n=7168, k=7168, a_block=1, b_block=128, out="bf16"),
        # a few tokens of one expert, an odd number of them
        dict(name="product 37x2816x2048", op="product", m=37, n=2816, k=2048, a_block=1, b_block=128, out="bf16"),
        # FPROP of the dense configuration
        dict(name="product 8192x5632x2048", op="product", m=8192, n=5632, k=2048, a_block=1, b_block=128, out="bf16"),
        # WGRAD of one expert: a ragged number of tokens is the summed index, both operands have scales along it
        dict(name="product 1408x2048x4109 f32", op="product", m=1408, n=2048, k=4109, a_block=1, b_block=1, out="f32"),
        # FPROP of the large configuration
        dict(name="product 16384x7168x7168", op="product", m=16384, n=7168, k=7168, a_block=1, b_block=128, out="bf16"),
        # a handful of tokens through the norm of the hidden stream
        dict(name="layer norm 5x2048", op="norm", rows=5, cols=2048, x="bf16", residual=True, beta=True),
        # the norm after a down projection of the large configuration: fp32 product plus the bf16 stream
        dict(name="layer norm 16384x7168 f32", op="norm", rows=16384, cols=7168, x="f32", residual=True, beta=True),
        # the same, backward: bf16 gradient, with the stream's own gradient added
        dict(name="layer norm back 8192x2048", op="norm_back", rows=8192, cols=2048, dy="bf16", x="bf16", dtotal=True),
        # an odd row count and width, fp32 gradient from a DGRAD product
        dict(name="layer norm back 3001x5000 f32", op="norm_back", rows=3001, cols=5000, dy="f32", x="bf16", dtotal=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "norm", "norm_back"])
    if op == "product":
        m, n, k = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            n, k = max(128, n // 128 * 128), max(128, k // 128 * 128)
        a_block, b_block = rng.choice([(1, 128), (1, 128), (1, 1), (128, 1), (128, 128)])
        while 1.0 * m * n * k > 8.4e11:
            m = m // 2 + 1
        return dict(op=op, m=m, n=n, k=k, a_block=a_block, b_block=b_block, out=rng.choice(["bf16", "f32"]))
    rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 64, 7168)
    if rng.random() < 0.7:
        cols = max(64, cols // 32 * 32)
    kind = rng.choice(["bf16", "f32"])
    if op == "quantize":
        row, col = rng.choice([(True, False), (True, True), (True, True), (False, True)])
        return dict(op=op, rows=rows, cols=cols, x=kind, block=rng.choice([1, 1, 128]), row=row, col=col)
    if op == "norm":
        return dict(op=op, rows=rows, cols=cols, x=kind, residual=rng.random() < 0.7, beta=rng.random() < 0.8)
    return dict(op=op, rows=rows, cols=cols, dy=kind, x=rng.choice(["bf16", "bf16", "f32"]), dtotal=rng.random() < 0.7)


# ----------------------------------------------------------------------------------- inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(gen, rows, cols, std=1.0):
    """N(0, std^2) with one element in a thousand fifty times larger."""
    x = torch.randn((rows, cols), generator=gen, device=DEV) * std
    big = torch.rand((rows, cols), generator=gen, device=DEV) < 1e-3
    return torch.where(big, 50.0 * x, x)


def _gradients(gen, rows, cols):
    """Heavy-tailed values around 1e-3: a normal over the root of a mean of squares."""
    x = torch.randn((rows, cols), generator=gen, device=DEV) * 1e-3
    return x * torch.rand((rows, cols), generator=gen, device=DEV).clamp_min(1e-2).rsqrt()


def _stream(gen, rows, cols):
    """A hidden stream: activations of a scale and an offset of their own in each row."""
    scale = 0.5 + 3.0 * torch.rand((rows, 1), generator=gen, device=DEV)
    return (_activations(gen, rows, cols) + torch.randn((rows, 1), generator=gen, device=DEV)) * scale


def _pitch(cols):
    """Bytes between rows of codes: the columns rounded up to 16."""
    return (cols + 15) // 16 * 16


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        # both operands along the summed index, as the quantizer leaves them; the weight of an FPROP, or two WGRAD operands
        a = _activations(gen, m, k)
        b = torch.randn((n, k), generator=gen, device=DEV) * 0.02 if case["b_block"] == 128 else _gradients(gen, n, k)
        for name, v, block in (("a", a, case["a_block"]), ("b", b, case["b_block"])):
            codes, s[name + "_scales"] = _quantized(v, block)
            pitched = torch.zeros((v.shape[0], _pitch(k)), dtype=torch.uint8, device=DEV)
            pitched[:, :k] = codes
            s[name + "_codes"] = pitched[:, :k]
        return s
    rows, cols = case["rows"], case["cols"]
    if op == "quantize":
        if case["block"] == 128:
            x = torch.randn((rows, cols), generator=gen, device=DEV) * 0.02
        else:
            x = _gradients(gen, rows, cols) if case["x"] == "f32" else _activations(gen, rows, cols)
        s["x"] = x.to(_dtype(case["x"]))
    elif op == "norm":
        s["x"] = _stream(gen, rows, cols).to(_dtype(case["x"]))
        s["residual"] = _activations(gen, rows, cols, 2.0).bfloat16() if case["residual"] else None
        s["gamma"] = (1.0 + 0.1 * torch.randn((cols,), generator=gen, device=DEV)).bfloat16()
        s["beta"] = (0.1 * torch.randn((cols,), generator=gen, device=DEV)).bfloat16() if case["beta"] else None
    else:
        s["x"] = _stream(gen, rows, cols).to(_dtype(case["x"]))
        v = s["x"].float()
        s["mean"] = v.mean(1)
        s["rstd"] = ((v - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
        s["gamma"] = (1.0 + 0.1 * torch.randn((cols,), generator=gen, device=DEV)).bfloat16()
        s["dy"] = _gradients(gen, rows, cols).to(_dtype(case["dy"]))
        s["dtotal"] = _gradients(gen, rows, cols).bfloat16() if case["dtotal"] else None
    return s


# ------------------------------------------------------------------------------ plain forms
def _blocks(v, block):
    """v, filled up with zeros, as [row blocks, rows, column blocks, columns]."""
    rows, cols = v.shape
    full = v.new_zeros((-(-rows // block) * block, -(-cols // BLOCK) * BLOCK))
    full[:rows, :cols] = v
    return full.view(full.shape[0] // block, block, full.shape[1] // BLOCK, BLOCK)


def _quantized(v, block):
    """E4M3 code bytes and fp32 scales of fp32 rows: scale s = amax / 448 (at least 2^-126) of each block of
    `block` rows and 128 columns, codes v * (1 / s) rounded to nearest even, a zero as +0."""
    rows, cols = v.shape
    b = _blocks(v, block)
    amax = b.abs().amax((1, 3))
    s = (amax / torch.full_like(amax, QMAX)).clamp_min(LEAST)  # a tensor: a number's reciprocal would be multiplied by
    inv = torch.ones_like(s) / s
    t = (b * inv[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    t = torch.where((t & 0x7F) == 0, torch.zeros_like(t), t)
    return t.reshape(b.shape[0] * block, -1)[:rows, :cols].contiguous(), s


def _values(codes):
    """The E4M3 values that code bytes stand for (their scales are outputs of their own)."""
    return codes.view(torch.float8_e4m3fn)


def _plain_quantize(s):
    c, x, out = s["case"], s["x"].float(), {}
    for name, wanted, v in (("row", c["row"], x), ("col", c["col"], x.T)):
        if wanted:
            codes, scales = _quantized(v, c["block"])
            out |= {name + "_codes": _values(codes), name + "_scales": scales}
    return out


def _restored(codes, scales, block):
    rows, cols = codes.shape
    unit = scales.repeat_interleave(block, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]
    return codes.view(torch.float8_e4m3fn).float() * unit


def _plain_product(s):
    c = s["case"]
    a, b = (_restored(s[n + "_codes"], s[n + "_scales"], c[n + "_block"]) for n in "ab")
    return {"d": (a @ b.T).to(_dtype(c["out"]))}


def _plain_norm(s):
    total = s["x"].float()
    if s["residual"] is not None:
        total = total + s["residual"].float()
    mean = total.mean(1)
    d = total - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
    y = d * rstd[:, None] * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    return {"y": y.bfloat16(), "total": total.bfloat16(), "mean": mean, "rstd": rstd}


def _plain_norm_back(s):
    h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    q = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (q - q.mean(1, keepdim=True) - h * (q * h).mean(1, keepdim=True))
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    return {"dx": dx.bfloat16(), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}


# -------------------------------------------------------------------- the library's operators
def _buffers(s):
    """Outputs, operand descriptions and workspaces, made on the first pass and kept, as a training loop keeps them."""
    if "own" in s:
        return s["own"]
    from rht_bit_block_gb300 import ufp4

    c, b = s["case"], {}
    op = c["op"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEV)

    if op == "quantize":
        for name, wanted, shape in (("row", c["row"], (c["rows"], c["cols"])), ("col", c["col"], (c["cols"], c["rows"]))):
            b[name] = None
            if wanted:
                b[name + "_codes"], b[name + "_scales"] = ufp4.alloc_fp8(*shape, c["block"], DEV)
                b[name] = ufp4.qtensor(b[name + "_codes"], b[name + "_scales"], *shape)
    elif op == "product":
        b["d"] = empty((c["m"], c["n"]), _dtype(c["out"]))
        b["a"] = ufp4.qtensor(s["a_codes"], s["a_scales"], c["m"], c["k"])
        b["b"] = ufp4.qtensor(s["b_codes"], s["b_scales"], c["n"], c["k"])
    elif op == "norm":
        rows, cols = c["rows"], c["cols"]
        b["y"], b["total"] = empty((rows, cols), torch.bfloat16), empty((rows, cols), torch.bfloat16)
        b["mean"], b["rstd"] = empty((rows,), torch.float32), empty((rows,), torch.float32)
    else:
        rows, cols = c["rows"], c["cols"]
        b["dx"] = empty((rows, cols), torch.bfloat16)
        b["dgamma"], b["dbeta"] = empty((cols,), torch.float32), empty((cols,), torch.float32)
        b["ws"] = empty((max(1, ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols)),), torch.uint8)
    s["own"] = b
    return b


def _own(s):
    from rht_bit_block_gb300 import ufp4

    c, b = s["case"], _buffers(s)
    op = c["op"]
    if op == "quantize":
        ufp4.ufp4_fp8_quantize(s["x"], b["row"], b["col"], block_rows=c["block"])
        out = {}
        for name in ("row", "col"):
            if c[name]:
                out |= {name + "_codes": _values(b[name + "_codes"]), name + "_scales": b[name + "_scales"]}
        return out
    if op == "product":
        ufp4.ufp4_fp8_gemm(b["a"], b["b"], b["d"], a_block_rows=c["a_block"], b_block_rows=c["b_block"])
        return {"d": b["d"]}
    if op == "norm":
        ufp4.ufp4_layer_norm(s["x"], s["gamma"], b["y"], b["mean"], b["rstd"], beta=s["beta"], residual=s["residual"],
                             total=b["total"], eps=EPS)
        return {"y": b["y"], "total": b["total"], "mean": b["mean"], "rstd": b["rstd"]}
    ufp4.ufp4_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], b["dx"],
                                  b["dgamma"], b["dbeta"], b["ws"], dtotal=s["dtotal"])
    return {"dx": b["dx"], "dgamma": b["dgamma"], "dbeta": b["dbeta"]}


def run(state):
    if own:
        return _own(state)
    plain = {"quantize": _plain_quantize, "product": _plain_product, "norm": _plain_norm, "norm_back": _plain_norm_back}
    return plain[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------- floors
def _scales(rows, cols, block):
    return -(-rows // block) * -(-cols // BLOCK)


def work(case):
    op = case["op"]
    if op == "product":
        m, n, k = 1.0 * case["m"], 1.0 * case["n"], 1.0 * case["k"]
        scales = _scales(case["m"], case["k"], case["a_block"]) + _scales(case["n"], case["k"], case["b_block"])
        return {"bytes": (m + n) * k + 4.0 * scales + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2.0 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    n = 1.0 * rows * cols
    if op == "quantize":
        outputs = (1 if case["row"] else 0) + (1 if case["col"] else 0)
        scales = (_scales(rows, cols, case["block"]) if case["row"] else 0) + \
            (_scales(cols, rows, case["block"]) if case["col"] else 0)
        return {"bytes": n * ((2 if case["x"] == "bf16" else 4) + outputs) + 4.0 * scales, "flops": n * (2 + 2 * outputs)}
    x = 2 if case["x"] == "bf16" else 4
    if op == "norm":
        return {"bytes": n * (x + (2 if case["residual"] else 0) + 4) + 8.0 * rows + cols * (4.0 if case["beta"] else 2.0),
                "flops": 9 * n}
    dy = 2 if case["dy"] == "bf16" else 4
    return {"bytes": n * (x + dy + 2 + (2 if case["dtotal"] else 0)) + 8.0 * rows + 10.0 * cols, "flops": 15 * n}


# ------------------------------------------------------------------- the definition, 64 bits
def _f64_codes(v, block):
    """E4M3 values and fp32 scales of fp64 rows from the number formats themselves: the scale, its reciprocal and the
    scaled value are each one operation rounded to fp32 (by definition); E4M3 has spacing 2^(k-3) for values in
    [2^k, 2^(k+1)), k >= -6, and is rounded half to even."""
    rows, cols = v.shape
    codes = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=v.device)
    scales = torch.empty((-(-rows // block), -(-cols // BLOCK)), dtype=torch.float32, device=v.device)
    for j in range(scales.shape[1]):
        part = v[:, j * BLOCK:(j + 1) * BLOCK]
        top = part.abs().amax(1)
        fill = torch.zeros((scales.shape[0] * block,), dtype=torch.float64, device=v.device)
        fill[:rows] = top
        s = (fill.view(-1, block).amax(1) / QMAX).float().clamp_min(LEAST)
        scales[:, j] = s
        inv = (1.0 / s.double()).float().double().repeat_interleave(block)[:rows, None]
        t = (part * inv).float().double()
        k = torch.frexp(t)[1].long().sub_(1).clamp_min_(-6)
        step = ((k + (1023 - 3)) << 52).view(torch.float64)  # 2^(k-3)
        codes[:, j * BLOCK:(j + 1) * BLOCK] = ((torch.round(t / step) * step) + 0.0).to(torch.float8_e4m3fn)
    return codes, scales


def _f64_operand(codes, scales, block):
    v = codes.view(torch.float8_e4m3fn).double()
    r = torch.arange(v.shape[0], device=v.device) // block
    k = torch.arange(v.shape[1], device=v.device) // BLOCK
    return v * scales.double()[r][:, k]


def exact(case, seed):
    op = case["op"]
    if op == "product" and 2.0 * case["m"] * case["n"] * case["k"] > 6e12:
        return None  # too long in 64 bits
    s = prepare(case, seed)
    if op == "quantize":
        out = {}
        for name, v in (("row", s["x"].double()), ("col", s["x"].double().T)):
            if case[name]:
                codes, scales = _f64_codes(v.contiguous(), case["block"])
                out |= {name + "_codes": codes, name + "_scales": scales}
        return out
    if op == "product":
        return {"d": torch.mm(_f64_operand(s["a_codes"], s["a_scales"], case["a_block"]),
                              _f64_operand(s["b_codes"], s["b_scales"], case["b_block"]).T)}
    if op == "norm":
        total = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
        var, mean = torch.var_mean(total, 1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        y = (total - mean[:, None]) * rstd[:, None] * s["gamma"].double()
        if s["beta"] is not None:
            y = y + s["beta"].double()
        return {"y": y, "total": total, "mean": mean, "rstd": rstd}
    rstd = s["rstd"].double()[:, None]
    centred = s["x"].double() - s["mean"].double()[:, None]
    dy = s["dy"].double()
    g = dy * s["gamma"].double()
    n = case["cols"]
    dx = rstd * g - rstd * (g.sum(1, keepdim=True) / n) - centred * rstd.pow(3) * ((g * centred).sum(1, keepdim=True) / n)
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].double()
    return {"dx": dx, "dgamma": (dy * centred * rstd).sum(0), "dbeta": dy.sum(0)}
