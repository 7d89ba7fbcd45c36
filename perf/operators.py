"""Cases for measuring the operators of a training step that sit between its GEMMs: the residual
RMS norm and the gated activation with their 8-bit activation checkpoints (forward and backward),
and the vocabulary loss with its gradient.

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
BLOCK = 32      # elements that share one checkpoint scale
QMAX = 448.0    # E4M3's largest value
EPS = 1e-6
IGNORED = -100
SILU, GELU = "silu", "gelu"


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of tokens through the norm of the hidden stream: launch latency
        dict(name="norm 5x2048", op="norm", rows=5, cols=2048, x="bf16", residual=True),
        # the norm after a down projection of the large configuration: fp32 GEMM output plus the bf16 stream
        dict(name="norm 16384x7168 f32", op="norm", rows=16384, cols=7168, x="f32", residual=True),
        # the same, backward: bf16 gradient of the head, with the stream's own gradient added
        dict(name="norm back 8192x2048", op="norm_back", rows=8192, cols=2048, dy="bf16", dtotal=True, remake=False),
        # an odd row count and width, fp32 gradient from a DGRAD GEMM, the normalised rows made again for WGRAD
        dict(name="norm back 3001x5000 f32", op="norm_back", rows=3001, cols=5000, dy="f32", dtotal=True, remake=True),
        # tokens of one small expert
        dict(name="glu 37x1408", op="glu", rows=37, cols=1408, x="bf16", act=SILU, packed=True),
        # the dense feed-forward block: gate and up are one fp32 GEMM output
        dict(name="glu 8192x5632 f32", op="glu", rows=8192, cols=5632, x="f32", act=SILU, packed=True),
        # an expert's ragged share of the tokens
        dict(name="glu back 4109x1408", op="glu_back", rows=4109, cols=1408, dy="bf16", act=GELU, packed=True, remake=False),
        # the large configuration, fp32 gradient from a DGRAD GEMM, the activation made again for WGRAD
        dict(name="glu back 16384x7168 f32", op="glu_back", rows=16384, cols=7168, dy="f32", act=SILU, packed=False,
             remake=True),
        # scoring a few tokens: the whole head is read once
        dict(name="loss 16x32000x2048", op="loss", tokens=16, vocab=32000, hidden=2048, ignored=0.0, z=0.0),
        # evaluation of a batch, some prompt tokens ignored
        dict(name="loss 8192x50001x2048", op="loss", tokens=8192, vocab=50001, hidden=2048, ignored=0.1, z=0.0),
        # a fine-tuning step: a third of the tokens are prompt and give no loss
        dict(name="loss step 2047x50001x2048", op="loss_step", tokens=2047, vocab=50001, hidden=2048, ignored=0.33, z=1e-4),
        # a pretraining step of the large configuration
        dict(name="loss step 4096x65536x7168", op="loss_step", tokens=4096, vocab=65536, hidden=7168, ignored=0.0, z=1e-4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "glu", "glu_back", "loss", "loss_step"])
    if op in ("loss", "loss_step"):
        tokens, hidden = _log_int(rng, 1, 8192), 8 * _log_int(rng, 32, 896)
        vocab = _log_int(rng, 1000, 130000)
        most = 1.9e12 / (1.0 if op == "loss" else 2.0)
        while 1.0 * tokens * vocab * hidden > most:
            tokens = tokens // 2 + 1
        return dict(op=op, tokens=tokens, vocab=vocab, hidden=hidden, ignored=rng.choice([0.0, 0.05, 0.5]),
                    z=rng.choice([0.0, 1e-4]))
    rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 64, 7168)
    if rng.random() < 0.7:
        cols = max(64, cols // 32 * 32)
    kind = rng.choice(["bf16", "f32"])
    if op == "norm":
        return dict(op=op, rows=rows, cols=cols, x=kind, residual=rng.random() < 0.7)
    if op == "norm_back":
        return dict(op=op, rows=rows, cols=cols, dy=kind, dtotal=rng.random() < 0.7, remake=rng.random() < 0.5)
    if op == "glu":
        return dict(op=op, rows=rows, cols=cols, x=kind, act=rng.choice([SILU, GELU]), packed=rng.random() < 0.7)
    return dict(op=op, rows=rows, cols=cols, dy=kind, act=rng.choice([SILU, GELU]), packed=rng.random() < 0.5,
                remake=rng.random() < 0.5)


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


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op in ("loss", "loss_step"):
        t, v, k = case["tokens"], case["vocab"], case["hidden"]
        s["h"] = torch.randn((t, k), generator=gen, device=DEV).bfloat16()
        s["w"] = (torch.randn((v, k), generator=gen, device=DEV) * (0.9 / math.sqrt(k))).bfloat16()
        targets = torch.randint(0, v, (t,), generator=gen, device=DEV)
        skip = torch.rand((t,), generator=gen, device=DEV) < case["ignored"]
        s["targets"] = torch.where(skip, torch.full_like(targets, IGNORED), targets)
        if op == "loss_step":
            s["weight"] = 0.5 + torch.rand((t,), generator=gen, device=DEV)
            s["scale"] = torch.full((1,), 1.0 / t, device=DEV)
        return s
    rows, cols = case["rows"], case["cols"]
    if op == "norm":
        s["x"] = _activations(gen, rows, cols).to(_dtype(case["x"]))
        s["residual"] = _activations(gen, rows, cols, 2.0).bfloat16() if case["residual"] else None
        s["gamma"] = (1.0 + 0.1 * torch.randn((cols,), generator=gen, device=DEV)).bfloat16()
    elif op == "norm_back":
        saved = _activations(gen, rows, cols, 2.0)
        s["rstd"] = (saved.square().mean(1) + EPS).rsqrt()
        s["codes"], s["scales"] = _checkpoint(saved)
        s["gamma"] = (1.0 + 0.1 * torch.randn((cols,), generator=gen, device=DEV)).bfloat16()
        s["dy"] = _gradients(gen, rows, cols).to(_dtype(case["dy"]))
        s["dtotal"] = _gradients(gen, rows, cols).bfloat16() if case["dtotal"] else None
    elif op == "glu":
        both = _activations(gen, rows, 2 * cols).to(_dtype(case["x"]))
        s["gate"], s["up"] = both[:, :cols], both[:, cols:]
        if not case["packed"]:
            s["gate"], s["up"] = s["gate"].contiguous(), s["up"].contiguous()
    else:
        s["gate_codes"], s["gate_scales"] = _checkpoint(_activations(gen, rows, cols))
        s["up_codes"], s["up_scales"] = _checkpoint(_activations(gen, rows, cols))
        s["dy"] = _gradients(gen, rows, cols).to(_dtype(case["dy"]))
    return s


# ------------------------------------------------------------------------------ plain forms
def _pow2(e):
    """2^e as fp32, exactly, for whole e in [-127, 127] (2^-127 is subnormal)."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def _checkpoint(v):
    """fp32 rows -> E4M3 code bytes and one E8M0 scale byte per 32: the scale is the least power of
    two 2^e with max |v| <= 448 * 2^e, the codes round v / 2^e to nearest even, a zero is +0."""
    rows, cols = v.shape
    pad = -cols % BLOCK
    b = torch.cat([v, v.new_zeros((rows, pad))], 1).reshape(rows, -1, BLOCK)
    mant, exp = torch.frexp(b.abs().amax(2))
    e = (exp - 9 + (mant > 0.875)).clamp(-127, 127)
    e = torch.where(mant == 0, torch.full_like(e, -127), e)
    t = (b * _pow2(-e).unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8)
    t = torch.where((t & 0x7F) == 0, torch.zeros_like(t), t)
    return t.reshape(rows, -1)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def _restore(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float()
    unit = _pow2(scales.to(torch.int32) - 127)
    return v * unit.repeat_interleave(BLOCK, 1)[:, : v.shape[1]]


def _values(codes):
    """The E4M3 values that checkpoint bytes stand for (their scales are outputs of their own)."""
    return codes.view(torch.float8_e4m3fn)


def _act(g, act):
    """act(g) and its derivative."""
    if act == SILU:
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    c, a = math.sqrt(2.0 / math.pi), 0.044715
    th = torch.tanh(c * (g + a * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * c * (1.0 + 3.0 * a * g * g)


def _plain_norm(s):
    total = s["x"].float()
    if s["residual"] is not None:
        total = total + s["residual"].float()
    rstd = 1.0 / torch.sqrt(total.square().mean(1) + EPS)
    y = total * rstd[:, None] * s["gamma"].float()
    codes, scales = _checkpoint(total)
    return {"y": y.bfloat16(), "total": total.bfloat16(), "rstd": rstd, "codes": _values(codes), "scales": scales}


def _plain_norm_back(s):
    xh = _restore(s["codes"], s["scales"]) * s["rstd"][:, None]
    dy, gamma = s["dy"].float(), s["gamma"].float()
    g = dy * gamma
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    out = {"dx": dx.bfloat16(), "dgamma": (dy * xh).sum(0)}
    if s["case"]["remake"]:
        out["y"] = (xh * gamma).bfloat16()
    return out


def _plain_glu(s):
    g, u = s["gate"].float(), s["up"].float()
    gc, gs = _checkpoint(g)
    uc, us = _checkpoint(u)
    return {"y": (_act(g, s["case"]["act"])[0] * u).bfloat16(), "gate_codes": _values(gc), "gate_scales": gs,
            "up_codes": _values(uc), "up_scales": us}


def _plain_glu_back(s):
    g, u = _restore(s["gate_codes"], s["gate_scales"]), _restore(s["up_codes"], s["up_scales"])
    dy = s["dy"].float()
    a, d = _act(g, s["case"]["act"])
    out = {"dgate": (dy * u * d).bfloat16(), "dup": (dy * a).bfloat16()}
    if s["case"]["remake"]:
        out["y"] = (a * u).bfloat16()
    return out


def _plain_loss(s, step):
    h, w, targets, z = s["h"].float(), s["w"].float(), s["targets"], s["case"]["z"]
    valid = targets >= 0
    at = targets.clamp_min(0)[:, None]
    logits = h @ w.T
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    loss = lse - logits.gather(1, at)[:, 0] + z * lse * lse
    zero = torch.zeros_like(lse)
    out = {"loss": torch.where(valid, loss, zero), "lse": torch.where(valid, lse, zero)}
    if step:
        del logits
        g = torch.where(valid, s["weight"] * s["scale"], zero)[:, None]
        dl = p * ((1.0 + 2.0 * z * lse)[:, None] * g / total)
        dl.scatter_add_(1, at, -g)
        dl = torch.where(valid[:, None], dl, torch.zeros_like(dl))
        out["dh"] = (dl @ w).bfloat16()
        out["dw"] = (dl.T @ torch.where(valid[:, None], h, torch.zeros_like(h))).bfloat16()
    return out


# -------------------------------------------------------------------- the library's operators
def _buffers(s):
    """Outputs, checkpoint descriptions and workspaces, made on the first pass and kept, as a training loop keeps them."""
    if "own" in s:
        return s["own"]
    from rht_bit_block_gb300 import ufp4

    c, b = s["case"], {}
    op = c["op"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEV)

    if op in ("loss", "loss_step"):
        t, v, k = c["tokens"], c["vocab"], c["hidden"]
        b["loss"], b["lse"] = empty((t,), torch.float32), empty((t,), torch.float32)
        need = ufp4.ufp4_head_loss_workspace_size(t, v, k)
        if op == "loss_step":
            b["dh"], b["dw"] = empty((t, k), torch.bfloat16), empty((v, k), torch.bfloat16)
            need = max(need, ufp4.ufp4_head_loss_backward_workspace_size(t, v, k))
        b["ws"] = empty((max(1, need),), torch.uint8)
    elif op == "norm":
        rows, cols = c["rows"], c["cols"]
        b["y"], b["total"] = empty((rows, cols), torch.bfloat16), empty((rows, cols), torch.bfloat16)
        b["rstd"] = empty((rows,), torch.float32)
        b["codes"], b["scales"] = ufp4.alloc_checkpoint(rows, cols, DEV)
        b["ckpt"] = ufp4.qtensor(b["codes"], b["scales"], rows, cols)
    elif op == "norm_back":
        rows, cols = c["rows"], c["cols"]
        b["dx"], b["dgamma"] = empty((rows, cols), torch.bfloat16), empty((cols,), torch.float32)
        b["y"] = empty((rows, cols), torch.bfloat16) if c["remake"] else None
        b["ckpt"] = ufp4.qtensor(s["codes"], s["scales"], rows, cols)
        b["ws"] = empty((max(1, ufp4.ufp4_rms_norm_backward_workspace_size(rows, cols)),), torch.uint8)
    elif op == "glu":
        rows, cols = c["rows"], c["cols"]
        b["y"] = empty((rows, cols), torch.bfloat16)
        for name in ("gate", "up"):
            b[name + "_codes"], b[name + "_scales"] = ufp4.alloc_checkpoint(rows, cols, DEV)
            b[name] = ufp4.qtensor(b[name + "_codes"], b[name + "_scales"], rows, cols)
    else:
        rows, cols = c["rows"], c["cols"]
        both = empty((rows, 2 * cols), torch.bfloat16)
        b["dgate"], b["dup"] = both[:, :cols], both[:, cols:]
        if not c["packed"]:
            b["dgate"], b["dup"] = empty((rows, cols), torch.bfloat16), empty((rows, cols), torch.bfloat16)
        b["y"] = empty((rows, cols), torch.bfloat16) if c["remake"] else None
        b["gate"] = ufp4.qtensor(s["gate_codes"], s["gate_scales"], rows, cols)
        b["up"] = ufp4.qtensor(s["up_codes"], s["up_scales"], rows, cols)
    s["own"] = b
    return b


def _own(s):
    from rht_bit_block_gb300 import ufp4

    c, b = s["case"], _buffers(s)
    op = c["op"]
    if op == "norm":
        ufp4.ufp4_rms_norm(s["x"], s["gamma"], b["y"], b["rstd"], residual=s["residual"], total=b["total"],
                           ckpt=b["ckpt"], eps=EPS)
        return {"y": b["y"], "total": b["total"], "rstd": b["rstd"], "codes": _values(b["codes"]), "scales": b["scales"]}
    if op == "norm_back":
        ufp4.ufp4_rms_norm_backward(s["dy"], b["ckpt"], s["rstd"], s["gamma"], b["dx"], b["dgamma"], b["ws"],
                                    dtotal=s["dtotal"], y=b["y"])
        out = {"dx": b["dx"], "dgamma": b["dgamma"]}
        return {**out, "y": b["y"]} if c["remake"] else out
    if op == "glu":
        ufp4.ufp4_glu(s["gate"], s["up"], b["y"], act=c["act"], ckpt_gate=b["gate"], ckpt_up=b["up"])
        return {"y": b["y"], "gate_codes": _values(b["gate_codes"]), "gate_scales": b["gate_scales"],
                "up_codes": _values(b["up_codes"]), "up_scales": b["up_scales"]}
    if op == "glu_back":
        ufp4.ufp4_glu_backward(s["dy"], b["gate"], b["up"], b["dgate"], b["dup"], act=c["act"], y=b["y"])
        out = {"dgate": b["dgate"], "dup": b["dup"]}
        return {**out, "y": b["y"]} if c["remake"] else out
    ufp4.ufp4_head_loss(s["h"], s["w"], s["targets"], b["loss"], b["lse"], b["ws"], z_loss=c["z"])
    out = {"loss": b["loss"], "lse": b["lse"]}
    if op == "loss_step":
        ufp4.ufp4_head_loss_backward(s["h"], s["w"], s["targets"], b["lse"], b["dh"], b["dw"], b["ws"],
                                     token_weight=s["weight"], scale=s["scale"], z_loss=c["z"])
        out |= {"dh": b["dh"], "dw": b["dw"]}
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_back":
        return _plain_norm_back(state)
    if op == "glu":
        return _plain_glu(state)
    if op == "glu_back":
        return _plain_glu_back(state)
    return _plain_loss(state, op == "loss_step")


# ----------------------------------------------------------------------------------- floors
def work(case):
    op = case["op"]
    if op in ("loss", "loss_step"):
        t, v, k = case["tokens"], case["vocab"], case["hidden"]
        valid = t * (1.0 - case["ignored"])  # ignored tokens need no logits
        if op == "loss":
            return {"bytes": 2.0 * k * (valid + v) + 16.0 * t, "flops": 2.0 * valid * v * k}
        return {"bytes": 4.0 * k * (t + v) + 20.0 * t, "flops": 6.0 * valid * v * k}
    n, rows = 1.0 * case["rows"] * case["cols"], 1.0 * case["rows"]
    ckpt = n + rows * math.ceil(case["cols"] / BLOCK)
    if op == "norm":
        x = 2 if case["x"] == "bf16" else 4
        return {"bytes": n * (x + (2 if case["residual"] else 0) + 4) + ckpt + 4 * rows + 2 * case["cols"], "flops": 8 * n}
    if op == "norm_back":
        dy = 2 if case["dy"] == "bf16" else 4
        extra = (2 if case["dtotal"] else 0) + (2 if case["remake"] else 0)
        return {"bytes": n * (dy + 2 + extra) + ckpt + 4 * rows + 6 * case["cols"], "flops": 12 * n}
    if op == "glu":
        return {"bytes": n * (2 * (2 if case["x"] == "bf16" else 4) + 2) + 2 * ckpt, "flops": 14 * n}
    dy = 2 if case["dy"] == "bf16" else 4
    return {"bytes": n * (dy + 4 + (2 if case["remake"] else 0)) + 2 * ckpt, "flops": 18 * n}


# ------------------------------------------------------------------- the definition, 64 bits
def _f64_codes(v):
    """E4M3 values and E8M0 bytes of fp64 rows from the number format itself: spacing 2^(k-3) for
    values in [2^k, 2^(k+1)), k >= -6, rounded half to even."""
    rows, cols = v.shape
    nb = (cols + BLOCK - 1) // BLOCK
    pad = torch.zeros((rows, nb * BLOCK), dtype=torch.float64, device=v.device)
    pad[:, :cols] = v
    b = pad.view(rows, nb, BLOCK)
    m = b.abs().amax(2)
    e = torch.ceil(torch.log2(m.clamp_min(1e-300) / QMAX))
    e = torch.where(QMAX * torch.pow(2.0, e - 1) >= m, e - 1, e)  # log2 may be a rounding off
    e = torch.where(QMAX * torch.pow(2.0, e) < m, e + 1, e)
    e = torch.where(m == 0, torch.full_like(e, -127.0), e.clamp_min(-127.0))
    t = b / torch.pow(2.0, e).unsqueeze(2)
    k = torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6)))
    k = torch.where(torch.pow(2.0, k + 1) <= t.abs(), k + 1, k)
    k = torch.where((torch.pow(2.0, k) > t.abs()) & (k > -6), k - 1, k)
    step = torch.pow(2.0, k - 3)
    q = torch.round(t / step) * step
    return q.view(rows, -1)[:, :cols].to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _f64_saved(codes, scales):
    value = codes.view(torch.float8_e4m3fn).double()
    unit = torch.pow(2.0, scales.double() - 127.0)
    return value * unit.repeat_interleave(BLOCK, 1)[:, : value.shape[1]]


def _f64_gate(g, act):
    if act == SILU:
        sig = torch.special.expit(g)
        return g * sig, sig + g * sig * torch.special.expit(-g)
    c = math.sqrt(2.0 / math.pi)
    inner = c * (g + 0.044715 * g ** 3)
    left = torch.special.expit(2.0 * inner)  # (1 + tanh(inner)) / 2
    return g * left, left + 2.0 * g * left * torch.special.expit(-2.0 * inner) * c * (1.0 + 0.134145 * g ** 2)


def exact(case, seed):
    op = case["op"]
    if op in ("loss", "loss_step"):
        products = 1.0 if op == "loss" else 3.0
        if 2.0 * products * case["tokens"] * case["vocab"] * case["hidden"] > 1.3e13:
            return None  # too long in 64 bits
    s = prepare(case, seed)
    if op == "norm":
        total = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
        # the sum of the inputs is an fp32 value by definition: the checkpoint and `total` are made from it
        total = total.float().double()
        rstd = (total.pow(2).sum(1) / case["cols"] + EPS).pow(-0.5)
        codes, scales = _f64_codes(total)
        return {"y": total * rstd[:, None] * s["gamma"].double(), "total": total, "rstd": rstd, "codes": codes, "scales": scales}
    if op == "norm_back":
        v, dy, gamma, rstd = _f64_saved(s["codes"], s["scales"]), s["dy"].double(), s["gamma"].double(), s["rstd"].double()[:, None]
        inner = (v * dy * gamma).sum(1, keepdim=True) / case["cols"]
        dx = rstd * dy * gamma - v * rstd.pow(3) * inner
        if s["dtotal"] is not None:
            dx = dx + s["dtotal"].double()
        out = {"dx": dx, "dgamma": (dy * v * rstd).sum(0)}
        return {**out, "y": v * rstd * gamma} if case["remake"] else out
    if op == "glu":
        g, u = s["gate"].double(), s["up"].double()
        gc, gs = _f64_codes(g)
        uc, us = _f64_codes(u)
        return {"y": _f64_gate(g, case["act"])[0] * u, "gate_codes": gc, "gate_scales": gs, "up_codes": uc, "up_scales": us}
    if op == "glu_back":
        g, u = _f64_saved(s["gate_codes"], s["gate_scales"]), _f64_saved(s["up_codes"], s["up_scales"])
        dy = s["dy"].double()
        a, d = _f64_gate(g, case["act"])
        out = {"dgate": dy * u * d, "dup": dy * a}
        return {**out, "y": a * u} if case["remake"] else out
    h, w, targets, z = s["h"].double(), s["w"].double(), s["targets"], case["z"]
    keep = torch.nonzero(targets >= 0)[:, 0]
    hk, tk = h[keep], targets[keep]
    logits = hk @ w.T
    lse_k = torch.logsumexp(logits, 1)
    loss, lse = torch.zeros(len(targets), dtype=torch.float64, device=DEV), torch.zeros(len(targets), dtype=torch.float64, device=DEV)
    rows = torch.arange(len(keep), device=DEV)
    loss[keep] = lse_k - logits[rows, tk] + z * lse_k ** 2
    lse[keep] = lse_k
    out = {"loss": loss, "lse": lse}
    if op == "loss_step":
        p = logits.sub_(lse_k[:, None]).exp_()
        p.mul_((1.0 + 2.0 * z * lse_k)[:, None])
        p[rows, tk] -= 1.0
        p.mul_((s["weight"].double() * s["scale"].double())[keep][:, None])
        dh = torch.zeros_like(h)
        dh[keep] = p @ w
        out |= {"dh": dh, "dw": p.T @ hk}
    return out
