"""The training-step operators in 64 bits (torch, any device), for their tests:
the checkpoint format element by element, and the formulas of the header."""
import math

import torch

BLOCK = 32


def encode(v):
    """(code bytes, scale bytes) of fp32 rows, in 64 bits: scale 2^e with e the
    least integer such that M <= 448 * 2^e (at least -127); E4M3 values have
    spacing 2^(k-3) in [2^k, 2^(k+1)), k >= -6, and bytes sign | (k+7) << 3 | f."""
    v = v.double().cpu()
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    p = torch.zeros((rows, nb * BLOCK), dtype=torch.float64)
    p[:, :cols] = v
    b = p.view(rows, nb, BLOCK)
    m = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    m = torch.where(bad, torch.zeros_like(m), m)
    e = torch.full_like(m, -127.0)
    for cand in range(121, -128, -1):                       # the last (least) that holds
        e = torch.where(m <= 448.0 * 2.0 ** cand, torch.full_like(e, float(cand)), e)
    t = (torch.where(bad[..., None], torch.zeros_like(b), b) * torch.pow(2.0, -e)[..., None])
    a = t.abs()
    mant, ex = torch.frexp(a)
    k = torch.clamp(ex - 1, min=-6).double()
    q = torch.round(a / torch.pow(2.0, k - 3)) * torch.pow(2.0, k - 3)  # half to even
    mant, ex = torch.frexp(q)
    k = torch.clamp(ex - 1, min=-6)
    f = (q / torch.pow(2.0, (k - 3).double())).long()       # 8..15 for normals, 0..7 below 2^-6
    byte = torch.where(f >= 8, ((k + 7).long() << 3) | (f & 7), f)
    byte = torch.where(byte == 0, byte, byte | ((t < 0).long() << 7))
    byte = torch.where(bad[..., None], torch.full_like(byte, 0x7F), byte)
    scale = torch.where(bad, torch.full_like(e, 255.0), e + 127).to(torch.uint8)
    return byte.view(rows, -1)[:, :cols].to(torch.uint8), scale


def decode(codes, scales):
    c = codes.cpu().long()
    e, f = (c >> 3) & 15, c & 7
    val = torch.where(e > 0, (8 + f).double() * torch.pow(2.0, (e - 10).double()), f.double() * 2.0 ** -9)
    val = torch.where((c & 0x7F) == 0x7F, torch.full_like(val, math.nan), val)
    val = torch.where(c >= 128, -val, val)
    unit = torch.pow(2.0, scales.cpu().double() - 127.0)
    return val * unit.repeat_interleave(BLOCK, 1)[:, :val.shape[1]]


def act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
    n = torch.sigmoid(-2 * c * (g + 0.044715 * g ** 3))
    return g * s, s + 2 * c * g * s * n * (1 + 3 * 0.044715 * g * g)


def norm(total, gamma, eps):
    total, gamma = total.double(), gamma.double()
    rstd = (total.square().mean(1) + eps).rsqrt()
    return total * rstd[:, None] * gamma, rstd


def norm_backward(s, rstd, gamma, dy):
    s, rstd, gamma, dy = s.double(), rstd.double()[:, None], gamma.double(), dy.double()
    h = s * rstd
    q = dy * gamma
    return rstd * (q - h * (q * h).mean(1, keepdim=True)), (dy * h).sum(0), h * gamma


def head(h, w, targets, z=0.0):
    """loss, lse (0 for ignored tokens), and the logits of the valid ones."""
    h, w = h.double(), w.double()
    keep = (targets >= 0) & (targets < w.shape[0])
    logits = h[keep] @ w.T
    l = torch.logsumexp(logits, 1)
    loss, lse = torch.zeros_like(h[:, 0]), torch.zeros_like(h[:, 0])
    lse[keep] = l
    loss[keep] = l - logits.gather(1, targets[keep][:, None])[:, 0] + z * l * l
    return loss, lse, logits, keep


def head_backward(h, w, targets, weight, scale, z=0.0):
    """dh, dw, and the sums of magnitudes |dl| |w| and |dl|^T |h| that bound their rounding."""
    _, lse, logits, keep = head(h, w, targets, z)
    h, w = h.double(), w.double()
    l, t = lse[keep], targets[keep]
    dl = torch.exp(logits - l[:, None]) * (1 + 2 * z * l)[:, None]
    dl[torch.arange(len(t), device=h.device), t] -= 1
    dl = dl * (weight.double()[keep][:, None] if weight is not None else 1.0)
    sc = float(scale) if scale is not None else 1.0
    dh, mh = torch.zeros_like(h), torch.zeros_like(h)
    dh[keep] = sc * (dl @ w)
    mh[keep] = abs(sc) * (dl.abs() @ w.abs())
    hk = h[keep]
    return dh, sc * (dl.T @ hk), mh, abs(sc) * (dl.abs().T @ hk.abs())
