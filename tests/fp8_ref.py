"""8-bit operands with a scale for each block of 128, and the layer norm, in 64 bits (torch), for their tests."""
import torch

from tests import train_ref

BLOCK = 128
LEAST = 2.0 ** -126


def nearest_e4m3(t):
    """Code bytes of fp64 values of at most 464 (above 448 they round to it): spacing 2^(k-3) in [2^k, 2^(k+1)), k >= -6."""
    a = t.abs()
    k = torch.clamp(torch.frexp(a)[1] - 1, min=-6).double()
    q = torch.round(a / torch.pow(2.0, k - 3)) * torch.pow(2.0, k - 3)  # half to even
    k = torch.clamp(torch.frexp(q)[1] - 1, min=-6)
    f = (q / torch.pow(2.0, (k - 3).double())).long()      # 8..15 for normals, 0..7 below 2^-6
    byte = torch.where(f >= 8, ((k + 7).long() << 3) | (f & 7), f)
    return torch.where(byte == 0, byte, byte | ((t < 0).long() << 7)).to(torch.uint8)


def quantize(x, block_rows):
    """(codes, scales) of bf16 or fp32 rows (CPU): scale, reciprocal and scaled value are each rounded to fp32."""
    x = x.double().cpu()
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // BLOCK)
    pad = torch.zeros((br * block_rows, bc * BLOCK), dtype=torch.float64)
    pad[:rows, :cols] = x
    b = pad.view(br, block_rows, bc, BLOCK)
    bad = ~torch.isfinite(b).all(3).all(1)
    nan = torch.isnan(b).any(3).any(1)
    m = torch.where(torch.isfinite(b), b, torch.zeros_like(b)).abs().amax((1, 3))
    s = (m / 448.0).float().clamp_min(LEAST)
    s = torch.where(bad, torch.full_like(s, float("inf")), s)
    s = torch.where(nan, torch.full_like(s, float("nan")), s)
    inv = (1.0 / s.double()).float().double()
    t = (torch.where(bad[:, None, :, None], torch.zeros_like(b), b) *
         torch.where(bad, torch.zeros_like(inv), inv)[:, None, :, None]).float().double()
    codes = nearest_e4m3(t)
    codes = torch.where(bad[:, None, :, None], torch.full_like(codes, 0x7F), codes)
    return codes.reshape(br * block_rows, -1)[:rows, :cols].contiguous(), s


def restore(codes, scales, block_rows):
    rows, cols = codes.shape
    val = train_ref.decode(codes, torch.full((rows, -(-cols // 32)), 127))  # units of 1
    s = scales.double().cpu()
    return val * s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def layer_norm(s, gamma, beta, eps):
    s = s.double().cpu()
    mean = s.mean(1)
    d = s - mean[:, None]
    rstd = (d.square().mean(1) + eps).rsqrt()
    y = d * rstd[:, None] * gamma.double().cpu()
    return (y if beta is None else y + beta.double().cpu()), mean, rstd


def layer_norm_backward(s, mean, rstd, gamma, dy):
    s, mean, rstd, gamma, dy = (t.double().cpu() for t in (s, mean, rstd, gamma, dy))
    h = (s - mean[:, None]) * rstd[:, None]
    q = dy * gamma
    dx = rstd[:, None] * (q - q.mean(1, keepdim=True) - h * (q * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0), h, q
