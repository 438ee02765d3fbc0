"""Plain 64-bit definitions of the 8-bit cache's operators, and bounds of what rounding may do to them."""
import math

import torch

E4M3, INT8 = 0, 1
TOP = {E4M3: 448.0, INT8: 127.0}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def values(codes, fmt):
    """Codes (uint8) as the numbers they stand for, fp64."""
    return codes.view(torch.float8_e4m3fn).double() if fmt == E4M3 else codes.view(torch.int8).double()


def step_of(x, fmt):
    """Distance between neighbouring code values at x (scale divided out)."""
    if fmt == INT8:
        return torch.ones_like(x)
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)


def nearest(x, fmt):
    """The code value nearest to x, ties to even, kept in range."""
    s = step_of(x, fmt)
    return (torch.round(x / s) * s).clamp(-TOP[fmt], TOP[fmt])


def exponent(top, fmt):
    """The smallest e in [-63, 63] with top <= largest code * 2^e, top a float."""
    e = -63
    while e < 63 and top > TOP[fmt] * 2.0 ** e:
        e += 1
    return e


def rotated(x, pos, inv_freq, inter=False, scale=1.0):
    """x [..., n, D] fp64 with its first 2 len(inv_freq) coordinates turned; pos [n]."""
    rot = 2 * inv_freq.numel()
    if rot == 0:
        return x
    a = pos.double()[:, None] * inv_freq.double().to(x.device)
    y = x[..., :rot]
    u, w = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :rot // 2], y[..., rot // 2:])
    u, w = u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()
    y = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((y * scale, x[..., rot:]), -1)


def attention(q, k, v, p, see, scale, cap=0.0, slopes=None):
    """One sequence in fp64: q [Hq, L, D], k, v [H, N, D], p [L] positions, see [L, N]. Returns the output, sum w |v|
    and the largest sum |q| |k| scale of a row."""
    Hq, L, D = q.shape
    H, N, _ = k.shape
    G = Hq // H
    ke, ve = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    x = (q @ ke.transpose(1, 2)) * scale
    size = ((q.abs() @ ke.abs().transpose(1, 2)) * abs(scale)).masked_fill(~see, 0.0)
    if cap:
        x = cap * torch.tanh(x / cap)
    if slopes is not None:
        t = torch.arange(N, device=q.device)
        x = x - slopes.double()[:, None, None] * (p[:, None] - t).abs()
    x = x.masked_fill(~see, -math.inf)
    top = x.amax(-1, keepdim=True) if N else torch.full((Hq, L, 1), -math.inf, device=q.device, dtype=torch.float64)
    w = torch.exp(x - torch.where(top == -math.inf, 0.0, top)).masked_fill(~see, 0.0)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return w @ ve, w @ ve.abs(), size.amax(-1, keepdim=True) if N else torch.zeros_like(total)


def bound(ref, wv, size, dtype, N, vmax, D, cap=0.0, slope=0.0, rounded=True):
    """How far an output element may be from `ref`.

    Scores: the query's fp16 rounding (2^-11 of each product where it was rotated; below 2^-14 of the row's largest,
    2^-25 of that: counted with the same term), fp32 sums of D products (D 2^-24), scale factors (3 x 2^-24), the cap
    (cap 2^-20: exp2, reciprocal and difference near 1), the bias (slope N 2^-23). An error d of every score moves the
    output by at most 2 d sum w |v|. Weights: fp16 (2^-11), below fp16's smallest normal an absolute 2^-25 of the
    largest, N times; exp2's own error and fp32 sums (2^-20). The output's rounding: half a step."""
    d = size * ((2.0 ** -11 if rounded else 2.0 ** -22) + (D + 8) * 2.0 ** -24) + cap * 2.0 ** -20 + slope * N * 2.0 ** -23
    return ref.abs() * (torch.finfo(dtype).eps / 2) + wv * (2.0 ** -11 + 2 * d + 2.0 ** -20) * 1.01 + N * 2.0 ** -25 * vmax + 2.0 ** -25
