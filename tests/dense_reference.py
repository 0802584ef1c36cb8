"""Plain 64-bit forms (CPU torch) of the dense feed-forward block, each with a bound of the error that
32-bit sums and the stated roundings may leave."""
import math

import torch

from block_reference import F32, act64, half_step

GROUP = 128


def slope64(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    c = 2 * math.sqrt(2 / math.pi)
    p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
    return p + z * p * (1 - p) * c * (1 + 0.134145 * z * z)


def product64(a, b):
    """(a b^T, bound) of 64-bit matrices: K/16 + 16 f32 additions, each off by at most one step (the
    tensor cores may truncate) of what has been summed; K split over a few parts adds as many."""
    K = a.shape[1]
    return a @ b.T, (K / 16 + 32) * 2 * F32 * (a.abs() @ b.abs().T)


# The activations have slopes of at most 1.2 and second slopes of at most 1.2; their own f32
# evaluation (an exponential, a division, three products) is good to 2^-19.
EVAL = 2.0 ** -19


def gated64(x, w, act):
    """(h, error of h before its rounding, gate, up, their errors) of 64-bit x, w."""
    F = w.shape[0] // 2
    z, off = product64(x, w)
    g, u, og, ou = z[:, :F], z[:, F:], off[:, :F], off[:, F:]
    a = act64(g, act)
    h = a * u
    err = 1.2 * og * (u.abs() + ou) + a.abs() * ou + EVAL * h.abs()
    return h, err, g, u, og, ou


def rounded(ref, err, dtype):
    return err + half_step(ref, dtype) * (1 + 2.0 ** -7)


def gated_bwd64(dh, x, w, g, u, og, ou, act, dtype):
    """{name: (reference, bound)}; g and u with their errors og, ou (0 from a checkpoint)."""
    a, s = act64(g, act), slope64(g, act)
    h = a * u
    eh = 1.2 * og * (u.abs() + ou) + a.abs() * ou + EVAL * h.abs()
    dg, du = dh * u * s, dh * a
    # the slope's terms are at most 1 + 1.2 |s - 1| in magnitude: its evaluation to 2^-19 of 1.2
    edg = dh.abs() * (1.2 * og * (u.abs() + ou) + 1.2 * ou + 1.2 * EVAL * u.abs())
    edu = dh.abs() * (1.2 * og + EVAL * a.abs())
    d = torch.cat([dg, du], dim=1)
    e = torch.cat([edg, edu], dim=1)
    e = rounded(d, e, dtype)  # rounded once, as the products' operand
    dx, ox = product64(d, w.T.contiguous())
    dw, ow = product64(d.T.contiguous(), x.T.contiguous())
    return dict(out=(h, rounded(h, eh, dtype)),
                d_x=(dx, rounded(dx, ox * 1.01 + e @ w.abs(), dtype)),
                d_w=(dw, rounded(dw, ow * 1.01 + e.T @ x.abs(), dtype)))


def linear_bwd64(dy, x, w, dtype):
    dx, ox = product64(dy, w.T.contiguous())
    dw, ow = product64(dy.T.contiguous(), x.T.contiguous())
    T = dy.shape[0]
    db = dy.sum(0)
    return dict(d_x=(dx, rounded(dx, ox, dtype)), d_w=(dw, rounded(dw, ow, dtype)),
                d_bias=(db, rounded(db, (T / 32 + 40) * F32 * dy.abs().sum(0), dtype)))


# -------------------------------------------------------------------------------- checkpoints
def groups64(v):
    v = torch.nn.functional.pad(v, (0, -v.shape[1] % GROUP))
    return v.view(v.shape[0], -1, GROUP)


def scales64(v):
    """The scale of each group of 64-bit [T, C]: the smallest power of two with max <= 448 scale."""
    b = groups64(v)
    top = torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b)).amax(dim=2)
    m, e = torch.frexp(top)
    k = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-118, 120)
    return torch.where(top > 0, torch.exp2(k.double()), torch.ones_like(top))


def e4m3_64(v):
    """Nearest E4M3 value, ties to even, of |v| <= 448; NaN of what is not finite."""
    fine = torch.isfinite(v)
    v = torch.where(fine, v, torch.zeros_like(v))
    _, e = torch.frexp(v)
    step = torch.exp2((e.clamp(min=-5) - 4).double())
    return torch.where(fine, torch.round(v / step) * step, torch.full_like(v, float("nan")))


def checkpoint64(v):
    """(values, scales) of 64-bit [T, C]."""
    s = scales64(v)
    q = e4m3_64(groups64(v) / s[:, :, None]) * s[:, :, None]
    return q.reshape(v.shape[0], -1)[:, :v.shape[1]], s


def restore64(codes, scale, C):
    """What codes and scales stand for, from the bits of E4M3."""
    c = codes.cpu().to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    mag = torch.where((c & 127) == 127, torch.full_like(mag, float("nan")), mag)
    v = torch.where(c >= 128, -mag, mag) * scale.cpu().double().repeat_interleave(GROUP, dim=1)
    return v[:, :C]


# ------------------------------------------------------------------------------- 4-bit weights
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)


def weights64(codes, scales, alpha):
    c = codes.cpu().long()
    v = torch.stack([E2M1[c & 15], E2M1[c >> 4]], dim=2).view(c.shape[0], -1)
    s = scales.cpu().view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1)
    return v * s * float(alpha)


def w4_sum64(x, w):
    """x w^T with the bound of product64, and bf16 x off by 2^-25 in f16 where it is small."""
    z, off = product64(x.cpu().double(), w)
    if x.dtype is torch.bfloat16:
        off = off + 2.0 ** -25 * torch.ones_like(x.cpu().double()) @ w.abs().T
    return z, off + 2 * F32 * z.abs()


def w4_linear64(x, w, bias, act, residual):
    z, off = w4_sum64(x, w)
    if bias is not None:
        z = z + bias.cpu().double()
        off = off + F32 * z.abs()
    a = act64(z, act)
    slope = {"none": 1.0, "silu": 1.2, "gelu_tanh": 1.2}.get(act)
    err = off * (2 * (z.abs() + off) if slope is None else slope)
    if act != "none":
        err = err + EVAL * a.abs()
    if residual is not None:
        r = residual.cpu().double()
        a, err = a + r, err + 2 * F32 * (a.abs() + r.abs())
    return a, rounded(a, err, x.dtype)


def w4_gated64(x, w, act):
    F = w.shape[0] // 2
    z, off = w4_sum64(x, w)
    g, u, og, ou = z[:, :F], z[:, F:], off[:, :F], off[:, F:]
    a = act64(g, act)
    h = a * u
    return h, rounded(h, 1.2 * og * (u.abs() + ou) + a.abs() * ou + EVAL * h.abs(), x.dtype)
