"""Plain 64-bit statements of the training operators (include/fc/train.h), in torch
on the CPU, each with a bound of what binary32 arithmetic adds to its result before
the rounding to 16 bits (layer_ref.step_bound counts that one)."""
from __future__ import annotations

import math

import torch

import layer_ref
from layer_ref import assert_within, dequantize  # noqa: F401  (the tests' shared helpers)

U = 2.0 ** -24          # a binary32 rounding, relative
# A row's sum: at most 64 additions in a thread and 32 across threads and waves, and
# the product with the rounded 1 / H.
SUM = 100 * U


def quantized(x, group):
    """The INT8 payload (codes, s, z) of x (16-bit, CPU) as fc_quantize_groups defines it,
    step by step in binary32."""
    g = x.float().unflatten(-1, (-1, group))
    mn, mx = g.amin(-1), g.amax(-1)
    s, z = ((mx - mn) / 255.0).half(), (mn + 0.0).half()
    sf = s.float()[..., None]
    inv = torch.where(sf > 0, 1.0 / torch.where(sf > 0, sf, 1.0), 0.0)
    q = ((g - z.float()[..., None]) * inv).round().clamp(0, 255)
    return q.flatten(-2).to(torch.uint8), s.view(torch.uint16), z.view(torch.uint16)


def held(payload, group):
    return dequantize(*payload, 8, group)


def layer_norm(x, w, b, eps, rms):
    """float64 -> dict of y, mean, rstd and their bounds (ey, emean, erstd)."""
    H = x.shape[-1]
    mean = torch.zeros(x.shape[0], 1, dtype=torch.float64) if rms else x.mean(-1, keepdim=True)
    em = torch.zeros_like(mean) if rms else SUM * x.abs().mean(-1, keepdim=True)
    c = x - mean
    ec = em + U * c.abs() * 2
    var = (c * c).mean(-1, keepdim=True)
    evar = SUM * var + 2 * (c.abs() * ec).mean(-1, keepdim=True) + (ec * ec).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    # v_rsq is off by an ulp, eps is added with one rounding
    erstd = rstd * (0.5 * evar * rstd * rstd * 1.01 + 4 * U)
    n = c * rstd
    en = ec * rstd + c.abs() * erstd + 2 * U * n.abs()
    ww = torch.ones(H, dtype=torch.float64) if w is None else w
    bb = torch.zeros(H, dtype=torch.float64) if b is None else b
    y = n * ww + bb
    return dict(y=y, ey=en * ww.abs() * 1.001 + 2 * U * ((n * ww).abs() + bb.abs()), mean=mean[:, 0], emean=em[:, 0],
                rstd=rstd[:, 0], erstd=erstd[:, 0])


def chain(T):
    """Additions that a sum over T rows passes through: a workgroup's rows (512 of them
    share many rows), the teams of its rows, and the join of the workgroups."""
    return min(T, T // 64 + 300) + 64


def layer_norm_backward(dy, x, mean, rstd, w, dres):
    """float64 (mean None: RMS) -> dict of dx, dw, db and their bounds."""
    H = x.shape[-1]
    m = torch.zeros_like(rstd) if mean is None else mean
    r = rstd[:, None]
    n = (x - m[:, None]) * r
    en = U * (3 * n.abs() + x.abs() * r)          # x of a payload is rounded too
    ww = torch.ones(H, dtype=torch.float64) if w is None else w
    g = dy * ww
    c2 = (g * n).mean(-1, keepdim=True)
    ec2 = SUM * (g * n).abs().mean(-1, keepdim=True) + (g.abs() * (en + 2 * U * n.abs())).mean(-1, keepdim=True)
    c1, ec1 = torch.zeros_like(c2), torch.zeros_like(c2)
    if mean is not None:
        c1 = g.mean(-1, keepdim=True)
        ec1 = (SUM + U) * g.abs().mean(-1, keepdim=True)
    dx = (g - c1 - n * c2) * r
    edx = r * (ec1 + n.abs() * ec2 + en * c2.abs() + 4 * U * (g.abs() + c1.abs() + (n * c2).abs())) * 1.001 + 2 * U * dx.abs()
    if dres is not None:
        dx = dx + dres
        edx = edx + 2 * U * (dx.abs() + dres.abs())
    k = chain(x.shape[0]) * U
    dw = (dy * n).sum(0)
    edw = (dy.abs() * en).sum(0) + k * (dy * n).abs().sum(0)
    return dict(dx=dx, edx=edx, dw=dw, edw=edw * 1.001, db=dy.sum(0), edb=k * dy.abs().sum(0) * 1.001)


def activation(z, act):
    """float64 -> (value, slope, bounds of both in binary32)."""
    if act == "none":
        return z, torch.ones_like(z), torch.zeros_like(z), torch.zeros_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).double(), torch.zeros_like(z), torch.zeros_like(z)
    if act == "gelu":
        p = torch.special.ndtr(z)
        extra = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        c = math.sqrt(8 / math.pi)
        u, du = (z, 1.0) if act == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z ** 2))
        p = torch.sigmoid(u)
        extra = z * p * torch.sigmoid(-u) * du
    # exp(v) carries v's roundings: |v| is at most z^2 / 2, |z| or 1.6 |z| + 0.072 |z|^3;
    # the fit of the normal distribution's tail is within 6e-7; results below 2^-126
    # are flushed
    rel = 2e-6 + 6e-7 * z * z
    tiny = 1e-36
    return z * p, p + extra, (z * p).abs() * rel + tiny, (p + extra.abs()) * rel + tiny


def linear(a, w, bias, act, mul, residual):
    """float64 [R, T, K] and [R, H, K] -> (y, bound, z, bound)."""
    wt = w.transpose(-1, -2).contiguous()
    z = torch.matmul(a, wt)
    mag = torch.matmul(a.abs(), wt.abs())
    ez = (2 * a.shape[-1] + 4) * U * mag
    if bias is not None:
        z = z + bias[:, None]
        ez = ez + 2 * U * (mag + bias.abs()[:, None])
    y, _, ey, _ = activation(z, act)
    ey = ey + 1.2 * ez          # no activation here is steeper than 1.13
    if mul is not None:
        y, ey = y * mul, ey * mul.abs() + U * (y * mul).abs()
    if residual is not None:
        ey = ey + U * (y.abs() + residual.abs()) * 1.001
        y = y + residual
    return y, ey, z, ez


def product(a, b):
    """a b for float64 [R, M, K], [R, K, N] -> (result, its binary32 bound)."""
    return torch.matmul(a, b), (2 * a.shape[-1] + 8) * U * torch.matmul(a.abs(), b.abs())


def activation_backward(dy, z, act, mul):
    """float64 -> dict of dz, dmul, db and their bounds."""
    value, slope, ev, es = activation(z, act)
    # z of a payload is rounded once; no slope changes faster than 1.1 per unit of z
    es = es + (0 if act in ("relu", "none") else 1.1) * U * z.abs()
    ev = ev + 1.2 * U * z.abs()
    m = torch.ones_like(z) if mul is None else mul
    dz = dy * m * slope
    edz = (dy * m).abs() * es * 1.001 + 5 * U * dz.abs()
    k = chain(z.shape[-2]) * U
    return dict(dz=dz, edz=edz, dmul=dy * value, edmul=dy.abs() * ev * 1.001 + 3 * U * (dy * value).abs(),
                db=dz.sum(-2), edb=edz.sum(-2) + k * dz.abs().sum(-2) * 1.001)


def assert_f32(got, ref, bound, what=""):
    """A binary32 result: the bound, and its own rounding."""
    got = got.cpu().double()
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)}"
    over = (got - ref).abs() - bound - U * ref.abs() - 1e-42
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert over.max().item() <= 0, f"{what}: {over.max().item()} over the bound"


__all__ = [n for n in dir() if not n.startswith("_")] + ["layer_ref"]
