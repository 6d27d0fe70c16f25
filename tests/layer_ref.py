"""Plain 64-bit statements of the transformer-block operators (include/fc/layer.h),
in torch on the CPU, and the error each 16-bit output may have.

A correctly rounded 16-bit result is off by at most half a step, u |ref| with
u = finfo.eps / 2 (or half the smallest subnormal); what the binary32
arithmetic before that rounding can add is bounded case by case below."""
from __future__ import annotations

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def step_bound(ref, dtype, extra):
    """|out - ref| for out = RN_dtype(v), |v - ref| <= extra."""
    f = torch.finfo(dtype)
    return (f.eps / 2) * (ref.abs() + extra) + extra + f.smallest_normal * f.eps / 2


def assert_within(got, ref, dtype, extra, what=""):
    got = got.cpu().double()
    assert got.shape == ref.shape
    # what binary32 cannot tell from an overflow of the 16-bit type is left to the caller
    over = (got - ref).abs() - step_bound(ref, dtype, extra)
    worst = over.max().item()
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert worst <= 0, f"{what}: {worst} over the bound at {tuple(torch.nonzero(over == over.max())[0].tolist())}"


# Relative error of a normed row in binary32: the squares are summed by at most
# 64 additions in a thread and 16 + 6 across them (each 2^-24), the mean, eps and
# v_rsq (1 ulp = 2^-23) follow, half of the sum's part reaches the root: under
# (43 + 1 + 2) * 2^-24; three more products and the final sum make 50 * 2^-24.
NORM_REL = 50 * 2.0 ** -24


def norms(x, residual, w_post, gate, gate_tokens, w_pre, res_scale, out_scale, eps):
    """All inputs float64 (or None). -> (h, its binary32 error bound, y, its bound)."""
    n = x
    if w_post is not None:
        n = w_post * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if gate is not None:
        rows = torch.arange(x.shape[0]) // gate_tokens
        n = n * gate.reshape(-1, x.shape[1])[rows]
    h = res_scale * residual + out_scale * n
    eh = NORM_REL * ((res_scale * residual).abs() + (out_scale * n).abs())
    if w_pre is None:
        return h, eh, None, None
    rstd = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    y = w_pre * h * rstd
    # an error of h moves the row's norm by at most the same relative amount
    rel_norm = torch.sqrt((eh * eh).mean(-1, keepdim=True)) * rstd
    ey = w_pre.abs() * eh * rstd * 1.001 + y.abs() * (NORM_REL + rel_norm * 1.001)
    return h, eh, y, ey


def unpack_codes(codes, bits):
    codes = codes.long()
    return codes if bits == 8 else torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def dequantize(codes, s, z, bits, group):
    q = unpack_codes(codes, bits).double()
    wide = [v.view(torch.float16).double().repeat_interleave(group, -1) for v in (s, z)]
    return q * wide[0] + wide[1]


def mx_quantize(x):
    """x [..., K] float64 -> (codes [..., Kp/2], scales [..., Kp/32]) uint8."""
    K = x.shape[-1]
    Kp = -(-K // 128) * 128
    p = torch.zeros(*x.shape[:-1], Kp, dtype=torch.float64)
    p[..., :K] = x
    b = p.reshape(*x.shape[:-1], Kp // 32, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros(1, dtype=torch.float64), b)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1].double() - 3, torch.tensor(-127.0, dtype=torch.float64))
    e = e.clamp(-127, 127)
    m = b.abs() / torch.exp2(e)[..., None]
    code = torch.zeros(m.shape, dtype=torch.uint8)
    for i in range(7):   # the borders lie halfway; a value on one goes to the even code
        mid = (GRID[i] + GRID[i + 1]) / 2
        code += ((m >= mid) if i % 2 else (m > mid)).to(torch.uint8)
    code += torch.signbit(b).to(torch.uint8) * 8
    code[bad] = 0
    scale = (e + 127).to(torch.uint8)
    scale[bad] = 255
    code = code.reshape(p.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def mx_dequantize(codes, scales, K):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = GRID[c & 7] * (1.0 - 2.0 * (c >> 3).double())
    e = torch.exp2(scales.double() - 127.0)
    e[scales == 255] = float("nan")
    return (v * e.repeat_interleave(32, -1))[..., :K]


def mx_product(a, w):
    """-> (sum, sum of magnitudes) of float64 [R, T, K] and [R, H, K]."""
    wt = w.transpose(-1, -2).contiguous()
    return torch.matmul(a, wt), torch.matmul(a.abs(), wt.abs())
