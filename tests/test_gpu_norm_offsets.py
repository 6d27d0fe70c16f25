"""The norm's backward pass where the mean is far above the deviations: n = (x - mean) * rstd
loses nothing to the mean, from 16-bit rows and from payloads, in every kernel that reads
them (rows in a wave, of a workgroup, read twice, by columns)."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc
import train_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
U = ref.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    fc.lib()
    yield


def _say(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


def _rows(T, H, dt, offset, deviation, seed):
    g = torch.Generator().manual_seed(seed)
    x = (offset + deviation * torch.randn(T, H, generator=g)).to(dt)
    mean = x.double().mean(-1)
    c = x.double() - mean[:, None]
    rstd = (1 / torch.sqrt((c * c).mean(-1) + 1e-5)).float()
    return (x, mean.float(), rstd, torch.randn(T, H, generator=g).to(dt), (1 + 0.3 * torch.randn(H, generator=g)).to(dt))


def _expected(dy, x, mean, rstd, w, en):
    """float64 -> (dx, its bound, dw, its bound) for an n that is off by en(n). A row's sums:
    ref.SUM; the last steps of dx: four roundings of its terms and one of the sum; dw: an
    fma a row and the join of ref.chain."""
    r = rstd[:, None]
    n = (x - mean[:, None]) * r
    en = en(n)
    g = dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * n).mean(-1, keepdim=True)
    ec1 = (ref.SUM + U) * g.abs().mean(-1, keepdim=True)
    ec2 = ref.SUM * (g * n).abs().mean(-1, keepdim=True) + (g.abs() * (en + 2 * U * n.abs())).mean(-1, keepdim=True)
    dx = (g - c1 - n * c2) * r
    edx = r * (ec1 + n.abs() * ec2 + en * c2.abs() + 4 * U * (g.abs() + c1.abs() + (n * c2).abs())) * 1.001 + 2 * U * dx.abs()
    edw = (dy.abs() * en).sum(0) + ref.chain(x.shape[0]) * U * (dy * n).abs().sum(0)
    return dx, edx, (dy * n).sum(0), edw * 1.001


# rows of a wave, of a workgroup (whole vectors and not), read twice; one row has the
# tightest bound of dw
SIZES = [(1, 64), (3, 100), (1, 1024), (2, 5003), (5, 8192), (1, 16384), (3, 20001)]
OFFSETS = [(F16, 1000.0, 1.0), (F16, 2000.0, 2.0), (F16, 30.0, 1.0), (BF16, -250.0, 2.0), (BF16, 30.0, 0.5)]


@pytest.mark.parametrize("dt,offset,deviation", OFFSETS)
@pytest.mark.parametrize("T,H", SIZES)
def test_backward_of_rows_far_from_zero(T, H, dt, offset, deviation):
    """x - mean is off by a rounding of the difference, n by one more."""
    _say(f"norm backward at offset {offset} T={T} H={H} {dt}")
    x, mean, rstd, dy, w = _rows(T, H, dt, offset, deviation, T + H)
    dx, dw, db = fc.fc_layer_norm_backward(*(t.cuda() for t in (dy, x, mean, rstd, w)))
    rx, ex, rw, ew = _expected(*(t.double() for t in (dy, x, mean, rstd, w)), lambda n: 2.001 * U * n.abs())
    ref.assert_within(dx, rx, dt, ex, "dx")
    ref.assert_f32(dw, rw, ew, "dw")


@pytest.mark.parametrize("dt,offset,deviation", OFFSETS)
@pytest.mark.parametrize("T,H,group", [(1, 64, 16), (3, 96, 24), (1, 1024, 128), (5, 8192, 64), (1, 16384, 128), (3, 20000, 40)])
def test_backward_of_payloads_far_from_zero(T, H, group, dt, offset, deviation):
    """n = q s rstd + (z - mean) rstd: the first factor is rounded once, the second term twice,
    n once; no term is larger than a group's range of the row."""
    _say(f"norm backward from a payload at offset {offset} T={T} H={H} g={group} {dt}")
    x, mean, rstd, dy, w = _rows(T, H, dt, offset, deviation, T + H)
    payload = ref.quantized(x, group)
    dx, dw, db = fc.fc_layer_norm_backward(dy.cuda(), tuple(t.cuda() for t in payload), mean.cuda(), rstd.cuda(), w.cuda())
    held = ref.held(payload, group)
    zero = payload[2].view(F16).double().repeat_interleave(group, -1)
    r = rstd.double()[:, None]
    rx, ex, rw, ew = _expected(*(t.double() for t in (dy, held, mean, rstd, w)), lambda n: 1.001 * U * (
        n.abs() + ((held - zero) * r).abs() + 2 * ((zero - mean.double()[:, None]) * r).abs()))
    ref.assert_within(dx, rx, dt, ex, "dx")
    ref.assert_f32(dw, rw, ew, "dw")


@pytest.mark.parametrize("T,H", SIZES)
def test_backward_of_constant_rows_whose_mean_times_rstd_overflows(T, H):
    """1e30 with rstd = 1e15: n is 0, dw too, and dx = rstd (g - mean(g))."""
    g = torch.Generator().manual_seed(H)
    x = torch.full((T, H), 1e30).to(BF16)
    mean, rstd = x[:, 0].float(), torch.full((T,), 1e15)
    dy = torch.randn(T, H, generator=g).to(BF16)
    dx, dw, db = fc.fc_layer_norm_backward(*(t.cuda() for t in (dy, x, mean, rstd)), dw=torch.ones(H, device="cuda"))
    d = dy.double()
    c1 = d.mean(-1, keepdim=True)
    bound = 1e15 * ((ref.SUM + U) * d.abs().mean(-1, keepdim=True) + 6 * U * (d.abs() + c1.abs()))
    ref.assert_within(dx, (d - c1) * rstd.double()[:, None], BF16, bound, "dx")
    assert (dw == 0).all()
    ref.assert_f32(db, d.sum(0), ref.chain(T) * U * d.abs().sum(0), "db")
