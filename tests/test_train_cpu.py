"""The training operators (include/fc/train.h) without a GPU: the library exports what
the header declares, rejects unsupported arguments before it touches a device pointer
(the pointers here are made up), the binding its own, and the 64-bit statements that
the GPU tests compare with agree with differentiation and with differences."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

import bit_activation_compression_amd as fc
import train_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_activation_compression_amd", "csrc")
NAN, INF = float("nan"), float("inf")
BIG = 2 ** 31 - 1


def P(i, off=0):
    """A 16-byte aligned pointer of its own region (64 MiB apart), never dereferenced."""
    return ctypes.c_void_p(0x10000000 + (i << 26) + off)


def test_exports_are_the_header_s():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fc", "train.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fc_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(fc.TRAIN_SYMBOLS)
    for n in names:
        assert hasattr(fc.lib(), n) and n in fc.__all__
    acts = re.findall(r"FC_ACT_([A-Z_]+) = (\d)", open(os.path.join(ROOT, "include", "fc", "train.h")).read())
    assert [(a.lower(), int(i)) for a, i in acts] == [(a, i) for i, a in enumerate(fc.ACTIVATIONS)]


def _norm(x=P(0), dt=1, T=8, H=256, w=P(1), b=P(2), eps=1e-5, rms=0, y=P(3), mean=P(4), rstd=P(5), codes=P(6), s=P(7),
          z=P(8), group=64):
    return fc.lib().fc_layer_norm(x, dt, T, H, w, b, eps, rms, y, mean, rstd, codes, s, z, group, None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(T=-1)), (2, dict(H=0)), (2, dict(H=65537)), (2, dict(group=0)), (2, dict(group=3)), (2, dict(group=100)),
    (7, dict(dt=2)), (10, dict(eps=0.0)), (10, dict(eps=NAN)), (10, dict(eps=INF)), (10, dict(eps=1e-39)), (10, dict(rms=1)),
    (1, dict(x=None)), (1, dict(y=None)), (1, dict(s=None)), (1, dict(z=None)), (1, dict(codes=None)),
    (4, dict(x=P(0, 8))), (4, dict(w=P(1, 2))), (4, dict(b=P(2, 4))), (4, dict(y=P(3, 8))), (4, dict(mean=P(4, 4))),
    (4, dict(rstd=P(5, 8))), (4, dict(codes=P(6, 1))), (4, dict(s=P(7, 2))),
    (9, dict(y=P(0))), (9, dict(y=P(0, 4080))), (9, dict(y=P(1))), (9, dict(mean=P(3, 4080))), (9, dict(codes=P(0, 16))),
    (9, dict(rstd=P(4, 16))), (9, dict(z=P(7))), (9, dict(s=P(6, 2032))),
    (0, dict(T=0, x=None, y=None, codes=None, s=None, z=None)), (0, dict(T=0, rms=1)),
])
def test_layer_norm_refuses(status, kw):
    assert _norm(**kw) == status


def _back(dy=P(0), x=None, codes=P(1), s=P(2), z=P(3), group=64, dt=1, T=8, H=256, mean=P(4), rstd=P(5), w=P(6), dres=P(7),
          dx=P(8), dw=P(9), db=P(10), ws=P(11), nbytes=1 << 26):
    return fc.lib().fc_layer_norm_backward(dy, x, codes, s, z, group, dt, T, H, mean, rstd, w, dres, dx, dw, db, ws, nbytes, None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(T=-1)), (2, dict(H=0)), (2, dict(H=65537)), (2, dict(group=4)), (2, dict(group=12)), (2, dict(group=96)),
    (7, dict(dt=3)), (1, dict(dy=None)), (1, dict(x=P(12))), (1, dict(codes=None)), (1, dict(s=None)), (1, dict(z=None)),
    (1, dict(rstd=None)), (1, dict(dx=None)), (1, dict(ws=None)), (5, dict(nbytes=0)), (5, dict(nbytes=2047)),
    (4, dict(dy=P(0, 8))), (4, dict(codes=P(1, 8))), (4, dict(s=P(2, 2))), (4, dict(mean=P(4, 4))), (4, dict(w=P(6, 8))),
    (4, dict(dres=P(7, 2))), (4, dict(dx=P(8, 8))), (4, dict(dw=P(9, 4))), (4, dict(db=P(10, 8))), (4, dict(ws=P(11, 8))),
    (9, dict(dx=P(0, 16))), (9, dict(dx=P(7, 16))), (9, dict(dx=P(1))), (9, dict(dw=P(0))), (9, dict(db=P(9, 1008))),
    (9, dict(ws=P(8))), (9, dict(ws=P(7, 16))), (9, dict(dx=P(6))), (9, dict(dw=P(5))), (9, dict(dx=P(4))),
    (9, dict(codes=None, x=P(8), s=None, z=None)), (9, dict(H=16384, dx=P(0))),
])
def test_layer_norm_backward_refuses(status, kw):
    assert _back(**kw) == status


def test_workspaces():
    B, G, A = (fc.fc_layer_norm_backward_workspace_bytes, fc.fc_linear_weight_grad_workspace_bytes,
               fc.fc_activation_backward_workspace_bytes)
    assert B(0, 64) == 0 and B(-1, 64) == 0 and B(5, 0) == 0 and B(5, 65537) == 0
    assert B(1, 8192) == 2 * 8192 * 4
    for T in (1, 100, 8192, 10 ** 6, BIG):
        for H in (1, 64, 513, 8192, 8193, 65536):
            assert 8 * H <= B(T, H) <= 512 * 8 * H
    assert G(0, 1, 8, 8) == G(1, 0, 8, 8) == G(1, 8, 0, 8) == G(1, 8, 8, 1 << 23) == G(BIG, BIG, 4096, 4096) == 0
    assert G(1, 1, 4096, 4096) == 0                        # one token is not split
    assert A(0, 1, 8) == A(1, 0, 8) == A(1, 8, 0) == A(BIG, BIG, 1 << 22) == 0
    assert A(1, 1, 64) == 0 and A(1, 8192, 8192) > 0
    for f, n in ((B, 2), (G, 4), (A, 3)):
        with pytest.raises(ValueError):
            f(*[2 ** 32 + 1] * n)


def _linear(a=P(0), w=P(1), dt=0, R=2, T=8, K=128, H=64, bias=P(2), act=3, mul=P(3), res=P(4), y=P(5), z=P(6), ws=P(7),
            nbytes=1 << 26):
    return fc.lib().fc_linear_act(a, w, dt, R, T, K, H, bias, act, mul, res, y, z, ws, nbytes, None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(R=0)), (2, dict(T=-1)), (2, dict(K=0)), (2, dict(H=0)), (2, dict(K=(1 << 22) + 1)), (2, dict(H=(1 << 22) + 1)),
    (2, dict(R=BIG)), (2, dict(T=BIG, H=1 << 12)), (10, dict(act=-1)), (10, dict(act=5)), (7, dict(dt=2)),
    (1, dict(a=None)), (1, dict(w=None)), (1, dict(y=None)),
    (4, dict(a=P(0, 8))), (4, dict(w=P(1, 2))), (4, dict(bias=P(2, 4))), (4, dict(mul=P(3, 8))), (4, dict(res=P(4, 8))),
    (4, dict(y=P(5, 8))), (4, dict(z=P(6, 8))),
    (9, dict(y=P(0))), (9, dict(y=P(1, 32752))), (9, dict(y=P(2))), (9, dict(y=P(3))), (9, dict(y=P(4, 16))), (9, dict(z=P(4))),
    (9, dict(z=P(5, 2032))), (9, dict(z=P(0, 4080))),
    (0, dict(T=0, a=None, w=None, y=None)),
])
def test_linear_act_refuses(status, kw):
    assert _linear(**kw) == status


def _input_grad(dy=P(0), w=P(1), dt=0, R=2, T=8, K=128, H=64, res=P(2), dx=P(3), ws=P(4), nbytes=1 << 26):
    return fc.lib().fc_linear_input_grad(dy, w, dt, R, T, K, H, res, dx, ws, nbytes, None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(R=0)), (2, dict(T=-1)), (2, dict(K=0)), (2, dict(H=(1 << 22) + 1)), (7, dict(dt=2)), (1, dict(dy=None)),
    (1, dict(w=None)), (1, dict(dx=None)), (4, dict(dy=P(0, 8))), (4, dict(res=P(2, 8))), (4, dict(dx=P(3, 2))),
    (9, dict(dx=P(0))), (9, dict(dx=P(1))), (9, dict(dx=P(2, 16))), (0, dict(T=0, dy=None, w=None, dx=None)),
])
def test_input_grad_refuses(status, kw):
    assert _input_grad(**kw) == status


def test_products_workspaces_are_checked():
    """Sums that are split: few outputs of long rows."""
    for call, size, at in ((_linear, fc.fc_linear_act_workspace_bytes, 5), (_input_grad, fc.fc_linear_input_grad_workspace_bytes, 3)):
        kw = dict(R=1, T=40, K=4096, H=128) if call is _linear else dict(R=1, T=40, K=128, H=4096)
        need = size(**kw)
        assert need > 0 and need % (40 * 128 * 4) == 0
        assert call(**kw, nbytes=need - 1) == 5
        assert call(**kw, ws=None) == 1
        assert call(**kw, ws=P(7, 8)) == 4
        for other in (0, 1, at):
            assert call(**kw, ws=P(other)) == 9
        assert call(**kw, ws=P(4 if call is _linear else 2)) == 9        # the residual
        assert size(1, 8192, 4096, 4096) == 0 and size(1, 0, 4096, 4096) == 0 and size(1, 1, 1 << 23, 8) == 0
    assert fc.fc_linear_act_workspace_bytes(1, 1, 4096, 64) == 0             # single tokens have none


def _weight_grad(dy=P(0), codes=P(1), s=P(2), z=P(3), group=32, dt=0, R=2, T=8, K=128, H=64, acc=0, dw=P(4), ws=P(5), nbytes=0):
    return fc.lib().fc_linear_weight_grad(dy, codes, s, z, group, dt, R, T, K, H, acc, dw, ws, nbytes, None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(R=0)), (2, dict(T=-1)), (2, dict(K=0)), (2, dict(H=0)), (2, dict(group=0)), (2, dict(group=4)), (2, dict(group=48)),
    (2, dict(group=20)), (2, dict(K=1 << 20, group=32)), (7, dict(dt=2)), (1, dict(dy=None)), (1, dict(codes=None)),
    (1, dict(s=None)), (1, dict(z=None)), (1, dict(dw=None)), (1, dict(T=0, dw=None)), (4, dict(dy=P(0, 8))),
    (4, dict(codes=P(1, 8))), (4, dict(s=P(2, 2))), (4, dict(dw=P(4, 4))), (4, dict(ws=P(5, 8))), (4, dict(T=0, dw=P(4, 4))),
    (9, dict(dw=P(0))), (9, dict(dw=P(1, 16))), (9, dict(dw=P(3))), (0, dict(T=0, acc=1, dy=None, codes=None, s=None, z=None)),
])
def test_weight_grad_refuses(status, kw):
    assert _weight_grad(**kw) == status


def test_weight_grad_workspace_is_checked():
    T = 1 << 16
    need = fc.fc_linear_weight_grad_workspace_bytes(1, T, 64, 64)
    if need:
        kw = dict(R=1, T=T, K=64, H=64, group=8)
        assert _weight_grad(**kw, nbytes=need - 1) == 5
        assert _weight_grad(**kw, ws=None) == 1
        assert _weight_grad(**kw, ws=P(4), nbytes=need) == 9
        assert _weight_grad(**kw, ws=P(1), nbytes=need) == 9


def _act(dy=P(0), codes=P(1), s=P(2), z=P(3), mc=P(4), ms=P(5), mz=P(6), group=32, dt=0, R=2, T=8, H=64, act=3, dz=P(7),
         dmul=P(8), db=P(9), ws=P(10), nbytes=1 << 20):
    return fc.lib().fc_activation_backward(dy, codes, s, z, mc, ms, mz, group, dt, R, T, H, act, dz, dmul, db, ws, nbytes, None)


NONE = dict(act=0, codes=None, s=None, z=None, mc=None, ms=None, mz=None, dz=None, dmul=None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(R=0)), (2, dict(T=-1)), (2, dict(H=0)), (2, dict(group=0)), (2, dict(group=12)), (2, dict(group=24)),
    (2, dict(H=1 << 20)), (2, dict(R=BIG, T=BIG, H=1 << 19)), (10, dict(act=-1)), (10, dict(act=5)), (7, dict(dt=2)),
    (1, dict(dy=None)), (1, dict(codes=None)), (1, dict(s=None)), (1, dict(z=None)), (1, dict(dz=None)), (1, dict(dmul=None)),
    (1, dict(mc=None)), (1, dict(ms=None)), (1, dict(mz=None)),
    (4, dict(dy=P(0, 8))), (4, dict(codes=P(1, 8))), (4, dict(mz=P(6, 2))), (4, dict(dz=P(7, 8))), (4, dict(dmul=P(8, 8))),
    (4, dict(db=P(9, 4))), (9, dict(dz=P(0, 16))), (9, dict(dz=P(1))), (9, dict(dmul=P(0))), (9, dict(dmul=P(7))),
    (9, dict(db=P(7))), (9, dict(db=P(6))), (9, dict(dz=P(4, 16))),
    (10, dict(act=0)), (10, dict(NONE, dz=P(7))), (10, dict(NONE, codes=P(1))), (1, dict(NONE, db=None)), (1, dict(NONE, dy=None)),
    (2, dict(NONE, H=(1 << 22) + 1)), (9, dict(NONE, db=P(0))), (0, dict(NONE, T=0, db=None)), (0, dict(T=0, db=None, dy=None)),
])
def test_activation_backward_refuses(status, kw):
    assert _act(**kw) == status


def test_activation_backward_workspace_is_checked():
    need = fc.fc_activation_backward_workspace_bytes(1, 8192, 4096)
    assert need
    kw = dict(NONE, R=1, T=8192, H=4096)
    assert _act(**kw, nbytes=need - 1) == 5
    assert _act(**kw, ws=None) == 1
    assert _act(**kw, ws=P(9), nbytes=need) == 9
    assert _act(**kw, ws=P(0, 4096), nbytes=need) == 9


def test_checks_under_sanitizers(tmp_path):
    """The checks' own code at the largest sizes, and that the library answers alike."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "driver")
    r = subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-O1", "-g", "-std=c++17",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "sanitize", "validate_train_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0 and "sanitize" in r.stderr:
        pytest.skip("sanitizer runtime not available")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = {}
    for line in r.stdout.splitlines():
        head, res = line.split(" : ")
        kind, *args = head.split()
        args, res = [int(a) for a in args], int(res)
        seen[kind, res] = seen.get((kind, res), 0) + 1
        if kind == "product":
            R, T, K, H = args
            # a NULL operand: a supported call gets that far
            assert _linear(a=None, R=R, T=T, K=K, H=H) == (res or (1 if T > 0 else 0)), line
        elif kind == "group":
            H, g = args
            st = _act(dy=None, R=1, T=1, H=H, group=g, db=None)
            assert st == (1 if res else 2), line
        else:
            R, T, H = args
            if H <= 1 << 22:
                assert _act(**dict(NONE, dy=None, R=R, T=T, H=H, ws=None)) == (1 if res else 2), line
    assert seen["product", 0] > 50 and seen["product", 2] > 50 and seen["group", 1] == 2


# --- the binding's own checks ------------------------------------------------

def test_binding_refuses_what_is_no_gpu_tensor_or_of_another_kind():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    f = torch.zeros(4)
    for call in (lambda: fc.fc_layer_norm(x), lambda: fc.fc_layer_norm(x[None]), lambda: fc.fc_layer_norm(x.float()),
                 lambda: fc.fc_layer_norm_backward(x, x, f, f), lambda: fc.fc_layer_norm_backward(x, x, None, f),
                 lambda: fc.fc_layer_norm_backward(x, x, f, f, rms=True),
                 lambda: fc.fc_linear_act(x, x), lambda: fc.fc_linear_act(x, x[:, :32]), lambda: fc.fc_linear_act(x[None], x),
                 lambda: fc.fc_linear_input_grad(x, x), lambda: fc.fc_linear_input_grad(x, x[:, :32]),
                 lambda: fc.fc_linear_weight_grad(x, (x, x, x)), lambda: fc.fc_linear_weight_grad(x, (x[None], x, x)),
                 lambda: fc.fc_linear_weight_grad(x, (x, x, x), accumulate=True),
                 lambda: fc.fc_activation_backward(x, "tanh"), lambda: fc.fc_activation_backward(x, "none"),
                 lambda: fc.fc_activation_backward(x, "gelu"), lambda: fc.fc_activation_backward(x, "none", bias=True)):
        with pytest.raises(ValueError):
            call()


# --- the 64-bit statements ---------------------------------------------------

def _leaf(t):
    return t.double().clone().requires_grad_()


@pytest.mark.parametrize("rms", [False, True])
def test_reference_layer_norm_gradients_are_autograd_s(rms):
    g = torch.Generator().manual_seed(1)
    x, dy, dres = (torch.randn(5, 24, generator=g, dtype=torch.float64) for _ in range(3))
    w, b = torch.randn(24, generator=g, dtype=torch.float64), torch.randn(24, generator=g, dtype=torch.float64)
    xl, wl, bl = _leaf(x), _leaf(w), _leaf(b)
    c = xl if rms else xl - xl.mean(-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-3) * wl + bl
    (y * dy).sum().backward()
    r = ref.layer_norm(x, w, b, 1e-3, rms)
    assert torch.allclose(r["y"], y.detach(), atol=1e-12)
    got = ref.layer_norm_backward(dy, x, None if rms else r["mean"], r["rstd"], w, dres)
    assert torch.allclose(got["dx"], xl.grad + dres, atol=1e-12)
    assert torch.allclose(got["dw"], wl.grad, atol=1e-12) and torch.allclose(got["db"], bl.grad, atol=1e-12)
    assert all((r[k] > 0).all() for k in ("ey", "erstd")) and all((got[k] > 0).all() for k in ("edx", "edw", "edb"))


@pytest.mark.parametrize("act", fc.ACTIVATIONS)
def test_reference_slopes_are_differences(act):
    z = torch.linspace(-12, 12, 2401, dtype=torch.float64) + 3e-3
    value, slope, ev, es = ref.activation(z, act)
    h = 1e-5
    up, down = ref.activation(z + h, act)[0], ref.activation(z - h, act)[0]
    assert ((up - down) / (2 * h) - slope).abs().max() < 1e-9
    assert slope.abs().max() < 1.13
    lib = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act]
    assert (value - lib(z)).abs().max() < 1e-14


def test_reference_linear_gradients_are_autograd_s():
    g = torch.Generator().manual_seed(2)

    def n(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)
    a, w, b, m, res, dy = n(2, 7, 6), n(2, 5, 6), n(2, 5), n(2, 7, 5), n(2, 7, 5), n(2, 7, 5)
    al, wl, bl, ml = (_leaf(t) for t in (a, w, b, m))
    z = torch.matmul(al, wl.transpose(-1, -2).contiguous()) + bl[:, None]
    y = torch.nn.functional.gelu(z) * ml + res
    (y * dy).sum().backward()
    ry, ey, rz, ez = ref.linear(a, w, b, "gelu", m, res)
    assert torch.allclose(ry, y.detach(), atol=1e-12) and torch.allclose(rz, z.detach(), atol=1e-12)
    r = ref.activation_backward(dy, rz, "gelu", m)
    assert torch.allclose(r["dmul"], ml.grad, atol=1e-12) and torch.allclose(r["db"], bl.grad, atol=1e-12)
    assert torch.allclose(ref.product(r["dz"], w)[0], al.grad, atol=1e-12)
    assert torch.allclose(ref.product(r["dz"].transpose(-1, -2).contiguous(), a)[0], wl.grad, atol=1e-12)


def test_reference_payload_is_within_half_a_step():
    x = torch.randn(9, 96, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[0] = 0.75
    p = ref.quantized(x, 24)
    g = x.double().unflatten(-1, (-1, 24))
    step = (g.amax(-1) - g.amin(-1)) / 255
    # half a code step, the fp16 roundings of zero and scale (255 times)
    tol = step * 0.5 + 2.0 ** -11 * (g.amin(-1).abs() + 255 * step) + 1e-6
    err = (ref.held(p, 24) - x.double()).abs().unflatten(-1, (-1, 24)).amax(-1)
    assert (err <= tol).all() and (ref.held(p, 24)[0] - 0.75).abs().max() == 0


def test_perf_plain_forms_match_their_definitions(monkeypatch):
    """perf/more_operators.py on the CPU, at small sizes: the plain forms against the 64-bit definitions."""
    import perf.more_operators as M
    monkeypatch.setattr(M, "DEV", "cpu")
    rng = random.Random(4)
    for case in M.listed() + [M.draw(rng) for _ in range(12)]:
        case = dict(case, T=min(case["T"], 6))
        if case["op"] == "linear":
            case.update(K=min(case["K"], 200), H=min(case["H"], 70))
        out, want = M.run(M.prepare(case, 1)), M.exact(case, 1)
        assert len(out) == len(want)
        for o, w in zip(out, want):
            assert o.shape == w.shape
            assert (o.double() - w).norm() <= 2.0 ** -8 * w.norm(), case
        assert M.work(case)["bytes"] > 0
