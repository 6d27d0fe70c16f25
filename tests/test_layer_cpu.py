"""The transformer-block operators (include/fc/layer.h) without a GPU: the
library exports what the header declares, rejects unsupported arguments before
it touches a device pointer (the pointers here are made up), and the 64-bit
statements that the GPU tests compare with agree with closed forms."""
import ctypes
import os
import re

import pytest
import torch

import bit_activation_compression_amd as fc
import layer_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fc", "layer.h")
NAN, INF = float("nan"), float("inf")


def P(i, off=0):
    """A 16-byte aligned pointer of its own region (64 MiB apart), never dereferenced."""
    return ctypes.c_void_p(0x10000000 + (i << 26) + off)


def test_exports_are_the_header_s():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fc_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(fc.LAYER_SYMBOLS)
    for n in names:
        assert hasattr(fc.lib(), n) and n in fc.__all__


def test_new_statuses_have_names():
    assert fc.fc_status_string(9).startswith("FC_ERR_OVERLAP")
    assert fc.fc_status_string(10).startswith("FC_ERR_VALUE")


X, RES, WPOST, GATE, WPRE, H_, Y_, C2, S2, Z2, WS = range(11)


def _norm(x=P(X), residual=P(RES), dt=1, T=8, H=256, w_post=P(WPOST), gate=P(GATE), gate_tokens=1,
          w_pre=P(WPRE), res_scale=1.0, out_scale=1.0, eps=1e-5, h=P(H_), y=P(Y_)):
    return fc.lib().fc_residual_norm(x, residual, dt, T, H, w_post, gate, gate_tokens, w_pre, res_scale,
                                     out_scale, eps, h, y, None)


@pytest.mark.parametrize("status,kw", [
    (2, dict(T=-1)), (2, dict(H=0)), (2, dict(H=65537)), (2, dict(gate_tokens=0)), (2, dict(gate_tokens=-3)),
    (7, dict(dt=2)),
    (10, dict(res_scale=NAN)), (10, dict(out_scale=INF)), (10, dict(eps=0.0)), (10, dict(eps=-1.0)),
    (10, dict(eps=NAN)), (10, dict(eps=INF)), (10, dict(eps=1e-39)),
    (1, dict(x=None)), (1, dict(residual=None)), (1, dict(h=None)), (1, dict(y=None)), (1, dict(w_pre=None)),
    (4, dict(x=P(X, 8))), (4, dict(residual=P(RES, 2))), (4, dict(w_post=P(WPOST, 4))),
    (4, dict(gate=P(GATE, 8))), (4, dict(w_pre=P(WPRE, 8))), (4, dict(h=P(H_, 8))), (4, dict(y=P(Y_, 8))),
    (9, dict(h=P(X))), (9, dict(y=P(X, 16))), (9, dict(y=P(RES))), (9, dict(h=P(RES, 16))), (9, dict(y=P(H_))),
    (9, dict(y=P(H_, 8 * 512 - 16))), (9, dict(h=P(WPOST))), (9, dict(y=P(WPRE, 496))), (9, dict(h=P(GATE, 7 * 512))),
    (0, dict(T=0, x=None, residual=None, h=None, y=None, w_pre=None, gate=None, w_post=None)),
])
def test_norm_refuses(status, kw):
    assert _norm(**kw) == status


def test_norm_gate_tokens_unused_without_gate():
    assert _norm(T=0, gate=None, gate_tokens=0) == 0


def _wire(codes=P(C2), s=P(S2), z=P(Z2), T=8, H=384, bits=4, group=96, dt=1, residual=P(RES), w_pre=P(WPRE),
          eps=1e-5, h=P(H_), y=P(Y_)):
    return fc.lib().fc_dequantize_residual_norm(codes, s, z, T, H, bits, group, dt, residual, None, None, 1,
                                                w_pre, 1.0, 1.0, eps, h, y, None)


@pytest.mark.parametrize("status,kw", [
    (3, dict(bits=5)), (2, dict(group=100)), (2, dict(group=3)), (2, dict(group=0)), (2, dict(H=0)),
    (2, dict(T=-1)), (2, dict(H=96 * 1000)), (7, dict(dt=-1)), (10, dict(eps=0.0)),
    (1, dict(codes=None)), (1, dict(s=None)), (1, dict(z=None)), (4, dict(z=P(Z2, 2))), (1, dict(y=None)),
    (9, dict(h=P(C2))), (9, dict(y=P(C2, 8 * 384 // 2 - 16))), (9, dict(y=P(Z2, 16))), (0, dict(T=0, codes=None)),
])
def test_wire_norm_refuses(status, kw):
    assert _wire(**kw) == status


def _allreduce(x=P(X), dt=1, R=2, T=8, H=256, b1=4, b2=4, group=128, residual=P(RES), w_pre=P(WPRE), eps=1e-5,
               h=P(H_), y=P(Y_), ws=P(WS), nbytes=1 << 20):
    return fc.lib().fc_allreduce_emulated_norm(x, dt, R, T, H, b1, b2, group, residual, None, None, 1, w_pre,
                                               1.0, 1.0, eps, h, y, ws, nbytes, None)


@pytest.mark.parametrize("status,kw", [
    (3, dict(b1=5)), (3, dict(b2=5)), (2, dict(R=3)), (2, dict(T=-1)), (2, dict(group=100)), (7, dict(dt=2)),
    (1, dict(ws=None)), (1, dict(x=None)), (4, dict(ws=P(WS, 8))), (10, dict(eps=0.0)),
    (5, dict(nbytes=100)), (9, dict(h=P(WS, 256))), (9, dict(x=P(WS))), (9, dict(residual=P(WS, 512))),
    (9, dict(w_pre=P(WS, 64))), (9, dict(h=P(X))), (0, dict(T=0, x=None, ws=None, nbytes=0)),
])
def test_allreduce_norm_refuses(status, kw):
    assert _allreduce(**kw) == status


def test_allreduce_norm_workspace_is_the_allreduce_s():
    need = fc.fc_workspace_bytes(2, 8, 256, 4, 128)
    assert _allreduce(nbytes=need - 1) == 5


def test_mxfp4_refuses():
    L = fc.lib()
    Q, D, M, N = L.fc_quantize_mxfp4, L.fc_dequantize_mxfp4, L.fc_matmul_mxfp4, L.fc_linear_mxfp4
    a, b, c, d, e, f = (P(i) for i in range(6))
    assert Q(a, 0, 0, 8, 128, b, c, None) == 2
    assert Q(a, 0, 1, -1, 128, b, c, None) == 2
    assert Q(a, 0, 1, 8, 0, b, c, None) == 2
    assert Q(a, 0, 1, 8, (1 << 22) + 1, b, c, None) == 2
    assert Q(a, 0, 1 << 30, 1 << 30, 128, b, c, None) == 2                     # more than 2^47 values
    assert D(a, b, 1 << 30, 1 << 30, 1 << 22, 0, c, None) == 2
    assert fc.fc_linear_mxfp4_workspace_bytes(1 << 30, 1 << 30, 1 << 22) == 0
    assert Q(a, 2, 1, 8, 128, b, c, None) == 7
    assert Q(None, 0, 1, 8, 128, b, c, None) == 1
    assert Q(a, 0, 1, 8, 128, b, P(2, 8), None) == 4
    assert Q(a, 0, 1, 8, 128, b, P(1, 16), None) == 9
    assert Q(a, 0, 1, 8, 128, P(0, 16), c, None) == 9
    assert Q(None, 0, 1, 0, 128, None, None, None) == 0
    assert D(a, b, 1, 8, 0, 0, c, None) == 2
    assert D(a, b, 1, 8, 128, 3, c, None) == 7
    assert D(a, None, 1, 8, 128, 0, c, None) == 1
    assert D(a, b, 1, 8, 128, 0, P(2, 2), None) == 4
    assert D(a, b, 1, 8, 128, 0, P(1, 16), None) == 9
    assert D(None, None, 1, 0, 128, 0, None, None) == 0
    assert M(a, b, c, d, 1, 8, 128, 0, 0, e, None) == 2
    assert M(a, b, c, d, 1, 8, 128, (1 << 24) + 1, 0, e, None) == 2
    assert M(a, b, c, d, 0, 8, 128, 64, 0, e, None) == 2
    assert M(a, b, c, d, 1 << 20, 1 << 20, 128, 1 << 20, 0, e, None) == 2    # more tiles than a grid has
    assert M(a, b, c, d, 1, 8, 128, 64, 2, e, None) == 7
    assert M(a, b, c, None, 1, 8, 128, 64, 0, e, None) == 1
    assert M(a, b, c, d, 1, 8, 128, 64, 0, P(4, 8), None) == 4
    assert M(a, b, c, d, 1, 8, 128, 64, 0, P(3, 16), None) == 9
    assert M(None, None, None, None, 1, 0, 128, 64, 0, None, None) == 0
    need = fc.fc_linear_mxfp4_workspace_bytes(1, 300, 128)
    assert need > 0
    assert N(a, b, c, 0, 1, 300, 128, 64, d, e, need - 1, None) == 5
    assert N(a, b, c, 0, 1, 300, 128, 64, d, None, need, None) == 1
    assert N(a, b, c, 0, 1, 300, 128, 64, d, P(4, 8), need, None) == 4
    assert N(a, b, c, 0, 1, 300, 128, 64, d, P(3, 16), need, None) == 9      # workspace in y
    assert N(a, b, c, 0, 1, 300, 128, 64, P(0, 16), e, need, None) == 9      # y in a
    assert N(a, b, c, 0, 1, 300, 0, 64, d, e, need, None) == 2
    assert N(a, b, c, 4, 1, 300, 128, 64, d, e, need, None) == 7
    assert N(None, None, None, 0, 1, 0, 128, 64, None, None, 0, None) == 0


def test_linear_workspace_holds_codes_and_scales():
    for R, T, K in [(1, 1000, 128), (4, 8192, 2048), (3, 777, 4100)]:
        Kp = -(-K // 128) * 128
        need = fc.fc_linear_mxfp4_workspace_bytes(R, T, K)
        assert need >= R * T * (Kp // 2 + Kp // 32) and need < R * T * (Kp // 2 + Kp // 32) + 256
    for bad in [(0, 8, 128), (1, -1, 128), (1, 8, 0), (1, 8, (1 << 22) + 1), (1, 0, 128)]:
        assert fc.fc_linear_mxfp4_workspace_bytes(*bad) == 0


def test_checks_under_sanitizers_match_the_library(tmp_path):
    """The checks' own code, built with address and undefined-behaviour sanitizers."""
    import shutil
    import subprocess
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "driver")
    r = subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-O1", "-g", "-std=c++17",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(ROOT, 'bit_activation_compression_amd', 'csrc')}",
                        os.path.join(ROOT, "tests", "sanitize", "validate_layer_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0 and "sanitize" in r.stderr:
        pytest.skip("sanitizer runtime not available")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-2000:]
    values = [0.0, 1.0, -2.0, 1e-39, 1e30, INF, -INF, NAN]
    refused = accepted = 0
    for line in r.stdout.splitlines():
        head, tail = line.split(" : ")
        kind, *args = head.split()
        args, got = [int(v) for v in args], [int(v) for v in tail.split()]
        if kind == "norm":
            T, H, gt, v, bad = args
            x = None if bad == 1 else P(0)
            h = x if bad == 2 else P(5, 8 if bad == 3 else 0)
            y = None if bad == 4 else P(6)
            res = h if bad == 5 else P(1)
            for st, kw in ((got[0], dict(out_scale=values[v])), (got[1], dict(eps=values[v]))):
                if st == 0 and T > 0:
                    accepted += 1          # not called: the pointers are made up
                    continue
                refused += st != 0
                assert _norm(x=x, residual=res, dt=1, T=T, H=H, w_post=P(2), gate=P(3), gate_tokens=gt, w_pre=P(4),
                             h=h, y=y, **kw) == st, line
        else:
            R, T, K, H = args
            if got[0] != 0:
                refused += 1
                assert fc.lib().fc_quantize_mxfp4(P(0), 1, R, T, K, P(1), P(2), None) == got[0], line
            if got[1] != 0:
                refused += 1
                assert fc.lib().fc_matmul_mxfp4(P(0), P(1), P(2), P(3), R, T, K, H, 1, P(4), None) == got[1], line
            assert got[2] == -(-K // 128) * 128 and got[3] == got[2] // 2
    assert refused > 1000 and accepted > 100


def test_binding_refuses_integers_past_32_bits():
    """ctypes would cut them down to values the library accepts."""
    m = torch.empty((4, 64), dtype=torch.bfloat16, device="meta")
    u8 = torch.empty((4, 32), dtype=torch.uint8, device="meta")
    u16 = torch.empty((4, 2), dtype=torch.uint16, device="meta")
    long_ = torch.empty(((1 << 32) + 4, 64), dtype=torch.bfloat16, device="meta")
    for call in [
        lambda: fc.fc_dequantize_residual_norm(u8, u16, u16, 4, 64, 4, (1 << 32) + 32, m),
        lambda: fc.fc_dequantize_residual_norm(u8, u16, u16, 4, 64, 4 - (1 << 32), 32, m),
        lambda: fc.fc_residual_norm(long_, long_),
    ]:
        with pytest.raises(ValueError, match="32 bits"):
            call()
    with pytest.raises(ValueError, match="32 bits"):
        fc._rows3(long_, "x")


def test_workspace_query_refuses_integers_past_32_bits():
    """(1, 2^32 + 8, 8192), cut to 32 bits, would be the workspace of 8 tokens."""
    for args in [(1, (1 << 32) + 8, 8192), ((1 << 32) + 1, 300, 128), (1, 300, (1 << 32) + 128), (1, 8 - (1 << 32), 8192)]:
        with pytest.raises(ValueError, match="32 bits"):
            fc.fc_linear_mxfp4_workspace_bytes(*args)
    # the largest that fit: refused by the library, and within its limits
    assert fc.fc_linear_mxfp4_workspace_bytes(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) == 0
    assert fc.fc_linear_mxfp4_workspace_bytes(1, 2 ** 31 - 1, 128) >= (2 ** 31 - 1) * 68


def test_weights_of_more_than_2_to_47_values_are_refused():
    """The limit on an operand's values holds for w as for a; R = 2 of the largest H and K meets it."""
    L, (a, b, c, d, e, f) = fc.lib(), (P(i) for i in range(6))
    H, K = 1 << 24, 1 << 22
    for T in (0, 1):
        assert L.fc_matmul_mxfp4(a, b, c, d, 3, T, K, H, 0, e, None) == 2
        assert L.fc_linear_mxfp4(a, b, c, 0, 3, T, K, H, d, e, 1 << 30, None) == 2
        assert L.fc_matmul_mxfp4(a, b, c, d, 1024, T, K, H // 512 + 1, 0, e, None) == 2
    assert L.fc_matmul_mxfp4(a, b, c, d, 2, 0, K, H, 0, e, None) == 0
    assert L.fc_linear_mxfp4(a, b, c, 0, 2, 0, K, H, d, e, 0, None) == 0
    assert L.fc_matmul_mxfp4(a, b, c, d, 1024, 0, K, H // 512, 0, e, None) == 0


# --- the 64-bit statements ---------------------------------------------------

def test_reference_quantizer_on_the_grid_ties_and_limits():
    g = ref.GRID
    # a block with 6 in it has E = 0: every grid value is its own code, signs kept
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :8], x[0, 8:16] = g, -g
    codes, scales = ref.mx_quantize(x)
    assert scales[0, 0] == 127 and scales[0, 1:].eq(0).all() and codes.shape == (1, 64)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten()
    assert c[:16].tolist() == list(range(16))
    # ties: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4; 7.9 saturates
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :9] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, 6.0])
    codes, scales = ref.mx_quantize(x)
    assert ref.mx_dequantize(codes, scales, 9)[0].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6]
    # scales: powers of two, the smallest and the largest
    for top, byte in [(1.0, 125), (1.99, 125), (2.0, 126), (2.0 ** -125, 0), (2.0 ** -124, 1), (2.0 ** 127, 252),
                      (0.0, 0), (2.0 ** -133, 0)]:
        x = torch.zeros(1, 32, dtype=torch.float64)
        x[0, 3] = top
        assert ref.mx_quantize(x)[1][0, 0] == byte
    x[0, 3] = INF
    x = torch.cat((x, torch.ones(1, 32, dtype=torch.float64)), 1)
    codes, scales = ref.mx_quantize(x)
    assert scales[0, 0] == 255 and scales[0, 1] == 125 and codes[0, :16].eq(0).all()
    assert torch.isnan(ref.mx_dequantize(codes, scales, 64)[0, :32]).all()


def test_reference_norms_closed_form():
    x = torch.full((2, 4), 3.0, dtype=torch.float64)
    one = torch.ones(4, dtype=torch.float64)
    h, eh, y, ey = ref.norms(x, 2 * x, one, 0.5 * one, 2, 4 * one, 0.25, 2.0, 0.0)
    assert torch.allclose(h, torch.full_like(h, 0.25 * 6 + 2 * 0.5)) and torch.allclose(y, torch.full_like(y, 4.0))
    assert (eh > 0).all() and (ey > 0).all()


def test_perf_plain_forms_match_their_definitions(monkeypatch):
    """perf/operators.py on the CPU, at small sizes: the plain forms against the 64-bit definitions."""
    import random

    import perf.operators as P
    monkeypatch.setattr(P, "DEV", "cpu")
    rng = random.Random(4)
    for case in P.listed() + [P.draw(rng) for _ in range(10)]:
        case = dict(case, T=min(case["T"], 5))
        if "R" in case:
            case.update(R=min(case["R"], 2), K=min(case["K"], 200), H=min(case["H"], 70))
        if case["op"] == "code":
            case["K"] = min(case["K"], 300)
        out, want = P.run(P.prepare(case, 1)), P.exact(case, 1)
        for o, w in zip(out if isinstance(out, list) else [out], want if isinstance(want, list) else [want]):
            assert o.shape == w.shape
            assert (o.double() - w).norm() <= 2.0 ** -8 * w.norm(), case
        assert P.work(case)["bytes"] > 0
