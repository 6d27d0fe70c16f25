"""More of the training operators on the GPU: the RMS norm's backward pass from payloads,
with and without the skip connection's gradient, in every kernel that reads them; calls with
workspaces that run on two streams at a time; activations of infinities, NaN and values
far from zero."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc
import train_ref as ref
from test_gpu_layer_norm import EPS, Guarded, _check_backward, _inputs, _on, _stats

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    fc.lib()
    yield


def _say(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


# rows side by side in a wave, several to a workgroup, one to a workgroup, read twice
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("rms,dres", [(True, False), (True, True), (False, True)])
@pytest.mark.parametrize("T,H,group", [(1, 8, 8), (70, 96, 24), (300, 512, 64), (33, 1040, 104), (700, 4096, 128), (20, 8192, 512),
                                       (30, 8200, 200), (150, 16384, 128)])
def test_backward_from_payload_rms_and_skip(T, H, group, rms, dres, dt):
    _say(f"backward from payload T={T} H={H} g={group} {dt} rms={rms} dres={dres}")
    d = _inputs(T, H, dt, T + H)
    mean, rstd = _stats(d["x"], rms)
    payload = ref.quantized(d["x"], group)
    dx, dw, db = Guarded((T, H), dt), Guarded((H,), torch.float32), Guarded((H,), torch.float32)
    args = (_on(d["dy"]), tuple(t.cuda() for t in payload), _on(mean), _on(rstd), _on(d["w"]))
    skip = _on(d["dres"]) if dres else None
    got = fc.fc_layer_norm_backward(*args, rms=rms, dres=skip, dx=dx.t, dw=dw.t, db=db.t)
    _check_backward(got, d, ref.held(payload, group), mean, rstd, dt, dres=dres)
    for g in (dx, dw, db):
        g.check()
    again = fc.fc_layer_norm_backward(*args, rms=rms, dres=skip)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    if dres:      # in place, over the skip connection's gradient
        over = fc.fc_layer_norm_backward(*args, rms=rms, dres=skip, dx=skip)
        for a, b in zip(got, over):
            assert torch.equal(a, b)


def test_two_streams_at_a_time():
    """Each stream has its own operands, outputs and workspaces, all made beforehand: the host
    only enqueues, far faster than the calls run, so that those of both streams overlap. Calls
    that split sums over workgroups, with workspaces that hold the other calls' leftovers."""
    R, T, K, H = 1, 4096, 1024, 1280
    g = torch.Generator(device="cuda").manual_seed(6)

    def n(*shape, dt=BF16):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    def one():
        d = dict(dy=n(R, T, H), x=n(T, K), w=n(R, H, K), b=n(R, H), few=n(R, 40, K), rows=n(T, K), pre=n(R, T, H))
        d["payload"] = fc.fc_quantize_groups(n(R, T, K), 8, 64)
        d["pz"] = fc.fc_quantize_groups(d["pre"], 8, 32)
        out = dict(y=n(R, 40, H), dx=n(R, 40, K), dw=n(R, H, K, dt=torch.float32), dz=n(R, T, H), db=n(R, H, dt=torch.float32),
                   dn=n(T, K), dg=n(K, dt=torch.float32), dbeta=n(K, dt=torch.float32))
        need = [fc.fc_linear_act_workspace_bytes(R, 40, K, H), fc.fc_linear_input_grad_workspace_bytes(R, 40, K, H),
                fc.fc_linear_weight_grad_workspace_bytes(R, T, K, H), fc.fc_activation_backward_workspace_bytes(R, T, H),
                fc.fc_layer_norm_backward_workspace_bytes(T, K)]
        assert min(need) > 0
        ws = torch.full((max(need),), 0x7F, dtype=torch.uint8, device="cuda")
        _, mean, rstd, _ = fc.fc_layer_norm(d["x"], stats=True)
        small, gain = d["dy"][:, :40].contiguous(), d["x"][0].clone()

        def calls(stream):
            kw = dict(workspace=ws, stream=stream)
            fc.fc_linear_act(d["few"], d["w"], d["b"], "gelu", y=out["y"], **kw)
            fc.fc_linear_input_grad(small, d["w"], dx=out["dx"], **kw)
            fc.fc_linear_weight_grad(d["dy"], d["payload"], dw=out["dw"], **kw)
            fc.fc_activation_backward(d["dy"], "silu", d["pz"], dz=out["dz"], db=out["db"], **kw)
            fc.fc_layer_norm_backward(d["rows"], d["x"], mean, rstd, gain, dx=out["dn"], dw=out["dg"],
                                      db=out["dbeta"], **kw)
        return calls, out

    sides = [one(), one()]
    want = []
    for calls, out in sides:
        calls(None)
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
    streams = [torch.cuda.Stream() for _ in sides]
    for turn in range(8):
        for _, out in sides:
            for t in out.values():
                t.fill_(3.0)
        torch.cuda.synchronize()
        for _ in range(12):
            for (calls, _), s in zip(sides, streams):
                calls(s)
        torch.cuda.synchronize()
        for (_, out), w in zip(sides, want):
            for k, v in out.items():
                assert torch.equal(v, w[k]), (turn, k)


FORMULAS = {"none": lambda z: z, "relu": lambda z: torch.where(z.isnan(), z, z.clamp_min(0)), "silu": lambda z: z / (1 + torch.exp(-z)),
            # (torch's own normal distribution function is 0 below -8.3)
            "gelu": lambda z: z * (0.5 * torch.special.erfc(z * -0.5 ** 0.5)),
            "gelu_tanh": lambda z: z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))) / 2}


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("act", list(fc.ACTIVATIONS))
@pytest.mark.parametrize("T,K", [(2, 64), (40, 72), (40, 4096), (40, 71)])
def test_activations_of_infinities_nan_and_far_values(T, K, act, dt):
    """Pre-activations that the bias gives: streamed weights, tiles, split sums, rows of odd length."""
    far = 3e4 if dt is F16 else 1e30
    inf, nan = float("inf"), float("nan")
    bias = torch.tensor([inf, -inf, nan, far, -far, 300.0, -300.0, 90.0, -90.0, 0.0, -0.0, 12.0, -12.0]).to(dt)
    H = len(bias)
    a, w = torch.zeros(T, K, dtype=dt, device="cuda"), torch.ones(H, K, dtype=dt, device="cuda")
    y, z = fc.fc_linear_act(a, w, bias.cuda(), act, z=True)
    want = FORMULAS[act](bias.double())
    y, z = y.cpu(), z.cpu()
    for t in range(T):
        assert torch.equal(z[t].isnan(), bias.isnan()) and torch.equal(z[t][~bias.isnan()], bias[~bias.isnan()])
        assert torch.equal(y[t].isnan(), want.isnan()), (y[t], want)
        ok = ~want.isnan()
        assert torch.equal(y[t][ok].isinf(), want[ok].isinf()) and torch.equal(y[t][ok].isinf() & (y[t][ok] > 0), want[ok] == inf)
        fin = torch.isfinite(want)
        # at |z| = 12 the tails keep their digits (ref.activation); below 1e-36 they are flushed
        rel = 2e-6 + 6e-7 * bias.double()[fin].clamp(-40, 40) ** 2
        ref.assert_within(y[t][fin], want[fin], dt, want[fin].abs() * rel + 1e-36, act)


@pytest.mark.parametrize("mul", [False, True])
@pytest.mark.parametrize("act", list(fc.ACTIVATIONS)[1:])
def test_activation_backward_far_from_zero(act, mul):
    """Values of a payload up to 1.6e7 on both sides: past 50 the slope is 0 or 1 to within
    |z| exp(-|z|) < 1e-20, the value 0 or z to within 50 times that."""
    T, H, group = 5, 64, 8
    scale = torch.tensor([[1.0, 64.0, 1000.0, 65504.0, 0.5, 8.0, 30000.0, 257.0]]).half().expand(T, H // group).contiguous()
    zero = -torch.where(scale > 256, torch.full_like(scale, 65504.0), 128 * scale)
    codes = torch.tensor([0, 1, 2, 3, 252, 253, 254, 255], dtype=torch.uint8).repeat(T, H // 8)
    payload = (codes, scale.view(torch.uint16), zero.contiguous().view(torch.uint16))
    z = ref.held(payload, group)
    keep = z.abs() > 50
    assert keep.sum() > T * H // 2 and z.max() > 1.5e7
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(22)).to(BF16)
    m = ref.quantized(torch.randn(T, H, generator=torch.Generator().manual_seed(23)).to(BF16), group)
    dz, dm, _ = fc.fc_activation_backward(dy.cuda(), act, _payload_on(payload), mul=_payload_on(m) if mul else None)
    factor = ref.held(m, group) if mul else torch.ones_like(z)
    want = torch.where(z > 0, dy.double() * factor, 0.0)
    # on the positive side ref.activation's 2e-6, and two products
    bound = (1e-18 + 2e-6 * (z > 0) + 3 * ref.U * (z > 0)) * (dy.double() * factor).abs()
    ref.assert_within(dz.cpu()[keep], want[keep], BF16, bound[keep], "dz")
    if mul:
        want = dy.double() * z.clamp_min(0)
        ref.assert_within(dm.cpu()[keep], want[keep], BF16, ((2e-6 + 4 * ref.U) * want.abs() + 1e-18 * dy.double().abs())[keep], "dmul")


def _payload_on(payload):
    return tuple(t.cuda() for t in payload)
