"""More of the training operators on the GPU: the RMS norm's backward pass from payloads,
with and without the skip connection's gradient, in every kernel that reads them."""
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
