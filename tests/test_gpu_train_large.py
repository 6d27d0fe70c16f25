"""Payloads whose kernels would take more threads than a launch counts in 32 bits."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc
import train_ref as ref
from test_gpu_train_products import _big, _codes

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    fc.lib()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _say(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


def test_weight_grad_of_more_than_2_to_35_values():
    """Groups that are no power of two are dequantized 8 values to a thread."""
    T, K, H, group = 65552, 524280, 512, 24
    assert T * K > 2 ** 35 and fc.fc_linear_weight_grad_workspace_bytes(1, T, K, H) >= 2 * T * K
    _say("payload")
    dy, (codes, s, z) = _big(T, H), _codes(T, K, group=group)
    torch.cuda.synchronize()
    _say("weight gradient of a large payload")
    dw = fc.fc_linear_weight_grad(dy, (codes, s, z))
    torch.cuda.synchronize()
    d = dy.double().t().contiguous()
    for c in (0, K // 2 // group * group, K - group):
        g = c // group
        scale, zero = (t[:, g:g + 1].contiguous().view(torch.float16).double() for t in (s, z))
        v = (codes[:, c:c + group].double() * scale + zero).float().to(BF16).double()
        assert ((dw[:, c:c + group].double() - d @ v).abs() <= (2 * T + 8) * ref.U * (d.abs() @ v.abs())).all(), c


def test_norm_with_a_payload_of_more_than_2_to_33_values():
    """Groups of 2, a thread to each in the quantizer; the norm as without it."""
    T, H, group = 131104, 65536, 2
    assert T * H // 2 > 2 ** 32
    x = torch.randn((4096, H), dtype=BF16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    x = x.repeat(T // 4096 + 1, 1)[:T].contiguous()
    codes = torch.full((T, H), 9, dtype=torch.uint8, device="cuda")
    _say("norm with a large payload")
    y, _, _, (codes, s, z) = fc.fc_layer_norm(x, group=group, payload=(codes, None, None))
    torch.cuda.synchronize()
    for t in (0, 32767, 32768, T // 2, T - 1):
        one = fc.fc_quantize_groups(x[None, t:t + 1], 8, group)
        for a, b in zip((codes, s, z), one):
            assert torch.equal(a[t].view(torch.uint8), b[0, 0].view(torch.uint8)), t
        assert torch.equal(y[t], fc.fc_layer_norm(x[t:t + 1])[0][0])
