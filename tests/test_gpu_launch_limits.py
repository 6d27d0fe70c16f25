"""Calls whose kernels would take 2^32 threads or more: the runtime does not refuse such a
launch but runs the threads modulo 2^32. The quantizers and dequantizers go in pieces, the
reduction refuses what does not fit."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _memory():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _say(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


def _need(gib):
    free, _ = torch.cuda.mem_get_info()
    if free < (gib + 8) * 2 ** 30:
        pytest.skip(f"needs ~{gib} GiB of free device memory")


def _ends(T, H, piece):
    """The first and last rows, and those around the pieces' borders."""
    cross = [c // H for c in range(piece, T * H, piece)]
    return sorted({t for c in [0, T - 2] + cross for t in range(max(c - 1, 0), min(c + 2, T))})


def test_dequantize_generic_past_2_to_35_values():
    T, H, group = 65552, 524280, 24
    assert T * H // 8 > 2 ** 32
    _need(110)
    _say("codes")
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (T, H), dtype=torch.uint8, device="cuda", generator=g)
    s = (torch.rand(T, H // group, device="cuda", generator=g) * 0.02 + 0.01).half()
    payload = codes, s.view(torch.uint16), (-128 * s).half().view(torch.uint16)
    out = torch.full((T, H), 7.0, dtype=F16, device="cuda")
    _say("dequantize in pieces")
    fc.fc_dequantize(*payload, T, H, 8, group, F16, out=out)
    torch.cuda.synchronize()
    for t in _ends(T, H, 2 ** 34):
        one = fc.fc_dequantize(*(r[t].clone() for r in payload), 1, H, 8, group, F16)
        assert torch.equal(out[t], one[0]), t
    _say("and in place, added to a residual")
    rows = _ends(T, H, 2 ** 34)
    out.fill_(1.0)
    fc.fc_dequantize_residual(*payload, T, H, 8, group, out, out=out)
    torch.cuda.synchronize()
    for t in rows:
        one = fc.fc_dequantize_residual(*(r[t].clone() for r in payload), 1, H, 8, group,
                                        torch.ones(1, H, dtype=F16, device="cuda"))
        assert torch.equal(out[t], one[0]), t


def test_quantize_generic_past_2_to_33_values():
    """Groups of 2: a thread to each."""
    T, H, group = 131104, 65536, 2
    assert T * H // 2 > 2 ** 32
    _need(45)
    x = torch.randn((4096, H), dtype=F16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    x = x.repeat(T // 4096 + 1, 1)[:T].contiguous()
    _say("quantize in pieces")
    codes = torch.full((1, T, H), 9, dtype=torch.uint8, device="cuda")
    codes, s, z = fc.fc_quantize_groups(x[None], 8, group, codes1=codes)
    torch.cuda.synchronize()
    for t in _ends(T, H, 2 ** 31):
        one = fc.fc_quantize_groups(x[None, t:t + 1].clone(), 8, group)
        for a, b in zip((codes, s, z), one):
            assert torch.equal(a[0, t].view(torch.uint8), b[0, 0].view(torch.uint8)), t
    _say("the reduction refuses it")
    with pytest.raises(fc.FcError, match="LAUNCH"):
        fc.fc_dequant_sum_requant(codes, s, z, 1, T, H, 8, group)


def test_quantize_and_dequantize_past_2_to_36_values():
    """Groups of the fast kernels: 16 values to a thread of the quantizer."""
    T, H, group = (2 ** 36 >> 16) + 16, 65536, 8192
    _need(175)
    x = torch.empty((T, H), dtype=BF16, device="cuda")
    rows = torch.randn((2048, H), dtype=BF16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    for t in range(0, T, 2048):
        x[t:t + 2048] = rows[:min(2048, T - t)]
    _say("quantize in pieces")
    codes = torch.full((1, T, H // 2), 0x99, dtype=torch.uint8, device="cuda")
    codes, s, z = fc.fc_quantize_groups(x[None], 4, group, codes1=codes)
    torch.cuda.synchronize()
    picked = _ends(T, H, 2 ** 34)
    for t in picked:
        one = fc.fc_quantize_groups(x[None, t:t + 1].clone(), 4, group)
        for a, b in zip((codes, s, z), one):
            assert torch.equal(a[0, t].view(torch.uint8), b[0, 0].view(torch.uint8)), t
    _say("dequantize in pieces, over the operand")
    x.zero_()
    fc.fc_dequantize(codes[0], s[0], z[0], T, H, 4, group, BF16, out=x)
    torch.cuda.synchronize()
    for t in picked:
        one = fc.fc_dequantize(*(r[0, t].clone() for r in (codes, s, z)), 1, H, 4, group, BF16)
        assert torch.equal(x[t], one[0]), t
