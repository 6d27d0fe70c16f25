"""MXFP4 on the GPU against the 64-bit statements (tests/layer_ref.py): the
quantizer and the dequantizer bit for bit over every 16-bit value and every
code and scale, the product bit for bit on operands whose sums binary32 holds
exactly and within the accumulation bound on others, and the three together
with the all-reduce as a transformer block runs them."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc
import layer_ref as ref

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


def _guarded(shape, dtype):
    n = 1
    for s in shape:
        n *= s
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((512 + n * size + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    def check():
        assert (raw[:512] == 0x5A).all() and (raw[512 + n * size:] == 0x5A).all()
    return raw[512:512 + n * size].view(dtype).view(shape), check


def _quantize(x):
    """GPU codes and scales of a CPU tensor, with the bytes around them checked."""
    Kp = -(-x.shape[-1] // 128) * 128
    codes, c1 = _guarded((*x.shape[:-1], Kp // 2), torch.uint8)
    scales, c2 = _guarded((*x.shape[:-1], Kp // 32), torch.uint8)
    fc.fc_quantize_mxfp4(x.cuda(), codes, scales)
    torch.cuda.synchronize()
    c1(), c2()
    return codes, scales


@pytest.mark.parametrize("dt", [BF16, F16])
def test_quantize_every_value(dt):
    """Every finite bit pattern, in blocks of neighbours (as neighbouring magnitudes) and in blocks
    whose scale another value sets."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
    bits = bits[torch.isfinite(bits.float())]
    bits = torch.cat((bits, torch.zeros(-len(bits) % 32, dtype=dt)))
    rows = [bits]
    for top in ([1.0, 1.75, 2.0 ** -10, 2.0 ** 15 - 16, 2.0 ** -24] if dt == F16
                else [1.0, 1.75, 2.0 ** 120, 2.0 ** 127, 2.0 ** -100, 2.0 ** -124, 2.0 ** -126, 2.0 ** -133]):
        small = bits[bits.float().abs() <= top]
        small = torch.cat((small, torch.zeros(-len(small) % 31, dtype=dt))).view(-1, 31)
        b = torch.cat((small, torch.full((len(small), 1), top, dtype=dt)), 1).flatten()
        rows.append(torch.cat((b, torch.zeros(-len(b) % 128, dtype=dt))))
    for i, x in enumerate(rows):
        _say(f"quantize every value {dt} set {i}")
        codes, scales = _quantize(x[None])
        want = ref.mx_quantize(x[None].double())
        assert torch.equal(scales.cpu(), want[1])
        assert torch.equal(codes.cpu(), want[0])


SHAPES = [(1, 1), (3, 31), (2, 32), (5, 33), (4, 100), (7, 127), (1, 128), (9, 129), (2, 250), (130, 256), (3, 4100),
          (65, 4096), (1000, 200), (2, 5, 96), (4, 33, 640), (1, 70001), (3, 65536)]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_shapes_and_back(shape, dt):
    _say(f"quantize {shape} {dt}")
    g = torch.Generator().manual_seed(sum(shape))
    x = (torch.randn(shape, generator=g) * torch.exp2(torch.randint(-8, 8, shape, generator=g).float())).to(dt)
    x[..., ::7] = 0
    codes, scales = _quantize(x)
    want = ref.mx_quantize(x.double())
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
    out, check = _guarded(shape, dt)
    fc.fc_dequantize_mxfp4(codes, scales, shape[-1], dt, out)
    torch.cuda.synchronize()
    check()
    assert torch.equal(out.cpu(), ref.mx_dequantize(*want, shape[-1]).to(dt))


@pytest.mark.parametrize("dt", [BF16, F16])
def test_non_finite_blocks(dt):
    x = torch.randn((4, 160), generator=torch.Generator().manual_seed(1)).to(dt)
    x[0, 5] = float("nan")
    x[1, 40] = float("inf")
    x[2, 159] = -float("inf")
    codes, scales = _quantize(x)
    want = ref.mx_quantize(x.double())
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
    out = fc.fc_dequantize_mxfp4(codes, scales, 160, dt).cpu()
    bad = torch.zeros(4, 160, dtype=torch.bool)
    bad[0, :32], bad[1, 32:64], bad[2, 128:] = True, True, True
    assert torch.equal(torch.isnan(out), bad)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_dequantize_every_code_and_scale(dt):
    """256 code pairs x 256 scales: exact, or rounded once, infinite past the type's range, NaN for 255."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)[None].repeat(256, 1)       # 512 values a row
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 16)
    out = fc.fc_dequantize_mxfp4(codes.cuda(), scales.cuda(), 512, dt).cpu()
    want = ref.mx_dequantize(codes, scales, 512).to(dt)     # at most 2 significant bits: one rounding
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(out[ok].view(torch.int16), want[ok].view(torch.int16))


# (R, T, K, H): single tokens, borders of every token and channel tile, odd sizes, short and long rows
PRODUCTS = [(1, 1, 128, 16), (1, 1, 32, 1), (2, 1, 2048, 512), (1, 2, 100, 7), (3, 5, 384, 33), (1, 8, 4096, 64),
            (4, 13, 640, 130), (1, 15, 256, 65), (2, 16, 1152, 256), (1, 17, 256, 300), (1, 31, 512, 128), (2, 32, 3584, 48),
            (1, 33, 896, 257), (2, 63, 384, 96), (1, 64, 7168, 160), (1, 65, 256, 64), (3, 77, 640, 515), (1, 100, 2176, 1000),
            (1, 127, 1000, 120), (2, 128, 512, 128), (1, 129, 384, 255), (1, 200, 4224, 264), (2, 255, 256, 256),
            (1, 256, 1024, 512), (1, 257, 896, 700), (2, 300, 128, 768), (1, 512, 2048, 1024), (1, 1000, 640, 1000),
            (4, 520, 256, 300), (1, 2048, 256, 2048), (2, 1030, 1152, 1300), (1, 4000, 128, 40), (1, 40, 128, 4000),
            (8, 3, 256, 2050), (1, 700, 96, 5)]


# enough tiles for the 128 and the 256 tile, and for several tiles per workgroup; K an even and an odd
# multiple of 128, shorter and longer than the stages in flight
PRODUCTS += [(4, 520, 256, 1300), (3, 1000, 384, 1160), (8, 600, 1408, 650), (2, 2300, 128, 1700),
             (8, 1300, 384, 1030), (8, 1300, 256, 2100), (4, 2050, 640, 1800), (1, 4000, 128, 3500), (2, 3000, 1408, 2100),
             (4, 100, 384, 4100), (4, 3, 2048, 4100), (2, 16, 1000, 8200)]


def _operands(R, T, K, H, seed, spread):
    g = torch.Generator().manual_seed(seed)
    Kp = -(-K // 128) * 128
    def side(rows):
        codes = torch.randint(0, 256, (R, rows, Kp // 2), generator=g, dtype=torch.uint8)
        codes[..., (K + 1) // 2:] = 0
        if K % 2:
            codes[..., K // 2] &= 15
        scales = torch.randint(127 - spread, 128 + spread, (R, rows, Kp // 32), generator=g).to(torch.uint8)
        scales[..., -(-K // 32):] = 0
        return codes, scales
    return *side(T), *side(H)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("R,T,K,H", PRODUCTS)
def test_product_exact(R, T, K, H, dt):
    """Scales of 1: every product is a multiple of 1/4 and every partial sum below 2^24 of them
    (K * 36 * 4 < 2^24), so binary32 holds the sum exactly in any order."""
    _say(f"product exact R={R} T={T} K={K} H={H} {dt}")
    assert K * 36 * 4 < 2 ** 24
    ac, as_, wc, ws = _operands(R, T, K, H, T + K + H, 0)
    y, check = _guarded((R, T, H), dt)
    fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc.cuda(), ws.cuda(), dt, y)
    torch.cuda.synchronize()
    check()
    want, _ = ref.mx_product(ref.mx_dequantize(ac, as_, K), ref.mx_dequantize(wc, ws, K))
    assert torch.equal(y.cpu(), want.to(torch.float32).to(dt))


# four and more of the 256 tiles per compute unit, and outputs past 128 MiB; rows of an odd length, of one
# that ends inside a tile, and whole ones
@pytest.mark.parametrize("R,T,K,H,dt", [(8, 2900, 640, 2901, BF16), (8, 2900, 1152, 2900, F16), (2, 8100, 256, 4352, BF16),
                                        (3, 1000, 384, 1161, F16), (5, 2500, 128, 2570, F16)])
def test_product_of_many_tiles(R, T, K, H, dt):
    _say(f"product of many tiles R={R} T={T} K={K} H={H} {dt}")
    ac, as_, wc, ws = _operands(R, T, K, H, T + K + H, 0)
    y, check = _guarded((R, T, H), dt)
    fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc.cuda(), ws.cuda(), dt, y)
    torch.cuda.synchronize()
    check()
    a, w = ref.mx_dequantize(ac, as_, K).float(), ref.mx_dequantize(wc, ws, K).float()
    for r in range(R):     # sums that binary32 holds exactly
        assert torch.equal(y[r].cpu(), (a[r] @ w[r].t().contiguous()).to(dt)), f"rank {r}"


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("R,T,K,H", PRODUCTS)
def test_product_scales(R, T, K, H, dt):
    """Scales of 2^-3 to 2^3, each its own: K additions of 2^-24 of the magnitudes' sum, and twice
    that for a matrix core that truncates where it aligns its terms."""
    _say(f"product scales R={R} T={T} K={K} H={H} {dt}")
    ac, as_, wc, ws = _operands(R, T, K, H, 3 * T + K + H, 3)
    y = fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc.cuda(), ws.cuda(), dt)
    torch.cuda.synchronize()
    want, mag = ref.mx_product(ref.mx_dequantize(ac, as_, K), ref.mx_dequantize(wc, ws, K))
    if dt == F16:
        assert want.abs().max() < 65504
    ref.assert_within(y, want, dt, mag * (K * 2.0 ** -23))
    again = fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc.cuda(), ws.cuda(), dt)
    assert torch.equal(y, again)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("R,T,K,H", PRODUCTS)
def test_linear_quantizes_its_activations(R, T, K, H, dt):
    """fc_linear_mxfp4 of integer activations: the product of fc_quantize_mxfp4's codes, exactly."""
    _say(f"linear R={R} T={T} K={K} H={H} {dt}")
    _, _, wc, ws = _operands(R, 1, K, H, K + H, 0)
    g = torch.Generator().manual_seed(T)
    # magnitudes 0..12 and a 4 in every block: scales of 1 or 2, codes rounded and saturated
    a = torch.randint(-12, 13, (R, T, K), generator=g).to(dt)
    a[..., ::32] = 4
    y, check = _guarded((R, T, H), dt)
    fc.fc_linear_mxfp4(a.cuda(), wc.cuda(), ws.cuda(), y)
    torch.cuda.synchronize()
    check()
    ac, as_ = ref.mx_quantize(a.double())
    want, _ = ref.mx_product(ref.mx_dequantize(ac, as_, K), ref.mx_dequantize(wc, ws, K))
    assert K * 72 * 4 < 2 ** 24
    assert torch.equal(y.cpu(), want.to(torch.float32).to(dt))


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_linear_real_activations(T):
    R, K, H = 2, 1000, 200
    g = torch.Generator().manual_seed(T)
    a = torch.randn((R, T, K), generator=g).to(BF16)
    a[:, :, 3] *= 50
    a[0, 0] = 0
    w = torch.randn((R, H, K), generator=g).to(BF16)
    wc, ws = fc.fc_quantize_mxfp4(w.cuda())
    y = fc.fc_linear_mxfp4(a.cuda(), wc, ws)
    q = fc.fc_quantize_mxfp4(a.cuda())
    want, mag = ref.mx_product(ref.mx_dequantize(*(v.cpu() for v in q), K), ref.mx_dequantize(wc.cpu(), ws.cpu(), K))
    ref.assert_within(y, want, BF16, mag * (K * 2.0 ** -23))
    assert (y[0, 0] == 0).all()


@pytest.mark.parametrize("T,H", [(1, 64), (16, 96), (50, 64), (300, 512)])
def test_nan_scales_stay_in_their_row_and_channel(T, H):
    K = 512
    g = torch.Generator().manual_seed(T)
    a = torch.randn((1, T, K), generator=g).to(BF16)
    a[0, T // 2, 400] = float("nan")
    ac, as_, wc, ws = _operands(1, T, K, H, 1, 1)
    ws[0, 7, 3] = 255
    bad = torch.zeros(1, T, H, dtype=torch.bool)
    bad[:, T // 2], bad[..., 7] = True, True
    y = fc.fc_linear_mxfp4(a.cuda(), wc.cuda(), ws.cuda())
    assert torch.equal(torch.isnan(y.cpu()), bad)
    y = fc.fc_matmul_mxfp4(*fc.fc_quantize_mxfp4(a.cuda()), wc.cuda(), ws.cuda(), BF16)
    assert torch.equal(torch.isnan(y.cpu()), bad)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_extreme_scales(T):
    """Products of 2^-127 and 2^120 scales: neither side alone fits a product in range."""
    K, H = 256, 48
    ac, as_, wc, ws = _operands(1, T, K, H, T, 0)
    as_[..., :] = 0
    ws[..., :] = 247
    y = fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc.cuda(), ws.cuda(), BF16)
    want, _ = ref.mx_product(ref.mx_dequantize(ac, as_, K), ref.mx_dequantize(wc, ws, K))
    assert torch.equal(y.cpu(), want.to(torch.float32).to(BF16))


def test_two_dimensional_operands_and_no_tokens():
    ac, as_, wc, ws = (v.cuda() for v in _operands(1, 5, 256, 40, 2, 1))
    y = fc.fc_matmul_mxfp4(ac, as_, wc, ws, BF16)
    y2 = fc.fc_matmul_mxfp4(ac[0], as_[0], wc[0], ws[0], BF16)
    assert y2.shape == (5, 40) and torch.equal(y[0], y2)
    empty = fc.fc_linear_mxfp4(torch.empty((2, 0, 256), dtype=BF16, device="cuda"), wc.repeat(2, 1, 1), ws.repeat(2, 1, 1))
    assert empty.shape == (2, 0, 40)
    c, s = fc.fc_quantize_mxfp4(torch.empty((0, 100), dtype=F16, device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0, 4)


def test_binding_refuses():
    x = torch.randn((4, 256), device="cuda").to(BF16)
    codes, scales = fc.fc_quantize_mxfp4(x)
    for call in [
        lambda: fc.fc_quantize_mxfp4(x.float()), lambda: fc.fc_quantize_mxfp4(x[0]), lambda: fc.fc_quantize_mxfp4(x[:, ::2]),
        lambda: fc.fc_quantize_mxfp4(x.cpu()), lambda: fc.fc_quantize_mxfp4(x, codes=codes[:3]),
        lambda: fc.fc_quantize_mxfp4(x, scales=scales.to(torch.int8)),
        lambda: fc.fc_dequantize_mxfp4(codes, scales, 100, BF16), lambda: fc.fc_dequantize_mxfp4(codes, scales[:3], 256, BF16),
        lambda: fc.fc_dequantize_mxfp4(codes, scales, 256, torch.float32),
        lambda: fc.fc_matmul_mxfp4(codes, scales, codes[None], scales[None], BF16),
        lambda: fc.fc_matmul_mxfp4(codes, scales, codes[:, :64].contiguous(), scales[:, :4].contiguous(), BF16),
        lambda: fc.fc_matmul_mxfp4(codes, scales, codes, scales, BF16, y=torch.empty((4, 5), dtype=BF16, device="cuda")),
        lambda: fc.fc_linear_mxfp4(x.float(), codes, scales), lambda: fc.fc_linear_mxfp4(x[:, :64].contiguous(), codes, scales),
        lambda: fc.fc_linear_mxfp4(x, codes, scales, y=torch.empty((4, 4), dtype=F16, device="cuda")),
    ]:
        with pytest.raises(ValueError):
            call()
    a = torch.randn((300, 256), device="cuda").to(BF16)
    with pytest.raises(fc.FcError) as e:
        fc.fc_linear_mxfp4(a, codes, scales, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    ws = torch.empty(fc.fc_linear_mxfp4_workspace_bytes(1, 300, 256) + 4096, dtype=torch.uint8, device="cuda")
    with pytest.raises(fc.FcError) as e:
        fc.fc_linear_mxfp4(a, codes, scales, y=ws[:2400].view(BF16).view(300, 4), workspace=ws)
    assert e.value.status == 9


def test_other_stream_and_graph_replays():
    R, K, H = 2, 1024, 512
    for T in (4, 300):
        a = torch.randn((R, T, K), device="cuda").to(BF16)
        wc, ws = fc.fc_quantize_mxfp4(torch.randn((R, H, K), device="cuda").to(BF16))
        y = fc.fc_linear_mxfp4(a, wc, ws)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y2 = fc.fc_linear_mxfp4(a, wc, ws, stream=side)
        side.synchronize()
        assert torch.equal(y, y2)
        need = max(fc.fc_linear_mxfp4_workspace_bytes(R, T, K), 1)
        work = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            fc.fc_linear_mxfp4(a, wc, ws, y2, work[0], stream=side)
        torch.cuda.synchronize()
        for i in range(4):
            a.copy_(torch.randn((R, T, K), device="cuda"))
            y2.zero_()
            torch.cuda.synchronize()
            graph.replay()
            fc.fc_linear_mxfp4(a, wc, ws, y, work[1])     # beside the replay, with a workspace of its own
            torch.cuda.synchronize()
            assert torch.equal(y, y2), f"T={T} replay {i}"


def test_more_rows_than_a_grid_row():
    """A grid row of 2^20 workgroups of 512 units of 8 values: rows of 128 (whole) and of 100 (padded)."""
    for K, rows in ((128, (1 << 25) + 70), (100, (1 << 25) + 70)):
        _say(f"quantize {rows} x {K}")
        g = torch.Generator(device="cuda").manual_seed(K)
        x = torch.randn((rows, K), generator=g, device="cuda", dtype=BF16)
        codes, scales = fc.fc_quantize_mxfp4(x)
        out = fc.fc_dequantize_mxfp4(codes, scales, K, BF16)
        torch.cuda.synchronize()
        at = torch.tensor([0, 1, (1 << 25) - 33, (1 << 25) - 1, 1 << 25, (1 << 25) + 32, rows - 1])
        want = ref.mx_quantize(x[at].cpu().double())
        assert torch.equal(codes[at].cpu(), want[0]) and torch.equal(scales[at].cpu(), want[1])
        assert torch.equal(out[at].cpu(), ref.mx_dequantize(*want, K).to(BF16))
        del x, codes, scales, out


def test_linear_of_more_channels_than_a_grid_row():
    """A grid row of 2^20 workgroups of 64 channels: 5 x 2^24 channels take more. Sums of
    128 products of multiples of 1/4 up to 36 are exact in binary32."""
    R, T, K, H = 5, 2, 128, 1 << 24
    _say(f"linear {R} x {T} x {K} x {H}")
    g = torch.Generator(device="cuda").manual_seed(5)
    wc = torch.randint(0, 256, (R, H, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.full((R, H, K // 32), 127, device="cuda", dtype=torch.uint8)
    a = torch.randint(-6, 7, (R, T, K), generator=g, device="cuda").to(BF16)
    y = fc.fc_linear_mxfp4(a, wc, ws)
    torch.cuda.synchronize()
    at = torch.tensor([0, 15, 16, 63, 64, (1 << 23) + 5, H - 65, H - 64, H - 1])
    aq = ref.mx_dequantize(*ref.mx_quantize(a.cpu().double()), K)
    for r in range(R):
        w = ref.mx_dequantize(wc[r, at].cpu(), ws[r, at].cpu(), K)
        assert torch.equal(y[r][:, at].cpu(), (aq[r] @ w.t()).to(BF16)), f"rank {r}"


def test_block_chain_captured():
    """The chain below in a graph, with eager work between the replays."""
    R, T, K, H = 4, 24, 512, 1024
    a = torch.randn((R, T, K), device="cuda").to(BF16)
    wc, ws = fc.fc_quantize_mxfp4(torch.randn((R, H, K), device="cuda").mul_(K ** -0.5).to(BF16))
    vc, vs = fc.fc_quantize_mxfp4(torch.randn((512, H), device="cuda").mul_(H ** -0.5).to(BF16))
    res = torch.randn((T, H), device="cuda").to(BF16)
    w = torch.ones(H, device="cuda", dtype=BF16)

    def buffers():
        e = lambda *s: torch.empty(s, dtype=BF16, device="cuda")
        b = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        return (e(R, T, H), e(T, H), e(T, H), e(T, 512), b(fc.fc_linear_mxfp4_workspace_bytes(R, T, K)),
                b(fc.fc_workspace_bytes(R, T, H, 4, 128)), b(fc.fc_linear_mxfp4_workspace_bytes(1, T, H)))

    def chain(y, h, n, out, w1, w2, w3):
        fc.fc_linear_mxfp4(a, wc, ws, y, w1)
        fc.fc_allreduce_emulated_norm(y, 4, 128, res, w_post=w, w_pre=w, h=h, y=n, workspace=w2)
        fc.fc_linear_mxfp4(n, vc, vs, out, w3)

    eager, captured = buffers(), buffers()
    chain(*eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(*captured)
    torch.cuda.synchronize()
    for i in range(4):
        a.copy_(torch.randn((R, T, K), device="cuda"))
        for v in captured[:4]:
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        chain(*eager)
        torch.cuda.synchronize()
        for e, c in zip(eager[:4], captured[:4]):
            assert torch.equal(e, c), f"replay {i}"


def test_block_chain():
    """The end of a transformer block under tensor parallelism: every rank's MXFP4 projection of its
    slice, the low-bit all-reduce of the partial sums, the residual update and both norms, and the
    next projection -- each step against its 64-bit statement on the step's own input."""
    R, T, K, H, bits, group = 4, 40, 512, 1024, 4, 128
    g = torch.Generator().manual_seed(11)
    a = torch.randn((R, T, K), generator=g).to(BF16)
    w = [torch.randn(s, generator=g).mul(s[-1] ** -0.5).to(BF16).cuda() for s in ((R, H, K), (K, H))]
    (wc, ws), (vc, vs) = (fc.fc_quantize_mxfp4(v) for v in w)
    residual = torch.randn((T, H), generator=g).to(BF16)
    ones = torch.ones(H, dtype=BF16)
    y = fc.fc_linear_mxfp4(a.cuda(), wc, ws)
    stream = residual.cuda()
    h, n, work = fc.fc_allreduce_emulated_norm(y, bits, group, stream, w_post=ones.cuda(), w_pre=ones.cuda(),
                                               gate=0.5 * ones.cuda(), h=stream)
    out = fc.fc_linear_mxfp4(n, vc, vs)
    torch.cuda.synchronize()
    want, mag = ref.mx_product(ref.mx_dequantize(*ref.mx_quantize(a.double()), K), ref.mx_dequantize(wc.cpu(), ws.cpu(), K))
    ref.assert_within(y, want, BF16, mag * (K * 2.0 ** -23), "projection")
    p = fc.workspace_views(work, R, T, H, bits, group)
    x = ref.dequantize(p["codes2"].cpu(), p["s2"].cpu(), p["z2"].cpu(), bits, group)
    # the reduced sum is within the two quantizations' steps of the sum of y
    s1 = p["s1"].cpu().view(torch.float16).double().repeat_interleave(group, -1).sum(0)
    s2 = p["s2"].cpu().view(torch.float16).double().repeat_interleave(group, -1)
    total = y.cpu().double().sum(0)
    assert ((x - total).abs() <= (s1 + s2) / 2 + 2.0 ** -10 * (total.abs() + y.cpu().double().abs().sum(0))).all()
    d = ones.double()
    hr, eh, nr, en = ref.norms(x, residual.double(), d, 0.5 * d, T, d, 1.0, 1.0, 1e-5)
    ref.assert_within(h, hr, BF16, eh, "h")
    ref.assert_within(n, nr, BF16, en, "n")
    q = ref.mx_quantize(n.cpu().double())
    want, mag = ref.mx_product(ref.mx_dequantize(*q, H)[None], ref.mx_dequantize(vc.cpu(), vs.cpu(), H)[None])
    ref.assert_within(out, want[0], BF16, mag[0] * (H * 2.0 ** -23), "next projection")


def test_product_of_the_most_tokens():
    """2^31 - 1 tokens, whose tiles' counts pass 32 bits where they are rounded up: 128 GiB of codes.
    Rows of ones at sampled tokens, zeros elsewhere; w = 1 gives K for the former."""
    T, K, dev = (1 << 31) - 1, 128, "cuda"
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 170 << 30:
        pytest.skip("needs 170 GiB of free device memory")
    _say(f"product of {T} tokens")
    at = torch.tensor([0, 1, 127, 128, (1 << 30) + 5, T - 257, T - 256, T - 129, T - 128, T - 1], device=dev)
    ac = torch.zeros((T, K // 2), dtype=torch.uint8, device=dev)
    as_ = torch.full((T, K // 32), 127, dtype=torch.uint8, device=dev)
    ac[at] = 0x22
    wc = torch.full((1, K // 2), 0x22, dtype=torch.uint8, device=dev)
    ws = torch.full((1, K // 32), 127, dtype=torch.uint8, device=dev)
    y, check = _guarded((T, 1), BF16)
    fc.fc_matmul_mxfp4(ac, as_, wc, ws, BF16, y)
    torch.cuda.synchronize()
    check()
    assert (y[at] == K).all()
    assert int(torch.count_nonzero(y)) == len(at)
    del ac, as_, wc, ws, y, check
    torch.cuda.empty_cache()


# one shape (T, K, H) for each kernel of the product on 256 compute units, but for the many-tile ones
TARGETS = {"split1 of 1 token": (1, 256, 64), "split1 of 32 tokens": (32, 256, 64), "split1 of 64 tokens": (64, 4096, 64),
           "64": (300, 256, 512), "64 in two rounds": (1408, 256, 3200), "128": (1024, 256, 4096), "256": (2176, 256, 4096)}


@pytest.mark.parametrize("target", TARGETS)
def test_small_scales(target):
    """Exponents that sum to e: sums are multiples of 2^(e - 2), which binary32 holds, among them
    subnormal ones, and one rounding takes them to bf16's subnormals. With both scales 2^-127 every
    sum is far below 2^-149: zeros."""
    T, K, H = TARGETS[target]
    ac, as_, wc, ws = _operands(1, T, K, H, 5, 0)
    as_[...] = 0
    for e in (-125, -135, -140, -254):
        _say(f"small scales {target}: 2^{e}")
        ws[...] = e + 254
        y = fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc.cuda(), ws.cuda(), BF16).cpu()
        want, _ = ref.mx_product(ref.mx_dequantize(ac, as_, K), ref.mx_dequantize(wc, ws, K))
        want = want.to(torch.float32).to(BF16)
        assert torch.equal(y, want)
        assert bool((want != 0).any()) == (e != -254)


@pytest.mark.parametrize("target", TARGETS)
@pytest.mark.parametrize("a_byte,w_byte", [(0, 247), (247, 0), (254, 0), (0, 254), (254, 1)])
def test_extreme_scales_in_every_kernel(target, a_byte, w_byte):
    """Neither scale alone leaves a product in binary32's range."""
    T, K, H = TARGETS[target]
    _say(f"extreme scales {target} {a_byte} {w_byte}")
    ac, as_, wc, ws = _operands(1, T, K, H, 6, 0)
    as_[...] = a_byte
    ws[...] = w_byte
    y = fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc.cuda(), ws.cuda(), BF16)
    want, _ = ref.mx_product(ref.mx_dequantize(ac, as_, K), ref.mx_dequantize(wc, ws, K))
    assert torch.equal(y.cpu(), want.to(torch.float32).to(BF16))


# (R, T, H) for each kernel; the last walks many tiles of 256 with the L2 prefetch
NAN_SHAPES = [(1, 1, 64), (1, 50, 64), (1, 64, 130), (1, 300, 512), (1, 1408, 3200), (3, 30, 8260), (1, 1024, 4096),
              (1, 2176, 4096), (2, 1000, 4360), (8, 2900, 2900)]


@pytest.mark.parametrize("R,T,H,K", [(*s, K) for s in NAN_SHAPES for K in (128, 384, 512, 640, 1152)]
                         + [(1, 50, 64, 4096), (1, 64, 130, 4224), (1, 2, 4200, 4224), (2, 16, 2100, 8192)])
def test_nan_scales_in_every_kernel(R, T, H, K):
    """NaN scales in the first and the last block of rows at the tiles' borders make those rows (of a)
    and channels (of w) NaN and no other: the row before one whose first scale is NaN ends in the
    same 16 bytes of scales where K is an odd multiple of 128. Elsewhere y is as without them."""
    _say(f"NaN scales R={R} T={T} K={K} H={H}")
    g = torch.Generator(device="cuda").manual_seed(T + K)
    def side(rows):
        codes = torch.randint(0, 256, (R, rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.randint(126, 129, (R, rows, K // 32), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
        return codes, scales
    ac, as_ = side(T)
    wc, ws = side(H)
    clean = fc.fc_matmul_mxfp4(ac, as_, wc, ws, BF16)
    bad = torch.zeros((R, T, H), dtype=torch.bool, device="cuda")
    def plant(scales, n, at):
        rows = sorted({r for r in at if r < n} | {n - 1}) if n > 1 else []
        for i, r in enumerate(rows):
            scales[i % R, r, 0 if i % 2 == 0 else -1] = 255
        return [(i % R, r) for i, r in enumerate(rows)]
    at = [1, 17, 32, 63, 64, 127, 128, 191, 255, 256, 511, 512, 640]
    for r, t in plant(as_, T, at):
        bad[r, t] = True
    for r, h in plant(ws, H, [c + 1 for c in at] + [2048, 2304]):
        bad[r, :, h] = True
    y, check = _guarded((R, T, H), BF16)
    fc.fc_matmul_mxfp4(ac, as_, wc, ws, BF16, y)
    torch.cuda.synchronize()
    check()
    assert torch.isfinite(clean).all()
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(torch.where(bad, 0.0, y.float()), torch.where(bad, 0.0, clean.float()))


@pytest.mark.parametrize("T,K,H", [(1, 384, 64), (5, 384, 4200), (1, 4224, 4200), (12, 1152, 17000)])
def test_nan_activations_quantized_in_place(T, K, H):
    """fc_linear_mxfp4 where the product quantizes: a NaN activation and NaN scales of w."""
    _say(f"linear NaN T={T} K={K} H={H}")
    g = torch.Generator().manual_seed(T)
    a = torch.randn((1, T, K), generator=g).to(BF16)
    a[0, T // 2, K - 1] = float("nan")
    _, _, wc, ws = _operands(1, 1, K, H, 1, 1)
    bad = torch.zeros(1, T, H, dtype=torch.bool)
    bad[:, T // 2] = True
    for h, block in ((1, 0), (16, -1), (H - 1, 0)):
        ws[0, h, block] = 255
        bad[..., h] = True
    assert fc.fc_linear_mxfp4_workspace_bytes(1, T, K) == 0
    y, check = _guarded((1, T, H), BF16)
    fc.fc_linear_mxfp4(a.cuda(), wc.cuda(), ws.cuda(), y)
    torch.cuda.synchronize()
    check()
    assert torch.equal(torch.isnan(y.cpu()), bad)


# Tiles of 64 two to a compute unit, more of them than fit the device at once, whole and odd multiples of
# 128, one and several stages; the same of the tiles of 128 and 256; split waves in two rounds, with each number of token blocks
SMALL_TILES = [(1, 1408, 128, 3200), (1, 1408, 384, 3200), (1, 1350, 1000, 3230), (1, 1390, 1280, 3137), (4, 40, 384, 8300),
               (4, 64, 896, 8257), (9, 3, 256, 4100), (9, 50, 640, 4101), (3, 17, 1408, 12000)]
LARGE_TILES = [(2, 2300, 512, 1700), (2, 2300, 1280, 1702), (8, 1300, 512, 2100), (8, 1300, 384, 2101)]
TWO_ROUNDS = [(1, 1, 4096, 4200), (1, 3, 4100, 8192), (2, 16, 8320, 2100), (1, 13, 8192, 4097), (1, 24, 4352, 8191), (2, 20, 4100, 4096)]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("R,T,K,H", SMALL_TILES + LARGE_TILES + TWO_ROUNDS)
def test_product_and_linear_in_every_kernel(R, T, K, H, dt):
    """Both calls where the sums are exact (K * 36 * 4 and, with activations that quantize to
    magnitudes of up to 12, K * 72 * 4 below 2^24 quarters)."""
    _say(f"every kernel R={R} T={T} K={K} H={H} {dt}")
    assert K * 72 * 4 < 2 ** 24
    ac, as_, wc, ws = _operands(R, T, K, H, T + K + H, 0)
    w = ref.mx_dequantize(wc, ws, K).float()
    wc, ws = wc.cuda(), ws.cuda()
    y, check = _guarded((R, T, H), dt)
    fc.fc_matmul_mxfp4(ac.cuda(), as_.cuda(), wc, ws, dt, y)
    torch.cuda.synchronize()
    check()
    a = ref.mx_dequantize(ac, as_, K).float()
    for r in range(R):     # sums that binary32 holds exactly
        assert torch.equal(y[r].cpu(), (a[r] @ w[r].t().contiguous()).to(dt)), f"rank {r}"
    g = torch.Generator().manual_seed(T)
    x = torch.randint(-12, 13, (R, T, K), generator=g).to(dt)
    x[..., ::32] = 4
    y, check = _guarded((R, T, H), dt)
    fc.fc_linear_mxfp4(x.cuda(), wc, ws, y)
    torch.cuda.synchronize()
    check()
    a = ref.mx_dequantize(*ref.mx_quantize(x.double()), K).float()
    for r in range(R):
        assert torch.equal(y[r].cpu(), (a[r] @ w[r].t().contiguous()).to(dt)), f"rank {r}"


def test_host_threads_on_streams_of_their_own():
    """Four threads at once, each on its stream with tensors of its own: the chain of norms, quantizing
    linear layers (few tokens and tiles) and the all-reduce gives what it gives alone."""
    import threading

    R, K, H = 2, 1024, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    wc, ws = fc.fc_quantize_mxfp4(n(R, H, K))
    gain = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16)

    def chain(a, res, stream=None):
        y = fc.fc_linear_mxfp4(a, wc, ws, stream=stream)
        h, v, _ = fc.fc_allreduce_emulated_norm(y, 4, 128, res, w_post=gain, w_pre=gain, stream=stream)
        h2, v2 = fc.fc_residual_norm(v, h, w_pre=gain, stream=stream)
        codes, scales = fc.fc_quantize_mxfp4(v2, stream=stream)
        return y, h, v, h2, v2, fc.fc_dequantize_mxfp4(codes, scales, H, BF16, stream=stream)

    inputs = [(n(R, T, K), n(T, H)) for T in (1, 5, 200, 700)]
    want = [chain(*i) for i in inputs]
    torch.cuda.synchronize()
    got, errors = [None] * len(inputs), []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got[i] = chain(*inputs[i], stream=stream)
            stream.synchronize()
        except Exception as e:     # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(inputs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
