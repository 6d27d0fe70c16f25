"""Linear layers with their epilogue, their gradients, and the activation's backward
pass on the GPU against their 64-bit statements (tests/train_ref.py): sizes at the
tiles' borders and odd ones, every activation, payload groups that end inside a
chunk's neighbours, long sums, no tokens, and one training step of a block's MLP with
all of them."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc
import train_ref as ref
from test_gpu_layer_norm import Guarded

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
ACTS = list(fc.ACTIVATIONS)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    fc.lib()
    yield


def _say(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


def _on(t):
    if isinstance(t, tuple):
        return tuple(x.cuda() for x in t)
    return None if t is None else t.cuda()


def _64(t):
    return None if t is None else t.double()


def _layer(R, T, K, H, dt, seed, bias=True, mul=True, skip=True):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(dt)
    return dict(a=n(R, T, K), w=n(R, H, K, scale=K ** -0.5), bias=n(R, H) if bias else None,
                mul=n(R, T, H) if mul else None, residual=n(R, T, H, scale=2.0) if skip else None)


def _check_linear(d, act, dt, what="", **kw):
    R, T, H = d["a"].shape[0], d["a"].shape[1], d["w"].shape[1]
    y, z = Guarded((R, T, H), dt), Guarded((R, T, H), dt)
    fc.fc_linear_act(_on(d["a"]), _on(d["w"]), _on(d["bias"]), act, mul=_on(d["mul"]), residual=_on(d["residual"]),
                     y=y.t, z=z.t, **kw)
    torch.cuda.synchronize()
    ry, ey, rz, ez = ref.linear(*(_64(d[k]) for k in ("a", "w", "bias")), act, _64(d["mul"]), _64(d["residual"]))
    ref.assert_within(z.t, rz, dt, ez, what + " z")
    ref.assert_within(y.t, ry, dt, ey, what + " y")
    y.check()
    z.check()


# (R, T, K, H): one token to many tiles of every kernel, sizes that no vector divides
SHAPES = [(1, 1, 1, 1), (1, 1, 8, 16), (1, 1, 4096, 256), (2, 1, 100, 48), (1, 2, 64, 33), (3, 5, 7, 9), (1, 8, 1024, 520),
          (1, 15, 200, 130), (1, 16, 512, 64), (4, 17, 96, 200), (1, 31, 2048, 40), (1, 33, 72, 1000), (2, 64, 640, 128),
          (1, 65, 65, 65), (1, 100, 1000, 127), (1, 127, 129, 257), (1, 128, 64, 256), (2, 129, 520, 384), (1, 200, 24, 8),
          (1, 256, 128, 256), (1, 257, 136, 264), (1, 333, 1001, 511), (1, 512, 64, 1024), (1, 700, 192, 768),
          (3, 300, 264, 520), (1, 1100, 56, 72), (1, 2050, 520, 300), (1, 1024, 1024, 2048), (1, 64, 8192, 64)]


# (R, T, K, H) of the largest tiles: whole rounds of them, and columns or rows left to
# smaller ones; ragged ones; a single stage, few and many; several ranks
LARGE_SHAPES = [(1, 4096, 200, 4096), (1, 8192, 72, 2816), (1, 2816, 136, 8192), (2, 2050, 64, 4104), (1, 4000, 1032, 4100),
                (4, 2048, 8, 2048), (1, 1500, 512, 4096), (1, 3300, 264, 3304)]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("R,T,K,H", LARGE_SHAPES)
def test_large_tiles(R, T, K, H, dt):
    """The linear layer, and the input gradient of a layer of H inputs and K outputs."""
    _say(f"large tiles {R}x{T}x{K}x{H} {dt}")
    d = _layer(R, T, K, H, dt, T + K, bias=True, mul=False, skip=True)
    _check_linear(d, "none", dt)
    w = d["w"].transpose(-1, -2).contiguous()
    dx = Guarded((R, T, H), dt)
    fc.fc_linear_input_grad(_on(d["a"]), _on(w), residual=_on(d["residual"]), dx=dx.t)
    want, bound = ref.product(d["a"].double(), w.double())
    want = want + d["residual"].double()
    ref.assert_within(dx.t, want, dt, bound + 4 * ref.U * (want.abs() + d["residual"].double().abs()), "dx")
    dx.check()


@pytest.mark.parametrize("stages", [1, 2, 3, 4, 7])
def test_large_tiles_of_few_stages(stages):
    """The first stages of the largest tiles, when their loads are the farthest behind: operands
    of small whole numbers, whose sums are exact, that no cache holds any more. What reads a
    stage before its last load has landed gives another sum."""
    T = H = 4096
    K = 64 * stages
    g = torch.Generator(device="cuda").manual_seed(stages)
    sets = [tuple(torch.randint(-2, 3, (1, n, K), generator=g, device="cuda").to(F16) for n in (T, H)) for _ in range(4)]
    flush = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    for i, (a, w) in enumerate(sets):
        _say(f"few stages {stages}, operands {i}")
        flush.fill_(float(i))
        y, _ = fc.fc_linear_act(a, w)
        # whole numbers of at most 4 * 448 < 2048: exact in binary32 and in fp16
        assert torch.equal(y[0].float(), a[0].float() @ w[0].float().T)


LARGE_WEIGHTS = [(200, 4096, 4096, 128), (72, 2816, 8192, 88), (130, 8192, 2816, 64), (65, 4104, 4096, 24), (40000, 64, 512, 64),
                 (5000, 512, 520, 8), (300, 2048, 2048, 32), (9000, 1024, 300, 16), (9000, 1032, 304, 24)]


@pytest.mark.parametrize("T,K,H,group", LARGE_WEIGHTS)
def test_weight_grad_large_tiles(T, K, H, group):
    """Many outputs: the values are made before the product, also from groups that are no
    power of two; summed into a gradient as well."""
    _say(f"weight grad large tiles {T}x{K}x{H} g={group}")
    dy = torch.randn(1, T, H, generator=torch.Generator().manual_seed(T)).to(BF16)
    payload = _payload(1, T, K, group, BF16, T)
    args = (_on(dy), _on(payload))
    dw = fc.fc_linear_weight_grad(*args)
    x = ref.held(payload, group).float().to(BF16).double()
    want, bound = ref.product(dy.double().transpose(-1, -2).contiguous(), x)
    ref.assert_f32(dw, want, bound, "dw")
    start = torch.randn(1, H, K, generator=torch.Generator().manual_seed(2))
    summed = fc.fc_linear_weight_grad(*args, dw=start.cuda(), accumulate=True)
    ref.assert_f32(summed, want + start.double(), bound + 2 * ref.U * (want.abs() + start.double().abs()), "dw summed")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("R,T,K,H", SHAPES)
def test_linear_shapes(R, T, K, H, dt):
    _say(f"linear {R}x{T}x{K}x{H} {dt}")
    _check_linear(_layer(R, T, K, H, dt, T + K + H), "silu", dt)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,H", [(3, 64, 72), (130, 48, 136), (130, 47, 131)])
def test_linear_activations(T, K, H, act, dt):
    """Weights large enough for pre-activations of -30 to 30."""
    _say(f"linear {act} {T}x{K}x{H} {dt}")
    d = _layer(1, T, K, H, dt, 5, mul=False, skip=False)
    d["w"] = (d["w"].float() * 8).to(dt)
    _check_linear(d, act, dt)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("mul", [False, True])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("T,K,H", [(4, 128, 160), (140, 128, 160), (140, 127, 161)])
def test_linear_optional_parts(T, K, H, bias, mul, skip):
    d = _layer(2, T, K, H, BF16, 6, bias, mul, skip)
    _check_linear(d, "gelu", BF16)
    y, z = fc.fc_linear_act(*(_on(d[k]) for k in ("a", "w", "bias")), "gelu", mul=_on(d["mul"]), residual=_on(d["residual"]))
    assert z is None
    full, _ = fc.fc_linear_act(*(_on(d[k]) for k in ("a", "w", "bias")), "gelu", mul=_on(d["mul"]), residual=_on(d["residual"]), z=True)
    assert torch.equal(y, full)


@pytest.mark.parametrize("T,K,H", [(1, 256, 512), (40, 96, 136), (300, 264, 520), (300, 263, 521)])
def test_linear_in_place_residual_and_two_dimensions(T, K, H):
    d = _layer(1, T, K, H, BF16, 7)
    two = {k: _on(v[0]) for k, v in d.items()}
    three, _ = fc.fc_linear_act(_on(d["a"]), _on(d["w"]), _on(d["bias"]), "relu", mul=_on(d["mul"]), residual=_on(d["residual"]))
    y, _ = fc.fc_linear_act(two["a"], two["w"], two["bias"], "relu", mul=two["mul"], residual=two["residual"], y=two["residual"])
    assert y.shape == (T, H) and y.data_ptr() == two["residual"].data_ptr()
    assert torch.equal(y, three[0])


@pytest.mark.parametrize("T,K,H", [(2, 128, 64), (20, 64, 136), (200, 264, 264), (200, 131, 264)])
def test_linear_nan_and_infinities_follow_the_formulas(T, K, H):
    """A NaN or an infinity of a token stays in its row, of a channel in its column; relu keeps a NaN."""
    d = _layer(1, T, K, H, BF16, 8, mul=False, skip=False)
    d["a"][0, 1, 3] = float("nan")
    d["w"][0, 5, K - 1] = float("inf")
    d["bias"][0, 9] = float("-inf")
    y, z = fc.fc_linear_act(_on(d["a"]), _on(d["w"]), _on(d["bias"]), "relu", z=True)
    y, z = y.cpu()[0], z.cpu()[0]
    assert torch.isnan(y[1]).all() and torch.isnan(z[1]).all()
    rows = [t for t in range(T) if t != 1]
    assert torch.isinf(z[rows, 5]).all() and (y[rows, 5] == z[rows, 5].clamp_min(0)).all()
    assert (z[rows, 9] == float("-inf")).all() and (y[rows, 9] == 0).all()
    cols = [h for h in range(H) if h not in (5, 9)]
    assert torch.isfinite(y[rows][:, cols]).all()


GRAD_SHAPES = [(1, 1, 8, 8), (1, 1, 256, 512), (2, 3, 40, 24), (1, 16, 64, 1000), (1, 33, 72, 65), (3, 65, 128, 100),
               (1, 100, 264, 127), (1, 128, 256, 64), (2, 129, 136, 200), (1, 257, 520, 264), (1, 300, 1000, 33),
               (1, 511, 64, 513), (1, 700, 768, 192), (1, 2000, 24, 16), (1, 1030, 1032, 520), (1, 130, 56, 2048),
               (1, 1100, 1024, 1000)]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("R,T,K,H", GRAD_SHAPES + [(1, 5, 7, 9), (1, 130, 131, 133), (1, 1, 1, 1), (2, 90, 301, 64)])
def test_input_grad_shapes(R, T, K, H, skip, dt):
    _say(f"input grad {R}x{T}x{K}x{H} {dt} skip={skip}")
    g = torch.Generator().manual_seed(T + K + H)
    dy = torch.randn(R, T, H, generator=g).to(dt)
    w = (torch.randn(R, H, K, generator=g) * H ** -0.5).to(dt)
    res = torch.randn(R, T, K, generator=g).to(dt) if skip else None
    dx = Guarded((R, T, K), dt)
    fc.fc_linear_input_grad(_on(dy), _on(w), residual=_on(res), dx=dx.t)
    want, bound = ref.product(dy.double(), w.double())
    if skip:
        want = want + res.double()
        bound = bound + 4 * ref.U * (want.abs() + res.double().abs())
    ref.assert_within(dx.t, want, dt, bound, "dx")
    dx.check()
    if skip:
        stream = _on(res)
        assert torch.equal(fc.fc_linear_input_grad(_on(dy), _on(w), residual=stream, dx=stream), dx.t)


def _payload(R, T, K, group, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R, T, K, generator=g) * 2 + 0.5).to(dt)
    return ref.quantized(x, group)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("i", range(len(GRAD_SHAPES)))
def test_weight_grad_shapes(i, dt):
    R, T, K, H = GRAD_SHAPES[i]
    group = [g for g in (8, 24, 40, 128, 32, 16, K) if K % g == 0][i % 2]
    _say(f"weight grad {R}x{T}x{K}x{H} g={group} {dt}")
    dy = torch.randn(R, T, H, generator=torch.Generator().manual_seed(i)).to(dt)
    payload = _payload(R, T, K, group, dt, i)
    dw = Guarded((R, H, K), torch.float32)
    args = (_on(dy), _on(payload))
    fc.fc_linear_weight_grad(*args, dw=dw.t)
    x = ref.held(payload, group).float().to(dt).double()      # rounded as fc_dequantize does
    want, bound = ref.product(dy.double().transpose(-1, -2).contiguous(), x)
    ref.assert_f32(dw.t, want, bound, "dw")
    dw.check()
    assert torch.equal(fc.fc_linear_weight_grad(*args), dw.t)
    start = torch.randn(R, H, K, generator=torch.Generator().manual_seed(1))
    summed = fc.fc_linear_weight_grad(*args, dw=start.cuda(), accumulate=True)
    ref.assert_f32(summed, want + start.double(), bound + 2 * ref.U * (want.abs() + start.double().abs()), "dw summed")


LONG_SUMS = [(5000, 64, 40, 8), (33000, 128, 72, 32), (20011, 520, 136, 104), (70001, 8, 8, 8), (9000, 264, 129, 24)]


@pytest.mark.parametrize("T,K,H,group", LONG_SUMS)
def test_weight_grad_long_sums(T, K, H, group):
    """Few outputs and many tokens: the sums are split, and joined in a fixed order."""
    _say(f"weight grad T={T} {K}x{H} g={group}")
    dy = torch.randn(1, T, H, generator=torch.Generator().manual_seed(T)).to(BF16)
    payload = _payload(1, T, K, group, BF16, T)
    args = (_on(dy), _on(payload))
    start = torch.randn(1, H, K, generator=torch.Generator().manual_seed(2))
    dw = fc.fc_linear_weight_grad(*args)
    x = ref.held(payload, group).float().to(BF16).double()
    want, bound = ref.product(dy.double().transpose(-1, -2).contiguous(), x)
    ref.assert_f32(dw, want, bound, "dw")
    summed = fc.fc_linear_weight_grad(*args, dw=start.cuda(), accumulate=True)
    ref.assert_f32(summed, want + start.double(), bound + 2 * ref.U * (want.abs() + start.double().abs()), "dw summed")
    assert torch.equal(fc.fc_linear_weight_grad(*args), dw)


def test_weight_grad_values_are_the_dequantizer_s():
    """One token with dy = 1: dw is the 16-bit value of each code."""
    for dt in (BF16, F16):
        payload = _on(_payload(1, 1, 1024, 32, dt, 3))
        dw = fc.fc_linear_weight_grad(torch.ones(1, 1, 8, dtype=dt, device="cuda"), payload)
        x = fc.fc_dequantize(payload[0][0], payload[1][0], payload[2][0], 1, 1024, 8, 32, dt)
        assert torch.equal(dw[0], x.float().expand(8, 1024))


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("mul", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("R,T,H,group", [(1, 1, 8, 8), (2, 37, 96, 24), (1, 300, 1032, 8)])
def test_activation_backward(R, T, H, group, act, bias, mul, dt):
    _say(f"activation backward {act} {R}x{T}x{H} g={group} {dt}")
    g = torch.Generator().manual_seed(T + H)
    dy = torch.randn(R, T, H, generator=g).to(dt)
    z = torch.randn(R, T, H, generator=g) * 3
    z[..., ::7] *= 4                                 # far out on both sides
    pz = ref.quantized(z.to(dt), group)
    pm = ref.quantized(torch.randn(R, T, H, generator=g).to(dt), group) if mul else None
    dz, dm, db = Guarded((R, T, H), dt), Guarded((R, T, H), dt), Guarded((R, H), torch.float32)
    got = fc.fc_activation_backward(_on(dy), act, _on(pz), mul=_on(pm), dz=dz.t, dmul=dm.t if mul else None, db=db.t if bias else None)
    assert (got[1] is None) == (not mul) and (got[2] is None) == (not bias)
    r = ref.activation_backward(dy.double(), ref.held(pz, group), act, ref.held(pm, group) if mul else None)
    ref.assert_within(dz.t, r["dz"], dt, r["edz"], "dz")
    if mul:
        ref.assert_within(dm.t, r["dmul"], dt, r["edmul"], "dmul")
    if bias:
        ref.assert_f32(db.t, r["db"], r["edb"], "db")
    for t in (dz, dm, db):
        t.check()
    over = _on(dy)
    again = fc.fc_activation_backward(over, act, _on(pz), mul=_on(pm), dz=over, bias=bias)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("R,T,H,group", [(1, 5000, 64, 16), (3, 2000, 520, 40), (1, 700, 8192, 128), (1, 3, 16384, 64), (40, 7, 24, 8)])
def test_activation_backward_sizes(R, T, H, group):
    _say(f"activation backward {R}x{T}x{H}")
    g = torch.Generator().manual_seed(R + T)
    dy = torch.randn(R, T, H, generator=g).to(BF16)
    pz = ref.quantized(torch.randn(R, T, H, generator=g).to(BF16), group)
    dz, _, db = fc.fc_activation_backward(_on(dy), "gelu_tanh", _on(pz), bias=True)
    r = ref.activation_backward(dy.double(), ref.held(pz, group), "gelu_tanh", None)
    ref.assert_within(dz, r["dz"], BF16, r["edz"], "dz")
    ref.assert_f32(db, r["db"], r["edb"], "db")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("R,T,H", [(1, 1, 1), (1, 3, 5), (2, 100, 7), (1, 4000, 9), (1, 513, 1001), (3, 2000, 64), (1, 300, 70001)])
def test_bias_grad(R, T, H, dt):
    _say(f"bias grad {R}x{T}x{H}")
    dy = torch.randn(R, T, H, generator=torch.Generator().manual_seed(T + H)).to(dt)
    db = Guarded((R, H), torch.float32)
    assert fc.fc_activation_backward(_on(dy), "none", db=db.t)[:2] == (None, None)
    r = ref.activation_backward(dy.double(), torch.zeros(R, T, H, dtype=torch.float64), "none", None)
    ref.assert_f32(db.t, r["db"], r["edb"], "db")
    db.check()


def test_no_tokens():
    e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")
    pay = lambda *s: (e(*s, dt=torch.uint8), e(*s[:-1], s[-1] // 8, dt=torch.uint16), e(*s[:-1], s[-1] // 8, dt=torch.uint16))
    w = torch.ones(2, 16, 24, dtype=BF16, device="cuda")
    y, z = fc.fc_linear_act(e(2, 0, 24), w, act="gelu", z=True)
    assert y.shape == (2, 0, 16) and z.shape == (2, 0, 16)
    assert fc.fc_linear_input_grad(e(2, 0, 16), w).shape == (2, 0, 24)
    ones = torch.ones(2, 16, 24, device="cuda")
    assert (fc.fc_linear_weight_grad(e(2, 0, 16), pay(2, 0, 24), dw=ones, accumulate=True) == 1).all()
    assert (fc.fc_linear_weight_grad(e(2, 0, 16), pay(2, 0, 24), dw=ones) == 0).all()
    db = torch.ones(2, 24, device="cuda")
    fc.fc_activation_backward(e(2, 0, 24), "silu", pay(2, 0, 24), db=db)
    assert (db == 0).all()


# --- sizes past 32 bits and grids past 2^20 workgroups -------------------------

def _codes(*shape, group):
    g = torch.Generator(device="cuda").manual_seed(3)
    c = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
    s = (torch.rand(*shape[:-1], shape[-1] // group, device="cuda", generator=g) * 0.02 + 0.01).half()
    return c, s.view(torch.uint16), (-128 * s).view(torch.uint16)


def _big(*shape):
    return torch.randn(shape, dtype=BF16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))


def test_operands_of_more_than_2_to_32_bytes():
    """300000 rows of 8192, checked at both ends."""
    T, H = 300000, 8192
    ends = [slice(0, 3), slice(T - 5, T)]
    x, w = _big(T, H), _big(H)
    _say("large norm")
    y, mean, rstd, payload = fc.fc_layer_norm(x, w, None, stats=True, group=512)
    for e in ends:
        r = ref.layer_norm(x[e].cpu().double(), w.cpu().double(), None, 1e-5, False)
        ref.assert_within(y[e], r["y"], BF16, r["ey"], "y")
        ref.assert_f32(rstd[e], r["rstd"], r["erstd"], "rstd")
        ref.assert_f32(mean[e], r["mean"], r["emean"], "mean")
        for got, want in zip(payload, ref.quantized(x[e].cpu(), 512)):
            assert torch.equal(got[e].cpu().contiguous().view(torch.uint8), want.view(torch.uint8))
    _say("large norm backward")
    dx, dw, db = fc.fc_layer_norm_backward(y, payload, mean, rstd, w)
    for e in ends:
        held = ref.held(tuple(t[e].cpu().contiguous() for t in payload), 512)
        r = ref.layer_norm_backward(y[e].cpu().double(), held, mean[e].cpu().double(), rstd[e].cpu().double(), w.cpu().double(), None)
        ref.assert_within(dx[e], r["dx"], BF16, r["edx"], "dx")
    for c in (0, H - 2):
        n = ((payload[0][:, c:c + 2].double() * payload[1].view(torch.float16)[:, [c // 512]].double()
              + payload[2].view(torch.float16)[:, [c // 512]].double()) - mean[:, None].double()) * rstd[:, None].double()
        d = y[:, c:c + 2].double()
        # each product is off by 4 roundings, the sum by its additions
        bound = (ref.chain(T) + 4) * ref.U * (d * n).abs().sum(0) + 4 * ref.U * d.abs().sum(0)
        assert ((dw[c:c + 2].double() - (d * n).sum(0)).abs() <= bound).all()
        assert ((db[c:c + 2].double() - d.sum(0)).abs() <= ref.chain(T) * ref.U * d.abs().sum(0)).all()
    del dx, x
    _say("large activation backward")
    dz, _, db = fc.fc_activation_backward(y, "relu", payload, bias=True)
    for e in ends:
        de = fc.fc_activation_backward(y[e].contiguous(), "relu", tuple(t[e].contiguous() for t in payload))[0]
        assert torch.equal(dz[e], de)
    del dz, payload
    _say("large input grad")
    w2, r2 = _big(64, H), _big(T, 64)
    dx = fc.fc_linear_input_grad(r2, w2)
    for e in ends:
        assert torch.equal(dx[e], fc.fc_linear_input_grad(r2[e].contiguous(), w2))
    del dx
    _say("large linear")
    a2 = _big(T, 64)
    out, _ = fc.fc_linear_act(a2, w2.t().contiguous())
    for e in ends:
        # few tokens of 64 k: the same order of sums in both kernels
        want = (a2[e].double() @ w2.double())
        assert ((out[e].double() - want).abs() <= 2.0 ** -8 * want.abs() + 136 * ref.U * (a2[e].double().abs() @ w2.double().abs())).all()
    del out
    _say("large weight grad")
    p = _codes(T, 64, group=32)
    dw = fc.fc_linear_weight_grad(y, p)
    v = fc.fc_dequantize(p[0], p[1], p[2], T, 64, 8, 32, BF16).double()
    for e in (slice(0, 4), slice(H - 4, H)):
        d = y[:, e].double().t().contiguous()
        assert ((dw[e].double() - d @ v).abs() <= (2 * T + 8) * ref.U * (d.abs() @ v.abs())).all()


@pytest.mark.parametrize("T", [1, 40])
def test_weights_of_more_than_2_to_32_bytes(T):
    H, K = 300000, 8192
    w, a = _big(H, K), _big(T, K)
    _say(f"large weights T={T}")
    y, _ = fc.fc_linear_act(a, w)
    for e in (slice(0, 5), slice(H - 5, H)):
        want, mag = a.double() @ w[e].double().t(), a.double().abs() @ w[e].double().abs().t()
        assert ((y[:, e].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2 * K + 4) * ref.U * mag).all()


def test_grids_of_more_than_2_to_20_workgroups():
    R = (1 << 20) + 77
    _say("many ranks, few tokens")
    a, w = _big(R, 1, 8), _big(R, 16, 8)
    y, _ = fc.fc_linear_act(a, w)
    tail = slice(R - 100, R)
    assert torch.equal(y[tail], fc.fc_linear_act(a[tail].clone(), w[tail].clone())[0])
    _say("many ranks, input and weight gradients")
    dy = _big(R, 9, 16)
    dx = fc.fc_linear_input_grad(dy, w)
    assert torch.equal(dx[tail], fc.fc_linear_input_grad(dy[tail].clone(), w[tail].clone()))
    p = _codes(R, 9, 8, group=8)
    dw = fc.fc_linear_weight_grad(dy, p)
    assert torch.equal(dw[tail], fc.fc_linear_weight_grad(dy[tail].clone(), tuple(t[tail].clone() for t in p)))
    _say("many ranks, activation backward")
    dz, _, db = fc.fc_activation_backward(dx, "silu", p, bias=True)
    dze, _, dbe = fc.fc_activation_backward(dx[tail].clone(), "silu", tuple(t[tail].clone() for t in p), bias=True)
    assert torch.equal(dz[tail], dze) and torch.equal(db[tail], dbe)
    _say("many rows of a norm")
    for rows, H in ((R, 520), (4 * R, 512)):
        x = _big(rows, H)
        y = fc.fc_layer_norm(x)[0]
        r = ref.layer_norm(x[-50:].cpu().double(), None, None, 1e-5, False)
        ref.assert_within(y[-50:], r["y"], BF16, r["ey"], "y")


def test_streams_do_not_share_workspaces():
    """Split products, weight and bias gradients on two streams at once, many times."""
    d = _layer(1, 40, 4096, 128, BF16, 21)
    dy, p = _big(6000, 128), _codes(6000, 64, group=16)
    calls = [lambda: fc.fc_linear_act(*(_on(d[k]) for k in ("a", "w", "bias")), "gelu")[0],
             lambda: fc.fc_linear_weight_grad(dy, p), lambda: fc.fc_activation_backward(dy, "none", bias=True)[2]]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([c() for c in calls])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


class _Block:
    """A pre-norm MLP block, x + W2 gelu(W1 norm(x) + b1) + b2, whose backward pass has the
    INT8 payloads of x, of the pre-activations and of W2's input alone."""

    def __init__(self, T, H, F, dt, seed):
        g = torch.Generator().manual_seed(seed)

        def n(*shape, scale=1.0):
            return (torch.randn(shape, generator=g) * scale).to(dt).cuda()
        self.x, self.dout = n(T, H, scale=2.0), n(T, H)
        self.w, self.b = (1 + n(H, scale=0.2).float()).to(dt), n(H, scale=0.1)
        self.w1, self.b1 = n(F, H, scale=H ** -0.5), n(F, scale=0.5)
        self.w2, self.b2 = n(H, F, scale=F ** -0.5), n(H, scale=0.5)

    def step(self, group):
        n, mean, rstd, px = fc.fc_layer_norm(self.x, self.w, self.b, stats=True, group=group)
        act, z = fc.fc_linear_act(n, self.w1, self.b1, "gelu", z=True)
        pz = tuple(t[0] for t in fc.fc_quantize_groups(z[None], 8, group))
        pact = tuple(t[0] for t in fc.fc_quantize_groups(act[None], 8, group))
        pn = tuple(t[0] for t in fc.fc_quantize_groups(n[None], 8, group))
        out, _ = fc.fc_linear_act(act, self.w2, self.b2, residual=self.x)
        db2 = fc.fc_activation_backward(self.dout, "none", bias=True)[2]
        dw2 = fc.fc_linear_weight_grad(self.dout, pact)
        dact = fc.fc_linear_input_grad(self.dout, self.w2)
        dz, _, db1 = fc.fc_activation_backward(dact, "gelu", pz, bias=True)
        dw1 = fc.fc_linear_weight_grad(dz, pn)
        dn = fc.fc_linear_input_grad(dz, self.w1)
        dx, dw, db = fc.fc_layer_norm_backward(dn, px, mean, rstd, self.w, dres=self.dout)
        return dict(out=out, dx=dx, w=dw, b=db, w1=dw1, b1=db1, w2=dw2, b2=db2)

    def reference(self):
        leaves = {k: getattr(self, k).cpu().double().requires_grad_() for k in ("x", "w", "b", "w1", "b1", "w2", "b2")}
        x = leaves["x"]
        c = x - x.mean(-1, keepdim=True)
        n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * leaves["w"] + leaves["b"]
        z = n @ leaves["w1"].t() + leaves["b1"]
        out = x + (z * torch.special.ndtr(z)) @ leaves["w2"].t() + leaves["b2"]
        out.backward(self.dout.cpu().double())
        r = {k: v.grad for k, v in leaves.items()}
        r["dx"] = r.pop("x")
        r["out"] = out.detach()
        return r


@pytest.mark.parametrize("T,H,F,group,dt", [(64, 128, 256, 32, BF16), (300, 256, 512, 64, F16), (77, 520, 1040, 8, BF16)])
def test_training_step_against_autograd(T, H, F, group, dt):
    """64-bit gradients of the uncompressed block. Each saved value is off by at most half a
    code step, (max - min) / 510 of its group, plus the rounding of its zero and scale: for
    groups of normal values of at most 256 that is under 1 / 60 of their deviation; and it
    is independent from value to value. A gradient that sums over them is off by a few
    percent of its root mean square, elementwise ones by a few percent of it too."""
    block = _Block(T, H, F, dt, T)
    got, want = block.step(group), block.reference()
    for k, w in want.items():
        err = (got[k].cpu().double() - w).square().mean().sqrt() / w.square().mean().sqrt()
        assert err < 0.03, (k, err.item())


def test_training_step_captured():
    block = _Block(96, 256, 512, BF16, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block.step(32)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.step(32)
    for turn in range(4):
        block.x.copy_(torch.randn(96, 256, generator=torch.Generator().manual_seed(turn)).to(BF16))
        block.dout.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        want = block.step(32)
        for k in out:
            assert torch.equal(out[k], want[k]), (turn, k)
