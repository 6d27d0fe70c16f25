"""Layer and RMS norm and their backward pass on the GPU against their 64-bit
statements (tests/train_ref.py): rows of every kind the kernels split differently,
both sources of the saved activations, gradients of shared weights over few and many
rows, and what lies around an output."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc
import train_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    fc.lib()
    yield


def _say(msg):
    print(f"[gpu] {msg}", file=sys.stderr, flush=True)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _inputs(T, H, dt, seed, offset=1.0):
    g = _gen(seed)
    x = torch.randn(T, H, generator=g) + offset * torch.randn(T, 1, generator=g)
    x[:, :: max(1, H // 3)] *= 8
    return dict(x=x.to(dt), w=(1 + 0.3 * torch.randn(H, generator=g)).to(dt), b=torch.randn(H, generator=g).to(dt),
                dy=torch.randn(T, H, generator=g).to(dt), dres=torch.randn(T, H, generator=g).to(dt))


class Guarded:
    """An output inside a larger buffer of a known pattern."""

    def __init__(self, shape, dt):
        n = 1
        for d in shape:
            n *= d
        size = torch.empty((), dtype=dt).element_size()
        self.at, self.end = 256, 256 + n * size
        self.raw = torch.full((self.end + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        self.t = self.raw[self.at:self.end].view(dt).view(shape)

    def check(self):
        assert (self.raw[:self.at] == 0x5A).all() and (self.raw[self.end:] == 0x5A).all()


# rows side by side in a wave, of a workgroup, read again; whole vectors and not
WIDTHS = [1, 2, 7, 8, 9, 16, 63, 64, 100, 128, 129, 255, 256, 511, 512, 513, 520, 1000, 1024, 2049, 4096, 5003, 8185,
          8192, 8193, 8200, 16384, 20001, 32768, 32769, 32776, 65536]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("H", WIDTHS)
def test_forward_widths(H, dt, rms):
    T = 7
    _say(f"layer norm H={H} {dt} rms={rms}")
    d = _inputs(T, H, dt, H)
    y, mean, rstd = Guarded((T, H), dt), Guarded((T,), torch.float32), Guarded((T,), torch.float32)
    fc.fc_layer_norm(d["x"].cuda(), d["w"].cuda(), d["b"].cuda(), EPS, rms=rms, y=y.t, mean=None if rms else mean.t, rstd=rstd.t)
    torch.cuda.synchronize()
    r = ref.layer_norm(d["x"].double(), d["w"].double(), d["b"].double(), EPS, rms)
    ref.assert_within(y.t, r["y"], dt, r["ey"], "y")
    ref.assert_f32(rstd.t, r["rstd"], r["erstd"], "rstd")
    if not rms:
        ref.assert_f32(mean.t, r["mean"], r["emean"], "mean")
    for g in (y, mean, rstd):
        g.check()


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,H", [(1, 64), (3, 96), (255, 40), (1000, 264), (700, 4096), (2100, 4096), (1030, 8192)])
def test_forward_token_counts(T, H, dt):
    _say(f"layer norm T={T} H={H} {dt}")
    d = _inputs(T, H, dt, T + H, offset=30.0)     # a mean far above the deviations
    y, mean, rstd, payload = fc.fc_layer_norm(d["x"].cuda(), d["w"].cuda(), None, 1e-3, stats=True)
    assert payload is None
    r = ref.layer_norm(d["x"].double(), d["w"].double(), None, 1e-3, False)
    ref.assert_within(y, r["y"], dt, r["ey"], "y")
    ref.assert_f32(mean, r["mean"], r["emean"], "mean")
    ref.assert_f32(rstd, r["rstd"], r["erstd"], "rstd")


@pytest.mark.parametrize("w", [False, True])
@pytest.mark.parametrize("b", [False, True])
@pytest.mark.parametrize("H", [72, 1032, 40000])
def test_forward_optional_parts(w, b, H):
    d = _inputs(5, H, BF16, 3)
    w, b = (d["w"] if w else None), (d["b"] if b else None)
    y, mean, rstd, _ = fc.fc_layer_norm(d["x"].cuda(), None if w is None else w.cuda(), None if b is None else b.cuda(), EPS)
    assert mean is None and rstd is None
    r = ref.layer_norm(d["x"].double(), None if w is None else w.double(), None if b is None else b.double(), EPS, False)
    ref.assert_within(y, r["y"], BF16, r["ey"], "y")


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,H,group", [(5, 8, 8), (33, 64, 8), (9, 64, 64), (70, 384, 128), (3, 512, 512), (7, 1024, 16),
                                       (4, 4096, 128), (2, 8192, 512), (6, 8192, 32), (3, 40960, 256), (2, 65536, 512),
                                       (1100, 8192, 128), (5, 96, 24), (3, 8192, 8192), (4, 1536, 2), (2, 40, 10)])
def test_forward_payload_is_the_quantizer_s(T, H, group, dt, rms):
    """Bit for bit, and the norm as without it; payloads beside it stay."""
    _say(f"payload T={T} H={H} g={group} {dt} rms={rms}")
    d = _inputs(T, H, dt, H + group)
    x, w = d["x"].cuda(), d["w"].cuda()
    codes, s, z = Guarded((T, H), torch.uint8), Guarded((T, H // group), torch.uint16), Guarded((T, H // group), torch.uint16)
    y, _, rstd, payload = fc.fc_layer_norm(x, w, None, EPS, rms=rms, stats=True, group=group, payload=(codes.t, s.t, z.t))
    plain, _, rstd2, _ = fc.fc_layer_norm(x, w, None, EPS, rms=rms, stats=True)
    want = fc.fc_quantize_groups(x[None], 8, group)
    for got, exp in zip(payload, want):
        assert torch.equal(got.view(torch.uint8), exp[0].view(torch.uint8))
    for got, exp in zip(payload, ref.quantized(d["x"], group)):
        assert torch.equal(got.cpu().view(torch.uint8), exp.view(torch.uint8))
    assert torch.equal(y, plain) and torch.equal(rstd, rstd2)
    for g in (codes, s, z):
        g.check()


@pytest.mark.parametrize("H", [96, 515, 9000, 40001])
def test_forward_zero_rows_infinities_and_nan_stay_in_their_rows(H):
    d = _inputs(6, H, BF16, 4)
    d["x"][0] = 0
    d["x"][2, H // 2] = float("nan")
    d["x"][4, H - 1] = float("inf")
    y = fc.fc_layer_norm(d["x"].cuda(), d["w"].cuda(), d["b"].cuda(), EPS)[0].cpu()
    assert torch.equal(y[0], d["b"])
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).any()
    keep = [1, 3, 5]
    r = ref.layer_norm(d["x"][keep].double(), d["w"].double(), d["b"].double(), EPS, False)
    ref.assert_within(y[keep], r["y"], BF16, r["ey"], "y")


def _check_backward(got, d, x, mean, rstd, dt, w=True, dres=True, what=""):
    r = ref.layer_norm_backward(d["dy"].double(), x, None if mean is None else mean.double(), rstd.double(),
                                d["w"].double() if w else None, d["dres"].double() if dres else None)
    dx, dw, db = got
    ref.assert_within(dx, r["dx"], dt, r["edx"], what + " dx")
    if dw is not None:
        ref.assert_f32(dw, r["dw"], r["edw"], what + " dw")
    if db is not None:
        ref.assert_f32(db, r["db"], r["edb"], what + " db")


def _stats(x, rms):
    m = None if rms else x.double().mean(-1)
    c = x.double() if rms else x.double() - m[:, None]
    return None if rms else m.float(), (1 / torch.sqrt((c * c).mean(-1) + EPS)).float()


def _on(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(H, dt, rms):
    T = 9
    _say(f"layer norm backward H={H} {dt} rms={rms}")
    d = _inputs(T, H, dt, H)
    mean, rstd = _stats(d["x"], rms)
    dx, dw, db = Guarded((T, H), dt), Guarded((H,), torch.float32), Guarded((H,), torch.float32)
    got = fc.fc_layer_norm_backward(_on(d["dy"]), _on(d["x"]), _on(mean), _on(rstd), _on(d["w"]), rms=rms, dres=_on(d["dres"]),
                                    dx=dx.t, dw=dw.t, db=db.t)
    _check_backward(got, d, d["x"].double(), mean, rstd, dt)
    for g in (dx, dw, db):
        g.check()


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,H,group", [(1, 8, 8), (5, 64, 8), (40, 64, 64), (300, 96, 24), (2000, 128, 32), (77, 512, 256),
                                       (600, 520, 8), (33, 1040, 104), (700, 4096, 128), (1200, 1024, 64), (20, 8192, 8192),
                                       (30, 8200, 200), (11, 40960, 512), (150, 16384, 128)])
def test_backward_from_payload(T, H, group, dt):
    """Row counts beyond the workgroups, groups of every kind, rows that are read again."""
    _say(f"backward from payload T={T} H={H} g={group} {dt}")
    d = _inputs(T, H, dt, T + H)
    mean, rstd = _stats(d["x"], False)
    payload = ref.quantized(d["x"], group)
    args = (_on(d["dy"]), tuple(t.cuda() for t in payload), _on(mean), _on(rstd), _on(d["w"]))
    got = fc.fc_layer_norm_backward(*args)
    _check_backward(got, d, ref.held(payload, group), mean, rstd, dt, dres=False)
    again = fc.fc_layer_norm_backward(*args)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("H", [40, 264, 4096, 8200])
@pytest.mark.parametrize("T", [1, 2, 513, 1025])
def test_backward_token_counts(T, H):
    _say(f"layer norm backward T={T} H={H}")
    d = _inputs(T, H, BF16, T + H)
    mean, rstd = _stats(d["x"], False)
    got = fc.fc_layer_norm_backward(_on(d["dy"]), _on(d["x"]), _on(mean), _on(rstd), _on(d["w"]), dres=_on(d["dres"]))
    _check_backward(got, d, d["x"].double(), mean, rstd, BF16)


@pytest.mark.parametrize("w,bias", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("H", [72, 2056, 12000])
def test_backward_optional_sums(w, bias, H):
    d = _inputs(21, H, F16, 8)
    mean, rstd = _stats(d["x"], False)
    got = fc.fc_layer_norm_backward(_on(d["dy"]), _on(d["x"]), _on(mean), _on(rstd), _on(d["w"]) if w else None, bias=bias)
    assert (got[1] is None) == (not w) and (got[2] is None) == (not bias)
    _check_backward(got, d, d["x"].double(), mean, rstd, F16, w=w, dres=False)


@pytest.mark.parametrize("H", [72, 517, 4096, 9001])
def test_backward_in_place(H):
    """dx over the skip connection's gradient, and over dy where no column sum reads it again."""
    d = _inputs(30, H, BF16, 9)
    mean, rstd = _stats(d["x"], False)
    args = (_on(d["x"]), _on(mean), _on(rstd), _on(d["w"]))
    want = fc.fc_layer_norm_backward(_on(d["dy"]), *args, dres=_on(d["dres"]))
    stream = _on(d["dres"])
    got = fc.fc_layer_norm_backward(_on(d["dy"]), *args, dres=stream, dx=stream)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    dy = _on(d["dy"])
    if H <= 8192:
        got = fc.fc_layer_norm_backward(dy, *args, dres=_on(d["dres"]), dx=dy)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    else:
        with pytest.raises(fc.FcError):
            fc.fc_layer_norm_backward(dy, *args, dx=dy)
        plain = fc.fc_layer_norm_backward(_on(d["dy"]), args[0], args[1], args[2], bias=False)
        assert torch.equal(fc.fc_layer_norm_backward(dy, args[0], args[1], args[2], bias=False, dx=dy)[0], plain[0])


def test_backward_nan_stays_in_its_row_and_columns():
    d = _inputs(8, 300, BF16, 10)
    mean, rstd = _stats(d["x"], False)
    d["dy"][3, 7] = float("nan")
    dx, dw, db = fc.fc_layer_norm_backward(_on(d["dy"]), _on(d["x"]), _on(mean), _on(rstd), _on(d["w"]))
    rows = torch.isnan(dx.cpu()).any(-1)
    assert rows.tolist() == [i == 3 for i in range(8)]
    for t in (dw, db):
        bad = torch.isnan(t.cpu())
        assert bad[7] and bad.sum() == 1


def test_no_rows():
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    f = torch.empty(0, dtype=torch.float32, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    y, mean, rstd, payload = fc.fc_layer_norm(e, w, None, stats=True, group=32)
    assert y.shape == (0, 64) and mean.shape == (0,) and payload[0].shape == (0, 64)
    dx, dw, db = fc.fc_layer_norm_backward(e, e, f, f, w, dw=torch.ones(64, device="cuda"), db=torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_other_stream_and_captured_graph():
    T, H, group = 40, 1024, 128
    d = {k: v.cuda() for k, v in _inputs(T, H, BF16, 11).items()}
    mean = rstd = None

    def step(stream=None):
        y, m, r, p = fc.fc_layer_norm(d["x"], d["w"], d["b"], EPS, stats=True, group=group, stream=stream)
        return (y, *fc.fc_layer_norm_backward(d["dy"], p, m, r, d["w"], dres=d["dres"], stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        d["x"].copy_(_inputs(T, H, BF16, 20 + turn)["x"])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), turn
    del mean, rstd
