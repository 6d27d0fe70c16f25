"""Block norms on the GPU against their 64-bit statement (tests/layer_ref.py):
every row shape the kernels split differently, optional parts, gates of each
kind, payloads of both widths with groups that end inside a vector, and the
rows around an output left as they were."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc
import layer_ref as ref

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


def _inputs(T, H, dt, gate_tokens, seed, post=True, gate=True, pre=True):
    g = torch.Generator().manual_seed(seed)
    def n(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(dt)
    x = n(T, H)
    x[:, :: max(1, H // 3)] *= 20
    return dict(x=x, residual=n(T, H, scale=3.0), w_post=(1 + n(H, scale=0.2)).to(dt) if post else None,
                gate=n(-(-T // gate_tokens), H) if gate else None, w_pre=(1 + n(H, scale=0.2)).to(dt) if pre else None)


def _cuda(d):
    return {k: v if v is None else v.cuda() for k, v in d.items()}


def _f64(d):
    return {k: v if v is None else v.double() for k, v in d.items()}


class Guarded:
    """A [T, H] output inside a larger buffer of a known pattern."""

    def __init__(self, T, H, dt):
        self.n = T * H
        self.raw = torch.full((256 + self.n + 256,), 0x5A5A, dtype=torch.int16, device="cuda")
        self.t = self.raw[256:256 + self.n].view(dt).view(T, H)

    def check(self):
        assert (self.raw[:256] == 0x5A5A).all() and (self.raw[256 + self.n:] == 0x5A5A).all()


def _check(got_h, got_y, d, gate_tokens, dt, res_scale, out_scale, eps=EPS, what=""):
    h, eh, y, ey = ref.norms(d["x"], d["residual"], d["w_post"], d["gate"], gate_tokens, d["w_pre"],
                             res_scale, out_scale, eps)
    ref.assert_within(got_h, h, dt, eh, what + " h")
    if y is None:
        assert got_y is None
    else:
        ref.assert_within(got_y, y, dt, ey, what + " y")


# every way the launcher splits rows, at its borders, and lengths that are not whole vectors
WIDTHS = [1, 2, 7, 8, 9, 63, 64, 511, 512, 513, 520, 1000, 1024, 2040, 2048, 2049, 4096, 5003, 8185, 8192, 8200,
          16384, 20001, 32768, 32770, 65536]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, dt):
    T = 5
    _say(f"norm H={H} {dt}")
    d = _inputs(T, H, dt, 2, H)
    h, y = Guarded(T, H, dt), Guarded(T, H, dt)
    fc.fc_residual_norm(**_cuda(d), gate_tokens=2, eps=EPS, res_scale=0.75, out_scale=1.5, h=h.t, y=y.t)
    torch.cuda.synchronize()
    _check(h.t, y.t, _f64(d), 2, dt, 0.75, 1.5)
    h.check()
    y.check()


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("H", [96, 4096, 8192])
@pytest.mark.parametrize("T", [1, 3, 255, 700, 1500])
def test_token_counts(T, H, dt):
    _say(f"norm T={T} H={H} {dt}")
    d = _inputs(T, H, dt, T, T + H)
    h, y = fc.fc_residual_norm(**_cuda(d), gate_tokens=T, eps=EPS)
    torch.cuda.synchronize()
    _check(h, y, _f64(d), T, dt, 1.0, 1.0)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 4, 100])
@pytest.mark.parametrize("pre", [False, True])
def test_optional_parts(post, gate, pre):
    T, H, dt = 10, 1032, BF16
    _say(f"norm post={post} gate={gate} pre={pre}")
    d = _inputs(T, H, dt, max(gate, 1), 9, post, gate > 0, pre)
    h, y = fc.fc_residual_norm(**_cuda(d), gate_tokens=gate or None, eps=1e-3, res_scale=-2.0, out_scale=0.1)
    torch.cuda.synchronize()
    _check(h, y, _f64(d), max(gate, 1), dt, -2.0, 0.1, 1e-3)


def test_gate_shapes():
    """[H] for all tokens; a row per token by default."""
    d = _cuda(_inputs(6, 64, BF16, 1, 3))
    per_token, _ = fc.fc_residual_norm(**d)
    again, _ = fc.fc_residual_norm(**d, gate_tokens=1)
    assert torch.equal(per_token, again)
    one = dict(d, gate=d["gate"][0].contiguous())
    a, _ = fc.fc_residual_norm(**one)
    b, _ = fc.fc_residual_norm(**dict(d, gate=d["gate"][:1].contiguous()), gate_tokens=6)
    assert torch.equal(a, b)


def test_in_place_residual():
    d = _cuda(_inputs(33, 2048, BF16, 1, 4))
    h, y = fc.fc_residual_norm(**d)
    stream = d["residual"].clone()
    h2, y2 = fc.fc_residual_norm(**dict(d, residual=stream), h=stream)
    assert h2.data_ptr() == stream.data_ptr()
    assert torch.equal(h, stream) and torch.equal(y, y2)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_zero_rows_infinities_and_nan_stay_in_their_rows(dt):
    T, H = 6, 515
    d = _inputs(T, H, dt, 1, 5)
    d["x"][0] = 0                       # a row that nothing is left of
    d["x"][1], d["residual"][1] = 0, 0
    d["x"][2, 7] = float("inf")
    d["residual"][4, 514] = float("nan")
    h, y = fc.fc_residual_norm(**_cuda(d), eps=EPS)
    torch.cuda.synchronize()
    h, y = h.cpu(), y.cpu()
    f = _f64(d)
    rows = [0, 1, 3, 5]
    part = {k: (v[rows] if k in ("x", "residual", "gate") else v) for k, v in f.items()}
    _check(h[rows], y[rows], part, 1, dt, 1.0, 1.0)
    assert (h[1] == 0).all() and (y[1] == 0).all()
    assert torch.isnan(h[2, 7]) and torch.isnan(y[2, 7])      # inf * (1 / inf)
    assert torch.isnan(h[4, 514]) and torch.isfinite(h[4, :514]).all() and torch.isnan(y[4]).all()


@pytest.mark.parametrize("dt", [BF16, F16])
def test_magnitudes(dt):
    """Rows from subnormals to the largest values binary32 can still square and sum."""
    H = 256
    scales = [1e-7, 1e-4, 1.0, 2000.0] if dt == F16 else [1e-38, 1e-20, 1e-4, 1.0, 1e4, 1e17]
    g = torch.Generator().manual_seed(6)
    x = (torch.randn(len(scales), H, generator=g) * torch.tensor(scales)[:, None]).to(dt)
    d = dict(x=x, residual=torch.zeros_like(x), w_post=None, gate=None, w_pre=torch.ones(H, dtype=dt))
    h, y = fc.fc_residual_norm(**_cuda(d), eps=1e-37)
    torch.cuda.synchronize()
    # bf16 rows of 1e-38: their squares underflow to nothing beside eps, in 64 bits too
    _check(h, y, _f64(d), 1, dt, 1.0, 1.0, 1e-37)


PAYLOADS = [  # (T, H, bits, group)
    (1, 8192, 4, 128), (64, 8192, 4, 128), (9, 4096, 8, 4096), (7, 4608, 8, 96), (7, 4608, 4, 96), (5, 30, 4, 6),
    (5, 30, 8, 10), (3, 2, 4, 2), (3, 2, 8, 2), (300, 1010, 4, 10), (300, 1010, 8, 2), (4, 640, 4, 8), (4, 640, 8, 160),
    (3, 5000, 4, 500), (2, 24576, 8, 24), (2, 65536, 4, 65536), (2, 65534, 8, 2), (2, 65534, 4, 65534), (2, 20002, 4, 146),
]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,H,bits,group", PAYLOADS)
def test_payload(T, H, bits, group, dt):
    _say(f"wire norm T={T} H={H} int{bits} g{group} {dt}")
    d = _inputs(T, H, dt, 3, T + H + bits)
    g = torch.Generator().manual_seed(H)
    codes = torch.randint(0, 256, (T, H * bits // 8), generator=g, dtype=torch.uint8)
    s = (torch.rand((T, H // group), generator=g) * 0.3).half()
    z = torch.randn((T, H // group), generator=g).half()
    x = ref.dequantize(codes, s, z, bits, group)
    d["x"] = x
    h, y = Guarded(T, H, dt), Guarded(T, H, dt)
    c = _cuda({k: v for k, v in d.items() if k != "x"})
    fc.fc_dequantize_residual_norm(codes.cuda(), s.view(torch.uint16).cuda(), z.view(torch.uint16).cuda(), T, H, bits,
                                   group, **c, gate_tokens=3, eps=EPS, res_scale=1.25, out_scale=0.5, h=h.t, y=y.t)
    torch.cuda.synchronize()
    # binary32 q * s + z is exact but for its last rounding, within the bound
    _check(h.t, y.t, _f64(d), 3, dt, 1.25, 0.5)
    h.check()
    y.check()


@pytest.mark.parametrize("R,T,H,b1,b2,group,dt", [
    (4, 16, 8192, 4, 4, 128, BF16), (8, 3, 8192, 4, 8, 128, BF16), (4, 1500, 4096, 4, 4, 128, F16),
    (3, 5, 576, 8, 4, 96, F16), (2, 2, 8, 4, 4, 2, BF16), (4, 4, 4096, 8, 8, 4096, F16), (1, 7, 256, 4, 4, 64, BF16),
])
def test_allreduce_norm(R, T, H, b1, b2, group, dt):
    """Payloads as fc_allreduce_emulated leaves them, and the norms of payload 2."""
    _say(f"allreduce norm R={R} T={T} H={H} int{b1}/{b2} g{group} {dt}")
    d = _cuda(_inputs(T, H, dt, 2, H + T))
    d.pop("x")
    g = torch.Generator().manual_seed(R)
    x = torch.randn((R, T, H), generator=g).to(dt).cuda()
    _, ws = fc.fc_allreduce_emulated(x, b1, group, bits2=b2)
    want = fc.workspace_views(ws, R, T, H, b1, group, b2)
    g2 = fc.fc_stage2_group(R, H, group)
    h1, y1 = fc.fc_dequantize_residual_norm(want["codes2"], want["s2"], want["z2"], T, H, b2, g2, **d, gate_tokens=2)
    h, y, ws2 = fc.fc_allreduce_emulated_norm(x, b1, group, **d, gate_tokens=2, bits2=b2)
    torch.cuda.synchronize()
    got = fc.workspace_views(ws2, R, T, H, b1, group, b2)
    for k in want:
        assert torch.equal(got[k].cpu(), want[k].cpu()), k
    assert torch.equal(h, h1) and torch.equal(y, y1)
    f = _f64({k: None if v is None else v.cpu() for k, v in d.items()})
    f["x"] = ref.dequantize(want["codes2"].cpu(), want["s2"].cpu(), want["z2"].cpu(), b2, g2)
    _check(h, y, f, 2, dt, 1.0, 1.0)


def test_no_tokens():
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    h, y = fc.fc_residual_norm(e, e.clone(), w_pre=torch.ones(64, dtype=BF16, device="cuda"))
    assert h.shape == y.shape == (0, 64)


@pytest.mark.parametrize("gate_tokens", [5, 1 << 31, (1 << 32) + 1])
def test_one_gate_row_for_any_longer_span(gate_tokens):
    d = _cuda(_inputs(5, 200, BF16, 1, 1))
    d["gate"] = d["gate"][:1]
    want = fc.fc_residual_norm(**dict(d, gate=d["gate"][0]))
    got = fc.fc_residual_norm(**dict(d, gate_tokens=gate_tokens))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refuses():
    d = _cuda(_inputs(4, 64, BF16, 1, 1))
    bad = [
        dict(x=d["x"].half()), dict(x=d["x"][:3]), dict(x=d["x"].cpu()), dict(residual=d["residual"].float()),
        dict(residual=d["residual"].t().contiguous().t()), dict(w_post=d["w_post"].float()), dict(w_pre=d["w_pre"][:32]),
        dict(gate=d["gate"][:3]), dict(gate=d["gate"], gate_tokens=2), dict(gate=d["gate"], gate_tokens=0),
        dict(gate=d["gate"][0], gate_tokens=1), dict(h=torch.empty(4, 63, dtype=BF16, device="cuda")),
        dict(y=torch.empty(4, 64, dtype=F16, device="cuda")), dict(w_pre=None, y=torch.empty(4, 64, dtype=BF16, device="cuda")),
        dict(residual=d["residual"][0]),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            fc.fc_residual_norm(**dict(d, **kw))
    for kw, status in [(dict(eps=0.0), 10), (dict(res_scale=float("nan")), 10), (dict(h=d["x"]), 9), (dict(y=d["residual"]), 9)]:
        with pytest.raises(fc.FcError) as e:
            fc.fc_residual_norm(**dict(d, **kw))
        assert e.value.status == status
    with pytest.raises(fc.FcError) as e:
        wide = torch.zeros(1, 65537, dtype=BF16, device="cuda")
        fc.fc_residual_norm(wide, wide.clone())
    assert e.value.status == 2
    q = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    m = torch.zeros(4, 2, dtype=torch.uint16, device="cuda")
    with pytest.raises(ValueError, match="codes2 holds"):
        fc.fc_dequantize_residual_norm(q[:2], m, m, 4, 64, 4, 32, d["residual"])
    with pytest.raises(ValueError, match="z2 holds"):
        fc.fc_dequantize_residual_norm(q, m, m[:1], 4, 64, 4, 32, d["residual"])
    with pytest.raises(fc.FcError) as e:
        fc.fc_dequantize_residual_norm(q, m, m, 4, 64, 4, 24, d["residual"])
    assert e.value.status == 2


def test_other_stream_and_graph_replays():
    """A call on a stream that is not the current one, and captured: every replay on new
    inputs equals the eager call."""
    T, H, R = 32, 4096, 4
    d = _cuda(_inputs(T, H, BF16, T, 8))
    d.pop("x")
    x = torch.randn((R, T, H), device="cuda").to(BF16)
    h, y, ws = fc.fc_allreduce_emulated_norm(x, 4, 128, **d, gate_tokens=T)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h2, y2, ws2 = fc.fc_allreduce_emulated_norm(x, 4, 128, **d, gate_tokens=T, stream=side)
    side.synchronize()
    assert torch.equal(h, h2) and torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fc.fc_allreduce_emulated_norm(x, 4, 128, **d, gate_tokens=T, h=h2, y=y2, workspace=ws2, stream=side)
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(torch.randn((R, T, H), device="cuda"))
        h2.zero_(), y2.zero_(), ws2.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        fc.fc_allreduce_emulated_norm(x, 4, 128, **d, gate_tokens=T, h=h, y=y, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(y, y2), f"replay {i}"


def _sampled(T, H, rows, dt, gate_tokens=1):
    """Inputs made on the GPU and the 64-bit check of some rows of the outputs."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(dt)
    res = torch.randn((T, H), generator=g, device="cuda").to(dt)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)
    h, y = fc.fc_residual_norm(x, res, w_post=w, w_pre=w, eps=EPS)
    torch.cuda.synchronize()
    at = torch.tensor(rows)
    d = dict(x=x[at].cpu().double(), residual=res[at].cpu().double(), w_post=w.cpu().double(), gate=None, w_pre=w.cpu().double())
    _check(h[at], y[at], d, 1, dt, 1.0, 1.0)
    return x, res, w, h, y


def test_outputs_past_the_cache():
    """Outputs of more than 256 MiB are stored past it; the rows are the same as one by one."""
    T, H = 8200, 8192
    _say("norm past the cache")
    rows = [0, 1, 4095, 8191, 8199]
    x, res, w, h, y = _sampled(T, H, rows, BF16)
    for r in rows:
        h1, y1 = fc.fc_residual_norm(x[r:r + 1], res[r:r + 1], w_post=w, w_pre=w, eps=EPS)
        # one vector per thread against two: other sums, so within a rounding of each other
        assert (h1 - h[r:r + 1]).abs().max() <= 2.0 ** -7 * h1.abs().max()


def test_more_rows_than_a_grid_row():
    T = (1 << 20) + 5
    _say("norm 2^20 + 5 rows")
    _sampled(T, 8, [0, 1, (1 << 20) - 1, 1 << 20, T - 1], F16)
    _sampled(T, 20, [3, (1 << 20) - 1, 1 << 20, T - 1], BF16)


# two vectors a thread: rows of 1025 to 2048 vectors, and from 2^23 elements on rows of more than 64; whole
# rows, rows that end inside a vector, groups of whole vectors and (146, 10: also inside one) of pairs
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,H", [(1777, 5003), (5, 8193), (5, 16383), (3, 8207), (16200, 519), (8400, 1001)])
def test_two_vectors_a_thread(T, H, dt):
    _say(f"norm, two vectors, T={T} H={H} {dt}")
    d = _inputs(T, H, dt, 1, H)
    h, y = Guarded(T, H, dt), Guarded(T, H, dt)
    fc.fc_residual_norm(**_cuda(d), gate_tokens=1, eps=EPS, res_scale=1.25, out_scale=-0.5, h=h.t, y=y.t)
    torch.cuda.synchronize()
    _check(h.t, y.t, _f64(d), 1, dt, 1.25, -0.5)
    h.check()
    y.check()


def _payload(T, H, bits, group, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (T, H * bits // 8), generator=g, dtype=torch.uint8)
    s = (torch.rand((T, H // group), generator=g) * 0.3).half()
    z = torch.randn((T, H // group), generator=g).half()
    return codes, s, z


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,H,bits,group", [
    (1100, 8192, 4, 128), (1030, 8192, 8, 128), (1900, 4608, 8, 96), (1900, 4608, 4, 96), (3, 12288, 4, 96), (2, 16384, 8, 16384),
    (3, 10010, 4, 10), (3, 10010, 8, 10), (900, 10010, 4, 10), (900, 10010, 8, 2), (2, 16382, 4, 16382), (840, 10074, 4, 146),
    (15000, 576, 4, 36)])
def test_payload_two_vectors_a_thread(T, H, bits, group, dt):
    _say(f"wire norm, two vectors, T={T} H={H} int{bits} g{group} {dt}")
    d = _inputs(T, H, dt, 3, T + H + bits)
    codes, s, z = _payload(T, H, bits, group, H)
    d["x"] = ref.dequantize(codes, s, z, bits, group)
    h, y = Guarded(T, H, dt), Guarded(T, H, dt)
    c = _cuda({k: v for k, v in d.items() if k != "x"})
    fc.fc_dequantize_residual_norm(codes.cuda(), s.view(torch.uint16).cuda(), z.view(torch.uint16).cuda(), T, H, bits,
                                   group, **c, gate_tokens=3, eps=EPS, res_scale=1.25, out_scale=0.5, h=h.t, y=y.t)
    torch.cuda.synchronize()
    _check(h.t, y.t, _f64(d), 3, dt, 1.25, 0.5)
    h.check()
    y.check()


@pytest.mark.parametrize("T,H,bits,group,pre", [(8200, 8192, 4, 128, True), (4200, 16382, 8, 2, True), (16500, 8192, 4, 128, False)])
def test_payload_outputs_past_the_cache(T, H, bits, group, pre):
    """Outputs of more than 256 MiB, with y and h alone; sampled rows."""
    _say(f"wire norm past the cache T={T} H={H} int{bits} g{group}")
    g = torch.Generator(device="cuda").manual_seed(T)
    codes = torch.randint(0, 256, (T, H * bits // 8), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand((T, H // group), generator=g, device="cuda") * 0.3).half()
    z = torch.randn((T, H // group), generator=g, device="cuda").half()
    res = torch.randn((T, H), generator=g, device="cuda").to(BF16)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    h, y = Guarded(T, H, BF16), Guarded(T, H, BF16)
    fc.fc_dequantize_residual_norm(codes, s.view(torch.uint16), z.view(torch.uint16), T, H, bits, group, res, w_post=w,
                                   w_pre=w if pre else None, eps=EPS, h=h.t, y=y.t if pre else None)
    torch.cuda.synchronize()
    h.check()
    y.check()
    at = torch.tensor([0, 1, 511, T // 2, T - 2, T - 1])
    wd = w.cpu().double()
    d = dict(x=ref.dequantize(codes[at].cpu(), s[at].cpu(), z[at].cpu(), bits, group), residual=res[at].cpu().double(),
             w_post=wd, gate=None, w_pre=wd if pre else None)
    _check(h.t[at], y.t[at] if pre else None, d, 1, BF16, 1.0, 1.0)
    if not pre:
        assert (y.raw == 0x5A5A).all()


@pytest.mark.parametrize("T,H", [(700, 9), (700, 515), (600, 1001), (500, 5003), (300, 8193), (100, 20001), (200, 32770), (60, 65535)])
def test_in_place_rows_that_end_inside_a_vector(T, H):
    """The load of such a row's last vector overlaps elements that other threads own and, in place,
    overwrite: the outputs are those of the call out of place."""
    _say(f"norm in place T={T} H={H}")
    d = _cuda(_inputs(T, H, F16, 1, H))
    h, y = fc.fc_residual_norm(**d)
    stream = d["residual"].clone()
    h2, y2 = fc.fc_residual_norm(**dict(d, residual=stream), h=stream)
    torch.cuda.synchronize()
    assert torch.equal(h, stream) and torch.equal(y, y2)


@pytest.mark.parametrize("T,H,bits,group", [(500, 10010, 4, 10), (300, 32770, 8, 290), (64, 65534, 4, 2), (1100, 8192, 4, 128)])
def test_payload_in_place(T, H, bits, group):
    _say(f"wire norm in place T={T} H={H} int{bits} g{group}")
    d = _cuda({k: v for k, v in _inputs(T, H, BF16, 1, H).items() if k != "x"})
    codes, s, z = _payload(T, H, bits, group, T)
    p = (codes.cuda(), s.view(torch.uint16).cuda(), z.view(torch.uint16).cuda(), T, H, bits, group)
    h, y = fc.fc_dequantize_residual_norm(*p, **d)
    stream = d["residual"].clone()
    h2, y2 = fc.fc_dequantize_residual_norm(*p, **dict(d, residual=stream), h=stream)
    torch.cuda.synchronize()
    assert torch.equal(h, stream) and torch.equal(y, y2)
