"""The training operators at the ends of their documented ranges: 2^31 - 1 tokens, rows of
2^22 values. Operands are zeros but for rows (or columns) at both ends, around the middle
and around 2^30, so that every output is known and every sum exact."""
from __future__ import annotations

import sys

import pytest
import torch

import bit_activation_compression_amd as fc

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T = 2 ** 31 - 1
ROWS = torch.tensor([0, 1, 63, 64, 255, 256, 2 ** 20, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 5, T - 257, T - 256, T - 64, T - 2, T - 1])
STEP = 1 << 27


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


def _whole(shape, seed):
    """Small whole numbers, not 0."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(1, 4, shape, generator=g) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
    return v.to(BF16).cuda()


def _all_rows(t, row, but):
    """Every row of t is `row`, but for the rows of `but`."""
    keep = t[but].clone()
    t[but] = row
    for i in range(0, t.shape[0], STEP):
        assert (t[i:i + STEP] == row).all(), i
    t[but] = keep


def test_norms_of_2_to_31_rows():
    H = 3
    _need(45)
    rows = ROWS.cuda()
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    small = _whole((len(rows), H), 1)
    x[rows] = small
    w = _whole((H,), 2)
    _say("norm of 2^31 - 1 rows")
    y, _, rstd, _ = fc.fc_layer_norm(x, w, rms=True, stats=True)
    ys, _, rs, _ = fc.fc_layer_norm(small, w, rms=True, stats=True)
    assert torch.equal(y[rows], ys) and torch.equal(rstd[rows], rs)
    _all_rows(y, torch.zeros(H, dtype=BF16, device="cuda"), rows)
    dy = y.zero_()
    grad = _whole((len(rows), H), 3)
    dy[rows] = grad
    _say("norm backward of 2^31 - 1 rows")
    dx, dw, db = fc.fc_layer_norm_backward(dy, x, None, rstd, w, rms=True)
    dxs, dws, dbs = fc.fc_layer_norm_backward(grad, small, None, rs, w, rms=True)
    assert torch.equal(dx[rows], dxs)
    _all_rows(dx, torch.zeros(H, dtype=BF16, device="cuda"), rows)
    assert torch.equal(db, grad.float().sum(0)) and torch.equal(dbs, db)
    # 15 products, in another order of sums
    assert ((dw - dws).abs() <= 32 * 2.0 ** -24 * (grad.float() * small.float() * rs[:, None]).abs().sum(0)).all()


@pytest.mark.parametrize("K,H", [(8, 8), (7, 5)])
def test_linear_and_input_grad_of_2_to_31_tokens(K, H):
    _need(75)
    rows = ROWS.cuda()
    a = torch.zeros(T, K, dtype=BF16, device="cuda")
    small = _whole((len(rows), K), 4)
    a[rows] = small
    w, bias = _whole((H, K), 5), _whole((H,), 6)
    _say(f"linear of 2^31 - 1 tokens, {K} x {H}")
    y, _ = fc.fc_linear_act(a, w, bias)
    _all_rows(y, bias, rows)
    assert torch.equal(y[rows].float(), small.float() @ w.float().t() + bias.float())
    del a
    torch.cuda.empty_cache()
    dy = y.zero_()
    grad = _whole((len(rows), H), 7)
    dy[rows] = grad
    _say("input gradient of 2^31 - 1 tokens")
    dx = torch.full((T, K), 7.0, dtype=BF16, device="cuda")
    fc.fc_linear_input_grad(dy, w, dx=dx)
    _all_rows(dx, torch.zeros(K, dtype=BF16, device="cuda"), rows)
    assert torch.equal(dx[rows].float(), grad.float() @ w.float())


@pytest.mark.parametrize("H", [8, 5])
def test_weight_grad_of_2_to_31_tokens(H):
    K, group = 8, 8
    _need(65)
    rows = ROWS.cuda()
    codes = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    s = torch.ones(T, 1, dtype=torch.float16, device="cuda")
    z = torch.full((T, 1), -2.0, dtype=torch.float16, device="cuda")
    codes[rows] = torch.randint(0, 5, (len(rows), K), generator=torch.Generator().manual_seed(8)).to(torch.uint8).cuda()
    dy = torch.zeros(T, H, dtype=BF16, device="cuda")
    grad = _whole((len(rows), H), 9)
    dy[rows] = grad
    _say("weight gradient of 2^31 - 1 tokens")
    dw = fc.fc_linear_weight_grad(dy, (codes, s.view(torch.uint16), z.view(torch.uint16)))
    assert torch.equal(dw, grad.float().t() @ (codes[rows].float() - 2))


def test_activation_backward_of_2_to_31_tokens():
    H = group = 8
    _need(100)
    rows = ROWS.cuda()
    codes = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    s = torch.ones(T, 1, dtype=torch.float16, device="cuda").view(torch.uint16)
    z = torch.full((T, 1), -2.0, dtype=torch.float16, device="cuda").view(torch.uint16)
    codes[rows] = torch.randint(0, 6, (len(rows), H), generator=torch.Generator().manual_seed(10)).to(torch.uint8).cuda()
    dy = torch.zeros(T, H, dtype=BF16, device="cuda")
    grad = _whole((len(rows), H), 11)
    dy[rows] = grad
    dz = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
    _say("activation backward of 2^31 - 1 tokens")
    _, _, db = fc.fc_activation_backward(dy, "relu", (codes, s, z), bias=True, dz=dz)
    want = grad.float() * (codes[rows] > 2)
    assert torch.equal(dz[rows].float(), want) and torch.equal(db, want.sum(0))
    _all_rows(dz, torch.zeros(H, dtype=BF16, device="cuda"), rows)
    _say("bias gradient of 2^31 - 1 tokens")
    assert torch.equal(fc.fc_activation_backward(dy, "none", bias=True)[2], grad.float().sum(0))


COLUMNS = [0, 1, 7, 8, 63, 64, 2 ** 21 - 1, 2 ** 21, 2 ** 22 - 65, 2 ** 22 - 64, 2 ** 22 - 8, 2 ** 22 - 1]


def _long_rows(n, seed):
    t = torch.zeros(n, 2 ** 22, dtype=BF16, device="cuda")
    t[:, COLUMNS] = _whole((n, len(COLUMNS)), seed)
    return t


@pytest.mark.parametrize("tokens,H", [(1, 48), (40, 128), (4096, 4096)])
def test_sums_of_2_to_22_values(tokens, H):
    """Streamed weights, split sums, and tiles of 256, whose operands are 2 GiB from the first row to the last."""
    _need(70)
    a, w = _long_rows(tokens, 12), _long_rows(H, 13)
    _say(f"linear of 2^22 inputs, {tokens} tokens, {H} outputs")
    y, _ = fc.fc_linear_act(a, w)
    assert torch.equal(y.float(), a[:, COLUMNS].float() @ w[:, COLUMNS].float().t())
    del w
    torch.cuda.empty_cache()
    _say("input gradient of 2^22 outputs")
    wt = torch.zeros(2 ** 22, 64, dtype=BF16, device="cuda")
    wt[COLUMNS] = _whole((len(COLUMNS), 64), 14)
    dx = fc.fc_linear_input_grad(a, wt)
    assert torch.equal(dx.float(), a[:, COLUMNS].float() @ wt[COLUMNS].float())


def test_rows_of_2_to_22_outputs():
    _need(10)
    K, tokens = 2 ** 22, 70
    w = _long_rows(16, 15)
    dy = _whole((tokens, 16), 16)
    _say("input gradient of 2^22 inputs")
    dx = torch.full((tokens, K), 7.0, dtype=BF16, device="cuda")
    fc.fc_linear_input_grad(dy, w, dx=dx)
    want = dy.float() @ w[:, COLUMNS].float()
    assert torch.equal(dx[:, COLUMNS].float(), want)
    dx[:, COLUMNS] = 0
    assert (dx == 0).all()
    _say("linear of 2^22 outputs, bias gradient")
    wt = torch.zeros(K, 8, dtype=BF16, device="cuda")
    wt[COLUMNS] = _whole((len(COLUMNS), 8), 17)
    a = _whole((tokens, 8), 18)
    y, _ = fc.fc_linear_act(a, wt)
    assert torch.equal(y[:, COLUMNS].float(), a.float() @ wt[COLUMNS].float().t())
    db = fc.fc_activation_backward(y, "none", bias=True)[2]
    assert torch.equal(db[COLUMNS], y[:, COLUMNS].float().sum(0)) and db.count_nonzero() <= len(COLUMNS)


@pytest.mark.parametrize("group", [524288, 8])
def test_payload_rows_of_524288_values(group):
    K, tokens, H = 524288, 130, 72
    g = torch.Generator(device="cuda").manual_seed(19)
    codes = torch.randint(0, 5, (tokens, K), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.ones(tokens, K // group, dtype=torch.float16, device="cuda").view(torch.uint16)
    z = torch.full((tokens, K // group), -2.0, dtype=torch.float16, device="cuda").view(torch.uint16)
    dy = _whole((tokens, H), 20)
    _say(f"weight gradient of payload rows of 524288, groups of {group}")
    dw = fc.fc_linear_weight_grad(dy, (codes, s, z))
    assert torch.equal(dw, dy.float().t() @ (codes.float() - 2))
    grad = _whole((tokens, K), 21)
    _say("activation backward")
    dz, dm, db = fc.fc_activation_backward(grad, "relu", (codes, s, z), mul=(codes, s, z), bias=True)
    x = codes.float() - 2
    assert torch.equal(dz.float(), grad.float() * x * (x > 0)) and torch.equal(dm.float(), grad.float() * x.clamp_min(0))
    assert torch.equal(db, dz.float().sum(0))
