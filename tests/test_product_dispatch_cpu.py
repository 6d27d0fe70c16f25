"""The rules that choose the products' tiles and splits, without a GPU: the launchers'
own code (csrc/fc_product_dispatch.h) in a build with address and undefined-behaviour
sanitizers. Every plan covers each output and each k once, at any size, and the GPU
tests' shapes reach every kernel."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """(R, M, N, K, large) -> (parts, (split, split_k), values, parts of sums, (split, split_k))."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("dispatch") / "driver")
    r = subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-O1", "-g", "-std=c++17", "-Wall",
                        f"-I{os.path.join(ROOT, 'bit_activation_compression_amd', 'csrc')}",
                        os.path.join(ROOT, "tests", "sanitize", "product_dispatch_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0 and "sanitize" in r.stderr:
        pytest.skip("sanitizer runtime not available")
    assert r.returncode == 0, r.stderr

    def run(shapes):
        text = "".join("%d %d %d %d %d\n" % tuple(s) for s in shapes)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr[-2000:]
        out = []
        for line in r.stdout.splitlines():
            v = [int(x) for x in line.split()]
            out.append(([tuple(v[:5]), tuple(v[5:10])], (v[10], v[11]), v[12], v[13], (v[14], v[15])))
        assert len(out) == len(shapes)
        return out
    return run


def _check(shape, plan):
    R, M, N, K, large = shape
    parts, (split, run), _, _, (wsplit, wrun) = plan
    real = [p for p in parts if p[0]]
    assert 1 <= len(real) <= 2 and parts[0][0], shape
    for tile, m0, m1, n0, n1 in real:
        assert tile in ((64, 128, 256) if large else (64, 128)) and 0 <= m0 < m1 <= M and 0 <= n0 < n1 <= N, shape
        assert m0 % 256 == 0 and n0 % 256 == 0
    # one part covers all; of two, the second has the columns or the rows that the first leaves
    if len(real) == 1:
        assert real[0][1:] == (0, M, 0, N), shape
    else:
        a, b = real
        assert a[1] == 0 and a[3] == 0
        assert (a[2] == M and b[1:] == (0, M, a[4], N)) or (a[4] == N and b[1:] == (a[2], M, 0, N)), shape
    for s, r in ((split, run), (wsplit, wrun)):
        assert s >= 1 and 1 <= r <= K and (s - 1) * r < K <= s * r, shape
        assert s == 1 or (r % 64 == 0 and r >= 512), shape


def test_plans_cover_everything_once(plans):
    rng = random.Random(7)
    shapes = []
    for _ in range(4000):
        def size(top):
            return max(1, int(round(2 ** rng.uniform(0, top))))
        shapes.append((size(4), size(14), size(14), size(15), rng.randrange(2)))
    for big in ((1, BIG, 1, 1), (1, 1, 1 << 22, 1 << 22), (1, 1 << 22, 1, BIG), (BIG, 1, 1, 1), (1, BIG, 16, 4096), (1, 1, 1, BIG),
                (1, BIG - 255, 8, 8), (7, 1 << 20, 1 << 12, 64), (1, 1 << 15, 1 << 20, 64)):
        shapes += [(*big, 0), (*big, 1)]
    for s, p in zip(shapes, plans(shapes)):
        _check(s, p)


def _kinds(plan, large):
    parts, (split, _), *_ = plan
    if split > 1:
        return {"split"}
    real = [p for p in parts if p[0]]
    if len(real) == 2:
        return {"columns left" if real[1][3] else "rows left"}
    return {str(real[0][0])}


def test_the_gpu_tests_reach_every_kernel(plans):
    import test_gpu_train_products as T
    fwd = [(R, t, H, K, int(K % 8 == 0)) for R, t, K, H in T.SHAPES + T.LARGE_SHAPES if t > 8]
    dx = [(R, t, K, H, int(K % 8 == 0 and H % 8 == 0)) for R, t, K, H in T.GRAD_SHAPES]
    dx += [(R, t, H, K, int(K % 8 == 0 and H % 8 == 0)) for R, t, K, H in T.LARGE_SHAPES]   # a layer of H inputs
    for shapes in (fwd, dx):
        seen = {0: set(), 1: set()}
        for s, p in zip(shapes, plans(shapes)):
            seen[s[4]] |= _kinds(p, s[4])
        assert seen[1] >= {"64", "128", "256", "columns left", "rows left", "split"}, seen
        assert any(s[4] == 0 for s in shapes)
    # weight gradients: codes or values, split or not, in every tile
    dw = [(R, H, K, t, 1) for R, t, K, H in T.GRAD_SHAPES] + [(1, H, K, t, 1) for t, K, H, _ in T.LONG_SUMS + T.LARGE_WEIGHTS]
    seen = {(p[2], p[3]) for p in plans(dw)}
    assert seen == {(0, 0), (0, 1), (1, 0), (1, 1)}, seen
    # (the tiles of what is read as values, and as codes: its splits are batches)
    tiles = {0: set(), 1: set()}
    for (R, M, N, K, _), p in zip(dw, plans(dw)):
        tiles[p[2]] |= {q[0] for q in plans([(R * p[4][0], M, N, K, p[2])])[0][0] if q[0]}
    assert tiles[0] == {64, 128} and tiles[1] == {64, 128, 256}, tiles


def test_the_measured_cases(plans):
    """The training shapes run in whole rounds of large tiles and the rest in middle ones."""
    (p,), = [plans([(1, 8192, 7168, 8192, 1)])]
    assert [q[0] for q in p[0]] == [256, 128]
    assert plans([(1, 8192, 8192, 8192, 1)])[0][0][0] == (256, 0, 8192, 0, 8192)
    assert plans([(1, 64, 4096, 4096, 1)])[0][1][0] == 8
