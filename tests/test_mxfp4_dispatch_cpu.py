"""The rules that choose the MXFP4 product's kernel, without a GPU: the launchers'
own code (csrc/fc_mxfp4_dispatch.h) in a build with address and
undefined-behaviour sanitizers, for a device of 256 compute units."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    """(R, T, K, H) shapes -> per shape: kernel of the coded product, of the 16-bit one, and
    the tokens' tiles of 256, 128 and 64."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("dispatch") / "driver")
    r = subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-O1", "-g", "-std=c++17", "-Wall",
                        f"-I{os.path.join(ROOT, 'bit_activation_compression_amd', 'csrc')}",
                        os.path.join(ROOT, "tests", "sanitize", "mxfp4_dispatch_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0 and "sanitize" in r.stderr:
        pytest.skip("sanitizer runtime not available")
    assert r.returncode == 0, r.stderr

    def run(shapes):
        text = "".join("%d %d %d %d\n" % tuple(s) for s in shapes)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr[-2000:]
        out = [line.split() for line in r.stdout.splitlines()]
        assert len(out) == len(shapes)
        return [(p, l, *map(int, t)) for p, l, *t in out]

    return run


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 63, 2 ** 31 - 64, 2 ** 31 - 128, 2 ** 31 - 255, 2 ** 31 - 256, 2 ** 31 - 257])
def test_tokens_up_to_the_largest_count(choose, T):
    """(1, T, 128, 16) is within the header's limits for every 32-bit T."""
    (product, linear, *tiles), = choose([(1, T, 128, 16)])
    assert tiles == [-(-T // b) for b in (256, 128, 64)]
    # one column of tiles: a round of 256 takes exactly half the rounds of 128, so 128 it is
    assert product == linear == "128"


@pytest.mark.parametrize("H", [1, 16, 17, 2 ** 24 - 1, 2 ** 24])
def test_channels_up_to_the_largest_count(choose, H):
    (product, linear, *_), (wide, *_) = choose([(1, 1, 128, H), (127, 16, 128, H)])
    assert (product, linear) == (("split1", "quantize1") if H <= 256 * 16 else ("64", "quantize0"))
    assert wide == ("split1" if 127 * -(-H // 16) <= 256 else "64")


def test_gpu_tests_reach_every_kernel(choose):
    """The shapes of test_gpu_mxfp4.py through the rules: every kernel, the tiles with one stage, with odd
    and even multiples of 128 and (those that stay for several) with more tiles than workgroups."""
    import test_gpu_mxfp4 as gpu
    kinds = ["split1", "split2", "64", "128", "256"]
    assert [p for p, *_ in choose([(1, *s) for s in gpu.TARGETS.values()])] == [n.split()[0] for n in gpu.TARGETS]
    nan = [(R, T, 384, H) for R, T, H in gpu.NAN_SHAPES]
    assert {p for p, *_ in choose(nan)} >= set(kinds) - {"split2"}
    exact = gpu.PRODUCTS + gpu.SMALL_TILES + gpu.LARGE_TILES + gpu.TWO_ROUNDS
    got = choose(exact)
    assert {p for p, *_ in got} == set(kinds)
    assert {l for _, l, *_ in got} == set(kinds) | {"quantize0", "quantize1", "quantize2"}
    # tiles and workgroups of a round on 256 units: (edge, workgroups a unit)
    for kind, (edge, per_unit) in {"64": (64, 2), "128": (128, 1), "256": (256, 1)}.items():
        again = [s for s, g in zip(exact, got) if g[0] == kind
                 and s[0] * -(-s[1] // edge) * -(-s[3] // edge) > 256 * per_unit]
        stages = {(-(-K // 128) + 1) // 2 for _, _, K, _ in again}
        assert {-(-K // 128) % 2 for _, _, K, _ in again} == {0, 1}, kind
        assert min(stages) == 1 and {s % 2 for s in stages} == {0, 1}, (kind, stages)
    for kind in kinds:
        assert {-(-K // 128) % 2 for (_, _, K, _), g in zip(exact, got) if g[0] == kind} == {0, 1}, kind
