"""What the header states of the Muon step's workspace and launches."""
import ctypes

import pytest
import torch

from lm_head_top_gb300 import kdkl

SMALL = 256


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(kdkl.LIB_PATH):
        from lm_head_top_gb300 import build
        build.build()
    return kdkl.load()


def _bytes(lib, shapes):
    table = (kdkl.kd_muon_matrix * len(shapes))()
    for row, (rows, cols) in zip(table, shapes):
        row.rows, row.cols = rows, cols
    return lib.kd_muon_workspace_size(table, len(shapes))


def _stated(shapes):
    up = lambda n: -(-n // 64) * 64  # noqa: E731
    return sum(8 * min(s) * (up(s[0]) + up(s[1])) + 12 * -(-s[0] * s[1] // 16384) for s in shapes)


@pytest.mark.parametrize("shapes", [
    [(1000, 1000)], [(193, 193)], [(129, 129)], [(129, 1)], [(257, 1)], [(1, 65536)], [(65536, 65536)], [(1, 1), (1000, 1000)],
    [(300, 200)] * 14, [(1000, 1000)] * 12 + [(2731, 1000)] * 6 + [(1000, 2731)] * 3,
    [(i + 1, 200 + i) for i in range(16)] * 3 + [(130, 130)], [(1024, 2816)] * 90])
def test_workspace_of_a_round(lib, shapes):
    stated, kinds = _stated(shapes), len({tuple(s) for s in shapes})
    got = _bytes(lib, shapes)
    if all(r <= 128 and c <= 256 or r <= 256 and c <= 128 for r, c in shapes):
        assert got == SMALL
        return
    assert got <= stated + 1024 * kinds + 1024
    if kinds <= 16:  # shapes past the sixteenth are another round's
        assert got >= stated


def test_workspace_of_rounds(lib):
    shapes = [(1024, 1024)] * 96 + [(2816, 1024)] * 48 + [(1024, 2816)] * 24
    assert _stated(shapes) > 3 * 2 ** 30  # two rounds of like size
    assert 0.5 * _stated(shapes) <= _bytes(lib, shapes) <= 0.52 * _stated(shapes)
    # one that needs more than 3 GiB has a round of its own
    big = [(20_000, 20_000)]
    assert _stated(big) <= _bytes(lib, big + [(1024, 2816)] * 20) <= _stated(big) + 4096
    assert _bytes(lib, [(128, 256), (256, 128), (1, 1)] * 300) == SMALL


@pytest.mark.gpu
@pytest.mark.parametrize("shapes,rounds", [
    ([(130, 300)], 1), ([(130, 300)] * 384, 1), ([(130, 300)] * 385, 2), ([(130, 200 + i) for i in range(16)], 1),
    ([(130, 200 + i) for i in range(17)], 2), ([(64, 20_000)] * 320, 2)])
@pytest.mark.parametrize("steps", [1, 5])
def test_launches(lib, shapes, rounds, steps):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    z = lambda: [torch.zeros(s, device="cuda") for s in shapes]  # noqa: E731
    h = kdkl.kd_muon_tensors(z(), z(), z())
    before = kdkl.kd_launch_count()
    kdkl.kd_muon_step(h, lr=0.1, steps=steps)
    assert kdkl.kd_launch_count() - before == rounds * (2 + 3 * steps)


@pytest.mark.gpu
@pytest.mark.parametrize("n,launches", [(1, 1), (384, 1), (385, 2)])
def test_launches_of_small_matrices(lib, n, launches):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    z = lambda: [torch.zeros(128, 256, device="cuda") for _ in range(n)]  # noqa: E731
    h = kdkl.kd_muon_tensors(z(), z(), z())
    before = kdkl.kd_launch_count()
    kdkl.kd_muon_step(h, lr=0.1)
    assert kdkl.kd_launch_count() - before == launches
