"""The Muon step's 22 bits: X against fp64 within a few times what the header states, by either
way of working on a matrix, with every mix of tiles, after one step and after five."""
import pytest
import torch

from _muon_halves import X_TOL, X_TOL_ONE, rank_one
from oracle import body_oracle as bo
from test_muon_gpu import TILES

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SMALL = [(16, 16), (17, 33), (33, 17), (64, 64), (100, 128), (128, 256), (256, 128)]
OTHERS = [(129, 200), (300, 300), (130, 700), (700, 130), (777, 777), (300, 1100), (1100, 300), (513, 1030)]


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _off(kdkl, grads, nesterov=True, **hyper):
    """Of the step alone, from parameters and momenta of zero."""
    params, momentum = [torch.zeros_like(g) for g in grads], [torch.zeros_like(g) for g in grads]
    kdkl.kd_muon_step(kdkl.kd_muon_tensors(params, grads, momentum), lr=1.0, scale="spectral", nesterov=nesterov, **hyper)
    for p, g in zip(params, grads):
        zero = torch.zeros_like(g)
        want = bo.muon(zero, g, zero, lr=1.0, scale="spectral", nesterov=nesterov, **hyper)[0]
        yield tuple(p.shape), float((p.double() - want).norm() / want.norm())


def _random(shapes, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(*s, generator=g, device="cuda") for s in shapes]


@pytest.mark.parametrize("shapes", [SMALL, OTHERS, SMALL + OTHERS], ids=["small", "others", "together"])
@pytest.mark.parametrize("seed", [0, 1])
def test_five_steps(kdkl, shapes, seed):
    # (u = (1 + mu) g rounded to fp32, and the update rounded once)
    for shape, off in _off(kdkl, _random(shapes, seed)):
        assert off <= X_TOL + 4 * U, (shape, off)


@pytest.mark.parametrize("shape", OTHERS)
def test_five_steps_of_one_matrix(kdkl, shape):
    for _, off in _off(kdkl, _random([shape], 3)):
        assert off <= X_TOL + 4 * U, off


@pytest.mark.parametrize("tiles", list(TILES))
def test_five_steps_with_every_mix_of_tiles(kdkl, tiles):
    for shape, off in _off(kdkl, _random(TILES[tiles], 4)):
        assert off <= X_TOL + 4 * U, (shape, off)


@pytest.mark.parametrize("shapes", [[(16, 2000), (16, 8192), (16, 20_000), (20_000, 16), (300, 20_000)],
                                    [(16, 16), (64, 64), (100, 250), (250, 100)], [(300, 300), (777, 777), (1024, 300)]],
                         ids=["long sums", "small", "others"])
def test_one_step_of_rank_one(kdkl, shapes):
    """A singular value of 1: all that S and its square are off is in X."""
    g = torch.Generator("cuda").manual_seed(5)
    grads = [rank_one(*s, g, "cuda") for s in shapes]
    for shape, off in _off(kdkl, grads, steps=1, nesterov=False):
        assert off <= X_TOL_ONE + 4 * U, (shape, off)


def test_more_than_a_round_holds_by_its_bytes(kdkl):
    """330 matrices of 64 x 20,000: 10.3 MB of workspace each, 3.4 GB, of which a round takes 3 GiB.
    Two rounds of like size, with a few of other shapes where they meet and at the end."""
    shapes = [(64, 20_000)] * 160 + [(200, 3000)] * 4 + [(64, 20_000)] * 170 + [(31, 47)]
    grads = _random(shapes, 6)
    params = [torch.zeros(s, device="cuda") for s in shapes]
    momentum = [torch.zeros(s, device="cuda") for s in shapes]
    h = kdkl.kd_muon_tensors(params, grads, momentum)
    each = sum(8 * min(s) * sum(-(-n // 64) * 64 for n in s) for s in shapes)
    assert each > 3 * 2 ** 30 and h.workspace_bytes < 0.55 * each  # two rounds
    ws = torch.full((h.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    kdkl.kd_muon_step(h, lr=1.0, scale="spectral", workspace=ws)
    assert kdkl.kd_kl_check_status(ws) == 0
    for i, (p, g) in enumerate(zip(params, grads)):
        zero = torch.zeros_like(g)
        want = bo.muon(zero, g, zero, lr=1.0, scale="spectral")[0]
        off = float((p.double() - want).norm() / want.norm())
        assert off <= X_TOL + 4 * U, (i, tuple(p.shape), off)
