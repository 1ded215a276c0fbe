"""What the tolerances of the Muon step's tests would notice: its arithmetic restated, whole and with
a part left out."""
import pytest
import torch

from _muon_halves import X_TOL, X_TOL_ONE, rank_one, x_of
from oracle import body_oracle as bo


def _off(u, steps=5, **k):
    zero = torch.zeros_like(u)
    want = bo.muon(zero, u, zero, lr=1.0, steps=steps, nesterov=False)[2]
    return float((x_of(u, steps, **k) - want).norm() / want.norm())


@pytest.mark.parametrize("shape", [(17, 33), (64, 64), (100, 128)])
def test_a_product_left_out(shape):
    u = torch.randn(*shape, generator=torch.Generator().manual_seed(1))
    assert _off(u) <= X_TOL / 5
    for which in range(3):
        for product in ((0, 1), (1, 0)):
            assert _off(u, drop=(which, product)) >= 5 * X_TOL, (which, product)


def test_sums_left_on_the_tensor_core():
    u = rank_one(16, 20_000, torch.Generator().manual_seed(2))
    assert _off(u, steps=1) <= X_TOL_ONE / 5
    assert _off(u, steps=1, blocks_a_sum=10 ** 6) >= 3 * X_TOL_ONE
