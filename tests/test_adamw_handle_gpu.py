"""The handle of kd_adamw_tensors holds the memory that it points to, whatever becomes of
the lists and tensors that it was made from."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _lists(n=3, count=5000):
    return [[torch.randn(count, device="cuda").abs() for _ in range(n)] for _ in range(4)]


def test_replaced_in_the_callers_list(kdkl):
    """A list that is filled anew every step: the tensors before stay, and are stepped."""
    lists = _lists()
    want = [[t.clone() for t in ts] for ts in lists]
    kdkl.kd_adamw_step(kdkl.kd_adamw_tensors(*want), lr=0.1)
    handle = kdkl.kd_adamw_tensors(*lists)
    held = [t.untyped_storage().data_ptr() for ts in lists for t in ts]
    params = list(lists[0])
    for ts in lists:
        ts[:] = []
    gc.collect()
    # nothing new is put where the handle points
    new = [torch.full((5000,), 7.0, device="cuda") for _ in range(64)]
    assert not {t.untyped_storage().data_ptr() for t in new} & set(held)
    kdkl.kd_adamw_step(handle, lr=0.1)
    assert all(torch.equal(a, b) for a, b in zip(params, want[0]))
    assert all((t == 7.0).all() for t in new)
    del handle, params


def test_a_tensors_data_is_exchanged(kdkl):
    lists = _lists()
    handle = kdkl.kd_adamw_tensors(*lists)
    held = {t.untyped_storage().data_ptr() for ts in lists for t in ts}
    for ts in lists:
        for t in ts:
            t.data = torch.zeros(5000, device="cuda")
    gc.collect()
    new = [torch.full((5000,), 7.0, device="cuda") for _ in range(64)]
    assert not {t.untyped_storage().data_ptr() for t in new} & held
    kdkl.kd_adamw_step(handle, lr=0.1)
    assert all((t == 7.0).all() for t in new) and not any(t.any() for ts in lists for t in ts)
