"""An AdamW step over no tensors (a process that owns none of a model's) does nothing,
with or without a clip coefficient."""
import torch

from lm_head_top_gb300 import kdkl


def test_no_tensors():
    handle = kdkl.kd_adamw_tensors([], [], [], [])
    assert kdkl.kd_adamw_step(handle, lr=1e-3) is None
    assert kdkl.kd_adamw_step(handle, lr=1e-3, grad_scale_dev=torch.ones(1)) is None
