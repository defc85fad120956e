"""Runs after the training tests: no kernel reported a problem (a wait that ran
out; in the bounds-checked build an address out of range)."""
import pytest
import torch


@pytest.mark.gpu
def test_device_status_is_clear_after_the_training_tests():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import tileblend as tbl
    assert tbl.tb_device_status() == tbl.TB_DEV_OK
