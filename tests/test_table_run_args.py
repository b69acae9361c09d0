"""What TableRun refuses before it allocates anything (no GPU needed)."""
import pytest
import torch

from fsdp_sharded_optimizer_zero_amd.runner import TableRun


def test_whole_parameters_need_a_body():
    """Without a body nothing reads them: each step would decay them."""
    with pytest.raises(ValueError, match="body"):
        TableRun(90, 24, 2, 8, 5, whole=[torch.ones(24)], device="cpu")
