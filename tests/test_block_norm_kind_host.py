"""An unknown kind of norm is refused alike by the workspace and by the calls."""
import pytest
import torch

import transformer_reduce_gb300 as L


def test_unknown_kinds_are_refused():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="kind must be"):
        L.block_norm_workspace(2, 8, 0, "batch", torch.float32, "cpu")
    with pytest.raises(ValueError, match="kind must be"):
        L.block_norm_fw(x, x, kind="batch")
