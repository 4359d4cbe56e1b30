"""The cache operators' check of where their workspace is, without a GPU."""
import types

import pytest
import torch

from compressed_sparse_kv_fp32_b200 import adamas


def test_workspace_on_the_host_is_refused():
    ws = types.SimpleNamespace(buffer=torch.zeros(256, dtype=torch.uint8), nbytes=256)
    with pytest.raises(ValueError, match="workspace must be on cuda:0, got cpu"):
        adamas._scratch(0, ws)


def test_workspace_of_another_device_is_refused():
    here = types.SimpleNamespace(get_device=lambda: 1, device=torch.device("cuda", 1), data_ptr=lambda: 4096)
    ws = types.SimpleNamespace(buffer=here, nbytes=256)
    with pytest.raises(ValueError, match="workspace must be on cuda:0, got cuda:1"):
        adamas._scratch(0, ws)
    assert adamas._scratch(1, ws) == (4096, 256)
