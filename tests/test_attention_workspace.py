"""The workspace that the binding hands to the library (runs without a GPU)."""
import pytest
import torch

from qat_nvfp4_quantize_amd import nvq


def test_workspace_is_counted_in_bytes_and_has_no_gaps():
    assert nvq._ws_args(None) == (None, 0)
    for t in (torch.empty(512, dtype=torch.uint8), torch.empty(8, 16, dtype=torch.float32)):
        assert nvq._ws_args(t) == (t.data_ptr(), 512)
    one = torch.empty(1, dtype=torch.uint8)
    for t in (one.expand(1 << 20), torch.empty(1024, dtype=torch.uint8)[::2], torch.empty(4, 256).t()):
        with pytest.raises(ValueError, match="contiguous"):
            nvq._ws_args(t)
