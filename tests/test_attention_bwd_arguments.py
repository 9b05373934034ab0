"""Arguments of the attention's backward pass that were taken for others, on the
host: no GPU."""
import pytest
import torch

from video_diffusion_transformer_non_b200 import binding


@pytest.mark.parametrize("n_split", [-1, 65, 255, 256, 257, 1 << 16])
def test_n_split_out_of_range(monkeypatch, n_split):
    """256 was taken as 0 and 257 as 1: only the low 8 bits reached the library."""
    monkeypatch.setattr(binding, "_DEVICE_TYPE", "cpu")
    x = torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="n_split"):
        binding.attention_bwd(x, x, x, x, x, torch.zeros((1, 2, 16)), n_split=n_split)
