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


@pytest.mark.parametrize("args", [
    (False, 60000, 60000, 128, 128, 64),            # 2 units for each of 3.6e9 heads
    (False, 1, 40000, 128 * 60000, 1, 64),          # row statistics and Q units
    (True, 65535, 65535, 2 ** 31 - 300, 2 ** 31 - 300, 128, binding.VIDATTN_SPLIT_KV(64)),
    (False, 4000, 4000, 1000, 1000, 64, binding.VIDATTN_SPLIT_KV(64))])
def test_workspace_of_refused_sizes(args):
    """More work units than a launch holds: vidattn_bwd refuses them, so the
    workspace query has no size for them either."""
    assert binding.bwd_workspace(*args) == -1
    ids, B, H, S_q, S_kv, D = args[:6]
    A = 1 << 20   # an aligned address that is never read
    seg = A if ids else None
    st = binding.load_library().vidattn_bwd(A, A, A, A, A, A, None, seg, seg, A, A, A, B, H, S_q,
                                            S_kv, D, 0.1, (args + (0,))[6], A, (1 << 63) - 1, None)
    assert st == 3   # VIDATTN_ERR_BAD_SHAPE


def test_workspace_of_the_largest_sizes():
    """Up to the limit it has one."""
    assert binding.bwd_workspace(False, 1, 8000, 128 * 60000, 1, 64) == 8000 * 60000 * 1024
    assert binding.bwd_workspace(False, 65535, 1, 1 << 21, 0, 64) > 0
