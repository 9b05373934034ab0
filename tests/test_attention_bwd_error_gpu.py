"""The backward pass after a wait of the library has run out (the error word is
set): its kernel leaves at once, as a whole; once the word is read and cleared,
the next call is right."""
import pytest
import torch

from test_attention_bwd_gpu import make
from video_diffusion_transformer_non_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,ids,n_split", [(64, None, 0), (128, "far", 0), (128, None, 3)])
def test_error_word(D, ids, n_split):
    x = make(2, 3, 700, 500, D, 50, ids)
    seg = x["seg_q"], x["seg_kv"]
    out, lse = binding.attention(x["q"], x["k"], x["v"], *seg)
    args = (x["dout"], x["q"], x["k"], x["v"], out, lse, *seg)
    want = binding.attention_bwd(*args, n_split=n_split)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    assert binding.selftest_timeout(1000) == 0
    for _ in range(3):
        binding.attention_bwd(*args, n_split=n_split)
    assert binding.device_status() != 0      # reads and clears
    assert binding.device_status() == 0
    got = binding.attention_bwd(*args, n_split=n_split)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
