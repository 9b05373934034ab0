"""Calls from threads of their own: a new thread has no current CUDA context until
a runtime call binds it, and the library is then already set up by another
thread, so that its first call there may be a driver call.  Results are the
main thread's, bit for bit, also for calls made at the same time."""
import threading

import pytest
import torch

from video_diffusion_transformer_non_b200 import autograd, binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def in_thread(fn):
    res = []

    def go():
        try:
            res.append(fn())
        except BaseException as e:   # handed to the test
            res.append(e)
    t = threading.Thread(target=go)
    t.start()
    t.join()
    if isinstance(res[0], BaseException):
        raise res[0]
    return res[0]


def data(S, D=64, H=2):
    return [torch.randn((1, H, S, D), device="cuda").to(BF) for _ in range(4)]


def test_first_calls_in_new_threads():
    """Set up here, then every call of new buffers in a thread of its own."""
    q, k, v, g = data(140)
    out, lse = binding.attention(q, k, v)
    binding.attention_bwd(g, q, k, v, out, lse)
    binding.layer_norm(q)
    turn = dict(grid=(2, 7, 10), bands=(16, 24, 24), freqs=binding.rope3d_frequencies((16, 24, 24)))
    binding.rope3d_scaled(q, k, **turn)
    q, k, v, g = data(150)
    out, lse = in_thread(lambda: binding.attention(q, k, v))
    grads = in_thread(lambda: binding.attention_bwd(g, q, k, v, out, lse))
    y = in_thread(lambda: binding.layer_norm(q))
    rot = in_thread(lambda: binding.rope3d_scaled(q, k, **turn))
    torch.cuda.synchronize()
    for a, b in zip((out, lse, *grads, *y, *rot),
                    (*binding.attention(q, k, v), *binding.attention_bwd(g, q, k, v, out, lse),
                     *binding.layer_norm(q), *binding.rope3d_scaled(q, k, **turn))):
        assert torch.equal(a, b)


def test_backward_in_autograds_thread_after_set_up():
    q, k, v, g = data(160)
    out, lse = binding.attention(q, k, v)
    binding.attention_bwd(g, q, k, v, out, lse)
    q, k, v, g = data(170)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out, lse = autograd.attention(*leaves)
    out.backward(g)
    want = binding.attention_bwd(g, q.detach(), k.detach(), v.detach(), out.detach(), lse.detach())
    for t, w in zip(leaves, want):
        assert torch.equal(t.grad, w)


def test_threads_at_once():
    """Four threads on streams of their own, many calls each."""
    sets = [data(200 + 64 * i) for i in range(4)]
    want = []
    for q, k, v, g in sets:
        out, lse = binding.attention(q, k, v)
        want.append(binding.attention_bwd(g, q, k, v, out, lse))
    torch.cuda.synchronize()
    errors = []

    def go(i):
        try:
            q, k, v, g = sets[i]
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    out, lse = binding.attention(q, k, v)
                    got = binding.attention_bwd(g, q, k, v, out, lse)
                stream.synchronize()
            for a, b in zip(got, want[i]):
                assert torch.equal(a, b)
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=go, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert binding.device_status() == 0
