"""The kernels' bounded wait (csrc/bounded_wait.h), compiled for the host: a wait
for other warps ends with them; the wait for copies and products in flight ahead
of a CTA's end does not, only at their phase or at the time limit."""
import os
import subprocess

from video_diffusion_transformer_non_b200 import build

PROGRAM = r"""
#include "bounded_wait.h"
#include <cstdio>
using namespace vidattn;

// polls until the end, and how it ended, of a wait whose phase passes at poll
// `lands` (never: < 0) while another warp has given up or not; a poll takes 1000 ns
template <bool kDrain>
void one(const char* name, long lands, bool gone, uint64_t limit, uint64_t since) {
  long polls = 0;
  const WaitEnd e = bounded_wait<kDrain>([&] { return ++polls == lands; }, [&] { return gone; },
                                         [&] { return uint64_t(5000 + 1000 * polls); }, limit, since);
  std::printf("%s %d %ld\n", name, int(e), polls);
}

int main() {
  one<false>("wait_now", 1, true, 1u << 30, 0);
  one<false>("wait_later", 5000, false, 1u << 30, 0);
  one<false>("wait_gone", 5000, true, 1u << 30, 0);
  one<false>("wait_never", -1, false, 1000000, 0);
  one<true>("drain_now", 1, true, 1u << 30, 0);
  one<true>("drain_gone", 5000, true, 1u << 30, 0);
  one<true>("drain_never", -1, true, 1000000, 0);
  one<true>("drain_since", -1, true, 1000000, 5000);
}
"""


def test_ends(tmp_path):
    src, exe = tmp_path / "wait.cpp", tmp_path / "wait"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, "-o", exe, src], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {n: (int(e), int(k)) for n, e, k in (x.split() for x in lines if x)}
    phase, gone, timeout = range(3)
    assert got["wait_now"] == (phase, 1) and got["drain_now"] == (phase, 1)
    assert got["wait_later"] == (phase, 5000)
    # the others are looked at every 256 polls
    assert got["wait_gone"][0] == gone and got["wait_gone"][1] <= 257
    assert got["drain_gone"] == (phase, 5000)
    # 1000 polls from the first look at the clock, or from `since`, to the next look
    assert got["wait_never"][0] == timeout and 1000 < got["wait_never"][1] <= 257 + 1000 + 256
    assert got["drain_never"][0] == timeout and 1000 < got["drain_never"][1] <= 257 + 1000 + 256
    assert got["drain_since"][0] == timeout and 1000 < got["drain_since"][1] <= 1000 + 257


def test_the_backward_kernel_leaves_with_drains():
    """Every wait ahead of the kernel's end that must not be cut short is one."""
    with open(os.path.join(build.CSRC, "bwd_kernel.cuh")) as f:
        text = f.read()
    unit = text[text.index("__device__ __forceinline__ void bwd_unit("):]
    for bar in ("a_full(k)", "b_full(k)", "fixed_full(which)"):
        assert f"bwd_drain({bar}" in unit
    assert unit.count("bwd_drain(done, 0") == 1
    assert "__syncthreads_or(threadIdx.x == 0 && *reinterpret_cast<volatile int*>(p.err) != 0)" \
        in unit
