// Host side of the layer norm (vidattn_layernorm, vidattn_layernorm_bwd):
// argument checks and the choice of kernel.  The operations are documented in
// include/vidattn.h, the kernels in layernorm.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include "../../include/vidattn.h"
#include "internal.h"
#include "layernorm.cuh"

namespace vidattn {
namespace {

using LnKernel = void (*)(const LnParams);

struct LnChoice {
  LnKernel kernel;
  int threads, rows;   // threads a CTA; rows a CTA takes at a time
  int ring, ring_max;  // bytes of shared memory, and with the most threads
};

// kLanes of a warp a row (0: the CTA), kC chunks of 8 features a thread; forward
// (backward) kRf (kRb) rows a thread at a time and registers for kFwd (kBwd) CTAs
// on an SM: the reductions leave a CTA idle, its other row or the next CTA fills
// in.  The backward pass has no registers for a second long row.
template <typename X, int kLanes, int kC, int kRf, int kRb, int kV, int kMaxThreads, int kFwd,
          int kBwd>
LnChoice ln_form(bool bwd, int threads) {
  using Frag = LnFrag<X, kC, kV>;
  const int piece = Frag::kWords * 4, tensors = bwd ? 2 : 1, rows = bwd ? kRb : kRf;
  const int stages = ln_stages(kMaxThreads, rows, tensors, piece);
  return LnChoice{bwd ? ln_bwd_kernel<X, kLanes, kC, kRb, kV, kMaxThreads, kBwd>
                      : ln_fwd_kernel<X, kLanes, kC, kRf, kV, kMaxThreads, kFwd>,
                  threads, kLanes ? threads / kLanes * rows : rows,
                  stages >= 2 ? stages * threads * rows * tensors * piece : 0,
                  stages >= 2 ? stages * kMaxThreads * rows * tensors * piece : 0};
}

// The smallest form that holds a row of N features in registers.  Forward, one
// and two rows at a time (bf16, us): 32760 x 5120 129 and 114, 16000 x 5119 172
// and 136, 32760 x 2560 63.5 and 65.6, 16000 x 8192 123 and 112, 100000 x 768 78
// and 63; 200000 x 384 62.4 and 63.5, so one there.  32760 x 6144 172 with one CTA
// on an SM, 141 with two.  Fewer rows than the device has warps of this form: one a
// warp (226 x 1001 fp32: 8.2, 10.2 with two).
template <typename X, int kV>
LnChoice ln_choose_x(bool bwd, int N, int64_t rows) {
  if (N <= 64) return ln_form<X, 8, 1, 2, 2, kV, kLnThreads, 3, 2>(bwd, kLnThreads);
  if (N <= 128) return ln_form<X, 16, 1, 2, 2, kV, kLnThreads, 3, 2>(bwd, kLnThreads);
  if (N <= 256) return ln_form<X, 32, 1, 2, 2, kV, kLnThreads, 3, 2>(bwd, kLnThreads);
  if (N <= 512) return ln_form<X, 32, 2, 1, 1, kV, kLnThreads, 2, 2>(bwd, kLnThreads);
  if (N <= 1024 && rows <= 148 * 8)
    return ln_form<X, 32, 4, 1, 1, kV, kLnThreads, 1, 1>(bwd, kLnThreads);
  if (N <= 1024) return ln_form<X, 32, 4, 2, 1, kV, kLnThreads, 1, 1>(bwd, kLnThreads);
  const int threads = (N + 511) / 512 * 32;
  if (threads <= 320) return ln_form<X, 0, 2, 2, 1, kV, 320, 2, 2>(bwd, threads);
  if (threads <= 384) return ln_form<X, 0, 2, 2, 1, kV, 384, 2, 1>(bwd, threads);
  if (threads <= 512) return ln_form<X, 0, 2, 2, 1, kV, 512, 1, 1>(bwd, threads);
  return ln_form<X, 0, 2, 1, 1, kV, 1024, 1, 1>(bwd, threads);
}
// piece: 16, 4 or 2, the bytes that every row's start and length are a multiple of.
LnChoice ln_choose(bool bwd, bool bf16, int piece, int N, int64_t rows) {
  if (!bf16)
    return piece == 16 ? ln_choose_x<float, 4>(bwd, N, rows) : ln_choose_x<float, 1>(bwd, N, rows);
  if (piece == 16) return ln_choose_x<uint16_t, 8>(bwd, N, rows);
  return piece == 4 ? ln_choose_x<uint16_t, 2>(bwd, N, rows) : ln_choose_x<uint16_t, 1>(bwd, N, rows);
}

// CTAs of a launch: enough for all rows, at most what the device holds at once
// (every CTA then walks over rows and reads the parameters once).
// A kernel's shared-memory limit is raised on its first use on a device (and
// again after vidattn_release).
struct LnReady {
  int epoch = -1, per_sm = 0;
};
std::mutex g_ln_mu;
std::map<std::pair<int, std::pair<LnKernel, int>>, LnReady> g_ln_ready;
int ln_grid(int dev, int sms, const LnChoice& c, int64_t rows) {
  const int now = host::epoch();
  int per_sm = 0;
  {
    std::lock_guard<std::mutex> lk(g_ln_mu);
    LnReady& r = g_ln_ready[{dev, {c.kernel, c.threads}}];
    if (r.epoch != now) {
      if (cudaFuncSetAttribute(c.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               c.ring_max) != cudaSuccess ||
          cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r.per_sm, c.kernel, c.threads, c.ring) !=
              cudaSuccess)
        return 0;
      r.epoch = now;
    }
    per_sm = r.per_sm;
  }
  if (per_sm < 1) return 0;
  return int(std::min<int64_t>((rows + c.rows - 1) / c.rows, int64_t(sms) * per_sm));
}
// The most CTAs a backward launch of these sizes uses on any device it runs
// on (sm_100a: at most 148 SMs x 2048 threads).
int64_t ln_bwd_parts(const LnChoice& c, int64_t rows) {
  return std::min<int64_t>((rows + c.rows - 1) / c.rows, 148 * (2048 / c.threads));
}

bool ln_apart(int B, int H, int S, int N, const int64_t s[3]) {
  const int64_t sizes[3] = {B, H, S};
  return host::rows_apart(sizes, s, N);
}
bool ln_in_place_ok(const void* in, const void* out, int B, int H, int S, const int64_t si[3],
                    const int64_t so[3]) {
  const int64_t sizes[3] = {B, H, S};
  return !host::over_another_layout(in, out, sizes, si, so);
}
// Any read layout: strides not negative.
bool ln_readable(const int64_t s[3]) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }
bool ln_on(const void* p, const int64_t s[3], int item, int bytes) {
  return host::aligned(p, bytes) && s[0] * item % bytes == 0 && s[1] * item % bytes == 0 &&
         s[2] * item % bytes == 0;
}
LnLayout ln_layout(int B, int H, int S, const int64_t s[3]) {
  const bool heads = H == 1 || s[1] == S * s[2];
  const bool batch = B == 1 || (heads && s[0] == (H == 1 ? S * s[2] : H * s[1]));
  return LnLayout{s[0], s[1], s[2], (S > 1 || (B == 1 && H == 1)) && heads && batch && s[2] <= INT_MAX};
}

bool ln_sizes_ok(int B, int H, int S, int N) {
  return B >= 1 && H >= 1 && S >= 0 && N >= 1 && N <= kLnMaxN &&
         int64_t(B) * H <= INT_MAX && int64_t(B) * H * S <= INT_MAX;
}
bool ln_type_ok(int t) { return t == VIDATTN_BF16 || t == VIDATTN_F32; }
int ln_item(int t) { return t == VIDATTN_BF16 ? 2 : 4; }

}  // namespace
}  // namespace vidattn

using namespace vidattn;

extern "C" {

VIDATTN_API int vidattn_layernorm(const void* x, const void* weight, const void* bias, void* y,
                                  float* mean, float* rstd, int B, int H, int S, int N,
                                  const int64_t* x_strides, const int64_t* y_strides, int x_type,
                                  int param_type, double eps, vidattn_stream_t stream_) {
  if (!x_strides || !y_strides) return VIDATTN_ERR_NULL;
  if (!ln_sizes_ok(B, H, S, N) || !ln_type_ok(x_type) || !ln_type_ok(param_type) ||
      !std::isfinite(eps) || eps < 0.0 || !ln_readable(x_strides) ||
      !ln_apart(B, H, S, N, y_strides))
    return VIDATTN_ERR_BAD_SHAPE;
  if (S == 0) return VIDATTN_OK;
  if (!x || !y) return VIDATTN_ERR_NULL;
  if (!ln_in_place_ok(x, y, B, H, S, x_strides, y_strides)) return VIDATTN_ERR_BAD_SHAPE;
  const int item = ln_item(x_type), pitem = ln_item(param_type);
  if (!host::aligned(x, item) || !host::aligned(y, item) || !host::aligned(weight, pitem) ||
      !host::aligned(bias, pitem) || !host::aligned(mean, 4) || !host::aligned(rstd, 4))
    return VIDATTN_ERR_MISALIGNED;
  int dev = 0, sms = 0;
  int* err = nullptr;
  const int st = host::device(&dev, &err, &sms);
  if (st != VIDATTN_OK) return st;
  LnParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = x;
  p.w = weight;
  p.b = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.lx = ln_layout(B, H, S, x_strides);
  p.ly = ln_layout(B, H, S, y_strides);
  p.rows = B * H * S;
  p.N = N;
  p.div_s = make_fastdiv(uint32_t(S));
  p.div_h = make_fastdiv(uint32_t(H));
  p.params_bf16 = param_type == VIDATTN_BF16;
  p.inv_n = 1.f / float(N);
  p.eps = float(eps);
  auto fits = [&](int bytes) {
    return N * item % bytes == 0 && ln_on(x, x_strides, item, bytes) &&
           ln_on(y, y_strides, item, bytes);
  };
  const LnChoice c = ln_choose(false, x_type == VIDATTN_BF16, fits(16) ? 16 : fits(4) ? 4 : 2, N,
                               p.rows);
  const int grid = ln_grid(dev, sms, c, p.rows);
  if (grid < 1) return VIDATTN_ERR_CUDA;
  c.kernel<<<grid, c.threads, c.ring, reinterpret_cast<cudaStream_t>(stream_)>>>(p);
  return cudaGetLastError() == cudaSuccess ? VIDATTN_OK : VIDATTN_ERR_CUDA;
}

VIDATTN_API int64_t vidattn_layernorm_bwd_workspace(int B, int H, int S, int N, int x_type) {
  if (!ln_sizes_ok(B, H, S, N) || !ln_type_ok(x_type)) return -1;
  const int64_t rows = int64_t(B) * H * S;
  const LnChoice c = ln_choose(true, x_type == VIDATTN_BF16, 16, N, rows);
  return (ln_bwd_parts(c, rows) * 2 * N * 4 + 255) & ~int64_t(255);
}

VIDATTN_API int vidattn_layernorm_bwd(const void* dy, const void* x, const float* mean,
                                      const float* rstd, const void* weight, void* dx,
                                      void* dweight, void* dbias, int B, int H, int S, int N,
                                      const int64_t* dy_strides, const int64_t* x_strides,
                                      const int64_t* dx_strides, int x_type, int param_type,
                                      void* workspace, int64_t workspace_bytes,
                                      vidattn_stream_t stream_) {
  if (!dy_strides || !x_strides || !dx_strides) return VIDATTN_ERR_NULL;
  if (!ln_sizes_ok(B, H, S, N) || !ln_type_ok(x_type) || !ln_type_ok(param_type) ||
      !ln_readable(x_strides) || !ln_readable(dy_strides) ||
      !ln_apart(B, H, S, N, dx_strides))
    return VIDATTN_ERR_BAD_SHAPE;
  const int item = ln_item(x_type), pitem = ln_item(param_type);
  const bool params = dweight || dbias;
  if (S > 0 && (!dy || !x || !mean || !rstd || !dx || (params && !workspace)))
    return VIDATTN_ERR_NULL;
  if (S > 0 && (!ln_in_place_ok(x, dx, B, H, S, x_strides, dx_strides) ||
                !ln_in_place_ok(dy, dx, B, H, S, dy_strides, dx_strides)))
    return VIDATTN_ERR_BAD_SHAPE;
  if (!host::aligned(x, item) || !host::aligned(dy, item) || !host::aligned(dx, item) ||
      !host::aligned(weight, pitem) || !host::aligned(dweight, pitem) ||
      !host::aligned(dbias, pitem) || !host::aligned(mean, 4) || !host::aligned(rstd, 4) ||
      (params && !host::aligned(workspace, 256)))
    return VIDATTN_ERR_MISALIGNED;
  if (S > 0 && params &&
      workspace_bytes < vidattn_layernorm_bwd_workspace(B, H, S, N, x_type))
    return VIDATTN_ERR_SCRATCH_LIMIT;
  if (S == 0 && !params) return VIDATTN_OK;
  int dev = 0, sms = 0;
  int* err = nullptr;
  const int st = host::device(&dev, &err, &sms);
  if (st != VIDATTN_OK) return st;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (S == 0) {   // sums over no rows
    bool ok = true;
    for (void* d : {dweight, dbias})
      if (d) ok = ok && cudaMemsetAsync(d, 0, size_t(N) * pitem, stream) == cudaSuccess;
    return ok ? VIDATTN_OK : VIDATTN_ERR_CUDA;
  }
  LnParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = x;
  p.dy = dy;
  p.w = weight;
  p.y = dx;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.part = params ? static_cast<float*>(workspace) : nullptr;
  p.lx = ln_layout(B, H, S, x_strides);
  p.ldy = ln_layout(B, H, S, dy_strides);
  p.ly = ln_layout(B, H, S, dx_strides);
  p.rows = B * H * S;
  p.N = N;
  p.div_s = make_fastdiv(uint32_t(S));
  p.div_h = make_fastdiv(uint32_t(H));
  p.params_bf16 = param_type == VIDATTN_BF16;
  p.inv_n = 1.f / float(N);
  auto fits = [&](int bytes) {
    return N * item % bytes == 0 && ln_on(x, x_strides, item, bytes) &&
           ln_on(dy, dy_strides, item, bytes) && ln_on(dx, dx_strides, item, bytes);
  };
  const LnChoice c = ln_choose(true, x_type == VIDATTN_BF16, fits(16) ? 16 : fits(4) ? 4 : 2, N,
                               p.rows);
  int grid = ln_grid(dev, sms, c, p.rows);
  if (grid < 1) return VIDATTN_ERR_CUDA;
  grid = int(std::min<int64_t>(grid, ln_bwd_parts(c, p.rows)));
  c.kernel<<<grid, c.threads, c.ring, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return VIDATTN_ERR_CUDA;
  if (params) {
    const unsigned blocks = (2 * N + 31) / 32;
    if (p.params_bf16)
      ln_params_grad_kernel<<<blocks, 1024, 0, stream>>>(
          p.part, grid, N, static_cast<uint16_t*>(dweight), static_cast<uint16_t*>(dbias));
    else
      ln_params_grad_kernel<<<blocks, 1024, 0, stream>>>(
          p.part, grid, N, static_cast<float*>(dweight), static_cast<float*>(dbias));
    if (cudaGetLastError() != cudaSuccess) return VIDATTN_ERR_CUDA;
  }
  return VIDATTN_OK;
}

}  // extern "C"
