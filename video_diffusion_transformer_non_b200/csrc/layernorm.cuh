// Layer norm of rows and its gradients, one memory-bound pass each.
//
//   y = xh w + b,  xh = (x - mean) rstd,  rstd = 1 / sqrt(var + eps)
//   with g = dy w, over the N features of a row:
//     dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum dy xh,  db = sum dy
//
// A row is held in registers by kLanes neighbouring threads, 8 features a
// thread and chunk, so that the mean, the variance about it and the result
// come from one read of the row.  Every thread keeps the same features for
// all its rows: weight and bias are read once, and the sums of dw and db over
// rows stay in its registers until the end; the CTAs' partial sums go to the
// workspace and are added by a second kernel in a fixed order.
//
// Rows of up to 1024 features belong to 8, 16 or 32 lanes of a warp, several
// rows in flight a thread (no barrier); longer ones to a CTA of ceil(N / 8)
// threads, the next rows' loads in flight while the present ones are reduced.
// Rows that lie on 16-byte boundaries with N a multiple of 8 move in 16-byte
// loads (8 neighbouring features a thread); any other N or stride takes the
// same code with single features, neighbouring lanes on neighbouring ones.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace vidattn {

constexpr int kLnMaxN = 16384;
constexpr int kLnThreads = 256;   // of the kernels with several rows a CTA

// Rows of a logical [B,H,S,N] array: strides in elements.
struct LnLayout {
  long long sb, sh, ss;
};

struct LnParams {
  const void *x, *dy, *w, *b;   // dy: backward only; w, b or null
  void* y;                      // y, or dx
  float *mean, *rstd;           // written by the forward (or null), read by the backward
  float* part;                  // backward: [gridDim.x][2][N] sums of dw and db, or null
  LnLayout lx, ldy, ly;
  int rows, N;
  FastDiv div_s, div_h;
  int params_bf16;
  float eps;
};

__device__ __forceinline__ long long ln_offset(const LnParams& p, const LnLayout& l, int row) {
  const uint32_t bh = fastdiv(uint32_t(row), p.div_s);
  const uint32_t s = uint32_t(row) - bh * p.div_s.d;
  const uint32_t b = fastdiv(bh, p.div_h);
  const uint32_t h = bh - b * p.div_h.d;
  return b * l.sb + h * l.sh + s * l.ss;
}

__device__ __forceinline__ float ln_bf16(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ __forceinline__ uint16_t ln_to_bf16(float v) {
  return static_cast<uint16_t>(pack_bf16x2(v, v) & 0xffffu);
}

// kC chunks of 8 features of one row, as read: X is float or uint16_t (bf16).
template <typename X, int kC, bool kVec>
struct LnFrag {
  static constexpr int kE = 8 * kC;
  static constexpr bool kBf16 = sizeof(X) == 2;
  static constexpr int kWords = kVec && kBf16 ? 4 * kC : kE;
  uint32_t r[kWords];

  // The row's feature that element e of this lane is.
  static __device__ __forceinline__ int col(int e, int lane, int lanes) {
    return kVec ? ((e >> 3) * lanes + lane) * 8 + (e & 7) : e * lanes + lane;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) r[i] = 0u;
  }
  // Features at and behind N read as 0.
  __device__ __forceinline__ void load(const X* row, int lane, int lanes, int N) {
    clear();
    if constexpr (kVec) {
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int at = (c * lanes + lane) * 8;
        if (at < N) {
#pragma unroll
          for (int k = 0; k < kWords / kC / 4; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(
                reinterpret_cast<const char*>(row + at) + 16 * k);
            uint32_t* d = r + c * (kWords / kC) + 4 * k;
            d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int at = e * lanes + lane;
        if (at < N) {
          if constexpr (kBf16) r[e] = uint32_t(row[at]) << 16;
          else r[e] = __float_as_uint(row[at]);
        }
      }
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (kVec && kBf16)
      return __uint_as_float((e & 1) ? r[e >> 1] & 0xffff0000u : r[e >> 1] << 16);
    else
      return __uint_as_float(r[e]);
  }
};

template <typename X, int kC, bool kVec>
__device__ __forceinline__ void ln_store(X* row, int lane, int lanes, int N,
                                         const float (&v)[8 * kC]) {
  if constexpr (kVec) {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int at = (c * lanes + lane) * 8;
      if (at >= N) continue;
      const float* s = v + 8 * c;
      uint4* d = reinterpret_cast<uint4*>(row + at);
      if constexpr (sizeof(X) == 2) {
        *d = make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]),
                        pack_bf16x2(s[6], s[7]));
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          d[k] = make_uint4(__float_as_uint(s[4 * k]), __float_as_uint(s[4 * k + 1]),
                            __float_as_uint(s[4 * k + 2]), __float_as_uint(s[4 * k + 3]));
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8 * kC; ++e) {
      const int at = e * lanes + lane;
      if (at < N) {
        if constexpr (sizeof(X) == 2) row[at] = ln_to_bf16(v[e]);
        else row[at] = v[e];
      }
    }
  }
}

// This thread's features of weight or bias (null: `none`).
template <int kC, bool kVec>
__device__ __forceinline__ void ln_params(const void* src, int bf16, int lane, int lanes, int N,
                                          float none, float (&v)[8 * kC]) {
#pragma unroll
  for (int e = 0; e < 8 * kC; ++e) {
    const int at = LnFrag<float, kC, kVec>::col(e, lane, lanes);
    v[e] = none;
    if (src != nullptr && at < N)
      v[e] = bf16 ? ln_bf16(__ldg(static_cast<const uint16_t*>(src) + at))
                  : __ldg(static_cast<const float*>(src) + at);
  }
}

// Sums over the lanes of a row: a part of a warp, or the CTA (kBlock), whose
// warps meet in shared memory (`buf`, 32 floats a value and call in turn).
template <bool kBlock, int kN>
__device__ __forceinline__ void ln_sum(float (&v)[kN], int lanes, float (*buf)[32]) {
  const int width = kBlock ? 32 : lanes;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= width) continue;
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if constexpr (kBlock) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kN; ++i) buf[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      v[i] = lane < n ? buf[i][lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
}

// The rows a thread works on: kR at a time.  kBlock: the CTA's kR next rows;
// else every group of kLanes threads has a row of its own in each of kR turns.
template <typename X, int kLanes, int kC, int kR, bool kVec, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) ln_fwd_kernel(const LnParams p) {
  constexpr bool kBlock = kLanes == 0;
  constexpr int kE = 8 * kC;
  using Frag = LnFrag<X, kC, kVec>;
  __shared__ float buf[kBlock ? 4 : 1][kR][32];
  const int lanes = kBlock ? blockDim.x : kLanes;
  const int lane = kBlock ? threadIdx.x : threadIdx.x % (kBlock ? 1 : kLanes);
  const int group = kBlock ? 0 : threadIdx.x / (kBlock ? 1 : kLanes);
  const int groups = kBlock ? 1 : kLnThreads / (kBlock ? 1 : kLanes);
  const X* x = static_cast<const X*>(p.x);
  X* y = static_cast<X*>(p.y);
  float w[kE], b[kE];
  ln_params<kC, kVec>(p.w, p.params_bf16, lane, lanes, p.N, 1.f, w);
  ln_params<kC, kVec>(p.b, p.params_bf16, lane, lanes, p.N, 0.f, b);
  const float n = float(p.N);
  const int64_t step = int64_t(gridDim.x) * groups * kR;
  int turn = 0;

  Frag next[kR];
  auto fetch = [&](int64_t base) {
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int64_t row = base + int64_t(i) * groups + group;
      if (row < p.rows) next[i].load(x + ln_offset(p, p.lx, int(row)), lane, lanes, p.N);
      else next[i].clear();
    }
  };
  int64_t base = int64_t(blockIdx.x) * groups * kR;
  if (base < p.rows) fetch(base);
  for (; base < p.rows; base += step, turn ^= 1) {
    Frag cur[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) cur[i] = next[i];
    if (kBlock && base + step < p.rows) fetch(base + step);
    float mean[kR], var[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      mean[i] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) mean[i] += cur[i].get(e);
    }
    ln_sum<kBlock>(mean, lanes, buf[kBlock ? 2 * turn : 0]);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      mean[i] /= n;
      var[i] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float d = cur[i].get(e) - mean[i];
        if (Frag::col(e, lane, lanes) < p.N) var[i] = fmaf(d, d, var[i]);
      }
    }
    ln_sum<kBlock>(var, lanes, buf[kBlock ? 2 * turn + 1 : 0]);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int64_t row = base + int64_t(i) * groups + group;
      const float rstd = 1.f / sqrtf(var[i] / n + p.eps);
      if (row < p.rows) {
        float v[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) v[e] = fmaf((cur[i].get(e) - mean[i]) * rstd, w[e], b[e]);
        ln_store<X, kC, kVec>(y + ln_offset(p, p.ly, int(row)), lane, lanes, p.N, v);
        if (lane == 0) {
          if (p.mean) p.mean[row] = mean[i];
          if (p.rstd) p.rstd[row] = rstd;
        }
      }
    }
    if (!kBlock && base + step < p.rows) fetch(base + step);
  }
}

template <typename X, int kLanes, int kC, int kR, bool kVec, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) ln_bwd_kernel(const LnParams p) {
  constexpr bool kBlock = kLanes == 0;
  constexpr int kE = 8 * kC;
  using Frag = LnFrag<X, kC, kVec>;
  __shared__ float buf[kBlock ? 2 : 1][2 * kR][32];
  // one row of partial sums of every warp
  __shared__ float sums[kBlock ? 1 : kLnThreads / 32][kBlock ? 1 : (kBlock ? 1 : kLanes) * kE];
  const int lanes = kBlock ? blockDim.x : kLanes;
  const int lane = kBlock ? threadIdx.x : threadIdx.x % (kBlock ? 1 : kLanes);
  const int group = kBlock ? 0 : threadIdx.x / (kBlock ? 1 : kLanes);
  const int groups = kBlock ? 1 : kLnThreads / (kBlock ? 1 : kLanes);
  const X* x = static_cast<const X*>(p.x);
  const X* dy = static_cast<const X*>(p.dy);
  X* dx = static_cast<X*>(p.y);
  float w[kE], dw[kE], db[kE];
  ln_params<kC, kVec>(p.w, p.params_bf16, lane, lanes, p.N, 1.f, w);
#pragma unroll
  for (int e = 0; e < kE; ++e) dw[e] = db[e] = 0.f;
  const float n = float(p.N);
  const int64_t step = int64_t(gridDim.x) * groups * kR;
  int turn = 0;

  Frag nx[kR], ng[kR];
  float nm[kR], nr[kR];
  auto fetch = [&](int64_t base) {
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int64_t row = base + int64_t(i) * groups + group;
      nm[i] = nr[i] = 0.f;
      if (row < p.rows) {
        nx[i].load(x + ln_offset(p, p.lx, int(row)), lane, lanes, p.N);
        ng[i].load(dy + ln_offset(p, p.ldy, int(row)), lane, lanes, p.N);
        nm[i] = __ldg(p.mean + row);
        nr[i] = __ldg(p.rstd + row);
      } else {
        nx[i].clear();
        ng[i].clear();
      }
    }
  };
  int64_t base = int64_t(blockIdx.x) * groups * kR;
  if (base < p.rows) fetch(base);
  for (; base < p.rows; base += step, turn ^= 1) {
    Frag cx[kR], cg[kR];
    float m[kR], r[kR], c[2 * kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) cx[i] = nx[i], cg[i] = ng[i], m[i] = nm[i], r[i] = nr[i];
    if (kBlock && base + step < p.rows) fetch(base + step);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float c1 = 0.f, c2 = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) {   // dy is 0 behind N
        const float xh = (cx[i].get(e) - m[i]) * r[i], g = cg[i].get(e);
        const float gw = g * w[e];
        c1 += gw;
        c2 = fmaf(gw, xh, c2);
        dw[e] = fmaf(g, xh, dw[e]);
        db[e] += g;
      }
      c[2 * i] = c1;
      c[2 * i + 1] = c2;
    }
    ln_sum<kBlock>(c, lanes, buf[kBlock ? turn : 0]);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int64_t row = base + int64_t(i) * groups + group;
      if (row < p.rows) {
        const float c1 = c[2 * i] / n, c2 = c[2 * i + 1] / n;
        float v[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const float xh = (cx[i].get(e) - m[i]) * r[i];
          v[e] = (fmaf(cg[i].get(e), w[e], -c1) - xh * c2) * r[i];
        }
        ln_store<X, kC, kVec>(dx + ln_offset(p, p.ly, int(row)), lane, lanes, p.N, v);
      }
    }
    if (!kBlock && base + step < p.rows) fetch(base + step);
  }
  if (p.part == nullptr) return;
  // this CTA's sums: the groups of a warp by shuffles, its warps in order
  float* part = p.part + int64_t(blockIdx.x) * 2 * p.N;
  if constexpr (kBlock) {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int at = Frag::col(e, lane, lanes);
      if (at < p.N) {
        part[at] = dw[e];
        part[p.N + at] = db[e];
      }
    }
  } else {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* v = which ? db : dw;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
#pragma unroll
        for (int o = 16; o >= kLanes; o >>= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
        if ((threadIdx.x & 31) < kLanes) sums[warp][e * kLanes + lane] = v[e];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < kLanes * kE; i += kLnThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kLnThreads / 32; ++k) t += sums[k][i];
        const int at = Frag::col(i / kLanes, i % kLanes, kLanes);
        if (at < p.N) part[which * p.N + at] = t;
      }
      __syncthreads();
    }
  }
}

// dw and db: the CTAs' partial sums [n_part][2][N] added in a fixed order, 32
// columns a CTA, a partial sum of each of 32 threads a column.
template <typename P>
__global__ void __launch_bounds__(1024)
    ln_params_grad_kernel(const float* __restrict__ part, int n_part, int N, P* dw, P* db) {
  __shared__ float s[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + tx;   // of 2 N
  float t = 0.f;
  if (i < 2 * N) {
#pragma unroll 8
    for (int k = ty; k < n_part; k += 32) t += __ldcg(part + int64_t(k) * 2 * N + i);
  }
  s[ty][tx] = t;
  __syncthreads();
  t = s[tx][ty];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int col = blockIdx.x * 32 + ty;
  if (tx != 0 || col >= 2 * N) return;
  P* out = col < N ? dw : db;
  if (out == nullptr) return;
  if constexpr (sizeof(P) == 2) out[col < N ? col : col - N] = ln_to_bf16(t);
  else out[col < N ? col : col - N] = t;
}

}  // namespace vidattn
