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
// Rows of up to 1024 features belong to 8, 16 or 32 lanes of a warp (no
// barrier); longer ones to a CTA with 16 features a thread.  What bounds the
// pass is how many bytes are in flight: rows go through a ring in shared memory,
// filled by cp.async up to three turns ahead, each thread copying and reading its
// own features (so the ring needs no barrier).  Rows on 16-byte boundaries with
// N a multiple of 16 bytes move in pieces of 16 bytes, the others in pieces of 4;
// bf16 rows on odd places or of odd length are put together from 4-byte pieces
// of neighbouring lanes, with a barrier a turn.
//
// Measured (B200): 32760 rows of 5120 bf16 in 113 us (5.9 TB/s, 91 % of the
// copy rate), backward 196 us (5.1 TB/s); 524160 rows of 128 in 55 us (4.9 TB/s),
// backward, from a [B,S,H,D] projection, 74 - 78 us (5.2 - 5.5 TB/s).  16000 rows,
// forward and backward: of 8192 bf16 113 and 164 us, of 5118 (pieces of 4 bytes)
// 90 and 154, of 5119 (odd) 135 and 238, of 5120 fp32 119 and 178, of 5119 fp32
// 148 and 227; 8000 rows of 16384: bf16 125 and 285, fp32 173 and 657 (backward
// without the ring).  Feature by feature through registers the rows of 5119 bf16
// took 258 and 572.  Instruction issue bounds it (51 - 64 % of the slots); a deeper
// ring, one CTA of twice the threads or 32 features a thread were slower.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx_train.cuh"

namespace vidattn {

constexpr int kLnMaxN = 16384;
constexpr int kLnThreads = 256;   // of the kernels with several rows a CTA

// Rows of a logical [B,H,S,N] array: strides in elements; flat: row r of all
// B * H * S lies at r * ss (below 2^31).
struct LnLayout {
  long long sb, sh, ss;
  int flat;
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
  float eps, inv_n;
};

__device__ __forceinline__ long long ln_offset(const LnParams& p, const LnLayout& l,
                                               uint32_t row) {
  if (l.flat) return (long long)(uint64_t(row) * uint32_t(l.ss));
  const uint32_t bh = fastdiv(row, p.div_s);
  const uint32_t s = row - bh * p.div_s.d;
  const uint32_t b = fastdiv(bh, p.div_h);
  const uint32_t h = bh - b * p.div_h.d;
  return b * l.sb + h * l.sh + s * l.ss;
}

__device__ __forceinline__ float ln_bf16(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ __forceinline__ uint16_t ln_to_bf16(float v) {
  return static_cast<uint16_t>(pack_bf16x2(v, v) & 0xffffu);
}

// Turns of the ring: up to 4 in 192 KB, or in 64 KB where several CTAs fit an SM
// (fewer than 2, backward with fp32 rows of more than 8192: they go through
// registers).
__host__ __device__ constexpr int ln_stages(int threads, int rows, int tensors, int bytes_a_thread) {
  const int stage = threads * rows * tensors * bytes_a_thread;
  int n = (threads <= 512 ? 65536 : 196608) / stage;
  if (n < 2 && 2 * stage <= 196608) n = 2;
  return n > 4 ? 4 : n;
}
__device__ __forceinline__ void ln_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ln_copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ln_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void ln_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// The row's feature that element e of a lane is: pieces of kV neighbouring
// features, neighbouring lanes on neighbouring pieces.
template <int kV>
__device__ __forceinline__ int ln_col(int e, int lane, int lanes) {
  return ((e / kV) * lanes + lane) * kV + e % kV;
}

// 8 kC features of one row, as read: X is float or uint16_t (bf16), in pieces
// of kV (16 or 4 bytes), of which N is a multiple.  bf16 with kV = 1: rows of
// any length on any place.  Their lanes hold pairs of features too; what is
// copied are the 4 aligned bytes that hold two features of the row, which on an
// odd place are one lane's second and the next one's first, and the one or two
// features left at the row's ends are read as they are used.
template <typename X, int kC, int kV>
struct LnFrag {
  static constexpr bool kOdd = sizeof(X) == 2 && kV == 1;
  static constexpr int kCols = kOdd ? 2 : kV;   // neighbouring features of a lane
  static constexpr int kE = 8 * kC;
  static constexpr int kPieces = kE / kCols;
  static constexpr int kPieceBytes = kCols * int(sizeof(X));
  static constexpr bool kPacked = sizeof(X) == 2;
  static constexpr int kWords = kPacked ? kE / 2 : kE;
  uint32_t r[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) r[i] = 0u;
  }
  // 1: the row starts on the second half of 4 aligned bytes
  static __device__ __forceinline__ int shift(const X* row) {
    return kOdd ? int(reinterpret_cast<uintptr_t>(row) >> 1) & 1 : 0;
  }
  // Features at and behind N read as 0.
  __device__ __forceinline__ void load(const X* row, int lane, int lanes, int N) {
    static_assert(!kOdd, "only rows of fp32 go without the ring");
    clear();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = (i * lanes + lane) * kCols;
      if (at >= N) continue;
      uint32_t* d = r + i * (kWords / kPieces);
      if constexpr (kPieceBytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + at);
        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
      } else {
        d[0] = *reinterpret_cast<const uint32_t*>(row + at);
      }
    }
  }
  // The same by way of shared memory: a piece every `pitch` bytes from `ring`,
  // a shared address of this thread's.
  static __device__ __forceinline__ void copy(uint32_t ring, uint32_t pitch, const X* row,
                                              int lane, int lanes, int N) {
    const int sh = shift(row);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = (i * lanes + lane) * kCols - sh;
      if constexpr (kOdd) {
        if (at >= 0 && at + 1 < N) ln_copy4(ring + i * pitch, row + at);
      } else {
        if (at >= N) continue;
        if constexpr (kPieceBytes == 16) ln_copy16(ring + i * pitch, row + at);
        else ln_copy4(ring + i * pitch, row + at);
      }
    }
  }
  static __device__ __forceinline__ uint32_t word(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
  }
  // kOdd: reads what other lanes of the row copied (a barrier lies between)
  __device__ __forceinline__ void read(uint32_t ring, uint32_t pitch, const X* row, int lane,
                                       int lanes, int N) {
    const int sh = shift(row);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = (i * lanes + lane) * kCols;
      uint32_t* d = r + i * (kWords / kPieces);
      if constexpr (kOdd) {
        const uint32_t mine = ring + i * pitch;
        d[0] = 0u;
        if (at >= N) continue;
        if (sh == 0) {
          d[0] = at + 1 < N ? word(mine) : uint32_t(row[at]);
        } else {
          const uint32_t next = lane + 1 < lanes ? mine + 4 : mine - 4 * lane + pitch;
          d[0] = at > 0 ? word(mine) >> 16 : uint32_t(row[0]);
          if (at + 2 < N) d[0] |= word(next) << 16;
          else if (at + 1 < N) d[0] |= uint32_t(row[at + 1]) << 16;
        }
      } else if constexpr (kPieceBytes == 16) {
        d[0] = d[1] = d[2] = d[3] = 0u;
        if (at < N)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                       : "r"(ring + i * pitch)
                       : "memory");
      } else {
        d[0] = at < N ? word(ring + i * pitch) : 0u;
      }
    }
  }
  // Elements 2 i and 2 i + 1.
  __device__ __forceinline__ float2 get2(int i) const {
    if constexpr (kPacked)
      return make_float2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
    else
      return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
  }
};
__device__ __forceinline__ float2 ln_both(float v) { return make_float2(v, v); }

template <typename X, int kC, int kV>
__device__ __forceinline__ void ln_store(X* row, int lane, int lanes, int N,
                                         const float2 (&v)[4 * kC]) {
  using Frag = LnFrag<X, kC, kV>;
  const int sh = Frag::shift(row);
#pragma unroll
  for (int i = 0; i < Frag::kPieces; ++i) {
    const int at = (i * lanes + lane) * Frag::kCols;
    if (at >= N) continue;
    const float2* s = v + i * Frag::kCols / 2;
    if constexpr (sizeof(X) == 4) {
      if constexpr (kV == 4)
        *reinterpret_cast<float4*>(row + at) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
      else
        row[at] = (i & 1) ? s[0].y : s[0].x;
    } else if constexpr (kV == 8) {
      *reinterpret_cast<uint4*>(row + at) =
          make_uint4(pack_bf16x2(s[0].x, s[0].y), pack_bf16x2(s[1].x, s[1].y),
                     pack_bf16x2(s[2].x, s[2].y), pack_bf16x2(s[3].x, s[3].y));
    } else {
      const uint32_t w = pack_bf16x2(s[0].x, s[0].y);
      if (!Frag::kOdd || (sh == 0 && at + 1 < N)) {
        *reinterpret_cast<uint32_t*>(row + at) = w;
      } else {
        row[at] = uint16_t(w & 0xffffu);
        if (at + 1 < N) row[at + 1] = uint16_t(w >> 16);
      }
    }
  }
}

// This thread's features of weight or bias (null: `none`).
template <typename P, int kC, int kCols>
__device__ __forceinline__ void ln_params_of(const P* src, int lane, int lanes, int N,
                                             float2 (&v)[4 * kC]) {
  P t[8 * kC];
#pragma unroll
  for (int e = 0; e < 8 * kC; ++e) {
    const int at = ln_col<kCols>(e, lane, lanes);
    t[e] = at < N ? __ldg(src + at) : P(0);
  }
#pragma unroll
  for (int e = 0; e < 4 * kC; ++e) {
    if constexpr (sizeof(P) == 2) v[e] = make_float2(ln_bf16(t[2 * e]), ln_bf16(t[2 * e + 1]));
    else v[e] = make_float2(t[2 * e], t[2 * e + 1]);
  }
}
template <int kC, int kCols>
__device__ __forceinline__ void ln_params(const void* src, int bf16, int lane, int lanes, int N,
                                          float none, float2 (&v)[4 * kC]) {
  if (src == nullptr) {
#pragma unroll
    for (int e = 0; e < 4 * kC; ++e) v[e] = ln_both(none);
  } else if (bf16) {
    ln_params_of<uint16_t, kC, kCols>(static_cast<const uint16_t*>(src), lane, lanes, N, v);
  } else {
    ln_params_of<float, kC, kCols>(static_cast<const float*>(src), lane, lanes, N, v);
  }
  // kept in registers, not read again for every row
#pragma unroll
  for (int e = 0; e < 4 * kC; ++e) asm volatile("" : "+f"(v[e].x), "+f"(v[e].y));
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
    for (int i = 0; i < kN; ++i) {   // every thread adds the warps' sums, in order
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < n; w += 4) {   // buf is zero behind the last warp
        const float4 u = *reinterpret_cast<const float4*>(&buf[i][w]);
        t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
      }
      v[i] = (t.x + t.y) + (t.z + t.w);
    }
  }
}

extern __shared__ uint4 ln_ring[];

// What both kernels share: the rows a thread works on, kR at a time (kBlock:
// the CTA's kR next rows; else every group of kLanes threads has a row of its
// own in each of kR turns), its features, and the ring.
template <typename X, int kLanes, int kC, int kR, int kV, int kMaxThreads, int kTensors>
struct LnWalk {
  static constexpr bool kBlock = kLanes == 0;
  using Frag = LnFrag<X, kC, kV>;
  static constexpr int kS = ln_stages(kMaxThreads, kR, kTensors, Frag::kWords * 4);
  static constexpr bool kRing = kS >= 2;
  int lanes, lane, groups, group;
  uint32_t row, step, pitch, stage, ring, in, out;   // in, out: ring addresses of this thread's
  __device__ __forceinline__ explicit LnWalk(const LnParams& p) {
    lanes = kBlock ? blockDim.x : kLanes;
    lane = kBlock ? threadIdx.x : threadIdx.x % (kBlock ? 1 : kLanes);
    group = kBlock ? 0 : threadIdx.x / (kBlock ? 1 : kLanes);
    groups = kBlock ? 1 : kLnThreads / (kBlock ? 1 : kLanes);
    row = blockIdx.x * groups * kR + group;
    step = gridDim.x * groups * kR;
    pitch = blockDim.x * Frag::kPieceBytes;
    stage = pitch * Frag::kPieces * kTensors * kR;
    ring = smem_u32(ln_ring) + threadIdx.x * Frag::kPieceBytes;
    in = out = ring;
  }
  // the CTA's first row of this turn decides whether the turn is made at all
  __device__ __forceinline__ bool any(const LnParams& p) const { return row - group < p.rows; }
  __device__ __forceinline__ uint32_t slot(uint32_t at, int i, int tensor) const {
    return at + (i * kTensors + tensor) * Frag::kPieces * pitch;
  }
  __device__ __forceinline__ void next(uint32_t& at) const {
    at += stage;
    if (at == ring + kS * stage) at = ring;
  }
};

template <typename X, int kLanes, int kC, int kR, int kV, int kMaxThreads, int kCtas>
__global__ void __launch_bounds__(kMaxThreads, kCtas) ln_fwd_kernel(const LnParams p) {
  using Walk = LnWalk<X, kLanes, kC, kR, kV, kMaxThreads, 1>;
  using Frag = typename Walk::Frag;
  constexpr bool kBlock = Walk::kBlock;
  constexpr int kE = 8 * kC, kS = Walk::kS;
  static_assert(kS >= 2, "every forward form has a ring");
  __shared__ __align__(16) float buf[kBlock ? 4 : 1][kR][32];
  if (kBlock) {
    for (int i = threadIdx.x; i < 4 * kR * 32; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  Walk t(p);
  const int lane = t.lane, lanes = t.lanes;
  const X* x = static_cast<const X*>(p.x);
  X* y = static_cast<X*>(p.y);
  auto fetch = [&](uint32_t row0) {
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const uint32_t row = row0 + i * t.groups;
      if (row < p.rows)
        Frag::copy(t.slot(t.in, i, 0), t.pitch, x + ln_offset(p, p.lx, row), lane, lanes, p.N);
    }
    t.next(t.in);
    ln_commit();
  };
#pragma unroll
  for (int k = 0; k < kS - 1; ++k) fetch(t.row + k * t.step);
  float2 w[kE / 2], b[kE / 2];
  ln_params<kC, Frag::kCols>(p.w, p.params_bf16, lane, lanes, p.N, 1.f, w);
  ln_params<kC, Frag::kCols>(p.b, p.params_bf16, lane, lanes, p.N, 0.f, b);
  for (int turn = 0; t.any(p); turn ^= 1, t.row += t.step) {
    Frag cur[kR];
    fetch(t.row + (kS - 1) * t.step);
    ln_wait<kS - 1>();
    if (Frag::kOdd) kBlock ? __syncthreads() : __syncwarp();
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const uint32_t row = min(t.row + i * t.groups, uint32_t(p.rows - 1));
      cur[i].read(t.slot(t.out, i, 0), t.pitch,
                  Frag::kOdd ? x + ln_offset(p, p.lx, row) : nullptr, lane, lanes, p.N);
    }
    t.next(t.out);
    float mean[kR], var[kR];
    float2 d[kR][kE / 2];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float2 s = ln_both(0.f);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        d[i][e] = cur[i].get2(e);
        s = fadd2(s, d[i][e]);
      }
      mean[i] = s.x + s.y;
    }
    ln_sum<kBlock>(mean, lanes, buf[kBlock ? 2 * turn : 0]);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      mean[i] *= p.inv_n;
      float2 s = ln_both(0.f);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        d[i][e] = fadd2(d[i][e], ln_both(-mean[i]));
        if (kV >= 2) {   // features behind N add nothing
          if (ln_col<Frag::kCols>(2 * e, lane, lanes) < p.N) s = ffma2(d[i][e], d[i][e], s);
        } else {
          if (ln_col<Frag::kCols>(2 * e, lane, lanes) < p.N) s.x = fmaf(d[i][e].x, d[i][e].x, s.x);
          if (ln_col<Frag::kCols>(2 * e + 1, lane, lanes) < p.N) s.y = fmaf(d[i][e].y, d[i][e].y, s.y);
        }
      }
      var[i] = s.x + s.y;
    }
    ln_sum<kBlock>(var, lanes, buf[kBlock ? 2 * turn + 1 : 0]);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const uint32_t row = t.row + i * t.groups;
      const float rstd = rsqrtf(fmaf(var[i], p.inv_n, p.eps));
      if (row < p.rows) {
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) d[i][e] = ffma2(fmul2(d[i][e], ln_both(rstd)), w[e], b[e]);
        ln_store<X, kC, kV>(y + ln_offset(p, p.ly, row), lane, lanes, p.N, d[i]);
        if (lane == 0) {
          if (p.mean) p.mean[row] = mean[i];
          if (p.rstd) p.rstd[row] = rstd;
        }
      }
    }
  }
}

template <typename X, int kLanes, int kC, int kR, int kV, int kMaxThreads, int kCtas>
__global__ void __launch_bounds__(kMaxThreads, kCtas) ln_bwd_kernel(const LnParams p) {
  using Walk = LnWalk<X, kLanes, kC, kR, kV, kMaxThreads, 2>;
  using Frag = typename Walk::Frag;
  constexpr bool kBlock = Walk::kBlock, kRing = Walk::kRing;
  constexpr int kE = 8 * kC, kS = Walk::kS;
  static_assert(kRing || kBlock, "only the longest rows go without the ring");
  // xh and g are kept from the sums to the result where registers allow
  constexpr bool kKeep = kC == 1 && kR <= 2 && kMaxThreads <= 320;
  __shared__ __align__(16) float buf[kBlock ? 2 : 1][2 * kR][32];
  if (kBlock) {
    for (int i = threadIdx.x; i < 4 * kR * 32; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  // one row of partial sums of every warp
  __shared__ float sums[kBlock ? 1 : kLnThreads / 32][kBlock ? 1 : (kBlock ? 1 : kLanes) * kE];
  Walk t(p);
  const int lane = t.lane, lanes = t.lanes;
  const X* x = static_cast<const X*>(p.x);
  const X* dy = static_cast<const X*>(p.dy);
  X* dx = static_cast<X*>(p.y);
  float2 w[kE / 2], dw[kE / 2], db[kE / 2];
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) dw[e] = db[e] = ln_both(0.f);
  Frag nx[kRing ? 1 : kR], ng[kRing ? 1 : kR];
  // the rows' statistics travel in the ring too, a copy for every warp (or group
  // of lanes): read from memory by all its threads, a turn ahead, they held up
  // the rows (long scoreboard stalls, 219 against 186 us without them)
  constexpr int kOwners = kBlock ? 32 : kLnThreads / (kBlock ? 1 : kLanes);
  __shared__ float2 stats[kRing ? kS : 1][kR][kOwners];
  const int owner = kBlock ? threadIdx.x >> 5 : t.group;
  const int owner_lane = kBlock ? threadIdx.x & 31 : lane;
  int st_in = 0, st_out = 0;
  float nm[kR], nr[kR];
  auto fetch = [&](uint32_t row0) {
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const uint32_t row = row0 + i * t.groups;
      if constexpr (kRing) {
        if (row < p.rows) {
          Frag::copy(t.slot(t.in, i, 0), t.pitch, x + ln_offset(p, p.lx, row), lane, lanes,
                     p.N);
          Frag::copy(t.slot(t.in, i, 1), t.pitch, dy + ln_offset(p, p.ldy, row), lane, lanes,
                     p.N);
          if (owner_lane < 2)
            ln_copy4(smem_u32(&stats[st_in][i][owner]) + 4 * owner_lane,
                     (owner_lane ? p.rstd : p.mean) + row);
        }
      } else if (row < p.rows) {
        nx[i].load(x + ln_offset(p, p.lx, row), lane, lanes, p.N);
        ng[i].load(dy + ln_offset(p, p.ldy, row), lane, lanes, p.N);
      } else {
        nx[i].clear();
        ng[i].clear();
      }
    }
    if constexpr (kRing) {
      t.next(t.in);
      st_in = st_in + 1 == kS ? 0 : st_in + 1;
      ln_commit();
    }
  };
  auto fetch_stats = [&](uint32_t row0) {   // one turn ahead
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const uint32_t row = row0 + i * t.groups;
      nm[i] = nr[i] = 0.f;
      if (row < p.rows) {
        nm[i] = __ldg(p.mean + row);
        nr[i] = __ldg(p.rstd + row);
      }
    }
  };
  if constexpr (!kRing) fetch_stats(t.row);
  if constexpr (kRing) {
#pragma unroll
    for (int k = 0; k < kS - 1; ++k) fetch(t.row + k * t.step);
  } else {
    fetch(t.row);
  }
  ln_params<kC, Frag::kCols>(p.w, p.params_bf16, lane, lanes, p.N, 1.f, w);
  for (int turn = 0; t.any(p); turn ^= 1, t.row += t.step) {
    Frag cx[kR], cg[kR];
    float m[kR], r[kR], c[2 * kR];
    if constexpr (!kRing) {
#pragma unroll
      for (int i = 0; i < kR; ++i) m[i] = -nm[i], r[i] = nr[i];
      fetch_stats(t.row + t.step);
    }
    if constexpr (kRing) {
      fetch(t.row + (kS - 1) * t.step);
      ln_wait<kRing ? kS - 1 : 0>();
      if (Frag::kOdd && kBlock) __syncthreads();
      else __syncwarp();   // the statistics came by two of the lanes
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float2 st = stats[st_out][i][owner];
        m[i] = -st.x, r[i] = st.y;
        const uint32_t row = min(t.row + i * t.groups, uint32_t(p.rows - 1));
        cx[i].read(t.slot(t.out, i, 0), t.pitch,
                   Frag::kOdd ? x + ln_offset(p, p.lx, row) : nullptr, lane, lanes, p.N);
        cg[i].read(t.slot(t.out, i, 1), t.pitch,
                   Frag::kOdd ? dy + ln_offset(p, p.ldy, row) : nullptr, lane, lanes, p.N);
        if (t.row + i * t.groups >= p.rows) {   // no row: no share
          cx[i].clear(), cg[i].clear();
          m[i] = r[i] = 0.f;
        }
      }
      t.next(t.out);
      st_out = st_out + 1 == kS ? 0 : st_out + 1;
    } else {
#pragma unroll
      for (int i = 0; i < kR; ++i) cx[i] = nx[i], cg[i] = ng[i];
      fetch(t.row + t.step);
    }
    float2 kx[kKeep ? kR : 1][kKeep ? kE / 2 : 1], kg[kKeep ? kR : 1][kKeep ? kE / 2 : 1];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float2 c1 = ln_both(0.f), c2 = ln_both(0.f);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {   // dy is 0 behind N
        const float2 xh = fmul2(fadd2(cx[i].get2(e), ln_both(m[i])), ln_both(r[i]));
        const float2 g = cg[i].get2(e), gw = fmul2(g, w[e]);
        c1 = fadd2(c1, gw);
        c2 = ffma2(gw, xh, c2);
        dw[e] = ffma2(g, xh, dw[e]);
        db[e] = fadd2(db[e], g);
        if (kKeep) kx[kKeep ? i : 0][kKeep ? e : 0] = xh, kg[kKeep ? i : 0][kKeep ? e : 0] = gw;
      }
      c[2 * i] = c1.x + c1.y;
      c[2 * i + 1] = c2.x + c2.y;
    }
    ln_sum<kBlock>(c, lanes, buf[kBlock ? turn : 0]);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const uint32_t row = t.row + i * t.groups;
      if (row < p.rows) {   // dx = r g - r c1 - xh r c2
        const float rn = -r[i] * p.inv_n;
        const float2 c1 = ln_both(c[2 * i] * rn), c2 = ln_both(c[2 * i + 1] * rn);
        float2 v[kE / 2];
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) {
          const float2 xh =
              kKeep ? kx[kKeep ? i : 0][kKeep ? e : 0]
                    : fmul2(fadd2(cx[i].get2(e), ln_both(m[i])), ln_both(r[i]));
          const float2 gw = kKeep ? kg[kKeep ? i : 0][kKeep ? e : 0] : fmul2(cg[i].get2(e), w[e]);
          v[e] = ffma2(xh, c2, ffma2(gw, ln_both(r[i]), c1));
        }
        ln_store<X, kC, kV>(dx + ln_offset(p, p.ly, row), lane, lanes, p.N, v);
      }
    }
  }
  if (p.part == nullptr) return;
  // this CTA's sums: the groups of a warp by shuffles, its warps in order
  float* part = p.part + int64_t(blockIdx.x) * 2 * p.N;
  auto value = [](const float2* v, int e) { return (e & 1) ? v[e / 2].y : v[e / 2].x; };
  if constexpr (kBlock) {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int at = ln_col<Frag::kCols>(e, lane, lanes);
      if (at < p.N) {
        part[at] = value(dw, e);
        part[p.N + at] = value(db, e);
      }
    }
  } else {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        float v = value(which ? db : dw, e);
#pragma unroll
        for (int o = 16; o >= kLanes; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) < kLanes) sums[warp][e * kLanes + lane] = v;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < kLanes * kE; i += kLnThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kLnThreads / 32; ++k) t += sums[k][i];
        const int at = ln_col<Frag::kCols>(i / kLanes, i % kLanes, kLanes);
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
