// Backward pass of the masked attention (fwd_kernel.cuh) for sm_100a.
//
// With P_ij = exp(scale q_i.k_j - lse_i) on the visible pairs (0 elsewhere),
// recomputed tile by tile from q, k and the forward's lse, and
// delta_i = dout_i.out_i - dlse_i:
//
//   dV = P^T dO      dP = dO V^T      dS = P (dP - delta)
//   dQ = scale dS K  dK = scale dS^T Q
//
// Two kinds of work units run in one launch.  A KV unit owns 128 keys, walks
// the query tiles that see them and keeps dK and dV in tensor memory (four
// products a tile pair: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO,
// dK += dS^T Q); a Q unit owns 128 queries, walks their key tiles and keeps dQ
// (three products: S, dP, dQ += dS K).  Recomputing S and dP in both costs
// 7 products where 5 would do, but every gradient is summed by one CTA in a
// fixed order: no atomics, no fp32 dQ in global memory, the same bits every
// time.  P and dS go from registers straight to tensor memory, as the A
// operand of the product that consumes them, and never touch shared memory.
//
// 640 threads: warps 0-15 compute P and dS, 32 columns of a tile row a thread
// (warp w: TMEM lanes 32 (w % 4) + [0, 32), columns 32 (w / 4) + [0, 32)); warp
// 16 issues the tcgen05.mma, warp 17 the TMA loads.
//
// Measured (B200): 8 heads of 32760 x 128 in 11.25 ms, 8 x 32760^2 pairs at 977
// TFLOP/s counting five products, 1368 counting the seven it does: the tensor
// core's sustained rate under the power cap.  A tile pair takes 1.48 us in a KV
// unit and 1.09 in a Q unit there; D = 64 takes 1.0 and 0.83, bound by the
// exponentials and issue slots.  A unit's set-up, first loads, drain and stores
// add about 4 us.
#pragma once
#include <climits>
#include <cstdint>
#include <cuda.h>

#include "bounded_wait.h"
#include "ptx_train.cuh"

namespace vidattn {

constexpr int kBwdSoftmaxWarps = 16;
constexpr int kBwdMmaWarp = 16, kBwdLoadWarp = 17;
constexpr int kBwdThreads = 640;   // 2 warps more: registers are dealt to 4 warps at a time
constexpr int kBwdMaxListed = 2944;   // tiles of a unit's range whose visits are kept as bits

struct BwdParams {
  // per 128-row query tile: -lse * log2(e) and -delta (row sees nothing or is
  // past S_q: -inf and 0, so its P and dS are 0), fp32 [B*H][n_q_tiles][2][128]
  const float* stats;
  const int32_t* seg_q;     // [B,S_q] or null
  const int32_t* seg_kv;    // [B,S_kv] or null
  const int4* q_sum;        // ids: [B,n_q_tiles] {min,max,uniform,0}, or null
  const int4* kv_sum;       // [B,n_kv_tiles]
  uint16_t* dq;             // bf16 [B,H,S_q,D]
  uint16_t* dk;             // bf16 [B,H,S_kv,D]
  uint16_t* dv;
  // split units: fp32 partial sums [n_kv_split][2][B*H][S_kv][D] (dK then dV,
  // dK unscaled) and [n_q_split][B*H][S_q][D], added up by bwd_combine_kernel
  float* part_kv;
  float* part_q;
  int* err;                 // device error word
  int BH, H, S_q, S_kv;
  int n_q_tiles, n_kv_tiles;
  int n_kv_split, n_q_split;
  int n_kv_units, n_q_units;   // B*H*tiles*split of each kind
  int kv_first;
  int causal, causal_off;
  float c;                  // scale * log2(e)
  float scale;
};

template <int D>
struct BwdCfg {
  static constexpr int kSub = D / 64;
  static constexpr int kSubBytes = 128 * 128;
  static constexpr int kTileBytes = kSub * kSubBytes;
  // Two stationary tiles and two rings of moving tiles.  A tile of ring A is
  // held from its score product to its gradient product, over more than a
  // whole step, so that ring has one stage more (with 2 a load had to land
  // between two products: 3500 cycles a step instead of 2100).  At D = 128
  // the seven tiles leave 3 KB for everything else.
  static constexpr int kStagesA = D == 128 ? 3 : 4, kStagesB = D == 128 ? 2 : 3;
  static constexpr int kOffFixed = 0;
  static constexpr int kOffRingA = 2 * kTileBytes;
  static constexpr int kOffRingB = kOffRingA + kStagesA * kTileBytes;
  static constexpr int kOffStats = kOffRingB + kStagesB * kTileBytes;   // [kStagesB][2][128] fp32
  static constexpr int kStatBytes = 2 * 128 * 4;
  static constexpr int kOffBar = kOffStats + kStagesB * kStatBytes;
  // fixed_full[2] a_full[] a_empty[] b_full[] b_empty[] s_full dp_full[2]
  // done s_free p_full ds_full[2]; the last four take an arrival of each
  // softmax warp.  With two dP tiles the softmax may be done with tile n + 1
  // before the tensor core's warp has looked for tile n, so dp_full and
  // ds_full alternate too: no barrier passes two phases unseen.
  static constexpr int kNumBars = 2 + 2 * (kStagesA + kStagesB) + 8;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;   // tmem addr, abort flag
  static constexpr int kOffList = kOffMisc + 16;            // visited tiles, masked tiles: bits
  static constexpr int kSmemBytes = kOffList + 2 * kBwdMaxListed / 8;
  static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory on sm_100");
  static constexpr uint32_t kTmemCols = 512;
  // Columns of tensor memory: dV (or dQ), dK, the scores S, and one or two dP
  // tiles; over a dP tile, once it is read, go P and dS (16 columns each per 32
  // of dP).  S is free for the next tile's scores as soon as it is in
  // registers.  With two dP tiles the next dP is computed beside the softmax
  // as well; a KV unit at D = 128 has room for one.
  static __host__ __device__ constexpr int dp_tiles(bool kv) { return kv && D == 128 ? 1 : 2; }
  static constexpr uint32_t kTmemAcc0 = 0;
  static constexpr uint32_t kTmemAcc1 = D;
  static __host__ __device__ constexpr uint32_t tmem_dp(bool kv, int n) {
    return 384u - 128u * ((n + 1) % dp_tiles(kv));
  }
  static __host__ __device__ constexpr uint32_t tmem_s(bool kv) {
    return 384u - 128u * dp_tiles(kv);
  }
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0);
  static constexpr uint32_t kIdescAcc = idesc_bf16_f32(128, D, 0, 1);
};

// A product's tcgen05.mma in one block, called by all lanes of a converged
// warp: one election, the first shared-memory descriptors, and fixed steps of
// their low words (16-byte units).  An election and a descriptor built from
// its address for every instruction made the issuing warp the slowest part:
// 60 - 120 cycles an instruction where N = 64 computes in 32.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // as smem_desc_sw128
__device__ __forceinline__ uint32_t bwd_desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

// D[128 x 128] (+)= A[128 x 64] B[128 x 64]^T, both K-major blocks in shared memory.
__device__ __forceinline__ void bwd_mma_ss4(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.u32 a, %1, 2;\n\tadd.u32 b, %2, 2;\n\t"
      "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
      "add.u32 a, %1, 4;\n\tadd.u32 b, %2, 4;\n\t"
      "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
      "add.u32 a, %1, 6;\n\tadd.u32 b, %2, 6;\n\t"
      "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

// D[128 x 128] = A[128 x D] B[128 x D]^T, both K-major tiles in shared memory.
template <int D>
__device__ __forceinline__ void bwd_issue_score(uint32_t d_tmem, uint32_t sA, uint32_t sB) {
  using C = BwdCfg<D>;
#pragma unroll
  for (int k = 0; k < C::kSub; ++k)
    bwd_mma_ss4(d_tmem, bwd_desc_lo(sA, 16) + k * (C::kSubBytes >> 4),
                bwd_desc_lo(sB, 16) + k * (C::kSubBytes >> 4), C::kIdescS, k > 0 ? 1u : 0u);
}

// Acc[128 x D] (+)= A[128 x 64] B[64 x D]: A bf16 in tensor memory, 32 values
// of a row in 16 columns, the next 32 from 32 columns on; B 64 rows of a
// shared tile (steps of 16 rows: 2048 bytes).
__device__ __forceinline__ void bwd_mma_ts4(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 a, b;\n\t.reg .b64 db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\tmov.b64 db, {b, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
      "add.u32 a, %1, 32;\n\tadd.u32 b, %2, 256;\n\tmov.b64 db, {b, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
      "add.u32 a, %1, 40;\n\tadd.u32 b, %2, 384;\n\tmov.b64 db, {b, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}
// Acc[128 x D] += A[128 x 128] B[128 x D].
template <int D>
__device__ __forceinline__ void bwd_issue_acc(uint32_t d_tmem, uint32_t a_tmem, uint32_t sB,
                                              bool accumulate) {
  using C = BwdCfg<D>;
  const uint32_t b = bwd_desc_lo(sB, C::kSubBytes);
  bwd_mma_ts4(d_tmem, a_tmem, b, C::kIdescAcc, accumulate ? 1u : 0u);
  bwd_mma_ts4(d_tmem, a_tmem + 64, b + 512, C::kIdescAcc, 1u);
}

// Bounded wait of a converged warp on an mbarrier phase, with one outcome for
// all lanes: false if the CTA has aborted, a wait of the launch has timed out
// or this one does (it then sets the abort flag and the device error word).  The
// polling is out of line: the phase has often passed already, and the kernel
// waits in many places.
constexpr uint64_t kBwdWaitTimeoutNs = 2000000000ull;
constexpr int kBwdErrTimeout = 1;   // bit of the device error word, as the forward's
static __device__ __noinline__ bool bwd_wait_slow(uint32_t bar, uint32_t parity,
                                                  volatile int* abort_flag, int* err) {
  const WaitEnd end = bounded_wait<false>(
      [&] { return mbar_try_wait(bar, parity); },
      [&] { return *abort_flag != 0 || *reinterpret_cast<volatile int*>(err) != 0; },
      [] { return globaltimer_ns(); }, kBwdWaitTimeoutNs);
  if (end != WaitEnd::kPhase) *abort_flag = 1;
  if (end == WaitEnd::kTimeout) atomicOr(err, kBwdErrTimeout);
  return __all_sync(0xffffffffu, end == WaitEnd::kPhase);
}
// The wait for loads or products in flight ahead of the CTA's end (a converged
// warp): it ends at their phase or at the time limit from `since`, not with a
// wait that ran out elsewhere.
static __device__ __noinline__ void bwd_drain(uint32_t bar, uint32_t parity, int* err,
                                              uint64_t since) {
  const WaitEnd end = bounded_wait<true>([&] { return mbar_try_wait(bar, parity); },
                                         [] { return false; }, [] { return globaltimer_ns(); },
                                         kBwdWaitTimeoutNs, since);
  if (end == WaitEnd::kTimeout) atomicOr(err, kBwdErrTimeout);
  __syncwarp();
}
__device__ __forceinline__ bool bwd_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int* err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return bwd_wait_slow(bar, parity, abort_flag, err);
}

// Two or three phases at once: their first looks overlap.
__device__ __forceinline__ bool bwd_wait2(uint32_t bar0, uint32_t par0, uint32_t bar1,
                                          uint32_t par1, volatile int* abort_flag, int* err) {
  const bool a = mbar_try_wait(bar0, par0), b = mbar_try_wait(bar1, par1);
  if (__all_sync(0xffffffffu, a && b)) return true;
  return bwd_wait_slow(bar0, par0, abort_flag, err) && bwd_wait_slow(bar1, par1, abort_flag, err);
}
__device__ __forceinline__ bool bwd_wait3(uint32_t bar0, uint32_t par0, uint32_t bar1,
                                          uint32_t par1, uint32_t bar2, uint32_t par2,
                                          volatile int* abort_flag, int* err) {
  const bool a = mbar_try_wait(bar0, par0), b = mbar_try_wait(bar1, par1),
             c = mbar_try_wait(bar2, par2);
  if (__all_sync(0xffffffffu, a && b && c)) return true;
  return bwd_wait_slow(bar0, par0, abort_flag, err) &&
         bwd_wait_slow(bar1, par1, abort_flag, err) && bwd_wait_slow(bar2, par2, abort_flag, err);
}

// Untiled bulk copy into shared memory (16-byte aligned, size a multiple of 16).
__device__ __forceinline__ void bulk_load_elect(uint32_t dst, const void* src, uint32_t bytes,
                                                uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      "\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// The other-side tiles a unit walks: positions [t0, t1) of its visit sequence,
// first + each set bit in turn (with ids), or first, first + 1, ...
struct BwdWalk {
  const uint32_t* bits;   // [kBwdMaxListed / 32] visited, then as many: needs the mask
  int first, n, start;    // n tiles from position `start` (relative to first)
  __device__ __forceinline__ int next(int pos) const {   // first visited position >= pos
    if (bits == nullptr) return pos;
    int w = pos >> 5;
    uint32_t x = bits[w] & (~0u << (pos & 31));
    while (x == 0u) x = bits[++w];
    return (w << 5) + __ffs(x) - 1;
  }
  __device__ __forceinline__ bool masked(int pos) const {
    return (bits[kBwdMaxListed / 32 + (pos >> 5)] >> (pos & 31)) & 1u;
  }
};

// Is any pair of (query tile i, key tile j) hidden?  kv_side: the unit owns
// the key tile (keys past S_kv are rows of its own that are never stored).
template <bool kv_side>
__device__ __forceinline__ bool bwd_pair_masked(const BwdParams& p, int b, int i, int j) {
  bool masked = false;
  if (!kv_side) masked = j == p.n_kv_tiles - 1 && (p.S_kv & 127) != 0;
  if (p.causal) masked = masked || j * 128 + 127 > i * 128 + p.causal_off;
  if (p.q_sum) {
    const int4 a = __ldg(p.q_sum + static_cast<int64_t>(b) * p.n_q_tiles + i);
    const int4 k = __ldg(p.kv_sum + static_cast<int64_t>(b) * p.n_kv_tiles + j);
    masked = masked || !(a.z && k.z && a.x == k.x);
  }
  return masked;
}

// Which of the 32 columns [x0, x0 + 32) of a score tile row are visible, as
// bits: lo <= column < hi, and the column's id equal to the row's.  Called by
// all lanes of a warp, whose rows differ and whose columns are the same: each
// lane reads one column's id, and every id among them (a few: runs) is compared
// with all of them by one ballot.
static __device__ __noinline__ uint32_t bwd_mask32(int x0, int lo, int hi, const int32_t* ids,
                                                  int n_ids, int my_id) {
  uint32_t m = 0;
  const int a = max(lo - x0, 0), e = min(hi - x0, 32);
  if (a < e) m = (~0u >> (32 - (e - a))) << a;
  if (ids != nullptr) {
    const int col = x0 + int(threadIdx.x & 31);
    const int id = col < n_ids ? __ldg(ids + col) : 0;
    uint32_t eq = 0, left = ~0u;
    while (left != 0u) {
      const int one = __shfl_sync(0xffffffffu, id, __ffs(left) - 1);
      const uint32_t same = __ballot_sync(0xffffffffu, id == one);
      if (one == my_id) eq = same;
      left &= ~same;
    }
    m &= eq;
  }
  return m;
}

// 32 scores of a row (r) to probabilities: 2^(c s + off), off the row's
// (kPerColumn false) or read per column from shared memory.  All on the
// special-function unit: a share of them as a polynomial on the FMA pipe costs
// issue slots here (D = 128, 8192 tokens: 693 us with 4 of 16, 671 with 2, 662
// with none; D = 64: 510, 498, 488).
template <bool kPerColumn>
__device__ __forceinline__ void bwd_probs32(const uint32_t (&r)[32], float c, float off,
                                            const float* offs, float (&pr)[32]) {
  const float2 c2 = make_float2(c, c);
#pragma unroll
  for (int x = 0; x < 32; x += 4) {
    float4 o = make_float4(off, off, off, off);
    if (kPerColumn) o = *reinterpret_cast<const float4*>(offs + x);
#pragma unroll
    for (int y = 0; y < 4; y += 2) {
      const int e = x + y;
      const float2 arg = ffma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), c2,
                               y == 0 ? make_float2(o.x, o.y) : make_float2(o.z, o.w));
      pr[e] = ex2(arg.x);
      pr[e + 1] = ex2(arg.y);
    }
  }
}

// dS = P (dP - delta) of 16 columns (r: dP), packed to bf16 pairs.
template <bool kPerColumn>
__device__ __forceinline__ void bwd_dscores16(const uint32_t (&r)[16], float nd, const float* nds,
                                              const float* pr, uint32_t* pk) {
#pragma unroll
  for (int x = 0; x < 16; x += 4) {
    float4 o = make_float4(nd, nd, nd, nd);
    if (kPerColumn) o = *reinterpret_cast<const float4*>(nds + x);
#pragma unroll
    for (int y = 0; y < 4; y += 2) {
      const int e = x + y;
      const float2 t = fadd2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                             y == 0 ? make_float2(o.x, o.y) : make_float2(o.z, o.w));
      const float2 ds = fmul2(make_float2(pr[e], pr[e + 1]), t);
      pk[e >> 1] = pack_bf16x2(ds.x, ds.y);
    }
  }
}

// 32 rows (a warp's lanes) x kCols columns of an accumulator from tensor
// memory, times mul, to bf16 (out) or as they are to fp32 (part), both at row
// pitch D.  have: the accumulator was written (a tile was visited); n_rows: of
// the 32 that exist.  A lane holds a row, so that its stores would touch 32
// rows with 16 bytes each; by way of `stage` (32 rows of kCols * 4 + 16 bytes,
// this warp's own) neighbouring lanes write neighbouring bytes instead (a KV
// unit's two gradients at D = 128: 3.4 us row by row).
template <int D, int kCols>
__device__ __forceinline__ void bwd_store_rows(uint32_t taddr, bool have, int n_rows, float mul,
                                               uint16_t* out, float* part, uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const bool wide = part != nullptr;
  const uint32_t pitch = kCols * (wide ? 4 : 2) + 16;   // 16 bytes off: rows meet other banks
  const uint32_t mine = stage + lane * pitch;
#pragma unroll 1
  for (int kk = 0; kk < kCols / 32; ++kk) {
    uint32_t o[32];
    if (have) {
      tmem_ld32(taddr + 32 * kk, o);
      tmem_ld_wait();
      reg_fence(o);
    } else {
#pragma unroll
      for (int x = 0; x < 32; ++x) o[x] = 0u;
    }
    if (wide) {
#pragma unroll
      for (int x = 0; x < 8; ++x)
        st_shared_v4(mine + kk * 128 + 16 * x, o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
    } else {
#pragma unroll
      for (int x = 0; x < 16; ++x)
        o[x] = pack_bf16x2(__uint_as_float(o[2 * x]) * mul, __uint_as_float(o[2 * x + 1]) * mul);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        st_shared_v4(mine + kk * 64 + 16 * x, o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
    }
  }
  __syncwarp();
  const int per_row = kCols * (wide ? 4 : 2) / 16;   // lanes that write one row
  char* dst = wide ? reinterpret_cast<char*>(part) : reinterpret_cast<char*>(out);
  const int64_t row_bytes = D * (wide ? 4 : 2);
#pragma unroll 4
  for (int i = lane; i < 32 * per_row; i += 32) {
    const int row = i / per_row, col = i % per_row;
    const uint4 v = ld_shared_v4(stage + row * pitch + col * 16);
    if (row < n_rows) *reinterpret_cast<uint4*>(dst + row * row_bytes + col * 16) = v;
  }
}

// One unit.  kKV: it owns key tile `own`; else query tile `own`.
template <int D, bool kKV>
__device__ __forceinline__ void bwd_unit(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                         const CUtensorMap& tm_v, const CUtensorMap& tm_do,
                                         const BwdParams& p, uint32_t sbase, uint8_t* smem,
                                         int bh, int own, int split, int n_split) {
  using C = BwdCfg<D>;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = bh / p.H;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  auto fixed_full = [&](int i) { return bar(i); };
  constexpr int kA = C::kStagesA, kB = C::kStagesB, kBars = 2 + 2 * (kA + kB);
  // stage and phase of position n of a ring
  auto a_full = [&](int n) { return bar(2 + n % kA); };
  auto a_empty = [&](int n) { return bar(2 + kA + n % kA); };
  auto b_full = [&](int n) { return bar(2 + 2 * kA + n % kB); };
  auto b_empty = [&](int n) { return bar(2 + 2 * kA + kB + n % kB); };
  auto a_par = [](int n) { return uint32_t(n / kA) & 1u; };
  auto b_par = [](int n) { return uint32_t(n / kB) & 1u; };
  constexpr int kX = C::dp_tiles(kKV);
  const uint32_t s_full = bar(kBars), done = bar(kBars + 3), s_free = bar(kBars + 4),
                 p_full = bar(kBars + 5);
  auto dp_full = [&](int n) { return bar(kBars + 1 + n % kX); };
  auto ds_full = [&](int n) { return bar(kBars + 6 + n % kX); };
  auto dp_par = [](int n) { return uint32_t(n / kX) & 1u; };
  const uint32_t sFix[2] = {sbase + C::kOffFixed, sbase + C::kOffFixed + C::kTileBytes};
  auto sA = [&](int n) { return sbase + C::kOffRingA + (n % kA) * C::kTileBytes; };
  auto sB = [&](int n) { return sbase + C::kOffRingB + (n % kB) * C::kTileBytes; };

  // ---------------------------------------------- the tiles this unit visits
  // without ids: a contiguous range; with ids: the bits of those that share an
  // id range with the unit's tile (a range of more than kBwdMaxListed tiles is
  // walked whole, each tile masked)
  BwdWalk walk{nullptr, 0, 0, 0};
  int end;
  if (kKV) {
    end = p.n_q_tiles;
    if (p.causal) {   // the first query row that sees key own * 128
      const int row = own * 128 - p.causal_off;
      walk.first = row <= 0 ? 0 : min(row / 128, end);
    }
  } else {
    end = p.n_kv_tiles;
    if (p.causal) {   // one past the last key row own * 128 + 127 sees
      const int last = min(own * 128 + 127, p.S_q - 1) + p.causal_off;
      end = last < 0 ? 0 : min(end, last / 128 + 1);
    }
  }
  int total = max(end - walk.first, 0);
  const int range = total;
  if (p.q_sum != nullptr && range <= kBwdMaxListed) {
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem + C::kOffList);
    const int4* mine = (kKV ? p.kv_sum : p.q_sum) +
                       static_cast<int64_t>(b) * (kKV ? p.n_kv_tiles : p.n_q_tiles) + own;
    const int4* other = (kKV ? p.q_sum : p.kv_sum) +
                        static_cast<int64_t>(b) * (kKV ? p.n_q_tiles : p.n_kv_tiles);
    const int4 me = __ldg(mine);
    for (int t0 = 32 * warp; t0 < range; t0 += kBwdThreads) {
      const int t = walk.first + t0 + lane;
      bool act = false, masked = false;
      if (t < end) {
        const int4 o = __ldg(other + t);
        act = !(o.y < me.x || o.x > me.y);
        masked = kKV ? bwd_pair_masked<kKV>(p, b, t, own) : bwd_pair_masked<kKV>(p, b, own, t);
      }
      const uint32_t w0 = __ballot_sync(0xffffffffu, act);
      const uint32_t w1 = __ballot_sync(0xffffffffu, masked);
      if (lane == 0) {
        bits[t0 / 32] = w0;
        bits[kBwdMaxListed / 32 + t0 / 32] = w1;
      }
    }
    __syncthreads();
    walk.bits = bits;
    total = 0;
    for (int w = 0; w < (range + 31) / 32; ++w) total += __popc(bits[w]);
  }
  const int t0 = int((int64_t(total) * split) / n_split);
  walk.n = int((int64_t(total) * (split + 1)) / n_split) - t0;
  walk.start = t0;
  if (walk.bits != nullptr && walk.n > 0) {   // the position of the t0-th set bit
    int left = t0, w = 0;
    for (; left >= __popc(walk.bits[w]); ++w) left -= __popc(walk.bits[w]);
    uint32_t x = walk.bits[w];
    for (; left > 0; --left) x &= x - 1u;
    walk.start = 32 * w + __ffs(x) - 1;
  }
  const int n_tiles = walk.n;
  // without ids the masked tiles are the first ones of a KV unit, the last
  // ones of a Q unit; ids beyond the bits: all
  int edge;
  if (kKV) {
    edge = p.causal ? (own * 128 + 127 - p.causal_off + 127) / 128 : 0;
    if (p.q_sum) edge = INT_MAX;
  } else {
    edge = (p.S_kv & 127) ? p.n_kv_tiles - 1 : p.n_kv_tiles;
    if (p.causal) edge = min(edge, max((own * 128 + p.causal_off + 1) >> 7, 0));
    if (p.q_sum) edge = 0;
  }
  auto masked_at = [&](int pos, int tile) {
    if (walk.bits) return walk.masked(pos);
    return kKV ? tile < edge : tile >= edge;
  };

  // The load warp's work.  KV unit: K and V stay; ring A holds Q, ring B dO and
  // the row statistics.  Q unit: Q and dO stay; ring A holds K, ring B V.
  int n_a = 0, n_b = 0;   // loads issued
  auto load = [&](int n, int tile, int which) {
    const CUtensorMap* map = which ? (kKV ? &tm_do : &tm_v) : (kKV ? &tm_q : &tm_k);
    const bool with_stats = kKV && which == 1;
    const uint32_t full = which ? b_full(n) : a_full(n), dst = which ? sB(n) : sA(n);
    mbar_arrive_expect_tx_elect(full, C::kTileBytes + (with_stats ? C::kStatBytes : 0));
    for (int s = 0; s < C::kSub; ++s)
      tma_load_3d_elect(dst + s * C::kSubBytes, map, full, s * 64, tile * 128, bh);
    if (with_stats)
      bulk_load_elect(sbase + C::kOffStats + (n % kB) * C::kStatBytes,
                      p.stats + (static_cast<int64_t>(bh) * p.n_q_tiles + tile) * 256,
                      C::kStatBytes, full);
    if (which) n_b = n + 1;
    else n_a = n + 1;
  };
  if (warp == kBwdLoadWarp && n_tiles > 0) {   // the first tiles, ahead of the CTA's set-up
    const int tile = walk.first + walk.next(walk.start);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const CUtensorMap* map = which ? (kKV ? &tm_v : &tm_do) : (kKV ? &tm_k : &tm_q);
      mbar_arrive_expect_tx_elect(fixed_full(which), C::kTileBytes);
      for (int s = 0; s < C::kSub; ++s)
        tma_load_3d_elect(sFix[which] + s * C::kSubBytes, map, fixed_full(which), s * 64,
                          own * 128, bh);
      load(0, tile, which);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc);

  if (warp == kBwdLoadWarp) {
    // -------------------------------------------------------------- loads
    bool ok = true;
    for (int n = 1, pos = n_tiles > 0 ? walk.next(walk.start) + 1 : 0; n < n_tiles && ok; ++n, ++pos) {
      pos = walk.next(pos);
      for (int which = 0; which < 2 && ok; ++which) {
        ok = bwd_wait(which ? b_empty(n) : a_empty(n), (which ? b_par(n) : a_par(n)) ^ 1u,
                             abort_flag, p.err);
        if (ok) load(n, walk.first + pos, which);
      }
    }
    // Every load has landed before the CTA can exit: where all went well the
    // products have waited for it, but this warp may have issued its last load
    // when another gave up.
    const uint64_t since = globaltimer_ns();
    for (int k = max(0, n_a - kA); k < n_a; ++k) bwd_drain(a_full(k), a_par(k), p.err, since);
    for (int k = max(0, n_b - kB); k < n_b; ++k) bwd_drain(b_full(k), b_par(k), p.err, since);
    for (int which = 0; which < 2 && n_tiles > 0; ++which)
      bwd_drain(fixed_full(which), 0, p.err, since);
    __syncwarp();
  } else if (warp == kBwdMmaWarp) {
    // -------------------------------------------------------- tensor core
    auto wait = [&](uint32_t b_, uint32_t parity) {
      return bwd_wait(b_, parity, abort_flag, p.err);
    };
    // scores of tile n, dP of tile n (their tiles have landed)
    auto scores = [&](int n) {
      tc_fence_after();
      bwd_issue_score<D>(tmem + C::tmem_s(kKV), sFix[0], sA(n));
      mma_commit_elect(s_full);
    };
    auto dprobs = [&](int n) {
      tc_fence_after();
      bwd_issue_score<D>(tmem + C::tmem_dp(kKV, n), sFix[1], sB(n));
      mma_commit_elect(dp_full(n));
      if (!kKV) mma_commit_elect(b_empty(n));
    };
    bool ok = true;
    if (n_tiles > 0) {
      ok = wait(fixed_full(0), 0) && wait(a_full(0), 0);
      if (ok) scores(0);
      ok = ok && wait(fixed_full(1), 0) && wait(b_full(0), 0);
      if (ok) dprobs(0);
    }
    for (int n = 0; n < n_tiles && ok; ++n) {
      const bool more = n + 1 < n_tiles;
      const uint32_t tp = uint32_t(n) & 1u;
      const uint32_t tX = tmem + C::tmem_dp(kKV, n);
      if (more) {
        // the next scores once these are in registers, and, into the other dP
        // tile (whose P and dS the products of tile n - 1 have read), the next
        // dP
        ok = kX == 2 ? bwd_wait3(s_free, tp, a_full(n + 1), a_par(n + 1), b_full(n + 1),
                                 b_par(n + 1), abort_flag, p.err)
                     : bwd_wait2(s_free, tp, a_full(n + 1), a_par(n + 1), abort_flag, p.err);
        if (!ok) break;
        scores(n + 1);
        if (kX == 2) dprobs(n + 1);
      }
      if (kKV && kX == 1) {   // P is ready before dS
        ok = wait(p_full, tp);
        if (!ok) break;
        tc_fence_after();
        bwd_issue_acc<D>(tmem + C::kTmemAcc0, tX, sB(n), n > 0);
      }
      ok = more && kX == 1 ? bwd_wait2(ds_full(n), dp_par(n), b_full(n + 1), b_par(n + 1),
                                       abort_flag, p.err)
                           : wait(ds_full(n), dp_par(n));
      if (!ok) break;
      tc_fence_after();
      if (kKV && kX == 2) bwd_issue_acc<D>(tmem + C::kTmemAcc0, tX, sB(n), n > 0);
      bwd_issue_acc<D>(tmem + (kKV ? C::kTmemAcc1 : C::kTmemAcc0), tX + 16, sA(n), n > 0);
      mma_commit_elect(a_empty(n));
      if (kKV) mma_commit_elect(b_empty(n));   // the statistics were read before ds_full
      if (more && kX == 1) dprobs(n + 1);   // over P and dS
    }
    // every product issued has finished before the epilogue and the release
    // of tensor memory
    mma_commit_elect(done);
    bwd_drain(done, 0, p.err, globaltimer_ns());
  } else if (warp < kBwdSoftmaxWarps) {
    // --------------------------------------------------------- P and dS
    const int quarter = warp >> 2;   // of a tile's columns
    const int x0 = 32 * quarter;
    const int r = ((warp & 3) << 5) + lane;
    const uint32_t tLane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = tLane + C::tmem_s(kKV) + x0;
    const int row = own * 128 + r;   // this thread's key (KV) or query row
    // one arrival a warp, after all its lanes
    auto arrive = [&](uint32_t b_) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_);
    };
    auto wait = [&](uint32_t b_, uint32_t parity) {
      const bool ok = bwd_wait(b_, parity, abort_flag, p.err);
      tc_fence_after();
      return ok;
    };
    float nlse = 0.f, ndelta = 0.f;
    if (!kKV) {
      const float* st = p.stats + (static_cast<int64_t>(bh) * p.n_q_tiles + own) * 256 + r;
      nlse = __ldg(st);
      ndelta = __ldg(st + 128);
    }
    // which of the 32 columns from x0 on (queries of a KV unit, keys of a Q
    // unit) this thread's row sees
    auto visible = [&](int x0) {
      int lo = 0, hi = kKV ? p.S_q : p.S_kv;
      if (p.causal) {
        if (kKV) lo = row - p.causal_off;
        else hi = min(hi, row + p.causal_off + 1);
      }
      const int32_t* ids = nullptr;
      int my_id = 0;
      if (p.q_sum) {
        const int32_t* own_ids = kKV ? p.seg_kv : p.seg_q;
        const int n_own = kKV ? p.S_kv : p.S_q;
        ids = (kKV ? p.seg_q : p.seg_kv) + static_cast<int64_t>(b) * (kKV ? p.S_q : p.S_kv);
        if (row < n_own) my_id = __ldg(own_ids + static_cast<int64_t>(b) * n_own + row);
      }
      return bwd_mask32(x0, lo, hi, ids, kKV ? p.S_q : p.S_kv, my_id);
    };
    bool ok = true;
    int pos = walk.start - 1;
    for (int n = 0; n < n_tiles; ++n) {
      pos = walk.next(pos + 1);
      const int tile = walk.first + pos;
      const bool masked = masked_at(pos, tile);
      const uint32_t vis = masked ? visible(tile * 128 + x0) : ~0u;
      const uint32_t tX = tLane + C::tmem_dp(kKV, n) + x0;
      const float* stats =
          reinterpret_cast<const float*>(smem + C::kOffStats + (n % kB) * C::kStatBytes) + x0;
      // the statistics of this query tile, then its scores
      ok = kKV ? bwd_wait2(b_full(n), b_par(n), s_full, uint32_t(n) & 1u, abort_flag, p.err)
               : bwd_wait(s_full, uint32_t(n) & 1u, abort_flag, p.err);
      if (!ok) break;
      tc_fence_after();
      float pr[32];
      {
        uint32_t rr[32];
        tmem_ld32(tS, rr);
        tmem_ld_wait();
        reg_fence(rr);
        arrive(s_free);
        bwd_probs32<kKV>(rr, p.c, nlse, stats, pr);
      }
      if (masked) {
#pragma unroll
        for (int x = 0; x < 32; ++x) pr[x] = (vis >> x) & 1 ? pr[x] : 0.f;
      }
      ok = wait(dp_full(n), dp_par(n));
      if (!ok) break;
      // P goes over the first 16 columns of dP, dS over the other 16, each once
      // they are in registers
      uint32_t rd[16], pk[16];
      tmem_ld16(tX, rd);
      if (kKV) {
#pragma unroll
        for (int x = 0; x < 16; ++x) pk[x] = pack_bf16x2(pr[2 * x], pr[2 * x + 1]);
      }
      tmem_ld_wait();
      reg_fence16(rd);
      if (kKV) tmem_st16(tX, pk);
      bwd_dscores16<kKV>(rd, ndelta, stats + 128, pr, pk);
      tmem_ld16(tX + 16, rd);
      if (kKV && kX == 1) {
        tmem_st_wait();
        arrive(p_full);
      }
      tmem_ld_wait();
      reg_fence16(rd);
      bwd_dscores16<kKV>(rd, ndelta, stats + 144, pr + 16, pk + 8);
      tmem_st16(tX + 16, pk);
      tmem_st_wait();
      arrive(ds_full(n));
    }
    // ------------------------------------------------------------ epilogue
    ok = ok && bwd_wait_slow(done, 0, abort_flag, p.err);
    if (ok) {
      tc_fence_after();
      // every load and product is over: the rings are free to stage the stores
      const bool have = n_tiles > 0;
      const int row0 = own * 128 + 32 * (warp & 3);   // this warp's first row
      constexpr int kStage = 32 * ((kKV ? D / 2 : 32) * 4 + 16);
      static_assert(kBwdSoftmaxWarps * kStage <= (C::kStagesA + C::kStagesB) * C::kTileBytes,
                    "stages in the rings");
      const uint32_t stage = sbase + C::kOffRingA + warp * kStage;
      if (kKV) {   // a quarter of the warps each: the halves of dV's and of dK's columns
        const bool is_dk = quarter >= 2;
        const int col = (quarter & 1) * (D / 2);
        const int64_t at = (static_cast<int64_t>(bh) * p.S_kv + row0) * D + col;
        float* part = nullptr;
        if (n_split > 1)
          part = p.part_kv + (int64_t(split) * 2 + (is_dk ? 0 : 1)) * p.BH * p.S_kv * D + at;
        bwd_store_rows<D, D / 2>(tLane + (is_dk ? C::kTmemAcc1 : C::kTmemAcc0) + col, have,
                                 min(p.S_kv - row0, 32), is_dk ? p.scale : 1.f,
                                 (is_dk ? p.dk : p.dv) + at, part, stage);
      } else if (quarter < D / 32) {   // 32 of dQ's columns each
        const int col = 32 * quarter;
        const int64_t at = (static_cast<int64_t>(bh) * p.S_q + row0) * D + col;
        float* part = nullptr;
        if (n_split > 1) part = p.part_q + int64_t(split) * p.BH * p.S_q * D + at;
        bwd_store_rows<D, 32>(tLane + C::kTmemAcc0 + col, have, min(p.S_q - row0, 32), p.scale,
                              p.dq + at, part, stage);
      }
    }
  }
}

// One CTA per unit: the kind with the longer units first, each kind with the
// split fastest, then the tile, then (b, h): the units of one head run close
// together and share its tiles in L2.  With the causal limit the longest tiles
// of a head go first.
template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    vidattn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_do, const BwdParams p) {
  using C = BwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sbase = smem_u32(smem_raw);
  uint8_t* smem = smem_raw;
  // a wait of an earlier CTA timed out: the results are already invalid.  One
  // thread's look decides for all: the word may change between two.
  if (__syncthreads_or(threadIdx.x == 0 && *reinterpret_cast<volatile int*>(p.err) != 0)) return;
  if (sbase & 1023u) {   // the tiles' swizzle needs the alignment asked for above
    if (threadIdx.x == 0) atomicOr(p.err, kBwdErrTimeout);
    return;
  }

  const int warp = threadIdx.x >> 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  // the load warp sets up the barriers, so that its first loads need not wait
  // for the other warps
  if (warp == kBwdLoadWarp) {
    if ((threadIdx.x & 31) == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_do);
      for (int i = 0; i < C::kNumBars; ++i)
        mbar_init(sbase + C::kOffBar + 8 * i,
                  i >= 2 + 2 * (C::kStagesA + C::kStagesB) + 4 ? kBwdSoftmaxWarps : 1);
      *reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4) = 0;
      fence_mbar_init();
    }
    __syncwarp();
  }
  if (warp == kBwdMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }

  int u = blockIdx.x;
  const int n_first = p.kv_first ? p.n_kv_units : p.n_q_units;
  const bool kv = (u < n_first) == (p.kv_first != 0);
  if (u >= n_first) u -= n_first;
  if (kv) {
    const int split = u % p.n_kv_split;
    u /= p.n_kv_split;
    bwd_unit<D, true>(tm_q, tm_k, tm_v, tm_do, p, sbase, smem, u / p.n_kv_tiles,
                            u % p.n_kv_tiles, split, p.n_kv_split);
  } else {
    const int split = u % p.n_q_split;
    u /= p.n_q_split;
    const int t = u % p.n_q_tiles;
    bwd_unit<D, false>(tm_q, tm_k, tm_v, tm_do, p, sbase, smem, u / p.n_q_tiles,
                             p.causal ? p.n_q_tiles - 1 - t : t, split, p.n_q_split);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kBwdMmaWarp) {
    tc_fence_after();
    tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(tmem_slot), C::kTmemCols);
  }
}

// Ahead of the main kernel, one CTA per 128-row tile: -lse log2(e) and -delta
// of a query tile of one (b, h) (blocks [0, BH * n_q_tiles); -inf and 0 for a
// row that sees nothing), and, with ids,
// the tile summaries {min, max, uniform, 0} of seg_q (by the blocks of head
// 0) and seg_kv (the blocks behind).  delta = dout . out - dlse: one pass
// over dout and out, 16 bytes a lane, D / 8 lanes a row.
template <int D>
__global__ void __launch_bounds__(256)
    bwd_prepare_kernel(const uint16_t* __restrict__ out, const uint16_t* __restrict__ dout,
                       const float* __restrict__ lse, const float* __restrict__ dlse,
                       const int32_t* __restrict__ seg_q, const int32_t* __restrict__ seg_kv,
                       float* __restrict__ stats, int4* __restrict__ q_sum,
                       int4* __restrict__ kv_sum, int BH, int H, int S_q, int S_kv,
                       int n_q_tiles, int n_kv_tiles) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 256 / kLanes;
  const int tid = threadIdx.x;
  const int64_t blk = blockIdx.x;
  const int64_t n_stat = static_cast<int64_t>(BH) * n_q_tiles;
  const int32_t* ids = nullptr;
  int4* sum = nullptr;
  int first = 0, len = 0;
  if (blk < n_stat) {
    const int bh = int(blk / n_q_tiles), tile = int(blk % n_q_tiles);
    float* st = stats + blk * 256;
    const int ch = tid % kLanes;
#pragma unroll
    for (int r0 = 0; r0 < 128; r0 += kRows) {
      const int r = r0 + tid / kLanes;
      const int row = tile * 128 + r;
      float acc = 0.f;
      const int64_t at = static_cast<int64_t>(bh) * S_q + row;
      if (row < S_q) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(out + at * D) + ch);
        const uint4 g = __ldg(reinterpret_cast<const uint4*>(dout + at * D) + ch);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          acc = fmaf(__uint_as_float(aw[x] << 16), __uint_as_float(gw[x] << 16), acc);
          acc = fmaf(__uint_as_float(aw[x] & 0xffff0000u), __uint_as_float(gw[x] & 0xffff0000u),
                     acc);
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      if (ch == 0) {
        float nl = -INFINITY, nd = 0.f;
        if (row < S_q) {
          const float l = __ldg(lse + at);
          if (l != -INFINITY) {   // else dlse may be a NaN, which 0 P would keep
            nl = -l * 1.44269504088896341f;
            nd = (dlse ? __ldg(dlse + at) : 0.f) - acc;
          }
        }
        st[r] = nl;
        st[128 + r] = nd;
      }
    }
    if (seg_q == nullptr || bh % H != 0) return;
    const int b = bh / H;
    ids = seg_q + static_cast<int64_t>(b) * S_q;
    sum = q_sum + static_cast<int64_t>(b) * n_q_tiles + tile;
    first = tile * 128;
    len = S_q;
  } else {
    const int64_t u = blk - n_stat;
    const int b = int(u / n_kv_tiles), tile = int(u % n_kv_tiles);
    ids = seg_kv + static_cast<int64_t>(b) * S_kv;
    sum = kv_sum + static_cast<int64_t>(b) * n_kv_tiles + tile;
    first = tile * 128;
    len = S_kv;
  }
  if (tid >= 32) return;
  int lo = INT_MAX, hi = INT_MIN;
  for (int x = tid; x < 128; x += 32) {
    if (first + x < len) {
      const int id = __ldg(ids + first + x);
      lo = min(lo, id);
      hi = max(hi, id);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (tid == 0) *sum = make_int4(lo, hi, lo == hi ? 1 : 0, 0);
}

// out[i] = mul * sum over splits of part[s * stride + i], rounded to bf16; 4
// values a thread, in split order.
__device__ __forceinline__ void bwd_combine4(const float* part, int64_t stride, int n_split,
                                             float mul, uint16_t* out, int64_t i) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < n_split; ++s) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(part + s * stride + 4 * i));
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  reinterpret_cast<uint2*>(out)[i] =
      make_uint2(pack_bf16x2(a.x * mul, a.y * mul), pack_bf16x2(a.z * mul, a.w * mul));
}

static __global__ void __launch_bounds__(256)
    bwd_combine_kernel(const float* __restrict__ part_kv, int n_kv_split, int64_t n_kv,
                       const float* __restrict__ part_q, int n_q_split, int64_t n_q, float scale,
                       uint16_t* __restrict__ dk, uint16_t* __restrict__ dv,
                       uint16_t* __restrict__ dq) {
  int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n_kv_split > 1) {
    if (i < n_kv / 4) return bwd_combine4(part_kv, 2 * n_kv, n_kv_split, scale, dk, i);
    i -= n_kv / 4;
    if (i < n_kv / 4) return bwd_combine4(part_kv + n_kv, 2 * n_kv, n_kv_split, 1.f, dv, i);
    i -= n_kv / 4;
  }
  if (n_q_split > 1 && i < n_q / 4) bwd_combine4(part_q, n_q, n_q_split, scale, dq, i);
}

}  // namespace vidattn
