// Host side of the attention's backward pass: argument checks, the workspace's
// layout, the split of long units and the launches.  The operation is
// documented in include/vidattn.h (vidattn_bwd), the kernels in bwd_kernel.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>

#include "../../include/vidattn.h"
#include "bwd_kernel.cuh"
#include "internal.h"

namespace vidattn {
namespace {

constexpr int kBwdMaxSplit = 64;

using BwdKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap,
                           const CUtensorMap, const BwdParams);
BwdKernel bwd_variant(int D) {
  return D == 128 ? vidattn_bwd_kernel<128> : vidattn_bwd_kernel<64>;
}
int bwd_smem(int D) { return D == 128 ? BwdCfg<128>::kSmemBytes : BwdCfg<64>::kSmemBytes; }

int tiles(int S) { return (S + 127) / 128; }

// Tile pairs that the causal limit leaves (all without it), in whole tiles.
int64_t bwd_pairs(int n_q, int n_kv, bool causal, int off) {
  if (!causal) return int64_t(n_q) * n_kv;
  // query tile i sees i + first key tiles, between none and all
  const int64_t first = (int64_t(off) + 127 >= 0 ? (off + 127) / 128 : -((-int64_t(off)) / 128)) + 1;
  const int64_t lo = std::min<int64_t>(std::max<int64_t>(1 - first, 0), n_q);
  const int64_t hi = std::min<int64_t>(std::max<int64_t>(n_kv - first, lo), n_q);
  return (hi - lo) * first + (hi * (hi - 1) - lo * (lo - 1)) / 2 + (n_q - hi) * n_kv;
}

// How many ranges a unit's visited tiles are split into.  A unit of `len`
// tiles costs `cost` products each, `share` is an SM's part of all products.
// With few units the longest bounds the launch; but each range has a start, a
// drain and fp32 sums of its own and the adding kernel follows, so a split has
// to shorten the longest unit by 15 products and by 0.7 shares.  Measured (H,
// S_q x S_kv, D = 128, us): 2, 4096^2, a unit of 1.3 shares: 60 whole, 66 in 2;
// 4, 1323^2, 1.9 shares but 11 tiles: 29 and 35; 4, 2398^2 causal, 2.1 shares:
// 41 and 47; 1, 4096^2, 2.7 shares: 58 whole, 43 in 2, 48 in 3; 1, 8192^2
// causal, 2.6 shares: 104 whole, 70 in 2; 1, 2048^2, 5.3 shares: 35 whole, 30
// in 2, 25 in 4, 29 in 6.
constexpr int kBwdMinTiles = 4;
int bwd_split(int len, int cost, int64_t share, int requested) {
  if (requested > 0) return requested;
  const int64_t unit = int64_t(len) * cost;
  share = std::max<int64_t>(share, 1);
  if (10 * unit <= 16 * share) return 1;
  int64_t n = (20 * unit + 13 * share) / (26 * share);   // unit / (1.3 share), to the nearest
  n = std::min({std::max<int64_t>(n, 2), int64_t(kBwdMaxSplit),
                std::max<int64_t>(len / kBwdMinTiles, 1)});
  return unit - unit / n < 15 + 7 * share / 10 ? 1 : int(n);
}

struct BwdPlan {
  int n_q, n_kv, kv_split, q_split;
  bool kv_first;   // the kind with the longer units goes first
  size_t stats, sums, part_kv, part_q, bytes;   // offsets, and the whole size
};

BwdPlan bwd_plan(bool ids, int B, int H, int S_q, int S_kv, int D, int flags) {
  BwdPlan r{};
  const int64_t BH = int64_t(B) * H;
  r.n_q = tiles(S_q);
  r.n_kv = tiles(S_kv);
  const int requested = (flags >> 8) & 0xFF;
  const bool causal = (flags & VIDATTN_CAUSAL) != 0;
  const int64_t share = BH * bwd_pairs(r.n_q, r.n_kv, causal, S_kv - S_q) * 7 / 148;
  r.kv_split = bwd_split(r.n_q, 4, share, requested);
  r.q_split = bwd_split(r.n_kv, 3, share, requested);
  r.kv_first = int64_t(r.n_q) * 4 * r.q_split >= int64_t(r.n_kv) * 3 * r.kv_split;
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  size_t at = 0;
  r.stats = at;
  at += up(size_t(BH) * r.n_q * 256 * 4);
  r.sums = at;
  if (ids) at += up(sizeof(int4) * size_t(B) * (size_t(r.n_q) + r.n_kv));
  r.part_kv = at;
  if (r.kv_split > 1) at += up(size_t(r.kv_split) * 2 * BH * S_kv * D * 4);
  r.part_q = at;
  if (r.q_split > 1) at += up(size_t(r.q_split) * BH * S_q * D * 4);
  r.bytes = at;
  return r;
}

// Do the grids of the kernels hold a call of these sizes (checked otherwise)?
bool bwd_fits(bool ids, int B, int H, int S_q, int S_kv, int D, int flags) {
  if (S_q == 0 || S_kv == 0) return true;   // no kernel runs
  const int64_t BH = int64_t(B) * H;
  if (BH * tiles(S_q) > INT_MAX || BH * tiles(S_kv) > INT_MAX) return false;
  const BwdPlan plan = bwd_plan(ids, B, H, S_q, S_kv, D, flags);
  return BH * plan.n_kv * plan.kv_split + BH * plan.n_q * plan.q_split <= INT_MAX &&
         BH * plan.n_q + (ids ? int64_t(B) * plan.n_kv : 0) <= INT_MAX;
}

// Raises the kernels' shared-memory limit once per device (and again after
// vidattn_release).
std::mutex g_bwd_mu;
std::map<int, int> g_bwd_ready;   // device -> 1 + the epoch of its set-up
int bwd_ready(int dev) {
  const int now = host::epoch() + 1;
  std::lock_guard<std::mutex> lk(g_bwd_mu);
  int& ready = g_bwd_ready[dev];
  if (ready != now) {
    for (int D : {64, 128})
      if (cudaFuncSetAttribute(bwd_variant(D), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               bwd_smem(D)) != cudaSuccess)
        return VIDATTN_ERR_CUDA;
    ready = now;
  }
  return VIDATTN_OK;
}

template <int D>
void launch_prepare(const void* out, const void* dout, const float* lse, const float* dlse,
                    const int32_t* seg_q, const int32_t* seg_kv, float* stats, int4* q_sum,
                    int4* kv_sum, int64_t blocks, int BH, int H, int S_q, int S_kv, int n_q,
                    int n_kv, cudaStream_t stream) {
  bwd_prepare_kernel<D><<<unsigned(blocks), 256, 0, stream>>>(
      static_cast<const uint16_t*>(out), static_cast<const uint16_t*>(dout), lse, dlse, seg_q,
      seg_kv, stats, q_sum, kv_sum, BH, H, S_q, S_kv, n_q, n_kv);
}

}  // namespace
}  // namespace vidattn

using namespace vidattn;

extern "C" {

VIDATTN_API int64_t vidattn_bwd_workspace(int has_ids, int B, int H, int S_q, int S_kv, int D,
                                          int flags) {
  if (B < 1 || H < 1 || B > 65535 || H > 65535 || S_q < 0 || S_kv < 0 || (D != 64 && D != 128) ||
      (flags & ~(VIDATTN_CAUSAL | VIDATTN_SPLIT_KV(0xFF))) ||
      ((flags >> 8) & 0xFF) > kBwdMaxSplit || S_q > INT_MAX - 256 || S_kv > INT_MAX - 256 ||
      !bwd_fits(has_ids != 0, B, H, S_q, S_kv, D, flags))
    return -1;
  return int64_t(bwd_plan(has_ids != 0, B, H, S_q, S_kv, D, flags).bytes);
}

VIDATTN_API int vidattn_bwd(const void* q, const void* k, const void* v, const void* out,
                            const void* dout, const float* lse, const float* dlse,
                            const int32_t* seg_q, const int32_t* seg_kv, void* dq, void* dk,
                            void* dv, int B, int H, int S_q, int S_kv, int D, float scale,
                            int flags, void* workspace, int64_t workspace_bytes,
                            vidattn_stream_t stream_) {
  using host::aligned;
  if (flags & ~(VIDATTN_CAUSAL | VIDATTN_SPLIT_KV(0xFF))) return VIDATTN_ERR_BAD_SHAPE;
  if (((flags >> 8) & 0xFF) > kBwdMaxSplit) return VIDATTN_ERR_BAD_SHAPE;
  if (S_q > 0 && (!q || !out || !dout || !lse || !dq)) return VIDATTN_ERR_NULL;
  if (S_kv > 0 && (!k || !v || !dk || !dv)) return VIDATTN_ERR_NULL;
  if ((seg_q == nullptr) != (seg_kv == nullptr)) return VIDATTN_ERR_SEG_PAIR;
  if (D != 64 && D != 128) return VIDATTN_ERR_UNSUPPORTED_D;
  if (B < 1 || H < 1 || B > 65535 || H > 65535 || S_q < 0 || S_kv < 0 || S_q > INT_MAX - 256 ||
      S_kv > INT_MAX - 256 || !std::isfinite(scale) ||
      !bwd_fits(seg_q != nullptr, B, H, S_q, S_kv, D, flags))
    return VIDATTN_ERR_BAD_SHAPE;
  for (const void* p : {q, k, v, out, dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if (!aligned(p, 16)) return VIDATTN_ERR_MISALIGNED;
  if (!aligned(lse, 4) || !aligned(dlse, 4) || !aligned(seg_q, 4) || !aligned(seg_kv, 4) ||
      !aligned(workspace, 256))
    return VIDATTN_ERR_MISALIGNED;
  if (S_q == 0 && S_kv == 0) return VIDATTN_OK;
  const BwdPlan plan = bwd_plan(seg_q != nullptr, B, H, S_q, S_kv, D, flags);
  const int64_t BH = int64_t(B) * H;
  const int64_t kv_units = BH * plan.n_kv * plan.kv_split;
  const int64_t n_units = kv_units + BH * plan.n_q * plan.q_split;
  if (S_q > 0 && S_kv > 0) {
    if (!workspace) return VIDATTN_ERR_NULL;
    if (workspace_bytes < int64_t(plan.bytes)) return VIDATTN_ERR_SCRATCH_LIMIT;
  }
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  int dev = 0, sms = 0;
  int* err = nullptr;
  int st = host::device(&dev, &err, &sms);
  if (st != VIDATTN_OK) return st;
  if (S_q == 0 || S_kv == 0) {   // no pairs: every gradient is zero
    bool ok = true;
    if (S_q > 0) ok = cudaMemsetAsync(dq, 0, size_t(BH) * S_q * D * 2, stream) == cudaSuccess;
    if (S_kv > 0)
      ok = cudaMemsetAsync(dk, 0, size_t(BH) * S_kv * D * 2, stream) == cudaSuccess &&
           cudaMemsetAsync(dv, 0, size_t(BH) * S_kv * D * 2, stream) == cudaSuccess;
    return ok ? VIDATTN_OK : VIDATTN_ERR_CUDA;
  }
  st = bwd_ready(dev);
  if (st != VIDATTN_OK) return st;
  CUtensorMap tq, tk, tv, tdo;
  if (!host::tensor_map(q, BH, S_q, D, &tq) || !host::tensor_map(k, BH, S_kv, D, &tk) ||
      !host::tensor_map(v, BH, S_kv, D, &tv) || !host::tensor_map(dout, BH, S_q, D, &tdo))
    return VIDATTN_ERR_CUDA;

  char* ws = static_cast<char*>(workspace);
  float* stats = reinterpret_cast<float*>(ws + plan.stats);
  int4* q_sum = seg_q ? reinterpret_cast<int4*>(ws + plan.sums) : nullptr;
  int4* kv_sum = seg_q ? q_sum + size_t(B) * plan.n_q : nullptr;
  const int64_t prep = BH * plan.n_q + (seg_q ? int64_t(B) * plan.n_kv : 0);
  auto prepare = D == 128 ? launch_prepare<128> : launch_prepare<64>;
  prepare(out, dout, lse, dlse, seg_q, seg_kv, stats, q_sum, kv_sum, prep, int(BH), H, S_q, S_kv,
          plan.n_q, plan.n_kv, stream);
  if (cudaGetLastError() != cudaSuccess) return VIDATTN_ERR_CUDA;

  BwdParams p{};
  p.stats = stats;
  p.seg_q = seg_q;
  p.seg_kv = seg_kv;
  p.q_sum = q_sum;
  p.kv_sum = kv_sum;
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  p.part_kv = reinterpret_cast<float*>(ws + plan.part_kv);
  p.part_q = reinterpret_cast<float*>(ws + plan.part_q);
  p.err = err;
  p.BH = int(BH);
  p.H = H;
  p.S_q = S_q;
  p.S_kv = S_kv;
  p.n_q_tiles = plan.n_q;
  p.n_kv_tiles = plan.n_kv;
  p.n_kv_split = plan.kv_split;
  p.n_q_split = plan.q_split;
  p.n_kv_units = int(kv_units);
  p.n_q_units = int(n_units - kv_units);
  p.kv_first = plan.kv_first;
  p.causal = (flags & VIDATTN_CAUSAL) ? 1 : 0;
  p.causal_off = S_kv - S_q;
  p.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.scale = scale;
  bwd_variant(D)<<<unsigned(n_units), kBwdThreads, bwd_smem(D), stream>>>(tq, tk, tv, tdo, p);
  if (cudaGetLastError() != cudaSuccess) return VIDATTN_ERR_CUDA;
  if (plan.kv_split > 1 || plan.q_split > 1) {
    const int64_t n_kv = BH * S_kv * D, n_q = BH * S_q * D;
    const int64_t items = (plan.kv_split > 1 ? n_kv / 2 : 0) + (plan.q_split > 1 ? n_q / 4 : 0);
    bwd_combine_kernel<<<unsigned((items + 255) / 256), 256, 0, stream>>>(
        p.part_kv, plan.kv_split, n_kv, p.part_q, plan.q_split, n_q, scale, p.dk, p.dv, p.dq);
    if (cudaGetLastError() != cudaSuccess) return VIDATTN_ERR_CUDA;
  }
  return VIDATTN_OK;
}

}  // extern "C"
