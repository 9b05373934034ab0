// Host-side state that vidattn.cu keeps and the library's other translation
// units use.
#pragma once
#include <cuda.h>

#include <algorithm>
#include <cstdint>
#include <utility>

namespace vidattn {
namespace host {

// The current device, its error word (device address) and its SM count, after
// the library's first-use set-up of that device.  Returns a vidattn_status.
int device(int* dev, int** err, int* sms);

// Tensor map of bf16 [BH, S, D] at ptr: box 64 x 128 x 1, 128-byte swizzle,
// rows past S read as zeros.
bool tensor_map(const void* ptr, int64_t BH, int64_t S, int D, CUtensorMap* out);

// Number of vidattn_release calls so far: per-device set-up kept elsewhere
// (kernel attributes) is valid only while it stands.
int epoch();

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Do the rows (N neighbouring elements each) of a [B,H,S,N] array with these
// sizes and strides of its first three axes lie apart?
inline bool rows_apart(const int64_t sizes[3], const int64_t strides[3], int64_t N) {
  std::pair<int64_t, int64_t> d[3];
  for (int i = 0; i < 3; ++i) d[i] = {strides[i], sizes[i]};
  std::sort(d, d + 3);
  int64_t end = N;   // one past the last element of what is laid out so far
  for (const auto& x : d) {
    if (x.second <= 1) continue;
    if (x.first < end) return false;
    end += x.first * (x.second - 1);
  }
  return true;
}

// An output over its own input: only with the input's strides (of the axes that
// have any extent), else some rows are written before they are read.
inline bool over_another_layout(const void* in, const void* out, const int64_t sizes[3],
                                const int64_t in_strides[3], const int64_t out_strides[3]) {
  if (in != out) return false;
  for (int i = 0; i < 3; ++i)
    if (sizes[i] > 1 && in_strides[i] != out_strides[i]) return true;
  return false;
}

}  // namespace host
}  // namespace vidattn
