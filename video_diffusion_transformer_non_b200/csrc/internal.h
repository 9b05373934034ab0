// Host-side state that vidattn.cu keeps and the library's other translation
// units use.
#pragma once
#include <cuda.h>

#include <cstdint>

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

}  // namespace host
}  // namespace vidattn
