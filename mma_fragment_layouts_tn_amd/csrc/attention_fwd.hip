// Forward attention kernels: fp16 and bf16, accumulators of 64, 128 and 256
// columns.  256 columns take 4 waves (a wave's accumulators and rows of Q
// fill half of the registers of a SIMD).
#include <hip/hip_runtime.h>

#include "attention.hpp"
#include "attention_launch.hpp"

namespace mfl {
namespace att {
namespace {
template <class T, int DC>
KernelRef pick(int algo) {
  switch (algo) {
    case 1:
      if constexpr (DC <= 128) return {(const void*)attention_tall<T, DC, 8>, 512};
      return {nullptr, 0};
    case 2: return {(const void*)attention_tall<T, DC, 4>, 256};
    case 3: return {(const void*)attention_flat<T, DC>, 64 * flat_waves<DC>()};
    default: return {nullptr, 0};
  }
}
template <class T>
KernelRef pick(int dc, int algo) {
  return dc == 64 ? pick<T, 64>(algo) : dc == 128 ? pick<T, 128>(algo) : pick<T, 256>(algo);
}
template <class T>
KernelRef join(int dc) {
  return {dc == 64    ? (const void*)attention_join<T, 64>
          : dc == 128 ? (const void*)attention_join<T, 128>
                      : (const void*)attention_join<T, 256>,
          256};
}
}  // namespace

KernelRef fwd_kernel(bool bf16, int dc, int algo) {
  return bf16 ? pick<__bf16>(dc, algo) : pick<_Float16>(dc, algo);
}
KernelRef join_kernel(bool bf16, int dc) { return bf16 ? join<__bf16>(dc) : join<_Float16>(dc); }
}  // namespace att
}  // namespace mfl
