// Attention gradient kernels: fp16 and bf16, accumulators of 64, 128 and 256
// columns.
#include <hip/hip_runtime.h>

#include "attention_bwd.hpp"
#include "attention_launch.hpp"

namespace mfl {
namespace att {
namespace {
template <class T>
KernelRef dq(int dc) {
  return {dc == 64    ? (const void*)attention_dq<T, 64>
          : dc == 128 ? (const void*)attention_dq<T, 128>
                      : (const void*)attention_dq<T, 256>,
          256};
}
template <class T>
KernelRef join(int dc) {
  return {dc == 64    ? (const void*)attention_dkv_join<T, 64>
          : dc == 128 ? (const void*)attention_dkv_join<T, 128>
                      : (const void*)attention_dkv_join<T, 256>,
          256};
}
}  // namespace

KernelRef dq_kernel(bool bf16, int dc) { return bf16 ? dq<__bf16>(dc) : dq<_Float16>(dc); }
KernelRef dkv_join_kernel(bool bf16, int dc) {
  return bf16 ? join<__bf16>(dc) : join<_Float16>(dc);
}
}  // namespace att
}  // namespace mfl
