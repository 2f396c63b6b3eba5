// Attention gradient kernels: fp16 and bf16, accumulators of 64, 128 and 256
// columns.
#include <hip/hip_runtime.h>

#include "attention_bwd.hpp"
#include "attention_launch.hpp"

namespace mfl {
namespace att {
namespace {
static_assert(dq_rows(64) == 32 * dq_waves<64>() && dq_rows(128) == 32 * dq_waves<128>() &&
                  dq_rows(256) == 32 * dq_waves<256>(),
              "rows per workgroup");
template <class T>
KernelRef dq(int dc) {
  return dc == 64    ? KernelRef{(const void*)attention_dq<T, 64>, 64 * dq_waves<64>()}
         : dc == 128 ? KernelRef{(const void*)attention_dq<T, 128>, 64 * dq_waves<128>()}
                     : KernelRef{(const void*)attention_dq<T, 256>, 64 * dq_waves<256>()};
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
