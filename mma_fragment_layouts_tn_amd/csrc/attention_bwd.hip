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
static_assert(dkv_keys(64) == 32 * dkv_waves<64>() && dkv_keys(128) == 32 * dkv_waves<128>() &&
                  dkv_keys(256) == 32 * dkv_waves<256>(),
              "keys per workgroup");
template <class T>
KernelRef dq(int dc) {
  return dc == 64    ? KernelRef{(const void*)attention_dq<T, 64>, 64 * dq_waves<64>()}
         : dc == 128 ? KernelRef{(const void*)attention_dq<T, 128>, 64 * dq_waves<128>()}
                     : KernelRef{(const void*)attention_dq<T, 256>, 64 * dq_waves<256>()};
}
template <class T>
KernelRef dkv(int dc) {
  return dc == 64    ? KernelRef{(const void*)attention_dkv<T, 64>, 64 * dkv_waves<64>()}
         : dc == 128 ? KernelRef{(const void*)attention_dkv<T, 128>, 64 * dkv_waves<128>()}
                     : KernelRef{(const void*)attention_dkv<T, 256>, 64 * dkv_waves<256>()};
}
}  // namespace

KernelRef dq_kernel(bool bf16, int dc) { return bf16 ? dq<__bf16>(dc) : dq<_Float16>(dc); }
KernelRef dkv_kernel(bool bf16, int dc) { return bf16 ? dkv<__bf16>(dc) : dkv<_Float16>(dc); }
}  // namespace att
}  // namespace mfl
