// Forward attention kernels: fp16 and bf16, accumulators of 64, 128 and 256
// columns.
#include <hip/hip_runtime.h>

#include "attention.hpp"
#include "attention_launch.hpp"

namespace mfl {
namespace att {
namespace {
template <class T, int DC>
KernelRef pick(int algo) {
  if (algo == 2) return {(const void*)attention_flat<T, DC>, 256};
  return {(const void*)attention_tall<T, DC>, 256};
}
template <class T>
KernelRef pick(int dc, int algo) {
  return dc == 64 ? pick<T, 64>(algo) : dc == 128 ? pick<T, 128>(algo) : pick<T, 256>(algo);
}
template <class T, int DC>
KernelRef other(int which) {
  switch (which) {
    case kPairTall: return {(const void*)attention_pair<T, DC, true>, 256};
    case kPairFlat: return {(const void*)attention_pair<T, DC, false>, 256};
    case kJoin: return {(const void*)attention_join<T, DC>, 256};
    default: return {(const void*)attention_join_tiles<T, DC>, 256};
  }
}
template <class T>
KernelRef other(int dc, int which) {
  return dc == 64 ? other<T, 64>(which) : dc == 128 ? other<T, 128>(which) : other<T, 256>(which);
}
}  // namespace

KernelRef fwd_kernel(bool bf16, int dc, int algo) {
  return bf16 ? pick<__bf16>(dc, algo) : pick<_Float16>(dc, algo);
}
KernelRef other_kernel(bool bf16, int dc, OtherKernel which) {
  return bf16 ? other<__bf16>(dc, which) : other<_Float16>(dc, which);
}
}  // namespace att
}  // namespace mfl
