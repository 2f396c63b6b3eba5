// Kernels of the gradients of the products of groups of rows: their sums are
// tied by hand, and the build checks every access to them in the generated
// code.
#include <hip/hip_runtime.h>

#include "grouped.hpp"

namespace mfl {
namespace grp {
namespace {
template <class T, class O>
KernelRef ref(bool gathered) {
  using S = Tiles256;
  return {gathered ? (const void*)grouped_backward<T, O, S, Weights256, true>
                   : (const void*)grouped_backward<T, O, S, Weights256, false>,
          S::Full::T, S::Full::BM, S::Full::BN, S::kParts};
}
}  // namespace

KernelRef backward_kernel(bool bf16, bool f32, bool gathered) {
  if (f32) return bf16 ? ref<__bf16, float>(gathered) : ref<_Float16, float>(gathered);
  return bf16 ? ref<__bf16, __bf16>(gathered) : ref<_Float16, _Float16>(gathered);
}
}  // namespace grp
}  // namespace mfl
