// Kernels of the products of groups of rows, D and dA: their sums are tied by
// hand, and the build checks every access to them in the generated code.
#include <hip/hip_runtime.h>

#include "grouped.hpp"

namespace mfl {
namespace grp {
namespace {
template <class T, class O, class S, bool PT>
KernelRef ref() {
  return {(const void*)grouped_rows<T, O, S, PT>, S::Full::T, S::Full::BM, S::Full::BN,
          S::kParts};
}
template <class T, class O, bool PT>
KernelRef by_tile(int algo) {
  return algo == kTile256 ? ref<T, O, Tiles256, PT>() : ref<T, O, Tiles128, PT>();
}
}  // namespace

KernelRef rows_kernel(bool bf16, bool f32, int algo) {
  if (f32) return bf16 ? by_tile<__bf16, float, false>(algo) : by_tile<_Float16, float, false>(algo);
  return bf16 ? by_tile<__bf16, __bf16, false>(algo) : by_tile<_Float16, _Float16, false>(algo);
}
KernelRef input_grad_kernel(bool bf16, int algo) {
  return bf16 ? by_tile<__bf16, __bf16, true>(algo) : by_tile<_Float16, _Float16, true>(algo);
}
}  // namespace grp
}  // namespace mfl
