// Kernels of the products of groups of rows: their sums are tied by hand, and the
// build checks every access to them in the generated code.
#include <hip/hip_runtime.h>

#include "grouped.hpp"

namespace mfl {
namespace grp {
namespace {
template <class T, class O, class S>
KernelRef ref() {
  return {(const void*)grouped_rows<T, O, S>, S::Full::T, S::Full::BM, S::Full::BN,
          S::kParts};
}
template <class T, class O>
KernelRef by_tile(int algo) {
  return algo == kTile256 ? ref<T, O, Tiles256>() : ref<T, O, Tiles128>();
}
}  // namespace

KernelRef rows_kernel(bool bf16, bool f32, int algo) {
  if (f32) return bf16 ? by_tile<__bf16, float>(algo) : by_tile<_Float16, float>(algo);
  return bf16 ? by_tile<__bf16, __bf16>(algo) : by_tile<_Float16, _Float16>(algo);
}
}  // namespace grp
}  // namespace mfl
