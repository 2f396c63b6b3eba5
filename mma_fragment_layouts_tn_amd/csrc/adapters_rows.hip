// Kernels of the shared projection with adapters on tiles through LDS: their
// sums are tied by hand, and the build checks every access to them in the
// generated code.
#include <hip/hip_runtime.h>

#include "adapters.hpp"

namespace mfl {
namespace grp {
namespace {
template <class T, class O, class S>
KernelRef ref() {
  return {(const void*)adapters_rows<T, O, S>, S::Full::T, S::Full::BM, S::Full::BN, S::kParts};
}
template <class T, class O>
KernelRef by_tile(int algo) {
  return algo == kTile256 ? ref<T, O, Tiles256>() : ref<T, O, Tiles128>();
}
}  // namespace

KernelRef down_rows_kernel(bool bf16) {
  using C = DownTile;
  return {bf16 ? (const void*)adapters_down_rows<__bf16>
               : (const void*)adapters_down_rows<_Float16>,
          kDownParts * C::T, C::BM, C::BN};
}
KernelRef adapters_kernel(bool bf16, bool f32, int algo) {
  if (f32) return bf16 ? by_tile<__bf16, float>(algo) : by_tile<_Float16, float>(algo);
  return bf16 ? by_tile<__bf16, __bf16>(algo) : by_tile<_Float16, _Float16>(algo);
}
}  // namespace grp
}  // namespace mfl
