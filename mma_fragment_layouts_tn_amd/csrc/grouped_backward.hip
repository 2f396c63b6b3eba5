// Kernels of the gradients of the products of groups of rows: their sums are
// tied by hand, and the build checks every access to them in the generated
// code.
#include <hip/hip_runtime.h>

#include "grouped.hpp"

namespace mfl {
namespace grp {
namespace {
template <class T, class O, class S, class W>
KernelRef ref(bool gathered) {
  return {gathered ? (const void*)grouped_backward<T, O, S, W, true>
                   : (const void*)grouped_backward<T, O, S, W, false>,
          S::Full::T, S::Full::BM, S::Full::BN, S::kParts};
}
template <class T, class O>
KernelRef by_tile(int algo, bool gathered) {
  return algo == kTile256 ? ref<T, O, Tiles256, Weights256>(gathered)
                          : ref<T, O, Tiles128, Tiles128>(gathered);
}
}  // namespace

KernelRef backward_kernel(bool bf16, bool f32, int algo, bool gathered) {
  if (f32)
    return bf16 ? by_tile<__bf16, float>(algo, gathered) : by_tile<_Float16, float>(algo, gathered);
  return bf16 ? by_tile<__bf16, __bf16>(algo, gathered)
              : by_tile<_Float16, _Float16>(algo, gathered);
}
}  // namespace grp
}  // namespace mfl
