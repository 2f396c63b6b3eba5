// Kernels of the adapters' down projection, and of the shared projection with
// adapters for few rows.
#include <hip/hip_runtime.h>

#include "adapters.hpp"

namespace mfl {
namespace grp {
namespace {
template <class T, int RM, int RN>
KernelRef down() {
  using F = FewTile<RM, RN>;
  return {(const void*)adapters_down<T, RM, RN>, F::T, F::BM, F::BN};
}
template <class T>
KernelRef down_by_size(int rm, int rn) {
  if (rn == 1) return rm == 4 ? down<T, 4, 1>() : rm == 2 ? down<T, 2, 1>() : down<T, 1, 1>();
  return rm == 4 ? down<T, 4, 2>() : rm == 2 ? down<T, 2, 2>() : down<T, 1, 2>();
}
template <class T, class O, int RM, int RN>
KernelRef few() {
  using F = FewTile<RM, RN>;
  return {(const void*)adapters_few<T, O, RM, RN>, F::T, F::BM, F::BN};
}
template <class T, class O>
KernelRef few_by_size(int rm, int rn) {
  if (rn == 1) return rm == 4 ? few<T, O, 4, 1>() : rm == 2 ? few<T, O, 2, 1>() : few<T, O, 1, 1>();
  return rm == 4 ? few<T, O, 4, 2>() : rm == 2 ? few<T, O, 2, 2>() : few<T, O, 1, 2>();
}
}  // namespace

KernelRef down_kernel(bool bf16, int rm, int rn) {
  return bf16 ? down_by_size<__bf16>(rm, rn) : down_by_size<_Float16>(rm, rn);
}
KernelRef adapters_few_kernel(bool bf16, bool f32, int rm, int rn) {
  if (f32) return bf16 ? few_by_size<__bf16, float>(rm, rn) : few_by_size<_Float16, float>(rm, rn);
  return bf16 ? few_by_size<__bf16, __bf16>(rm, rn) : few_by_size<_Float16, _Float16>(rm, rn);
}
}  // namespace grp
}  // namespace mfl
