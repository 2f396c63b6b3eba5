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
  if (rn == 1) return rm == 2 ? down<T, 2, 1>() : down<T, 1, 1>();
  return rm == 2 ? down<T, 2, 2>() : down<T, 1, 2>();
}
template <class T, int RM>
KernelRef first() {
  using F = FewTile<RM, 4>;
  return {(const void*)adapters_first<T, RM, 4>, F::T, F::BM, F::BN};
}
template <class T>
KernelRef first_by_size(int rm) {
  return rm == 4 ? first<T, 4>() : rm == 2 ? first<T, 2>() : first<T, 1>();
}
template <class T, class O, int RN>
KernelRef one_by_rank(int ra) {
  const void* f = ra == 4   ? (const void*)adapters_one<T, O, RN, 4>
                  : ra == 2 ? (const void*)adapters_one<T, O, RN, 2>
                            : (const void*)adapters_one<T, O, RN, 1>;
  using F = OneTile<RN>;
  return {f, F::T, F::BM, F::BN};
}
template <class T, class O>
KernelRef one(int rn, int ra) {
  return rn == 1 ? one_by_rank<T, O, 1>(ra) : one_by_rank<T, O, 2>(ra);
}
}  // namespace

KernelRef adapters_one_kernel(bool bf16, bool f32, int rn, int ra) {
  return f32 ? bf16 ? one<__bf16, float>(rn, ra) : one<_Float16, float>(rn, ra)
         : bf16 ? one<__bf16, __bf16>(rn, ra) : one<_Float16, _Float16>(rn, ra);
}
KernelRef down_kernel(bool bf16, int rm, int rn) {
  return bf16 ? down_by_size<__bf16>(rm, rn) : down_by_size<_Float16>(rm, rn);
}
KernelRef adapters_first_kernel(bool bf16, int rm) {
  return bf16 ? first_by_size<__bf16>(rm) : first_by_size<_Float16>(rm);
}
KernelRef adapters_join_kernel(bool bf16, bool f32) {
  const void* f = f32 ? bf16 ? (const void*)adapters_join<__bf16, float>
                             : (const void*)adapters_join<_Float16, float>
                  : bf16 ? (const void*)adapters_join<__bf16, __bf16>
                         : (const void*)adapters_join<_Float16, _Float16>;
  return {f, kJoinThreads};
}
}  // namespace grp
}  // namespace mfl
