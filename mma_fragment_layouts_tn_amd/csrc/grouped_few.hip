// Kernels of the products of groups of few rows, of the places of a list of
// choices, and of the sum of a token's results.
#include <hip/hip_runtime.h>

#include "grouped.hpp"
#include "rows.hpp"

namespace mfl {
namespace grp {
namespace {
template <class T, class O, int RM, int RN>
KernelRef few() {
  using F = FewTile<RM, RN>;
  return {(const void*)grouped_few<T, O, RM, RN>, F::T, F::BM, F::BN};
}
template <class T, class O>
KernelRef few_by_size(int rm, int rn) {
  if (rm == 4) return few<T, O, 4, 2>();
  if (rm == 2) return few<T, O, 2, 2>();
  return rn == 2 ? few<T, O, 1, 2>() : few<T, O, 1, 1>();
}
}  // namespace

KernelRef few_kernel(bool bf16, bool f32, int rm, int rn) {
  if (f32) return bf16 ? few_by_size<__bf16, float>(rm, rn) : few_by_size<_Float16, float>(rm, rn);
  return bf16 ? few_by_size<__bf16, __bf16>(rm, rn) : few_by_size<_Float16, _Float16>(rm, rn);
}
KernelRef count_kernel(bool i64, int groups) {
  const void* f = groups <= 256 ? i64 ? (const void*)group_count<int64_t, 256>
                                      : (const void*)group_count<int32_t, 256>
                  : i64         ? (const void*)group_count<int64_t, kMaxGroups>
                                : (const void*)group_count<int32_t, kMaxGroups>;
  return {f, 64 * sort_waves(groups)};
}
KernelRef place_kernel(bool i64, int groups) {
  const void* f = groups <= 256 ? i64 ? (const void*)group_place<int64_t, 256>
                                      : (const void*)group_place<int32_t, 256>
                  : i64         ? (const void*)group_place<int64_t, kMaxGroups>
                                : (const void*)group_place<int32_t, kMaxGroups>;
  return {f, 64 * sort_waves(groups)};
}
KernelRef combine_kernel(bool bf16, bool f32) {
  const void* f = f32 ? bf16 ? (const void*)combine_sum<__bf16, float>
                             : (const void*)combine_sum<_Float16, float>
                  : bf16 ? (const void*)combine_sum<__bf16, __bf16>
                         : (const void*)combine_sum<_Float16, _Float16>;
  return {f, kCombineThreads};
}
KernelRef combine_grad_kernel(bool bf16) {
  return {bf16 ? (const void*)combine_gradient<__bf16> : (const void*)combine_gradient<_Float16>,
          kCombineThreads};
}
}  // namespace grp
}  // namespace mfl
