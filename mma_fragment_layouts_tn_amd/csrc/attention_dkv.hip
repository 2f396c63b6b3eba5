// Kernels of the gradients of keys and values: fp16 and bf16, accumulators of
// 64, 128 and 256 columns.  A source of its own: their sums are tied by hand,
// and the build checks every access to them in the generated code.
#include <hip/hip_runtime.h>

#include "attention_bwd.hpp"
#include "attention_launch.hpp"

namespace mfl {
namespace att {
namespace {
template <class T, int DC, int KW, int RW, int KB>
KernelRef dkv_ref() {
  static_assert(dkv_keys(DC) == 32 * KW * KB && dkv_chunk(DC) == 32 * RW, "tile");
  return {(const void*)attention_dkv<T, DC, KW, RW, KB>, 64 * KW * RW};
}
template <class T>
KernelRef dkv(int dc) {
  return dc == 64    ? dkv_ref<T, 64, 2, 2, 2>()
         : dc == 128 ? dkv_ref<T, 128, 4, 1, 2>()
                     : dkv_ref<T, 256, 4, 1, 1>();
}
}  // namespace

KernelRef dkv_kernel(bool bf16, int dc) { return bf16 ? dkv<__bf16>(dc) : dkv<_Float16>(dc); }
}  // namespace att
}  // namespace mfl
