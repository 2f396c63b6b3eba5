// Kernel instances of attention, picked by type and head-dimension class (the
// accumulators' columns: 64, 128 or 256), defined in attention_fwd.hip and
// attention_bwd.hip.
#pragma once

#include <stdint.h>

namespace mfl {
namespace att {

struct FwdParams;
struct CombineParams;
struct BwdParams;

// kernel and its threads; null for a class that is not built
struct KernelRef {
  const void* fn;
  int threads;
};
KernelRef fwd_kernel(bool bf16, int dc, int algo);   // algo: MFL_ATTENTION_TALL, _TALL_4, _FLAT
KernelRef join_kernel(bool bf16, int dc);
KernelRef dq_kernel(bool bf16, int dc);
KernelRef dkv_kernel(bool bf16, int dc);
KernelRef dkv_join_kernel(bool bf16, int dc);

// columns of the accumulators for a head dimension
constexpr int dim_class(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// rows (forward, dQ) and keys (dK, dV) per workgroup
constexpr int tile_rows(int algo) { return algo == 3 ? 32 : algo == 2 ? 128 : 256; }
constexpr int dq_rows(int dc) { return dc == 256 ? 128 : 256; }
#ifndef K64
#define K64 128
#define C64 64
#endif
#ifndef K128
#define K128 256
#define C128 32
#endif
constexpr int dkv_keys(int dc) { return dc == 64 ? K64 : dc == 128 ? K128 : 128; }
constexpr int dkv_chunk(int dc) { return dc == 256 ? 32 : dc == 64 ? C64 : C128; }

}  // namespace att
}  // namespace mfl
