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

// kernel and its threads
struct KernelRef {
  const void* fn;
  int threads;
};
KernelRef fwd_kernel(bool bf16, int dc, int algo);   // algo: MFL_ATTENTION_TALL, _FLAT
// two problems in one launch; joins of all rows, of the tiles split
enum OtherKernel { kPairTall, kPairFlat, kJoin, kJoinTiles };
KernelRef other_kernel(bool bf16, int dc, OtherKernel which);
KernelRef dq_kernel(bool bf16, int dc);
KernelRef dkv_kernel(bool bf16, int dc);
KernelRef dkv_join_kernel(bool bf16, int dc);

// columns of the accumulators for a head dimension
constexpr int dim_class(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// rows (forward, dQ) and keys (dK, dV) per workgroup
constexpr int tile_rows(int algo) { return algo == 2 ? 16 : 128; }
constexpr int kDqRows = 128;
constexpr int dkv_keys(int dc) { return dc == 128 ? 256 : 128; }
// rows that a workgroup of dK and dV takes at a time
constexpr int dkv_chunk(int dc) { return dc == 64 ? 64 : 32; }
// units of its steps (attention_dkv): beside a tile's steps, least of a share
constexpr int kDkvFixed = 8, kDkvLeast = 6;

}  // namespace att
}  // namespace mfl
