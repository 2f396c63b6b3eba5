// Kernel arguments and instances of the products by groups of rows.
#pragma once

#include <stdint.h>

namespace mfl {
namespace grp {

// D(m, n) = sum_c Q(m, c) P(n, c), see grouped.hpp.  Strides in elements.
struct GroupedParams {
  const void* p;
  const void* q;
  void* d;
  const int* offsets;          // groups + 1 places
  const int* rows;             // row of each place, or null
  int groups, places;
  int m, n, k;                 // extents; m or k is the group's places
  int ldp, ldq, ldd;
  int p_rows, q_rows;          // rows that a gathered operand has
  int slots, tiles_n, band;    // tiles along m (of all groups, at most), along n; order (0: down
                               // each column)
  int64_t p_group, d_group;
};

// Adapters beside a shared projection (adapters.hpp): g is the shared product
// (p = W), down the down projection (p = A, n = rank); q = x, offsets and rows
// in both.
struct AdapterParams {
  GroupedParams g, down;
  const void* up;              // B
  const float* scale;          // of each group, or null: 1
  int* owner;                  // workspace: the group of each place that has one,
  float* h;                    // scale h, places x rank,
  float* part;                 // sums over parts of the contraction, splits x places x n
  int64_t up_group;
  int rank, ldup;
  int down_blocks, splits, part_k;
};

struct SortParams {
  const void* ids;
  int* rows;
  int* offsets;
  int* slots;
  int* table;                  // choices of each group in each chunk
  int64_t count, chunk;
  int top, groups, bits;       // bits: of the numbers 0 .. groups
};

struct CombineRows {
  const void* x;
  const void* dout;
  const int* slots;
  const int* rows;
  const float* weights;
  void* out;
  void* dx;
  float* dw;
  int64_t tokens, ldx, ldo, lddx;
  int top, n, x_rows;
};

constexpr int kMaxGroups = 4096;
constexpr int kExact = 256;    // groups whose tiles are numbered without gaps, fewer than
constexpr int kFill = 256;     // workgroups that occupy every CU

struct KernelRef {
  const void* fn;
  int threads, bm = 0, bn = 0;
  int parts = 1;               // that a tile may be cut into
};

// kernels by type and size of tile, each in a source of its own
enum Algo { kAuto, kFew, kTile128, kTile256 };
KernelRef rows_kernel(bool bf16, bool f32, int algo);                   // D
KernelRef few_kernel(bool bf16, bool f32, int row_blocks, int column_blocks);
KernelRef backward_kernel(bool bf16, bool f32, bool gathered);   // dA and dB
KernelRef down_kernel(bool bf16, int row_blocks, int column_blocks);
KernelRef down_rows_kernel(bool bf16);
KernelRef adapters_one_kernel(bool bf16, bool f32, int column_blocks, int rank_blocks);
KernelRef adapters_first_kernel(bool bf16, int row_blocks);
KernelRef adapters_join_kernel(bool bf16, bool f32);
KernelRef adapters_kernel(bool bf16, bool f32, int algo);
KernelRef count_kernel(bool i64, int groups);
KernelRef place_kernel(bool i64, int groups);
KernelRef combine_kernel(bool bf16, bool f32);
KernelRef combine_grad_kernel(bool bf16);

}  // namespace grp
}  // namespace mfl
