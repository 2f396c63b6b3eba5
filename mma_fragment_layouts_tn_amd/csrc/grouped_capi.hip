// C ABI of the products by groups of rows (mfl_grouped.h): argument checks,
// choice of kernel, launches.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/mfl_grouped.h"
#include "grouped_launch.hpp"

namespace {

using namespace mfl::grp;

constexpr int64_t kMaxCount = (int64_t)INT_MAX - (1 << 16);
constexpr int64_t kMaxExtent = (int64_t)1 << 21;     // n, k, strides between rows
constexpr int64_t kMaxGroupStride = (int64_t)1 << 42;
constexpr int64_t kMaxGather = ((int64_t)1 << 30) - 1;   // elements a gathered operand spans

bool aligned(const void* p) { return (uintptr_t)p % 16 == 0; }
bool aligned4(const void* p) { return (uintptr_t)p % 4 == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool half_type(int32_t t) { return t == MFL_F16 || t == MFL_BF16; }

// a launch has fewer than 2^32 threads
bool fits(const KernelRef& k, int64_t blocks) { return blocks < ((int64_t)1 << 32) / k.threads; }

int launch(const KernelRef& k, int64_t blocks, void* params, void* stream, void* more = nullptr,
           void* rest = nullptr) {
  if (blocks == 0) return MFL_OK;
  if (!fits(k, blocks)) return MFL_E_TOO_LARGE;
  void* args[] = {params, more, rest};   // (a kernel takes as many as it has)
  const hipError_t e = hipLaunchKernel(k.fn, dim3((unsigned)blocks), dim3(k.threads), args, 0,
                                       (hipStream_t)stream);
  return e == hipSuccess ? MFL_OK : MFL_E_LAUNCH;
}

// a stride between rows of `width` elements
int check_stride(int64_t ld, int64_t width) {
  if (ld < 0 || ld < width) return MFL_E_LEADING_DIM;
  if (ld > kMaxExtent) return MFL_E_TOO_LARGE;
  return ld % 8 ? MFL_E_MISALIGNED : MFL_OK;
}
// between the groups' matrices of rows x width elements; an output's do not overlap
int check_group_stride(int64_t s, int64_t rows, int64_t ld, int64_t width, int64_t groups,
                       bool output) {
  if (s < 0) return MFL_E_LEADING_DIM;
  if (s > kMaxGroupStride) return MFL_E_TOO_LARGE;
  if (s % 8) return MFL_E_MISALIGNED;
  if (output && groups > 1 && rows > 0 && s < (rows - 1) * ld + width) return MFL_E_ALIAS;
  return MFL_OK;
}

int check_places(int64_t groups, int64_t places) {
  if (groups < 0 || places < 0) return MFL_E_NEGATIVE_DIM;
  if (groups == 0) return MFL_E_UNSUPPORTED;
  if (groups > kMaxGroups || places > kMaxCount) return MFL_E_TOO_LARGE;
  return MFL_OK;
}

int check_grouped(const mfl_grouped_t& a, const void* A, const void* B, const int32_t* offsets,
                  const int32_t* rows, const void* D) {
  if (a.a_rows < 0 || a.n < 0 || a.k < 0) return MFL_E_NEGATIVE_DIM;
  int rc = check_places(a.groups, a.places);
  if (rc) return rc;
  if (!half_type(a.dtype) || (a.out != a.dtype && a.out != MFL_F32) || a.algo < MFL_GROUPED_AUTO ||
      a.algo > MFL_GROUPED_TILE_256)
    return MFL_E_UNSUPPORTED;
  if (a.n == 0 || a.k == 0) return MFL_E_UNSUPPORTED;
  if (a.a_rows > kMaxCount || a.n > kMaxExtent || a.k > kMaxExtent) return MFL_E_TOO_LARGE;
  if (a.n % 8 || a.k % 8) return MFL_E_MISALIGNED;
  if (!rows && a.a_rows < a.places) return MFL_E_UNSUPPORTED;
  if (!offsets || !B || (a.places > 0 && (!A || !D))) return MFL_E_NULL_POINTER;
  if ((rc = check_stride(a.lda, a.k)) || (rc = check_stride(a.ldb, a.k)) ||
      (rc = check_stride(a.ldd, a.n)) ||
      (rc = check_group_stride(a.b_group, a.n, a.ldb, a.k, a.groups, false)))
    return rc;
  if (rows && a.a_rows * a.lda > kMaxGather) return MFL_E_TOO_LARGE;
  if (!aligned(A) || !aligned(B) || !aligned(D) || !aligned4(offsets) || !aligned4(rows))
    return MFL_E_MISALIGNED;
  return MFL_OK;
}
bool is_one_of(const void* p, std::initializer_list<const void*> others) {
  for (const void* x : others)
    if (p && p == x) return true;
  return false;
}
int check_forward(const mfl_grouped_t& a, const void* A, const void* B, const int32_t* offsets,
                  const int32_t* rows, const void* D) {
  const int rc = check_grouped(a, A, B, offsets, rows, D);
  return rc ? rc : is_one_of(D, {A, B, offsets, rows}) ? MFL_E_ALIAS : MFL_OK;
}

// `bm`-place tiles over the groups and what is behind them, at most; the
// kernels number the tiles of few groups without gaps, those of more with
// empty ones between (group_spot)
int64_t tile_slots(int64_t places, int64_t groups, int64_t bm) {
  const int64_t held = groups < kExact && places < groups + 1 ? places : groups + 1;
  return places / bm + held;
}

struct Choice {
  int algo;
  KernelRef kernel;
  int64_t slots, tiles_n;
  // workgroups; cutting the last round's tiles adds less than a round
  int64_t blocks() const { return slots * tiles_n + (kernel.parts > 1 ? kFill : 0); }
};

Choice with(KernelRef k, int algo, const mfl_grouped_t& a, int64_t n) {
  return {algo, k, tile_slots(a.places, a.groups, k.bm), ceil_div(n, k.bn)};
}

// Kernel for `places` rows of `groups` matrices of n x k.  The lengths are on
// the device, so the rule goes by their mean.  Microseconds, bf16, weights from
// memory (not the caches), half of the groups half of the mean and half three
// halves of it:
//
//   groups mean    n     k   FEW  128  256
//        2   16  4096  4096   19   49   26   FEW shares a contraction between
//        8  100   256   256   5.3  6.6  6.5  waves, as long as its small tiles do
//       32   16   256  1024   7.7   14  9.9  not read weights and rows too often
//        8   48  1024  1024   16    14   10
//       32   16  1024  1024   21    20   17
//        8   48  1024   256   8.8  7.2  6.9  256 has more loads under way, and cuts
//        8   48  1024  4096   44    59   28  what is left of a round
//       32  400  1024  1024    -    46   38
//        8   48  4096   256   24   8.4  9.5  128 has two workgroups per CU, which
//       32  200  1024   256   59    10   14  counts where a tile is a few steps,
//        8  200  4096  4096    -    86   96  and where a little over half of one
//       32  200  1024  4096    -    95  111  round of 256's tiles cannot be cut
//
// The rule gives two of these rows to the slower kernel: 8 of 48 by 1024 x 256 to
// 128, for 0.3 us, and the last to 256 (`round` is 164 there, beyond 5/8 of the
// 256; on another device 106 us, 99 by 128).
int choose_algo(int64_t places, int64_t groups, int64_t n, int64_t k, bool few) {
  const int64_t mean = ceil_div(places, groups), held = places < groups ? places : groups,
                across = ceil_div(n, 256), tiles = held * across;
  const bool narrow = tiles <= 16 && (k <= 512 || mean <= 64);
  if (few && tiles <= 64 && mean * tiles <= (narrow ? 2048 : 768)) return kFew;
  const int64_t round = (places / 256 + held / 2) * across;     // 256's tiles, about
  if (mean > 128 && round > kFill / 2 && round <= kFill * 5 / 8) return kTile128;
  return k < 512 && mean < 512 ? kTile128 : kTile256;
}

Choice choose(const mfl_grouped_t& a) {
  const bool bf16 = a.dtype == MFL_BF16, f32 = a.out == MFL_F32;
  const int64_t mean = ceil_div(a.places, a.groups);
  const int algo = a.algo ? a.algo : choose_algo(a.places, a.groups, a.n, a.k, true);
  if (algo != kFew) return with(rows_kernel(bf16, f32, algo), algo, a, a.n);
  const int rm = mean <= 10 ? 1 : mean <= 24 ? 2 : 4;
  const int64_t held = a.places < a.groups ? a.places : a.groups;
  const int rn = held * ceil_div(a.n, 32) >= 2 * kFill ? 2 : 1;
  return with(few_kernel(bf16, f32, rm, rn), algo, a, a.n);
}

// The walk over tiles: bands of this many slots.  FEW goes down each column,
// so that the tiles of one group, which read the same weights, follow each
// other.
void place(GroupedParams& p, const Choice& c) {
  p.slots = (int)c.slots;
  p.tiles_n = (int)c.tiles_n;
  p.band = c.algo == kFew ? 0 : c.algo == kTile256 ? 4 : 8;
}

// Both gradients, in one launch: the kernel, and each one's tiles.  (Tiles of
// 128 x 128 are no faster anywhere: 16 groups of 42 rows, 1024 x 512, 16 us
// either way, 8 of 1024, 4096 x 2048, 321 and 269.)
struct Backward {
  Choice da, db;
};
Backward choose_backward(const mfl_grouped_t& f, bool gathered) {
  const bool bf16 = f.dtype == MFL_BF16, f32 = f.out == MFL_F32;
  Backward r;
  const KernelRef k = backward_kernel(bf16, f32, gathered);
  r.da = with(k, kTile256, f, f.k);
  r.db = {kTile256, k, f.groups * ceil_div(f.n, k.bm), ceil_div(f.k, k.bn)};
  return r;
}

int check_backward(const mfl_grouped_grad_t& a, const void* dD, const void* A, const void* B,
                   const int32_t* offsets, const int32_t* rows, const void* dA, const void* dB) {
  const mfl_grouped_t& f = a.f;
  int rc = check_grouped(f, A, B, offsets, rows, dD);
  if (rc) return rc;
  if (f.algo != MFL_GROUPED_AUTO) return MFL_E_ALGO_CASE;
  if ((rc = check_stride(a.ldda, f.k)) || (rc = check_stride(a.lddb, f.k)) ||
      (rc = check_group_stride(a.db_group, f.n, a.lddb, f.k, f.groups, true)))
    return rc;
  if (!aligned(dA) || !aligned(dB)) return MFL_E_MISALIGNED;
  if (is_one_of(dA, {dD, A, B, offsets, rows, dB}) || is_one_of(dB, {dD, A, B, offsets, rows}))
    return MFL_E_ALIAS;
  const Backward r = choose_backward(f, rows != nullptr);
  return fits(r.da.kernel, r.da.blocks() + r.db.blocks()) ? MFL_OK : MFL_E_TOO_LARGE;
}

int check_adapters(const mfl_adapters_t& a, const void* x, const void* W, const void* A,
                   const void* B, const int32_t* offsets, const int32_t* rows, const float* scale,
                   const void* D) {
  if (a.x_rows < 0 || a.n < 0 || a.k < 0 || a.rank < 0) return MFL_E_NEGATIVE_DIM;
  int rc = check_places(a.groups, a.places);
  if (rc) return rc;
  if (!half_type(a.dtype) || (a.out != a.dtype && a.out != MFL_F32) || a.algo < MFL_GROUPED_AUTO ||
      a.algo > MFL_GROUPED_TILE_256)
    return MFL_E_UNSUPPORTED;
  if (a.n == 0 || a.k == 0 || a.rank == 0) return MFL_E_UNSUPPORTED;
  if (a.x_rows > kMaxCount || a.n > kMaxExtent || a.k > kMaxExtent || a.rank > kMaxExtent)
    return MFL_E_TOO_LARGE;
  if (a.n % 8 || a.k % 8 || a.rank % 8) return MFL_E_MISALIGNED;
  if (!rows && a.x_rows < a.places) return MFL_E_UNSUPPORTED;
  if (!offsets || !W || !A || !B || (a.places > 0 && (!x || !D))) return MFL_E_NULL_POINTER;
  if ((rc = check_stride(a.ldx, a.k)) || (rc = check_stride(a.ldw, a.k)) ||
      (rc = check_stride(a.lda, a.k)) || (rc = check_stride(a.ldb, a.rank)) ||
      (rc = check_stride(a.ldd, a.n)) ||
      (rc = check_group_stride(a.a_group, a.rank, a.lda, a.k, a.groups, false)) ||
      (rc = check_group_stride(a.b_group, a.n, a.ldb, a.rank, a.groups, false)))
    return rc;
  if (rows && a.x_rows * a.ldx > kMaxGather) return MFL_E_TOO_LARGE;
  if (!aligned(x) || !aligned(W) || !aligned(A) || !aligned(B) || !aligned(D) ||
      !aligned4(offsets) || !aligned4(rows) || !aligned4(scale))
    return MFL_E_MISALIGNED;
  return is_one_of(D, {x, W, A, B, offsets, rows, scale}) ? MFL_E_ALIAS : MFL_OK;
}

// The shared product is on tiles of places whatever their group; the down
// projection on tiles of one group.
struct AdaptersPlan {
  Choice down, all;
  bool one;                    // one launch, no workspace
  int64_t splits, part_k;      // FEW: parts of the contraction
  int64_t h_at, part_at, bytes;
  int64_t join_blocks;
};
// Whether the problem is small enough for one launch, and its tiles.  Each of
// its workgroups reads 16 rows of x, 32 or 16 of W and A's; a contraction
// longer than that allows is better shared by workgroups, and beyond some 64 MB
// in all, or a workgroup per CU where they are long, the reading takes longer
// than a second launch.  Microseconds, bf16, weights from memory:
//
//   rows  adapters  rank    n     k    32    16  two launches
//      1         1    16   64    64   3.7         5.5
//     48         8    16  256   256   4.5         9.1
//   1000         8    16  256   256   8.7        17.7
//     48         8    16 1024  1024   7.7        10.8
//     48        64    16 1024  1024    23          11    (214 MB)
//      1         1    16 4096  4096    18    14    17
//     48         8    16  256  4096          13    15
//     16         8    16 1024  4096          21    15    (512 workgroups)
//      1         1    64 4096  4096    32    27    22
bool one_launch(const mfl_adapters_t& a, Choice* c) {
  if (a.rank > 64) return false;
  const int ra = a.rank <= 16 ? 1 : a.rank <= 32 ? 2 : 4;
  for (int rn = 2; rn; --rn) {
    const KernelRef k = adapters_one_kernel(a.dtype == MFL_BF16, a.out == MFL_F32, rn, ra);
    *c = {kFew, k, tile_slots(a.places, a.groups, k.bm), ceil_div(a.n, k.bn)};
    const int64_t each = (k.bm + k.bn + 16 * ra) * a.k, tiles = c->blocks();
    if (rn == 2 ? each <= 64 * 2048 && tiles <= 1024 && tiles * each <= (32 << 20)
                : each <= 48 * 4096 && tiles <= kFill)
      return true;
  }
  return false;
}
// FEW: tiles of the shared product (*all) and of the down projection, two
// launches.
Choice few_down(const mfl_adapters_t& a, Choice* all) {
  const bool bf16 = a.dtype == MFL_BF16;
  const KernelRef k = adapters_first_kernel(bf16, a.places <= 16 ? 1 : a.places <= 32 ? 2 : 4);
  *all = {kFew, k, ceil_div(a.places, k.bm), ceil_div(a.n, k.bn)};
  const KernelRef d = down_kernel(bf16, 1, 1);
  return {kFew, d, tile_slots(a.places, a.groups, d.bm), ceil_div(a.rank, d.bn)};
}
// The kernel: FEW as long as both find room in one round, or nearly, and the
// down projection of the requests does where each has an adapter of its own.
// Microseconds, bf16, x and weights from memory; tiles of both:
//
//   rows  adapters  rank    n     k          FEW  TILE
//    192         1    16 4096  4096  192+14   46    48
//    300         4    16 1024  1024   80+23   15    19
//    500         4    32 1024  1024  128+72   20    20
//   1000         4    16  256  4096   64+67   26    46
//   2000         4    16  256  4096  128+130  40    45
//   1000         4    64  256  1024   64+268  25    23
//     64        64    64 1024  4096   16+272  52    72
//    128        64    64 4096  4096  128+292  74    69
//   1000         4    64   64  4096   16+268  51    47
//
// (The first and the fifth row go to TILE, a few workgroups beyond the rule; with
// x in the caches that is the faster one there, 45 and 39.)
int adapters_algo(const mfl_adapters_t& a) {
  Choice all;
  const int64_t down = few_down(a, &all).blocks(), tiles = all.blocks(), sum = tiles + down;
  const bool few = sum <= kFill * 3 / 4 ||
                   (a.places <= 192 && tiles <= kFill / 4 && sum <= kFill * 11 / 8);
  return few ? kFew : choose_algo(a.places, 1, a.n, a.k, false);
}
AdaptersPlan plan_adapters(const mfl_adapters_t& a) {
  const bool bf16 = a.dtype == MFL_BF16, f32 = a.out == MFL_F32;
  AdaptersPlan r{};
  if (a.algo <= kFew && one_launch(a, &r.all)) {
    r.one = true;
    return r;
  }
  const int algo = a.algo ? a.algo : adapters_algo(a);
  if (algo == kFew) {
    r.down = few_down(a, &r.all);
  } else {
    const int64_t mean = ceil_div(a.places, a.groups);
    const KernelRef k = adapters_kernel(bf16, f32, algo),
                    d = mean > 24 ? down_rows_kernel(bf16)
                                  : down_kernel(bf16, mean <= 10 ? 1 : 2, a.rank <= 16 ? 1 : 2);
    r.all = {algo, k, ceil_div(a.places, k.bm), ceil_div(a.n, k.bn)};
    r.down = {kFew, d, tile_slots(a.places, a.groups, d.bm), ceil_div(a.rank, d.bn)};
  }
  r.h_at = ceil_div(4 * a.places, 16) * 16;
  // (h takes 4 bytes each; a TILE with an fp32 D is documented to take 6)
  r.part_at = r.h_at + ceil_div(a.places * a.rank * (algo != kFew && f32 ? 6 : 4), 16) * 16;
  if (algo == kFew) {
    // one round of the chip (a workgroup per CU) with the down projection's,
    // 256 of the contraction each at least
    const int64_t tiles = r.all.blocks(), most = ceil_div(a.k, 256),
                  free = kFill - r.down.blocks();
    r.splits = tiles > 0 && free > tiles ? free / tiles : 1;
    if (r.splits > most) r.splits = most;
    r.part_k = ceil_div(ceil_div(a.k, r.splits), 32) * 32;
    r.splits = ceil_div(a.k, r.part_k);
    r.join_blocks = ceil_div(a.places * (a.n / 4), 256);
  }
  r.bytes = r.part_at + 4 * r.splits * a.places * a.n;
  return r;
}
int64_t first_blocks(const AdaptersPlan& r) {
  return r.all.algo == kFew ? r.down.blocks() + r.all.blocks() * r.splits : r.all.blocks();
}

struct SortPlan {
  int64_t chunk, blocks, bytes;
};
SortPlan plan_sort(const mfl_group_rows_t& a) {
  SortPlan r;
  // 16 waves of up to 256 choices, or 4 for many groups (sort_waves)
  const int64_t wide = a.groups <= 256 ? 1024 : 256, unit = 4 * wide;
  // One workgroup alone for two chunks too, with the waves of one: 8,192 choices
  // of 64 groups 12.0 us, as by two launches, whose calls cost 4 us more;
  // 12,288 16.5 and 12.4.
  const int64_t alone = a.groups <= 256 ? 2 * unit : unit;
  r.chunk = a.count <= alone ? ceil_div(a.count > 0 ? a.count : 1, wide) * wide
                             : unit * (a.count > 256 * unit ? ceil_div(a.count, 256 * unit) : 1);
  r.blocks = a.count ? ceil_div(a.count, r.chunk) : 1;
  r.bytes = r.blocks > 1 ? 4 * r.blocks * (a.groups + 1) : 0;
  return r;
}

int check_sort(const mfl_group_rows_t& a, const void* ids, const int32_t* rows,
               const int32_t* offsets, const int32_t* slots) {
  if (a.top < 0) return MFL_E_NEGATIVE_DIM;
  const int rc = check_places(a.groups, a.count);
  if (rc) return rc;
  if (a.ids_type != MFL_I32 && a.ids_type != MFL_I64) return MFL_E_UNSUPPORTED;
  if (a.top == 0 || a.count % a.top) return MFL_E_UNSUPPORTED;
  if (!offsets || (a.count > 0 && (!ids || !rows || !slots))) return MFL_E_NULL_POINTER;
  if ((uintptr_t)ids % (a.ids_type == MFL_I64 ? 8 : 4) || !aligned4(rows) || !aligned4(offsets) ||
      !aligned4(slots))
    return MFL_E_MISALIGNED;
  return is_one_of(rows, {ids, offsets, slots}) || is_one_of(slots, {ids, offsets}) ||
                 is_one_of(offsets, {ids})
             ? MFL_E_ALIAS
             : MFL_OK;
}

// a thread per eight columns of a token; a wave per place or choice
int64_t sum_blocks(const mfl_combine_t& a) { return ceil_div(a.tokens * (a.n / 8), 256); }
int64_t grad_blocks(const mfl_combine_t& a) {
  const int64_t choices = a.tokens * a.top;
  return ceil_div(a.x_rows > choices ? a.x_rows : choices, 4);
}

int check_combine(const mfl_combine_t& a, const void* X, const int32_t* slots,
                  const float* weights, const void* out) {
  if (a.tokens < 0 || a.top < 0 || a.n < 0 || a.x_rows < 0) return MFL_E_NEGATIVE_DIM;
  if (!half_type(a.dtype) || (a.out != a.dtype && a.out != MFL_F32)) return MFL_E_UNSUPPORTED;
  if (a.n == 0 || a.top > 64) return MFL_E_UNSUPPORTED;
  if (a.tokens > kMaxCount || a.x_rows > kMaxCount || a.tokens * a.top > kMaxCount ||
      a.n > kMaxExtent)
    return MFL_E_TOO_LARGE;
  if (a.n % 8) return MFL_E_MISALIGNED;
  if (a.tokens > 0 && (!out || (a.top > 0 && !slots))) return MFL_E_NULL_POINTER;
  if (a.tokens > 0 && a.x_rows > 0 && !X) return MFL_E_NULL_POINTER;
  int rc;
  if ((rc = check_stride(a.ldx, a.n)) || (rc = check_stride(a.ldo, a.n))) return rc;
  if (!aligned(X) || !aligned(out) || !aligned4(slots) || !aligned4(weights))
    return MFL_E_MISALIGNED;
  return fits(combine_kernel(false, false), sum_blocks(a)) ? MFL_OK : MFL_E_TOO_LARGE;
}

CombineRows combine_params(const mfl_combine_t& a, const void* X, const int32_t* slots,
                           const float* weights) {
  CombineRows p{};
  p.x = X;
  p.slots = slots;
  p.weights = weights;
  p.tokens = a.tokens;
  p.ldx = a.ldx;
  p.ldo = a.ldo;
  p.top = (int)a.top;
  p.n = (int)a.n;
  p.x_rows = (int)a.x_rows;
  return p;
}

}  // namespace

extern "C" {

int group_rows_plan(const mfl_group_rows_t* a, const void* ids, const int32_t* rows,
                    const int32_t* offsets, const int32_t* slots, int64_t* workspace_bytes) {
  if (!a) return MFL_E_NULL_POINTER;
  const int rc = check_sort(*a, ids, rows, offsets, slots);
  if (rc) return rc;
  if (workspace_bytes) *workspace_bytes = plan_sort(*a).bytes;
  return MFL_OK;
}

int group_rows(const mfl_group_rows_t* a, const void* ids, int32_t* rows, int32_t* offsets,
               int32_t* slots, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_sort(*a, ids, rows, offsets, slots);
  if (rc) return rc;
  const SortPlan plan = plan_sort(*a);
  if (plan.bytes > 0 && (!workspace || !aligned(workspace) || workspace_bytes < plan.bytes))
    return MFL_E_WORKSPACE;
  SortParams p{};
  p.ids = ids;
  p.rows = rows;
  p.offsets = offsets;
  p.slots = slots;
  p.table = (int*)workspace;
  p.count = a->count;
  p.chunk = plan.chunk;
  p.top = (int)a->top;
  p.groups = (int)a->groups;
  while (p.groups >> p.bits) ++p.bits;
  const bool i64 = a->ids_type == MFL_I64;
  if (plan.blocks > 1 && (rc = launch(count_kernel(i64, p.groups), plan.blocks, &p, stream)))
    return rc;
  return launch(place_kernel(i64, p.groups), plan.blocks, &p, stream);
}

int gemm_tn_grouped_plan(const mfl_grouped_t* a, const void* A, const void* B,
                         const int32_t* offsets, const int32_t* rows, const void* D,
                         int32_t* algo) {
  if (!a) return MFL_E_NULL_POINTER;
  const int rc = check_forward(*a, A, B, offsets, rows, D);
  if (rc) return rc;
  const Choice c = choose(*a);
  if (!fits(c.kernel, c.blocks())) return MFL_E_TOO_LARGE;
  if (algo) *algo = c.algo;
  return MFL_OK;
}

int gemm_tn_grouped(const mfl_grouped_t* a, const void* A, const void* B, const int32_t* offsets,
                    const int32_t* rows, void* D, void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  const int rc = check_forward(*a, A, B, offsets, rows, D);
  if (rc) return rc;
  const Choice c = choose(*a);
  if (!fits(c.kernel, c.blocks())) return MFL_E_TOO_LARGE;
  if (a->places == 0) return MFL_OK;
  GroupedParams p{};
  p.p = B;
  p.q = A;
  p.d = D;
  p.offsets = offsets;
  p.rows = rows;
  p.groups = (int)a->groups;
  p.places = (int)a->places;
  p.n = (int)a->n;
  p.k = (int)a->k;
  p.ldp = (int)a->ldb;
  p.ldq = (int)a->lda;
  p.ldd = (int)a->ldd;
  p.q_rows = (int)a->a_rows;
  p.p_group = a->b_group;
  place(p, c);
  return launch(c.kernel, c.blocks(), &p, stream);
}

int gemm_tn_grouped_backward_plan(const mfl_grouped_grad_t* a, const void* dD, const void* A,
                                  const void* B, const int32_t* offsets, const int32_t* rows,
                                  const void* dA, const void* dB) {
  if (!a) return MFL_E_NULL_POINTER;
  return check_backward(*a, dD, A, B, offsets, rows, dA, dB);
}

int gemm_tn_grouped_backward(const mfl_grouped_grad_t* a, const void* dD, const void* A,
                             const void* B, const int32_t* offsets, const int32_t* rows, void* dA,
                             void* dB, void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_backward(*a, dD, A, B, offsets, rows, dA, dB);
  if (rc) return rc;
  const mfl_grouped_t& f = a->f;
  const Backward r = choose_backward(f, rows != nullptr);
  GroupedParams x{};           // dA
  x.p = B;
  x.q = dD;
  x.d = dA;
  x.offsets = offsets;
  x.groups = (int)f.groups;
  x.places = (int)f.places;
  x.n = (int)f.k;
  x.k = (int)f.n;
  x.ldp = (int)f.ldb;
  x.ldq = (int)f.ldd;
  x.ldd = (int)a->ldda;
  x.p_group = f.b_group;
  place(x, r.da);
  GroupedParams y{};           // dB
  y.p = A;
  y.q = dD;
  y.d = dB;
  y.offsets = offsets;
  y.rows = rows;
  y.groups = (int)f.groups;
  y.places = (int)f.places;
  y.m = (int)f.n;
  y.n = (int)f.k;
  y.ldp = (int)f.lda;
  y.ldq = (int)f.ldd;
  y.ldd = (int)a->lddb;
  y.p_rows = (int)f.a_rows;
  y.d_group = a->db_group;
  place(y, r.db);
  int first = dA && f.places > 0 ? (int)r.da.blocks() : 0;
  return launch(r.da.kernel, first + (dB ? r.db.blocks() : 0), &x, stream, &y, &first);
}

int gemm_tn_adapters_plan(const mfl_adapters_t* a, const void* x, const void* W, const void* A,
                          const void* B, const int32_t* offsets, const int32_t* rows,
                          const float* scale, const void* D, int32_t* algo,
                          int64_t* workspace_bytes) {
  if (!a) return MFL_E_NULL_POINTER;
  const int rc = check_adapters(*a, x, W, A, B, offsets, rows, scale, D);
  if (rc) return rc;
  const AdaptersPlan r = plan_adapters(*a);
  if (!r.one && (!fits(r.down.kernel, r.down.blocks()) || !fits(r.all.kernel, first_blocks(r)) ||
                 !fits(adapters_join_kernel(false, false), r.join_blocks)))
    return MFL_E_TOO_LARGE;
  if (algo) *algo = r.all.algo;
  if (workspace_bytes) *workspace_bytes = r.bytes;
  return MFL_OK;
}

int gemm_tn_adapters(const mfl_adapters_t* a, const void* x, const void* W, const void* A,
                     const void* B, const int32_t* offsets, const int32_t* rows,
                     const float* scale, void* D, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  int64_t need = 0;
  int rc = gemm_tn_adapters_plan(a, x, W, A, B, offsets, rows, scale, D, nullptr, &need);
  if (rc) return rc;
  if (a->places == 0) return MFL_OK;
  if (need > 0 && (!workspace || !aligned(workspace) || workspace_bytes < need))
    return MFL_E_WORKSPACE;
  const AdaptersPlan r = plan_adapters(*a);
  AdapterParams p{};
  p.g.q = x;
  p.g.offsets = offsets;
  p.g.rows = rows;
  p.g.groups = (int)a->groups;
  p.g.places = (int)a->places;
  p.g.k = (int)a->k;
  p.g.ldq = (int)a->ldx;
  p.g.q_rows = (int)a->x_rows;
  p.down = p.g;
  p.down.p = A;
  p.down.n = (int)a->rank;
  p.down.ldp = (int)a->lda;
  p.down.p_group = a->a_group;
  p.g.p = W;
  p.g.d = D;
  p.g.n = (int)a->n;
  p.g.ldp = (int)a->ldw;
  p.g.ldd = (int)a->ldd;
  place(p.g, r.all);
  p.up = B;
  p.scale = scale;
  p.up_group = a->b_group;
  p.rank = (int)a->rank;
  p.ldup = (int)a->ldb;
  if (r.one) return launch(r.all.kernel, r.all.blocks(), &p, stream);
  place(p.down, r.down);
  p.owner = (int*)workspace;
  p.h = (float*)((char*)workspace + r.h_at);
  p.part = (float*)((char*)workspace + r.part_at);
  if (r.all.algo == kFew) {
    p.down_blocks = (int)r.down.blocks();
    p.splits = (int)r.splits;
    p.part_k = (int)r.part_k;
    rc = launch(r.all.kernel, first_blocks(r), &p, stream);
    return rc ? rc : launch(adapters_join_kernel(a->dtype == MFL_BF16, a->out == MFL_F32),
                            r.join_blocks, &p, stream);
  }
  rc = launch(r.down.kernel, r.down.blocks(), &p, stream);
  return rc ? rc : launch(r.all.kernel, r.all.blocks(), &p, stream);
}

int combine_rows(const mfl_combine_t* a, const void* X, const int32_t* slots,
                 const float* weights, void* out, void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  const int rc = check_combine(*a, X, slots, weights, out);
  if (rc) return rc;
  if (is_one_of(out, {X, slots, weights})) return MFL_E_ALIAS;
  CombineRows p = combine_params(*a, X, slots, weights);
  p.out = out;
  return launch(combine_kernel(a->dtype == MFL_BF16, a->out == MFL_F32),
                sum_blocks(*a), &p, stream);
}

int combine_rows_backward(const mfl_combine_t* a, int64_t lddx, const void* dout, const void* X,
                          const int32_t* slots, const int32_t* rows, const float* weights,
                          void* dX, float* dw, void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_combine(*a, X, slots, weights, dout);
  if (rc) return rc;
  if (a->out != a->dtype) return MFL_E_UNSUPPORTED;
  if (!fits(combine_grad_kernel(false), grad_blocks(*a))) return MFL_E_TOO_LARGE;
  if (a->x_rows > 0 && (!rows || !dX)) return MFL_E_NULL_POINTER;
  if (dw && !weights) return MFL_E_UNSUPPORTED;
  rc = check_stride(lddx, a->n);
  if (rc) return rc;
  if (!aligned(dX) || !aligned4(rows) || !aligned4(dw)) return MFL_E_MISALIGNED;
  if (is_one_of(dX, {X, dout, slots, rows, weights, dw}) ||
      is_one_of(dw, {X, dout, slots, rows, weights}))
    return MFL_E_ALIAS;
  CombineRows p = combine_params(*a, X, slots, weights);
  p.dout = dout;
  p.rows = rows;
  p.dx = dX;
  p.dw = dw;
  p.lddx = lddx;
  return launch(combine_grad_kernel(a->dtype == MFL_BF16), grad_blocks(*a), &p, stream);
}

}  // extern "C"
