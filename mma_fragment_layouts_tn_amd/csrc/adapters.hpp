// Low-rank adapters of many requests beside a shared projection:
//
//   D(r, n) = sum_k x(r, k) W(n, k) + s_g sum_j h(r, j) B(g, n, j)
//   h(r, j) = sum_k x(r, k) A(g, j, k)             r = rows[place], place in group g
//
// Small problems take one launch (adapters_one), others two.  The first forms
// s_g h for every place (few columns: the kernel for few rows, by group).  The
// second is the shared product on tiles of places whatever their group, so
// that W is read for all of them together, and adds the low-rank terms of the
// tile's groups to its sums before they are rounded.  A group's term reaches
// the rows of its own places alone, so infinities in one adapter stay with its
// requests.
//
// s_g h is held in fp32.  Where it is a matrix operand (many rows) it is taken
// apart there, into three numbers of the operands' type that add up to it.
#pragma once

#include "grouped.hpp"

namespace mfl {
namespace grp {

// two 16-bit values with an exponent of all ones in either
template <class T>
__device__ __forceinline__ bool not_finite(unsigned u) {
  constexpr unsigned e = std::is_same<T, __bf16>::value ? 0x7f80u : 0x7c00u;
  return (u & e) == e || (u >> 16 & e) == e;
}
__device__ __forceinline__ bool not_finite(float x) { return !(__builtin_fabsf(x) < INFINITY); }

// An fp32 number as a sum of kPieces numbers of T, cut off, not rounded: 24
// bits are three times bf16's 8, or twice fp16's 11 and two more.  bf16 has fp32's
// range.  fp16's ends at 65504 and, downwards, in steps of 2^-24: numbers that
// are taken apart together are scaled by a power of two (scale_of) that brings
// the largest of them between 2^14 and 2^15, and those far below it are off by
// 2^-38 of it at the most.  take(): the next number of each of eight.
constexpr int kPieces = 3;
template <class T>
struct Pieces;
template <>
struct Pieces<__bf16> {
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ Vec8<__bf16> take(float (&left)[8]) {
    u32x4_t x;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const unsigned a = __float_as_uint(left[2 * q]), b = __float_as_uint(left[2 * q + 1]);
      x[q] = __builtin_amdgcn_perm(b, a, 0x07060302);
      left[2 * q] -= __uint_as_float(a & 0xffff0000u);
      left[2 * q + 1] -= __uint_as_float(b & 0xffff0000u);
    }
    return __builtin_bit_cast(Vec8<__bf16>, x);
  }
};
template <>
struct Pieces<_Float16> {
  static constexpr bool kScaled = true;
  // Exponent of the factor's inverse, from the largest magnitude of each of a
  // row's lanes, l, l ^ 16, l ^ 32 and l ^ 48.
  static __device__ __forceinline__ int scale_of(float top) {
    const att::Halves q = att::quarters(top);
    top = att::both_max(fmaxf(q.lower, q.upper));
    return (int)(__float_as_uint(top) >> 23) - 126 - 15;
  }
  static __device__ __forceinline__ Vec8<_Float16> take(float (&left)[8]) {
    Vec8<_Float16> x;
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
      const auto y = __builtin_amdgcn_cvt_pkrtz(left[q], left[q + 1]);
      x[q] = (_Float16)y[0];
      x[q + 1] = (_Float16)y[1];
      left[q] = __builtin_fmaf((float)x[q], -1.0f, left[q]);
      left[q + 1] = __builtin_fmaf((float)x[q + 1], -1.0f, left[q + 1]);
    }
    return x;
  }
};

// Mma's instruction with the sums in ordinary registers: the compiler keeps the
// results of its own all in the one kind or all in the other.  settle() is what
// follows the last.
template <class T>
__device__ __forceinline__ void mma_low(const Vec8<T>& p, const Vec8<T>& q, floatx4& c) {
  if constexpr (std::is_same<T, __bf16>::value)
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(p), "v"(q));
  else
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(p), "v"(q));
}

// Four values of s_g h of a place, columns n .. n + 3, and the place's group.
__device__ __forceinline__ void keep(const AdapterParams& p, int place, int group, int n,
                                     floatx4 h) {
  h *= p.scale ? p.scale[group] : 1.0f;
  if (n == 0) p.owner[place] = group;
  *(floatx4*)(p.h + (int64_t)place * p.rank + n) = h;
}

// h of a tile of one group's places, few rows
template <class T, int RM, int RN>
__device__ __forceinline__ void down_few(const AdapterParams& p, floatx4* sums, int id) {
  using F = FewTile<RM, RN>;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const GroupSpot spot = group_spot<1>(p.down, id, F::BM);
  if (spot.spot.parts == 0 || spot.at.group == p.down.groups) return;
  const Place at = spot.at;
  const int n0 = spot.spot.tn * F::BN;
  few_tile<T, RM, RN>(p.down, at, n0, (const T*)p.down.p + at.group * p.down.p_group, 0, p.down.k,
                      sums, w, lane);
  // (a thread reads what it added itself)
  for (int x = tid; x < RM * RN * 64; x += F::T) {
    const int l = x & 63, j = (x >> 6) % RN, i = (x >> 6) / RN;
    const int m = 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m < at.count && n < p.rank) keep(p, at.first + m, at.group, n, sums[x]);
  }
}
template <class T, int RM, int RN>
__global__ void __launch_bounds__(64 * kFewWaves, 1) adapters_down(const AdapterParams p) {
  __shared__ floatx4 sums[kFewWaves * RM * RN * 64];
  down_few<T, RM, RN>(p, sums, blockIdx.x);
}

// the group of a place that has one, else -1
__device__ __forceinline__ int owner_of(const AdapterParams& p, int place) {
  const int g = place < p.g.offsets[p.g.groups] ? p.owner[place] : -1;
  return (unsigned)g < (unsigned)p.g.groups ? g : -1;
}
// Lanes whose number differs from the lane's before them; the first is one.
// (The exchange ahead of the condition: behind `lane == 0 ||` lane 0 would be
// off, and what lane 1 reads from it undefined.)
__device__ __forceinline__ unsigned long long run_starts(int own, int lane) {
  const int before = __shfl_up(own, 1);
  return __ballot(lane == 0 || own != before);
}
// row of x and D at a place, -1 where it is outside
__device__ __forceinline__ int row_at(const GroupedParams& p, int place) {
  const int r = p.rows ? p.rows[place] : place;
  return (unsigned)r < (unsigned)p.q_rows ? r : -1;
}

// Few rows, first launch: the workgroups of the down projection, and those of
// the shared product, which depend on nothing of theirs.  A tile's contraction
// is shared out to `splits` workgroups, so that W is read by all CUs in wide
// tiles (with a quarter of the columns per workgroup instead x is read four
// times as often, and bounds the launch: 48 rows by 4096 x 4096 20 us, so 14.7).
template <class T, int RM, int RN>
__global__ void __launch_bounds__(64 * kFewWaves, 1) adapters_first(const AdapterParams p) {
  using F = FewTile<RM, RN>;
  __shared__ floatx4 sums[kFewWaves * RM * RN * 64];
  if ((int)blockIdx.x < p.down_blocks) return down_few<T, 1, 1>(p, sums, blockIdx.x);
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int id = blockIdx.x - p.down_blocks, split = id % p.splits;
  const int slot = id / p.splits % p.g.slots, n0 = id / p.splits / p.g.slots * F::BN;
  const Place at{0, slot * F::BM, min(p.g.places - slot * F::BM, F::BM), false};
  const int from = split * p.part_k;
  few_tile<T, RM, RN>(p.g, at, n0, (const T*)p.g.p, from, min(from + p.part_k, p.g.k), sums, w,
                      lane);
  float* part = p.part + (int64_t)split * p.g.places * p.g.n;
  for (int x = tid; x < RM * RN * 64; x += F::T) {
    const int l = x & 63, j = (x >> 6) % RN, i = (x >> 6) / RN;
    const int m = 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m < at.count && n < p.g.n)
      *(floatx4*)(part + (int64_t)(at.first + m) * p.g.n + n) = sums[x];
  }
}

// Second launch: a thread adds the parts of four results in order, and their
// low-rank terms, rank multiplications each.
constexpr int kJoinThreads = 256;
template <class T, class O>
__global__ void __launch_bounds__(kJoinThreads) adapters_join(const AdapterParams p) {
  const int64_t x = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int wide = p.g.n / 4, place = (int)(x / wide), n = 4 * (int)(x - (int64_t)place * wide);
  if (place >= p.g.places) return;
  const int64_t plane = (int64_t)p.g.places * p.g.n;
  const float* part = p.part + (int64_t)place * p.g.n + n;
  floatx4 y{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) y += *(const floatx4*)(part + s * plane);
  const int g = owner_of(p, place), row = row_at(p.g, place);
  if (row < 0) return;
  if (g >= 0) {
    const float* h = p.h + (int64_t)place * p.rank;
    const T* b = (const T*)p.up + g * p.up_group + (int64_t)n * p.ldup;
    floatx4 low{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
    for (int c = 0; c < p.rank; c += 8) {
      const floatx4 h0 = *(const floatx4*)(h + c), h1 = *(const floatx4*)(h + c + 4);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const Vec8<T> bv = att::load8(b + v * p.ldup + c);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          low[v] = __builtin_fmaf(e < 4 ? h0[e % 4] : h1[e % 4], (float)bv[e], low[v]);
      }
    }
    y += low;
  }
  Out<O>::store4((O*)p.g.d + (int64_t)row * p.g.ldd + n, y);
}

// Small problems, one launch: a tile of 16 places of one group (or of none) by
// 16 RN columns forms its own h beside the shared product, as RA atoms more of
// the same contraction, and adds the low-rank term a result per thread.  h is
// formed again for every tile; what it saves is a launch, the workspace and the
// wait between the two: 48 rows of 256, rank 16, to 256 columns 4.5 us where
// two launches take 9.1, one row of 4096 to 4096 columns (RN = 1) 14 and 17.
// What bounds it is the latency of one pass over the contraction.  B's row is
// asked for ahead of the product.
template <int RN>
struct OneTile {
  static constexpr int BM = 16, BN = 16 * RN, T = 64 * kFewWaves;
  static_assert(BM * BN <= T, "a result per thread");
};
template <class T, class O, int RN, int RA>
__global__ void __launch_bounds__(64 * kFewWaves, 1) adapters_one(const AdapterParams p) {
  using F = OneTile<RN>;
  constexpr int NB = 2 * RA;
  __shared__ floatx4 sums[kFewWaves * (RN + RA) * 64];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const GroupSpot spot = group_spot<1>(p.g, blockIdx.x, F::BM);
  if (spot.spot.parts == 0) return;
  const Place at = spot.at;
  const int n0 = spot.spot.tn * F::BN;
  const bool has = at.group < p.g.groups;
  const int group = has ? at.group : 0;
  // the thread's result
  const int m = tid / F::BN, nn = tid % F::BN, n = n0 + nn;
  const bool mine = m < at.count && n < p.g.n;      // (at most 16 rows)
  const int row = mine ? row_at(p.g, at.first + m) : -1;
  const float scale = p.scale ? p.scale[group] : 1.0f;
  u32x4_t b[NB];
  const __amdgpu_buffer_rsrc_t rb =
      buffer((const T*)p.up + group * p.up_group + (int64_t)n0 * p.ldup, kWhole);
#pragma unroll
  for (int c = 0; c < NB; ++c)
    b[c] = __builtin_amdgcn_raw_buffer_load_b128(
        rb, has && mine && 8 * c < p.rank ? 2u * (nn * p.ldup + 8 * c) : kOutside, 0, 0);

  const int r = lane & 15;
  const unsigned c16 = 16u * (lane >> 4);
  unsigned q_off[1], p_off[RN + RA];
  few_rows<T, 1>(p.g, at, lane, q_off);
#pragma unroll
  for (int j = 0; j < RN; ++j)
    p_off[j] = n0 + 16 * j + r < p.g.n ? 2u * (16 * j + r) * p.g.ldp + c16 : kOutside;
#pragma unroll
  for (int j = 0; j < RA; ++j)
    p_off[RN + j] =
        has && 16 * j + r < p.rank ? 2u * (16 * j + r) * p.down.ldp + c16 : kOutside;
  const __amdgpu_buffer_rsrc_t rw = buffer((const T*)p.g.p + (int64_t)n0 * p.g.ldp, kWhole),
                               ra = buffer((const T*)p.down.p + group * p.down.p_group, kWhole);
  few_product<T, 1, RN + RA>(
      few_base<T>(p.g, at), q_off,
      [&](int j, bool in, int off) {
        const unsigned x = in ? p_off[j] : kOutside;
        return j < RN ? __builtin_amdgcn_raw_buffer_load_b128(rw, x, off, 0)
                      : __builtin_amdgcn_raw_buffer_load_b128(ra, x, off, 0);
      },
      0, p.g.k, spot.spot.tn + 3 * at.group, sums, w, lane);
  __syncthreads();
  if (row < 0) return;
  // value j of the place's columns from atom `atom` on
  auto value = [&](int atom, int j) {
    return ((const float*)sums)[((atom + j / 16) * 64 + m + 16 * (j % 16 / 4)) * 4 + j % 4];
  };
  float y = value(0, nn), low = 0.0f;
  if (has) {
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      if (8 * c >= p.rank) break;
      const Vec8<T> bv = as16(b[c], T());
#pragma unroll
      for (int e = 0; e < 8; ++e)
        low = __builtin_fmaf(scale * value(RN, 8 * c + e), (float)bv[e], low);
    }
    y += low;
  }
  ((O*)p.g.d)[(int64_t)row * p.g.ldd + n] = (O)y;
}

// What adapters_rows leaves out: the products of which a factor is not finite,
// for the place's columns n .. n + 3 (else -0, which changes no sum).
template <class T>
__device__ __forceinline__ floatx4 rest(const AdapterParams& p, int place, int n) {
  floatx4 low{-0.0f, -0.0f, -0.0f, -0.0f};
  const int g = owner_of(p, place);
  if (g < 0) return low;
  const T* b = (const T*)p.up + g * p.up_group + (int64_t)n * p.ldup;
  const float* h = p.h + (int64_t)place * p.rank;
  for (int c = 0; c < p.rank; ++c)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float x = h[c], y = (float)b[v * p.ldup + c];
      if (not_finite(x) || not_finite(y)) low[v] += x * y;
    }
  return low;
}

// h of a tile of one group's places, many rows: x is read once per 64 columns
// of the rank, and reading it is the work.  What bounds it is the latency of
// what a CU can have under way (its LDS), so the tiles are small, to go to more
// CUs, and the contraction is shared by kDownParts sets of two waves with
// stages of their own.  5,001 rows of 4096, rank 64: 16 us; with 64 rows per
// tile 19 (two sets) to 24 (four), straight from memory (down_few) 29.
constexpr int kDownParts = 4;
using DownTile = Tile<32, 64, 2, 1, 3>;
template <class T>
__global__ void __launch_bounds__(kDownParts * DownTile::T, 1) adapters_down_rows(
    const AdapterParams p) {
  using C = DownTile;
  __shared__ __attribute__((aligned(1024))) char smem[kDownParts * C::LDS];
  const int lane = threadIdx.x & 63, part = uniform(threadIdx.x / C::T),
            w = uniform(threadIdx.x >> 6) % C::W;
  const GroupSpot x = group_spot<1>(p.down, blockIdx.x, C::BM);
  if (x.spot.parts == 0 || x.at.group == p.down.groups) return;
  const int n0 = x.spot.tn * C::BN;
  const int steps = ((p.down.k + 63) / 64 + kDownParts - 1) / kDownParts;
  const int from = 64 * steps * part;         // (beyond k: out of range, zeros)
  GroupedParams d = p.down;
  d.k -= from;
  d.q = (const T*)d.q + from;
  RowsSource<C, false> src;
  src.init(d, x.at, n0, (const T*)d.p + x.at.group * d.p_group + from, w, lane);
  floatx4 acc[C::RM][C::RN];
  product<T, C, false, false>((lds_c)smem + part * C::LDS, steps, src, acc, w, lane);
  floatx4* sums = (floatx4*)smem;
  __syncthreads();
  if (part > 0)
#pragma unroll
    for (int j = 0; j < C::RN; ++j)
      sums[(((part - 1) * C::W + w) * C::RN + j) * 64 + lane] = acc[0][j];
  __syncthreads();
  const int m = 16 * w + (lane & 15);
  if (part > 0 || m >= x.at.count) return;
#pragma unroll
  for (int j = 0; j < C::RN; ++j) {
    floatx4 h = acc[0][j];
#pragma unroll
    for (int v = 1; v < kDownParts; ++v) h += sums[(((v - 1) * C::W + w) * C::RN + j) * 64 + lane];
    const int n = n0 + column_of(lane, j);
    if (n < p.rank) keep(p, x.at.first + m, x.at.group, n, h);
  }
}

// Tiles through LDS.  The low-rank term of each run of places of one group is
// a few matrix instructions more, on fragments straight from memory (a few KB
// that every workgroup of a row of tiles reads): rows of other groups multiply B
// by zeros, and 16 rows without one of the run are passed over.  bf16's add to
// the tile's own sums; fp16's are scaled.  What is not finite in B, which must
// not reach those other rows, or in s_g h, of whose infinities the pieces would
// make NaN, is left out there and added to the sums of its own rows afterwards.
// 5,001 rows of 4096 x 4096, fp16, with the down projection: 147 us without an
// adapter, 167 with 8 of rank 16, 186 of rank 64.  (s_g h as two 16-bit numbers,
// stored and read back, takes as long: bf16, rank 64, 172 us and 171.)
template <class T, class O, class C>
__device__ __forceinline__ void adapters_tile(const AdapterParams& p, char* smem, int first,
                                              int count, int n0) {
  constexpr int RN = C::RN, WROWS = 16 * C::RM, H = (C::RM + 3) / 4, HM = C::RM < 4 ? C::RM : 4;
  static_assert(H * HM == C::RM, "runs are found 64 rows at a time");
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const GroupedParams& g = p.g;
  RowsSource<C, false> src;
  src.init(g, Place{0, first, count, false}, n0, (const T*)g.p, w, lane);
  // the groups of the wave's places, 64 a time (asked for ahead of the product)
  const int m0 = first + (w % C::WM) * WROWS, nw = n0 + (w / C::WM) * 64;
  int own[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int at = m0 + 64 * h + lane;
    own[h] = lane < 16 * HM && at < first + count ? owner_of(p, at) : -1;
  }
  floatx4 acc[C::RM][RN];
  product<T, C, false, false>((lds_c)smem, (g.k + 63) / 64, src, acc, w, lane);

  // s_g h is an operand in pieces.  Where they are scaled, per row and 32 columns
  // of the rank, those columns' sums are registers of their own, scaled back when
  // they are added.
  constexpr bool SCALED = Pieces<T>::kScaled;
  const int r = lane & 15, c8 = 8 * (lane >> 4);
  bool bad = false;       // something was left out
  if (!SCALED) tied<C>(acc);
  // For 32 columns of the rank of a run: B, and s_g h of 16 rows at a time.  The
  // next ones are on their way while some are multiplied.
  struct Columns {
    u32x4_t x[RN];
  };
  struct Rows {
    u32x4_t x[2];
  };
  struct Step {
    int a, b, group, c;   // places a .. b - 1 of 64, columns c ..; group < 0: none
    unsigned long long starts;
  };
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int at = m0 + 64 * h;
    const __amdgpu_buffer_rsrc_t rh = buffer(p.h + (int64_t)at * p.rank, kWhole);
    auto load_b = [&](const Step& s) {
      Columns y;
      const __amdgpu_buffer_rsrc_t rb =
          buffer((const T*)p.up + max(s.group, 0) * p.up_group + (int64_t)nw * p.ldup, kWhole);
      const int c = s.group < 0 ? p.rank : s.c + c8;
#pragma unroll
      for (int j = 0; j < RN; ++j) {
        const int n = 16 * (r >> 2) + 4 * j + (r & 3);
        y.x[j] = __builtin_amdgcn_raw_buffer_load_b128(
            rb, c < p.rank && nw + n < g.n ? 2u * (n * p.ldup + c) : kOutside, 0, 0);
      }
      return y;
    };
    auto load_h = [&](const Step& s, int i) {
      Rows y;
      const int c = s.group < 0 ? p.rank : s.c + c8, m = 16 * i + r;
      const unsigned x = c < p.rank && m >= s.a && m < s.b ? 4u * (m * p.rank + c) : kOutside;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        y.x[e] = __builtin_amdgcn_raw_buffer_load_b128(rh, x, 16 * e, 0);
      return y;
    };
    auto finite = [&](Columns& y) {
#pragma unroll
      for (int j = 0; j < RN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const unsigned u = y.x[j][e];
          const bool z = not_finite<T>(u);
          y.x[j][e] = z ? 0u : u;
          bad |= z;
        }
    };
    auto use = [&](const Columns& b, const Rows& y, int i) {
      float left[8];
      unsigned top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const unsigned u = y.x[e / 4][e % 4];
        left[e] = __uint_as_float(u);
        top = max(top, u & 0x7fffffffu);
      }
      if (__any(top >= 0x7f800000u)) {
        bad = true;
        top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          left[e] = not_finite(left[e]) ? 0.0f : left[e];
          top = max(top, __float_as_uint(left[e]) & 0x7fffffffu);
        }
      }
      floatx4 low[RN];
      int ex = 0;
      if constexpr (SCALED) {
        ex = Pieces<T>::scale_of(__uint_as_float(top));
#pragma unroll
        for (int e = 0; e < 8; ++e) left[e] = __builtin_amdgcn_ldexpf(left[e], -ex);
#pragma unroll
        for (int j = 0; j < RN; ++j) low[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int v = 0; v < kPieces; ++v) {
        const Vec8<T> piece = Pieces<T>::take(left);
#pragma unroll
        for (int j = 0; j < RN; ++j) {
          if constexpr (SCALED)
            mma_low<T>(as16(b.x[j], T()), piece, low[j]);
          else
            Mma<T>::run(as16(b.x[j], T()), piece, acc[4 * h + i][j]);
        }
      }
      if constexpr (SCALED) {
        att::settle();
#pragma unroll
        for (int j = 0; j < RN; ++j) {
          asm volatile("" : "+v"(low[j]), "+a"(acc[4 * h + i][j]));
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[4 * h + i][j][v] += __builtin_amdgcn_ldexpf(low[j][v], ex);
          asm volatile("" : "+a"(acc[4 * h + i][j]));     // (else all leave their AGPRs at once)
        }
      }
    };
    auto advance = [&](Step s) {
      if (s.group >= 0 && (s.c += 32) < p.rank) return s;
      s.c = 0;
      do {
        if (!s.starts) {
          s.group = -1;
          return s;
        }
        s.a = __builtin_ctzll(s.starts);
        s.starts &= s.starts - 1;
        s.b = s.starts ? __builtin_ctzll(s.starts) : 64;
        s.group = __builtin_amdgcn_readlane(own[h], s.a);
      } while (s.group < 0);
      return s;
    };
    Step s = advance(Step{0, 0, -1, 0, run_starts(own[h], lane)});
    Columns b = load_b(s);
    Rows y = load_h(s, s.a / 16);
    while (s.group >= 0) {
      const Step to = advance(s);
      const Columns next = load_b(to);      // (of no step: nothing is read)
      const Rows ahead = load_h(to, to.a / 16);
      finite(b);
#pragma unroll
      for (int i = 0; i < HM; ++i)
        if (16 * i < s.b && 16 * i + 16 > s.a) {
          const Rows then = load_h(s, i + 1);
          use(b, y, i);
          y = then;
        }
      y = ahead;
      b = next;
      s = to;
    }
  }
  if (!SCALED) settled<C>(acc);
  if (__any(bad))
#pragma unroll 1
    for (int x = 0; x < C::RM * RN; ++x) {
      const int m = m0 - first + 16 * (x / RN) + r, n = nw + column_of(lane, x % RN);
      floatx4 y{-0.0f, -0.0f, -0.0f, -0.0f};
      if (m < count && n < g.n) y = rest<T>(p, first + m, n);
#pragma unroll
      for (int i = 0; i < C::RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j)
        {
          if (x == RN * i + j) acc[i][j] += y;
          asm volatile("" : "+a"(acc[i][j]));
        }
    }
  store_rows<O, C, true>(acc, n0, g.n, w, lane, [&](int m) {
    const int row = m < count ? row_at(g, first + m) : -1;
    return row < 0 ? nullptr : (O*)g.d + (int64_t)row * g.ldd;
  });
}

template <class T, class O, class S>
__global__ void __launch_bounds__(S::Full::T, 1) adapters_rows(const AdapterParams p) {
  using C = typename S::Full;
  __shared__ __attribute__((aligned(1024))) char smem[S::kLds];
  const Spot s = spot_of<S::kParts>(blockIdx.x, p.g.slots, p.g.tiles_n, p.g.band, INT_MAX);
  if (s.parts == 0) return;
  const Place at{0, s.tm * C::BM, min(p.g.places - s.tm * C::BM, C::BM), false};
  by_rows<S>(s, at, s.tn * C::BN, p.g.n, [&](auto c, const Place& x, int n0) {
    adapters_tile<T, O, decltype(c)>(p, smem, x.first, x.count, n0);
  });
}

}  // namespace grp
}  // namespace mfl
