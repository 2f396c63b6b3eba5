// Low-rank adapters of many requests beside a shared projection:
//
//   D(r, n) = sum_k x(r, k) W(n, k) + s_g sum_j h(r, j) B(g, n, j)
//   h(r, j) = sum_k x(r, k) A(g, j, k)             r = rows[place], place in group g
//
// Two launches.  The first forms s_g h for every place (few columns: the
// kernel for few rows, by group).  The second is the shared product on tiles
// of places whatever their group, so that W is read for all of them together,
// and adds the low-rank terms of the tile's groups to its sums before they
// are rounded.  A group's term reaches the rows of its own places alone, so
// infinities in one adapter stay with its requests.
//
// s_g h is kept to fp32's accuracy: as fp32 values where the second kernel
// multiplies them out itself (few rows), and as two 16-bit numbers (three
// with fp32 results) that add up to it where they are a matrix operand.
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

// 16-bit numbers that stand for an fp32 value.  Each leaves half a step, 2^-8
// (bf16) or 2^-11 (fp16) of what it stands for: two 2^-16 or 2^-22, far below
// a 16-bit result's own rounding, three 2^-24, an fp32 result's.
template <class O>
constexpr int pieces_of() {
  return sizeof(O) == 4 ? 3 : 2;
}

// s_g h of a tile of one group's places.  p.g: q = x, p = A, n = rank.
template <class T, int RM, int RN>
__global__ void __launch_bounds__(64 * kFewWaves, 1) adapters_down(const AdapterParams p) {
  using F = FewTile<RM, RN>;
  __shared__ floatx4 sums[kFewWaves * RM * RN * 64];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const GroupSpot spot = group_spot<1>(p.g, blockIdx.x, F::BM);
  if (spot.spot.parts == 0 || spot.at.group == p.g.groups) return;
  const Place at = spot.at;
  const int n0 = spot.spot.tn * F::BN;
  few_tile<T, RM, RN>(p.g, at, n0, (const T*)p.g.p + at.group * p.g.p_group, sums, w, lane);
  const float s = p.scale ? p.scale[at.group] : 1.0f;
  if (n0 == 0)
    for (int m = tid; m < at.count; m += F::T) p.owner[at.first + m] = at.group;
  // (a thread reads what it added itself)
  for (int x = tid; x < RM * RN * 64; x += F::T) {
    const int l = x & 63, j = (x >> 6) % RN, i = (x >> 6) / RN;
    const int m = 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m >= at.count || n >= p.rank) continue;
    floatx4 h = sums[x] * s;
    const int64_t place = at.first + m;
    if (p.h) {
      *(floatx4*)(p.h + place * p.rank + n) = h;
      continue;
    }
    typedef T vec4 __attribute__((ext_vector_type(4)));
    for (int c = 0; c < p.pieces; ++c) {
      vec4 y;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        y[v] = (T)h[v];
        const float z = (float)y[v];
        h[v] = not_finite(z) ? 0.0f : h[v] - z;
      }
      *(vec4*)((T*)p.hp + (place * p.pieces + c) * p.rank + n) = y;
    }
  }
}

// the group of a place that has one, else -1
__device__ __forceinline__ int owner_of(const AdapterParams& p, int place) {
  const int g = place < p.g.offsets[p.g.groups] ? p.owner[place] : -1;
  return (unsigned)g < (unsigned)p.g.groups ? g : -1;
}
// row of x and D at a place, -1 where it is outside
__device__ __forceinline__ int row_at(const GroupedParams& p, int place) {
  const int r = p.rows ? p.rows[place] : place;
  return (unsigned)r < (unsigned)p.q_rows ? r : -1;
}

// Few rows: every thread adds its own results' low-rank terms, rank
// multiplications each.
template <class T, class O, int RM, int RN>
__global__ void __launch_bounds__(64 * kFewWaves, 1) adapters_few(const AdapterParams p) {
  using F = FewTile<RM, RN>;
  __shared__ floatx4 sums[kFewWaves * RM * RN * 64];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const Spot s = spot_of<1>(blockIdx.x, p.g.slots, p.g.tiles_n, p.g.slots, INT_MAX);
  const Place at{0, s.tm * F::BM, min(p.g.places - s.tm * F::BM, F::BM)};
  const int n0 = s.tn * F::BN;
  few_tile<T, RM, RN>(p.g, at, n0, (const T*)p.g.p, sums, w, lane);
  for (int x = tid; x < RM * RN * 64; x += F::T) {
    const int l = x & 63, j = (x >> 6) % RN, i = (x >> 6) / RN;
    const int m = 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m >= at.count || n >= p.g.n) continue;
    const int place = at.first + m, g = owner_of(p, place), row = row_at(p.g, place);
    floatx4 y = sums[x];
    if (g >= 0) {
      const float* h = p.h + (int64_t)place * p.rank;
      const T* b = (const T*)p.up + g * p.up_group + (int64_t)n * p.ldup;
      floatx4 low{0.0f, 0.0f, 0.0f, 0.0f};
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
    if (row >= 0) Out<O>::store4((O*)p.g.d + (int64_t)row * p.g.ldd + n, y);
  }
}

// what adapters_rows leaves out: the pairs of B's numbers of which one is not
// finite, for the place's columns n .. n + 3
template <class T>
__device__ __forceinline__ floatx4 rest(const AdapterParams& p, int place, int n, int pieces) {
  floatx4 low{0.0f, 0.0f, 0.0f, 0.0f};
  const int g = owner_of(p, place);
  if (g < 0) return low;
  const T* b = (const T*)p.up + g * p.up_group + (int64_t)n * p.ldup;
  const T* h = (const T*)p.hp + (int64_t)place * pieces * p.rank;
  for (int c = 0; c < p.rank; c += 2) {
    float s[2] = {};
    for (int x = pieces; x--;)
      for (int e = 0; e < 2; ++e) s[e] += (float)h[x * p.rank + c + e];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float b0 = (float)b[v * p.ldup + c], b1 = (float)b[v * p.ldup + c + 1];
      if (not_finite(b0) || not_finite(b1)) low[v] += s[0] * b0 + s[1] * b1;
    }
  }
  return low;
}

// Tiles through LDS.  The low-rank term of each run of places of one group is
// a few matrix instructions more into the same sums, on fragments straight
// from memory (a few KB that every workgroup of a row of tiles reads): rows
// of other groups multiply B by zeros.  What is not finite in B is left out
// there, so that it cannot reach them, and added to its own rows at the end.
template <class T, class O, class C>
__device__ __forceinline__ void adapters_tile(const AdapterParams& p, char* smem, int first,
                                              int count, int n0) {
  constexpr int NPC = pieces_of<O>(), RN = C::RN, WROWS = 16 * C::RM, H = (C::RM + 3) / 4,
                HM = C::RM < 4 ? C::RM : 4;
  static_assert(H * HM == C::RM, "runs are found 64 rows at a time");
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const GroupedParams& g = p.g;
  RowsSource<C, false> src;
  src.init(g, Place{0, first, count}, n0, (const T*)g.p, w, lane);
  floatx4 acc[C::RM][RN];
  product<T, C, false, false>((lds_c)smem, (g.k + 63) / 64, src, acc, w, lane);

  const int m0 = first + (w % C::WM) * WROWS, nw = n0 + (w / C::WM) * 64;
  const int r = lane & 15, c8 = 8 * (lane >> 4);
  bool bad = false;       // something in B that is not finite
  tied<C>(acc);
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int at = m0 + 64 * h;
    const int own =
        lane < 16 * HM && at + lane < first + count ? owner_of(p, at + lane) : -1;
    unsigned long long starts = __ballot(lane == 0 || own != __shfl_up(own, 1));
    while (starts) {
      const int a = __builtin_ctzll(starts);
      starts &= starts - 1;
      const int b = starts ? __builtin_ctzll(starts) : 64;
      const int grp = __builtin_amdgcn_readlane(own, a);
      if (grp < 0) continue;
      const __amdgpu_buffer_rsrc_t rb =
          buffer((const T*)p.up + grp * p.up_group + (int64_t)nw * p.ldup, kWhole);
      const __amdgpu_buffer_rsrc_t rh =
          buffer((const T*)p.hp + (int64_t)at * NPC * p.rank, kWhole);
      for (int c0 = 0; c0 < p.rank; c0 += 32) {
        const bool in = c0 + c8 < p.rank;
        u32x4_t fp[RN], fq[NPC][HM];
#pragma unroll
        for (int j = 0; j < RN; ++j) {
          const int n = 16 * (r >> 2) + 4 * j + (r & 3);
          fp[j] = __builtin_amdgcn_raw_buffer_load_b128(
              rb, in && nw + n < g.n ? 2u * (n * p.ldup + c0 + c8) : kOutside, 0, 0);
        }
#pragma unroll
        for (int x = 0; x < NPC; ++x)
#pragma unroll
          for (int i = 0; i < HM; ++i) {
            const int m = 16 * i + r;
            fq[x][i] = __builtin_amdgcn_raw_buffer_load_b128(
                rh, in && m >= a && m < b ? 2u * ((m * NPC + x) * p.rank + c0 + c8) : kOutside, 0,
                0);
          }
        bool out = false;
#pragma unroll
        for (int j = 0; j < RN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned u = fp[j][e];
            const bool z = not_finite<T>(u);
            fp[j][e] = z ? 0u : u;
            out |= z;
          }
        bad |= out;
#pragma unroll
        for (int x = 0; x < NPC; ++x)
#pragma unroll
          for (int i = 0; i < HM; ++i)
#pragma unroll
            for (int j = 0; j < RN; ++j)
              Mma<T>::run(as16(fp[j], T()), as16(fq[x][i], T()), acc[4 * h + i][j]);
      }
    }
  }
  settled<C>(acc);
  auto row_of = [&](int m) {
    const int row = m < count ? row_at(g, first + m) : -1;
    return row < 0 ? nullptr : (O*)g.d + (int64_t)row * g.ldd;
  };
  store_rows<O, C, true>(acc, n0, g.n, w, lane, row_of);
  if (!__any(bad)) return;
  // (each lane reads what it stored: a sum with an infinity or NaN does not
  // depend on the rounding of its finite part)
#pragma unroll 1
  for (int x = 0; x < C::RM * RN; ++x) {
    const int m = m0 - first + 16 * (x / RN) + r, n = nw + column_of<true>(lane, x % RN);
    O* row = row_of(m);
    if (!row || n >= g.n) continue;
    floatx4 y = rest<T>(p, first + m, n, NPC);
#pragma unroll
    for (int v = 0; v < 4; ++v) y[v] += (float)row[n + v];
    Out<O>::store4(row + n, y);
  }
}

template <class T, class O, class S>
__global__ void __launch_bounds__(S::Full::T, 1) adapters_rows(const AdapterParams p) {
  using C = typename S::Full;
  __shared__ __attribute__((aligned(1024))) char smem[S::kLds];
  const Spot s = spot_of<S::kParts>(blockIdx.x, p.g.slots, p.g.tiles_n, p.g.band, INT_MAX);
  if (s.parts == 0) return;
  const Place at{0, s.tm * C::BM, min(p.g.places - s.tm * C::BM, C::BM)};
  by_rows<S>(s, at, [&](auto c, const Place& x) {
    adapters_tile<T, O, decltype(c)>(p, smem, x.first, x.count, s.tn * C::BN);
  });
}

}  // namespace grp
}  // namespace mfl
