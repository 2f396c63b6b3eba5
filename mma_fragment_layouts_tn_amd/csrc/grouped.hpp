// Products whose weights are chosen per row: experts' layers (grouped by
// expert, forward and both gradients) and low-rank adapters beside a shared
// projection.
//
// Every kernel here computes, on a tile of m x n,
//
//   D(m, n) = sum_c Q(m, c) P(n, c)
//
// and issues the matrix instruction with P first, so that lane l's four
// accumulators of an atom are four adjacent columns n = 4 (l / 16) + v of row
// m = l % 16: results leave the registers as vectors along D's rows.
//
//            D                       Q                       P
//   rows     D, a row per place      A rows (gathered), c=k  B[g], c = k
//   dA       dA, a row per place     dD rows, c = n          B[g], c = n, transposed
//   dB       dB[g], m = n, n = k     dD, c = place, transp.  A (gathered), c = place, transp.
//
// Transposed: the contraction is the strided direction in memory.  Such a
// tile lies in LDS as it does in memory (a row per c) and its fragments come
// from the transposing LDS read, so no operand is rearranged anywhere.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <type_traits>

#include "attention.hpp"
#include "grouped_launch.hpp"

namespace mfl {
namespace grp {

using att::barrier;
using att::BoolC;
using att::Elem;
using att::floatx4;
using att::lds_c;
using att::lds_s4;
using att::lds_t;
using att::shortx4;
using att::Span;
using att::span_of;
using att::uniform;
using att::Vec8;

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

constexpr unsigned kOutside = 0x80000000u;   // a lane's offset beyond any descriptor's range
constexpr int kWhole = 0x7fffffff;

// acc += P Q^T on one atom, the accumulator tied to one AGPR tuple (with the
// builtin the compiler rotates a wave's tuples through copies in the loop).
// It sees no hazards through the statement: two wait states ahead of it cover
// operands assembled by vector instructions, settle() what follows the last.
template <class T>
struct Mma;
template <>
struct Mma<_Float16> {
  static __device__ __forceinline__ void run(const Vec8<_Float16>& p, const Vec8<_Float16>& q,
                                             floatx4& c) {
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(p), "v"(q));
  }
};
template <>
struct Mma<__bf16> {
  static __device__ __forceinline__ void run(const Vec8<__bf16>& p, const Vec8<__bf16>& q,
                                             floatx4& c) {
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(p), "v"(q));
  }
};

// A tile of BM x BN by WM x WN waves, BC contraction elements per step, NST
// stages.  Each wave 16 RM x 64.
template <int BM_, int BN_, int WM_, int WN_, int NST_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BC = 64;
  static constexpr int W = WM * WN, T = 64 * W;
  static constexpr int RM = BM / WM / 16, RN = BN / WN / 16;
  static constexpr int P_BYTES = BN * BC * 2, Q_BYTES = BM * BC * 2;
  static constexpr int NST = NST_, STAGE = P_BYTES + Q_BYTES, LDS = NST * STAGE;
  static constexpr int NP = P_BYTES / 1024 / W, NQ = Q_BYTES / 1024 / W, NI = NP + NQ;
  static_assert(RN == 4, "the order of P's rows in LDS is made for 64 columns per wave");
  static_assert(NP * W * 1024 == P_BYTES && NQ * W * 1024 == Q_BYTES, "loads divide over waves");
  static_assert(LDS <= 160 * 1024, "stages fit LDS");
};

// Tiles of 256 x 256 by 8 waves of 128 x 64, two per SIMD, one workgroup per
// CU.  The tiles of a launch's last, incomplete round are cut in up to kParts,
// one part to a workgroup, as long as those find room in the round, and a tile
// of few rows is computed as the smaller one: 68 tiles by 8 are 2 rounds and a
// little, not 3 (by_rows).
//
// A smaller tile's step is over before the loads of the next have come (a
// quarter's: 0.7 us a step with two stages, where its instructions take 0.25),
// so it keeps as many stages as LDS holds.
struct Tiles256 {
  using Full = Tile<256, 256, 2, 4>;
  using Half = Tile<128, 256, 2, 4, 3>;
  using Quarter = Tile<64, 256, 2, 4, 4>;
  using Corner = Tile<128, 128, 4, 2, 5>;
  using Eighth = Tile<64, 128, 4, 2, 6>;
  static constexpr int kParts = 8, kLds = Quarter::LDS;
  static_assert(kLds >= Corner::LDS && kLds >= Eighth::LDS, "one size for all");
};
// the same where both operands are transposed
struct Weights256 {
  using Full = Tile<256, 256, 2, 4>;
  using Half = Tile<128, 256, 2, 4>;
  using Corner = Tile<128, 128, 4, 2>;
  static constexpr int kParts = 4, kLds = Full::LDS;
};
// Tiles of 128 x 128 by 4 waves of 64 x 64, two workgroups per CU.
struct Tiles128 {
  using Full = Tile<128, 128, 2, 2>;
  static constexpr int kParts = 1, kLds = Full::LDS;
};

// P's rows in LDS (contraction contiguous): row 16 j + 4 q + v of a wave's 64
// holds column 16 q + 4 j + v, so the four atoms' accumulators of a lane are
// 16 adjacent columns.  Its own inverse.
MFL_HD constexpr int perm64(int r) {
  return (r & ~63) | ((r >> 2) & 3) << 4 | ((r >> 4) & 3) << 2 | (r & 3);
}

// The sums are as vector instructions wrote them, and the wait states before a
// matrix instruction takes them have passed.
template <class C>
__device__ __forceinline__ void tied(floatx4 (&acc)[C::RM][C::RN]) {
#pragma unroll
  for (int i = 0; i < C::RM; ++i)
#pragma unroll
    for (int j = 0; j < C::RN; ++j) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 4" ::);
}
// The matrix instructions' results are written: the sums may be moved or read.
template <class C>
__device__ __forceinline__ void settled(floatx4 (&acc)[C::RM][C::RN]) {
  att::settle();
#pragma unroll
  for (int i = 0; i < C::RM; ++i)
#pragma unroll
    for (int j = 0; j < C::RN; ++j) asm volatile("" : "+a"(acc[i][j]));
}

// ------------------------------------------------------- fragment reads
// Contraction-contiguous tile, rows of 64 elements (lds_offset<64>): the
// fragment of rows 16 i + l % 16, sub-step kk.
template <class T>
struct Straight {
  unsigned at;
  static __device__ __forceinline__ Straight of(int row0, int lane) {
    const int r = lane & 15;
    return Straight{2u * lds_offset<64>(row0 + r, 8 * (lane >> 4))};
  }
  __device__ __forceinline__ Vec8<T> read(lds_c stage, int i, int kk) const {
    using ptr = const __attribute__((address_space(3))) Vec8<T>*;
    return *(ptr)(stage + ((at ^ (64u * kk)) + 2048u * i));
  }
};
constexpr bool straight_addresses_hold() {
  for (int r = 0; r < 16; ++r)
    for (int c = 0; c < 4; ++c)
      for (int i = 0; i < 8; ++i)
        for (int kk = 0; kk < 2; ++kk)
          if (2 * lds_offset<64>(16 * i + r, 32 * kk + 8 * c) !=
              ((2 * lds_offset<64>(r, 8 * c)) ^ (64 * kk)) + 2048 * i)
            return false;
  return true;
}
static_assert(straight_addresses_hold(), "sub-steps by XOR, atoms by offset");

// Transposed tile, 64 rows (one per c) of R elements (lds_offset_mn<R>): two
// reads of four rows each fill the fragment.
template <class T, int R>
struct Transposed {
  unsigned at;
  static __device__ __forceinline__ Transposed of(int row0, int lane) {
    const int s = lane & 15, blk = lane >> 4;
    return Transposed{2u * lds_offset_mn<R>(row0 + 4 * (s & 3), 8 * blk + (s >> 2))};
  }
  __device__ __forceinline__ Vec8<T> read(lds_c stage, int i, int kk) const {
    const lds_c a = stage + ((at ^ (32u * i)) + 64u * R * kk);
    const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)a);
    const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(a + 8 * R));
    return __builtin_bit_cast(Vec8<T>, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};
template <int R>
constexpr bool transposed_addresses_hold() {
  for (int row0 = 0; row0 < R; row0 += 64)
    for (int s = 0; s < 4; ++s)
      for (int k = 0; k < 32; ++k)
        for (int i = 0; i < (R - row0 >= 128 && row0 % 128 == 0 ? 8 : 4); ++i)
          for (int kk = 0; kk < 2; ++kk)
            if (2 * lds_offset_mn<R>(row0 + 16 * i + 4 * s, 32 * kk + k) !=
                ((2 * lds_offset_mn<R>(row0 + 4 * s, k)) ^ (32 * i)) + 64 * R * kk)
              return false;
  return true;
}
static_assert(transposed_addresses_hold<128>() && transposed_addresses_hold<256>(),
              "atoms by XOR, sub-steps by offset");

template <class T, int R, bool TR>
struct ReaderOf {
  using type = Straight<T>;
};
template <class T, int R>
struct ReaderOf<T, R, true> {
  using type = Transposed<T, R>;
};

// ------------------------------------------------------------ pipeline
// `steps` steps of 64 contraction elements into acc.  issue(kt, i, stage)
// sends load i (of the wave's NI) of step kt into the stage at `stage`;
// ahead(kt) is called a step before the loads of step kt are issued.
//
// A step is two sub-steps of 32.  The first one's matrix instructions run
// while the second one's fragments are read; then every wave has its loads of
// the next step and is done with this stage (the barrier); the second one's
// run while the next stage's first fragments are read and the loads of the
// step NST further go into this stage, one by one between the instructions.
template <class T, class C, bool PT, bool QT, class Source>
__device__ __forceinline__ void product(lds_c ring, int steps, Source& src,
                                        floatx4 (&acc)[C::RM][C::RN], int w, int lane) {
  constexpr int RM = C::RM, RN = C::RN, NI = C::NI;
  const typename ReaderOf<T, C::BN, PT>::type rp =
      ReaderOf<T, C::BN, PT>::type::of((w / C::WM) * (C::BN / C::WN), lane);
  const typename ReaderOf<T, C::BM, QT>::type rq =
      ReaderOf<T, C::BM, QT>::type::of((w % C::WM) * (C::BM / C::WM), lane);
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  tied<C>(acc);
  if (steps > 0) {
    Vec8<T> fp[2][RN], fq[2][RM];
    // fragment read r in the order the instructions take them
    auto read = [&](int r, int buf, int kk, lds_c stage) {
      if (r == 0)
        fq[buf][0] = rq.read(stage + C::P_BYTES, 0, kk);
      else if (r <= RN)
        fp[buf][r - 1] = rp.read(stage, r - 1, kk);
      else
        fq[buf][r - RN] = rq.read(stage + C::P_BYTES, r - RN, kk);
    };
    constexpr int kReads = RM + RN, kMma = RM * RN, kSlots = kMma / 2;
    auto group = [&](int buf, lds_c stage, auto loads, int kt, lds_c to) {
#pragma unroll
      for (int g = 0; g < kMma; ++g) {
        if (C::W > 4) {           // two waves of the workgroup per SIMD take turns
          if (g == 0) __builtin_amdgcn_s_setprio(1);
          if (g == kMma / 2) __builtin_amdgcn_s_setprio(0);
        }
        Mma<T>::run(fp[buf][g % RN], fq[buf][g / RN], acc[g / RN][g % RN]);
        if (g < kSlots)
#pragma unroll
          for (int r = g * kReads / kSlots; r < (g + 1) * kReads / kSlots; ++r)
            read(r, 1 - buf, 1 - buf, stage);
        if constexpr (decltype(loads)::value)
#pragma unroll
          for (int i = g * NI / kMma; i < (g + 1) * NI / kMma; ++i) src.issue(kt, i, to);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    using Yes = BoolC<true>;
    using No = BoolC<false>;
    // the stage read now, the next one, and where the loads go: distinct for
    // the compiler, which otherwise lets every transposing read wait for them
    constexpr int NST = C::NST, HEAD = Source::kAhead;
    static_assert(HEAD == 0 || NST == 2, "ahead() reaches one step");
    auto step = [&](int kt, lds_c __restrict__ from, lds_c __restrict__ next,
                    lds_c __restrict__ to) {
      group(0, from, No(), 0, to);
      att::wait_vm<(NST - 2) * NI>();
      barrier();
      group(1, next, Yes(), kt + NST, to);
      src.ahead(kt + NST + 1);
    };
#pragma unroll
    for (int st = 0; st < NST; ++st) {
      src.ahead(st);
#pragma unroll
      for (int i = 0; i < NI; ++i) src.issue(st, i, ring + st * C::STAGE);
    }
    src.ahead(NST);
    att::wait_vm<(NST - 1) * NI + HEAD>();
    barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(r, 0, 0, ring);
    // One body for every step (several would need the sums at the same
    // registers where they meet): the loads behind the last step are out of
    // range and move nothing, the fragments read behind it are not used.
    lds_c from = ring, last = ring + (NST - 1) * C::STAGE;
    for (int kt = 0; kt < steps; ++kt) {
      const lds_c next = from == last ? ring : from + C::STAGE;
      step(kt, from, next, from);
      from = next;
    }
    att::wait_vm<0>();
    settled<C>(acc);       // (inside the condition: where the paths meet is too late)
  }
}

// ---------------------------------------------------- where loads come from
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00027000);
}
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, lds_c to, unsigned lane_off,
                                         int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_t)to, 16, lane_off, off, 0, 0);
}

// R rows with the contraction contiguous, `k` elements of it: LDS run j holds
// rows 8 j .. 8 j + 7.  at(row): byte offset of a row, or kOutside.
template <int N>
struct RowLoads {
  __amdgpu_buffer_rsrc_t r;
  unsigned off[N];
  int col;           // of the even runs; 32 further or nearer in the odd ones
  int k, run0;
  template <class At>
  __device__ __forceinline__ void init(const void* base, int k_, int w, int lane, At at) {
    r = buffer(base, kWhole);
    k = k_;
    run0 = w * N;
    col = 8 * ((lane & 7) ^ ((lane >> 4) & 3));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = 8 * (run0 + i) + (lane >> 3);
      const unsigned x = at(row);
      off[i] = x == kOutside ? x : x + 2u * column(i);
    }
  }
  // (swz<8> of a row is its bits 1 - 3, bit 3 of them the run's parity)
  __device__ __forceinline__ int column(int i) const { return col ^ (((run0 + i) & 1) * 32); }
  __device__ __forceinline__ void issue(int kt, int i, lds_c to) const {
    const unsigned x = column(i) < k - 64 * kt ? off[i] : kOutside;
    load_lds(r, to + (run0 + i) * 1024, x, 128 * kt);
  }
};

// A transposed tile of R columns from column col0 on (of `width`): LDS run j
// holds 512 / R rows.
template <int R, int N>
struct ColumnLoads {
  static constexpr int RUN = 512 / R, CPR = R / 8;
  unsigned off[N];   // column's byte offset within a row, kOutside past the width
  int row0;          // the lane's row within run 0 of the wave
  int run0;
  __device__ __forceinline__ void init(int col0, int width, int w, int lane) {
    run0 = w * N;
    row0 = RUN * run0 + lane / CPR;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col0 + 8 * ((lane % CPR) ^ mn_swz(row0 + RUN * i));
      off[i] = c < width ? 2u * c : kOutside;
    }
  }
};

// rows follow each other, `count` of them, `ld` elements apart
template <int R, int N>
struct PlainColumns : ColumnLoads<R, N> {
  using Base = ColumnLoads<R, N>;
  const char* base;
  int64_t count;
  int ld, width;
  __device__ __forceinline__ void init(const void* b, int64_t n, int ld_, int col0, int width_,
                                       int w, int lane) {
    Base::init(col0, width_, w, lane);
    base = (const char*)b;
    count = n;
    ld = ld_;
    width = width_;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (this->off[i] != kOutside) this->off[i] += 2u * (this->row0 + Base::RUN * i) * ld;
  }
  __device__ __forceinline__ void issue(int kt, int i, lds_c to) const {
    const int64_t left = count - 64 * (int64_t)kt;
    const int rows = left < 64 ? (int)left : 64;
    const __amdgpu_buffer_rsrc_t r = buffer(base + (int64_t)kt * 128 * ld,
                                            rows > 0 ? 2 * ((rows - 1) * ld + width) : 0);
    load_lds(r, to + (this->run0 + i) * 1024, this->off[i], 0);
  }
};

// the rows index[0] .. index[count - 1] of `total` rows; a number outside
// counts as a row of zeros
template <int R, int N>
struct GatheredColumns : ColumnLoads<R, N> {
  using Base = ColumnLoads<R, N>;
  __amdgpu_buffer_rsrc_t r;
  const int* index;
  int ld, total, count;
  int next[N];       // indices of the step whose loads are issued next
  __device__ __forceinline__ void init(const void* b, const int* index_, int n, int ld_, int total_,
                                       int col0, int width, int w, int lane) {
    Base::init(col0, width, w, lane);
    r = buffer(b, kWhole);
    index = index_;
    ld = ld_;
    total = total_;
    count = n;
  }
  __device__ __forceinline__ void ahead(int kt) {
    const int left = min(max(count - 64 * kt, 0), 64);
    const __amdgpu_buffer_rsrc_t list = buffer(index + 64 * (int64_t)kt, 4 * left);
#pragma unroll
    for (int i = 0; i < N; ++i)
      next[i] = __builtin_amdgcn_raw_buffer_load_b32(list, 4 * (this->row0 + Base::RUN * i), 0, 0);
  }
  __device__ __forceinline__ void issue(int kt, int i, lds_c to) const {
    const int row = next[i];
    const bool ok = 64 * kt + this->row0 + Base::RUN * i < count &&
                    (unsigned)row < (unsigned)total && this->off[i] != kOutside;
    unsigned x = 2u * row * ld + this->off[i];
    asm volatile("" : "+v"(x));     // (else formed in a branch of its own)
    load_lds(r, to + (this->run0 + i) * 1024, ok ? x : kOutside, 0);
  }
};

// ---------------------------------------------------------- rows of groups
struct Place {
  int group, first, count;    // the tile's first place, its places
  bool small;                 // the group's matrix is read by two tiles at most
};

// Workgroups go to the 8 XCDs in turn; renumbered, each XCD has a run of
// consecutive numbers (as tile_of_block).
__device__ __forceinline__ int in_runs(int id, int n) {
  const int q = n / 8, r = n % 8, x = id % 8;
  return x * q + min(x, r) + id / 8;
}
// number -> tile, in bands `band` tiles tall
__device__ __forceinline__ TileIndex tile_at(int lin, int tiles_m, int tiles_n, int band) {
  const int g = lin / (band * tiles_n), in = lin - g * band * tiles_n;
  const int rows = min(tiles_m - g * band, band);
  return TileIndex{g * band + in % rows, in / rows};
}

// A workgroup's tile of `tiles_m` x `tiles_n`, or its part of one: those of
// the last round of kFill workgroups are cut into up to PARTS.
struct Spot {
  int tm, tn, part, parts;    // parts 0: nothing to do
};
// `each` numbers at a time are dealt out to the XCDs.
template <int PARTS>
__device__ __forceinline__ Spot spot_of(int id, int tiles_m, int tiles_n, int band, int each) {
  const int n = tiles_m * tiles_n;
  int whole = n, parts = 1;
  if constexpr (PARTS > 1) {
    const int rest = n % kFill;
    while (rest > 0 && parts < PARTS && rest * parts * 2 <= kFill) parts *= 2;
    if (parts > 1) whole = n - rest;
  }
  int lin, part = 0;
  if (id < whole) {
    const int from = id / each * each;
    lin = from + in_runs(id - from, min(each, whole - from));
    parts = 1;
  } else {
    const int cut = (n - whole) * parts;
    if (id - whole >= cut) return Spot{0, 0, 0, 0};
    const int x = in_runs(id - whole, cut);
    lin = whole + x / parts;
    part = x % parts;
  }
  const TileIndex t = tile_at(lin, tiles_m, tiles_n, band);
  return Spot{t.tm, t.tn, part, parts};
}

// Tiles of `bm` places, none across two groups; the places behind the last
// group are a group of their own (group == p.groups).
//
// Up to kExact - 1 groups every wave counts the tiles of all of them, 64
// groups a time, so that the tiles are numbered without gaps and the launch's
// workgroups beyond them are the last ones.  (With the numbering below, 4096
// rows in one group left two of 18 slots empty, which made one of the 8 XCDs
// idle and the others run a second round: 793 TFLOP/s where it gives 1,270.)
// For more groups, group g takes the numbers from start(g) / bm + g on, as
// attention's tiles of sequences, some of them empty, and the last round is not
// cut: 1,024 choices of 255 groups of 512 x 2048 take 104 us, of 256 127; 65,536
// choices 215 and 263.
constexpr int kSmall = 256;
struct GroupSpot {
  Spot spot;
  Place at;
};
template <int PARTS>
__device__ __forceinline__ GroupSpot group_spot(const GroupedParams& p, int id, int bm) {
  auto held = [&](int g) { return min(max(p.offsets[g], 0), p.places); };
  GroupSpot r;
  if (p.groups >= kExact) {
    r.spot = spot_of<1>(id, p.slots, p.tiles_n, p.band ? p.band : p.slots, INT_MAX);
    if (r.spot.parts == 0) return r;
    auto first = [&](int g) { return held(g) / bm + g; };
    const int g = att::find_sequence(p.groups + 1, r.spot.tm, first);
    const int a = uniform(held(g)), b = uniform(g < p.groups ? held(g + 1) : p.places);
    const int t = r.spot.tm - (a / bm + g);
    r.at = Place{g, a + t * bm, t < 0 ? 0 : min(max(b - a, 0) - t * bm, bm), b - a <= kSmall};
    if (r.at.count <= 0) r.spot.parts = 0;
    return r;
  }
  constexpr int NB = kExact / 64;
  const int lane = threadIdx.x & 63;
  int start[NB], len[NB], before[NB], total = 0;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int g = 64 * b + lane;
    start[b] = g <= p.groups ? held(g) : 0;
    const int end = g < p.groups ? held(g + 1) : p.places;
    len[b] = g <= p.groups ? max(end - start[b], 0) : 0;
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (64 * b > p.groups) break;
    const int mine = (len[b] + bm - 1) / bm;
    int scan = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int t = __shfl_up(scan, d);
      if (lane >= d) scan += t;
    }
    before[b] = total + scan - mine;
    total += __builtin_amdgcn_readlane(scan, 63);
  }
  r.spot = spot_of<PARTS>(id, total, p.tiles_n, p.band ? p.band : max(total, 1), INT_MAX);
  if (r.spot.parts == 0) return r;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (64 * b > p.groups) break;
    const unsigned long long m = __ballot(len[b] > 0 && before[b] <= r.spot.tm);
    if (!m) continue;
    const int l = 63 - __builtin_clzll(m);
    const int t = r.spot.tm - __builtin_amdgcn_readlane(before[b], l);
    const int n = __builtin_amdgcn_readlane(len[b], l);
    r.at = Place{64 * b + l, __builtin_amdgcn_readlane(start[b], l) + t * bm, min(n - t * bm, bm),
                 n <= kSmall};
  }
  return r;
}

template <class O>
struct Out;
template <>
struct Out<float> {
  static __device__ __forceinline__ void store4(float* p, const floatx4& x) { *(floatx4*)p = x; }
};
template <class O>
struct Out {
  typedef O vec4 __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ void store4(O* p, const floatx4& x) {
    *(vec4*)p = vec4{(O)x[0], (O)x[1], (O)x[2], (O)x[3]};
  }
};

// Columns of a lane's accumulators (P's order in LDS as perm64): atom j's four
// from column_of(lane, j) on.
__device__ __forceinline__ int column_of(int lane, int j) { return 16 * (lane >> 4) + 4 * j; }

// Exchanges between two lanes of which one bit differs: afterwards a lane with
// the bit clear has both lanes' a, one with the bit set both lanes' b, in the
// order of the lanes.
template <int BIT>
__device__ __forceinline__ void exchange(unsigned& a, unsigned& b, int lane) {
  if constexpr (BIT == 5 || BIT == 4) {
    const auto r = BIT == 5 ? __builtin_amdgcn_permlane32_swap(a, b, false, false)
                            : __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
  } else {
    static_assert(BIT == 3 || BIT == 2, "lane bits 2 to 5");
    const bool set = lane >> BIT & 1;
    const int send = (int)(set ? a : b);
    const unsigned got = BIT == 3
                             ? __builtin_amdgcn_mov_dpp(send, 0x128, 0xf, 0xf, false)   // row_ror:8
                             : __builtin_amdgcn_ds_swizzle(send, 0x101f);                // xor 4
    a = set ? got : a;
    b = set ? b : got;
  }
}

// The wave's rows, row_of(m) for row m of the tile (null: none), columns <
// width.  An accumulator tuple is four columns of a row: stored as they are, a
// row's 128-byte lines are written a quarter at a time, and the L2s put them
// together.  Exchanges between lanes make 16 columns per lane (which P's order
// in LDS does for tiles that have it) and then, of 16 rows by 64 columns, whole
// rows per store, 8 lanes a line, which need not stay in the L2s.  D, dA and dB
// of 8192 places, 8 groups of 4096 x 2048: 447 us by quarters (510 if those are
// non-temporal), 419 by lines, 401 if non-temporal; D of 16384 places, 2048 x
// 4096, 260 and 251.
template <class O, class C, bool PERM, class RowOf>
__device__ __forceinline__ void store_rows(const floatx4 (&acc)[C::RM][C::RN], int col0, int width,
                                           int w, int lane, RowOf row_of) {
  constexpr int NW = sizeof(O);          // dwords of four values (2 or 4 bytes each)
  const int m0 = (w % C::WM) * (16 * C::RM), n0 = col0 + (w / C::WM) * 64 + 16 * (lane >> 4);
#pragma unroll
  for (int i = 0; i < C::RM; ++i) {
    unsigned u[4][NW];                   // columns 4 x of the lane's 16
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if constexpr (NW == 4) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float f = acc[i][x][v];
          u[x][v] = __float_as_uint(f);
        }
      } else {
        typedef O vec4 __attribute__((ext_vector_type(4)));
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        const floatx4 f = acc[i][x];
        const u32x2 p = __builtin_bit_cast(u32x2, vec4{(O)f[0], (O)f[1], (O)f[2], (O)f[3]});
        u[x][0] = p[0];
        u[x][1] = p[1];
      }
    }
    if constexpr (!PERM) {
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        exchange<5>(u[0][v], u[2][v], lane);
        exchange<5>(u[1][v], u[3][v], lane);
        exchange<4>(u[0][v], u[1][v], lane);
        exchange<4>(u[2][v], u[3][v], lane);
      }
    }
    // pieces of 16 bytes: bits of the row for bits of the piece
    u32x4_t piece[NW];
    if constexpr (NW == 4) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        exchange<3>(u[0][v], u[2][v], lane);
        exchange<3>(u[1][v], u[3][v], lane);
        exchange<2>(u[0][v], u[1][v], lane);
        exchange<2>(u[2][v], u[3][v], lane);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) piece[x] = u32x4_t{u[x][0], u[x][1], u[x][2], u[x][3]};
    } else {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        exchange<3>(u[0][v], u[2][v], lane);
        exchange<3>(u[1][v], u[3][v], lane);
      }
      piece[0] = u32x4_t{u[0][0], u[0][1], u[1][0], u[1][1]};
      piece[1] = u32x4_t{u[2][0], u[2][1], u[3][0], u[3][1]};
    }
    constexpr int ROWS = 16 / NW, COLS = 16 / NW;    // rows of a store, columns of a piece
    const int n = n0 + COLS * ((lane & 15) / ROWS);
    if (n >= width) continue;
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      O* row = row_of(m0 + 16 * i + ROWS * x + (lane & 15) % ROWS);
      if (row) __builtin_nontemporal_store(piece[x], (u32x4_t*)(row + n));
    }
  }
}
// rows follow each other
template <class O, class C, bool PERM>
__device__ __forceinline__ void store_tile(O* base, int64_t ld, int rows, int col0, int width,
                                           const floatx4 (&acc)[C::RM][C::RN], int w, int lane) {
  store_rows<O, C, PERM>(acc, col0, width, w, lane,
                         [&](int m) { return m < rows ? base + (int64_t)m * ld : nullptr; });
}

template <class O, class C>
__device__ __forceinline__ void zero_tile(O* base, int64_t ld, int rows, int col0, int width,
                                          int tid) {
  for (int x = tid; x < rows * (C::BN / 4); x += C::T) {
    const int m = x / (C::BN / 4), n = col0 + 4 * (x % (C::BN / 4));
    if (n < width) Out<O>::store4(base + (int64_t)m * ld + n, floatx4{0.0f, 0.0f, 0.0f, 0.0f});
  }
}

template <class C, bool PT>
struct RowsSource {
  static constexpr int kAhead = 0;    // loads of ahead()
  RowLoads<C::NQ> q;
  typename std::conditional<PT, PlainColumns<C::BN, C::NP>, RowLoads<C::NP>>::type p;
  // The step that the contraction begins with (it goes round), the same for
  // tiles of the same weights.  Weights that few tiles read come straight from
  // memory, and where their rows lie a power of two apart, workgroups in step
  // would all ask the same channels: 64 groups of 8 rows, 1024 x 2048, 67 us in
  // step, 55 so, 48 with rows of 2112.
  int begin = 0, steps = 0;
  __device__ __forceinline__ void start(int id, int k) {
    steps = (k + 63) / 64;
    begin = id % steps;
  }
  // the tile's places against columns n0 .. of the matrix P
  template <class T>
  __device__ __forceinline__ void init(const GroupedParams& a, const Place& at, int n0, const T* P,
                                       int w, int lane) {
    if (a.rows)
      q.init(a.q, a.k, w, lane, [&](int row) {
        const int r = a.rows[at.first + min(row, at.count - 1)];
        return row < at.count && (unsigned)r < (unsigned)a.q_rows ? 2u * (unsigned)r * a.ldq
                                                                  : kOutside;
      });
    else
      q.init((const T*)a.q + (int64_t)at.first * a.ldq, a.k, w, lane,
             [&](int row) { return row < at.count ? 2u * row * a.ldq : kOutside; });
    if constexpr (PT)
      p.init(P, a.k, a.ldp, n0, a.n, w, lane);
    else
      p.init(P + (int64_t)n0 * a.ldp, a.k, w, lane, [&](int row) {
        const int n = perm64(row);
        return n0 + n < a.n ? 2u * n * a.ldp : kOutside;
      });
  }
  __device__ __forceinline__ void ahead(int) {}
  __device__ __forceinline__ void issue(int kt, int i, lds_c to) const {
    if (kt < steps) {
      kt += begin;
      kt = kt < steps ? kt : kt - steps;
    }
    if (i < C::NP)
      p.issue(kt, i, to);
    else
      q.issue(kt, i - C::NP, to + C::P_BYTES);
  }
};

// a tile of places of one group against columns n0 ..
template <class T, class O, class C, bool PT>
__device__ __forceinline__ void rows_tile(const GroupedParams& p, char* smem, const Place& at,
                                          int n0) {
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  O* D = (O*)p.d + (int64_t)at.first * p.ldd;
  if (at.group == p.groups) {       // of no group: no result, or no gradient
    if constexpr (PT) zero_tile<O, C>(D, p.ldd, at.count, n0, p.n, tid);
    return;
  }
  RowsSource<C, PT> src;
  src.init(p, at, n0, (const T*)p.p + at.group * p.p_group, w, lane);
  if (!PT && at.small) src.start(at.group * p.tiles_n + n0 / C::BN, p.k);
  floatx4 acc[C::RM][C::RN];
  product<T, C, PT, false>((lds_c)smem, (p.k + 63) / 64, src, acc, w, lane);
  store_tile<O, C, !PT>(D, p.ldd, at.count, n0, p.n, acc, w, lane);
}

// A part of a tile of places against columns n0 ..; f with the tile that fits
// it.  The rows there are, to 64, 128 or 256, and 256 columns are halved in
// turn, so that a part reads as little as it can for its results.  What a part
// has under way is what LDS holds, and few parts are bound by the latency of
// it: 2 groups of 150 places, 2048 x 4096, cut by rows alone 46 us, so 29; both
// gradients of 666 places, 16 groups of 1024 x 512, 20 and 17.
template <class S, class F>
__device__ __forceinline__ void by_rows(const Spot& spot, Place at, int n0, int width, F f) {
  if constexpr (S::kParts == 1) {
    f(typename S::Full(), at, n0);
  } else {
    int rows = at.count <= 64 ? 64 : at.count <= 128 ? 128 : 256, cols = 256;
    if (spot.parts > 1) rows == 256 ? rows = 128 : cols = 128;
    if (spot.parts > 2) cols == 256 ? cols = 128 : rows = 64;
    if (spot.parts > 4) rows = 64;
    const int across = 256 / cols, m = spot.part / across * rows;
    n0 += spot.part % across * cols;
    at.first += m;
    at.count = min(at.count - m, rows);
    if (at.count <= 0 || n0 >= width) return;
    if (cols == 128)
      at.count <= 64 ? f(typename S::Eighth(), at, n0) : f(typename S::Corner(), at, n0);
    else if (at.count <= 64)
      f(typename S::Quarter(), at, n0);
    else if (at.count <= 128)
      f(typename S::Half(), at, n0);
    else
      f(typename S::Full(), at, n0);
  }
}

// D = A B[g]^T (PT false) or dA = dD B[g] (PT true): workgroup `id`'s part
template <class T, class O, class S, bool PT>
__device__ __forceinline__ void rows_part(const GroupedParams& p, char* smem, int id) {
  using C = typename S::Full;
  const GroupSpot x = group_spot<S::kParts>(p, id, C::BM);
  if (x.spot.parts == 0) return;
  by_rows<S>(x.spot, x.at, x.spot.tn * C::BN, p.n, [&](auto c, const Place& at, int n0) {
    rows_tile<T, O, decltype(c), PT>(p, smem, at, n0);
  });
}
template <class T, class O, class S>
__global__ void __launch_bounds__(S::Full::T, 1) grouped_rows(const GroupedParams p) {
  __shared__ __attribute__((aligned(1024))) char smem[S::kLds];
  rows_part<T, O, S, false>(p, smem, blockIdx.x);
}

template <class C, bool GATHER>
struct WeightsSource {
  static constexpr int kAhead = GATHER ? C::NP : 0;
  typename std::conditional<GATHER, GatheredColumns<C::BN, C::NP>,
                            PlainColumns<C::BN, C::NP>>::type p;
  PlainColumns<C::BM, C::NQ> q;
  __device__ __forceinline__ void ahead(int kt) {
    if constexpr (GATHER) p.ahead(kt);
  }
  __device__ __forceinline__ void issue(int kt, int i, lds_c to) const {
    if (i < C::NP)
      p.issue(kt, i, to);
    else
      q.issue(kt, i - C::NP, to + C::P_BYTES);
  }
};

template <class T, class O, class C, bool GATHER>
__device__ __forceinline__ void weights_tile(const GroupedParams& p, char* smem, int g, int m0,
                                             int n0) {
  static_assert(C::BM % 128 == 0 && C::BN % 128 == 0, "swizzle of transposed tiles");
  if (m0 >= p.m || n0 >= p.n) return;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const Span s = span_of(p.offsets, g, p.places);
  WeightsSource<C, GATHER> src;
  if constexpr (GATHER)
    src.p.init(p.p, p.rows + s.begin, s.len, p.ldp, p.p_rows, n0, p.n, w, lane);
  else
    src.p.init((const T*)p.p + (int64_t)s.begin * p.ldp, s.len, p.ldp, n0, p.n, w, lane);
  src.q.init((const T*)p.q + (int64_t)s.begin * p.ldq, s.len, p.ldq, m0, p.m, w, lane);
  floatx4 acc[C::RM][C::RN];
  product<T, C, true, true>((lds_c)smem, (s.len + 63) / 64, src, acc, w, lane);
  store_tile<O, C, false>((O*)p.d + g * p.d_group + (int64_t)m0 * p.ldd, p.ldd, p.m - m0, n0, p.n,
                          acc, w, lane);
}

// dB[g] = sum over the group's places of dD^T A: workgroup `id`'s part
template <class T, class O, class W, bool GATHER>
__device__ __forceinline__ void weights_part(const GroupedParams& p, char* smem, int id) {
  using C = typename W::Full;
  // slots: tiles of one group's rows times groups
  const int per = p.slots / p.groups;
  // (each group's tiles to all XCDs: with a run of the whole launch to each,
  // groups of 492 to 1800 places took 203 us where equal ones take 146)
  const Spot x = spot_of<W::kParts>(id, p.slots, p.tiles_n, min(p.band, per), per * p.tiles_n);
  if (x.parts == 0) return;
  const int g = x.tm / per;
  const int m0 = (x.tm - g * per) * C::BM, n0 = x.tn * C::BN;
  if constexpr (W::kParts > 1) {
    if (x.parts == 4)
      return weights_tile<T, O, typename W::Corner, GATHER>(
          p, smem, g, m0 + (x.part >> 1) * W::Corner::BM, n0 + (x.part & 1) * W::Corner::BN);
    if (x.parts == 2)
      return weights_tile<T, O, typename W::Half, GATHER>(p, smem, g, m0 + x.part * W::Half::BM,
                                                          n0);
  }
  weights_tile<T, O, C, GATHER>(p, smem, g, m0, n0);
}

// Both gradients in one launch: the first `first` workgroups are dA's, the
// others dB's.
template <class T, class O, class S, class W, bool GATHER>
__global__ void __launch_bounds__(S::Full::T, 1) grouped_backward(const GroupedParams da,
                                                                  const GroupedParams db,
                                                                  int first) {
  static_assert((int)S::Full::T == (int)W::Full::T && S::kLds >= W::kLds, "one workgroup for both");
  __shared__ __attribute__((aligned(1024))) char smem[S::kLds];
  if ((int)blockIdx.x < first)
    rows_part<T, T, S, true>(da, smem, blockIdx.x);
  else
    weights_part<T, O, W, GATHER>(db, smem, blockIdx.x - first);
}

// ------------------------------------------------------------- few rows
// Tiles of 16 RM places by 16 RN columns for groups of few rows, where the
// weights' bytes are the work: no LDS stages, every fragment straight from
// memory.  The workgroup's eight waves share the contraction, U sub-steps of
// 32 a time (64 U consecutive bytes of each row per wave); their sums are
// added through LDS in the order of the waves.  One token's two experts, 2048 x
// 4096, 33.6 MB of weights: 8.9 us, of which the bytes alone take 6.6.
constexpr int kFewWaves = 8;
// sub-steps a time: two of those are in registers beside the sums
constexpr int few_depth(int rm, int rn) { return rm + rn > 3 ? 2 : 4; }

template <int RM, int RN>
struct FewTile {
  static constexpr int BM = 16 * RM, BN = 16 * RN, T = 64 * kFewWaves;
};

__device__ __forceinline__ att::Vec8<_Float16> as16(const u32x4_t& u, _Float16) {
  return __builtin_bit_cast(att::Vec8<_Float16>, u);
}
__device__ __forceinline__ att::Vec8<__bf16> as16(const u32x4_t& u, __bf16) {
  return __builtin_bit_cast(att::Vec8<__bf16>, u);
}

// The contraction from `from` to k (begun at another place by tiles of other
// weights, as RowsSource::start, by tiles of the same weights at the same).
// q_off: byte offsets of the lane's rows (kOutside: zeros); load_p(j, in, off):
// its 16 bytes of atom j's row at off, zeros without `in`.  After it
// sums[(i RN + j) * 64 + lane] holds the four values of atom (i, j).
template <class T, int RM, int RN, class LoadP>
__device__ __forceinline__ void few_product(__amdgpu_buffer_rsrc_t rq, const unsigned (&q_off)[RM],
                                            LoadP load_p, int from, int k, int begin,
                                            floatx4* sums, int w, int lane) {
  constexpr int U = few_depth(RM, RN), W = kFewWaves;
  floatx4 acc[RM][RN];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  struct Part {
    u32x4_t p[U][RN], q[U][RM];
  };
  auto load = [&](Part& x, int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = k0 + 32 * u + 8 * (lane >> 4) < k;
#pragma unroll
      for (int j = 0; j < RN; ++j)
        x.p[u][j] = load_p(j, in, 2 * k0 + 64 * u);
#pragma unroll
      for (int i = 0; i < RM; ++i)
        x.q[u][i] = __builtin_amdgcn_raw_buffer_load_b128(
            rq, in ? q_off[i] : kOutside, 2 * k0 + 64 * u, 0);
    }
  };
  auto use = [&](const Part& x) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j)
          acc[i][j] = Elem<T>::mma16(as16(x.p[u][j], T()), as16(x.q[u][i], T()), acc[i][j]);
  };
  // The waves take the pieces of 32 U in turn, from piece `begin` on and round;
  // two at a time, so that one is on its way while the other is used.
  Part a, b;
  const int pieces = (k - from + 32 * U - 1) / (32 * U);
  const int first = begin % max(pieces, 1);
  auto place = [&](int v) {
    const int c = v + first;
    return from + 32 * U * (c < pieces ? c : c - pieces);
  };
  int v = w;
  if (v < pieces) {
    load(a, place(v));
    for (; v + W < pieces; v += 2 * W) {
      load(b, place(v + W));
      use(a);
      if (v + 2 * W < pieces) load(a, place(v + 2 * W));
      use(b);
    }
    if (v < pieces) use(a);
  }
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) sums[((w * RM + i) * RN + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int x = threadIdx.x; x < RM * RN * 64; x += 64 * W) {
    floatx4 t = sums[x];
#pragma unroll
    for (int v = 1; v < W; ++v) t += sums[v * RM * RN * 64 + x];
    sums[x] = t;
  }
}

// byte offsets of the lane's rows of Q
template <class T, int RM>
__device__ __forceinline__ void few_rows(const GroupedParams& p, const Place& at, int lane,
                                         unsigned (&off)[RM]) {
  const unsigned c = 16u * (lane >> 4);
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int row = 16 * i + (lane & 15);
    if (p.rows) {
      const int a = p.rows[at.first + min(row, at.count - 1)];
      off[i] = row < at.count && (unsigned)a < (unsigned)p.q_rows
                   ? 2u * (unsigned)a * p.ldq + c : kOutside;
    } else {
      off[i] = row < at.count ? 2u * row * p.ldq + c : kOutside;
    }
  }
}
// Q of a tile, as few_rows counts it
template <class T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t few_base(const GroupedParams& p,
                                                           const Place& at) {
  return buffer((const T*)p.q + (p.rows ? 0 : (int64_t)at.first * p.ldq), kWhole);
}

// the tile's places against columns n0 .. of the matrix P
template <class T, int RM, int RN>
__device__ __forceinline__ void few_tile(const GroupedParams& p, const Place& at, int n0,
                                         const T* P, int from, int k, floatx4* sums, int w,
                                         int lane) {
  const int r = lane & 15;
  const unsigned c = 16u * (lane >> 4);
  unsigned q_off[RM], p_off[RN];
  few_rows<T, RM>(p, at, lane, q_off);
#pragma unroll
  for (int j = 0; j < RN; ++j)
    p_off[j] = n0 + 16 * j + r < p.n ? 2u * (16 * j + r) * p.ldp + c : kOutside;
  const __amdgpu_buffer_rsrc_t rp = buffer(P + (int64_t)n0 * p.ldp, kWhole);
  few_product<T, RM, RN>(
      few_base<T>(p, at), q_off,
      [&](int j, bool in, int off) {
        return __builtin_amdgcn_raw_buffer_load_b128(rp, in ? p_off[j] : kOutside, off, 0);
      },
      from, k, n0 / (16 * RN) + 3 * at.group, sums, w, lane);
}

// D = A B[g]^T, groups of few rows
template <class T, class O, int RM, int RN>
__global__ void __launch_bounds__(64 * kFewWaves, 1) grouped_few(const GroupedParams p) {
  using F = FewTile<RM, RN>;
  __shared__ floatx4 sums[kFewWaves * RM * RN * 64];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const GroupSpot s = group_spot<1>(p, blockIdx.x, F::BM);
  if (s.spot.parts == 0 || s.at.group == p.groups) return;
  const Place at = s.at;
  const int n0 = s.spot.tn * F::BN;
  few_tile<T, RM, RN>(p, at, n0, (const T*)p.p + at.group * p.p_group, 0, p.k, sums, w, lane);
  // (a thread stores what it added itself)
  for (int x = tid; x < RM * RN * 64; x += F::T) {
    const int l = x & 63, j = (x >> 6) % RN, i = (x >> 6) / RN;
    const int m = 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m < at.count && n < p.n)
      Out<O>::store4((O*)p.d + (int64_t)(at.first + m) * p.ldd + n, sums[x]);
  }
}

}  // namespace grp
}  // namespace mfl
