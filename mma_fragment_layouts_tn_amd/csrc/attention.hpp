// Attention kernels: the chain's two products with the softmax between them.
//
// Row r of a kv head's rows is (token r / G, query head kv * G + r % G): the G
// query heads of a group are rows of one product, so a tile of rows reads
// each key and value once for the whole group, and a single token fills G
// rows instead of one.
//
//   forward   S^T = K Q^T, P = exp2(c S - m), O^T = V^T P^T
//
// As in the chain the first product is issued transposed: lane l's
// accumulators hold the scores of row l % 32, so maximum, exponent and sum of
// a row are in-lane work plus one exchange between the two halves of the
// wave, and the weights are the second product's operand as they are.  Value
// i of an accumulator is key 8 (i / 4) + 4 (l / 32) + i % 4: two runs of four
// consecutive keys per 16-wide K chunk, which is what two transposing LDS
// reads of V deliver, so neither operand is permuted in memory.  The second
// product is transposed too (its columns are the rows of Q): rescaling O by a
// new maximum is one factor per lane.
#pragma once

#include <hip/hip_runtime.h>

#include "gemm_tile.hpp"

namespace mfl {
namespace att {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef short shortx8 __attribute__((ext_vector_type(8)));
using lds_t = __attribute__((address_space(3))) void*;
using lds_s4 = __attribute__((address_space(3))) shortx4*;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A row's reference maximum follows its running maximum only once that is
// 2^kSlack ahead: weights stay below 2^8, the accumulators need no rescaling
// in most steps, and the quotient at the end is the same.
constexpr float kSlack = 8.0f;

template <class T>
struct Elem;
template <>
struct Elem<_Float16> {
  typedef _Float16 vec8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ floatx16 mma(vec8 a, vec8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ floatx4 mma16(vec8 a, vec8 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  // The sum tied to accumulation registers (mma_tied) or to ordinary ones
  // (mma_begin from zero, mma_add): the compiler keeps the results of its own
  // matrix instructions all in the one kind or all in the other.  It does not
  // see these instructions' wait states; the kernels that use them say how
  // they are kept.
  static __device__ __forceinline__ void mma_begin(vec8 a, vec8 b, floatx16& c) {
    asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ void mma_add(vec8 a, vec8 b, floatx16& c) {
    asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ void mma_tied(vec8 a, vec8 b, floatx16& c) {
    asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0"
                 : "+a"(c)
                 : "v"(a), "v"(b));
  }
};
template <>
struct Elem<__bf16> {
  typedef __bf16 vec8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ floatx16 mma(vec8 a, vec8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ floatx4 mma16(vec8 a, vec8 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // The sum tied to accumulation registers (mma_tied) or to ordinary ones
  // (mma_begin from zero, mma_add): the compiler keeps the results of its own
  // matrix instructions all in the one kind or all in the other.  It does not
  // see these instructions' wait states; the kernels that use them say how
  // they are kept.
  static __device__ __forceinline__ void mma_begin(vec8 a, vec8 b, floatx16& c) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ void mma_add(vec8 a, vec8 b, floatx16& c) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ void mma_tied(vec8 a, vec8 b, floatx16& c) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0"
                 : "+a"(c)
                 : "v"(a), "v"(b));
  }
};
template <class T>
using Vec8 = typename Elem<T>::vec8;

// Between the last matrix instruction of a loop and the first use of its
// sums: the wait states that the compiler does not see for tied sums, nor
// always across blocks for others.
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// One launch of the forward kernels.  Sequence s of `batch` owns query tokens
// [seq_q[s], seq_q[s+1]) (or q_len tokens each, from s * q_len, when seq_q is
// null) and keys: [seq_k[s], seq_k[s+1]) of the packed keys, or lengths[s]
// keys of cache s (k_batch, v_batch elements apart), or all total_k keys.
// Token n's address is (n / q_inner) * q_batch + (n % q_inner) * q_tok.
struct FwdParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;                 // (tokens, heads) or null
  float* part_o;              // splits x rows x DC, null: one split, out written
  float2* part_ml;            // splits x rows
  const int* seq_q;
  const int* seq_k;
  const int* lengths;
  int batch, q_len, total_q, total_k;
  int q_inner;
  int heads_kv, group, dim, causal;
  int splits, split0, slots;  // key splits of this launch, index of the first
  int part_keys;              // a tile takes a split per part_keys keys (0: all of them)
  int64_t rows;               // tokens * heads: the rows of one split
  int64_t q_batch, q_tok, q_head, k_batch, k_tok, k_head, v_batch, v_tok, v_head;
  int64_t o_batch, o_tok, o_head;
  float scale_log2;           // scale * log2(e) > 0
};

struct CombineParams {
  const float* part_o;
  const float2* part_ml;
  void* o;
  float* lse;
  int64_t rows;
  int splits, dim, heads, q_inner;
  int64_t o_batch, o_tok, o_head;
};

// The tile that a share cut off at its end: first key, keys (0: none), the
// last share that it went on in, its number (attention_dkv).
struct DkvCut {
  int key, keys, last, number;
};

struct BwdParams {
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;
  float* stats;               // 2 x heads x tokens: lse * log2(e), then rowsum(dout * out)
  void* dq;
  void* dk;
  void* dv;
  const int* seq_q;
  const int* seq_k;
  int batch, total_q, total_k;
  int heads_kv, group, dim, causal, slots_q, slots_k;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head, do_tok, do_head;
  int64_t dq_tok, dq_head, dk_tok, dk_head, dv_tok, dv_head;
  float scale, scale_log2;
  // dK, dV: workgroups per kv head, 0: one per tile; sums of the tiles cut, a
  // place per part and kv head (dkv_place), dK then dV of the keys of a tile
  int shares, by_tile;
  DkvCut* cuts;               // one per share
  float* partials;
};

// ------------------------------------------------------------- LDS tiles
// Rows of DC elements, 16-byte chunk c of row r stored at chunk c ^ swz(r).
// Straight reads (one chunk of 16 consecutive rows) and transposing reads (4
// consecutive chunks of 4 rows, or 2 chunks of 8 rows, consecutive ones) all
// spread over the banks: swz differs over 16 rows (DC = 64, two rows per pass
// of the banks: over 8 pairs of rows), over 4 rows already in its upper bits,
// over 8 rows in all but the lowest.
template <int DC>
MFL_HD constexpr int swz_row(int r) {
  return (DC >= 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2) | ((r >> 2) & 1) << 1 | ((r >> 3) & 1);
}
template <int DC>
MFL_HD constexpr int tile_off(int r, int d) {
  return r * DC + (((d >> 3) ^ swz_row<DC>(r)) << 3) + (d & 7);
}
template <int DC>
constexpr bool swizzle_spreads() {
  const int row_groups = DC / 8 < 16 ? DC / 8 : 16;     // 16-byte groups of a row within 256 bytes
  const int per_pass = 16 / row_groups;                 // rows per 256 bytes
  for (int base = 0; base < 64; base += 16) {
    unsigned seen = 0;
    for (int i = 0; i < 16; ++i) {
      const int r = base + i;
      seen |= 1u << (((r % per_pass) * row_groups + ((0 ^ swz_row<DC>(r)) % row_groups)) & 15);
    }
    if (seen != 0xffffu) return false;
  }
  for (int r0 = 0; r0 < 64; r0 += 4) {
    unsigned seen = 0;
    for (int i = 0; i < 16; ++i) {
      const int r = r0 + i / 4;
      seen |= 1u << (((r % per_pass) * row_groups + (((i % 4) ^ swz_row<DC>(r)) % row_groups)) & 15);
    }
    if (seen != 0xffffu) return false;
  }
  for (int r0 = 0; r0 < 64; r0 += 8) {
    unsigned seen = 0;
    for (int i = 0; i < 16; ++i) {
      const int r = r0 + i / 2;
      seen |= 1u << (((r % per_pass) * row_groups + (((i % 2) ^ swz_row<DC>(r)) % row_groups)) & 15);
    }
    if (seen != 0xffffu) return false;
  }
  return true;
}
static_assert(swizzle_spreads<64>() && swizzle_spreads<128>() && swizzle_spreads<256>(),
              "both kinds of LDS reads must touch every bank group once");

template <bool B>
struct BoolC {
  static constexpr bool value = B;
};

template <class T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p, 16), 16);
  return v;
}

// A lane's place in a stage for both kinds of fragment reads, as LDS byte
// addresses.  Tiles start at multiples of 4 KiB, so the address of another
// chunk is the address of the first one XOR a constant, and other rows (32
// and 16 further, where the swizzle is the same) are constant offsets: two
// registers serve every read of a stage.
//
// The compiler lets a transposing read wait for every direct-to-LDS load in
// flight unless it can tell them apart, which would take away the loads'
// lead.  The kernels' steps are therefore functions of two restricted
// pointers, to the stage they read (`stage` here) and to the ring they fill,
// and every such read is addressed from the first.  What orders a read behind the
// loads it needs is its address, which at() forms behind the wait.
using lds_c = __attribute__((address_space(3))) char*;
template <class T, int DC>
struct Reader {
  unsigned s, t;
  lds_c stage;
  // straight: row l % 32, d = 8 (l / 32)
  // transposed: of each 16 lanes, lane i supplies 4 elements of key i / 4
  static __device__ __forceinline__ Reader of(int lane) {
    const int i = lane & 15, blk = lane >> 4;
    return Reader{2u * tile_off<DC>(lane & 31, 8 * (lane >> 5)),
                  2u * tile_off<DC>(4 * (blk >> 1) + (i >> 2), 16 * (blk & 1) + 4 * (i & 3)),
                  nullptr};
  }
  // in the stage at `base`, `more` bytes on; opaque, so that the addresses
  // below are formed where they are used instead of held in registers
  __device__ __forceinline__ Reader at(lds_c base, unsigned more = 0) const {
    const unsigned b = (unsigned)(uintptr_t)base + more;
    Reader r{s + b, t + b, base};
    asm volatile("" : "+v"(r.s), "+v"(r.t));
    return r;
  }
  // operand fragment of rows 32 b .. 32 b + 31, K chunk kk, `more` bytes on
  __device__ __forceinline__ Vec8<T> straight(int b, int kk, int more = 0) const {
    using ptr = const __attribute__((address_space(3))) Vec8<T>*;
    return *(ptr)((s ^ (32u * kk)) + 64 * b * DC + more);
  }
  // transposed: rows d = 32 db + l % 32; values the keys
  // 16 kc + 4 (l / 32) + 0..3 and 8 further
  __device__ __forceinline__ Vec8<T> transposed(int kc, int db, int more = 0) const {
    const unsigned x = t ^ (64u * db);
    const shortx4 lo = read_tr(x + 32 * kc * DC + more);
    const shortx4 hi = read_tr((x ^ 16u) + 32 * kc * DC + 16 * DC + more);
    return __builtin_bit_cast(Vec8<T>, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  __device__ __forceinline__ shortx4 read_tr(unsigned address) const {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)in_stage(address));
  }
  __device__ __forceinline__ lds_c in_stage(unsigned address) const {
    return stage + (int)(address - (unsigned)(uintptr_t)stage);
  }
};
// what Reader takes for granted of the tile's layout
template <int DC>
constexpr bool reader_addresses_hold() {
  for (int r = 0; r < 32; ++r)
    for (int kk = 0; kk < DC / 16; ++kk)
      for (int h = 0; h < 2; ++h)
        if (tile_off<DC>(r + 32, 16 * kk + 8 * h) !=
            (tile_off<DC>(r, 8 * h) ^ (16 * kk)) + 32 * DC)
          return false;
  for (int r = 0; r < 8; ++r)
    for (int d = 0; d < 32; d += 4)
      for (int db = 0; db < DC / 32; ++db) {
        const int x = tile_off<DC>(r, d) ^ (32 * db);
        if (tile_off<DC>(16 + r, 32 * db + d) != x + 16 * DC ||
            tile_off<DC>(16 + r + 8, 32 * db + d) != (x ^ 8) + 24 * DC)
          return false;
      }
  return true;
}
static_assert(reader_addresses_hold<64>() && reader_addresses_hold<128>() &&
                  reader_addresses_hold<256>(),
              "chunks by XOR, rows by offset");

// LDS reads of this wave done, then the workgroup barrier
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// at most VM vector-memory operations of this wave in flight
template <int VM>
__device__ __forceinline__ void wait_vm() {
  static_assert(VM >= 0 && VM < 64, "vmcnt has 6 bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (((VM >> 4) & 3) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
}

// maximum and sum over lanes l and l ^ 32: the exchange leaves the lower
// half's value in one register of every lane, the upper half's in the other
struct Halves {
  float lower, upper;
};
__device__ __forceinline__ Halves halves(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned a = r[0], b = r[1];   // (a bit cast of r[i] itself reads element 0)
  return Halves{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
// the same over rows of 16 lanes: 0 and 1, 2 and 3
__device__ __forceinline__ Halves quarters(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned a = r[0], b = r[1];
  return Halves{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ float both_max(float x) {
  const Halves h = halves(x);
  return fmaxf(h.lower, h.upper);
}
__device__ __forceinline__ float both_sum(float x) {
  const Halves h = halves(x);
  return h.lower + h.upper;
}
__device__ __forceinline__ float all4_max(float x) {   // lanes l, l ^ 16, l ^ 32, l ^ 48
  const Halves h = quarters(both_max(x));
  return fmaxf(h.lower, h.upper);
}
__device__ __forceinline__ float all4_sum(float x) {
  const Halves h = quarters(both_sum(x));
  return h.lower + h.upper;
}
// x, but not for the optimiser: a first step told apart by it stays a branch
// in the loop's body (a copy of the body for it would hide from the compiler
// that its loads and the other steps' reads are apart)
__device__ __forceinline__ int hidden(int x) {
  asm volatile("" : "+s"(x));
  return x;
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// ---------------------------------------------------- tiles of sequences
// Tiles of BM rows, none across two sequences, without a table: sequence s
// takes the slots from first(s) = start(s) / BM + s on.  floor(b) - floor(a) + 1
// >= ceil(b - a), so every sequence finds room, first() grows strictly, and
// a slot's sequence is found by comparing 64 candidates at a time.
template <class F>
__device__ __forceinline__ int find_sequence(int batch, int slot, F first) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, at = lo + lane * step;
    const bool ok = at < hi && first(at) <= slot;
    const int n = max(1, (int)__popcll(__ballot(ok)));
    lo = uniform(lo + (n - 1) * step);
    hi = min(lo + step, hi);
  }
  return lo;
}

struct Span {
  int begin, len;
};
// sequence s of the offsets, held inside [0, total] whatever they are
__device__ __forceinline__ Span span_of(const int* seq, int s, int total) {
  const int a = min(max(seq[s], 0), total), b = min(max(seq[s + 1], 0), total);
  return Span{uniform(a), uniform(max(b - a, 0))};
}

struct Place {
  int q0, lq, lk, tile;     // first token and count, keys, tile within the sequence
  int64_t k_off, v_off;     // element offsets of key 0
  bool any;                 // the slot holds a tile
};

__device__ __forceinline__ Place place_of(const FwdParams& p, int slot, int bm) {
  Place r;
  int s, first;
  if (p.seq_q) {
    auto f = [&](int i) {
      return (int)((int64_t)min(max(p.seq_q[i], 0), p.total_q) * p.group / bm) + i;
    };
    s = find_sequence(p.batch, slot, f);
    const Span q = span_of(p.seq_q, s, p.total_q);
    r.q0 = q.begin;
    r.lq = q.len;
    first = uniform(f(s));
  } else {
    const int per = (int)(((int64_t)p.q_len * p.group + bm - 1) / bm);
    s = slot / per;
    first = s * per;
    r.q0 = s * p.q_len;
    r.lq = s < p.batch ? p.q_len : 0;
    s = min(s, p.batch - 1);
  }
  r.tile = slot - first;
  r.any = r.tile >= 0 && (int64_t)r.tile * bm < (int64_t)r.lq * p.group;
  if (p.seq_k) {
    const Span k = span_of(p.seq_k, s, p.total_k);
    r.lk = k.len;
    r.k_off = (int64_t)k.begin * p.k_tok;
    r.v_off = (int64_t)k.begin * p.v_tok;
  } else {
    r.lk = p.lengths ? uniform(min(max(p.lengths[s], 0), p.total_k)) : p.total_k;
    r.k_off = (int64_t)s * p.k_batch;
    r.v_off = (int64_t)s * p.v_batch;
  }
  return r;
}

// keys that the tile's last row sees; the splits they take; whether those go
// to the workspace
__device__ __forceinline__ int seen_of(const FwdParams& p, const Place& at, int bm) {
  const int last = min((int)(((int64_t)at.tile * bm + bm - 1) / p.group), at.lq - 1);
  return uniform(max(p.causal ? min(last + at.lk - at.lq, at.lk - 1) + 1 : at.lk, 0));
}
__device__ __forceinline__ int parts_of(const FwdParams& p, int seen) {
  if (p.part_keys == 0) return p.splits;
  return uniform(min(max((seen + p.part_keys - 1) / p.part_keys, 1), p.splits));
}
__device__ __forceinline__ bool to_parts(const FwdParams& p, int parts) {
  return p.part_o && (p.part_keys == 0 || parts > 1);
}

// ------------------------------------------------ direct-to-LDS staging
// One wave instruction fills 1024 consecutive LDS bytes; each lane fetches
// the 16 bytes its place stands for.  Buffer loads: a tile's rows past the
// sequence's end and columns past the head dimension are out of the buffer's
// range, and the hardware stores zeros for them, so every load of every tile
// is one instruction on a descriptor made once per tile and a 32-bit offset
// per lane that never changes.  (Addresses formed per lane, with a choice
// between the tensor and a block of zeros, cost a fifth of the gradients'
// step in vector instructions.)  Loads move at most 64 bytes a clock into
// LDS, and a wave that issues several in a row stands still meanwhile: the
// kernels issue them one by one between matrix instructions.
constexpr int kMaxTokenStride = 1 << 23;   // elements: 64 rows stay within 2^30 bytes

template <class T, int DC>
struct Fetch {
  static constexpr int ROWS = 512 / DC;   // tile rows per instruction
  __amdgpu_buffer_rsrc_t r;
  // the tile's rows `row0` .. of `end` rows at `base`
  static __device__ __forceinline__ Fetch of(const T* base, int64_t stride, int row0, int end,
                                             int dim) {
    return at(base + (int64_t)row0 * stride, stride, end - row0, dim);
  }
  // `rows` rows (any number) from `row` on
  static __device__ __forceinline__ Fetch at(const T* row, int64_t stride, int rows, int dim) {
    const int bytes = rows > 0 ? 2 * ((min(rows, 64) - 1) * (int)stride + dim) : 0;
    return Fetch{__builtin_amdgcn_make_buffer_rsrc((void*)row, 0, bytes, 0x00027000)};
  }
  // instruction i of the tile
  __device__ __forceinline__ void issue(int64_t stride, int dim, lds_c tile, int i,
                                        int lane) const {
    const int row = (8 * lane) / DC, c = ((8 * lane) % DC) / 8;
    const int col = 8 * (c ^ swz_row<DC>(row) ^ swz_row<DC>(i * ROWS));
    const unsigned off = col < dim ? 2u * (row * (int)stride + col) : 0x80000000u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_t)(tile + i * 1024), 16, off,
                                             2 * i * ROWS * (int)stride, 0, 0);
  }
};
// the swizzle of a sum of rows without common bits
template <int DC>
constexpr bool swizzle_is_linear() {
  for (int r = 0; r < 64; ++r)
    for (int i = 512 / DC; i < 64; i += 512 / DC)
      if (r < 512 / DC && swz_row<DC>(i + r) != (swz_row<DC>(i) ^ swz_row<DC>(r))) return false;
  return true;
}
static_assert(swizzle_is_linear<64>() && swizzle_is_linear<128>() && swizzle_is_linear<256>(),
              "a lane's column of another instruction by XOR");
// 8 values of a row from the two halves of the wave: value i of block x is
// d = 8 (i / 4) + 4 (l / 32) + i % 4; after the exchange lane l holds
// d = 8 (q + l / 32) + 0..7 of the pair of groups q, q + 1
template <class T>
__device__ __forceinline__ uint4 gather8(const floatx16& x, int q, float f) {
  typedef T vec4 __attribute__((ext_vector_type(4)));
  union {
    vec4 v;
    unsigned u[2];
  } a, b;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a.v[e] = (T)(x[4 * q + e] * f);
    b.v[e] = (T)(x[4 * (q + 1) + e] * f);
  }
  const auto s0 = __builtin_amdgcn_permlane32_swap(a.u[0], b.u[0], false, false);
  const auto s1 = __builtin_amdgcn_permlane32_swap(a.u[1], b.u[1], false, false);
  return make_uint4(s0[0], s1[0], s0[1], s1[1]);
}

// the transposed accumulators of one row per lane, times f, as row elements
template <class T, int DC>
__device__ __forceinline__ void store_row(T* row, const floatx16 (&acc)[DC / 32], float f, int dim,
                                          int lane, bool valid) {
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const uint4 u = gather8<T>(acc[db], q, f);
      const int d = 32 * db + 8 * (q + (lane >> 5));
      if (valid && d < dim) *(uint4*)(row + d) = u;
    }
}

template <int N>
__device__ __forceinline__ void zero(floatx16 (&a)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) a[j][i] = 0.0f;
}

// 8 weights of a 32-key block, K chunk c (0, 1), as an operand fragment
template <class T>
__device__ __forceinline__ Vec8<T> pack8(const floatx16& s, int c) {
  Vec8<T> r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = (T)s[8 * c + e];
  return r;
}

// A wave's rows: lane l and lane l ^ 32 hold row l % 32 of the 32 from `row0`
// on; rows past the last repeat it and are not stored.
struct RowOf {
  int head, n;        // query head, token
  int limit;          // last visible key
  bool valid;
};
__device__ __forceinline__ RowOf row_of(int r, int lq, int lk, int group, int kvh, int q0,
                                        int causal) {
  const int last = lq * group - 1, c = min(r, last);
  const int t = c / group;
  RowOf x;
  x.valid = r <= last;
  x.n = q0 + t;
  x.head = kvh * group + (c - t * group);
  x.limit = causal ? min(t + lk - lq, lk - 1) : lk - 1;
  return x;
}

// Running softmax of the lane's row over the scores in st: the reference that
// the weights are formed with (in units of log2), after updating the maximum m
// and, if it grew by more than the slack, the lane's share l of the sum and
// the accumulators.
template <int NB, int ND>
__device__ __forceinline__ float new_reference(const floatx16 (&st)[NB], floatx16 (&acc)[ND],
                                               float& m, float& l, float c) {
  float top = -INFINITY;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, st[b][i]);
  top = both_max(top) * c;
  if (__any(top - m > kSlack)) {       // m = -inf at first: inf > slack, or nan for no key
    const float to = fmaxf(m, top);
    const float f = __builtin_amdgcn_exp2f(m - (to == -INFINITY ? 0.0f : to));
    l *= f;
#pragma unroll
    for (int j = 0; j < ND; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][i] *= f;
    m = to;
  }
  return m == -INFINITY ? 0.0f : m;
}

// bits 0 .. n - 1 (none for n <= 0, all for n > 31)
__device__ __forceinline__ unsigned low_bits(int n) {
  return n > 31 ? ~0u : n > 0 ? (1u << n) - 1u : 0u;
}
// all bits of x where bit r of the mask is set, else those of y
__device__ __forceinline__ float select_bit(unsigned mask, int r, float x, float y) {
  unsigned m = (unsigned)__builtin_amdgcn_sbfe((int)mask, r, 1);
  asm("" : "+v"(m));   // two instructions, not a test and a choice
  return __builtin_bit_cast(float, (m & __builtin_bit_cast(unsigned, x)) |
                                       (~m & __builtin_bit_cast(unsigned, y)));
}
// keys past the row's limit get -inf
template <int NB>
__device__ __forceinline__ void mask_keys(floatx16 (&st)[NB], int key0, int limit, int lane) {
  const int room = limit - key0 - 4 * (lane >> 5);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const unsigned seen = low_bits(room + 1 - 32 * b);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      st[b][i] = select_bit(seen, 8 * (i / 4) + i % 4, st[b][i], -INFINITY);
  }
}

// ------------------------------------------------------ forward, tall
// Four waves of 32 rows each over chunks of 64 keys staged in a ring of NST
// LDS stages (K and V of a chunk together), shared by the workgroup: 64 KB, so
// that two workgroups fit a CU up to 128 columns.  Eight waves in one
// workgroup per CU took 1 - 6 % longer on long prompts and 30 % on 2048 tokens
// (62 against 49 us).
//
// Bound by matrix and vector instructions that take turns: 8192 causal tokens,
// 32/8 heads of 128, fp16, take 556 us (989 TFLOP/s; a large library product
// reaches 1,500).  The matrix pipe is busy for 58 % of the cycles, vector
// instructions are issued in 52 %, both at once in 20 %.  The maximum over a
// chunk and the first half of its weights run with no matrix instruction of
// the wave in flight, and the second wave of the SIMD fills only some of it.
// With loads, LDS reads, exponentials and maxima all taken out 419 us of 568
// were left (one device).  Scores formed one chunk ahead of their weights, so
// that a wave's own matrix instructions cover its softmax, took 2 % longer
// (the copies of the scores, one product more per tile); raised wave priority
// around the products, 4 slots of lead and alternating sums changed nothing.
template <int DC>
MFL_HD constexpr int tall_stages() {
  return DC == 64 ? 4 : 2;
}

template <class T, int DC>
__device__ __forceinline__ void tall_rows(const FwdParams& p, T* smem, int bid) {
  constexpr int W = 4, BM = 32 * W, CK = 64, NST = tall_stages<DC>(), KS = DC / 16, ND = DC / 32;
  constexpr int TILE = CK * DC, NI = TILE / 512 / W;   // elements, loads per matrix and wave
  static_assert(NI >= 1, "loads");
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int kvh = bid % p.heads_kv;
  bid /= p.heads_kv;
  // last splits first (only the longest tiles have them; between the others'
  // workgroups the empty ones would leave shader engines idle), last rows
  // first (with a causal mask the longest)
  const int split = p.splits - 1 - bid / p.slots, slot = p.slots - 1 - bid % p.slots;
  const Place at = place_of(p, slot, BM);
  if (!at.any) return;
  const int seen = seen_of(p, at, BM), parts = parts_of(p, seen);
  if (split >= parts) return;

  const RowOf row = row_of(at.tile * BM + 32 * w + (lane & 31), at.lq, at.lk, p.group, kvh, at.q0,
                           p.causal);
  const int chunks = (seen + CK - 1) / CK;
  const int c0 = (int)((int64_t)chunks * split / parts);
  const int c1 = (int)((int64_t)chunks * (split + 1) / parts);
  // chunks before `cut` hide nothing from any of the wave's rows
  const int cut = min(max((uniform(row.limit) + 1) / CK, c0), c1);

  const T* K = (const T*)p.k + at.k_off + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + at.v_off + (int64_t)kvh * p.v_head;
  const lds_c ring = (lds_c)smem;
  auto stage_of = [&](int c) { return (c - c0) % NST * 4 * TILE; };
  // load j of chunk c: K, then V
  struct Next {
    Fetch<T, DC> k, v;
  };
  auto next_chunk = [&](int c) {
    const int end = c < c1 ? at.lk : 0;
    return Next{Fetch<T, DC>::of(K, p.k_tok, c * CK, end, p.dim),
                Fetch<T, DC>::of(V, p.v_tok, c * CK, end, p.dim)};
  };
  auto issue = [&](const Next& n, lds_c to, int j) {
    if (j < NI)
      n.k.issue(p.k_tok, p.dim, to, w * NI + j, lane);
    else
      n.v.issue(p.v_tok, p.dim, to + 2 * TILE, w * NI + j - NI, lane);
  };

  const int64_t qn = (int64_t)(row.n / p.q_inner) * p.q_batch + (row.n % p.q_inner) * p.q_tok;
  const T* Q = (const T*)p.q + qn + row.head * p.q_head;
  Vec8<T> qf[KS];
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    const int d = 16 * kk + 8 * (lane >> 5);
    if (d < p.dim)
      qf[kk] = load8(Q + d);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[kk][e] = (T)0.0f;
  }
  floatx16 acc[ND];
  zero(acc);
  float m = -INFINITY, l = 0.0f;
  const Reader<T, DC> reader = Reader<T, DC>::of(lane);
  // chunk c, while chunk c + NST - 1 is fetched; `to` is the whole ring.
  // Every step issues 2 NI loads (of nothing past the last chunk), so what is
  // in flight is known by count.
  auto step = [&](int c, lds_c __restrict__ from, lds_c __restrict__ to, auto masked) {
    if (c == hidden(c0)) {
#pragma unroll
      for (int s = 0; s < NST - 1; ++s) {
        const Next nx = next_chunk(c0 + s);
#pragma unroll
        for (int j = 0; j < 2 * NI; ++j) issue(nx, to + 4 * s * TILE, j);
      }
    }
    // chunk c has landed here, and after the barrier everywhere; its
    // predecessor's stage is free
    wait_vm<(NST - 2) * 2 * NI>();
    barrier();
    const Next nx = next_chunk(c + NST - 1);
    const lds_c fill = to + stage_of(c + NST - 1);
    const int key0 = c * CK;
    const Reader<T, DC> rd = reader.at(from);
    // 2 KS slots of one matrix instruction each for S, as many for O, pinned
    // in this order: fragments are read RA slots ahead (left to itself the
    // compiler reads each just before its use), the next chunk's loads are
    // spread out, and the weights of keys 32 - 63 are formed under the first
    // half of O.
    constexpr int RA = 2, N = 4 * KS;
    Vec8<T> fr[RA + 1], pf[4];
    auto read = [&](int n) {
      if (n >= N) return;
      Vec8<T>& f = fr[n % (RA + 1)];
      if (n < 2 * KS)
        f = rd.straight(n / KS, n % KS);
      else
        f = rd.transposed((n - 2 * KS) / ND, n % ND, 2 * TILE);
    };
    auto load_at = [&](int n) {
#pragma unroll
      for (int j = 0; j < 2 * NI; ++j)
        if ((2 * j + 1) * N / (8 * NI) == n) issue(nx, fill, j);
      __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int n = 0; n < RA; ++n) read(n);
    floatx16 st[2];
    zero(st);
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n) {
      read(n + RA);
      st[n / KS] = Elem<T>::mma(fr[n % (RA + 1)], qf[n % KS], st[n / KS]);
      load_at(n);
    }
    if constexpr (decltype(masked)::value) mask_keys(st, key0, row.limit, lane);
    const float ref = new_reference(st, acc, m, l, p.scale_log2);
    float sum = 0.0f;
    auto weight = [&](int v) {
      const float w_ =
          __builtin_amdgcn_exp2f(__builtin_fmaf(st[v / 16][v % 16], p.scale_log2, -ref));
      st[v / 16][v % 16] = w_;
      sum += w_;
      if (v % 8 == 7) pf[v / 8] = pack8<T>(st[v / 16], v / 8 % 2);
    };
#pragma unroll
    for (int v = 0; v < 16; ++v) weight(v);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 2 * KS; n < N; ++n) {
      const int k = n - 2 * KS;
      read(n + RA);
      acc[k % ND] = Elem<T>::mma(fr[n % (RA + 1)], pf[k / ND], acc[k % ND]);
      if (k < KS)
#pragma unroll
        for (int v = 16 + 16 * k / KS; v < 16 + 16 * (k + 1) / KS; ++v) weight(v);
      load_at(n);
    }
    l += sum;
  };
  int c = c0;
  if (c < cut) {
    do step(c, ring + stage_of(c), ring, BoolC<false>{});
    while (++c < cut);
    settle();
  }
  if (c < c1) {
    do step(c, ring + stage_of(c), ring, BoolC<true>{});
    while (++c < c1);
    settle();
  }
  wait_vm<0>();

  l = both_sum(l);
  const int64_t out_row = (int64_t)row.n * (p.heads_kv * p.group) + row.head;
  if (to_parts(p, parts)) {
    const int64_t at_row = (int64_t)(p.split0 + split) * p.rows + out_row;
    if (row.valid && lane < 32) p.part_ml[at_row] = make_float2(m, l);
    if (row.valid && l != 0.0f) {
      float* po = p.part_o + at_row * DC + 4 * (lane >> 5);
#pragma unroll
      for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(floatx4*)(po + 32 * db + 8 * q) = floatx4{acc[db][4 * q], acc[db][4 * q + 1],
                                                      acc[db][4 * q + 2], acc[db][4 * q + 3]};
    }
    return;
  }
  const int64_t on = (int64_t)(row.n / p.q_inner) * p.o_batch + (row.n % p.q_inner) * p.o_tok;
  store_row<T, DC>((T*)p.o + on + row.head * p.o_head, acc, l == 0.0f ? 0.0f : 1.0f / l, p.dim,
                   lane, row.valid);
  if (p.lse && row.valid && lane < 32)
    p.lse[out_row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <class T, int DC>
__global__ void __launch_bounds__(256, DC == 256 ? 1 : 2) attention_tall(const FwdParams p) {
  static_assert(4 * tall_stages<DC>() * 64 * DC <= 160 * 1024, "staging");
  __shared__ __attribute__((aligned(4096))) T smem[tall_stages<DC>() * 2 * 64 * DC];
  tall_rows<T, DC>(p, smem, blockIdx.x);
}

// ------------------------------------------------------ forward, flat
// Few rows, long keys: 16 rows per workgroup (v_mfma 16x16x32: a decoding
// step's rows, a group of heads times the new tokens, rarely fill more), whose
// 4 waves take turns over chunks of 32 keys.  Each wave has a buffer of its
// own for the K and the V of one chunk; the next K is fetched as soon as the
// scores are formed, the next V after the second product, so a wave always has
// half a chunk in flight, no wave waits for another before the end, and two
// workgroups fit a CU (DC <= 128).  The W partial rows are joined in LDS.
// Bound by latency at few keys, by memory at many: one token of 32/8 heads of
// 128 against 8192 keys takes 6.9 us in 32 parts (7.9 in 16) and 4.4 - 6.8 to
// join them.
//
// Lane l holds row l % 16; value v of the scores of keys 16 b .. 16 b + 15 is
// key 16 b + 4 (l / 16) + v.  The second product's operand takes the values of
// both 16-key blocks: per lane two runs of 4 keys, as two transposing reads
// deliver V.
constexpr int kFlatWaves = 4;
template <class T, int DC>
constexpr int flat_elems() {            // LDS: buffers, then (maximum, sum) per wave and row
  return kFlatWaves * (2 * 32 * DC + 64);
}

template <class T, int DC>
__device__ __forceinline__ void flat_rows(const FwdParams& p, T* smem, int bid) {
  constexpr int W = kFlatWaves, BM = 16, CK = 32, KS = DC / 32, ND = DC / 16, TILE = CK * DC,
                NI = TILE / 512;
  float2(*ml)[16] = (float2(*)[16])(smem + W * 2 * TILE);
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int kvh = bid % p.heads_kv;
  bid /= p.heads_kv;
  const int split = p.splits - 1 - bid / p.slots, slot = p.slots - 1 - bid % p.slots;
  const Place at = place_of(p, slot, BM);
  if (!at.any) return;
  const int seen = seen_of(p, at, BM), parts = parts_of(p, seen);
  if (split >= parts) return;

  const int r16 = lane & 15, quad = lane >> 4;
  const RowOf row = row_of(at.tile * BM + r16, at.lq, at.lk, p.group, kvh, at.q0, p.causal);
  const int chunks = (seen + CK - 1) / CK;
  const int c0 = (int)((int64_t)chunks * split / parts);
  const int c1 = (int)((int64_t)chunks * (split + 1) / parts);
  const T* K = (const T*)p.k + at.k_off + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + at.v_off + (int64_t)kvh * p.v_head;
  const lds_c mine = (lds_c)smem + w * 4 * TILE;
  const int64_t qn = (int64_t)(row.n / p.q_inner) * p.q_batch + (row.n % p.q_inner) * p.q_tok;
  const T* Q = (const T*)p.q + qn + row.head * p.q_head;
  Vec8<T> qf[KS];
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    const int d = 32 * kk + 8 * quad;
    if (d < p.dim)
      qf[kk] = load8(Q + d);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[kk][e] = (T)0.0f;
  }
  floatx4 acc[ND];
#pragma unroll
  for (int j = 0; j < ND; ++j) acc[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  // byte offsets of the lane's reads (see Reader)
  const unsigned s0 = 2u * tile_off<DC>(r16, 8 * quad);
  const unsigned t0 = 2u * tile_off<DC>(4 * quad + (r16 >> 2), 4 * (r16 & 3));
  auto fetch = [&](const T* x, int64_t stride, int c, lds_c to) {
    const Fetch<T, DC> f = Fetch<T, DC>::of(x, stride, c * CK, c < c1 ? at.lk : 0, p.dim);
#pragma unroll
    for (int j = 0; j < NI; ++j) f.issue(stride, p.dim, to, j, lane);
  };
  auto reads_done = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](int c, lds_c __restrict__ from, lds_c __restrict__ to) {
    if (c == hidden(c0 + w)) {
      fetch(K, p.k_tok, c, to);
      fetch(V, p.v_tok, c, to + 2 * TILE);
    }
    wait_vm<NI>();                       // K has landed, V may be in flight
    unsigned s = s0 + (unsigned)(uintptr_t)from;
    asm volatile("" : "+v"(s));
    floatx4 st[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      st[b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        using ptr = const __attribute__((address_space(3))) Vec8<T>*;
        st[b] = Elem<T>::mma16(*(ptr)((s ^ (64u * kk)) + 32 * b * DC), qf[kk], st[b]);
      }
    }
    reads_done();
    fetch(K, p.k_tok, c + W, to);
    const int room = row.limit - c * CK - 4 * quad;
    const unsigned visible = low_bits(room + 1);
    float top = -INFINITY;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st[b][e] = select_bit(visible, 16 * b + e, st[b][e], -INFINITY);
        top = fmaxf(top, st[b][e]);
      }
    top = all4_max(top) * p.scale_log2;
    if (__any(top - m > kSlack)) {
      const float next = fmaxf(m, top);
      const float f = __builtin_amdgcn_exp2f(m - (next == -INFINITY ? 0.0f : next));
      l *= f;
#pragma unroll
      for (int j = 0; j < ND; ++j) acc[j] *= f;
      m = next;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    Vec8<T> pf;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = __builtin_amdgcn_exp2f(__builtin_fmaf(st[i / 4][i % 4], p.scale_log2, -ref));
      l += v;
      pf[i] = (T)v;
    }
    wait_vm<NI>();                       // V has landed, the next K may be in flight
    unsigned t = t0 + (unsigned)(uintptr_t)from;
    asm volatile("" : "+v"(t));
    auto read_tr = [&](unsigned address) {
      return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s4)(from + (int)(address - (unsigned)(uintptr_t)from)));
    };
#pragma unroll
    for (int db = 0; db < ND; ++db) {
      const unsigned x = (t ^ (32u * db)) + 2 * TILE;
      const shortx4 lo = read_tr(x), hi = read_tr(x + 32 * DC);
      acc[db] = Elem<T>::mma16(
          __builtin_bit_cast(Vec8<T>, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)), pf,
          acc[db]);
    }
    reads_done();
    fetch(V, p.v_tok, c + W, to + 2 * TILE);
  };
  int c = c0 + w;
  if (c < c1) {
    do step(c, mine, mine);
    while ((c += W) < c1);
    settle();
  }
  wait_vm<0>();
  // join: every wave scales its rows to the common maximum and leaves them in
  // LDS (16-byte group g of row r at g ^ r)
  l = all4_sum(l);
  if (lane < 16) ml[w][lane] = make_float2(m, l);
  __syncthreads();
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < W; ++i) top = fmaxf(top, ml[i][r16].x);
  const float f = __builtin_amdgcn_exp2f(m - (top == -INFINITY ? 0.0f : top));
  float* rows = (float*)smem + w * BM * DC;
#pragma unroll
  for (int db = 0; db < ND; ++db)
    *(floatx4*)(rows + r16 * DC + 4 * ((4 * db + quad) ^ r16)) = acc[db] * f;
  __syncthreads();
  // 4 elements of a row per thread and turn
  constexpr int GROUPS = DC / 4;
  const int heads = p.heads_kv * p.group;
  for (int x = threadIdx.x; x < BM * GROUPS; x += 64 * W) {
    const int rr = x / GROUPS, g = x % GROUPS;
    const RowOf o = row_of(at.tile * BM + rr, at.lq, at.lk, p.group, kvh, at.q0, p.causal);
    if (!o.valid) continue;
    float mt = -INFINITY, lt = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) mt = fmaxf(mt, ml[i][rr].x);
    const float mr = mt == -INFINITY ? 0.0f : mt;
    floatx4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      lt += ml[i][rr].y * __builtin_amdgcn_exp2f(ml[i][rr].x - mr);
      sum += *(const floatx4*)((const float*)smem + (i * BM + rr) * DC + 4 * (g ^ rr));
    }
    const int64_t out_row = (int64_t)o.n * heads + o.head;
    if (to_parts(p, parts)) {
      const int64_t at_row = (int64_t)(p.split0 + split) * p.rows + out_row;
      if (g == 0) p.part_ml[at_row] = make_float2(mt, lt);
      if (lt != 0.0f) *(floatx4*)(p.part_o + at_row * DC + 4 * g) = sum;
      continue;
    }
    const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
    if (4 * g < p.dim) {
      typedef T vec4 __attribute__((ext_vector_type(4)));
      const int64_t on = (int64_t)(o.n / p.q_inner) * p.o_batch + (o.n % p.q_inner) * p.o_tok;
      vec4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = (T)(sum[e] * inv);
      *(vec4*)((T*)p.o + on + o.head * p.o_head + 4 * g) = y;
    }
    if (p.lse && g == 0)
      p.lse[out_row] = lt == 0.0f ? -INFINITY : (mt + __builtin_amdgcn_logf(lt)) * kLn2;
  }
}

template <class T, int DC>
__global__ void __launch_bounds__(64 * kFlatWaves, DC == 256 ? 1 : 2)
    attention_flat(const FwdParams p) {
  __shared__ __attribute__((aligned(4096))) T smem[flat_elems<T, DC>()];
  flat_rows<T, DC>(p, smem, blockIdx.x);
}

// Two problems in one launch, for decoding behind a prefix: the first `n0`
// workgroups work on `a` (the prefix, tall or flat rows), the others on `b`
// (the sequences' own keys, flat rows).  The prefix is bound by the matrix
// pipe when many rows share it, the own keys by memory; side by side on a CU
// each fills the other's waits.  64 tokens of 32/8 heads of 128 behind 8192
// keys with up to 1000 own: 35 us, in two launches one after the other 55; 128
// behind 32768 keys with 256 - 2048 own: 181 us, two launches 249 (740 MB of
// keys and values, 4.1 TB/s of a large copy's 4.77, and 71 GFLOP).  Every tile
// of rows stages the whole prefix: those 128 tokens are four tiles of 128 rows
// per kv head and read it four times, from the caches mostly.
template <class T, int DC, bool TALL>
__global__ void __launch_bounds__(256, DC == 256 ? 1 : 2)
    attention_pair(const FwdParams a, const FwdParams b, int n0) {
  constexpr int E0 = TALL ? tall_stages<DC>() * 2 * 64 * DC : 0, E1 = flat_elems<T, DC>();
  __shared__ __attribute__((aligned(4096))) T smem[E0 > E1 ? E0 : E1];
  const int bid = blockIdx.x;
  if (bid < n0) {
    if constexpr (TALL)
      tall_rows<T, DC>(a, smem, bid);
    else
      flat_rows<T, DC>(a, smem, bid);
  } else {
    flat_rows<T, DC>(b, smem, bid - n0);
  }
}

// ------------------------------------------------------ joining splits
// One wave: the weights of a row's splits from their maxima and sums (a split
// per lane), then their accumulators in split order, 8 in flight.
template <class T, int DC>
__device__ __forceinline__ void join_row(const float* part_o, const float2* part_ml, int64_t rows,
                                         int64_t row, int splits, int dim, T* out, float* lse) {
  const int lane = threadIdx.x & 63;
  constexpr int E = DC / 64;
  typedef float vecE __attribute__((ext_vector_type(E)));
  // 64 splits at a time; what came before carries over as one more
  float m = -INFINITY, l = 0.0f;
  vecE sum;
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.0f;
  for (int s0 = 0; s0 < splits; s0 += 64) {
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (s0 + lane < splits) ml = part_ml[(s0 + lane) * rows + row];
    float top = ml.x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    top = fmaxf(top, m);
    const float ref = top == -INFINITY ? 0.0f : top;
    // (a split without visible keys has weight 0, and nothing was written)
    const float f = ml.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml.x - ref);
    const float old = __builtin_amdgcn_exp2f(m - ref);
    float part = ml.y * f;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) part += __shfl_xor(part, d);
    l = l * old + part;
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] *= old;
    m = top;
    const int n = min(splits - s0, 64);
    for (int i = 0; i < n; i += 8) {
      vecE v[8];
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = __shfl(f, i + j);
        const int s = s0 + i + j;
        if (i + j < n && g[j] != 0.0f)
          v[j] = *(const vecE*)(part_o + (s * rows + row) * DC + E * lane);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < n && g[j] != 0.0f)
#pragma unroll
          for (int e = 0; e < E; ++e) sum[e] += v[j][e] * g[j];
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (E * lane < dim) {
    typedef T outE __attribute__((ext_vector_type(E)));
    outE y;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = (T)(sum[e] * inv);
    *(outE*)(out + E * lane) = y;
  }
  if (lse && lane == 0) *lse = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// every row, one wave each: decoding behind a prefix, where each has its parts
template <class T, int DC>
__global__ void __launch_bounds__(256) attention_join(const CombineParams p) {
  const int64_t row = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
  if (row >= p.rows) return;
  const int n = (int)(row / p.heads), head = (int)(row % p.heads);
  join_row<T, DC>(p.part_o, p.part_ml, p.rows, row, p.splits, p.dim,
                  (T*)p.o + (int64_t)(n / p.q_inner) * p.o_batch + (n % p.q_inner) * p.o_tok +
                      head * p.o_head,
                  p.lse ? p.lse + row : nullptr);
}

// The rows of the tiles that took more than one split, one after the other
// where a workgroup has `each` > 4 of them.  Rows of no sequence are in no
// tile: nothing is known of their parts, and nothing is written.
template <class T, int DC>
__global__ void __launch_bounds__(256) attention_join_tiles(const FwdParams p, int bm, int each) {
  int bid = blockIdx.x;
  const int kvh = bid % p.heads_kv;
  bid /= p.heads_kv;
  const int per = bm / each;
  const Place at = place_of(p, bid / per, bm);
  if (!at.any) return;
  const int parts = parts_of(p, seen_of(p, at, bm));
  if (parts == 1) return;
  for (int i = 0; i < each; i += 4) {
    const int r = at.tile * bm + each * (bid % per) + i + uniform(threadIdx.x >> 6);
    const RowOf row = row_of(r, at.lq, at.lk, p.group, kvh, at.q0, p.causal);
    if (!row.valid) return;
    const int64_t out_row = (int64_t)row.n * (p.heads_kv * p.group) + row.head;
    join_row<T, DC>(p.part_o, p.part_ml, p.rows, out_row, parts, p.dim,
                    (T*)p.o + row.n * p.o_tok + row.head * p.o_head,
                    p.lse ? p.lse + out_row : nullptr);
  }
}

}  // namespace att
}  // namespace mfl
