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
};
template <>
struct Elem<__bf16> {
  typedef __bf16 vec8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ floatx16 mma(vec8 a, vec8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <class T>
using Vec8 = typename Elem<T>::vec8;

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
};

// ------------------------------------------------------------- LDS tiles
// Rows of DC elements, 16-byte chunk c of row r stored at chunk c ^ swz(r).
// Straight reads (one chunk of 16 consecutive rows) and transposing reads (4
// consecutive chunks of 4 consecutive rows) both spread over the banks: swz
// differs over 16 rows (DC = 64, two rows per pass of the banks: over 8 pairs
// of rows), and over 4 rows (2 pairs) already in its upper bits.
template <int DC>
MFL_HD constexpr int swz_row(int r) {
  return DC >= 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
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
  return true;
}
static_assert(swizzle_spreads<64>() && swizzle_spreads<128>() && swizzle_spreads<256>(),
              "both kinds of LDS reads must touch every bank group once");

// Where no key or column is, the direct-to-LDS loads read zeros (for a
// query's log-sum-exp: infinity, which makes its weights zero).
static __device__ const uint4 kZeros = {0u, 0u, 0u, 0u};
static __device__ const float kInfinity = INFINITY;

template <class T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p, 16), 16);
  return v;
}

// The operand fragment of rows r..r+31 (lane: row l % 32, d = d0 + 8 (l / 32))
template <class T, int DC>
__device__ __forceinline__ Vec8<T> frag(const T* tile, int r, int d) {
  return *(const Vec8<T>*)&tile[tile_off<DC>(r, d)];
}

// Transposed: lane (row d0 + l % 32, values: the keys k0 + 4 (l / 32) + 0..3
// and 8 further) of a tile stored key by key
template <class T, int DC>
__device__ __forceinline__ Vec8<T> frag_tr(const T* tile, int k0, int d0, int lane) {
  const int s = lane & 15, blk = lane >> 4;
  const int r = k0 + 4 * (blk >> 1) + (s >> 2), d = d0 + 16 * (blk & 1) + 4 * (s & 3);
  const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(&tile[tile_off<DC>(r, d)]));
  const shortx4 hi =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(&tile[tile_off<DC>(r + 8, d)]));
  return __builtin_bit_cast(Vec8<T>, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

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
__device__ __forceinline__ float both_max(float x) {
  const Halves h = halves(x);
  return fmaxf(h.lower, h.upper);
}
__device__ __forceinline__ float both_sum(float x) {
  const Halves h = halves(x);
  return h.lower + h.upper;
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

// ------------------------------------------------ direct-to-LDS staging
// One wave instruction fills 1024 consecutive LDS bytes; each lane fetches
// the 16 bytes its place stands for.
template <class T, int DC>
struct Fetch {
  static constexpr int ROWS = 512 / DC;   // tile rows per instruction
  // instruction i of a tile whose row 0 is key `key0`: rows with key >= end
  // and columns past `dim` are zeros
  static __device__ __forceinline__ void issue(const T* base, int64_t stride, int key0, int end,
                                               int dim, T* tile, int i, int lane) {
    const int r = i * ROWS + (8 * lane) / DC, c = ((8 * lane) % DC) / 8;
    const int col = 8 * (c ^ swz_row<DC>(r)), key = key0 + r;
    const void* g = base + (int64_t)key * stride + col;
    if (key >= end || col >= dim) g = &kZeros;
    __builtin_amdgcn_global_load_lds(g, (lds_t)(tile + i * 512), 16, 0, 0);
  }
};

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

// Running softmax of the lane's row over the scores in st: updates the
// reference maximum m (in units of log2), the lane's share l of the sum and
// the accumulators, leaves the weights in st.
template <int NB, int ND>
__device__ __forceinline__ void softmax_step(floatx16 (&st)[NB], floatx16 (&acc)[ND], float& m,
                                             float& l, float c) {
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
  const float ref = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(st[b][i], c, -ref));
      st[b][i] = w;
      sum += w;
    }
  l += sum;
}

// keys past the row's limit get -inf
template <int NB>
__device__ __forceinline__ void mask_keys(floatx16 (&st)[NB], int key0, int limit, int lane) {
  const int room = limit - key0 - 4 * (lane >> 5);
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (32 * b + 8 * (i / 4) + i % 4 > room) st[b][i] = -INFINITY;
}

// ------------------------------------------------------ forward, tall
// W waves of 32 rows each over chunks of 64 keys staged in a ring of NST LDS
// stages (K and V of a chunk together), shared by the workgroup.
template <int DC>
MFL_HD constexpr int tall_stages(int waves) {
  return DC == 256 ? 2 : waves == 8 ? 4 : DC == 64 ? 4 : 2;
}

template <class T, int DC, int W>
__global__ void __launch_bounds__(64 * W) attention_tall(const FwdParams p) {
  constexpr int BM = 32 * W, CK = 64, NST = tall_stages<DC>(W), KS = DC / 16, ND = DC / 32;
  constexpr int TILE = CK * DC, NI = CK * DC / 512 / W;   // elements, instructions per matrix and wave
  static_assert(NI >= 1 && 4 * NST * TILE <= 160 * 1024, "staging");
  __shared__ __attribute__((aligned(1024))) T smem[NST * 2 * TILE];
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  int bid = blockIdx.x;
  const int kvh = bid % p.heads_kv;
  bid /= p.heads_kv;
  const int split = bid % p.splits;
  const int slot = p.slots - 1 - bid / p.splits;         // the longest rows first
  const Place at = place_of(p, slot, BM);
  if (!at.any) return;

  const int r0 = at.tile * BM + 32 * w;
  const RowOf row = row_of(r0 + (lane & 31), at.lq, at.lk, p.group, kvh, at.q0, p.causal);
  const int first_row_limit = uniform(row.limit);
  // no work for a wave whose rows are all past the last one
  const int wave_limit =
      r0 < at.lq * p.group ? __builtin_amdgcn_readlane(row.limit, 31) : -1;
  // keys of this workgroup: to its last row's limit, its share of them
  const int last_t = min((int)(((int64_t)at.tile * BM + BM - 1) / p.group), at.lq - 1);
  const int seen = max(p.causal ? min(last_t + at.lk - at.lq, at.lk - 1) + 1 : at.lk, 0);
  const int chunks = (seen + CK - 1) / CK;
  const int c0 = (int)((int64_t)chunks * split / p.splits);
  const int c1 = (int)((int64_t)chunks * (split + 1) / p.splits);

  const T* K = (const T*)p.k + at.k_off + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + at.v_off + (int64_t)kvh * p.v_head;
  auto issue = [&](int c) {
    if (c >= c1) return;
    T* st = smem + ((c - c0) % NST) * 2 * TILE;
#pragma unroll
    for (int j = 0; j < NI; ++j)
      Fetch<T, DC>::issue(K, p.k_tok, c * CK, at.lk, p.dim, st, w * NI + j, lane);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      Fetch<T, DC>::issue(V, p.v_tok, c * CK, at.lk, p.dim, st + TILE, w * NI + j, lane);
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

#pragma unroll
  for (int s = 0; s < NST - 1; ++s) issue(c0 + s);
  for (int c = c0; c < c1; ++c) {
    // chunk c has landed here, and after the barrier everywhere; its
    // predecessor's stage is free
    const int ahead = min(c1 - 1 - c, NST - 2);
    if (ahead >= 2) wait_vm<(NST > 3 ? 2 : 0) * 2 * NI>();
    else if (ahead == 1) wait_vm<(NST > 2 ? 1 : 0) * 2 * NI>();
    else wait_vm<0>();
    barrier();
    issue(c + NST - 1);
    const int key0 = c * CK;
    if (key0 > wave_limit) continue;
    const T* sk = smem + ((c - c0) % NST) * 2 * TILE;
    const T* sv = sk + TILE;
    floatx16 st[2];
    zero(st);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
        st[b] = Elem<T>::mma(
            frag<T, DC>(sk, 32 * b + (lane & 31), 16 * kk + 8 * (lane >> 5)), qf[kk], st[b]);
    if (key0 + CK - 1 > first_row_limit) mask_keys(st, key0, row.limit, lane);
    softmax_step(st, acc, m, l, p.scale_log2);
#pragma unroll
    for (int kc = 0; kc < 4; ++kc) {
      const Vec8<T> pf = pack8<T>(st[kc / 2], kc % 2);
#pragma unroll
      for (int db = 0; db < ND; ++db)
        acc[db] = Elem<T>::mma(frag_tr<T, DC>(sv, 16 * kc, 32 * db, lane), pf, acc[db]);
    }
  }

  l = both_sum(l);
  const int64_t out_row = (int64_t)row.n * (p.heads_kv * p.group) + row.head;
  if (p.part_o) {
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

// ------------------------------------------------------ forward, flat
// Few rows, long keys: 32 rows per workgroup, whose W waves take turns over
// chunks of 32 keys.  Each wave has its own ring of stages, so no wave waits
// for another before the end, where the W partial rows are joined in LDS.
template <int DC>
MFL_HD constexpr int flat_waves() { return DC == 256 ? 2 : 4; }
template <int DC>
MFL_HD constexpr int flat_stages() { return DC == 64 ? 4 : 2; }

template <class T, int DC>
__global__ void __launch_bounds__(64 * flat_waves<DC>()) attention_flat(const FwdParams p) {
  constexpr int W = flat_waves<DC>(), NST = flat_stages<DC>(), CK = 32, KS = DC / 16,
                ND = DC / 32, TILE = CK * DC, NI = TILE / 512, BM = 32;
  static_assert(2 * (NST - 1) * NI < 64, "loads in flight");
  constexpr int RING = NST * 2 * TILE;                   // elements per wave
  __shared__ __attribute__((aligned(1024))) T smem[W * RING];
  __shared__ float2 ml[W][32];
  static_assert(2 * W * RING >= 4 * W * 32 * DC, "the partial rows fit in the rings");
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  int bid = blockIdx.x;
  const int kvh = bid % p.heads_kv;
  bid /= p.heads_kv;
  const int split = bid % p.splits;
  const int slot = p.slots - 1 - bid / p.splits;
  const Place at = place_of(p, slot, BM);
  if (!at.any) return;

  const RowOf row = row_of(at.tile * BM + (lane & 31), at.lq, at.lk, p.group, kvh, at.q0, p.causal);
  const int first_row_limit = uniform(row.limit);
  const int seen = max(__builtin_amdgcn_readlane(row.limit, 31) + 1, 0);
  const int chunks = (seen + CK - 1) / CK;
  const int c0 = (int)((int64_t)chunks * split / p.splits);
  const int c1 = (int)((int64_t)chunks * (split + 1) / p.splits);
  const T* K = (const T*)p.k + at.k_off + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + at.v_off + (int64_t)kvh * p.v_head;
  T* ring = smem + w * RING;
  const int mine = max((c1 - c0 - w + W - 1) / W, 0);    // chunks c0 + w, + W, ...
  auto issue = [&](int i) {
    if (i >= mine) return;
    T* st = ring + (i % NST) * 2 * TILE;
    const int key0 = (c0 + w + i * W) * CK;
#pragma unroll
    for (int j = 0; j < NI; ++j) Fetch<T, DC>::issue(K, p.k_tok, key0, at.lk, p.dim, st, j, lane);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      Fetch<T, DC>::issue(V, p.v_tok, key0, at.lk, p.dim, st + TILE, j, lane);
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
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) issue(s);
  for (int i = 0; i < mine; ++i) {
    // this wave's reads of the stage of chunk i - 1 are done: refill it
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    issue(i + NST - 1);
    const int ahead = min(mine - 1 - i, NST - 1);
    if (ahead >= 3) wait_vm<(NST > 3 ? 3 : 0) * 2 * NI>();
    else if (ahead == 2) wait_vm<(NST > 2 ? 2 : 0) * 2 * NI>();
    else if (ahead == 1) wait_vm<2 * NI>();
    else wait_vm<0>();
    __builtin_amdgcn_sched_barrier(0);
    const T* sk = ring + (i % NST) * 2 * TILE;
    const T* sv = sk + TILE;
    const int key0 = (c0 + w + i * W) * CK;
    floatx16 st[1];
    zero(st);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
      st[0] = Elem<T>::mma(frag<T, DC>(sk, lane & 31, 16 * kk + 8 * (lane >> 5)), qf[kk], st[0]);
    if (key0 + CK - 1 > first_row_limit) mask_keys(st, key0, row.limit, lane);
    softmax_step(st, acc, m, l, p.scale_log2);
#pragma unroll
    for (int kc = 0; kc < 2; ++kc) {
      const Vec8<T> pf = pack8<T>(st[0], kc);
#pragma unroll
      for (int db = 0; db < ND; ++db)
        acc[db] = Elem<T>::mma(frag_tr<T, DC>(sv, 16 * kc, 32 * db, lane), pf, acc[db]);
    }
  }
  // join: every wave scales its rows to the common maximum and leaves them in
  // LDS (16-byte group g of row r at g ^ (r & 15))
  l = both_sum(l);
  if (lane < 32) ml[w][lane] = make_float2(m, l);
  __syncthreads();
  const int r = lane & 31;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < W; ++i) top = fmaxf(top, ml[i][r].x);
  const float ref = top == -INFINITY ? 0.0f : top;
  const float f = __builtin_amdgcn_exp2f(m - ref);
  float* rows = (float*)smem + w * 32 * DC;
#pragma unroll
  for (int db = 0; db < ND; ++db)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int g = (8 * db + 2 * q + (lane >> 5)) ^ (r & 15);
      *(floatx4*)(rows + r * DC + 4 * g) =
          floatx4{acc[db][4 * q] * f, acc[db][4 * q + 1] * f, acc[db][4 * q + 2] * f,
                  acc[db][4 * q + 3] * f};
    }
  __syncthreads();
  // 4 elements of a row per thread and turn
  constexpr int GROUPS = DC / 4;
  const int heads = p.heads_kv * p.group;
  for (int x = threadIdx.x; x < 32 * GROUPS; x += 64 * W) {
    const int rr = x / GROUPS, g = x % GROUPS;
    const RowOf o = row_of(at.tile * BM + rr, at.lq, at.lk, p.group, kvh, at.q0, p.causal);
    if (!o.valid) continue;
    float mt = -INFINITY, lt = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) mt = fmaxf(mt, ml[i][rr].x);
    const float mr = mt == -INFINITY ? 0.0f : mt;
    floatx4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      lt += ml[i][rr].y * __builtin_amdgcn_exp2f(ml[i][rr].x - mr);
      s += *(const floatx4*)((const float*)smem + (i * 32 + rr) * DC + 4 * (g ^ (rr & 15)));
    }
    const int64_t out_row = (int64_t)o.n * heads + o.head;
    if (p.part_o) {
      const int64_t at_row = (int64_t)(p.split0 + split) * p.rows + out_row;
      if (g == 0) p.part_ml[at_row] = make_float2(mt, lt);
      if (lt != 0.0f) *(floatx4*)(p.part_o + at_row * DC + 4 * g) = s;
      continue;
    }
    const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
    if (4 * g < p.dim) {
      typedef T vec4 __attribute__((ext_vector_type(4)));
      const int64_t on = (int64_t)(o.n / p.q_inner) * p.o_batch + (o.n % p.q_inner) * p.o_tok;
      vec4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = (T)(s[e] * inv);
      *(vec4*)((T*)p.o + on + o.head * p.o_head + 4 * g) = y;
    }
    if (p.lse && g == 0)
      p.lse[out_row] = lt == 0.0f ? -INFINITY : (mt + __builtin_amdgcn_logf(lt)) * kLn2;
  }
}

// ------------------------------------------------------ joining splits
// One wave per row: the splits' weights from their maxima and sums, then
// their accumulators in split order.
template <class T, int DC>
__global__ void __launch_bounds__(256) attention_join(const CombineParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= p.rows) return;
  float top = -INFINITY;
  for (int s = lane; s < p.splits; s += 64) top = fmaxf(top, p.part_ml[s * p.rows + row].x);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  const float ref = top == -INFINITY ? 0.0f : top;
  constexpr int E = DC / 64;
  typedef float vecE __attribute__((ext_vector_type(E)));
  vecE sum;
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.0f;
  float l = 0.0f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = p.part_ml[s * p.rows + row];
    if (ml.y == 0.0f) continue;        // no key of the split is visible
    const float f = __builtin_amdgcn_exp2f(ml.x - ref);
    l += ml.y * f;
    const vecE v = *(const vecE*)(p.part_o + (s * p.rows + row) * DC + E * lane);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] += v[e] * f;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int n = (int)(row / p.heads), head = (int)(row % p.heads);
  T* o = (T*)p.o + (int64_t)(n / p.q_inner) * p.o_batch + (n % p.q_inner) * p.o_tok +
         head * p.o_head;
  if (E * lane < p.dim) {
#pragma unroll
    for (int e = 0; e < E; ++e) o[E * lane + e] = (T)(sum[e] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[row] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace att
}  // namespace mfl
