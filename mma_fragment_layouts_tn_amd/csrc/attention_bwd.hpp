// Gradients of attention, without atomics: one kernel owns rows of queries
// and walks the keys (dQ), one owns keys and walks the rows (dK, dV).  Both
// compute the weights again from the log-sum-exp:
//
//   P = exp2(c Q K^T - lse log2 e),  dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,  delta = rowsum(dO O)
//
// Seven products instead of the five a single kernel would need, for sums
// whose order is fixed: a run gives the same bits every time, and the rows of
// a group's heads are added in the registers of one wave.
#pragma once

#include "attention.hpp"
#include "attention_launch.hpp"

namespace mfl {
namespace att {

// Sequence of a slot over the query tokens' rows or the keys; slots past the
// last sequence's share out the tokens behind it (`spare`: which share).
struct BwdPlace {
  int q0, lq, k0, lk, tile, spare;
  bool any;
};
__device__ __forceinline__ BwdPlace bwd_place(const BwdParams& p, int slot, int bm, bool rows) {
  const int* seq = rows ? p.seq_q : p.seq_k;
  const int total = rows ? p.total_q : p.total_k, mult = rows ? p.group : 1;
  BwdPlace r;
  int s = 0;
  r.spare = -1;
  if (seq) {
    auto f = [&](int i) { return (int)((int64_t)min(max(seq[i], 0), total) * mult / bm) + i; };
    s = find_sequence(p.batch, slot, f);
    r.tile = slot - uniform(f(s));
    r.spare = slot - uniform(f(p.batch));
  } else {
    r.tile = slot;
  }
  const Span q = p.seq_q ? span_of(p.seq_q, s, p.total_q) : Span{0, p.total_q};
  const Span k = p.seq_k ? span_of(p.seq_k, s, p.total_k) : Span{0, p.total_k};
  r.q0 = q.begin;
  r.lq = q.len;
  r.k0 = k.begin;
  r.lk = k.len;
  const int64_t len = rows ? (int64_t)r.lq * p.group : r.lk;
  r.any = r.tile >= 0 && (int64_t)r.tile * bm < len;
  return r;
}

// rows [from, to) of a gradient (row r: token r / group of the heads
// kvh * group + r % group) set to zero by the workgroup
template <class T>
__device__ __forceinline__ void zero_rows(T* base, int64_t tok, int64_t head, int group, int kvh,
                                          int64_t from, int64_t to, int dim, int threads) {
  const int per = dim / 8;
  for (int64_t x = threadIdx.x; x < (to - from) * per; x += threads) {
    const int64_t r = from + x / per;
    T* o = base + r / group * tok + (kvh * group + r % group) * head + 8 * (x % per);
    *(uint4*)o = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ------------------------------------------------------------------- dQ
// Four waves of 32 rows each, as the forward kernel's tall form, over chunks of
// 64 keys; also forms the rows' log-sum-exps in base 2 and deltas, which the
// kernel of dK and dV reads.  delta is the fp32 sum over the 16-bit out, dS is
// rounded to 16 bits as the third product's operand.  Error of dQ and dK: 0.0027
// of their norm (bf16; fp16 0.0003), where the results' own rounding alone is
// 0.0017.  With an exact delta it would be 0.0024, with an unrounded dS 0.0021;
// delta is exact only after all keys, too late for this kernel but for a fourth
// product (P K), and dS in two halves is a fourth product as well.  In fp16 a
// dS beyond 65504 is infinite.
//
// 8192 tokens in 4 sequences, 32/8 heads of 128, bf16: 278 us, 1,020 TFLOP/s,
// the matrix pipe busy for 55 % of the cycles, vector instructions issued in
// 40 %, both at once in 20 %.  Reads placed by the compiler, one before each
// use: 315; 8 waves in one workgroup per CU 316.
template <class T, int DC>
__global__ void __launch_bounds__(256, DC == 256 ? 1 : 2) attention_dq(const BwdParams p) {
  constexpr int W = 4, NST = tall_stages<DC>(), BM = 32 * W, CK = 64, KS = DC / 16, ND = DC / 32,
                TILE = CK * DC, NI = TILE / 512 / W, RA = 2;
  static_assert(BM == kDqRows, "rows per workgroup");
  __shared__ __attribute__((aligned(1024))) T smem[NST * 2 * TILE];
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int kvh = blockIdx.x % p.heads_kv, heads = p.heads_kv * p.group;
  const int slot = p.slots_q - 1 - blockIdx.x / p.heads_kv;
  const BwdPlace at = bwd_place(p, slot, BM, true);
  if (!at.any) {
    if (at.spare >= 0) {
      const int64_t end = (int64_t)p.total_q * p.group;
      const int64_t from =
          (int64_t)min(max(p.seq_q[p.batch], 0), p.total_q) * p.group + (int64_t)at.spare * BM;
      zero_rows<T>((T*)p.dq, p.dq_tok, p.dq_head, p.group, kvh, from, min(from + BM, end), p.dim,
                   64 * W);
    }
    return;
  }
  const int r0 = at.tile * BM + 32 * w;
  const RowOf row = row_of(r0 + (lane & 31), at.lq, at.lk, p.group, kvh, at.q0, p.causal);
  const int last_t = min((int)(((int64_t)at.tile * BM + BM - 1) / p.group), at.lq - 1);
  const int seen = max(p.causal ? min(last_t + at.lk - at.lq, at.lk - 1) + 1 : at.lk, 0);
  const int chunks = (seen + CK - 1) / CK;
  // chunks before `cut` hide nothing from any of the wave's rows
  const int cut = min(max((uniform(row.limit) + 1) / CK, 0), chunks);
  const T* K = (const T*)p.k + (int64_t)at.k0 * p.k_tok + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + (int64_t)at.k0 * p.v_tok + (int64_t)kvh * p.v_head;
  const lds_c ring = (lds_c)smem;
  // load j of chunk c: K, then V
  struct Next {
    Fetch<T, DC> k, v;
  };
  auto next_chunk = [&](int c) {
    const int end = c < chunks ? at.lk : 0;
    return Next{Fetch<T, DC>::of(K, p.k_tok, c * CK, end, p.dim),
                Fetch<T, DC>::of(V, p.v_tok, c * CK, end, p.dim)};
  };
  auto issue = [&](const Next& n, lds_c to, int j) {
    if (j < NI)
      n.k.issue(p.k_tok, p.dim, to, w * NI + j, lane);
    else
      n.v.issue(p.v_tok, p.dim, to + 2 * TILE, w * NI + j - NI, lane);
  };

  const T* Q = (const T*)p.q + row.n * p.q_tok + row.head * p.q_head;
  const T* O = (const T*)p.o + row.n * p.o_tok + row.head * p.o_head;
  const T* G = (const T*)p.dout + row.n * p.do_tok + row.head * p.do_head;
  Vec8<T> qf[KS], gf[KS];
  float delta = 0.0f;
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    const int d = 16 * kk + 8 * (lane >> 5);
    if (d < p.dim) {
      qf[kk] = load8(Q + d);
      gf[kk] = load8(G + d);
      const Vec8<T> of = load8(O + d);
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)gf[kk][e], (float)of[e], delta);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[kk][e] = gf[kk][e] = (T)0.0f;
    }
  }
  delta = both_sum(delta);
  float lse2 = p.lse[(int64_t)row.n * heads + row.head];
  lse2 = lse2 == -INFINITY ? INFINITY : lse2 * kLog2e;   // no visible key: weights 0
  if (row.valid && lane < 32) {
    p.stats[(int64_t)row.head * p.total_q + row.n] = lse2;
    p.stats[(int64_t)(heads + row.head) * p.total_q + row.n] = delta;
  }
  floatx16 acc[ND];
  zero(acc);

  const Reader<T, DC> reader = Reader<T, DC>::of(lane);
  // chunk c, while chunk c + NST - 1 is fetched; every step issues 2 NI loads
  auto step = [&](int c, lds_c __restrict__ from, lds_c __restrict__ to, auto masked) {
    if (c == hidden(0)) {
#pragma unroll
      for (int s = 0; s < NST - 1; ++s) {
        const Next nx = next_chunk(s);
#pragma unroll
        for (int j = 0; j < 2 * NI; ++j) issue(nx, to + 4 * s * TILE, j);
      }
    }
    wait_vm<(NST - 2) * 2 * NI>();
    barrier();
    const Next nx = next_chunk(c + NST - 1);
    const lds_c fill = to + (c + NST - 1) % NST * 4 * TILE;
    const Reader<T, DC> rd = reader.at(from);
    // Six products of KS slots of one matrix instruction each, pinned in this
    // order: S and dP of keys 0 - 31, S and dP of keys 32 - 63, dQ of both.
    // The weights of the first block are formed under the second's S, its
    // score gradients under the second's dP, the second's under the first's
    // dQ.  Fragments are read RA slots ahead (left to itself the compiler
    // reads each just before its use), the next chunk's loads are spread out.
    floatx16 st[2][1], dp[2][1];
    Vec8<T> fr[RA + 1], df[2][2];
    unsigned seen_keys[2];
    auto read = [&](int n) {
      if (n >= 6 * KS) return;
      const int ph = n / KS, kk = n % KS;
      Vec8<T>& f = fr[n % (RA + 1)];
      if (ph < 4)
        f = rd.straight(ph / 2, kk, ph % 2 ? 2 * TILE : 0);
      else
        f = rd.transposed(2 * (ph - 4) + kk / ND, kk % ND);
    };
    // unit u of 32: value u % 16; 0 - 15 weights, 16 - 31 score gradients
    auto work = [&](int b, int u) {
      const int i = u % 16;
      if (u < 16) {
        float x = __builtin_amdgcn_exp2f(__builtin_fmaf(st[b][0][i], p.scale_log2, -lse2));
        if constexpr (decltype(masked)::value)
          x = select_bit(seen_keys[b], 8 * (i / 4) + i % 4, x, 0.0f);
        st[b][0][i] = x;
      } else {
        dp[b][0][i] = st[b][0][i] * (dp[b][0][i] - delta);
        if (i % 8 == 7) df[b][i / 8] = pack8<T>(dp[b][0], i / 8);
      }
    };
    auto fill_slot = [&](int n) {
      const int ph = n / KS, m = n % KS;
      // units of a phase: 16 (phases 2, 3) or 32 (4) over KS slots
      const int each = ph == 4 ? 32 : 16;
      if (ph >= 2 && ph <= 4)
#pragma unroll
        for (int u = each * m / KS; u < each * (m + 1) / KS; ++u)
          work(ph == 4 ? 1 : 0, ph == 3 ? 16 + u : u);
#pragma unroll
      for (int j = 0; j < 2 * NI; ++j)
        if ((2 * j + 1) * 6 * KS / (8 * NI) == n) issue(nx, fill, j);
      __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (decltype(masked)::value)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        seen_keys[b] = low_bits(row.limit + 1 - c * CK - 32 * b - 4 * (lane >> 5));
#pragma unroll
    for (int n = 0; n < RA; ++n) read(n);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      zero(st[b]);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const int n = 2 * b * KS + kk;
        read(n + RA);
        st[b][0] = Elem<T>::mma(fr[n % (RA + 1)], qf[kk], st[b][0]);
        fill_slot(n);
      }
      zero(dp[b]);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const int n = (2 * b + 1) * KS + kk;
        read(n + RA);
        dp[b][0] = Elem<T>::mma(fr[n % (RA + 1)], gf[kk], dp[b][0]);
        fill_slot(n);
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const int n = (4 + b) * KS + kk;
        read(n + RA);
        acc[kk % ND] = Elem<T>::mma(fr[n % (RA + 1)], df[b][kk / ND], acc[kk % ND]);
        fill_slot(n);
      }
  };
  int c = 0;
  if (c < cut) {
    do step(c, ring + c % NST * 4 * TILE, ring, BoolC<false>{});
    while (++c < cut);
    settle();
  }
  if (c < chunks) {
    do step(c, ring + c % NST * 4 * TILE, ring, BoolC<true>{});
    while (++c < chunks);
    settle();
  }
  wait_vm<0>();
  store_row<T, DC>((T*)p.dq + row.n * p.dq_tok + row.head * p.dq_head, acc, p.scale, p.dim, lane,
                   row.valid);
}

// ------------------------------------------------------------- dK and dV
// KW x RW waves: wave w holds the 32 KB keys of key group w % KW and takes
// block w / KW of each chunk's 32-row blocks; the row groups' sums are added
// in LDS at the end.  Chunks of RC query tokens of one head at a time, over
// the heads of the group.  Scores come with the rows in the registers and the
// key in the lane (S = Q K^T, A operand from LDS), so P and dS are the B
// operands of dV^T = dO^T P and dK^T = Q^T dS as they are, and every fragment
// read from LDS serves the KB key blocks of the wave.
//
// With KB = 2 and 128 columns a wave's sums take all 256 accumulation
// registers, one wave per SIMD; K of the tile is held in registers, V in LDS.
// Two waves of 32 keys each instead issue twice the LDS reads, waits and
// scalar instructions per matrix instruction, and those, not the matrix pipe,
// set their pace: 4,600 cycles for 2,048 of matrix work, here 3,600.
//
// 8192 tokens in 4 sequences, 32/8 heads of 128, bf16: 411 us, 920 TFLOP/s,
// the matrix pipe busy for 47 % of the cycles, vector instructions issued in
// 28 %, both at once in 12 %; with one wave per SIMD what it waits for is not
// filled.  Reads 1, 3 or 4 slots ahead instead of 2 change nothing.  The join
// takes 26 us more, for the partial sums written and read.  At 128 and 256
// columns 65 and 81 registers are spilled (224 and 256 bytes per lane), all of
// them around the steps of a tile, none in them.
//
// The chunks that the causal mask cuts come first, in a loop of their own: the
// mask as a branch inside one loop made the compiler spill accumulators.
struct DkvSteps {
  int first, cut, last;     // chunks: first that sees the tile, first without
                            // hidden keys, last of the sequence
  int steps;                // over the heads of the group
};
__device__ __forceinline__ DkvSteps dkv_steps(const BwdParams& p, int lq, int lk, int tile, int bn,
                                              int rc) {
  DkvSteps r;
  const int off = lk - lq, j0 = tile * bn;
  r.last = (lq + rc - 1) / rc - 1;
  r.first = r.cut = 0;
  if (p.causal) {           // token t sees the keys up to t + off
    r.first = max(j0 - off, 0) / rc;
    r.cut = max((max(j0 + bn - 1 - off, 0) + rc - 1) / rc, r.first);
    r.first = min(r.first, r.last + 1);
    r.cut = min(r.cut, r.last + 1);
  }
  r.steps = (r.last + 1 - r.first) * p.group;
  return r;
}

// Equal shares.  With a causal mask the tiles of a sequence differ in steps by
// as much as its length, and with one tile or equal parts of a tile per
// workgroup the last ones ran alone: 443 us, and 21 for the join, for 8192
// tokens in 4 sequences where the CUs were busy for 286.  So the units of all
// tiles of a kv head, in order (a tile's steps, and kDkvFixed more for its
// loads and stores), are cut into p.shares ranges of `each`, one per
// workgroup: 411 us, and 26 for the join.  Up to two tiles of a share are cut,
// and their sums go to the workspace; the one that goes on in the next share is
// noted in p.cuts, and attention_dkv_join adds its sums in order.
//
// Places.  A part is a share and a tile, and from each part to the next one or
// both grow: with tiles numbered in order, share + number is another place
// for each, shares + tiles - 1 in all.  Where there are more tiles than shares
// it is two places per share (the tile that began in an earlier share, the
// one that goes on in the next).  A tile's number is its slot (bwd_place): no
// less than the tiles before it, less than slots_k whatever the offsets are.
__device__ __forceinline__ int64_t dkv_place(const BwdParams& p, int share, int number,
                                             bool began) {
  return p.by_tile ? share + number : 2 * share + (began ? 1 : 0);
}
struct DkvUnits {
  int64_t n, r, c, group;   // chunks of rows; chunks per tile; chunks before the diagonal
  bool causal;
  // units of tiles 0 .. t - 1: group * sum of (n - max(0, i r - c))
  __device__ __forceinline__ int64_t before(int64_t t) const {
    int64_t hidden_chunks = 0;
    if (causal) {
      const int64_t i0 = c < 0 ? 0 : c / r + 1, m = t - i0;
      if (m > 0) hidden_chunks = r * ((i0 + t - 1) * m / 2) - c * m;
    }
    return t * (kDkvFixed + group * n) - group * hidden_chunks;
  }
};
__device__ __forceinline__ DkvUnits units_of(const BwdParams& p, int lq, int lk, int bn, int rc) {
  const int off = lk - lq;
  // ceil(off / rc), off of either sign
  const int c = off >= 0 ? (off + rc - 1) / rc : -(-off / rc);
  return DkvUnits{(lq + rc - 1) / rc, bn / rc, c, p.group, p.causal != 0};
}
struct Lens {
  int q0, lq, k0, lk;
};
__device__ __forceinline__ Lens lens_of(const BwdParams& p, int s) {
  if (!p.seq_k) return Lens{0, p.total_q, 0, p.total_k};
  const int q0 = min(max(p.seq_q[s], 0), p.total_q), q1 = min(max(p.seq_q[s + 1], 0), p.total_q);
  const int k0 = min(max(p.seq_k[s], 0), p.total_k), k1 = min(max(p.seq_k[s + 1], 0), p.total_k);
  return Lens{q0, max(q1 - q0, 0), k0, max(k1 - k0, 0)};
}
// the sequence that holds unit u and its first unit, and all units of a head
struct DkvFound {
  int s;
  int64_t base, total;
};
__device__ __forceinline__ DkvFound find_units(const BwdParams& p, int64_t u, int bn, int rc) {
  const int lane = threadIdx.x & 63;
  DkvFound r{0, 0, 0};
  for (int s0 = 0; s0 < p.batch; s0 += 64) {
    const int s = s0 + lane;
    int64_t sum = 0;
    if (s < p.batch) {
      const Lens l = lens_of(p, s);
      sum = units_of(p, l.lq, l.lk, bn, rc).before((l.lk + bn - 1) / bn);
    }
    const int64_t own = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int64_t y = __shfl_up((long long)sum, d);
      if (lane >= d) sum += y;
    }
    const int64_t base = r.total + sum - own;
    const int n = (int)__popcll(__ballot(s < p.batch && base <= u));   // bases never fall
    if (n > 0) {
      r.s = uniform(s0 + n - 1);
      r.base = __shfl((long long)base, n - 1);
    }
    r.total += __shfl((long long)sum, 63);
  }
  return r;
}
__device__ __forceinline__ int64_t dkv_each(int64_t total, int shares) {
  return max((total + shares - 1) / shares, (int64_t)kDkvLeast);
}
// largest t in [0, n) with before(t) <= u
__device__ __forceinline__ int find_tile(const DkvUnits& x, int n, int64_t u) {
  return find_sequence(n, 0, [&](int t) { return x.before(t) <= u ? 0 : 1; });
}

template <class T, int DC, int KW, int RW, int KB>
struct DkvShape {
  // V of the tile in registers beside K (else in LDS for all steps)
  static constexpr bool VREG = DC == 64;
  static constexpr int W = KW * RW, NST = DC == 256 ? 2 : 4, BN = 32 * KW * KB, RC = 32 * RW,
                       TILE = RC * DC, NI = TILE / 512 / W,
                       PER = 2 * NI + 1;                 // loads per wave and stage
  static constexpr int STATS = NST * 2 * TILE + (VREG ? 0 : BN * DC), ELEMS = STATS + NST * 256;
  static_assert(KB <= 2 && NI >= 1, "key blocks, loads");
  static_assert((RW - 1) * KW * 32 * DC * 4 <= NST * 4 * TILE, "sums fit in the stages");
};

// steps [first, first + steps) of a tile; `part`: where the sums go if these
// are not all of its steps
template <class T, int DC, int KW, int RW, int KB>
__device__ __forceinline__ void dkv_tile(const BwdParams& p, T* smem, const BwdPlace& at, int kvh,
                                         const DkvSteps& all, int first, int steps, float* part) {
  using S = DkvShape<T, DC, KW, RW, KB>;
  constexpr bool VREG = S::VREG;
  constexpr int W = S::W, NST = S::NST, BN = S::BN, RC = S::RC, TILE = S::TILE, NI = S::NI,
                PER = S::PER, KS = DC / 16, ND = DC / 32;
  float(*sstat)[2][64] = (float(*)[2][64])(smem + S::STATS);
  const lds_c ring = (lds_c)smem, sv = ring + NST * 4 * TILE;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6), kw = w % KW, rw = w / KW;
  const int heads = p.heads_kv * p.group;
  const int j0 = at.tile * BN + 32 * KB * kw, off = at.lk - at.lq;

  // Steps in order: the cut chunks of every head, then the others, each from
  // the last chunk down, so that the workgroups of one kv head, whose first
  // chunks differ, fetch the same chunks at about the same time.
  struct Cursor {
    int head, c, lo, hi;
  };
  auto cursor_at = [&](int s) {
    const int cut_steps = (all.cut - all.first) * p.group;
    Cursor u;
    const bool cut = s < cut_steps;
    u.lo = cut ? all.first : all.cut;
    u.hi = cut ? all.cut - 1 : all.last;
    if (!cut) s -= cut_steps;
    const int n = max(u.hi + 1 - u.lo, 1);
    u.head = uniform(s / n);
    u.c = u.hi - uniform(s % n);
    return u;
  };
  auto move = [&](Cursor& u) {
    if (--u.c >= u.lo) return;
    if (++u.head == p.group) {     // the cut chunks are done
      u.head = 0;
      u.lo = all.cut;
      u.hi = all.last;
    }
    u.c = u.hi;
  };
  const int cut_here =
      min(max((all.cut - all.first) * p.group - first, 0), steps);   // steps of the first loop
  int left = steps;                                                  // steps to fetch
  Cursor ahead = cursor_at(first), now = ahead;

  // the loads of a step, one by one
  struct Next {
    Fetch<T, DC> q, g;
    __amdgpu_buffer_rsrc_t stat;
  };
  auto advance = [&]() {
    const int t = ahead.c * RC, head = kvh * p.group + ahead.head;
    const int rows = left > 0 ? at.lq - t : 0;
    const int64_t n = (int64_t)at.q0 + t;
    Next x;
    x.q = Fetch<T, DC>::at((const T*)p.q + n * p.q_tok + head * p.q_head, p.q_tok, rows, p.dim);
    x.g =
        Fetch<T, DC>::at((const T*)p.dout + n * p.do_tok + head * p.do_head, p.do_tok, rows, p.dim);
    // even waves fetch the log-sum-exps, odd waves the deltas, 64 at a time
    // (several waves the same: every wave has as many loads in flight)
    x.stat = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.stats + ((int64_t)(w & 1) * heads + head) * p.total_q + n), 0,
        uniform(rows > 64 ? 256 : rows > 0 ? 4 * rows : 0), 0x00027000);
    --left;
    move(ahead);
    return x;
  };
  auto issue = [&](const Next& n, lds_c to, int stage, int j) {
    if (j < NI)
      n.q.issue(p.q_tok, p.dim, to, w * NI + j, lane);
    else if (j < 2 * NI)
      n.g.issue(p.do_tok, p.dim, to + 2 * TILE, w * NI + j - NI, lane);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(n.stat, (lds_t)(&sstat[stage][w & 1][0]), 4,
                                               4u * lane, 0, 0, 0);
  };
  const T* K = (const T*)p.k + (int64_t)at.k0 * p.k_tok + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + (int64_t)at.k0 * p.v_tok + (int64_t)kvh * p.v_head;
  Vec8<T> kf[KB][KS], vf[VREG ? KB : 1][VREG ? KS : 1];
#pragma unroll
  for (int x = 0; x < KB; ++x)
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int d = 16 * kk + 8 * (lane >> 5);
      const int64_t n = min(j0 + 32 * x + (lane & 31), at.lk - 1);
      Vec8<T> none;
#pragma unroll
      for (int e = 0; e < 8; ++e) none[e] = (T)0.0f;
      kf[x][kk] = d < p.dim ? load8(K + n * p.k_tok + d) : none;
      if constexpr (VREG) vf[x][kk] = d < p.dim ? load8(V + n * p.v_tok + d) : none;
    }
  // (64 rows at a time: what a descriptor covers)
  constexpr int NV = 64 * DC / 512 / W;
#pragma unroll
  for (int b = 0; !VREG && b < BN / 64; ++b) {
    const Fetch<T, DC> f = Fetch<T, DC>::of(V, p.v_tok, at.tile * BN + 64 * b, at.lk, p.dim);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      f.issue(p.v_tok, p.dim, sv + 128 * b * DC, w * NV + j, lane);
  }
  floatx16 dk[KB][ND], dv[KB][ND];
#pragma unroll
  for (int x = 0; x < KB; ++x) {
    zero(dk[x]);
    zero(dv[x]);
  }

  // 32 rows of a stage in 4 KS KB slots of one matrix instruction each,
  // pinned in this order: S, dP, dV, dK.  Weight i of a key block is formed
  // under dP (i < 8) or the first half of dV, its score gradient under the
  // second half of dV (i < 8) or the first half of dK: what an instruction
  // takes is ready half a phase before, and the vector work is spread over
  // three of the four phases.  Fragments are read RA fragments ahead; the next
  // stage's loads are spread over the slots.
    constexpr int RA = 2, H = KS / 2;
  auto block = [&](const Reader<T, DC>& rd, const Reader<T, DC>& rv, const float* stat, int tb,
                   const Next& nx, lds_c to, int stage, auto masked) {
    floatx16 st[KB], dp[KB];
    const float* ps = stat + 4 * (lane >> 5);
    Vec8<T> fr[RA + 1], fv[RA + 1][KB], pf[KB][2], df[KB][2];
    // bit r: row r of the 32 (+ 4 in the upper half of the wave) sees the
    // lane's key
    unsigned rows[KB];
    if constexpr (decltype(masked)::value)
#pragma unroll
      for (int x = 0; x < KB; ++x)
        rows[x] = ~low_bits(j0 + 32 * x + (lane & 31) - off - tb - 4 * (lane >> 5));
    auto read = [&](int n) {
      if (n >= 4 * KS) return;
      const int ph = n / KS, kk = n % KS;
      Vec8<T>& f = fr[n % (RA + 1)];
      if (ph == 0) f = rd.straight(0, kk);
      if (ph == 1) f = rd.straight(0, kk, 2 * TILE);
      if (ph == 1 && !VREG)
#pragma unroll
        for (int x = 0; x < KB; ++x) fv[n % (RA + 1)][x] = rv.straight(x, kk);
      if (ph == 2) f = rd.transposed(kk / ND, kk % ND, 2 * TILE);
      if (ph == 3) f = rd.transposed(kk / ND, kk % ND);
    };
    // Vector work: unit u of 32 covers value u % 16; units 0 - 15 form the
    // weights, 16 - 31 the score gradients.  Unit 0 starts with dP's slot 0,
    // and a quarter of the units goes to each half phase (the first two
    // quarters' first eight values to all of dP).  Rows' log-sum-exps and
    // deltas come four at a time, read a group ahead.
    floatx4 stats[2];
    auto read_stats = [&](int g) {   // g 0 - 3: log-sum-exps, 4 - 7: deltas
      if (g < 8) stats[g % 2] = *(const floatx4*)(ps + (g / 4) * 64 + 8 * (g % 4));
    };
    auto unit = [&](int x, int u) {
      const int i = u % 16;
      if (u < 16) {
        float v = __builtin_amdgcn_exp2f(
            __builtin_fmaf(st[x][i], p.scale_log2, -stats[u / 4 % 2][i % 4]));
        if constexpr (decltype(masked)::value)
          v = select_bit(rows[x], 8 * (i / 4) + i % 4, v, 0.0f);
        st[x][i] = v;
      } else {
        dp[x][i] = st[x][i] * (dp[x][i] - stats[u / 4 % 2][i % 4]);
      }
      if (i % 8 == 7) {
        Vec8<T>& f = u < 16 ? pf[x][i / 8] : df[x][i / 8];
        f = pack8<T>(u < 16 ? st[x] : dp[x], i / 8);
        asm volatile("" : "+v"(f));   // here, not where it is used
      }
    };
    // units of slot n's frag: 8 over dP's KS, then 8 over each half phase
    auto units_from = [&](int n) {
      const int m = n - KS;
      return m <= 0 ? 0 : m <= KS ? 8 * m / KS : m >= 2 * KS + H ? 32 : 8 + 8 * (m - KS) / H;
    };
    auto load_at = [&](int n) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if ((2 * j + 1) * 4 * KS / (2 * PER) == n) issue(nx, to, stage, j);
    };
    // Before the first use of st (dp): its last instruction has run for the
    // 8 passes that the first of the next product waited for the matrix pipe,
    // and for 16 more here, with KB = 2 for 8 passes of the other key block's
    // too (19 are asked for).
    auto scores_done = [&](floatx16(&z)[KB]) {
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (KB == 1)
        asm volatile("s_nop 7\n\ts_nop 7" : "+v"(z[0]));
      else
        asm volatile("s_nop 7\n\ts_nop 7" : "+v"(z[0]), "+v"(z[KB - 1]));
      __builtin_amdgcn_sched_barrier(0);
    };
    // after the matrix instruction of slot (n, x): its share of vector work
    // and loads
    auto fill = [&](int n, int x) {
#pragma unroll
      for (int u = units_from(n); u < units_from(n + 1); ++u) {
        if (x == 0 && u % 4 == 0) read_stats(u / 4 + 1);
        unit(x, u);
      }
      if (x == KB - 1) load_at(n);
      __builtin_amdgcn_sched_barrier(0);
    };
    read_stats(0);
#pragma unroll
    for (int n = 0; n < RA; ++n) read(n);
#pragma unroll
    for (int m = 0; m < KS; ++m) {
      read(m + RA);
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        if (m == 0)
          Elem<T>::mma_begin(fr[0], kf[x][0], st[x]);
        else
          Elem<T>::mma_add(fr[m % (RA + 1)], kf[x][m], st[x]);
        fill(m, x);
      }
    }
#pragma unroll
    for (int m = 0; m < KS; ++m) {
      const int n = KS + m;
      read(n + RA);
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        const Vec8<T>& vx = VREG ? vf[VREG ? x : 0][VREG ? m : 0] : fv[n % (RA + 1)][x];
        if (m == 0)
          Elem<T>::mma_begin(fr[n % (RA + 1)], vx, dp[x]);
        else
          Elem<T>::mma_add(fr[n % (RA + 1)], vx, dp[x]);
        if (m == 0 && x == 0) scores_done(st);
        fill(n, x);
      }
    }
#pragma unroll
    for (int m = 0; m < KS; ++m) {
      const int n = 2 * KS + m;
      read(n + RA);
      if (KB == 1 && m == H) asm volatile("s_nop 1");   // pf[0][1] is a slot old
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        Elem<T>::mma_tied(fr[n % (RA + 1)], pf[x][m / ND], dv[x][m % ND]);
        if (m == H && x == 0) scores_done(dp);
        fill(n, x);
      }
    }
#pragma unroll
    for (int m = 0; m < KS; ++m) {
      const int n = 3 * KS + m;
      read(n + RA);
      if (KB == 1 && m % H == 0) asm volatile("s_nop 1");
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        Elem<T>::mma_tied(fr[n % (RA + 1)], df[x][m / ND], dk[x][m % ND]);
        fill(n, x);
      }
    }
  };

  const Reader<T, DC> reader = Reader<T, DC>::of(lane);
  // step it, while step it + NST - 1 is fetched; every step issues PER loads
  auto step = [&](int it, lds_c __restrict__ from, lds_c __restrict__ to, auto masked) {
    if (it == hidden(0)) {
#pragma unroll
      for (int s = 0; s < NST - 1; ++s) {
        const Next nx = advance();
#pragma unroll
        for (int j = 0; j < PER; ++j) issue(nx, to + 4 * s * TILE, s, j);
      }
    }
    wait_vm<(NST - 2) * PER>();
    barrier();
    const Next nx = advance();
    const int stage = (it + NST - 1) % NST;
    block(reader.at(from, 64 * DC * rw), reader.at(sv, 64 * DC * KB * kw),
          &sstat[it % NST][0][32 * rw], now.c * RC + 32 * rw, nx, to + stage * 4 * TILE, stage,
          masked);
  };
  // the sums may be moved or read from here on
  auto settled = [&]() {
    settle();
#pragma unroll
    for (int x = 0; x < KB; ++x)
#pragma unroll
      for (int db = 0; db < ND; ++db) asm volatile("" : "+a"(dk[x][db]), "+a"(dv[x][db]));
  };
  // (settled inside the conditions: where the paths meet is too late)
  int it = 0;
  if (it < cut_here) {
    do {
      step(it, ring + it % NST * 4 * TILE, ring, BoolC<true>{});
      move(now);
    } while (++it < cut_here);
    settled();
  }
  if (it < steps) {
    do {
      step(it, ring + it % NST * 4 * TILE, ring, BoolC<false>{});
    } while (++it < steps);
    settled();
  }
  wait_vm<0>();
  // the row groups' sums: group 0 adds the others', register by register
  if constexpr (RW > 1) {
    floatx4* sums = (floatx4*)smem;
    auto add = [&](floatx16 (&x)[ND]) {
      __syncthreads();
      if (rw > 0) {
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sums[((w - KW) * ND * 4 + 4 * db + q) * 64 + lane] =
                floatx4{x[db][4 * q], x[db][4 * q + 1], x[db][4 * q + 2], x[db][4 * q + 3]};
      }
      __syncthreads();
      if (rw == 0) {
#pragma unroll
        for (int g = 0; g < RW - 1; ++g)
#pragma unroll
          for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const floatx4 y = sums[((g * KW + w) * ND * 4 + 4 * db + q) * 64 + lane];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[db][4 * q + e] += y[e];
            }
      }
    };
#pragma unroll
    for (int x = 0; x < KB; ++x) {
      add(dk[x]);
      add(dv[x]);
    }
  }
  const bool whole = steps == all.steps;
#pragma unroll
  for (int x = 0; x < KB; ++x) {
    const int key = j0 + 32 * x + (lane & 31);
    const bool valid = key < at.lk && rw == 0;
    const int64_t n = (int64_t)at.k0 + min(key, at.lk - 1);
    if (!whole) {
      float* o = part + (32 * KB * kw + 32 * x + (lane & 31)) * DC + 4 * (lane >> 5);
      if (valid)
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            *(floatx4*)(o + 32 * db + 8 * q) =
                floatx4{dk[x][db][4 * q], dk[x][db][4 * q + 1], dk[x][db][4 * q + 2],
                        dk[x][db][4 * q + 3]};
            *(floatx4*)(o + BN * DC + 32 * db + 8 * q) =
                floatx4{dv[x][db][4 * q], dv[x][db][4 * q + 1], dv[x][db][4 * q + 2],
                        dv[x][db][4 * q + 3]};
          }
    } else {
      store_row<T, DC>((T*)p.dk + n * p.dk_tok + kvh * p.dk_head, dk[x], p.scale, p.dim, lane,
                       valid);
      store_row<T, DC>((T*)p.dv + n * p.dv_tok + kvh * p.dv_head, dv[x], 1.0f, p.dim, lane, valid);
    }
  }
}

// A workgroup per kv head and share, or, where there are tiles enough to fill
// the chip many times (p.shares = 0), per tile.
template <class T, int DC, int KW, int RW, int KB>
__global__ void __launch_bounds__(64 * KW * RW) attention_dkv(const BwdParams p) {
  using S = DkvShape<T, DC, KW, RW, KB>;
  constexpr int BN = S::BN, RC = S::RC;
  // one object: with a second one the compiler's bookkeeping of direct-to-LDS
  // loads makes every read wait for all of them
  __shared__ __attribute__((aligned(4096))) T smem[S::ELEMS];
  const int kvh = blockIdx.x % p.heads_kv, w = blockIdx.x / p.heads_kv;
  const int parts = p.shares ? p.shares : p.slots_k;
  if (p.seq_k) {            // keys behind the last sequence
    const int end = min(max(p.seq_k[p.batch], 0), p.total_k);
    const int64_t rest = p.total_k - end;
    const int64_t from = end + rest * w / parts, to = end + rest * (w + 1) / parts;
    zero_rows<T>((T*)p.dk, p.dk_tok, p.dk_head, 1, kvh, from, to, p.dim, 64 * S::W);
    zero_rows<T>((T*)p.dv, p.dv_tok, p.dv_head, 1, kvh, from, to, p.dim, 64 * S::W);
  }
  BwdPlace at;
  int64_t u = 0, end = 0, base = 0;     // units left: [u, end); base: the sequence's first
  int64_t each = 0;
  int s = 0;
  if (p.shares) {
    const int64_t total = find_units(p, 0, BN, RC).total;
    each = dkv_each(total, p.shares);
    u = w * each;
    end = min(u + each, total);
    if (kvh == 0 && threadIdx.x == 0) p.cuts[w] = DkvCut{0, 0, 0, 0};
    if (u >= end) return;
    const DkvFound f = find_units(p, u, BN, RC);
    s = f.s;
    base = f.base;
    const Lens l = lens_of(p, s);
    at = BwdPlace{uniform(l.q0), uniform(l.lq), uniform(l.k0), uniform(l.lk), 0, 0, true};
    at.tile = uniform(
        find_tile(units_of(p, at.lq, at.lk, BN, RC), (at.lk + BN - 1) / BN, u - base));
  } else {
    at = bwd_place(p, w, BN, false);
    if (!at.any) return;
  }
  for (;;) {
    const DkvSteps all = dkv_steps(p, at.lq, at.lk, at.tile, BN, RC);
    int first = 0, steps = all.steps;
    bool mine = true;
    float* part = nullptr;
    if (p.shares) {
      const int64_t a = base + units_of(p, at.lq, at.lk, BN, RC).before(at.tile) + kDkvFixed;
      first = uniform((int)max(u - a, (int64_t)0));
      steps = uniform((int)(min(max(end - a, (int64_t)0), (int64_t)all.steps) - first));
      mine = all.steps ? steps > 0 : u <= a - kDkvFixed;
      const int number = at.k0 / BN + s + at.tile;
      part = p.partials + (dkv_place(p, w, number, u <= a) * p.heads_kv + kvh) * (2 * BN * DC);
      if (u <= a && steps > 0 && steps < all.steps && kvh == 0 && threadIdx.x == 0)
        p.cuts[w] = DkvCut{at.k0 + at.tile * BN, min(BN, at.lk - at.tile * BN),
                           (int)((a + all.steps - 1) / each), number};
      u = a + all.steps;
    }
    if (mine) dkv_tile<T, DC, KW, RW, KB>(p, smem, at, kvh, all, first, steps, part);
    if (u >= end) return;
    if (++at.tile * (int64_t)BN >= at.lk) {
      Lens l;
      base = u;
      do l = lens_of(p, ++s);           // (there are units left, so there is one)
      while (l.lk == 0);
      at = BwdPlace{uniform(l.q0), uniform(l.lq), uniform(l.k0), uniform(l.lk), 0, 0, true};
    }
    __syncthreads();                    // the tile's reads of LDS are done
  }
}

// The sums of the tile that a share cut off at its end, over the shares that
// it went on in, in order; a workgroup per share, kv head and 32 keys, 8
// elements of dK and dV per thread and turn.
template <class T, int DC>
__global__ void __launch_bounds__(256) attention_dkv_join(const BwdParams p, int bn) {
  int bid = blockIdx.x;
  const int kvh = bid % p.heads_kv;
  bid /= p.heads_kv;
  const int w = bid / (bn / 32);
  const DkvCut cut = p.cuts[w];
  const int w1 = cut.last;
  const int j0 = 32 * (bid % (bn / 32)), per = p.dim / 8;
  for (int i = threadIdx.x; i < min(32, cut.keys - j0) * per; i += 256) {
    const int key = j0 + i / per, d = 8 * (i % per);
    float k[8] = {}, v[8] = {};
    for (int g0 = w; g0 <= w1; g0 += 4) {     // four parts in flight
      floatx4 y[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int g = min(g0 + j, w1);
        const float* o = p.partials +
                         (dkv_place(p, g, cut.number, g == w) * p.heads_kv + kvh) *
                             (2 * bn * DC) +
                         key * DC + d;
        y[j][0] = *(const floatx4*)o;
        y[j][1] = *(const floatx4*)(o + 4);
        y[j][2] = *(const floatx4*)(o + bn * DC);
        y[j][3] = *(const floatx4*)(o + bn * DC + 4);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (g0 + j <= w1)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            k[e] += y[j][e / 4][e % 4];
            v[e] += y[j][2 + e / 4][e % 4];
          }
    }
    Vec8<T> y, z;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = (T)(k[e] * p.scale);
      z[e] = (T)v[e];
    }
    const int64_t n = (int64_t)cut.key + key;
    *(Vec8<T>*)((T*)p.dk + n * p.dk_tok + kvh * p.dk_head + d) = y;
    *(Vec8<T>*)((T*)p.dv + n * p.dv_tok + kvh * p.dv_head + d) = z;
  }
}

}  // namespace att
}  // namespace mfl
