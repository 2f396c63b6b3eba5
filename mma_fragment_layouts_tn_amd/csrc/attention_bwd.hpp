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
template <int DC>
MFL_HD constexpr int dq_waves() { return DC == 256 ? 4 : 8; }
template <int DC>
MFL_HD constexpr int dq_stages() { return DC == 256 ? 2 : 4; }

template <class T, int DC>
__global__ void __launch_bounds__(64 * dq_waves<DC>()) attention_dq(const BwdParams p) {
  constexpr int W = dq_waves<DC>(), NST = dq_stages<DC>(), BM = 32 * W, CK = 64, KS = DC / 16,
                ND = DC / 32, TILE = CK * DC, NI = TILE / 512 / W;
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
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int key0 = c * CK + 32 * b;
      floatx16 st[1], dp[1];
      zero(st);
      zero(dp);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) st[0] = Elem<T>::mma(rd.straight(b, kk), qf[kk], st[0]);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        dp[0] = Elem<T>::mma(rd.straight(b, kk, 2 * TILE), gf[kk], dp[0]);
#pragma unroll
        for (int j = 0; j < NI; ++j)
          if ((2 * j + 1) * KS / (2 * NI) == kk) {
            pin_loads();
            issue(nx, fill, b * NI + j);
            pin_loads();
          }
      }
      if constexpr (decltype(masked)::value) mask_keys(st, key0, row.limit, lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float w_ = __builtin_amdgcn_exp2f(__builtin_fmaf(st[0][i], p.scale_log2, -lse2));
        st[0][i] = w_ * (dp[0][i] - delta);
      }
#pragma unroll
      for (int kc = 0; kc < 2; ++kc) {
        const Vec8<T> df = pack8<T>(st[0], kc);
#pragma unroll
        for (int db = 0; db < ND; ++db)
          acc[db] = Elem<T>::mma(rd.transposed(2 * b + kc, db), df, acc[db]);
      }
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
// With KB = 2 a wave's sums take all 256 accumulation registers, one wave per
// SIMD, and K and V of the tile stay in LDS.  Two waves of 32 keys each instead issue twice the LDS
// reads, waits and scalar instructions per matrix instruction, and those, not
// the matrix pipe, set their pace: 4,600 cycles for 2,048 of matrix work.
//
// A tile's steps (chunks of all heads) are shared out over as many workgroups
// as dkv_steps() says, in order; with more than one, their sums go to the
// workspace and attention_dkv_join adds them in order.  The chunks that the
// causal mask cuts come first, in a loop of their own: the mask as a branch
// inside one loop made the compiler spill accumulators.
struct DkvSteps {
  int first, cut, last;     // chunks: first that sees the tile, first without
                            // hidden keys, last of the sequence
  int steps, parts;
};
__device__ __forceinline__ DkvSteps dkv_steps(const BwdParams& p, const BwdPlace& at, int bn,
                                              int rc) {
  DkvSteps r;
  const int off = at.lk - at.lq, j0 = at.tile * bn;
  r.last = (at.lq + rc - 1) / rc - 1;
  r.first = r.cut = 0;
  if (p.causal) {           // token t sees the keys up to t + off
    r.first = max(j0 - off, 0) / rc;
    r.cut = max((max(j0 + bn - 1 - off, 0) + rc - 1) / rc, r.first);
    r.first = min(r.first, r.last + 1);
    r.cut = min(r.cut, r.last + 1);
  }
  r.steps = (r.last + 1 - r.first) * p.group;
  r.parts = min(max((r.steps + p.part_steps - 1) / p.part_steps, 1), p.max_parts);
  return r;
}

template <class T, int DC, int KW, int RW, int KB>
__global__ void __launch_bounds__(64 * KW * RW) attention_dkv(const BwdParams p) {
  // the tile's K and V in registers (else in LDS for all steps)
  constexpr bool KREG = true, VREG = DC == 64;
  constexpr int W = KW * RW, NST = DC == 256 ? 2 : 4, BN = 32 * KW * KB, RC = 32 * RW,
                KS = DC / 16, ND = DC / 32, TILE = RC * DC, NI = TILE / 512 / W,
                PER = 2 * NI + 1;                        // loads per wave and stage
  static_assert(KB <= 2 && NI >= 1, "key blocks, loads");
  static_assert((RW - 1) * KW * 32 * DC * 4 <= NST * 4 * TILE, "sums fit in the stages");
  // one object: with a second one the compiler's bookkeeping of direct-to-LDS
  // loads makes every read wait for all of them
  constexpr int HELD = (KREG ? 0 : 1) + (VREG ? 0 : 1);
  __shared__ __attribute__((aligned(4096))) T smem[NST * 2 * TILE + HELD * BN * DC + NST * 256];
  float(*sstat)[2][64] = (float(*)[2][64])(smem + NST * 2 * TILE + HELD * BN * DC);
  const lds_c ring = (lds_c)smem, sv = ring + NST * 4 * TILE,
              sk = sv + (VREG ? 0 : 2 * BN * DC);
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6), kw = w % KW, rw = w / KW;
  int bid = blockIdx.x;
  const int kvh = bid % p.heads_kv, heads = p.heads_kv * p.group;
  bid /= p.heads_kv;
  // the tiles' last parts first: only the longest tiles have them
  const int slot = bid % p.slots_k, part = p.max_parts - 1 - bid / p.slots_k;
  const BwdPlace at = bwd_place(p, slot, BN, false);
  if (!at.any) {
    if (at.spare >= 0 && part == 0) {
      const int64_t from =
          (int64_t)min(max(p.seq_k[p.batch], 0), p.total_k) + (int64_t)at.spare * BN;
      const int64_t to = min(from + BN, (int64_t)p.total_k);
      zero_rows<T>((T*)p.dk, p.dk_tok, p.dk_head, 1, kvh, from, to, p.dim, 64 * W);
      zero_rows<T>((T*)p.dv, p.dv_tok, p.dv_head, 1, kvh, from, to, p.dim, 64 * W);
    }
    return;
  }
  const DkvSteps all = dkv_steps(p, at, BN, RC);
  if (part >= all.parts) return;
  const int first = uniform((int)((int64_t)all.steps * part / all.parts));
  const int steps = uniform((int)((int64_t)all.steps * (part + 1) / all.parts)) - first;
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
  Vec8<T> kf[KREG ? KB : 1][KREG ? KS : 1], vf[VREG ? KB : 1][VREG ? KS : 1];
#pragma unroll
  for (int x = 0; x < KB; ++x)
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int d = 16 * kk + 8 * (lane >> 5);
      const int64_t n = min(j0 + 32 * x + (lane & 31), at.lk - 1);
      Vec8<T> none;
#pragma unroll
      for (int e = 0; e < 8; ++e) none[e] = (T)0.0f;
      if constexpr (KREG) kf[x][kk] = d < p.dim ? load8(K + n * p.k_tok + d) : none;
      if constexpr (VREG) vf[x][kk] = d < p.dim ? load8(V + n * p.v_tok + d) : none;
    }
  // (64 rows at a time: what a descriptor covers)
  constexpr int NV = 64 * DC / 512 / W;
#pragma unroll
  for (int b = 0; b < BN / 64; ++b) {
    const Fetch<T, DC> f = Fetch<T, DC>::of(V, p.v_tok, at.tile * BN + 64 * b, at.lk, p.dim);
    const Fetch<T, DC> g = Fetch<T, DC>::of(K, p.k_tok, at.tile * BN + 64 * b, at.lk, p.dim);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!VREG) f.issue(p.v_tok, p.dim, sv + 128 * b * DC, w * NV + j, lane);
      if (!KREG) g.issue(p.k_tok, p.dim, sk + 128 * b * DC, w * NV + j, lane);
    }
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
      if ((ph == 0 && !KREG) || (ph == 1 && !VREG))
#pragma unroll
        for (int x = 0; x < KB; ++x)
          fv[n % (RA + 1)][x] = rv.straight(x, kk, ph == 0 ? (int)(sk - sv) : 0);
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
        const Vec8<T>& kx = KREG ? kf[KREG ? x : 0][KREG ? m : 0] : fv[m % (RA + 1)][x];
        if (m == 0)
          Elem<T>::mma_begin(fr[0], kx, st[x]);
        else
          Elem<T>::mma_add(fr[m % (RA + 1)], kx, st[x]);
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
    if (rw > 0) return;
  }
#pragma unroll
  for (int x = 0; x < KB; ++x) {
    const int key = j0 + 32 * x + (lane & 31);
    const bool valid = key < at.lk;
    const int64_t n = (int64_t)at.k0 + min(key, at.lk - 1);
    if (all.parts > 1) {
      const int64_t stride = (int64_t)p.total_k * p.heads_kv * DC;
      float* o = p.partials + 2 * part * stride + (n * p.heads_kv + kvh) * DC + 4 * (lane >> 5);
      if (valid)
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            *(floatx4*)(o + 32 * db + 8 * q) =
                floatx4{dk[x][db][4 * q], dk[x][db][4 * q + 1], dk[x][db][4 * q + 2],
                        dk[x][db][4 * q + 3]};
            *(floatx4*)(o + stride + 32 * db + 8 * q) =
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

// The parts' sums of a tile whose steps were shared out, in part order; a
// workgroup per tile, kv head and 32 keys, 8 elements of dK and dV per thread
// and turn.
template <class T, int DC>
__global__ void __launch_bounds__(256) attention_dkv_join(const BwdParams p, int bn, int rc) {
  int bid = blockIdx.x;
  const int kvh = bid % p.heads_kv;
  bid /= p.heads_kv;
  const BwdPlace at = bwd_place(p, bid / (bn / 32), bn, false);
  if (!at.any) return;
  const int parts = dkv_steps(p, at, bn, rc).parts;
  if (parts == 1) return;
  const int j0 = at.tile * bn + 32 * (bid % (bn / 32)), per = p.dim / 8;
  const int64_t stride = (int64_t)p.total_k * p.heads_kv * DC;
  for (int x = threadIdx.x; x < min(32, at.lk - j0) * per; x += 256) {
    const int64_t n = (int64_t)at.k0 + j0 + x / per;
    const int d = 8 * (x % per);
    const float* i = p.partials + (n * p.heads_kv + kvh) * DC + d;
    float k[8] = {}, v[8] = {};
    for (int g = 0; g < parts; ++g, i += 2 * stride)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        k[e] += i[e];
        v[e] += i[stride + e];
      }
    Vec8<T> a, b;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = (T)(k[e] * p.scale);
      b[e] = (T)v[e];
    }
    *(Vec8<T>*)((T*)p.dk + n * p.dk_tok + kvh * p.dk_head + d) = a;
    *(Vec8<T>*)((T*)p.dv + n * p.dv_tok + kvh * p.dv_head + d) = b;
  }
}

}  // namespace att
}  // namespace mfl
