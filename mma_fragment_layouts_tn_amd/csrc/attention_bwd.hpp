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
  const int first_row_limit = uniform(row.limit);
  const int last_t = min((int)(((int64_t)at.tile * BM + BM - 1) / p.group), at.lq - 1);
  const int seen = max(p.causal ? min(last_t + at.lk - at.lq, at.lk - 1) + 1 : at.lk, 0);
  const int chunks = (seen + CK - 1) / CK;
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
  auto step = [&](int c, lds_c __restrict__ from, lds_c __restrict__ to) {
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
      if (key0 + 31 > first_row_limit) mask_keys(st, key0, row.limit, lane);
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
  for (int c = 0; c < chunks; ++c) step(c, ring + c % NST * 4 * TILE, ring);
  wait_vm<0>();
  store_row<T, DC>((T*)p.dq + row.n * p.dq_tok + row.head * p.dq_head, acc, p.scale, p.dim, lane,
                   row.valid);
}

// ------------------------------------------------------------- dK and dV
// KW x RW waves: wave w holds the 32 keys of key group w % KW and takes block
// w / KW of each chunk's 32-row blocks; the row groups' sums are added in LDS
// at the end.  Chunks of RC query tokens of one head at a time,
// over the heads of the group.  Scores come with the rows in the registers
// and the key in the lane (S = Q K^T, A operand from LDS), so P and dS are
// the B operands of dV^T = dO^T P and dK^T = Q^T dS as they are.
//
// A tile's steps (chunks of all heads) are shared out over as many workgroups
// as dkv_parts() says, in order; with more than one, their sums go to the
// workspace and attention_dkv_join adds them in order.
template <int DC>
MFL_HD constexpr int dkv_rows() { return DC == 256 ? 32 : 64; }

struct DkvSteps {
  int t0, per_head, steps, parts;
};
// first token that sees the tile's first key, chunks per head, chunks in all,
// workgroups they are shared out over
__device__ __forceinline__ DkvSteps dkv_steps(const BwdParams& p, const BwdPlace& at, int bn,
                                              int rc) {
  DkvSteps r;
  r.t0 = p.causal ? max(at.tile * bn - (at.lk - at.lq), 0) / rc * rc : 0;
  r.per_head = r.t0 < at.lq ? (at.lq - r.t0 + rc - 1) / rc : 0;
  r.steps = r.per_head * p.group;
  r.parts = min(max((r.steps + p.part_steps - 1) / p.part_steps, 1), p.max_parts);
  return r;
}

template <class T, int DC, int KW, int RW>
__global__ void __launch_bounds__(64 * KW * RW) attention_dkv(const BwdParams p) {
  constexpr int W = KW * RW, NST = DC == 64 ? 4 : DC == 128 ? 3 : 2, BN = 32 * KW,
                RC = dkv_rows<DC>(), KS = DC / 16, ND = DC / 32, TILE = RC * DC,
                NI = TILE / 512 / W, PER = 2 * NI + 1;   // loads per wave and stage
  static_assert(RC == 32 * RW, "every row group has a block of each chunk");
  static_assert(RW == 1 || (RW - 1) * KW * 32 * DC * 4 <= NST * 4 * TILE, "sums fit in the stages");
  // one object: with a second one the compiler's bookkeeping of direct-to-LDS
  // loads makes every read wait for all of them
  __shared__ __attribute__((aligned(4096))) T smem[NST * 2 * TILE + BN * DC + NST * 256];
  float(*sstat)[2][64] = (float(*)[2][64])(smem + NST * 2 * TILE + BN * DC);
  const lds_c ring = (lds_c)smem, sv = ring + NST * 4 * TILE;   // sv: the tile's V, for all steps
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
  const int first = (int)((int64_t)all.steps * part / all.parts);
  const int steps = (int)((int64_t)all.steps * (part + 1) / all.parts) - first;
  const int j0 = at.tile * BN + 32 * kw, off = at.lk - at.lq, t0 = all.t0;
  // The step fetched next.  Chunks start at multiples of RC and are walked
  // from the sequence's end, so the workgroups of one head, whose first tokens
  // differ, fetch the same chunks at the same time.
  const int t_last = (at.lq - 1) / RC * RC;
  int next = 0, next_head = kvh * p.group, next_t = t_last;
  if (all.per_head > 0) {
    next_head += first / all.per_head;
    next_t -= first % all.per_head * RC;
  }
  int t = next_t;
  struct Next {
    Fetch<T, DC> q, g;
    __amdgpu_buffer_rsrc_t stat;
    int stage;
  };
  auto advance = [&]() {
    const int end = next < steps ? at.lq : 0;
    Next n;
    n.stage = next % NST;
    n.q = Fetch<T, DC>::of((const T*)p.q + (int64_t)at.q0 * p.q_tok + next_head * p.q_head, p.q_tok,
                           next_t, end, p.dim);
    n.g = Fetch<T, DC>::of((const T*)p.dout + (int64_t)at.q0 * p.do_tok + next_head * p.do_head,
                           p.do_tok, next_t, end, p.dim);
    // even waves fetch the log-sum-exps, odd waves the deltas, 64 at a time
    // (several waves the same: every wave has as many loads in flight)
    n.stat = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.stats + ((int64_t)(w & 1) * heads + next_head) * p.total_q + at.q0 + next_t), 0,
        4 * max(min(end - next_t, 64), 0), 0x00027000);
    ++next;
    next_t -= RC;
    if (next_t < t0) {
      next_t = t_last;
      ++next_head;
    }
    return n;
  };
  auto issue = [&](const Next& n, lds_c to, int j) {
    if (j < NI)
      n.q.issue(p.q_tok, p.dim, to, w * NI + j, lane);
    else if (j < 2 * NI)
      n.g.issue(p.do_tok, p.dim, to + 2 * TILE, w * NI + j - NI, lane);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(n.stat, (lds_t)(&sstat[n.stage][w & 1][0]), 4,
                                               4u * lane, 0, 0, 0);
  };
  const int key = j0 + (lane & 31);
  const int64_t n = (int64_t)at.k0 + min(key, at.lk - 1);
  const T* K = (const T*)p.k + n * p.k_tok + (int64_t)kvh * p.k_head;
  Vec8<T> kf[KS];
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    const int d = 16 * kk + 8 * (lane >> 5);
    if (d < p.dim)
      kf[kk] = load8(K + d);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) kf[kk][e] = (T)0.0f;
  }
  const T* V = (const T*)p.v + (int64_t)at.k0 * p.v_tok + (int64_t)kvh * p.v_head;
  // (64 rows at a time: what a descriptor covers)
  constexpr int NV = 64 * DC / 512 / W;
#pragma unroll
  for (int b = 0; b < BN / 64; ++b) {
    const Fetch<T, DC> f = Fetch<T, DC>::of(V, p.v_tok, at.tile * BN + 64 * b, at.lk, p.dim);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      f.issue(p.v_tok, p.dim, sv + 128 * b * DC, w * NV + j, lane);
  }
  floatx16 dk[ND], dv[ND];
  zero(dk);
  zero(dv);

  // 32 rows of a stage, the tokens from tb on, in 4 KS slots of one matrix
  // instruction each, pinned in this order: S; dP, under which P is formed;
  // dV, under which dS is formed; dK.  Fragments are read RA slots ahead; the
  // next stage's loads are spread over the slots.
#ifndef RAV
#define RAV 2
#endif
  constexpr int RA = RAV;
  auto block = [&](const Reader<T, DC>& rd, const Reader<T, DC>& rv, const float* stat, int tb,
                   const Next& nx, lds_c to) {
    auto load_at = [&](int n) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if ((2 * j + 1) * 4 * KS / (2 * PER) == n) issue(nx, to, j);
    };
    floatx16 st, dp;
#pragma unroll
    for (int i = 0; i < 16; ++i) st[i] = dp[i] = 0.0f;
    const float* ps = stat + 4 * (lane >> 5);
    Vec8<T> fr[RA + 1], fv[RA + 1], pf[2], df[2];
    // values formed per slot of dP and dV, in groups of four with one read of
    // their rows' log-sum-exps and deltas
    // Bit r: row r of the 32 (+ 4 in the upper half of the wave) exists and
    // sees the lane's key.  Two instructions per weight in every block; as a
    // branch taken by the few blocks that need it, it made the compiler spill
    // accumulators.
    const int from = max((p.causal ? key - off - tb : 0) - 4 * (lane >> 5), 0);
    const int to_ = at.lq - tb - 4 * (lane >> 5);
    const unsigned rows = low_bits(to_) & ~low_bits(from);
    constexpr int E = 16 / KS, NQ = (RA * E + 3) / 4 + 1;
    floatx4 stats[NQ];
    auto read = [&](int n) {
      if (n >= 4 * KS) return;
      const int ph = n / KS, kk = n % KS;
      if ((ph == 1 || ph == 2) && kk * E % 4 == 0)
        stats[(4 * (ph - 1) + kk * E / 4) % NQ] =
            *(const floatx4*)(ps + (ph - 1) * 64 + 8 * (kk * E / 4));
      Vec8<T>& f = fr[n % (RA + 1)];
      if (ph == 0) f = rd.straight(0, kk);
      if (ph == 1) {
        f = rd.straight(0, kk, 2 * TILE);
        fv[n % (RA + 1)] = rv.straight(0, kk);
      }
      if (ph == 2) f = rd.transposed(kk / ND, kk % ND, 2 * TILE);
      if (ph == 3) f = rd.transposed(kk / ND, kk % ND);
    };
#pragma unroll
    for (int n = 0; n < RA; ++n) read(n);
#pragma unroll
    for (int n = 0; n < KS; ++n) {
      read(n + RA);
      st = Elem<T>::mma(fr[n % (RA + 1)], kf[n], st);
      load_at(n);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < KS; ++m) {
      const int n = KS + m;
      read(n + RA);
      dp = Elem<T>::mma(fr[n % (RA + 1)], fv[n % (RA + 1)], dp);
      load_at(n);
#pragma unroll
      for (int i = m * E; i < m * E + E; ++i)
        st[i] = select_bit(rows, 8 * (i / 4) + i % 4,
                           __builtin_amdgcn_exp2f(__builtin_fmaf(
                               st[i], p.scale_log2, -stats[i / 4 % NQ][i % 4])),
                           0.0f);
      if (m * E + E == 8) pf[0] = pack8<T>(st, 0);
      if (m * E + E == 16) pf[1] = pack8<T>(st, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < KS; ++m) {
      const int n = 2 * KS + m;
      read(n + RA);
      dv[m % ND] = Elem<T>::mma(fr[n % (RA + 1)], pf[m / ND], dv[m % ND]);
      load_at(n);
#pragma unroll
      for (int i = m * E; i < m * E + E; ++i)
        dp[i] = st[i] * (dp[i] - stats[(4 + i / 4) % NQ][i % 4]);
      if (m * E + E == 8) df[0] = pack8<T>(dp, 0);
      if (m * E + E == 16) df[1] = pack8<T>(dp, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < KS; ++m) {
      const int n = 3 * KS + m;
      read(n + RA);
      dk[m % ND] = Elem<T>::mma(fr[n % (RA + 1)], df[m / ND], dk[m % ND]);
      load_at(n);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  const Reader<T, DC> reader = Reader<T, DC>::of(lane);
  // step it on the tokens from t on, while step it + NST - 1 is fetched; every
  // step issues PER loads
  auto step = [&](int it, lds_c __restrict__ from, lds_c __restrict__ to,
                  lds_c __restrict__ values) {
    if (it == hidden(0)) {
#pragma unroll
      for (int s = 0; s < NST - 1; ++s) {
        const Next nx = advance();
#pragma unroll
        for (int j = 0; j < PER; ++j) issue(nx, to + 4 * s * TILE, j);
      }
    }
    wait_vm<(NST - 2) * PER>();
    barrier();
    const Next nx = advance();
    block(reader.at(from, 64 * DC * rw), reader.at(values, 64 * DC * kw), &sstat[it % NST][0][32 * rw],
          t + 32 * rw, nx, to + (it + NST - 1) % NST * 4 * TILE);
  };
  for (int it = 0; it < steps; ++it) {
    step(it, ring + it % NST * 4 * TILE, ring, sv);
    t = t - RC < t0 ? t_last : t - RC;
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
    add(dk);
    add(dv);
    if (rw > 0) return;
  }
  const bool valid = key < at.lk;
  if (all.parts > 1) {
    const int64_t stride = (int64_t)p.total_k * p.heads_kv * DC;
    float* o = p.partials + 2 * part * stride + (n * p.heads_kv + kvh) * DC + 4 * (lane >> 5);
    if (valid)
#pragma unroll
      for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          *(floatx4*)(o + 32 * db + 8 * q) = floatx4{dk[db][4 * q], dk[db][4 * q + 1],
                                                     dk[db][4 * q + 2], dk[db][4 * q + 3]};
          *(floatx4*)(o + stride + 32 * db + 8 * q) = floatx4{
              dv[db][4 * q], dv[db][4 * q + 1], dv[db][4 * q + 2], dv[db][4 * q + 3]};
        }
    return;
  }
  store_row<T, DC>((T*)p.dk + n * p.dk_tok + kvh * p.dk_head, dk, p.scale, p.dim, lane, valid);
  store_row<T, DC>((T*)p.dv + n * p.dv_tok + kvh * p.dv_head, dv, 1.0f, p.dim, lane, valid);
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
