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
  const int wave_limit =
      r0 < at.lq * p.group ? __builtin_amdgcn_readlane(row.limit, 31) : -1;
  const int last_t = min((int)(((int64_t)at.tile * BM + BM - 1) / p.group), at.lq - 1);
  const int seen = max(p.causal ? min(last_t + at.lk - at.lq, at.lk - 1) + 1 : at.lk, 0);
  const int chunks = (seen + CK - 1) / CK;
  const T* K = (const T*)p.k + (int64_t)at.k0 * p.k_tok + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + (int64_t)at.k0 * p.v_tok + (int64_t)kvh * p.v_head;
  auto issue = [&](int c) {
    if (c >= chunks) return;
    T* st = smem + (c % NST) * 2 * TILE;
#pragma unroll
    for (int j = 0; j < NI; ++j)
      Fetch<T, DC>::issue(K, p.k_tok, c * CK, at.lk, p.dim, st, w * NI + j, lane);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      Fetch<T, DC>::issue(V, p.v_tok, c * CK, at.lk, p.dim, st + TILE, w * NI + j, lane);
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

#pragma unroll
  for (int s = 0; s < NST - 1; ++s) issue(s);
  for (int c = 0; c < chunks; ++c) {
    const int ahead = min(chunks - 1 - c, NST - 2);
    if (ahead >= 2) wait_vm<(NST > 3 ? 2 : 0) * 2 * NI>();
    else if (ahead == 1) wait_vm<(NST > 2 ? 1 : 0) * 2 * NI>();
    else wait_vm<0>();
    barrier();
    issue(c + NST - 1);
    const T* sk = smem + (c % NST) * 2 * TILE;
    const T* sv = sk + TILE;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int key0 = c * CK + 32 * b;
      if (key0 > wave_limit) break;
      floatx16 st[1], dp[1];
      zero(st);
      zero(dp);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
        st[0] = Elem<T>::mma(
            frag<T, DC>(sk, 32 * b + (lane & 31), 16 * kk + 8 * (lane >> 5)), qf[kk], st[0]);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
        dp[0] = Elem<T>::mma(
            frag<T, DC>(sv, 32 * b + (lane & 31), 16 * kk + 8 * (lane >> 5)), gf[kk], dp[0]);
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
          acc[db] =
              Elem<T>::mma(frag_tr<T, DC>(sk, 32 * b + 16 * kc, 32 * db, lane), df, acc[db]);
      }
    }
  }
  store_row<T, DC>((T*)p.dq + row.n * p.dq_tok + row.head * p.dq_head, acc, p.scale, p.dim, lane,
                   row.valid);
}

// ------------------------------------------------------------- dK and dV
// W waves of 32 keys; chunks of RC query tokens of one head at a time, over
// the heads of the group.  Scores come with the rows in the registers and the
// key in the lane (S = Q K^T, A operand from LDS), so P and dS are the B
// operands of dV^T = dO^T P and dK^T = Q^T dS as they are.
template <int DC>
MFL_HD constexpr int dkv_waves() { return 4; }
template <int DC>
MFL_HD constexpr int dkv_rows() { return DC == 256 ? 32 : 64; }

template <class T, int DC>
__global__ void __launch_bounds__(64 * dkv_waves<DC>()) attention_dkv(const BwdParams p) {
  constexpr int W = dkv_waves<DC>(), NST = DC == 64 ? 4 : 3, BN = 32 * W, RC = dkv_rows<DC>(),
                KS = DC / 16, ND = DC / 32, TILE = RC * DC, NI = TILE / 512 / W,
                PER = 2 * NI + 1;                        // loads per wave and stage
  __shared__ __attribute__((aligned(1024))) T smem[NST * 2 * TILE];
  __shared__ __attribute__((aligned(256))) float sstat[NST][2][64];
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int kvh = blockIdx.x % p.heads_kv, heads = p.heads_kv * p.group;
  const int slot = blockIdx.x / p.heads_kv;
  const BwdPlace at = bwd_place(p, slot, BN, false);
  if (!at.any) {
    if (at.spare >= 0) {
      const int64_t from = (int64_t)min(max(p.seq_k[p.batch], 0), p.total_k) + at.spare * BN;
      const int64_t to = min(from + BN, (int64_t)p.total_k);
      zero_rows<T>((T*)p.dk, p.dk_tok, p.dk_head, 1, kvh, from, to, p.dim, 64 * W);
      zero_rows<T>((T*)p.dv, p.dv_tok, p.dv_head, 1, kvh, from, to, p.dim, 64 * W);
    }
    return;
  }
  const int j0 = at.tile * BN + 32 * w, off = at.lk - at.lq;
  const int key = j0 + (lane & 31), held = min(key, at.lk - 1);
  // first token that sees the workgroup's first key
  const int t0 = p.causal ? max(at.tile * BN - off, 0) : 0;
  const int per_head = t0 < at.lq ? (at.lq - t0 + RC - 1) / RC : 0;
  const int steps = per_head * p.group;
  auto issue = [&](int it) {
    if (it >= steps) return;
    const int g = it / per_head, t = t0 + (it - g * per_head) * RC, head = kvh * p.group + g;
    T* st = smem + (it % NST) * 2 * TILE;
    const T* Q = (const T*)p.q + (int64_t)at.q0 * p.q_tok + head * p.q_head;
    const T* G = (const T*)p.dout + (int64_t)at.q0 * p.do_tok + head * p.do_head;
#pragma unroll
    for (int j = 0; j < NI; ++j)
      Fetch<T, DC>::issue(Q, p.q_tok, t, at.lq, p.dim, st, w * NI + j, lane);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      Fetch<T, DC>::issue(G, p.do_tok, t, at.lq, p.dim, st + TILE, w * NI + j, lane);
    // even waves fetch the log-sum-exps, odd waves the deltas, 64 at a time
    // (two waves the same: every wave has as many loads in flight)
    const int n = t + lane, which = w & 1;
    const float* src =
        p.stats + ((int64_t)which * heads + head) * p.total_q + at.q0 + n;
    const void* s = n < at.lq ? (const void*)src
                              : which ? (const void*)&kZeros : (const void*)&kInfinity;
    __builtin_amdgcn_global_load_lds(s, (lds_t)(&sstat[it % NST][which][0]), 4, 0, 0);
  };
  const T* K = (const T*)p.k + ((int64_t)at.k0 + held) * p.k_tok + (int64_t)kvh * p.k_head;
  const T* V = (const T*)p.v + ((int64_t)at.k0 + held) * p.v_tok + (int64_t)kvh * p.v_head;
  Vec8<T> kf[KS], vf[KS];
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    const int d = 16 * kk + 8 * (lane >> 5);
    if (d < p.dim) {
      kf[kk] = load8(K + d);
      vf[kk] = load8(V + d);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) kf[kk][e] = vf[kk][e] = (T)0.0f;
    }
  }
  floatx16 dk[ND], dv[ND];
  zero(dk);
  zero(dv);

#pragma unroll
  for (int s = 0; s < NST - 1; ++s) issue(s);
  for (int it = 0; it < steps; ++it) {
    const int ahead = min(steps - 1 - it, NST - 2);
    if (ahead >= 2) wait_vm<(NST > 3 ? 2 : 0) * PER>();
    else if (ahead == 1) wait_vm<PER>();
    else wait_vm<0>();
    barrier();
    issue(it + NST - 1);
    const int t = t0 + (it % per_head) * RC;
    const T* sq = smem + (it % NST) * 2 * TILE;
    const T* sg = sq + TILE;
#pragma unroll
    for (int b = 0; b < RC / 32; ++b) {
      // tokens tb .. tb + 31 see keys up to tb + 31 + off
      const int tb = t + 32 * b;
      if (tb >= at.lq || (p.causal && tb + 31 + off < j0)) continue;
      floatx16 st[1], dp[1];
      zero(st);
      zero(dp);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
        st[0] = Elem<T>::mma(frag<T, DC>(sq, 32 * b + (lane & 31), 16 * kk + 8 * (lane >> 5)),
                             kf[kk], st[0]);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
        dp[0] = Elem<T>::mma(frag<T, DC>(sg, 32 * b + (lane & 31), 16 * kk + 8 * (lane >> 5)),
                             vf[kk], dp[0]);
      if (p.causal && tb + off < j0 + 31) {
        const int from = key - off - tb - 4 * (lane >> 5);   // first row that sees the key
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (8 * (i / 4) + i % 4 < from) st[0][i] = -INFINITY;
      }
      const float* ps = &sstat[it % NST][0][32 * b + 4 * (lane >> 5)];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const floatx4 ls = *(const floatx4*)(ps + 8 * q);
        const floatx4 de = *(const floatx4*)(ps + 64 + 8 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * q + e;
          st[0][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(st[0][i], p.scale_log2, -ls[e]));
          dp[0][i] = st[0][i] * (dp[0][i] - de[e]);
        }
      }
#pragma unroll
      for (int kc = 0; kc < 2; ++kc) {
        const Vec8<T> pf = pack8<T>(st[0], kc), df = pack8<T>(dp[0], kc);
#pragma unroll
        for (int db = 0; db < ND; ++db)
          dv[db] = Elem<T>::mma(frag_tr<T, DC>(sg, 32 * b + 16 * kc, 32 * db, lane), pf, dv[db]);
#pragma unroll
        for (int db = 0; db < ND; ++db)
          dk[db] = Elem<T>::mma(frag_tr<T, DC>(sq, 32 * b + 16 * kc, 32 * db, lane), df, dk[db]);
      }
    }
  }
  const bool valid = key < at.lk;
  const int64_t n = (int64_t)at.k0 + held;
  store_row<T, DC>((T*)p.dk + n * p.dk_tok + kvh * p.dk_head, dk, p.scale, p.dim, lane, valid);
  store_row<T, DC>((T*)p.dv + n * p.dv_tok + kvh * p.dv_head, dv, 1.0f, p.dim, lane, valid);
}

}  // namespace att
}  // namespace mfl
