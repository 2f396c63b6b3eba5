// C ABI of attention (mfl_attention.h): argument checks, choice of kernel and
// splits, launches.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mfl_attention.h"
#include "attention.hpp"
#include "attention_bwd.hpp"
#include "attention_launch.hpp"

namespace {

using namespace mfl::att;

constexpr int64_t kMaxCount = (int64_t)INT_MAX - (1 << 16);
constexpr int64_t kMaxStride = (int64_t)1 << 40;   // elements; products with a count fit int64

// between tokens: tiles of tokens are addressed with 32-bit offsets
int check_token_strides(std::initializer_list<int64_t> strides) {
  for (int64_t s : strides)
    if (s > kMaxTokenStride) return MFL_E_TOO_LARGE;
  return MFL_OK;
}

bool aligned(const void* p) { return (uintptr_t)p % 16 == 0; }

int check_strides(std::initializer_list<int64_t> strides) {
  for (int64_t s : strides) {
    if (s < 0) return MFL_E_LEADING_DIM;
    if (s > kMaxStride) return MFL_E_TOO_LARGE;
    if (s % 8) return MFL_E_MISALIGNED;
  }
  return MFL_OK;
}

// no two elements of an output share an address: sorted by stride, each
// extent must reach past everything the smaller ones cover
struct Axis {
  int64_t count, stride;
};
int check_output(int64_t dim, Axis a, Axis b, Axis c) {
  Axis x[3] = {a, b, c};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (x[j].stride < x[i].stride) {
        const Axis t = x[i];
        x[i] = x[j];
        x[j] = t;
      }
  __int128 span = dim;
  for (const Axis& y : x) {
    if (y.count <= 1) continue;
    if (y.stride < span) return MFL_E_ALIAS;
    span += (__int128)(y.count - 1) * y.stride;
  }
  return MFL_OK;
}

int check_heads(int32_t dtype, int64_t batch, int64_t heads_q, int64_t heads_kv, int64_t dim,
                float scale) {
  if (heads_q < 0 || heads_kv < 0 || dim < 0 || batch < 0) return MFL_E_NEGATIVE_DIM;
  if (dtype != MFL_F16 && dtype != MFL_BF16) return MFL_E_UNSUPPORTED;
  if (batch == 0 || heads_kv == 0 || heads_q == 0 || heads_q % heads_kv) return MFL_E_UNSUPPORTED;
  if (dim == 0 || dim % 8 || dim > 256) return MFL_E_UNSUPPORTED;
  if (!(scale > 0.0f) || !isfinite(scale * kLog2e)) return MFL_E_UNSUPPORTED;
  if (heads_q > (1 << 16) || batch > (1 << 24)) return MFL_E_TOO_LARGE;
  return MFL_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t clamp(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// slots of `bm`-row tiles over the sequences (find_sequence)
int64_t tile_slots(int64_t rows, int64_t batch, int64_t bm, bool packed) {
  return packed ? rows / bm + batch : ceil_div(rows, bm);
}

struct Choice {
  int algo;
  int64_t splits, slots, part_keys;
};

// one part's partial rows, and all of them
int64_t plane_bytes(int64_t rows, int dc) { return rows * (4 * (int64_t)dc + 8); }
int64_t partial_bytes(int64_t rows, int64_t splits, int dc) {
  return splits > 1 ? splits * plane_bytes(rows, dc) : 0;
}

// Workgroups that occupy every CU.
constexpr int64_t kFill = 256;
// Partial rows at most, where the number of parts is chosen here.
constexpr int64_t kPartialBytes = (int64_t)1 << 28;

// Kernel and parts of packed attention.  The host knows the sums of the
// lengths, not each one (they are on the device), so the rules go by means.
//
// FLAT (16 rows, 4 waves share the keys) against TALL (128 rows, each wave
// all keys), 32 query and 8 key heads of 128, bf16, causal: 1 token 4.5 and
// 5.1 us, 16 tokens against 8192 keys 18 and 20, 128 tokens 5.5 and 7.3, 256
// tokens 7.6 and 9.6, but 512 tokens 16.1 and 14.4 and 2048 tokens 102 and 49.
// So FLAT where a sequence has up to 64 rows, or where its workgroups are at
// most two per CU and the keys are few (64 tokens against 8192 keys: 35 and
// 30, both split).
//
// By the means a batch of a long prompt and many single tokens counts as the
// latter, and one sequence far longer than many others keeps one part:
// 2048 tokens beside 200 single ones 122 us in FLAT and 61 in TALL, one token
// against 131072 keys beside 32 against 100 1348 us in one part and 164 in 32.
// A caller that knows the lengths gives algo and splits.
//
// Parts: where the tiles leave CUs idle, a tile's keys are shared out to
// workgroups, as many as make two per CU with the mean of the keys, if that
// saves more than it costs: a workgroup takes 18 ns per key (TALL, 128
// columns) or 6.4 ns (FLAT); partial rows are written and read at 4 TB/s, and
// the launch that joins them takes 4 us.  64 tokens against 8192 keys: 150 us
// in one part, 30 in 16; 1024 against 1024: 25 and 43 in two.
//
// A plane of partial rows per part: one sequence may have most of the keys, so
// the planes are as many as all keys would take, up to 256 MiB (7 planes at
// least; equal lengths take 2 - 4 where planes are that large), and a longer
// sequence gets longer parts.  32 sequences of 32 tokens against 8192 keys:
// 294 us with 15 planes, 338 with 64 (1.1 GB, and as many workgroups that find
// nothing to do); 64 tokens against 65536 keys beside 15 times 64 against 256:
// 177 with 15 and with 32, 377 with 4.
Choice choose(int64_t rows, int64_t batch, bool packed, int64_t keys, int64_t heads_kv, int dc,
              int algo, int64_t splits) {
  Choice c;
  const int64_t mean_rows = ceil_div(rows, batch), mean_keys = ceil_div(keys, batch);
  if (algo == MFL_ATTENTION_AUTO) {
    const bool few = ceil_div(rows, 16) * heads_kv <= 2 * kFill && mean_keys <= 2048;
    algo = mean_rows <= 64 || few ? MFL_ATTENTION_FLAT : MFL_ATTENTION_TALL;
  }
  c.algo = algo;
  c.slots = tile_slots(rows, batch, tile_rows(algo), packed);
  c.splits = splits;
  c.part_keys = 0;
  if (splits == 0) {
    c.splits = 1;
    const int64_t tiles = ceil_div(rows, tile_rows(algo)),
                  wgs = (tiles > batch ? tiles : batch) * heads_kv,
                  least = algo == MFL_ATTENTION_FLAT ? 256 : 512;
    if (rows > 0 && wgs <= kFill) {
      const int64_t fair = ceil_div(mean_keys, 2 * kFill / wgs),
                    part = clamp(ceil_div(fair, 64) * 64, least, INT_MAX / 2),
                    saved = (mean_keys - part) * (algo == MFL_ATTENTION_FLAT ? 64 : 180) * dc / 1280,
                    bytes = ceil_div(mean_keys, part) * rows * heads_kv * dc * 8;
      if (saved > 4000 + bytes / 4000) {
        c.part_keys = part;
        c.splits = clamp(ceil_div(keys, part), 1,
                         clamp(kPartialBytes / plane_bytes(rows * heads_kv, dc), 1, 64));
      }
    }
  }
  return c;
}

// Workgroups of a launch: every kernel here has 256 threads, and a launch has
// fewer than 2^32.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;

bool grid_fits(const Choice& c, int64_t heads_kv) {
  return (__int128)c.slots * heads_kv * c.splits <= kMaxBlocks;
}

// Rows per workgroup of the join by tiles: one per wave, or two where there
// are more workgroups than are resident at a time (20,000 rows 15.4 and
// 11.4 us, 3,000 rows 4 and 6).
int join_rows(const Choice& c, int64_t heads_kv) {
  return c.slots * (tile_rows(c.algo) / 4) * heads_kv > 16 * kFill ? 8 : 4;
}
int64_t join_blocks(const Choice& c, int64_t heads_kv) {
  return c.slots * (tile_rows(c.algo) / join_rows(c, heads_kv)) * heads_kv;
}

constexpr int kJoinRows = 4;   // of the join of all rows: one per wave

int launch(KernelRef k, int64_t blocks, void** args, void* stream) {
  if (blocks == 0) return MFL_OK;
  const hipError_t e = hipLaunchKernel(k.fn, dim3((unsigned)blocks), dim3(k.threads), args, 0,
                                       (hipStream_t)stream);
  return e == hipSuccess ? MFL_OK : MFL_E_LAUNCH;
}

int run(KernelRef k, int64_t blocks, void* params, void* stream, int a = 0, int b = 0) {
  void* args[] = {params, &a, &b};   // (a kernel takes as many as it has)
  return launch(k, blocks, args, stream);
}

void place_choice(FwdParams& p, const Choice& c) {
  p.splits = (int)c.splits;
  p.slots = (int)c.slots;
  p.part_keys = (int)c.part_keys;
}

int run_forward(FwdParams& p, const Choice& c, bool bf16, int dc, void* stream) {
  place_choice(p, c);
  return run(fwd_kernel(bf16, dc, c.algo), c.slots * p.heads_kv * c.splits, &p, stream);
}

int run_join(const FwdParams& p, int splits, bool bf16, int dc, void* stream) {
  CombineParams j{};
  j.part_o = p.part_o;
  j.part_ml = p.part_ml;
  j.o = p.o;
  j.lse = p.lse;
  j.rows = p.rows;
  j.splits = splits;
  j.dim = p.dim;
  j.heads = p.heads_kv * p.group;
  j.q_inner = p.q_inner;
  j.o_batch = p.o_batch;
  j.o_tok = p.o_tok;
  j.o_head = p.o_head;
  return run(other_kernel(bf16, dc, kJoin), ceil_div(p.rows, kJoinRows), &j, stream);
}

int check_packed(const mfl_attention_t& a, const void* q, const void* k, const void* v,
                 const int32_t* seq_q, const int32_t* seq_k, const void* out, const float* lse) {
  if (a.total_q < 0 || a.total_k < 0) return MFL_E_NEGATIVE_DIM;
  int rc = check_heads(a.dtype, a.batch, a.heads_q, a.heads_kv, a.head_dim, a.scale);
  if (rc) return rc;
  if ((a.causal != 0 && a.causal != 1) || a.algo < 0 || a.algo > MFL_ATTENTION_FLAT ||
      a.splits < 0 || a.splits > 1024)
    return MFL_E_UNSUPPORTED;
  if (!seq_q != !seq_k) return MFL_E_NULL_POINTER;
  if (!seq_q && a.batch != 1) return MFL_E_NULL_POINTER;
  if (a.total_q > kMaxCount || a.total_k > kMaxCount || a.total_q * a.heads_q > kMaxCount)
    return MFL_E_TOO_LARGE;
  if (a.total_q > 0 && (!q || !out)) return MFL_E_NULL_POINTER;
  if (a.total_q > 0 && a.total_k > 0 && (!k || !v)) return MFL_E_NULL_POINTER;
  rc = check_strides({a.q_token, a.q_head, a.k_token, a.k_head, a.v_token, a.v_head, a.out_token,
                      a.out_head});
  if (!rc) rc = check_token_strides({a.q_token, a.k_token, a.v_token});
  if (rc) return rc;
  if (!aligned(q) || !aligned(k) || !aligned(v) || !aligned(out) || (uintptr_t)lse % 4 ||
      (uintptr_t)seq_q % 4 || (uintptr_t)seq_k % 4)
    return MFL_E_MISALIGNED;
  if (out && (out == q || out == k || out == v)) return MFL_E_ALIAS;
  return check_output(a.head_dim, {a.total_q, a.out_token}, {a.heads_q, a.out_head}, {1, 0});
}

int plan_packed(const mfl_attention_t& a, bool packed, Choice& c, int64_t& bytes) {
  const int dc = dim_class(a.head_dim);
  c = choose(a.total_q * (a.heads_q / a.heads_kv), a.batch, packed, a.total_k, a.heads_kv, dc,
             a.algo, a.splits);
  if (!grid_fits(c, a.heads_kv) || (c.splits > 1 && join_blocks(c, a.heads_kv) > kMaxBlocks))
    return MFL_E_TOO_LARGE;
  bytes = partial_bytes(a.total_q * a.heads_q, c.splits, dc);
  return MFL_OK;
}

int check_workspace(const void* workspace, int64_t have, int64_t need) {
  if (need == 0) return MFL_OK;
  return !workspace || !aligned(workspace) || have < need ? MFL_E_WORKSPACE : MFL_OK;
}

// the partial rows, then the (maximum, sum) pairs
void place_partials(FwdParams& p, void* workspace, int64_t splits, int dc) {
  p.part_o = (float*)workspace;
  p.part_ml = (float2*)((char*)workspace + 4 * splits * p.rows * dc);
}

// Shares of dK and dV per kv head (0: a workgroup per tile), and the workspace.
struct BackwardPlan {
  int64_t slots_q, slots_k, shares, bytes, cuts_at, partials_at;
  bool by_tile;
};

BackwardPlan plan_backward(const mfl_attention_t& f, bool packed) {
  const int dc = dim_class(f.head_dim);
  const int64_t group = f.heads_q / f.heads_kv;
  BackwardPlan r;
  // one slot more than tiles can need: the tokens behind the last sequence
  r.slots_q = tile_slots(f.total_q * group, f.batch, kDqRows, packed) + (packed ? 1 : 0);
  r.slots_k = tile_slots(f.total_k, f.batch, dkv_keys(dc), packed);
  r.bytes = r.cuts_at = r.partials_at = 8 * f.heads_q * f.total_q;   // the statistics first
  r.shares = 0;
  r.by_tile = false;
  // Equal shares cost the partial sums of the tiles cut and their join (256 KB
  // per part at 128 columns; 26 us for 8192 tokens, 8 key heads).  With a
  // causal mask they pay until there are many tiles per CU (that case: 440 us
  // with the join, 769 a tile each); without one tiles differ little, and from
  // two per CU on a tile each is as good (16 key heads of 64, 600 tiles: 91
  // and 93 us).  Every workgroup walks the sequences' lengths to find its
  // share, so not for more than 256 sequences.
  const int64_t tiles = r.slots_k * f.heads_kv;
  if (f.batch <= 256 && tiles < (f.causal ? 8 : 2) * kFill) {
    // One round of the chip, or two to four if that leaves fewer CUs idle by
    // more than a sixteenth of them: every share more is a cut more, a place
    // in the workspace and sums to join.  dK, dV and dQ of 4096 tokens, 24
    // query and 3 key heads of 128: 384 us in one round of 255 and 462 in three
    // of 256; 40 and 20 heads 596 in one of 240, 735 in four of 255.
    int64_t best = 0;
    for (int64_t rounds = 1; rounds <= 4; ++rounds) {
      const int64_t n = rounds * kFill / f.heads_kv, busy = n * f.heads_kv * 1024 / rounds;
      if (busy > best + (rounds > 1 ? kFill * 64 : 0)) {
        best = busy;
        r.shares = n;
      }
    }
    // no more than the steps that there can be would fill
    const int64_t chunks = ceil_div(f.total_q, dkv_chunk(dc)) + f.batch;
    r.shares = clamp(r.slots_k * (chunks * group + kDkvFixed) / kDkvLeast, 1, r.shares);
    r.partials_at = ceil_div(r.cuts_at + r.shares * (int64_t)sizeof(DkvCut), 16) * 16;
    const int64_t numbered = r.shares + r.slots_k - 1;     // dkv_place
    r.by_tile = numbered < 2 * r.shares;
    r.bytes = r.partials_at +
              (r.by_tile ? numbered : 2 * r.shares) * f.heads_kv * 8 * dkv_keys(dc) * dc;
  }
  return r;
}

int check_backward(const mfl_attention_grad_t& a, const void* dout, const void* q, const void* k,
                   const void* v, const void* out, const float* lse, const int32_t* seq_q,
                   const int32_t* seq_k, const void* dq, const void* dk, const void* dv) {
  mfl_attention_t f = a.f;
  f.algo = MFL_ATTENTION_AUTO;
  f.splits = 0;
  int rc = check_packed(f, q, k, v, seq_q, seq_k, out, lse);
  if (rc) return rc;
  if (f.total_q > 0 && (!dout || !lse || !dq)) return MFL_E_NULL_POINTER;
  if (f.total_k > 0 && (!dk || !dv)) return MFL_E_NULL_POINTER;
  rc = check_strides({a.dout_token, a.dout_head, a.dq_token, a.dq_head, a.dk_token, a.dk_head,
                      a.dv_token, a.dv_head});
  if (!rc) rc = check_token_strides({a.dout_token});
  if (rc) return rc;
  // rows past a sequence's end must lie past its rows
  if ((f.total_q > 1) && (f.q_token < f.head_dim || a.dout_token < f.head_dim))
    return MFL_E_LEADING_DIM;
  const void* grads[3] = {dq, dk, dv};
  const void* inputs[6] = {dout, q, k, v, out, lse};
  if (!aligned(dout)) return MFL_E_MISALIGNED;
  for (int i = 0; i < 3; ++i) {
    if (!aligned(grads[i])) return MFL_E_MISALIGNED;
    for (const void* x : inputs)
      if (grads[i] && grads[i] == x) return MFL_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (grads[i] && grads[i] == grads[j]) return MFL_E_ALIAS;
  }
  rc = check_output(f.head_dim, {f.total_q, a.dq_token}, {f.heads_q, a.dq_head}, {1, 0});
  if (rc) return rc;
  rc = check_output(f.head_dim, {f.total_k, a.dk_token}, {f.heads_kv, a.dk_head}, {1, 0});
  if (rc) return rc;
  rc = check_output(f.head_dim, {f.total_k, a.dv_token}, {f.heads_kv, a.dv_head}, {1, 0});
  if (rc) return rc;
  const BackwardPlan r = plan_backward(f, seq_q != nullptr);
  if (r.slots_q * f.heads_kv > kMaxBlocks || r.slots_k * f.heads_kv > kMaxBlocks)
    return MFL_E_TOO_LARGE;
  return MFL_OK;
}

int check_prefix(const mfl_attention_prefix_t& a, const void* q, const void* prefix_k,
                 const void* prefix_v, const void* k, const void* v, const int32_t* lengths,
                 const void* out, const float* lse) {
  if (a.q_tokens < 0 || a.prefix < 0 || a.capacity < 0) return MFL_E_NEGATIVE_DIM;
  int rc = check_heads(a.dtype, a.batch, a.heads_q, a.heads_kv, a.head_dim, a.scale);
  if (rc) return rc;
  if (a.algo < 0 || a.algo > MFL_ATTENTION_FLAT || a.splits_prefix < 0 ||
      a.splits_prefix > 1024 || a.splits_own < 0 || a.splits_own > 1024)
    return MFL_E_UNSUPPORTED;
  if (a.q_tokens > kMaxCount || a.prefix > kMaxCount || a.capacity > kMaxCount)
    return MFL_E_TOO_LARGE;
  if ((__int128)a.batch * a.q_tokens * a.heads_q > kMaxCount) return MFL_E_TOO_LARGE;
  if (a.q_tokens > 0) {
    if (!q || !out) return MFL_E_NULL_POINTER;
    if (a.prefix > 0 && (!prefix_k || !prefix_v)) return MFL_E_NULL_POINTER;
    if (a.capacity > 0 && (!k || !v || !lengths)) return MFL_E_NULL_POINTER;
  }
  rc = check_strides({a.q_batch, a.q_token, a.q_head, a.prefix_k_token, a.prefix_k_head,
                      a.prefix_v_token, a.prefix_v_head, a.k_batch, a.k_token, a.k_head,
                      a.v_batch, a.v_token, a.v_head, a.out_batch, a.out_token, a.out_head});
  if (!rc) rc = check_token_strides({a.prefix_k_token, a.prefix_v_token, a.k_token, a.v_token});
  if (rc) return rc;
  if (!aligned(q) || !aligned(prefix_k) || !aligned(prefix_v) || !aligned(k) || !aligned(v) ||
      !aligned(out) || (uintptr_t)lse % 4 || (uintptr_t)lengths % 4)
    return MFL_E_MISALIGNED;
  if (out && (out == q || out == prefix_k || out == prefix_v || out == k || out == v))
    return MFL_E_ALIAS;
  return check_output(a.head_dim, {a.batch, a.out_batch}, {a.q_tokens, a.out_token},
                      {a.heads_q, a.out_head});
}

struct PrefixPlan {
  Choice prefix, own;      // splits 0: the part has no launch
  int64_t bytes;
};

int plan_prefix(const mfl_attention_prefix_t& a, PrefixPlan& r) {
  const int dc = dim_class(a.head_dim);
  const int64_t group = a.heads_q / a.heads_kv, rows = a.batch * a.q_tokens * group;
  r.prefix.algo = a.algo ? a.algo : rows <= 64 ? MFL_ATTENTION_FLAT : MFL_ATTENTION_TALL;
  r.own.algo = MFL_ATTENTION_FLAT;
  r.prefix.slots = ceil_div(rows, tile_rows(r.prefix.algo));
  r.own.slots = a.batch * ceil_div(a.q_tokens * group, tile_rows(MFL_ATTENTION_FLAT));
  r.prefix.part_keys = r.own.part_keys = 0;
  // each part gets a workgroup per CU
  auto parts = [&](int64_t slots, int64_t keys, int64_t least) {
    const int64_t wgs = slots * a.heads_kv;
    return clamp(wgs > 0 ? kFill / wgs : 1, 1, clamp(keys / least, 1, 64));
  };
  r.prefix.splits = a.splits_prefix ? a.splits_prefix : parts(r.prefix.slots, a.prefix, 128);
  r.own.splits = a.splits_own ? a.splits_own : parts(r.own.slots, a.capacity, 256);
  // Half as many of the prefix where the own keys alone give two workgroups
  // per CU, as long as none walks more than 4096 keys (64 sequences behind
  // 8192 keys: 8 parts 40 us, 16 parts 48; 256 sequences: 2 and 4 parts 137 and
  // 142; 128 behind 32768: 8 and 4 parts 172 and more than 205).
  const int64_t half = r.prefix.splits / 2;
  if (!a.splits_prefix && half > 0 && r.own.slots * a.heads_kv >= 2 * kFill && a.capacity > 0 &&
      ceil_div(a.prefix, half) <= 4096)
    r.prefix.splits = half;
  if (a.prefix == 0) r.prefix.splits = 0;
  if (a.capacity == 0) r.own.splits = a.prefix == 0 ? 1 : 0;
  if (!grid_fits(r.prefix, a.heads_kv) || !grid_fits(r.own, a.heads_kv) ||
      (__int128)(r.prefix.slots * r.prefix.splits + r.own.slots * r.own.splits) * a.heads_kv >
          kMaxBlocks ||
      (r.prefix.splits + r.own.splits > 1 &&
       ceil_div(a.batch * a.q_tokens * a.heads_q, kJoinRows) > kMaxBlocks))
    return MFL_E_TOO_LARGE;
  r.bytes = partial_bytes(a.batch * a.q_tokens * a.heads_q, r.prefix.splits + r.own.splits, dc);
  return MFL_OK;
}

}  // namespace

extern "C" {

int attention_packed_plan(const mfl_attention_t* a, const void* q, const void* k, const void* v,
                          const int32_t* seq_q, const int32_t* seq_k, const void* out,
                          const float* lse, int32_t* algo, int32_t* splits,
                          int64_t* workspace_bytes) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_packed(*a, q, k, v, seq_q, seq_k, out, lse);
  if (rc) return rc;
  Choice c;
  int64_t bytes;
  rc = plan_packed(*a, seq_q != nullptr, c, bytes);
  if (rc) return rc;
  if (algo) *algo = c.algo;
  if (splits) *splits = (int32_t)c.splits;
  if (workspace_bytes) *workspace_bytes = bytes;
  return MFL_OK;
}

int attention_packed(const mfl_attention_t* a, const void* q, const void* k, const void* v,
                     const int32_t* seq_q, const int32_t* seq_k, void* out, float* lse,
                     void* workspace, int64_t workspace_bytes, void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_packed(*a, q, k, v, seq_q, seq_k, out, lse);
  if (rc) return rc;
  Choice c;
  int64_t bytes;
  rc = plan_packed(*a, seq_q != nullptr, c, bytes);
  if (rc) return rc;
  rc = check_workspace(workspace, workspace_bytes, bytes);
  if (rc) return rc;
  if (a->total_q == 0) return MFL_OK;
  const int dc = dim_class(a->head_dim);
  FwdParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = out;
  p.lse = lse;
  p.seq_q = seq_q;
  p.seq_k = seq_k;
  p.batch = (int)a->batch;
  p.q_len = (int)a->total_q;
  p.total_q = (int)a->total_q;
  p.total_k = (int)a->total_k;
  p.q_inner = INT_MAX;
  p.heads_kv = (int)a->heads_kv;
  p.group = (int)(a->heads_q / a->heads_kv);
  p.dim = (int)a->head_dim;
  p.causal = a->causal;
  p.rows = a->total_q * a->heads_q;
  p.q_tok = a->q_token;
  p.q_head = a->q_head;
  p.k_tok = a->k_token;
  p.k_head = a->k_head;
  p.v_tok = a->v_token;
  p.v_head = a->v_head;
  p.o_tok = a->out_token;
  p.o_head = a->out_head;
  p.scale_log2 = a->scale * kLog2e;
  const bool bf16 = a->dtype == MFL_BF16;
  if (c.splits > 1) place_partials(p, workspace, c.splits, dc);
  rc = run_forward(p, c, bf16, dc, stream);
  if (rc || c.splits == 1) return rc;
  // by tiles: rows of no sequence have no partial sums and stay as they were
  return run(other_kernel(bf16, dc, kJoinTiles), join_blocks(c, p.heads_kv), &p, stream,
             tile_rows(c.algo), join_rows(c, p.heads_kv));
}

int attention_packed_backward_plan(const mfl_attention_grad_t* a, const void* dout,
                                   const void* q, const void* k, const void* v, const void* out,
                                   const float* lse, const int32_t* seq_q, const int32_t* seq_k,
                                   const void* dq, const void* dk, const void* dv,
                                   int64_t* workspace_bytes) {
  if (!a) return MFL_E_NULL_POINTER;
  const int rc = check_backward(*a, dout, q, k, v, out, lse, seq_q, seq_k, dq, dk, dv);
  if (rc) return rc;
  if (workspace_bytes) *workspace_bytes = plan_backward(a->f, seq_q != nullptr).bytes;
  return MFL_OK;
}

int attention_packed_backward(const mfl_attention_grad_t* a, const void* dout, const void* q,
                              const void* k, const void* v, const void* out, const float* lse,
                              const int32_t* seq_q, const int32_t* seq_k, void* dq, void* dk,
                              void* dv, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_backward(*a, dout, q, k, v, out, lse, seq_q, seq_k, dq, dk, dv);
  if (rc) return rc;
  const mfl_attention_t& f = a->f;
  const BackwardPlan plan = plan_backward(f, seq_q != nullptr);
  rc = check_workspace(workspace, workspace_bytes, plan.bytes);
  if (rc) return rc;
  const int dc = dim_class(f.head_dim);
  const bool bf16 = f.dtype == MFL_BF16;
  BwdParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = out;
  p.dout = dout;
  p.lse = lse;
  p.stats = (float*)workspace;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.seq_q = seq_q;
  p.seq_k = seq_k;
  p.batch = (int)f.batch;
  p.total_q = (int)f.total_q;
  p.total_k = (int)f.total_k;
  p.heads_kv = (int)f.heads_kv;
  p.group = (int)(f.heads_q / f.heads_kv);
  p.dim = (int)f.head_dim;
  p.causal = f.causal;
  // (a single token's stride is not read, but must lead past its row)
  p.q_tok = f.total_q > 1 ? f.q_token : f.head_dim;
  p.q_head = f.q_head;
  p.k_tok = f.k_token;
  p.k_head = f.k_head;
  p.v_tok = f.v_token;
  p.v_head = f.v_head;
  p.o_tok = f.out_token;
  p.o_head = f.out_head;
  p.do_tok = f.total_q > 1 ? a->dout_token : f.head_dim;
  p.do_head = a->dout_head;
  p.dq_tok = a->dq_token;
  p.dq_head = a->dq_head;
  p.dk_tok = a->dk_token;
  p.dk_head = a->dk_head;
  p.dv_tok = a->dv_token;
  p.dv_head = a->dv_head;
  p.scale = f.scale;
  p.scale_log2 = f.scale * kLog2e;
  p.slots_q = (int)plan.slots_q;
  p.slots_k = (int)plan.slots_k;
  p.shares = (int)plan.shares;
  p.by_tile = plan.by_tile;
  p.cuts = (DkvCut*)((char*)workspace + plan.cuts_at);
  p.partials = (float*)((char*)workspace + plan.partials_at);
  if (f.total_q > 0) {
    rc = run(dq_kernel(bf16, dc), plan.slots_q * p.heads_kv, &p, stream);
    if (rc) return rc;
  }
  if (f.total_k == 0) return MFL_OK;
  rc = run(dkv_kernel(bf16, dc), (plan.shares ? plan.shares : plan.slots_k) * p.heads_kv, &p,
           stream);
  if (rc || plan.shares <= 1) return rc;
  return run(dkv_join_kernel(bf16, dc), plan.shares * (dkv_keys(dc) / 32) * p.heads_kv, &p, stream,
             dkv_keys(dc));
}

int attention_prefix_plan(const mfl_attention_prefix_t* a, const void* q, const void* prefix_k,
                          const void* prefix_v, const void* k, const void* v,
                          const int32_t* lengths, const void* out, const float* lse,
                          int32_t* algo, int32_t* splits_prefix, int32_t* splits_own,
                          int64_t* workspace_bytes) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_prefix(*a, q, prefix_k, prefix_v, k, v, lengths, out, lse);
  if (rc) return rc;
  PrefixPlan r;
  rc = plan_prefix(*a, r);
  if (rc) return rc;
  if (algo) *algo = r.prefix.algo;
  if (splits_prefix) *splits_prefix = (int32_t)r.prefix.splits;
  if (splits_own) *splits_own = (int32_t)r.own.splits;
  if (workspace_bytes) *workspace_bytes = r.bytes;
  return MFL_OK;
}

int attention_prefix(const mfl_attention_prefix_t* a, const void* q, const void* prefix_k,
                     const void* prefix_v, const void* k, const void* v, const int32_t* lengths,
                     void* out, float* lse, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  if (!a) return MFL_E_NULL_POINTER;
  int rc = check_prefix(*a, q, prefix_k, prefix_v, k, v, lengths, out, lse);
  if (rc) return rc;
  PrefixPlan r;
  rc = plan_prefix(*a, r);
  if (rc) return rc;
  rc = check_workspace(workspace, workspace_bytes, r.bytes);
  if (rc) return rc;
  if (a->q_tokens == 0) return MFL_OK;
  const int dc = dim_class(a->head_dim);
  const bool bf16 = a->dtype == MFL_BF16;
  const int splits = (int)(r.prefix.splits + r.own.splits);
  FwdParams p{};
  p.q = q;
  p.o = out;
  p.lse = lse;
  p.q_inner = (int)a->q_tokens;
  p.heads_kv = (int)a->heads_kv;
  p.group = (int)(a->heads_q / a->heads_kv);
  p.dim = (int)a->head_dim;
  p.rows = a->batch * a->q_tokens * a->heads_q;
  p.total_q = (int)(a->batch * a->q_tokens);
  p.q_batch = a->q_batch;
  p.q_tok = a->q_token;
  p.q_head = a->q_head;
  p.o_batch = a->out_batch;
  p.o_tok = a->out_token;
  p.o_head = a->out_head;
  p.scale_log2 = a->scale * kLog2e;
  if (splits > 1) place_partials(p, workspace, splits, dc);
  FwdParams x = p;               // one sequence of all rows against the prefix
  x.k = prefix_k;
  x.v = prefix_v;
  x.batch = 1;
  x.q_len = p.total_q;
  x.total_k = (int)a->prefix;
  x.k_tok = a->prefix_k_token;
  x.k_head = a->prefix_k_head;
  x.v_tok = a->prefix_v_token;
  x.v_head = a->prefix_v_head;
  FwdParams y = p;               // each sequence's rows against its own keys
  y.k = k;
  y.v = v;
  y.lengths = lengths;
  y.batch = (int)a->batch;
  y.q_len = (int)a->q_tokens;
  y.total_k = (int)a->capacity;
  y.causal = 1;
  y.k_batch = a->k_batch;
  y.k_tok = a->k_token;
  y.k_head = a->k_head;
  y.v_batch = a->v_batch;
  y.v_tok = a->v_token;
  y.v_head = a->v_head;
  y.split0 = (int)r.prefix.splits;
  place_choice(x, r.prefix);
  place_choice(y, r.own);
  const int64_t nx = r.prefix.slots * r.prefix.splits * p.heads_kv,
                ny = r.own.slots * r.own.splits * p.heads_kv;
  if (nx == 0) {
    rc = run(fwd_kernel(bf16, dc, MFL_ATTENTION_FLAT), ny, &y, stream);
  } else if (ny == 0) {
    rc = run(fwd_kernel(bf16, dc, r.prefix.algo), nx, &x, stream);
  } else {
    const KernelRef f = other_kernel(
        bf16, dc, r.prefix.algo == MFL_ATTENTION_FLAT ? kPairFlat : kPairTall);
    int n0 = (int)nx;
    void* args[] = {&x, &y, &n0};
    rc = launch(f, nx + ny, args, stream);
  }
  if (rc) return rc;
  return splits > 1 ? run_join(p, splits, bf16, dc, stream) : MFL_OK;
}

}  // extern "C"
