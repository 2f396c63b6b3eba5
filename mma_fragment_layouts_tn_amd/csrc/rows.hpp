// Kernels around the products by groups of rows: the places of a list of
// choices, and the sum of a token's results with its gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grouped_launch.hpp"

namespace mfl {
namespace grp {

// ------------------------------------------------------------ group_rows
// A stable counting sort.  Choices go to workgroups in chunks, within one to
// its W waves in runs, so that (group, workgroup, wave, position) is the order
// of the places: every wave counts its run, the counts before its own in that
// order are where its first choice of each group goes, and a second walk over
// the run gives each choice the number of equal ones before it.  Nothing
// depends on the order that waves run in.  Up to one chunk that is one launch;
// more chunks are counted by a launch before.
//
// Memory traffic is the choices twice and the results once (524,288 of them:
// 8 MB, 2 us); what bounds it is latency, of the walks (64 choices per wave at
// a time, their loads eight times that) and of the sums over chunks (every
// workgroup's, kSumAhead chunks at a time): 524,288 choices of 256 groups are
// counted in 3.8 us and placed in 13.8, 1,024 of 64 placed in 4.6.  (All of a
// chunk's sums under way at once, and the choices held from the first walk to
// the second, 18.2 us for both launches instead of 17.6.)
constexpr int kWalk = 8;          // loads of 64 choices under way
constexpr int kSumAhead = 16;

// waves of a workgroup: their counts of G groups fit LDS
constexpr int sort_waves(int G) { return G <= 256 ? 16 : 4; }

template <class I>
__device__ __forceinline__ int key_of(const void* ids, int64_t c, int groups) {
  const I x = ((const I*)ids)[c];
  return x >= 0 && x < groups ? (int)x : groups;
}

// f(first choice of 64, the lane's key) over [a, b), 64 apart
template <class I, class F>
__device__ __forceinline__ void walk(const SortParams& p, int64_t a, int64_t b, int lane, F f) {
  for (int64_t c = a; c < b; c += 64 * kWalk) {
    int key[kWalk];
#pragma unroll
    for (int s = 0; s < kWalk; ++s) {
      const int64_t x = c + 64 * s + lane;
      key[s] = x < b ? key_of<I>(p.ids, x, p.groups) : 0;
    }
#pragma unroll
    for (int s = 0; s < kWalk; ++s)
      if (c + 64 * s < b) f(c + 64 * s, key[s]);
  }
}

struct Run {
  int64_t first, end;     // this wave's choices
};
template <int W>
__device__ __forceinline__ Run run_of(const SortParams& p, int w) {
  const int64_t a = (int64_t)blockIdx.x * p.chunk, b = min(a + p.chunk, p.count);
  const int64_t per = p.chunk / W;
  return Run{min(a + w * per, b), min(a + (w + 1) * per, b)};
}

// counts of a chunk, per group (the last: no group)
template <class I, int G, int W = sort_waves(G)>
__global__ void __launch_bounds__(64 * W) group_count(const SortParams p) {
  __shared__ int hist[G + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  for (int g = tid; g <= p.groups; g += 64 * W) hist[g] = 0;
  __syncthreads();
  const Run run = run_of<W>(p, tid >> 6);
  walk<I>(p, run.first, run.end, lane, [&](int64_t c, int key) {
    if (c + lane < run.end) atomicAdd(&hist[key], 1);
  });
  __syncthreads();
  for (int g = tid; g <= p.groups; g += 64 * W)
    p.table[(int64_t)blockIdx.x * (p.groups + 1) + g] = hist[g];
}

template <class I, int G, int W = sort_waves(G)>
__global__ void __launch_bounds__(64 * W) group_place(const SortParams p) {
  constexpr int T = 64 * W;
  // hist[w][g]: wave w's choices of group g, then the place of its next one
  __shared__ int hist[W][G + 1];
  __shared__ int before[G + 1], all[G + 1];   // in the chunks before, in all of them
  __shared__ int sums[W];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = p.groups + 1;
  for (int g = tid; g < n; g += T) {
    before[g] = all[g] = 0;
#pragma unroll
    for (int v = 0; v < W; ++v) hist[v][g] = 0;
  }
  __syncthreads();
  const Run run = run_of<W>(p, w);
  walk<I>(p, run.first, run.end, lane, [&](int64_t c, int key) {
    if (c + lane < run.end) atomicAdd(&hist[w][key], 1);
  });
  if (gridDim.x > 1) {
    // the threads as rows of columns of the table, as many rows as there are
    const int wide = (n + 63) / 64 * 64, rows = T / wide > 1 ? T / wide : 1;
    const int blocks = gridDim.x, me = blockIdx.x;
    for (int g = tid % wide; g < n && tid < rows * wide; g += T) {
      int sum = 0, mine = 0;
      for (int b0 = tid / wide; b0 < blocks; b0 += rows * kSumAhead) {
        int t[kSumAhead];
#pragma unroll
        for (int x = 0; x < kSumAhead; ++x) {
          const int b = b0 + x * rows;
          t[x] = p.table[(int64_t)min(b, blocks - 1) * n + g];
          t[x] = b < blocks ? t[x] : 0;
        }
#pragma unroll
        for (int x = 0; x < kSumAhead; ++x) {
          sum += t[x];
          mine += b0 + x * rows < me ? t[x] : 0;
        }
      }
      atomicAdd(&all[g], sum);
      atomicAdd(&before[g], mine);
    }
  }
  __syncthreads();
  // Groups in runs of consecutive ones per thread, then a scan over the
  // threads: the places of the groups before.
  const int per = (n + T - 1) / T;
  int mine = 0;
  for (int x = 0; x < per; ++x) {
    const int g = tid * per + x;
    if (g >= n) break;
    int at = before[g], count = all[g];
    // this chunk's waves in turn
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const int t = hist[v][g];
      hist[v][g] = at;
      at += t;
    }
    if (gridDim.x == 1) count = at;
    before[g] = mine;       // from here on: within the thread's run, so far
    mine += count;
  }
  int scan = mine;          // inclusive over the wave's lanes
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(scan, d);
    if (lane >= d) scan += t;
  }
  if (lane == 63) sums[w] = scan;
  __syncthreads();
  int base = scan - mine;
  for (int v = 0; v < w; ++v) base += sums[v];
  for (int x = 0; x < per; ++x) {
    const int g = tid * per + x;
    if (g >= n) break;
    const int s = before[g] + base;
    if (blockIdx.x == 0) p.offsets[g] = s;
#pragma unroll
    for (int v = 0; v < W; ++v) hist[v][g] += s;
  }
  __syncthreads();
  volatile int* next = hist[w];
  walk<I>(p, run.first, run.end, lane, [&](int64_t c0, int key) {
    const int64_t c = c0 + lane;
    const bool in = c < run.end;
    // lanes of the same key
    unsigned long long same = __ballot(in);
    for (int bit = 0; bit < p.bits; ++bit) {
      const bool set = (key >> bit) & 1;
      const unsigned long long m = __ballot(set);
      same &= set ? m : ~m;
    }
    const int earlier = __popcll(same & ((1ull << lane) - 1));
    const int at = in ? next[key] + earlier : 0;
    // (a wave's LDS operations are done in order: the read above, this write,
    // the next round's read)
    if (in && earlier == 0) next[key] = at + __popcll(same);
    if (in) {
      p.rows[at] = (int)((unsigned)c / (unsigned)p.top);
      p.slots[c] = key < p.groups ? at : -1;
    }
  });
}

// ---------------------------------------------------------- combine_rows
template <class T>
struct Eight {
  typedef T vec __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ void load(const void* p, int64_t e, float (&x)[8]) {
    const vec v = *(const vec*)((const T*)p + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
  }
  static __device__ __forceinline__ void store(void* p, int64_t e, const float (&x)[8]) {
    vec v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)x[i];
    *(vec*)((T*)p + e) = v;
  }
};

// Eight columns of a token per thread, its rows one after the other: X is
// read once and out written once, which is all there is to do: 8,191 tokens of
// two rows of 4096, bf16, 37 us, 5.4 TB/s.
constexpr int kCombineThreads = 256;
template <class T, class O>
__global__ void __launch_bounds__(kCombineThreads) combine_sum(const CombineRows p) {
  const int chunks = p.n / 8;
  const int64_t x = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
  const int64_t t = x / chunks;
  if (t >= p.tokens) return;
  const int c = 8 * (int)(x - t * chunks);
  float sum[8] = {};
  const int* slots = p.slots + t * p.top;
  const float* weights = p.weights ? p.weights + t * p.top : nullptr;
#pragma unroll 4
  for (int j = 0; j < p.top; ++j) {
    const int s = slots[j];
    if ((unsigned)s >= (unsigned)p.x_rows) continue;
    const float w = weights ? weights[j] : 1.0f;
    float y[8];
    Eight<T>::load(p.x, (int64_t)s * p.ldx + c, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w, y[i], sum[i]);
  }
  Eight<O>::store(p.out, t * p.ldo + c, sum);
}

// A wave per place: it finds its place among its token's choices, reads the
// token's dout (which the token's other places read too: from L2) and its row
// of X once, and writes its row of dX.  The dot product of the two is dw.  The
// same 8,191 tokens 61 us, 5.5 TB/s.
template <class T>
__global__ void __launch_bounds__(kCombineThreads) combine_gradient(const CombineRows p) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * (kCombineThreads / 64) +
                    __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // choice i: no place, or one of another token's
  if (p.dw && i < p.tokens * p.top && lane == 0) {
    const int s = p.slots[i];
    if ((unsigned)s >= (unsigned)p.x_rows || p.rows[s] != i / p.top) p.dw[i] = 0.0f;
  }
  if (i >= p.x_rows) return;
  const int64_t t = p.rows[i];
  const bool token = t >= 0 && t < p.tokens;
  const int s = token && lane < p.top ? p.slots[t * p.top + lane] : -1;
  unsigned long long mine = __ballot(token && s == i);
  float w = 0.0f;
  for (unsigned long long m = mine; m; m &= m - 1)
    w += p.weights ? p.weights[t * p.top + __builtin_ctzll(m)] : 1.0f;
  float dot = 0.0f;
  for (int c = 8 * lane; c < p.n; c += 512) {
    float g[8] = {}, y[8];
    if (mine) {
      Eight<T>::load(p.dout, t * p.ldo + c, g);
      if (p.dw) {
        Eight<T>::load(p.x, i * p.ldx + c, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = __builtin_fmaf(g[e], y[e], dot);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] *= w;
    }
    Eight<T>::store(p.dx, i * p.lddx + c, g);
  }
  if (!p.dw || !mine) return;
#pragma unroll
  for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
  if (lane < p.top && (mine >> lane & 1)) p.dw[t * p.top + lane] = dot;
}

}  // namespace grp
}  // namespace mfl
