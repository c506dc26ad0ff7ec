// The k largest logits of every row and the log-sum-exp of all the others, in one pass over the row.
//
// A workgroup takes a segment of a row (the whole row where there are rows enough to fill the
// device). The k-th largest of the threads' maxima over their first vectors is a lower bound t of the
// k-th largest logit; from there on an element above the bound is a candidate and goes, as a 64-bit
// key (value's order in the upper half, falling index in the lower, so that no two are the same),
// into a buffer in LDS, and any other adds 2^(x log2 e - ref) to its thread's sum. Candidates are few
// (for random order about k per group-sized part of the segment). When the buffer could run over, it
// is sorted, the k largest stay, the bound rises to the k-th, and the others join the sums; the end
// does the same. The sum of the others is never formed by subtracting the listed ones, which would
// lose what is left where the list holds nearly all of the row.
//
// Every set and every order of additions depends on the data alone, not on the order in which
// candidates reach the buffer, so results are the same bits every time.
//
// This file is compiled with the IEEE mode off, like the row kernels: NaN is outside the contract.

#include <stdint.h>

#include <algorithm>

#include "opd_internal.h"
#include "opd_rows.h"

namespace opd {
namespace {

constexpr int kGroupVec = 4;  // vectors per thread between two checks of the buffer

// Unsigned keys in the order of the values (-0 as +0, so that equal values go by index).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t make_key(float x, int index) {
  return ((uint64_t)order_key(x) << 32) | (uint32_t)~index;
}

// A thread's share of the log-sum-exp of the elements that are not listed: sum * 2^ref.
struct Rest {
  float ref = kNoRef, sum = 0.f;
  // ref may lag the largest exponent by up to 24: 2^24 an element leaves fp32 range to spare
  __device__ __forceinline__ void raise(float m) {
    const float c = m * kLog2e;
    if (c > ref + 24.f) {
      sum *= ex2(ref - c);
      ref = c;
    }
  }
  __device__ __forceinline__ void add(float x) { sum += ex2(__builtin_fmaf(x, kLog2e, -ref)); }
};

struct Shared {
  uint64_t keys[kTopkCap];
  float part[kThreads];
  float pair[kThreads / 64][2];
  float bound;
  int count;
};

// Sorts the n buffered keys (largest first), keeps the k largest, and adds the others to the threads'
// sums in the order of their rank. Returns the number kept. All threads call it.
__device__ int settle(Shared& S, int n, int k, Rest& rest) {
  const int tid = threadIdx.x;
  int m = 2;
  while (m < n) m <<= 1;
  for (int i = n + tid; i < m; i += kThreads) S.keys[i] = 0;
  __syncthreads();
  for (int size = 2; size <= m; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = tid; i < m / 2; i += kThreads) {
        const int a = 2 * i - (i & (stride - 1)), b = a + stride;
        const uint64_t x = S.keys[a], y = S.keys[b];
        const bool falling = (a & size) == 0;
        if ((x < y) == falling) {
          S.keys[a] = y;
          S.keys[b] = x;
        }
      }
      __syncthreads();
    }
  for (int i = k + tid; i < n; i += kThreads) {
    if (S.keys[i] == 0) continue;  // (a segment's list that was not full)
    const float x = key_value((uint32_t)(S.keys[i] >> 32));
    rest.raise(x);
    rest.add(x);
  }
  const int kept = min(n, k);
  if (tid == 0) {
    S.count = kept;
    S.bound = n >= k ? key_value((uint32_t)(S.keys[k - 1] >> 32)) : kNegInf;
  }
  __syncthreads();
  return kept;
}

// Joins the threads' sums; thread 0 has the result.
__device__ void join_rest(Shared& S, Rest& rest) {
  wave_lse(rest.ref, rest.sum);
  if ((threadIdx.x & 63) == 0) {
    S.pair[threadIdx.x >> 6][0] = rest.ref;
    S.pair[threadIdx.x >> 6][1] = rest.sum;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    rest.ref = S.pair[0][0];
    rest.sum = S.pair[0][1];
    for (int w = 1; w < kThreads / 64; ++w) lse_join(rest.ref, rest.sum, S.pair[w][0], S.pair[w][1]);
  }
}

// Writes a row's answer: the first `kept` keys (an entry that is not there: index -1) and the sum.
__device__ void write_row(const TopkParams& P, const Shared& S, int row, int kept, const Rest& rest) {
  for (int i = threadIdx.x; i < P.k; i += kThreads) {
    const uint64_t key = i < kept ? S.keys[i] : 0;
    const bool there = key != 0;
    P.values[(int64_t)row * P.k + i] = there ? key_value((uint32_t)(key >> 32)) : kNegInf;
    P.index[(int64_t)row * P.k + i] = there ? (int32_t)~(uint32_t)key : -1;
  }
  if (threadIdx.x == 0)  // the exponents are of fp32's log2(e), so that one is divided out
    P.rest_lse[row] = rest.sum > 0.f
                          ? (float)(((double)rest.ref + (double)lg2(rest.sum)) / (double)kLog2e)
                          : kNegInf;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_topk(TopkParams P) {
  using V = Vec<BF16>;
  constexpr int EPV = V::EPV;
  __shared__ Shared S;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / P.n_seg, seg = blockIdx.x - row * P.n_seg;
  const uint8_t* yr = P.y + (int64_t)row * P.ld_bytes;
  const int v0 = seg * P.seg_vec, v1 = min(v0 + P.seg_vec, P.nvec);
  const int k = P.k;
  Rest rest;
  if (tid == 0) S.count = 0;

  u32x4 raw[kGroupVec];
  auto load = [&](int g0) {
#pragma unroll
    for (int u = 0; u < kGroupVec; ++u) {
      const int v = g0 + u * kThreads + tid;
      raw[u] = v < v1 ? load16_nt(yr + (int64_t)v * 16) : u32x4{0, 0, 0, 0};
    }
  };
  // Elements of vector v, NaN-free; those past the vocabulary are not there (`valid` of them are).
  auto valid_of = [&](int v) { return v < v1 ? min(EPV, P.vocab - v * EPV) : 0; };

  load(v0);
  {  // the first bound: the k-th largest of the threads' maxima
    float m = kNegInf;
#pragma unroll
    for (int u = 0; u < kGroupVec; ++u) {
      const int valid = valid_of(v0 + u * kThreads + tid);
      float x[EPV];
      V::unpack(raw[u], x);
#pragma unroll
      for (int e = 0; e < EPV; ++e)
        if (e < valid) m = fmaxf(m, x[e]);
    }
    S.part[tid] = m;
    __syncthreads();
    int above = 0;
    for (int i = 0; i < kThreads; ++i) {
      const float o = S.part[i];
      above += (o > m || (o == m && i < tid)) ? 1 : 0;
    }
    if (above == k - 1) S.bound = m;
    __syncthreads();
  }
  float bound = S.bound;
  // Until the buffer has once been cut to k, an element equal to the bound may belong to the list;
  // from then on it cannot: k keys at or above the bound are held, and its index is higher than theirs.
  bool strict = false;
  int n = 0;
  auto above = [&](float x) { return strict ? x > bound : x >= bound; };
  auto append = [&](float x, int index) {
    const int at = atomicAdd(&S.count, 1);
    if (at < kTopkCap) S.keys[at] = make_key(x, index);
  };

  for (int g0 = v0; g0 < v1; g0 += kThreads * kGroupVec) {
    if (g0 != v0) load(g0);
#pragma unroll
    for (int u = 0; u < kGroupVec; ++u) {
      const int v = g0 + u * kThreads + tid;
      const int valid = valid_of(v);
      float x[EPV];
      V::unpack(raw[u], x);
      float m = kNegInf;
#pragma unroll
      for (int e = 0; e < EPV; ++e)
        if (e < valid && !above(x[e])) m = fmaxf(m, x[e]);
      rest.raise(m);
#pragma unroll
      for (int e = 0; e < EPV; ++e)
        if (e < valid) {
          if (above(x[e]))
            append(x[e], v * EPV + e);
          else
            rest.add(x[e]);
        }
    }
    __syncthreads();
    const int total = S.count;
    __syncthreads();
    if (total <= kTopkCap) {
      n = total;
      if (n > kTopkCap / 2) {
        n = settle(S, n, k, rest);
        if (n == k) {
          bound = S.bound;
          strict = true;
        }
      }
      continue;
    }
    // More candidates than places: back to the n keys of before the group, then one vector per thread
    // at a time, cutting before the buffer could run over.
    const float old_bound = bound;
    const bool old_strict = strict;
    __syncthreads();
    if (tid == 0) S.count = n;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kGroupVec; ++u) {
      if (n + kThreads * EPV > kTopkCap) {
        n = settle(S, n, k, rest);
        if (n == k) {
          bound = S.bound;
          strict = true;
        }
      }
      const int v = g0 + u * kThreads + tid;
      const int valid = valid_of(v);
      float x[EPV];
      V::unpack(raw[u], x);
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        const bool was = old_strict ? x[e] > old_bound : x[e] >= old_bound;
        if (e < valid && was) {  // (the others are in the sum already)
          if (above(x[e])) {
            append(x[e], v * EPV + e);
          } else {
            rest.raise(x[e]);
            rest.add(x[e]);
          }
        }
      }
      __syncthreads();
      n = S.count;
      __syncthreads();
    }
  }
  const int kept = settle(S, n, k, rest);
  join_rest(S, rest);
  if (P.n_seg == 1) {
    write_row(P, S, row, kept, rest);
  } else {
    uint64_t* keys = P.seg_keys + (int64_t)blockIdx.x * k;
    for (int i = tid; i < k; i += kThreads) keys[i] = i < kept ? S.keys[i] : 0;
    if (tid == 0) {
      P.seg_lse[2 * (int64_t)blockIdx.x] = rest.ref;
      P.seg_lse[2 * (int64_t)blockIdx.x + 1] = rest.sum;
    }
  }
}

// One workgroup per row: the segments' keys together are few enough to be sorted at once.
__global__ void __launch_bounds__(kThreads) k_topk_merge(TopkParams P) {
  __shared__ Shared S;
  const int tid = threadIdx.x, row = blockIdx.x;
  const int total = P.n_seg * P.k;
  const uint64_t* keys = P.seg_keys + (int64_t)row * total;
  for (int i = tid; i < total; i += kThreads) S.keys[i] = keys[i];
  Rest rest;
  for (int i = tid; i < P.n_seg; i += kThreads) {
    const float* p = P.seg_lse + 2 * ((int64_t)row * P.n_seg + i);
    lse_join(rest.ref, rest.sum, p[0], p[1]);
  }
  __syncthreads();
  const int kept = settle(S, total, P.k, rest);
  join_rest(S, rest);
  write_row(P, S, row, kept, rest);
}

}  // namespace

void topk_split(int64_t n_rows, int32_t nvec, int32_t k, int32_t* n_seg, int32_t* seg_vec) {
  // One workgroup per row once the rows alone give every CU two; with fewer, enough segments for that,
  // of at least two vectors per thread, and at most as many as one workgroup can merge.
  int64_t seg = n_rows > 0 ? (512 + n_rows - 1) / n_rows : 1;
  seg = std::min<int64_t>(seg, (nvec + 2 * kThreads - 1) / (2 * kThreads));
  seg = std::min<int64_t>(seg, kTopkCap / k);
  seg = std::max<int64_t>(seg, 1);
  *seg_vec = (int32_t)((nvec + seg - 1) / seg);
  *n_seg = (nvec + *seg_vec - 1) / *seg_vec;
}

hipError_t launch_topk(const TopkParams& p, int in_bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.n_rows * p.n_seg));
  if (in_bf16)
    hipLaunchKernelGGL(k_topk<true>, grid, dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL(k_topk<false>, grid, dim3(kThreads), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.n_seg == 1) return e;
  hipLaunchKernelGGL(k_topk_merge, dim3((unsigned)p.n_rows), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace opd
