// The k largest logits of every row and the log-sum-exp of all the others, in one pass over the row.
//
// A workgroup takes a segment of a row (the whole row where there are rows enough to fill the device).
// Its first vectors are loaded into registers at once; the k-th largest of the maxima of groups of
// threads over them is a lower bound of the k-th largest logit. From there on an element at or above the
// bound is a candidate and goes, as a 64-bit key (value's order in the upper half, falling index in the
// lower, so that no two are the same), into a buffer in LDS, and any other adds 2^((x - bound) log2 e) to
// its thread's sum; what is not in registers is streamed past the same bound. Candidates are few (for
// random order k times the segment's length over the held part's). They are ranked by counting, the k
// largest are the answer, and the others join the sums in the order of their rank. The sum of the others
// is never formed by subtracting the listed ones, which would lose what is left where the list holds
// nearly all of the row; where the bound turns out to be no reference for it (all others so far below
// that their terms vanish), the segment is gone over once more for the sum alone.
//
// When the buffer would run over (rows of equal values; rising rows), it is cut to the k largest and the
// bound raised to the k-th, after every few vectors if need be. Every set and every order of additions
// depends on the data alone, not on the order in which candidates reach the buffer, so results are the
// same bits every time.
//
// This file is compiled with the IEEE mode off, like the row kernels: NaN is outside the contract.

#include <stdint.h>

#include <algorithm>

#include "opd_internal.h"
#include "opd_rows.h"

namespace opd {
namespace {

constexpr int kLoose = 4;        // vectors in flight per thread of what is not held
constexpr int kBatch = 256;      // threads that append between two checks where the buffer runs over
constexpr int kRankMost = 512;   // candidates up to which ranking by counting beats sorting
constexpr uint32_t kKeyNegInf = 0x007fffffu;

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

// A thread's share of a log-sum-exp: sum * 2^ref. The reference may lag the largest exponent by up to
// 24: 2^24 an element leaves fp32 range to spare.
struct Rest {
  float ref = kNoRef, sum = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float c = x * kLog2e;
    if (c > ref + 24.f) {
      sum *= ex2(ref - c);
      ref = c;
    }
    sum += ex2(__builtin_fmaf(x, kLog2e, -ref));
  }
};

// The bound: elements at or above it are candidates. Once the buffer has been cut to k it is the next
// number above the k-th: k keys above that are held, and the index of an element equal to the k-th that
// comes later is higher than theirs.
__device__ __forceinline__ float bound_after_cut(float kth) { return key_value(order_key(kth) + 1u); }

// The sum of a thread's elements that were no candidates, relative to the bound (none is above it).
struct Low {
  float ref, sum = 0.f;
  __device__ __forceinline__ void rebase(float bound) {
    const float r = fmaxf(bound * kLog2e, kNoRef);
    sum *= ex2(ref - r);
    ref = r;
  }
};

// Ends the arithmetic of a vector here: the compiler would otherwise keep vectors in unpacked form and put
// their sums off together, which costs the registers that the row needs.
__device__ __forceinline__ void settle(u32x4& v, Low& low) { asm volatile("" : "+v"(v), "+v"(low.sum)); }

struct Shared {
  uint64_t keys[kTopkCap];
  uint64_t sorted[kRankMost];
  uint32_t maxima[512];
  float pair[16][2];
  float bound;
  int count;
};

// The first bound: the k-th largest of m maxima' keys in S.maxima (one wave; m a multiple of 64), as far as
// its upper `bits` bits say, rounded down; -inf where there are not k.
template <int M>
__device__ void find_bound(Shared& S, int k, int bits) {
  const int lane = thread_x() & 63;
  uint32_t key[M / 64];
#pragma unroll
  for (int i = 0; i < M / 64; ++i) key[i] = S.maxima[i * 64 + lane];
  uint32_t p = 0;
  for (int b = 31; b >= 32 - bits; --b) {
    const uint32_t q = p | (1u << b);
    int n = 0;
#pragma unroll
    for (int i = 0; i < M / 64; ++i) n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] >= q));
    if (n >= k) p = q;
  }
  if (lane == 0) S.bound = key_value(max(p, kKeyNegInf));
}

// Orders the n keys in S.keys (largest first), keeps the k largest there and adds the others to the
// threads' sums in the order of their rank. Returns the number kept; S.bound is the k-th's value. All T
// threads call it.
template <int T>
__device__ int cut(Shared& S, int n, int k, Rest& rest) {
  const int tid = thread_x();
  const uint64_t* from = S.keys;
  if (n <= kRankMost) {
    for (int i = tid; i < n; i += T) {
      const uint64_t mine = S.keys[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += S.keys[j] > mine ? 1 : 0;
      S.sorted[rank] = mine;
    }
    lds_barrier();
    from = S.sorted;
  } else {
    int m = 1024;
    while (m < n) m <<= 1;
    for (int i = n + tid; i < m; i += T) S.keys[i] = 0;
    lds_barrier();
    for (int size = 2; size <= m; size <<= 1)
      for (int stride = size >> 1; stride > 0; stride >>= 1) {
        for (int i = tid; i < m / 2; i += T) {
          const int a = 2 * i - (i & (stride - 1)), b = a + stride;
          const uint64_t x = S.keys[a], y = S.keys[b];
          if ((x < y) == ((a & size) == 0)) {
            S.keys[a] = y;
            S.keys[b] = x;
          }
        }
        lds_barrier();
      }
  }
  for (int i = k + tid; i < n; i += T) rest.add(key_value((uint32_t)(from[i] >> 32)));
  const int kept = min(n, k);
  if (from != S.keys)
    for (int i = tid; i < kept; i += T) S.keys[i] = from[i];
  if (tid == 0) {
    S.count = kept;
    S.bound = n >= k ? key_value((uint32_t)(from[k - 1] >> 32)) : kNegInf;
  }
  lds_barrier();
  return kept;
}

// Joins the threads' sums; the first wave has the result.
template <int T>
__device__ void join_rest(Shared& S, Rest& rest) {
  const int tid = thread_x();
  wave_lse(rest.ref, rest.sum);
  if ((tid & 63) == 0) {
    S.pair[tid >> 6][0] = rest.ref;
    S.pair[tid >> 6][1] = rest.sum;
  }
  lds_barrier();
  if (tid < 64) {
    rest.ref = tid < T / 64 ? S.pair[tid][0] : kNoRef;
    rest.sum = tid < T / 64 ? S.pair[tid][1] : 0.f;
    wave_lse(rest.ref, rest.sum);
  }
}

// Writes a row's answer: the first `kept` keys (an entry that is not there: index -1) and the sum.
template <int T>
__device__ void write_row(const TopkParams& P, const Shared& S, int row, int kept, const Rest& rest) {
  for (int i = thread_x(); i < P.k; i += T) {
    const uint64_t key = i < kept ? S.keys[i] : 0;
    P.values[(int64_t)row * P.k + i] = key ? key_value((uint32_t)(key >> 32)) : kNegInf;
    P.index[(int64_t)row * P.k + i] = key ? (int32_t)~(uint32_t)key : -1;
  }
  if (thread_x() == 0)  // the exponents are of fp32's log2(e), so that one is divided out
    P.rest_lse[row] = rest.sum > 0.f
                          ? (float)(((double)rest.ref + (double)lg2(rest.sum)) / (double)kLog2e)
                          : kNegInf;
}

// One vector: candidates into the buffer, the others into the sum. The few lanes with candidates are taken
// one by one, the wave's first lanes trying one element each.
template <bool BF16>
__device__ __forceinline__ void take(Shared& S, float bound, Low& low, const u32x4& raw, float (&x)[Vec<BF16>::EPV],
                                     int first, int end) {
  using V = Vec<BF16>;
  constexpr int EPV = V::EPV;
  float m = x[0];
#pragma unroll
  for (int e = 1; e < EPV; ++e) m = fmaxf(m, x[e]);
  uint64_t lanes = __builtin_amdgcn_ballot_w64(m >= bound);
  if (lanes) {
    const int lane = thread_x() & 63;
    do {
      const int from = __builtin_ctzll(lanes);
      lanes &= lanes - 1;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (uint32_t)__builtin_amdgcn_readlane((int)raw[j], from);
      const int at = __builtin_amdgcn_readlane(first, from) + lane;
      const int j = BF16 ? lane >> 1 : lane;
      const uint32_t word = j == 0 ? w[0] : j == 1 ? w[1] : j == 2 ? w[2] : w[3];
      const float v = __uint_as_float(!BF16 || (lane & 1) ? word & (BF16 ? 0xffff0000u : ~0u) : word << 16);
      if (lane < EPV && v >= bound && at < end) {
        const int place = atomicAdd(&S.count, 1);
        if (place < kTopkCap) S.keys[place] = make_key(v, at);
      }
    } while (lanes);
#pragma unroll
    for (int e = 0; e < EPV; ++e) x[e] = x[e] >= bound ? kNegInf : x[e];
  }
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < EPV; ++e) s += ex2(__builtin_fmaf(x[e], kLog2e, -low.ref));
  low.sum += s;
}

// The candidates of one vector per thread again, in batches of threads, cutting the buffer before it could
// run over (`was`: the bound that take() went by; the others are in the sum already). All threads.
template <int EPV, int T>
__device__ void take_again(Shared& S, float& bound, float was, Rest& rest, const float (&x)[EPV], int first, int end,
                           int& n, int k) {
  for (int b = 0; b < T / kBatch; ++b) {
    if (n + kBatch * EPV > kTopkCap) {
      n = cut<T>(S, n, k, rest);
      if (n == k) bound = bound_after_cut(S.bound);
    }
    if (thread_x() / kBatch == b) {
#pragma unroll
      for (int e = 0; e < EPV; ++e)
        if (x[e] >= was && first + e < end) {
          if (x[e] >= bound)
            S.keys[atomicAdd(&S.count, 1)] = make_key(x[e], first + e);
          else
            rest.add(x[e]);
        }
    }
    lds_barrier();
    n = S.count;
    lds_barrier();
  }
}

// One workgroup of T threads per (row, segment); H vectors per thread are held. M: maxima that the first
// bound is found from.
template <bool BF16, int T, int H, int M>
__global__ void __launch_bounds__(T) k_topk(TopkParams P) {
  using V = Vec<BF16>;
  constexpr int EPV = V::EPV;
  constexpr int U = kLoose;
  __shared__ Shared S;
  const int tid = thread_x();
  const int row = group_x(), seg = group_y();
  const int v0 = seg * P.seg_vec, n_vec = min(P.seg_vec, P.nvec - v0), k = P.k;
  const int base = v0 * EPV, end = min((v0 + n_vec) * EPV, P.vocab);  // tokens [base, end)
  const RowBuf in = row_buf(P.y + (int64_t)row * P.ld_bytes + (int64_t)v0 * 16, (uint32_t)n_vec * 16u);
  if (tid == 0) S.count = 0;

  // Vector v + tid; its elements past the segment's end become -inf.
  auto unpack = [&](u32x4& raw, int v, float (&x)[EPV]) {
    V::unpack(raw, x);
    if (base + (v + T) * EPV > end) {
#pragma unroll
      for (int e = 0; e < EPV; ++e) x[e] = base + (v + tid) * EPV + e < end ? x[e] : kNegInf;
    }
  };

  u32x4 held[H];
#pragma unroll
  for (int i = 0; i < H; ++i) held[i] = buf_load16<kStream>(in, (uint32_t)tid * 16u, (uint32_t)(i * T) * 16u);
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < H; ++i)
    if (i * T < n_vec) {
      if (base + (i * T + T) * EPV > end) {
        float x[EPV];
        unpack(held[i], i * T, x);
#pragma unroll
        for (int e = 0; e < EPV; ++e) m = fmaxf(m, x[e]);
      } else {
        m = V::max(held[i], m);
      }
      asm volatile("" : "+v"(held[i]), "+v"(m));
    }
  {
    constexpr int G = T / M;  // threads per maximum: neighbours
    static_assert(G == 1 || G == 2 || G == 4, "maxima of one, two or four lanes");
    float g = V::max_value(m);
    if (G >= 2) g = fmaxf(g, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(g), 0xB1, 0xF, 0xF, true)));
    if (G >= 4) g = fmaxf(g, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(g), 0x4E, 0xF, 0xF, true)));
    // (-inf is also what a group without elements has: no maximum, so that fewer than k of them are seen)
    if (tid % G == 0) S.maxima[tid / G] = g > kNegInf ? order_key(g) : 0u;
  }
  lds_barrier();
  if (tid < 64) find_bound<M>(S, k, BF16 ? 16 : 24);
  lds_barrier();
  float bound = S.bound;
  Rest rest;
  Low low;
  low.ref = fmaxf(bound * kLog2e, kNoRef);
#pragma unroll
  for (int i = 0; i < H; ++i)
    if (i * T < n_vec) {
      float x[EPV];
      unpack(held[i], i * T, x);
      take<BF16>(S, bound, low, held[i], x, base + (i * T + tid) * EPV, end);
      settle(held[i], low);
    }
  // What has been gone over ends at vector g1: the held ones, then U per thread at a time.
  int n = 0, g0 = 0, g1 = H * T;
  for (;;) {
    if (g0 > 0) {
      u32x4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = buf_load16<kStream>(in, (uint32_t)tid * 16u, (uint32_t)(g0 + u * T) * 16u);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[EPV];
        unpack(raw[u], g0 + u * T, x);
        take<BF16>(S, bound, low, raw[u], x, base + (g0 + u * T + tid) * EPV, end);
        settle(raw[u], low);
      }
    }
    const bool last = g1 >= n_vec;
    lds_barrier();
    const int total = S.count;
    lds_barrier();
    if (total <= kTopkCap) {
      n = total;
    } else {
      // more candidates than places: back to the keys of before, and those vectors again
      if (tid == 0) S.count = n;
      lds_barrier();
      const float was = bound;
      for (int v = g0; v < g1 && v < n_vec; v += T) {
        u32x4 raw = buf_load16<kCached>(in, (uint32_t)tid * 16u, (uint32_t)v * 16u);
        float x[EPV];
        unpack(raw, v, x);
        take_again<EPV, T>(S, bound, was, rest, x, base + (v + tid) * EPV, end, n, k);
      }
      low.rebase(bound);
    }
    if (last) break;
    if (n > kTopkCap / 4) {
      n = cut<T>(S, n, k, rest);
      if (n == k) bound = bound_after_cut(S.bound);
      low.rebase(bound);
    }
    g0 = g1;
    g1 += U * T;
  }
  const int kept = cut<T>(S, n, k, rest);
  // The bound was a reference for the sum if the terms add up to something (2^-40 of the bound's own
  // leaves those below fp32's smallest number 2^86 times less); else the others again, by themselves.
  {
    float t = wave_sum(low.sum);
    if ((tid & 63) == 0) S.pair[tid >> 6][0] = t;
    lds_barrier();
    t = 0.f;
    for (int w = 0; w < T / 64; ++w) t += S.pair[w][0];
    lds_barrier();
    if (t >= 0x1p-40f) {
      lse_join(rest.ref, rest.sum, low.ref, low.sum);
    } else {
      rest = Rest{};
      const uint64_t least = kept == k ? S.keys[k - 1] : 0;
      for (int v = 0; v < n_vec; v += T) {
        u32x4 raw = buf_load16<kCached>(in, (uint32_t)tid * 16u, (uint32_t)v * 16u);
        float x[EPV];
        unpack(raw, v, x);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const int i = base + (v + tid) * EPV + e;
          if (i < end && make_key(x[e], i) < least) rest.add(x[e]);
        }
      }
    }
  }
  join_rest<T>(S, rest);
  if (P.n_seg == 1) {
    write_row<T>(P, S, row, kept, rest);
  } else {
    const int64_t unit = (int64_t)row * P.n_seg + seg;
    uint64_t* keys = P.seg_keys + unit * k;
    for (int i = tid; i < k; i += T) keys[i] = i < kept ? S.keys[i] : 0;
    if (tid == 0) {
      P.seg_lse[2 * unit] = rest.ref;
      P.seg_lse[2 * unit + 1] = rest.sum;
    }
  }
}

// One workgroup per row joins the segments' lists and sums: again a bound from the threads' maxima, the keys
// at or above it ranked, the others added to the sums by the threads that loaded them.
__global__ void __launch_bounds__(kThreads) k_topk_merge(TopkParams P) {
  constexpr int T = kThreads, R = kTopkCap / T;
  __shared__ Shared S;
  const int tid = thread_x(), row = group_x(), k = P.k;
  const int total = P.n_seg * k;
  const uint64_t* keys = P.seg_keys + (int64_t)row * total;
  uint64_t mine[R];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    mine[i] = i * T + tid < total ? keys[i * T + tid] : 0;
    m = max(m, (uint32_t)(mine[i] >> 32));
  }
  Rest rest;
  for (int i = tid; i < P.n_seg; i += T) {
    const float* p = P.seg_lse + 2 * ((int64_t)row * P.n_seg + i);
    lse_join(rest.ref, rest.sum, p[0], p[1]);
  }
  if (tid == 0) S.count = 0;
  S.maxima[tid] = m;
  lds_barrier();
  if (tid < 64) find_bound<T>(S, k, 32);
  lds_barrier();
  const float bound = S.bound;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (mine[i] == 0) continue;  // (a list that was not full)
    const float x = key_value((uint32_t)(mine[i] >> 32));
    if (x >= bound)
      S.keys[atomicAdd(&S.count, 1)] = mine[i];
    else
      rest.add(x);
  }
  lds_barrier();
  const int kept = cut<T>(S, S.count, k, rest);
  join_rest<T>(S, rest);
  write_row<T>(P, S, row, kept, rest);
}

constexpr int kWholeRows = 192;  // rows from which a workgroup per row is faster than split rows

template <bool BF16, int T, int H, int M>
hipError_t launch(const TopkParams& p, hipStream_t s) {
  hipLaunchKernelGGL((k_topk<BF16, T, H, M>), dim3((unsigned)p.n_rows, (unsigned)p.n_seg), dim3(T), 0, s, p);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_rows(const TopkParams& p, hipStream_t s) {
  if (p.seg_vec <= 256 * 8) return launch<BF16, 256, 8, 256>(p, s);
  if (p.seg_vec <= 512 * 10) return launch<BF16, 512, 10, 512>(p, s);
  if (p.n_rows < 512) return p.k <= 96 ? launch<BF16, 1024, 19, 256>(p, s) : launch<BF16, 1024, 19, 512>(p, s);
  return p.k <= 96 ? launch<BF16, 512, 12, 256>(p, s) : launch<BF16, 512, 12, 512>(p, s);
}

}  // namespace

void topk_split(int64_t n_rows, int32_t nvec, int32_t k, int32_t* n_seg, int32_t* seg_vec) {
  // Few rows: segments for two workgroups of 256 threads per CU, of at least four vectors per thread, and at
  // most as many as one workgroup can merge.
  int64_t seg = 1;
  if (n_rows > 0 && n_rows < kWholeRows) {
    seg = (1024 + n_rows - 1) / n_rows;
    seg = std::min<int64_t>(seg, (nvec + 4 * kThreads - 1) / (4 * kThreads));
    seg = std::min<int64_t>(seg, kTopkCap / k);
    seg = std::max<int64_t>(seg, 1);
  }
  *seg_vec = (int32_t)(((nvec + seg - 1) / seg + 7) / 8 * 8);
  *n_seg = (nvec + *seg_vec - 1) / *seg_vec;
}

hipError_t launch_topk(const TopkParams& p, int in_bf16, hipStream_t s) {
  const hipError_t e = in_bf16 ? launch_rows<true>(p, s) : launch_rows<false>(p, s);
  if (e != hipSuccess || p.n_seg == 1) return e;
  hipLaunchKernelGGL(k_topk_merge, dim3((unsigned)p.n_rows), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace opd
