// Distillation from a teacher's top logits: loss, statistics and gradient of drafter rows against k
// listed target logits and the log-sum-exp of the target's others.
//
// The classes of a row are its k listed tokens and, as one, all the others. With p the drafter's and q
// the teacher's distribution over the classes (fp32, logarithms to base 2 inside):
//   reverse  term_c = p_c (ln p_c - ln q_c),  g_c = [unclipped] (ln p_c - ln q_c + 1), S = sum p_c g_c,
//            d_c = alpha p_c (g_c - S)
//   forward  term_c = q_c (ln q_c - ln p_c),  u_c = [unclipped] q_c, Q = sum u_c, d_c = alpha (Q p_c - u_c)
//   and d_c += (1 - alpha) (p_c - [c = a]); the gradient of a listed token is w d_c, that of any other
//   token j its share of its class's: w d_rest 2^(z_j log2 e - L), L the log2-sum over the others.
// So a row costs one exp2 an element for L and one for the gradient, and HBM bounds it. The others'
// sum leaves the listed tokens out element by element (a bitmap of the segment in LDS names them)
// instead of subtracting them from the row's sum, which would lose what is left where the drafter has
// learned the list.
//
// This file is compiled with the IEEE mode off, like the row kernels: NaN is outside the contract.

#include <stdint.h>

#include <algorithm>

#include "opd_internal.h"
#include "opd_rows.h"

namespace opd {
namespace {

constexpr int kSegVec = 4096;   // most vectors of a segment: its bitmap has one byte a vector
constexpr int kWaves = kThreads / 64;
constexpr float kLn2 = 0.69314718055994530942f;
static_assert(kTopkMax <= kThreads, "one thread per listed token");

struct Shared {
  int32_t index[kTopkMax];
  uint32_t listed[kSegVec / 4];  // bit e of byte v: element e of the segment's vector v is listed
  float red[kWaves][2];
};

__device__ float block_sum(Shared& S, float x) {
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) S.red[threadIdx.x >> 6][0] = x;
  __syncthreads();
  float t = S.red[0][0];
  for (int w = 1; w < kWaves; ++w) t += S.red[w][0];
  return t;
}

__device__ float block_max(Shared& S, float x) {
  x = wave_max(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) S.red[threadIdx.x >> 6][0] = x;
  __syncthreads();
  float t = S.red[0][0];
  for (int w = 1; w < kWaves; ++w) t = fmaxf(t, S.red[w][0]);
  return t;
}

// Entry threadIdx.x of the row's list: its token, or -1 where there is none that counts.
__device__ int list_entry(const TopkLossParams& P, Shared& S, int row, bool report) {
  const int tid = threadIdx.x;
  int idx = tid < P.k ? P.top_index[(int64_t)row * P.k + tid] : -1;
  if (idx >= P.vocab) {
    if (report) atomicOr(P.flags, kFlagBadToken);
    idx = -1;
  }
  if (tid < kTopkMax) S.index[tid] = idx;
  __syncthreads();
  bool twice = false;
  for (int i = 0; i < tid && i < P.k; ++i) twice |= S.index[i] == idx;
  if (idx >= 0 && twice) {
    if (report) atomicOr(P.flags, kFlagBadList);
    idx = -1;
  }
  return idx;
}

// Marks the listed tokens of vectors [v0, v0 + kSegVec) in S.listed.
template <int EPV>
__device__ void mark_listed(Shared& S, int idx, int v0) {
  for (int i = threadIdx.x; i < kSegVec / 4; i += kThreads) S.listed[i] = 0u;
  __syncthreads();
  const int v = idx >= 0 ? idx / EPV - v0 : -1;
  if (v >= 0 && v < kSegVec) atomicOr(&S.listed[v >> 2], 1u << (8 * (v & 3) + idx % EPV));
  __syncthreads();
}

// What a row's classes give: thread i has listed token i's derivative, every thread the rest's.
struct RowResult {
  float loss, divergence, lse;
  float d;       // d loss / d z of this thread's listed token
  float d_rest;  // derivative of the class of all others
};

// rest_ref, rest_l2: reference and log2 of the sum over the tokens not listed.
template <bool BF16>
__device__ RowResult row_classes(const TopkLossParams& P, Shared& S, int row, int idx, float rest_ref, float rest_l2) {
  const int tid = threadIdx.x;
  const uint8_t* zr = P.z + (int64_t)row * P.ld_bytes;
  const float t = idx >= 0 ? P.top_logit[(int64_t)row * P.k + tid] : kNegInf;
  const float z = idx >= 0 ? Vec<BF16>::elem(zr, idx) : kNegInf;
  const float t_rest = P.rest_lse ? P.rest_lse[row] : kNegInf;
  RowResult r;
  const float t_top = block_max(S, t);
  if (!(t_top > kNegInf)) {  // nothing listed: the row takes no part
    r.loss = r.divergence = r.d = r.d_rest = 0.f;
    const float zm = fmaxf(block_max(S, z) * kLog2e, rest_ref);
    const float sum = block_sum(S, ex2(__builtin_fmaf(z, kLog2e, -zm))) + ex2((rest_ref - zm) + rest_l2);
    r.lse = (float)(((double)zm + (double)lg2(sum)) / (double)kLog2e);
    return r;
  }
  // the drafter's distribution over the classes
  const float zm = fmaxf(block_max(S, z) * kLog2e, rest_ref);
  const float ez = __builtin_fmaf(z, kLog2e, -zm), ez_rest = (rest_ref - zm) + rest_l2;
  const float lz = lg2(block_sum(S, ex2(ez)) + ex2(ez_rest));
  r.lse = (float)(((double)zm + (double)lz) / (double)kLog2e);
  const float lp = (ez - lz) * kLn2, lp_rest = (ez_rest - lz) * kLn2;
  const float p = ex2(ez - lz), p_rest = ex2(ez_rest - lz);
  // the teacher's
  const float tm = fmaxf(t_top, t_rest) * kLog2e;
  const float et = __builtin_fmaf(t, kLog2e, -tm), et_rest = __builtin_fmaf(t_rest, kLog2e, -tm);
  const float lt = lg2(block_sum(S, ex2(et)) + ex2(et_rest));
  const float lq = (et - lt) * kLn2, lq_rest = (et_rest - lt) * kLn2;
  const float q = ex2(et - lt), q_rest = ex2(et_rest - lt);
  // its top-1: the lowest token of the largest logit
  float best = t == t_top ? (float)idx : 3e38f;  // (indices below 2^24 are exact)
  best = -block_max(S, -best);
  const float hard = idx >= 0 && (float)idx == best ? 1.f : 0.f;
  // (0 ln 0 = 0; a listed token of another's probability 0 has an infinite term, clipped for any tau)
  float term, term_rest, d, d_rest, sum;
  if (P.kl == OPD_KL_REVERSE) {
    term = p > 0.f ? p * (lp - lq) : 0.f;
    term_rest = p_rest > 0.f ? p_rest * (lp_rest - lq_rest) : 0.f;
    const bool in = term <= P.tau && term < __builtin_inff() && p > 0.f;
    const bool in_rest = term_rest <= P.tau && term_rest < __builtin_inff() && p_rest > 0.f;
    const float g = in ? lp - lq + 1.f : 0.f, g_rest = in_rest ? lp_rest - lq_rest + 1.f : 0.f;
    sum = block_sum(S, p * g) + p_rest * g_rest;
    d = p * (g - sum);
    d_rest = p_rest * (g_rest - sum);
  } else {
    term = q > 0.f ? q * (lq - lp) : 0.f;
    term_rest = q_rest > 0.f ? q_rest * (lq_rest - lp_rest) : 0.f;
    const float u = term <= P.tau && term < __builtin_inff() ? q : 0.f;
    const float u_rest = term_rest <= P.tau && term_rest < __builtin_inff() ? q_rest : 0.f;
    sum = block_sum(S, u) + u_rest;
    d = __builtin_fmaf(sum, p, -u);
    d_rest = __builtin_fmaf(sum, p_rest, -u_rest);
  }
  r.divergence = block_sum(S, idx >= 0 ? fminf(term, P.tau) : 0.f) + fminf(term_rest, P.tau);
  const float ce = -block_sum(S, hard > 0.f ? lp : 0.f);
  const float beta = 1.f - P.alpha;
  r.loss = (P.alpha > 0.f ? P.alpha * r.divergence : 0.f) + (beta > 0.f ? beta * ce : 0.f);
  const float w = P.grad_loss ? P.grad_loss[row] : 1.f;
  r.d = w * __builtin_fmaf(P.alpha, d, beta * (p - hard));
  r.d_rest = w * __builtin_fmaf(P.alpha, d_rest, beta * p_rest);
  return r;
}

// One workgroup per (row, segment): reference and sum of the segment's tokens that are not listed.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_topk_loss_sums(TopkLossParams P) {
  using V = Vec<BF16>;
  constexpr int EPV = V::EPV;
  __shared__ Shared S;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / P.n_seg, seg = blockIdx.x - row * P.n_seg;
  const uint8_t* zr = P.z + (int64_t)row * P.ld_bytes;
  const int v0 = seg * P.seg_vec, v1 = min(v0 + P.seg_vec, P.nvec);
  const int idx = list_entry(P, S, row, false);
  mark_listed<EPV>(S, idx, v0);
  float ref = kNoRef, sum = 0.f;
  for (int v = v0 + tid; v < v1; v += kThreads) {
    float x[EPV];
    V::unpack(load16(zr + (int64_t)v * 16), x);
    const uint32_t out = reinterpret_cast<const uint8_t*>(S.listed)[v - v0];
    float m = kNegInf;
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      if ((out >> e & 1) || v * EPV + e >= P.vocab) x[e] = kNegInf;
      m = fmaxf(m, x[e]);
    }
    const float c = m * kLog2e;
    if (c > ref + 24.f) {  // (the sum's exponents stay below 24 + the number of terms' logarithm)
      sum *= ex2(ref - c);
      ref = c;
    }
#pragma unroll
    for (int e = 0; e < EPV; ++e) sum += ex2(__builtin_fmaf(x[e], kLog2e, -ref));
  }
  wave_lse(ref, sum);
  if ((tid & 63) == 0) {
    S.red[tid >> 6][0] = ref;
    S.red[tid >> 6][1] = sum;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWaves; ++w) lse_join(ref, sum, S.red[w][0], S.red[w][1]);
    P.seg_lse[2 * (int64_t)blockIdx.x] = ref;
    P.seg_lse[2 * (int64_t)blockIdx.x + 1] = sum;
  }
}

// One workgroup per row: joins the segments' sums; loss and statistics.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_topk_loss_row(TopkLossParams P) {
  __shared__ Shared S;
  const int tid = threadIdx.x, row = blockIdx.x;
  const int idx = list_entry(P, S, row, true);
  float ref = kNoRef, sum = 0.f;
  for (int i = 0; i < P.n_seg; ++i) {  // every thread the same additions
    const float* p = P.seg_lse + 2 * ((int64_t)row * P.n_seg + i);
    lse_join(ref, sum, p[0], p[1]);
  }
  const float l2 = sum > 0.f ? lg2(sum) : kNegInf;
  const RowResult r = row_classes<BF16>(P, S, row, idx, ref, l2);
  if (tid == 0) {
    P.loss[row] = r.loss;
    float* st = P.row_stats + 4 * (int64_t)row;
    st[0] = ref;
    st[1] = l2;
    st[2] = r.lse;
    st[3] = r.divergence;
  }
}

// One workgroup per (row, segment): the gradient.
template <bool BF16, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads) k_topk_loss_grad(TopkLossParams P) {
  using V = Vec<BF16>;
  using O = Vec<OUT_BF16>;
  constexpr int EPV = V::EPV;
  __shared__ Shared S;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / P.n_seg, seg = blockIdx.x - row * P.n_seg;
  const uint8_t* zr = P.z + (int64_t)row * P.ld_bytes;
  uint8_t* dr = P.dz + (int64_t)row * P.ld_dz_bytes;
  const int v0 = seg * P.seg_vec, v1 = min(v0 + P.seg_vec, P.nvec);
  const int idx = list_entry(P, S, row, false);
  const float ref = P.row_stats[4 * (int64_t)row], l2 = P.row_stats[4 * (int64_t)row + 1];
  const RowResult r = row_classes<BF16>(P, S, row, idx, ref, l2);
  // 2^(z log2 e - L) with L = ref + l2 rounded once, and what the rounding lost made up in the factor
  const bool others = l2 > kNegInf;
  const float L = others ? ref + l2 : 0.f;
  const float factor = others ? r.d_rest * ex2(l2 - (L - ref)) : 0.f;
  for (int v = v0 + tid; v < v1; v += kThreads) {
    float x[EPV];
    V::unpack(load16(zr + (int64_t)v * 16), x);
#pragma unroll
    for (int e = 0; e < EPV; ++e) x[e] = others ? factor * ex2(__builtin_fmaf(x[e], kLog2e, -L)) : 0.f;
    const int valid = P.vocab - v * EPV;
#pragma unroll
    for (int e = 0; e < EPV; ++e)
      if (e < valid) O::put(dr, v * EPV + e, x[e]);
  }
  __syncthreads();  // the listed tokens' places are written over, in this order
  const int v = idx >= 0 ? idx / EPV : -1;
  if (v >= v0 && v < v1) O::put(dr, idx, r.d);
}

}  // namespace

void topk_loss_split(int64_t n_rows, int32_t nvec, int32_t* n_seg, int32_t* seg_vec) {
  // Segments of at most kSegVec vectors; more of them where the rows alone do not fill the device.
  int64_t seg = n_rows > 0 ? (1024 + n_rows - 1) / n_rows : 1;
  seg = std::min<int64_t>(seg, (nvec + 2 * kThreads - 1) / (2 * kThreads));
  seg = std::max<int64_t>(seg, (nvec + kSegVec - 1) / kSegVec);
  *seg_vec = (int32_t)((nvec + seg - 1) / seg);
  *n_seg = (nvec + *seg_vec - 1) / *seg_vec;
}

hipError_t launch_topk_loss_fwd(const TopkLossParams& p, int in_bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.n_rows * p.n_seg));
  if (in_bf16)
    hipLaunchKernelGGL(k_topk_loss_sums<true>, grid, dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL(k_topk_loss_sums<false>, grid, dim3(kThreads), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (in_bf16)
    hipLaunchKernelGGL(k_topk_loss_row<true>, dim3((unsigned)p.n_rows), dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL(k_topk_loss_row<false>, dim3((unsigned)p.n_rows), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_topk_loss_bwd(const TopkLossParams& p, int in_bf16, int out_bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.n_rows * p.n_seg));
  if (in_bf16 && out_bf16)
    hipLaunchKernelGGL((k_topk_loss_grad<true, true>), grid, dim3(kThreads), 0, s, p);
  else if (in_bf16)
    hipLaunchKernelGGL((k_topk_loss_grad<true, false>), grid, dim3(kThreads), 0, s, p);
  else if (out_bf16)
    hipLaunchKernelGGL((k_topk_loss_grad<false, true>), grid, dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL((k_topk_loss_grad<false, false>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace opd
