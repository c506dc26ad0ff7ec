// Penalties for repeated tokens, biases and grammar masks on the logits of packed draft blocks.
//
// Per element (token v, row j of block b; c_v its count in the request's output up to the row,
// known_v whether prompt or output has it):
//   x1 = known_v ? (x > 0 ? x / rho : x rho) : x,  x2 = x1 - f c_v - g [c_v > 0] + bias_v,
//   out = masked ? masked_value : x2,
// one read and one write of every logit, so HBM bounds it: the token counts must not cost a pass of
// their own. A workgroup takes a tile of one block's vocabulary and all of the block's rows (or
// every gridDim.z-th group of kRowGroup rows): it scans the request's history once, counting the
// tile's tokens in LDS, turns the counts into one fp32 number to subtract and two bits per token
// (known; counted in the output), and streams its rows past that state. The proposals of a block's
// earlier rows are added on the way, by the thread that holds the token.

#include <stdint.h>

#include "opd_internal.h"
#include "opd_rows.h"

namespace opd {
namespace {

constexpr int kTileVec = 1024;  // 16-byte vectors of a row that a workgroup takes
constexpr int kRowGroup = 16;   // rows of a block that share one scan of the history

__device__ __forceinline__ int clamp_len(const int32_t* p, int b, int most, bool* bad) {
  const int n = p ? p[b] : most;
  if (n < 0 || n > most) *bad = true;
  return min(max(n, 0), most);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_adjust(AdjustParams P) {
  using V = Vec<BF16>;
  constexpr int EPV = V::EPV;
  constexpr int kTok = kTileVec * EPV;
  __shared__ float sub[kTok];  // first a bias entry's number, then the token's count, then what to subtract
  __shared__ uint32_t known[kTok / 32], counted[kTok / 32];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int start = P.offsets[b], end = P.offsets[b + 1];
  const bool first = blockIdx.x == 0 && blockIdx.z == 0;
  if (start < 0 || end < start || end > P.n_rows) {
    if (first && tid == 0) atomicOr(P.flags, kFlagBadOffsets);
    return;
  }
  const int nb = end - start;
  const int v0 = blockIdx.x * kTileVec;
  const int v1 = min(v0 + kTileVec, P.nvec);
  const int t0 = v0 * EPV;
  const unsigned nt = (unsigned)(min(v1 * EPV, P.vocab) - t0);  // tokens of the tile

  if ((int)blockIdx.x == (int)gridDim.x - 1 && P.mask) {  // the last tile's workgroup is for empty masks
    for (int j0 = blockIdx.z * kRowGroup; j0 < nb; j0 += gridDim.z * kRowGroup)
      for (int j = j0; j < min(j0 + kRowGroup, nb); ++j) {
        const int mr = P.mask_row ? P.mask_row[start + j] : start + j;
        if (mr < 0) continue;
        if (mr >= P.n_masks) {
          if (tid == 0) atomicOr(P.flags, kFlagBadList);
          continue;
        }
        const uint32_t* m = reinterpret_cast<const uint32_t*>(P.mask + (int64_t)mr * P.ld_mask_bytes);
        const int words = (P.vocab + 31) / 32;
        bool any = false;
        for (int w0 = 0; w0 < words && !any; w0 += kThreads) {
          const int w = w0 + tid;
          uint32_t bits = w < words ? m[w] : 0u;
          if (w == words - 1 && (P.vocab & 31)) bits &= (1u << (P.vocab & 31)) - 1u;
          any = __syncthreads_or(bits != 0u);
        }
        if (!any && tid == 0) atomicOr(P.flags, kFlagEmptyMask);
      }
    return;
  }

  const float rho = P.repetition ? P.repetition[b] : 1.f;
  const float inv_rho = 1.f / rho;
  const float freq = P.frequency ? P.frequency[b] : 0.f;
  const float pres = P.presence ? P.presence[b] : 0.f;
  bool bad_list = false, bad_token = false;
  const int n_hist = P.history ? clamp_len(P.history_len, b, P.max_history, &bad_list) : 0;
  int n_prompt = 0;
  if (P.history && P.prompt_len) n_prompt = clamp_len(P.prompt_len, b, n_hist, &bad_list);
  const int n_bias = P.bias_tokens ? clamp_len(P.bias_len, b, P.max_bias, &bad_list) : 0;
  const int32_t* hist = P.history + (int64_t)b * P.ld_history;
  const int32_t* btok = P.bias_tokens + (int64_t)b * P.ld_bias;
  const float* bval = P.bias_values + (int64_t)b * P.ld_bias;
  uint32_t* count = reinterpret_cast<uint32_t*>(sub);

  for (int j0 = blockIdx.z * kRowGroup; j0 < nb; j0 += gridDim.z * kRowGroup) {
    const int rows = min(kRowGroup, nb - j0);
    __syncthreads();  // the previous group's rows are done with the state
    for (int i = tid; i < kTok; i += kThreads) count[i] = 0u;
    for (int i = tid; i < kTok / 32; i += kThreads) known[i] = counted[i] = 0u;
    __syncthreads();
    // Which bias entries count: the last of a token's, found as the largest number in its slot.
    uint64_t mine = 0;  // entries tid, tid + kThreads, ... of this thread that count
    if (n_bias) {
      for (int i = tid; i < n_bias; i += kThreads) {
        const unsigned t = (unsigned)(btok[i] - t0);
        if ((unsigned)btok[i] >= (unsigned)P.vocab) bad_token = true;
        else if (t < nt) atomicMax(&count[t], (uint32_t)i + 1u);
      }
      __syncthreads();
      int q = 0;
      for (int i = tid; i < n_bias; i += kThreads, ++q) {
        const unsigned t = (unsigned)(btok[i] - t0);
        if ((unsigned)btok[i] < (unsigned)P.vocab && t < nt && count[t] == (uint32_t)i + 1u) mine |= 1ull << q;
      }
      __syncthreads();
      q = 0;
      for (int i = tid; i < n_bias; i += kThreads, ++q)
        if (mine >> q & 1) count[btok[i] - t0] = 0u;
      __syncthreads();
    }
    // Counts: the history, then the proposals of the block's rows before this group.
    const int n_draft = P.draft ? j0 : 0;
    for (int i = tid; i < n_hist + n_draft; i += kThreads) {
      const int tok = i < n_hist ? hist[i] : P.draft[start + i - n_hist];
      if ((unsigned)tok >= (unsigned)P.vocab) {
        bad_token = true;
        continue;
      }
      const unsigned t = (unsigned)(tok - t0);
      if (t < nt) {
        atomicOr(&known[t >> 5], 1u << (t & 31));
        if (i >= n_prompt) atomicAdd(&count[t], 1u);
      }
    }
    __syncthreads();
    for (int w = tid; w < kTok / 32; w += kThreads) {
      uint32_t bits = 0;
      for (int i = 0; i < 32; ++i) {
        const uint32_t c = count[32 * w + i];
        sub[32 * w + i] = c ? __builtin_fmaf(freq, (float)c, pres) : 0.f;
        bits |= (c ? 1u : 0u) << i;
      }
      counted[w] = bits;
    }
    __syncthreads();
    if (mine) {
      int q = 0;
      for (int i = tid; i < n_bias; i += kThreads, ++q)
        if (mine >> q & 1) sub[btok[i] - t0] -= bval[i];
    }
    __syncthreads();

    for (int v = v0 + tid; v < v1; v += kThreads) {
      const int e0 = (v - v0) * EPV;
      float s[EPV];
#pragma unroll
      for (int e = 0; e < EPV; ++e) s[e] = sub[e0 + e];
      uint32_t kn = known[e0 >> 5] >> (e0 & 31), co = counted[e0 >> 5] >> (e0 & 31);
      const int valid = P.vocab - v * EPV;
      for (int j = 0; j < rows; ++j) {
        const int row = start + j0 + j;
        if (j && P.draft) {  // the previous row's proposal is part of the output from here on
          const int tok = P.draft[row - 1] - t0 - e0;
#pragma unroll
          for (int e = 0; e < EPV; ++e)
            if (tok == e && e < valid) {
              s[e] += freq + ((co >> e & 1) ? 0.f : pres);
              co |= 1u << e;
              kn |= 1u << e;
            }
        }
        float x[EPV];
        V::unpack(load16(P.x + (int64_t)row * P.ld_bytes + (int64_t)v * 16), x);
        uint32_t allowed = 0xffu;
        if (P.mask) {
          const int mr = P.mask_row ? P.mask_row[row] : row;
          if (mr >= 0 && mr < P.n_masks) {
            const uint8_t* m = P.mask + (int64_t)mr * P.ld_mask_bytes;
            allowed = BF16 ? m[v] : (uint32_t)m[v >> 1] >> (4 * (v & 1));
          }
        }
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const float mul = (kn >> e & 1) ? (x[e] > 0.f ? inv_rho : rho) : 1.f;
          x[e] = (allowed >> e & 1) ? __builtin_fmaf(x[e], mul, -s[e]) : P.masked_value;
        }
        uint8_t* o = P.out + (int64_t)row * P.ld_out_bytes;
        if (valid >= EPV) {
          store16_nt(o + (int64_t)v * 16, V::pack(x));
        } else {
#pragma unroll
          for (int e = 0; e < EPV; ++e)
            if (e < valid) V::put(o, v * EPV + e, x[e]);
        }
      }
    }
  }
  if (blockIdx.x == 0) {  // one tile sees every list whole
    if (P.draft)
      for (int j = tid; j < nb; j += kThreads) bad_token |= (unsigned)P.draft[start + j] >= (unsigned)P.vocab;
    if (bad_token) atomicOr(P.flags, kFlagBadToken);
    if (bad_list) atomicOr(P.flags, kFlagBadList);
  }
}

}  // namespace

hipError_t launch_adjust(const AdjustParams& p, int in_bf16, hipStream_t s) {
  const int tiles = (p.nvec + kTileVec - 1) / kTileVec + (p.mask ? 1 : 0);
  // row groups of a block of average length, one for each layer of the grid
  int64_t z = (p.n_rows + (int64_t)p.n_blocks * kRowGroup - 1) / ((int64_t)p.n_blocks * kRowGroup);
  z = z < 1 ? 1 : z > 4096 ? 4096 : z;
  for (int b0 = 0; b0 < p.n_blocks; b0 += 65535) {  // the grid's second dimension ends there
    AdjustParams q = p;
    q.n_blocks = p.n_blocks - b0 < 65535 ? p.n_blocks - b0 : 65535;
    q.offsets += b0;
    if (q.history) q.history += (int64_t)b0 * p.ld_history;
    if (q.history_len) q.history_len += b0;
    if (q.prompt_len) q.prompt_len += b0;
    if (q.repetition) q.repetition += b0;
    if (q.frequency) q.frequency += b0;
    if (q.presence) q.presence += b0;
    if (q.bias_tokens) q.bias_tokens += (int64_t)b0 * p.ld_bias;
    if (q.bias_values) q.bias_values += (int64_t)b0 * p.ld_bias;
    if (q.bias_len) q.bias_len += b0;
    const dim3 grid((unsigned)tiles, (unsigned)q.n_blocks, (unsigned)z);
    if (in_bf16)
      hipLaunchKernelGGL(k_adjust<true>, grid, dim3(kThreads), 0, s, q);
    else
      hipLaunchKernelGGL(k_adjust<false>, grid, dim3(kThreads), 0, s, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace opd
