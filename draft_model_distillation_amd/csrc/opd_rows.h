// Device helpers shared by the kernels on single rows of logits (opd_adjust.hip, opd_topk.hip,
// opd_topk_loss.hip): 16-byte loads and stores, conversion to and from fp32, and (reference, sum)
// pairs of a log-sum-exp in powers of two.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace opd {

constexpr float kLog2e = 1.44269504088896340736f;  // rounded to fp32; its multiples are exponents of 2
constexpr float kNegInf = -__builtin_inff();
// A reference below every finite logit's exponent and above -inf, so that differences stay defined.
constexpr float kNoRef = -1e30f;

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x4 load16(const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); }
__device__ __forceinline__ u32x4 load16_nt(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}
__device__ __forceinline__ void store16_nt(uint8_t* p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
}

// fp32 -> bf16 bits, to nearest, ties to even; NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}

// 16 bytes of logits as EPV floats and back (bf16 -> fp32 is exact).
template <bool BF16>
struct Vec;
template <>
struct Vec<true> {
  static constexpr int EPV = 8;
  static constexpr int SIZE = 2;
  __device__ __forceinline__ static void unpack(u32x4 v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static u32x4 pack(const float (&x)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_bits(x[2 * i]) | (bf16_bits(x[2 * i + 1]) << 16);
    return v;
  }
  __device__ __forceinline__ static float elem(const uint8_t* row, int i) {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
  }
  __device__ __forceinline__ static void put(uint8_t* row, int i, float f) {
    reinterpret_cast<uint16_t*>(row)[i] = (uint16_t)bf16_bits(f);
  }
};
template <>
struct Vec<false> {
  static constexpr int EPV = 4;
  static constexpr int SIZE = 4;
  __device__ __forceinline__ static void unpack(u32x4 v, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
  }
  __device__ __forceinline__ static u32x4 pack(const float (&x)[4]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(x[i]);
    return v;
  }
  __device__ __forceinline__ static float elem(const uint8_t* row, int i) {
    return reinterpret_cast<const float*>(row)[i];
  }
  __device__ __forceinline__ static void put(uint8_t* row, int i, float f) { reinterpret_cast<float*>(row)[i] = f; }
};

// A running sum of 2^(x log2(e)) kept as sum * 2^ref. ref is at least kNoRef.
__device__ __forceinline__ void lse_join(float& ref, float& sum, float ref2, float sum2) {
  const float r = fmaxf(ref, ref2);
  sum = sum * ex2(ref - r) + sum2 * ex2(ref2 - r);
  ref = r;
}

// Joins the pairs of a wave's 64 lanes (a fixed tree; every lane gets the result).
__device__ __forceinline__ void wave_lse(float& ref, float& sum) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const float r2 = __shfl_xor(ref, m), s2 = __shfl_xor(sum, m);
    lse_join(ref, sum, r2, s2);
  }
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}

}  // namespace opd
