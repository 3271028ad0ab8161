// Device helpers shared by the HIP kernels of the QLoRA NF4 library (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qn {

// NF4 levels, codes 0..15, as IEEE binary32 bit patterns.  These are the
// sixteen values of the NF4 table on the page "QLoRA: NF4 storage, gradients
// and local integration" (section "Exact CPU teaching quantizer and adapter
// gradient path"); every one of them is exactly an fp32 number.
constexpr uint32_t kNF4Bits[16] = {
    0xbf800000u, 0xbf3239b1u, 0xbf066b30u, 0xbeca32a0u, 0xbe91a24du, 0xbe3d353fu,
    0xbdba7871u, 0x00000000u, 0x3da2faffu, 0x3e24cae3u,
    0x3e7c04ddu, 0x3ead033au, 0x3ee1a4b8u, 0x3f1007abu, 0x3f3913b3u, 0x3f800000u};

// FP4 code values, codes 0..15 (code c: sign bit 3, magnitude index c & 7),
// as binary32 bit patterns: the E2M1 levels {0, 0.0625, 2, 3, 4, 6, 8, 12}
// / 12 (course notebook FT-02, "Exercise 3: NF4 vs FP4 at equal memory",
// prints them to four decimals: 0, 0.0052, 0.1667, 0.25, 0.3333, 0.5,
// 0.6667, 1), each rounded to fp32.
constexpr uint32_t kFP4Bits[16] = {
    0x00000000u, 0x3baaaaabu, 0x3e2aaaabu, 0x3e800000u, 0x3eaaaaabu, 0x3f000000u,
    0x3f2aaaabu, 0x3f800000u, 0x80000000u, 0xbbaaaaabu, 0xbe2aaaabu, 0xbe800000u,
    0xbeaaaaabu, 0xbf000000u, 0xbf2aaaabu, 0xbf800000u};

// Codebooks of the 4-bit codes.
constexpr int kCodeNF4 = 0, kCodeFP4 = 1;

// Level k of codebook cb, as a bit pattern (cb and k known at compile time
// give an immediate).
__host__ __device__ constexpr uint32_t level_bits(int cb, int k) {
  return cb == kCodeFP4 ? kFP4Bits[k] : kNF4Bits[k];
}

constexpr int kBlock = 64;        // first-level block (weights per absmax scale)
constexpr int kGroup = 256;       // second-level block (scales per fp32 scale2)
constexpr float kE4M3Max = 448.f; // largest finite OCP FP8 E4M3FN value

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float as_f32(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t as_u32(float f) { return __float_as_uint(f); }

// Two fp32 -> packed bf16x2 (low half = a), round to nearest even
// (v_cvt_pk_bf16_f32 on gfx950).
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  f32x2 v = {a, b};
  bf16x2 h = __builtin_convertvector(v, bf16x2);
  return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ float bf16_lo(uint32_t p) { return as_f32(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return as_f32(p & 0xffff0000u); }

// sum over s < S of part[s * count + i], added in slice order (loads issued
// eight at a time)
__device__ __forceinline__ float slice_sum(const float* __restrict__ part, int64_t count, int S,
                                           int64_t i) {
  float acc = part[i];
  for (int s0 = 1; s0 < S; s0 += 8) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = s0 + k < S ? part[(int64_t)(s0 + k) * count + i] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k < S) acc += v[k];
  }
  return acc;
}

// OCP FP8 E4M3FN byte -> fp32 (exact).  Exponent bias 7, three mantissa
// bits, subnormals m * 2^-9; the NaN pattern is never produced here.
__device__ __forceinline__ float e4m3_to_f32(uint32_t q) {
  uint32_t e = (q >> 3) & 15u, m = q & 7u;
  float v = e ? as_f32(((e + 120u) << 23) | (m << 20)) : (float)m * 0x1p-9f;
  return as_f32(as_u32(v) | ((q & 0x80u) << 24));
}

// fp32 -> OCP FP8 E4M3FN byte, round to nearest even; magnitudes past the
// largest finite value saturate to 448.  Input must be finite.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint32_t sign = (as_u32(x) >> 24) & 0x80u;
  float a = __builtin_fabsf(x);
  uint32_t mag;
  if (a < 0x1p-6f) {
    // subnormal range: quantum 2^-9, result 0..8 (8 = smallest normal)
    mag = (uint32_t)__builtin_rintf(a * 512.f);
  } else {
    uint32_t b = as_u32(a);
    // keep 3 mantissa bits, round half to even on the 20 dropped bits
    uint32_t r = b + 0x7ffffu + ((b >> 20) & 1u);
    mag = (r >> 20) - (120u << 3);
  }
  if (mag > 126u) mag = 126u;
  return sign | mag;
}

// Dequant scale s'_b = fmaf(e4m3(q_b), s2_g, mu): one rounding.
__device__ __forceinline__ float dq_scale(uint32_t q, float s2, float mu) {
  return __builtin_fmaf(e4m3_to_f32(q), s2, mu);
}

// Where a state's block scales come from: the double-quantized codes
// (absmax == null) or fp32 block scales as they are (double quantization
// off).
struct ScaleSrc {
  const uint8_t* qscale;
  const float* scale2;
  const float* offset;
  const float* absmax;
};

// 8-bit activation checkpoints: 64 columns of a row share the scale
// 2^(E-127); E from the block's largest magnitude (its bf16 bits without the
// sign).  127 = 1.984375 x 2^6 is bf16, so only the significand 255/128 above
// it needs the next power of two; the largest finite magnitude, 255 x 2^120,
// has none that bf16 can hold (64 x 2^122 is infinite) and saturates at
// 127 x 2^121.
constexpr int kAct8Block = 64;
constexpr uint32_t kAct8NaN = 255;  // E of a block with a NaN or an infinity
__device__ __forceinline__ uint32_t act8_exp(uint32_t absmax_bits) {
  if (absmax_bits >= 0x7f80u) return kAct8NaN;
  const int e = (int)(absmax_bits >> 7) - 6 + ((absmax_bits & 0x7fu) == 0x7fu ? 1 : 0);
  return (uint32_t)min(max(e, 1), 248);
}
// what a value is multiplied by to become its code, and back
__device__ __forceinline__ float act8_inv(uint32_t E) {
  return E == kAct8NaN ? 0.f : as_f32((254u - E) << 23);
}
__device__ __forceinline__ float act8_scale(uint32_t E) {
  return as_f32(E == kAct8NaN ? 0x7fc00000u : E << 23);
}
// code of a value (a block's NaN or infinity: whatever, the block reads NaN)
__device__ __forceinline__ int act8_code(float x, float inv) {
  return (int)fminf(fmaxf(__builtin_rintf(x * inv), -127.f), 127.f);
}

// bf16 or fp32 elements as fp32, and back (round to nearest even)
__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const uint16_t* p) { return as_f32((uint32_t)*p << 16); }
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return (uint16_t)(pack_bf16x2(x, 0.f) & 0xffffu);
}
__device__ __forceinline__ void store_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_f32(uint16_t* p, float x) { *p = to_bf16(x); }

// A lane's value from the lane that DPP control CTRL names (every lane has
// one for the controls used here).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xb1, kDppXor2 = 0x4e;              // quad_perm
constexpr int kDppMirror8 = 0x141, kDppMirror16 = 0x140;     // row_half_mirror, row_mirror

// Reductions over a wave, the result in every lane: within rows of 16 by DPP,
// across them by the two permlane swaps.  f joins two values.
template <typename F>
__device__ __forceinline__ uint32_t reduce_8_lanes(uint32_t x, F f) {
  x = f(x, dpp<kDppXor1>(x));
  x = f(x, dpp<kDppXor2>(x));
  return f(x, dpp<kDppMirror8>(x));
}
template <typename F>
__device__ __forceinline__ uint32_t reduce_wave(uint32_t x, F f) {
  x = reduce_8_lanes(x, f);
  x = f(x, dpp<kDppMirror16>(x));
  auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = f(a[0], a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return f(b[0], b[1]);
}
__device__ __forceinline__ float wave_sum(float x) {
  return as_f32(reduce_wave(as_u32(x), [](uint32_t a, uint32_t b) {
    return as_u32(as_f32(a) + as_f32(b));
  }));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
  return reduce_wave(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t max_of_8_lanes(uint32_t x) {
  return reduce_8_lanes(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}

}  // namespace qn
