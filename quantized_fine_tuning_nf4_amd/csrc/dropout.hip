// Dropout of an activation without a stored mask (generator and element order in
// qn_device.h).
#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
constexpr int kThreads = 256;
constexpr int kU = 2;  // blocks of eight elements a thread takes, their loads together

// out = kept ? x scale : 0 over n elements, eight a thread and turn.  out may be x.  Ten
// rounds of Philox 4x32, two 32 x 32 -> 64 bit products each, make the bits of eight
// elements; two such blocks a thread keep loads in flight beside them, and HBM is the bound:
// 8192x4096 bf16 22.2 us (134 MB, 6.05 TB/s); 1003x1001 fp32 3.6, latency.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_dropout(const T* x, int64_t n, Drop d, float scale,
                                                      T* out) {
  constexpr int W = sizeof(T) / 2;  // 16-byte words of eight elements
  const int64_t blocks = n >> 3;
  const uint64_t offset = drop_offset(d);
  const uint32_t all = d.on ? 0u : 0x00010001u;  // (a threshold of zero drops nothing)
  const int64_t b0 = (int64_t)blockIdx.x * (kThreads * kU) + threadIdx.x;
  u32x4 v[kU][W];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t b = b0 + u * kThreads;
    if (b < blocks)
#pragma unroll
      for (int w = 0; w < W; ++w)
        v[u][w] = *reinterpret_cast<const u32x4_any*>(x + 8 * b + 8 / W * w);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t b = b0 + u * kThreads;
    if (b > blocks || (b == blocks && (n & 7) == 0)) continue;
    const u32x4 words = philox(d, offset, (uint64_t)b);
    if (b == blocks) {  // the last elements, fewer than eight
      const uint32_t keep = d.on ? keep_byte(words, d.less) : 255u;
      for (int j = 0; j < (int)(n & 7); ++j) {
        const float f = load_f32(x + 8 * b + j);
        store_f32(out + 8 * b + j, (keep >> j) & 1u ? f * scale : 0.f);
      }
      continue;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t k = __builtin_bit_cast(uint32_t, kept(words[q], d.less)) | all;
      const uint32_t lo = 0u - (k & 1u), hi = 0u - (k >> 16);
      if constexpr (W == 1) {
        const uint32_t p = v[u][0][q];
        v[u][0][q] = pack_bf16x2(bf16_lo(p) * scale, bf16_hi(p) * scale) &
                     ((lo & 0xffffu) | (hi & 0xffff0000u));
      } else {
        u32x4& p = v[u][q >> 1];
        p[2 * (q & 1)] = as_u32(as_f32(p[2 * (q & 1)]) * scale) & lo;
        p[2 * (q & 1) + 1] = as_u32(as_f32(p[2 * (q & 1) + 1]) * scale) & hi;
      }
    }
#pragma unroll
    for (int w = 0; w < W; ++w)
      *reinterpret_cast<u32x4_any*>(out + 8 * b + 8 / W * w) = v[u][w];
  }
}

}  // namespace

hipError_t launch_dropout(const void* x, bool f32, int64_t n, const Drop& d, float scale,
                          void* out, hipStream_t st) {
  if (n <= 0) return hipSuccess;
  const int64_t wgs = ((n + 7) / 8 + kThreads * kU - 1) / (kThreads * kU);
  if (f32)
    hipLaunchKernelGGL(k_dropout<float>, dim3((unsigned)wgs), dim3(kThreads), 0, st,
                       static_cast<const float*>(x), n, d, scale, static_cast<float*>(out));
  else
    hipLaunchKernelGGL(k_dropout<uint16_t>, dim3((unsigned)wgs), dim3(kThreads), 0, st,
                       static_cast<const uint16_t*>(x), n, d, scale, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

}  // namespace qn
