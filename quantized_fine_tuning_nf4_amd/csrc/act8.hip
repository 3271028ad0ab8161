// Activation checkpoints in 8 bits: codes int8 with one power-of-two scale
// for every 64 columns of a row (format in the header).
#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

// One wave per block of 64 columns, one column per lane.
__global__ __launch_bounds__(256) void k_act8_pack(const uint16_t* __restrict__ x, int64_t M,
                                                   int64_t K, int64_t nb, int8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ exps) {
  const int lane = threadIdx.x & 63;
  const int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (b >= M * nb) return;  // whole wave
  const int64_t m = b / nb, c = (b - m * nb) * kAct8Block + lane;
  const bool in = c < K;
  const uint32_t v = in ? x[m * K + c] : 0u;
  uint32_t top = v & 0x7fffu;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  const uint32_t E = act8_exp(top);
  if (in) codes[m * K + c] = E == kAct8NaN ? 0 : (int8_t)act8_code(as_f32(v << 16), act8_inv(E));
  if (lane == 0) exps[b] = (uint8_t)E;
}

__global__ __launch_bounds__(256) void k_act8_unpack(const int8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ exps, int64_t M,
                                                     int64_t K, int64_t nb,
                                                     uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (b >= M * nb) return;
  const int64_t m = b / nb, c = (b - m * nb) * kAct8Block + lane;
  if (c < K) out[m * K + c] = to_bf16((float)codes[m * K + c] * act8_scale(exps[b]));
}

}  // namespace

hipError_t launch_act8_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                            hipStream_t st) {
  const int64_t nb = (K + kAct8Block - 1) / kAct8Block;
  if (M == 0) return hipSuccess;
  hipLaunchKernelGGL(k_act8_pack, dim3((unsigned)((M * nb + 3) / 4)), dim3(256), 0, st, x, M, K, nb,
                     codes, exps);
  return hipGetLastError();
}

hipError_t launch_act8_unpack(const int8_t* codes, const uint8_t* exps, int64_t M, int64_t K,
                              uint16_t* out, hipStream_t st) {
  const int64_t nb = (K + kAct8Block - 1) / kAct8Block;
  if (M == 0) return hipSuccess;
  hipLaunchKernelGGL(k_act8_unpack, dim3((unsigned)((M * nb + 3) / 4)), dim3(256), 0, st, codes,
                     exps, M, K, nb, out);
  return hipGetLastError();
}

}  // namespace qn
