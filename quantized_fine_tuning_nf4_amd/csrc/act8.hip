// Activation checkpoints in 8 bits: codes int8 with one power-of-two scale
// for every 64 columns of a row (format in the header).
//
// Both directions stream: a thread takes chunks of 16 columns, 32 bytes of
// bf16 on one side and 16 codes on the other, four lanes to a block.  With K a
// multiple of 64 (FLAT) blocks run on from row to row and the whole tensor is
// one run of chunks; otherwise a row's last block and its last chunk are
// partial, and rows start on any byte (vector accesses need no alignment on
// this target).
//
// Both are bound by HBM: 177 MB each for 4096 x 14336, 30.3 us packing and 31.0
// unpacking (5.8 and 5.7 TB/s, a large copy's rate).  A wave for every block, a
// column a lane, took 129 us each: 2-byte requests, and six exchanges for a
// maximum.  At 77 x 1000 a kernel takes 5 us, nearly all of it the start of the
// launch and two trips to memory.
#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
constexpr int kThreads = 256;
constexpr int kChunk = 16;           // columns of a chunk
constexpr int kPerBlock = kAct8Block / kChunk;
constexpr int kU = 2;                // chunks of a thread, loaded together

// Where chunk i of the run lies: its first element, its columns in the row
// (<= 0: past the row's end) and its block.
struct Place {
  int64_t at, block;
  int left;
};
template <bool FLAT>
__device__ __forceinline__ Place place(uint32_t i, uint32_t K, uint32_t nb) {
  if constexpr (FLAT) return Place{(int64_t)i * kChunk, (int64_t)(i / kPerBlock), kChunk};
  const uint32_t per_row = nb * kPerBlock, m = i / per_row, c = i - m * per_row;
  return Place{(int64_t)m * K + c * kChunk, (int64_t)m * nb + c / kPerBlock, (int)(K - c * kChunk)};
}

template <bool FLAT>
__global__ __launch_bounds__(kThreads) void k_act8_pack(const uint16_t* __restrict__ x, uint32_t K,
                                                        uint32_t nb, uint32_t chunks,
                                                        int8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ exps) {
  const uint32_t i0 = blockIdx.x * (kThreads * kU) + threadIdx.x;
  u32x4 a[kU], b[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t i = i0 + u * kThreads;
    a[u] = b[u] = u32x4{0u, 0u, 0u, 0u};
    if (i >= chunks) continue;
    const Place p = place<FLAT>(i, K, nb);
    if (p.left >= kChunk) {
      a[u] = *reinterpret_cast<const u32x4_any*>(x + p.at);
      b[u] = *reinterpret_cast<const u32x4_any*>(x + p.at + 8);
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        if (j < p.left) {
          const uint32_t v = (uint32_t)x[p.at + j] << (16 * (j & 1));
          if (j < 8)
            a[u][j >> 1] |= v;
          else
            b[u][(j - 8) >> 1] |= v;
        }
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t i = i0 + u * kThreads;
    uint32_t top = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      top = max(top, max(a[u][q] & 0x7fffu, (a[u][q] >> 16) & 0x7fffu));
      top = max(top, max(b[u][q] & 0x7fffu, (b[u][q] >> 16) & 0x7fffu));
    }
    top = max(top, dpp<kDppXor1>(top));
    top = max(top, dpp<kDppXor2>(top));
    const uint32_t E = act8_exp(top);
    const float inv = act8_inv(E);
    if (i >= chunks) continue;
    const Place p = place<FLAT>(i, K, nb);
    u32x4 c = {0u, 0u, 0u, 0u};
    if (E != kAct8NaN) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = q < 2 ? a[u][2 * q] : b[u][2 * q - 4];
        const uint32_t hi = q < 2 ? a[u][2 * q + 1] : b[u][2 * q - 3];
        c[q] = ((uint32_t)act8_code(bf16_lo(lo), inv) & 0xffu) |
               (((uint32_t)act8_code(bf16_hi(lo), inv) & 0xffu) << 8) |
               (((uint32_t)act8_code(bf16_lo(hi), inv) & 0xffu) << 16) |
               ((uint32_t)act8_code(bf16_hi(hi), inv) << 24);
      }
    }
    if (p.left >= kChunk) {
      *reinterpret_cast<u32x4_any*>(codes + p.at) = c;
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        if (j < p.left) codes[p.at + j] = (int8_t)(c[j >> 2] >> (8 * (j & 3)));
    }
    if (i % kPerBlock == 0) exps[p.block] = (uint8_t)E;
  }
}

template <bool FLAT>
__global__ __launch_bounds__(kThreads) void k_act8_unpack(const int8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ exps,
                                                          uint32_t K, uint32_t nb, uint32_t chunks,
                                                          uint16_t* __restrict__ out) {
  const uint32_t i0 = blockIdx.x * (kThreads * kU) + threadIdx.x;
  u32x4 c[kU];
  uint32_t E[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t i = i0 + u * kThreads;
    c[u] = u32x4{0u, 0u, 0u, 0u};
    E[u] = 0u;
    if (i >= chunks) continue;
    const Place p = place<FLAT>(i, K, nb);
    E[u] = exps[p.block];
    if (p.left >= kChunk) {
      c[u] = *reinterpret_cast<const u32x4_any*>(codes + p.at);
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        if (j < p.left) c[u][j >> 2] |= (uint32_t)(uint8_t)codes[p.at + j] << (8 * (j & 3));
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t i = i0 + u * kThreads;
    if (i >= chunks) continue;
    const Place p = place<FLAT>(i, K, nb);
    const float scale = act8_scale(E[u]);
    uint32_t w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t v = c[u][q >> 1] >> (16 * (q & 1));
      w[q] = pack_bf16x2((float)(int8_t)v * scale, (float)(int8_t)(v >> 8) * scale);
    }
    if (p.left >= kChunk) {
      *reinterpret_cast<u32x4_any*>(out + p.at) = u32x4{w[0], w[1], w[2], w[3]};
      *reinterpret_cast<u32x4_any*>(out + p.at + 8) = u32x4{w[4], w[5], w[6], w[7]};
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        if (j < p.left) out[p.at + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// Calls f(first row, rows, chunks) for slabs of rows whose chunks have 32-bit
// numbers.
template <typename F>
hipError_t by_slabs(int64_t M, int64_t nb, F&& f) {
  const int64_t per_row = nb * kPerBlock, most = (((int64_t)1 << 31) - 1) / per_row;
  for (int64_t m = 0; m < M; m += most) {
    const int64_t rows = M - m < most ? M - m : most;
    const uint32_t chunks = (uint32_t)(rows * per_row);
    f(m, dim3((chunks + kThreads * kU - 1) / (kThreads * kU)), chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_act8_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                            hipStream_t st) {
  const int64_t nb = (K + kAct8Block - 1) / kAct8Block;
  return by_slabs(M, nb, [&](int64_t m, dim3 grid, uint32_t chunks) {
    if (K % kAct8Block == 0)
      hipLaunchKernelGGL(k_act8_pack<true>, grid, dim3(kThreads), 0, st, x + m * K, (uint32_t)K,
                         (uint32_t)nb, chunks, codes + m * K, exps + m * nb);
    else
      hipLaunchKernelGGL(k_act8_pack<false>, grid, dim3(kThreads), 0, st, x + m * K, (uint32_t)K,
                         (uint32_t)nb, chunks, codes + m * K, exps + m * nb);
  });
}

hipError_t launch_act8_unpack(const int8_t* codes, const uint8_t* exps, int64_t M, int64_t K,
                              uint16_t* out, hipStream_t st) {
  const int64_t nb = (K + kAct8Block - 1) / kAct8Block;
  return by_slabs(M, nb, [&](int64_t m, dim3 grid, uint32_t chunks) {
    if (K % kAct8Block == 0)
      hipLaunchKernelGGL(k_act8_unpack<true>, grid, dim3(kThreads), 0, st, codes + m * K,
                         exps + m * nb, (uint32_t)K, (uint32_t)nb, chunks, out + m * K);
    else
      hipLaunchKernelGGL(k_act8_unpack<false>, grid, dim3(kThreads), 0, st, codes + m * K,
                         exps + m * nb, (uint32_t)K, (uint32_t)nb, chunks, out + m * K);
  });
}

}  // namespace qn
