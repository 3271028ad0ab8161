// MXFP4: matrices in 4 bits with a power-of-two scale for every 32 columns of a row
// (format in the header), into the format and back, and the linear's product on two
// of them with the adapter term.
#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr int kThreads = 256;

// eight columns of a row from column c as fp32 (zero past the row's end K)
__device__ __forceinline__ void load8(const uint16_t* row, int64_t c, int64_t K, float v[8]) {
  if (c + 8 <= K) {
    const u32x4 w = *reinterpret_cast<const u32x4_any*>(row + c);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf16_lo(w[q]);
      v[2 * q + 1] = bf16_hi(w[q]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = c + q < K ? load_f32(row + c + q) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* row, int64_t c, int64_t K, float v[8]) {
  if (c + 8 <= K) {
    const u32x4 a = *reinterpret_cast<const u32x4_any*>(row + c);
    const u32x4 b = *reinterpret_cast<const u32x4_any*>(row + c + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = as_f32(a[q]);
      v[4 + q] = as_f32(b[q]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = c + q < K ? row[c + q] : 0.f;
  }
}
__device__ __forceinline__ void store8(uint16_t* row, int64_t c, int64_t K, const float v[8]) {
  if (c + 8 <= K) {
    *reinterpret_cast<u32x4_any*>(row + c) =
        u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
              pack_bf16x2(v[6], v[7])};
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < K) row[c + q] = to_bf16(v[q]);
  }
}
__device__ __forceinline__ void store8(float* row, int64_t c, int64_t K, const float v[8]) {
  if (c + 8 <= K) {
    *reinterpret_cast<u32x4_any*>(row + c) = u32x4{as_u32(v[0]), as_u32(v[1]), as_u32(v[2]),
                                                   as_u32(v[3])};
    *reinterpret_cast<u32x4_any*>(row + c + 4) = u32x4{as_u32(v[4]), as_u32(v[5]), as_u32(v[6]),
                                                       as_u32(v[7])};
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < K) row[c + q] = v[q];
  }
}

// eight values of a block with exponent E as codes, the first in the low bits
__device__ __forceinline__ uint32_t encode8(const float v[8], uint32_t E) {
  const float inv = mx4_inv(E);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.f, 3);
  return E == kMx4NaN ? 0u : c;
}
// and back
__device__ __forceinline__ void decode8(uint32_t c, float scale, float v[8]) {
#define QN_PAIR(q)                                                                       \
  {                                                                                      \
    const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, q);                 \
    v[2 * q] = p[0] * scale;                                                             \
    v[2 * q + 1] = p[1] * scale;                                                         \
  }
  QN_PAIR(0) QN_PAIR(1) QN_PAIR(2) QN_PAIR(3)
#undef QN_PAIR
}

// A workgroup takes 32 rows x 256 columns, a step of the scales' layout: pass p,
// thread t -> row 8 p + t / 32, columns 8 (t % 32) .. + 7; four lanes to a block.  The
// 256 scale bytes leave together.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx4_quant(const T* __restrict__ x, int64_t rows,
                                                        int64_t K, int J,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
  __shared__ uint8_t sc[256];
  const int t = threadIdx.x;
  const int64_t R = blockIdx.x / J, j = blockIdx.x - R * J;
  const int64_t c = j * kMx4Step + 8 * (t & 31);
  float v[4][8];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t row = 32 * R + 8 * p + (t >> 5);
    load8(x + min(row, rows - 1) * K, c, K, v[p]);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int n = 8 * p + (t >> 5);
    const int64_t row = 32 * R + n;
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) top = max(top, as_u32(v[p][q]) & 0x7fffffffu);
    top = max(top, dpp<kDppXor1>(top));
    top = max(top, dpp<kDppXor2>(top));
    // (past the matrix: a scale of one, so that a product may read it)
    const bool in = row < rows && c - 8 * (t & 3) < K;
    const uint32_t E = in ? mx4_exp(top) : 127u;
    if ((t & 3) == 0) sc[mx4_scale_at(n, (t & 31) >> 2)] = (uint8_t)E;
    if (row < rows)
      *reinterpret_cast<uint32_t*>(codes + row * 128 * J + 128 * j + 4 * (t & 31)) =
          in ? encode8(v[p], E) : 0u;
  }
  __syncthreads();
  if (t < 64)
    reinterpret_cast<uint32_t*>(scales + (int64_t)blockIdx.x * 256)[t] =
        reinterpret_cast<const uint32_t*>(sc)[t];
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx4_dequant(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          int64_t rows, int64_t K, int J,
                                                          T* __restrict__ out) {
  const int t = threadIdx.x;
  const int64_t R = blockIdx.x / J, j = blockIdx.x - R * J;
  const int64_t c = j * kMx4Step + 8 * (t & 31);
  uint32_t w[4], E[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int n = 8 * p + (t >> 5);
    w[p] = *reinterpret_cast<const uint32_t*>(codes + min(32 * R + n, rows - 1) * 128 * J +
                                              128 * j + 4 * (t & 31));
    E[p] = scales[(int64_t)blockIdx.x * 256 + mx4_scale_at(n, (t & 31) >> 2)];
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t row = 32 * R + 8 * p + (t >> 5);
    if (row >= rows || c >= K) continue;
    float v[8];
    decode8(w[p], mx4_scale(E[p]), v);
    store8(out + row * K, c, K, v);
  }
}

// y[M, N] = x W^T + s u B^T.  A wave takes 32 rows of W (the MFMA's A operand, so
// that a lane ends with four columns of y in a row) and 32 rows of x; lane l holds row
// l % 16 and block 4 t + l / 16 of the step's eight in product t.
__global__ __launch_bounds__(kThreads) void k_mx4_mm(
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs, int64_t M, int64_t N, int J,
    const float* __restrict__ u, const uint16_t* __restrict__ B, int r, float s,
    uint16_t* __restrict__ y, uint32_t cols_wgs) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, n = lane & 15;
  const uint32_t bm = blockIdx.x / cols_wgs, bn = blockIdx.x - bm * cols_wgs;
  const int64_t n0 = 32 * ((int64_t)bn * 4 + wave), m0 = 32 * (int64_t)bm;
  if (n0 >= N) return;
  const uint8_t *wp[2], *xp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    wp[i] = wc + min(n0 + 16 * i + n, N - 1) * 128 * J + 16 * g;
    xp[i] = xc + min(m0 + 16 * i + n, M - 1) * 128 * J + 16 * g;
  }
  const uint32_t* wsp = reinterpret_cast<const uint32_t*>(ws + (n0 / 32) * J * 256) + lane;
  const uint32_t* xsp = reinterpret_cast<const uint32_t*>(xs + (m0 / 32) * J * 256) + lane;
  f32x4 acc[2][2] = {};
  for (int j = 0; j < J; ++j) {
    const int sw = (int)wsp[64 * j], sx = (int)xsp[64 * j];
    i32x8 a[2][2], b[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const u32x4 p = *reinterpret_cast<const u32x4*>(wp[i] + 128 * j + 64 * t);
        const u32x4 q = *reinterpret_cast<const u32x4*>(xp[i] + 128 * j + 64 * t);
        a[i][t] = i32x8{(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
        b[i][t] = i32x8{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
      }
#define QN_MM(i, k, t)                                                                      \
  acc[i][k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(                             \
      a[i][t], b[k][t], acc[i][k], 4, 4, 2 * i + t, sw, 2 * k + t, sx)
    QN_MM(0, 0, 0); QN_MM(0, 1, 0); QN_MM(1, 0, 0); QN_MM(1, 1, 0);
    QN_MM(0, 0, 1); QN_MM(0, 1, 1); QN_MM(1, 0, 1); QN_MM(1, 1, 1);
#undef QN_MM
  }
  // lane: row m0 + 16 k + l % 16 of y, columns n0 + 16 i + 4 (l / 16) + q
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t m = m0 + 16 * k + n;
    if (m >= M) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = n0 + 16 * i + 4 * g + q;
        if (col >= N) continue;
        float low = 0.f;
        for (int e = 0; e < r; ++e) low += u[m * r + e] * load_f32(B + col * r + e);
        y[m * N + col] = to_bf16(acc[i][k][q] + s * low);
      }
  }
}

// out[k][n] = W[n][k] as bf16, row length ldt (zero for rows <= n < ldt).  A
// workgroup takes 32 rows x 256 columns as above, through LDS.
__global__ __launch_bounds__(kThreads) void k_mx4_dequant_t(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
    int64_t K, int J, uint16_t* __restrict__ out, int64_t ldt, BwdAux aux, int aux_wgs) {
  constexpr int PITCH = 32 + 2;  // values of a column of the tile
  __shared__ uint16_t tile[256 * PITCH];
  const int t = threadIdx.x;
  if ((int)blockIdx.x < aux_wgs) {  // one job per thread
    const int64_t i = (int64_t)blockIdx.x * kThreads + t;
    if (i < bwd_aux_count(aux)) bwd_aux_at(aux, i);
    return;
  }
  const int64_t d = (int64_t)blockIdx.x - aux_wgs, R = d / J, j = d - R * J;
  const int64_t rr = (rows + 31) / 32;  // (ldt may go past the scales' last 32 rows)
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int n = 8 * p + (t >> 5);
    const int64_t row = 32 * R + n;
    float v[8] = {};
    if (row < rows) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + row * 128 * J + 128 * j +
                                                            4 * (t & 31));
      decode8(w, mx4_scale(scales[(min(R, rr - 1) * J + j) * 256 +
                                  mx4_scale_at(n, (t & 31) >> 2)]), v);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) tile[(8 * (t & 31) + q) * PITCH + n] = to_bf16(v[q]);
  }
  __syncthreads();
  // thread: column t of the step, 32 values
  const int64_t k = j * kMx4Step + t;
  if (k >= K) return;
  uint16_t* dst = out + k * ldt + 32 * R;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = *reinterpret_cast<const uint32_t*>(tile + t * PITCH + 8 * c + 2 * q);
    *reinterpret_cast<u32x4*>(dst + 8 * c) = u32x4{w[0], w[1], w[2], w[3]};
  }
}

}  // namespace

hipError_t launch_mx4_quant(const void* x, bool f32, int64_t rows, int64_t K, uint8_t* codes,
                            uint8_t* scales, hipStream_t st) {
  const int64_t J = mx4_steps(K);
  const dim3 grid((unsigned)((rows + 31) / 32 * J));
  if (f32)
    hipLaunchKernelGGL(k_mx4_quant<float>, grid, dim3(kThreads), 0, st,
                       static_cast<const float*>(x), rows, K, (int)J, codes, scales);
  else
    hipLaunchKernelGGL(k_mx4_quant<uint16_t>, grid, dim3(kThreads), 0, st,
                       static_cast<const uint16_t*>(x), rows, K, (int)J, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx4_dequant(const Mx4& w, bool f32, void* out, hipStream_t st) {
  const int64_t J = mx4_steps(w.cols);
  const dim3 grid((unsigned)((w.rows + 31) / 32 * J));
  if (f32)
    hipLaunchKernelGGL(k_mx4_dequant<float>, grid, dim3(kThreads), 0, st, w.codes, w.scales,
                       w.rows, w.cols, (int)J, static_cast<float*>(out));
  else
    hipLaunchKernelGGL(k_mx4_dequant<uint16_t>, grid, dim3(kThreads), 0, st, w.codes, w.scales,
                       w.rows, w.cols, (int)J, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

hipError_t launch_mx4_dequant_t(const Mx4& w, uint16_t* out, int64_t ldt, const BwdAux& aux,
                                hipStream_t st) {
  const int64_t J = mx4_steps(w.cols), wgs = (bwd_aux_count(aux) + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(k_mx4_dequant_t, dim3((unsigned)(wgs + ldt / 32 * J)), dim3(kThreads), 0, st,
                     w.codes, w.scales, w.rows, w.cols, (int)J, out, ldt, aux, (int)wgs);
  return hipGetLastError();
}

hipError_t launch_mx4_mm(const Mx4& w, const uint8_t* xc, const uint8_t* xs, int64_t M,
                         const float* u, const uint16_t* B, int r, float s, uint16_t* y,
                         hipStream_t st) {
  const uint32_t cols_wgs = (uint32_t)((w.rows + 127) / 128);
  const dim3 grid(cols_wgs * (uint32_t)((M + 31) / 32));  // (at most 2^31)
  hipLaunchKernelGGL(k_mx4_mm, grid, dim3(kThreads), 0, st, w.codes, w.scales, xc, xs, M, w.rows,
                     (int)mx4_steps(w.cols), u, B, r, s, y, cols_wgs);
  return hipGetLastError();
}

}  // namespace qn
