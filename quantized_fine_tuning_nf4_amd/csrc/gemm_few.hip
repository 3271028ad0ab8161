// bf16 product of few rows with the adapter term:
//
//   C[M, Nc] (bf16) = A[M, R] Bm[Nc, R]^T + s V[M, r] L[Nc, r]^T (.) mask
//
// the same as gemm_bf16.hip's, for batches of up to 128 rows, where that kernel has too
// few tiles to fill the chip (M = 1, Nc = 5112, R = 2688: 40 workgroups walk 42 steps).
// Here a workgroup takes 16 NT rows of Bm, straight into registers, and up to 64 rows of A
// (16 MT), its eight waves the steps of 32 in turn and a block of 16 ranks each; their
// sums meet in LDS.  Bound by Bm from memory for a few rows, else by A from the second
// level cache, which the workgroups of a block of rows all read.  M = 1, Nc = 5112,
// R = 2688 9.0 us (27 MB of Bm), M = 100, 1024 and 1024 7.7; by tiles 23 and 12.4.
#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
constexpr int kWaves = 8;

// ranks j .. j + 7 of a row of L (bf16) and of V (fp32), zero past r
__device__ __forceinline__ u32x4 ranks(const uint16_t* row, int j, int r) {
  if (j + 8 <= r) return *reinterpret_cast<const u32x4_any*>(row + j);
  if (j >= r) return u32x4{0u, 0u, 0u, 0u};
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (j + q < r) w[q >> 1] |= (uint32_t)row[j + q] << (16 * (q & 1));
  return u32x4{w[0], w[1], w[2], w[3]};
}
__device__ __forceinline__ void ranks(const float* row, int j, int r, f32x4 v[2]) {
  if (j + 8 <= r) {
    v[0] = __builtin_bit_cast(f32x4, *reinterpret_cast<const u32x4_any*>(row + j));
    v[1] = __builtin_bit_cast(f32x4, *reinterpret_cast<const u32x4_any*>(row + j + 4));
    return;
  }
  v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (j >= r) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q >> 2][q & 3] = j + q < r ? row[j + q] : 0.f;
}

template <int MT, int NT>
__global__ __launch_bounds__(64 * kWaves) void k_gemm_few(
    const uint16_t* __restrict__ A, int64_t lda, int64_t R, const uint16_t* __restrict__ Bm,
    int64_t ldb, int M, int64_t Nc, const float* __restrict__ V, const uint16_t* __restrict__ L,
    int r, float s, uint16_t* __restrict__ C, const uint8_t* __restrict__ mask, int col_wgs) {
  constexpr int ROWS = 16 * NT, PITCH = ROWS + 4, THREADS = 64 * kWaves;
  constexpr int U = MT * NT >= 4 ? 4 : 8;  // steps whose loads go out together
  __shared__ __attribute__((aligned(16))) float sums[kWaves][16 * MT][PITCH];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mb = (int)blockIdx.x / col_wgs;  // a batch past 64 rows goes in two
  const int64_t c0 = (int64_t)((int)blockIdx.x - mb * col_wgs) * ROWS;
  A += (int64_t)mb * 16 * MT * lda;
  V += (int64_t)mb * 16 * MT * r;
  C += (int64_t)mb * 16 * MT * Nc;
  if (mask) mask += (int64_t)mb * 16 * MT * Nc / 8;
  M = min(M - mb * 16 * MT, 16 * MT);
  const uint16_t *ap[MT], *bp[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) ap[i] = A + (int64_t)min(16 * i + n, M - 1) * lda + 8 * g;
#pragma unroll
  for (int i = 0; i < NT; ++i) bp[i] = Bm + min(c0 + 16 * i + n, Nc - 1) * ldb + 8 * g;
  const int64_t lim = R - 8 * g;  // columns left for this lane's chunk (R % 8 == 0)
  const int steps = (int)((R + 31) / 32);
  // a block of 16 ranks is a wave's: its operands and keep bits go out first
  const int jl = 16 * wave + 8 * (g & 1);
  const bool share = 16 * wave < r;
  u32x4 lb[NT];
  f32x4 va[MT][2];
  uint32_t kb[MT][NT];
  if (share) {
#pragma unroll
    for (int i = 0; i < NT; ++i) lb[i] = ranks(L + min(c0 + 16 * i + n, Nc - 1) * r, jl, r);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = min(16 * m + n, M - 1);
      ranks(V + row * r, jl, r, va[m]);
      if (mask)  // (Nc % 64 == 0: a byte is half a tile's columns)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          kb[m][i] = mask[((row * Nc + min(c0 + 16 * i, Nc - 16)) >> 3) + (g >> 1)] >> (4 * (g & 1));
    }
  }
  f32x4 acc[MT][NT] = {};
  for (int s0 = wave * U; s0 < steps; s0 += U * kWaves) {
    u32x4 a[U][MT], b[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t off = 32 * (int64_t)(s0 + u);
      const bool in = off < lim;  // past the row: its first columns, zero in both operands
#pragma unroll
      for (int i = 0; i < NT; ++i)
        b[u][i] = *reinterpret_cast<const u32x4*>(bp[i] + (in ? off : -8 * g));
#pragma unroll
      for (int i = 0; i < MT; ++i)
        a[u][i] = *reinterpret_cast<const u32x4*>(ap[i] + (in ? off : -8 * g));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = 32 * (int64_t)(s0 + u) < lim;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (!in) b[u][i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (!in) a[u][m] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, b[u][i]), __builtin_bit_cast(bf16x8, a[u][m]), acc[m][i],
              0, 0, 0);
      }
    }
  }
  // the wave's ranks of the adapter term: lane groups 0 and 1 carry the bf16 high part of
  // s V, 2 and 3 its remainder; what is dropped counts as zero
  if (share) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = s * va[m][q >> 1][2 * (q & 1)], z = s * va[m][q >> 1][2 * (q & 1) + 1];
        const uint32_t hi = pack_bf16x2(x, z);
        w[q] = g >= 2 ? pack_bf16x2(x - bf16_lo(hi), z - bf16_hi(hi)) : hi;
      }
      const bf16x8 v = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        f32x4 low = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lb[i]), v,
                                                            f32x4{}, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (!mask || ((kb[m][i] >> q) & 1)) acc[m][i][q] += low[q];
      }
    }
  }
  // lane: row 16 m + n of C, columns 16 i + 4 g + 0 .. 3
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i)
      *reinterpret_cast<f32x4*>(&sums[wave][16 * m + n][16 * i + 4 * g]) = acc[m][i];
  __syncthreads();
  const int c = tid % ROWS;
  if (c0 + c >= Nc) return;
  for (int m = tid / ROWS; m < M; m += THREADS / ROWS) {
    float t = sums[0][m][c];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t += sums[w][m][c];
    C[(int64_t)m * Nc + c0 + c] = to_bf16(t);
  }
}

template <int MT, int NT>
hipError_t launch(const uint16_t* A, int64_t lda, int64_t R, const uint16_t* Bm, int64_t ldb,
                  int64_t M, int64_t Nc, const float* V, const uint16_t* L, int r, float s,
                  uint16_t* C, const uint8_t* mask, hipStream_t st) {
  const int col_wgs = (int)((Nc + 16 * NT - 1) / (16 * NT));
  hipLaunchKernelGGL((k_gemm_few<MT, NT>), dim3((unsigned)(col_wgs * ((M + 16 * MT - 1) / (16 * MT)))),
                     dim3(64 * kWaves), 0, st, A, lda, R, Bm, ldb, (int)M, Nc, V, L, r, s, C, mask,
                     col_wgs);
  return hipGetLastError();
}

}  // namespace

// 32 rows of Bm a workgroup instead of 16 where there are enough of them.  Every
// workgroup's pass over A against the tiles' steps: M = 16, Nc = 4096, R = 14336 (the
// whole backward) 81 us instead of 123, M = 1, 2688 and 5112 50 and 80, but M = 64, 14336
// and 4096 97 and 68, M = 128, 4096 and 4096 70 and 58.
static bool wide_tiles(int64_t Nc) { return Nc >= 16 * 512; }
bool gemm_few_ok(int64_t M, int64_t Nc) {
  return M <= 128 && M * Nc <= ((int64_t)1 << 18) * (wide_tiles(Nc) ? 2 : 1);
}

hipError_t launch_gemm_few(const uint16_t* A, int64_t lda, int64_t R, const uint16_t* Bm,
                           int64_t ldb, int64_t M, int64_t Nc, const float* V, const uint16_t* L,
                           int r, float s, uint16_t* C, hipStream_t st, const uint8_t* mask) {
  if (M <= 0) return hipSuccess;
  if (M > 128 || r > 16 * kWaves || (mask && Nc % 64 != 0) || R < 8 || R % 8 != 0 || R > ldb) return hipErrorInvalidValue;
  const bool wide = wide_tiles(Nc);
#define QN_FEW(MT)                                                                          \
  return wide ? launch<MT, 2>(A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, mask, st)            \
              : launch<MT, 1>(A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, mask, st)
  if (M <= 16) QN_FEW(1);
  if (M <= 32) QN_FEW(2);
  QN_FEW(4);
#undef QN_FEW
}

}  // namespace qn
