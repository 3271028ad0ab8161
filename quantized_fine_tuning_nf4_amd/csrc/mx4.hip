// MXFP4: matrices in 4 bits with a power-of-two scale for every 32 columns of a row
// (format in the header), into the format and back, and the linear's product on two
// of them with the adapter term.
#include <algorithm>
#include <type_traits>

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
    const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row + c));
    const u32x4 b = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row + c + 4));
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

// f(0), f(1), .. f(N - 1), each with its index as a constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}

// ---- Into the format: E = floor(log2 max |x|) - 2 + 127 per block of 32 columns, codes
// the nearest levels of x 2^(127 - E) (hardware conversion, ties to the even code, 6 at
// most).  A workgroup takes 32 rows x 256 columns, a step of the scales' layout: pass p,
// thread t -> row 8 p + t / 32, columns 8 (t % 32) .. + 7; four lanes to a block.  The
// 256 scale bytes leave together.  Bound by HBM: 4096x14336 fp32 49.4 us (271 MB, 5.5
// TB/s), 8192x4096 bf16 18.4 (85 MB, 4.6 TB/s); small matrices by one pass's latency (77x1000
// 3.8 us).  fp32 matrices (weights, read once) come by streaming loads, with ordinary ones
// 62.6 us; bf16 ones, activations that the kernel before may have left in the caches, by
// ordinary loads, and streaming ones take as long (18.4).
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

// ---- And back, one rounding to T at most (fp32: none), the same tile.  Bound by HBM's
// writes: 4096x14336 fp32 44.0 us (266 MB, 6.05 TB/s), 77x1000 bf16 2.9.
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

// ---- The linear's input: x [M, K] bf16 read once, into MXFP4 and, with the adapter, u =
// drop(x) A^T.  A workgroup takes 16 RT rows and one of S slices of the steps (256
// columns each), its waves a step in turn.  Lane (g, n) = (l / 16, l % 16) holds columns
// 8 g .. 8 g + 7 of row n in each block of 32: an operand of the bf16 product for u as it
// is, and a quarter of the block, whose largest magnitude meets over the four lanes of
// the row by two exchanges (two blocks a word).  Four blocks' codes are turned around
// between those lanes, so that each stores one block's 16 bytes.  With one slice the
// waves' sums of u meet in LDS, and the workgroup writes u and (s u) as the
// product's epilogue takes it; else the slices' sums are written, for the product's
// workgroups to add (few rows) or for k_mx4_u.  With DROP each lane draws its eight elements' keep bits
// (one counter) and masks the operand of u alone.  u's products are in the same pass, since x
// is the larger part of the bytes: 8192x4096 at r = 16 20.3 us (85 MB, 4.2 TB/s), with
// dropout 24.0-25.0: the Philox rounds (20 wide multiplies for eight elements) fill the
// vector units beside the loads; at r = 64 37 us, A's four tiles of ranks from the L2 in
// every workgroup.  Few rows: eight slices, 16x14336 7.4 us, 1x4096 4.6, latency.
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}
// the eight codes of a lane's part of a block (the words by themselves: a bit cast of a
// vector's element is one of its first)
__device__ __forceinline__ uint32_t encode8(u32x4 v, uint32_t E) {
  const float scale = mx4_scale(E);
  const uint32_t v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v0), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v1), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v2), scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v3), scale, 3);
  return E == kMx4NaN ? 0u : c;
}
// B [N, r] as the product's epilogue takes it: 16 rows and 16 ranks are 512 bytes, 16 of
// them rows n's ranks 8 h .. 8 h + 7 at 16 h + n (zero past N and r); piece i of them
__device__ __forceinline__ void order_b(const uint16_t* B, int64_t N, int r, int nj, int64_t i,
                                        uint16_t* out) {
  const int n = (int)(i & 15), h = (int)(i >> 4) & 1;
  const int64_t t = i >> 5, row = t / nj * 16 + n;
  const int j = (int)(t % nj) * 16 + 8 * h;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (row < N) {
    if (r % 8 == 0) {
      if (j < r) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(B + row * r + j);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = v[q];
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (j + q < r) w[q >> 1] |= (uint32_t)B[row * r + j + q] << (16 * (q & 1));
    }
  }
  reinterpret_cast<u32x4*>(out)[i] = u32x4{w[0], w[1], w[2], w[3]};
}

template <int RT, int NJ, bool DROP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx4_x(
    const uint16_t* __restrict__ x, int64_t M, int64_t K, int J, int S, Drop d,
    const uint16_t* __restrict__ A, const uint16_t* __restrict__ B, int64_t N, int r, float s,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, float* __restrict__ u,
    float* __restrict__ upart, uint16_t* __restrict__ su, uint16_t* __restrict__ bo, int b_wgs) {
  constexpr int PITCH = 16 * RT + 4;
  __shared__ __attribute__((aligned(16))) float sums[WAVES][16 * NJ][PITCH];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if ((int)blockIdx.x < b_wgs) {
    const int64_t i = (int64_t)blockIdx.x * (64 * WAVES) + tid;
    if (i < (N + 15) / 16 * NJ * 32) order_b(B, N, r, NJ, i, bo);
    return;
  }
  const int64_t bid = (int64_t)blockIdx.x - b_wgs, rt = bid / S;
  const int z = (int)(bid - rt * S);
  const int j0 = (int)((int64_t)J * z / S), j1 = (int)((int64_t)J * (z + 1) / S);
  const int64_t m0 = 16 * RT * rt;
  const uint64_t offset = DROP ? drop_offset(d) : 0;
  const uint16_t* xp[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) xp[i] = x + min(m0 + 16 * i + n, M - 1) * K + 8 * g;
  const uint16_t* ap[NJ];
#pragma unroll
  for (int q = 0; q < NJ; ++q) ap[q] = A + (int64_t)min(16 * q + n, r - 1) * K + 8 * g;
  f32x4 acc[RT][NJ] = {};
  for (int j = j0 + wave; j < j1; j += WAVES) {
    const int64_t k0 = (int64_t)j * kMx4Step;
    const int blocks = (int)min((K - k0) / kMx4Block, (int64_t)8);  // (K is a multiple of 64)
    u32x4 v[RT][8];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int b = 0; b < 8; ++b)  // past the row: its first columns, zeroed below
        v[i][b] = *reinterpret_cast<const u32x4*>(xp[i] + (b < blocks ? k0 + 32 * b : 0));
    constexpr int CB = NJ == 1 ? 8 : NJ == 2 ? 4 : 2;  // blocks whose rows of A come together
    unrolled<8 / CB>([&](auto c_t) {
      constexpr int c = decltype(c_t)::value * CB;
      u32x4 a[CB][NJ];
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int q = 0; q < NJ; ++q)
          a[b][q] = *reinterpret_cast<const u32x4*>(ap[q] + (c + b < blocks ? k0 + 32 * (c + b) : 0));
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const bool in = c + b < blocks;
#pragma unroll
        for (int q = 0; q < NJ; ++q)
          if (!in || 16 * q + n >= r) a[b][q] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if (!in) v[i][c + b] = u32x4{0u, 0u, 0u, 0u};
          u32x4 w = v[i][c + b];
          if constexpr (DROP) {
            const int64_t m = min(m0 + 16 * i + n, M - 1);
            w = drop8(w, philox(d, offset, (uint64_t)(m * K + k0 + 32 * (c + b) + 8 * g) >> 3),
                      d.less);
          }
#pragma unroll
          for (int q = 0; q < NJ; ++q)
            acc[i][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a[b][q]), acc[i][q], 0, 0,
                0);
        }
      }
    });
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t m = m0 + 16 * i + n;
      uint32_t e0 = 0, e1 = 0;  // exponents of blocks g and g + 4
      u32x4 out[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t c[4];
#pragma unroll
        for (int p = 0; p < 2; ++p) {  // two blocks at a time
          const u32x4 a = v[i][4 * h + 2 * p], b = v[i][4 * h + 2 * p + 1];
          const uint32_t mask = 0x7fff7fffu;
          const uint32_t ma = pk_max(pk_max(a[0] & mask, a[1] & mask),
                                     pk_max(a[2] & mask, a[3] & mask));
          const uint32_t mb = pk_max(pk_max(b[0] & mask, b[1] & mask),
                                     pk_max(b[2] & mask, b[3] & mask));
          uint32_t top = pk_max(__builtin_amdgcn_perm(mb, ma, 0x05040100u),
                                __builtin_amdgcn_perm(mb, ma, 0x07060302u));
          const auto s16 = __builtin_amdgcn_permlane16_swap(top, top, false, false);
          top = pk_max(s16[0], s16[1]);
          const auto s32 = __builtin_amdgcn_permlane32_swap(top, top, false, false);
          top = pk_max(s32[0], s32[1]);
          const uint32_t Ea = mx4_exp(top << 16), Eb = mx4_exp(top & 0xffff0000u);
          c[2 * p] = encode8(a, Ea);
          c[2 * p + 1] = encode8(b, Eb);
          uint32_t& e = h ? e1 : e0;
          e = g == 2 * p ? Ea : g == 2 * p + 1 ? Eb : e;
        }
        // c[b] of lane g -> word g of block b at lane b
        auto t0 = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
        auto t1 = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
        auto w0 = __builtin_amdgcn_permlane16_swap(t0[0], t1[0], false, false);
        auto w1 = __builtin_amdgcn_permlane16_swap(t0[1], t1[1], false, false);
        out[h] = u32x4{w0[0], w0[1], w1[0], w1[1]};
      }
      if (m < M) {
        uint8_t* dst = codes + m * 128 * J + 128 * j + 16 * g;
        *reinterpret_cast<u32x4*>(dst) = out[0];
        *reinterpret_cast<u32x4*>(dst + 64) = out[1];
        *reinterpret_cast<uint16_t*>(scales + ((m >> 5) * J + j) * 256 + 4 * lane +
                                     2 * ((m >> 4) & 1)) = (uint16_t)(e0 | (e1 << 8));
      }
    }
  }
  // lane: rank 16 q + n, rows 16 i + 4 g + 0 .. 3
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int q = 0; q < NJ; ++q)
      *reinterpret_cast<f32x4*>(&sums[wave][16 * q + n][16 * i + 4 * g]) = acc[i][q];
  __syncthreads();
  float* dst = S > 1 ? upart + (int64_t)z * M * r : u;
  for (int e = tid; e < 16 * RT * 16 * NJ; e += 64 * WAVES) {
    const int row = e / (16 * NJ), j = e % (16 * NJ);
    float t = sums[0][j][row];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) t += sums[w][j][row];
    sums[0][j][row] = t;  // (read and written by this thread alone)
    if (j < r && m0 + row < M) dst[(m0 + row) * r + j] = t;
  }
  if (!su) return;
  __syncthreads();
  // (s u): 16 rows and 16 ranks are 1 KB in the order of the product's lanes
  for (int e = tid; e < 64 * RT * NJ; e += 64 * WAVES) {
    const int l = e & 63, q = (e >> 6) % NJ, i = (e >> 6) / NJ;
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int j = 16 * q + 8 * ((l >> 4) & 1) + 2 * p, row = 16 * i + (l & 15);
      const float a = j < r ? s * sums[0][j][row] : 0.f;
      const float b = j + 1 < r ? s * sums[0][j + 1][row] : 0.f;
      const uint32_t hi = pack_bf16x2(a, b);
      w[p] = l >= 32 ? pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi)) : hi;
    }
    reinterpret_cast<u32x4*>(su)[((rt * RT + i) * NJ + q) * 64 + l] = u32x4{w[0], w[1], w[2], w[3]};
  }
}

// u = the sum of its S slices in slice order, and (s u) as above: a thread takes eight
// ranks of a row (zero past M and r).
constexpr int kThreadsU = 64;  // (few threads in all: over many compute units)
__global__ __launch_bounds__(kThreadsU) void k_mx4_u(const float* __restrict__ upart, int S,
                                                     int64_t M, int r, int nj, float s,
                                                     float* __restrict__ u,
                                                     uint16_t* __restrict__ su, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreadsU + threadIdx.x;
  if (i >= n) return;
  const int l = (int)(i & 31);
  const int64_t t = i >> 5, row = t / nj * 16 + (l & 15);
  const int j = (int)(t % nj) * 16 + 8 * (l >> 4), left = row < M ? min(r - j, 8) : 0;
  float v[8] = {};
  const float* p = upart + row * r + j;
  if (left == 8) {
#pragma unroll 4
    for (int z = 0; z < S; ++z) {
      const u32x4 a = *reinterpret_cast<const u32x4_any*>(p + z * M * r);
      const u32x4 b = *reinterpret_cast<const u32x4_any*>(p + z * M * r + 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] += as_f32(a[q]);
        v[4 + q] += as_f32(b[q]);
      }
    }
  } else {
    for (int z = 0; z < S; ++z)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < left) v[q] += p[z * M * r + q];
  }
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < left) u[row * r + j + q] = v[q];
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float a = s * v[2 * q], b = s * v[2 * q + 1];
    hi[q] = pack_bf16x2(a, b);
    lo[q] = pack_bf16x2(a - bf16_lo(hi[q]), b - bf16_hi(hi[q]));
  }
  reinterpret_cast<u32x4*>(su)[t * 64 + l] = u32x4{hi[0], hi[1], hi[2], hi[3]};
  reinterpret_cast<u32x4*>(su)[t * 64 + 32 + l] = u32x4{lo[0], lo[1], lo[2], lo[3]};
}

// ---- The product of many rows.  Workgroup tile BM x BN (rows of x, rows of W), WVM x WVN
// waves of TM x TN tiles of v_mfma_scale_f32_16x16x128_f8f6f4.  A step is 256 columns:
// rows of 128 bytes of codes and 256 scale bytes per 32 rows go from global memory
// straight into LDS, NST stages deep.  Chunk c (16 bytes, a block) of row y sits at unit
// c ^ ((y >> 1) & 7), so that 16 rows of a fragment read sit on distinct banks.  In
// half t of a step lane (g, n) = (l / 16, l % 16) takes row n's block 4 t + g, whose scale
// is byte 2 (tile % 2) + t of the lane's four.
// 8192x4096x4096 at r = 16 69.0 us, 3.98 PFLOP/s (256 x 256 tiles, 109 MB read, 67 written).
// Three things hold it: the clock (4096x4096x16384, 4.87 PFLOP/s, takes 113 us at 1.88 GHz on
// random operands and 87 at 2.43 GHz on zeros, by the same instructions: power), issue (on
// either operands MFMAs are 62% of the cycles; the instruction alone reaches 5.7 PFLOP/s
// with one wave a SIMD and 7.3 with two, on random operands) and what a round of tiles costs
// outside its steps, some 6 us (at the rate of 16384 columns the two rounds take 56 us).
// 32x32x64 tiles take 75 us; four stages for many tiles, loads or barriers elsewhere in the
// step and wave priorities change nothing or lose.  301x50021x1000 22.5 us:
// 2.3 rounds of tiles take three, of four steps each, whose first stage and output nothing
// overlaps (the call 26.8 us, with 256 rows of x, two rounds, 22.6), and rows of an odd
// length (with 50016 columns 22.6, 50024 25.1, though no more bytes are written); 64 x 128
// tiles 24.6 and 64 x 64 27.2 (two stages deep), eight waves 23.1.
template <int WVM, int WVN, int TM, int TN, int STAGES>
struct MxGeo {
  static constexpr int NST = STAGES;
  static constexpr int WAVES = WVM * WVN, THREADS = 64 * WAVES;
  static constexpr int BM = 16 * TM * WVM, BN = 16 * TN * WVN;
  static constexpr int XB = BM * 128, WB = BN * 128;   // codes of a stage
  static constexpr int XS = XB + WB, WS = XS + BM * 8;  // its scales
  static constexpr int SL = (BM + BN + 127) / 128;     // loads of scales, 1 KB each
  static constexpr int STB = XS + 1024 * SL;           // bytes of a stage
  // output staging of a wave: half its rows at a time
  static constexpr int OUTP = 32 * TN + 16, OUTW = 8 * TM * OUTP;
  static constexpr int LDS_MAIN = NST * STB > WAVES * OUTW ? NST * STB : WAVES * OUTW;
  static constexpr int LDS_V = LDS_MAIN, LDS_L = LDS_V + BM * 64;  // r <= 16: s u and B
  static constexpr int LDS_BYTES = LDS_L + BN * 32;
  static constexpr int XL = BM / 8 / WAVES, WL = BN / 8 / WAVES;   // loads of codes of a wave
  static_assert(LDS_BYTES <= 160 * 1024 && WAVES % SL == 0, "LDS");
};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rs(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(lo | (hi << 32)), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
__device__ __forceinline__ void dma16(rsrc_t rs, uint32_t voff, uint32_t soff, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void barrier_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ i32x8 frag4(u32x4 v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

template <int WVM, int WVN, int TM, int TN, int NST, bool ONE>
__global__ __launch_bounds__(64 * WVM * WVN, 2) void k_mx4_gemm(
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs, int64_t M, int64_t N, int J,
    const uint16_t* __restrict__ su, const uint16_t* __restrict__ bo, int nj,
    uint16_t* __restrict__ y, int tiles_m, int tiles_n) {
  using G = MxGeo<WVM, WVN, TM, TN, NST>;
  constexpr int BM = G::BM, BN = G::BN, STB = G::STB, XL = G::XL, WL = G::WL, LPS = XL + WL;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WVN, wn = wave % WVN;

  // tile order: each XCD (they take workgroups round robin) a contiguous run of the
  // tiles, which go down up to four tile rows at a time and then across the columns, so
  // that the workgroups that share an L2 share rows of both operands
  const int ntiles = tiles_m * tiles_n, xcd = blockIdx.x & 7;
  const int bid = xcd * (ntiles >> 3) + min(xcd, ntiles & 7) + (blockIdx.x >> 3);
  const int grp = bid / (4 * tiles_n), in = bid - grp * 4 * tiles_n;
  const int deep = min(4, tiles_m - 4 * grp);
  int tm = 4 * grp + in % deep, tn = in / deep;
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int mrows = (int)min((int64_t)BM, M - m0), nrows = (int)min((int64_t)BN, N - n0);
  const int pitch = 128 * J;

  // loads: instruction i of wave w covers rows 8 (XL w + i) + l / 8 (rows past the matrix
  // repeat its last one: nothing of them is stored)
  const rsrc_t rx = make_rs(xc + m0 * pitch, (uint32_t)(mrows * pitch));
  const rsrc_t rw = make_rs(wc + n0 * pitch, (uint32_t)(nrows * pitch));
  uint32_t xoff[XL], woff[WL];
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int row = 8 * (XL * wave + i) + (lane >> 3);
    xoff[i] = (uint32_t)(min(row, mrows - 1) * pitch + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
  }
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int row = 8 * (WL * wave + i) + (lane >> 3);
    woff[i] = (uint32_t)(min(row, nrows - 1) * pitch + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
  }
  // scales: 1 KB (four groups of 32 rows) a wave, those of x first; there are more waves
  // than that, and the upper ones load the same again
  constexpr bool MIXED = BM % 128 != 0;  // (groups of x and of W in one load)
  const int sq = wave % G::SL, xg = (mrows + 31) >> 5, wg = (nrows + 31) >> 5;
  const int sg = 4 * sq + (lane >> 4);  // group of the tile
  const bool sx = MIXED ? sg < BM / 32 : sq < BM / 128;
  const int sk = sx ? min(sg, xg - 1) : min(sg - BM / 32, wg - 1);
  const uint8_t* sbase = sx ? xs + m0 / 32 * J * 256 : ws + n0 / 32 * J * 256;
  const rsrc_t rs = make_rs(sbase, MIXED ? 0u : (uint32_t)((sx ? xg : wg) * J * 256));
  const uint32_t soff = (uint32_t)(sk * J * 256 + 16 * (lane & 15));
  // load q (0 .. LPS) of step st
  auto load_one = [&](int q, int st, int stage) {
    uint8_t* base = smem + stage * STB;
    const uint32_t so = (uint32_t)st * 128;
    if (q < XL)
      dma16(rx, xoff[q], so, base + 1024 * (XL * wave + q));
    else if (q < LPS)
      dma16(rw, woff[q - XL], so, base + G::XB + 1024 * (WL * wave + q - XL));
    else if constexpr (MIXED)
      __builtin_amdgcn_global_load_lds((global_void*)(sbase + soff + 2 * so),
                                       (lds_void*)(base + G::XS + 1024 * sq), 16, 0, 0);
    else
      dma16(rs, soff, 2 * so, base + G::XS + 1024 * sq);
  };

  // fragment reads
  const int n = lane & 15, g = lane >> 4;
  int roff[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) roff[t] = n * 128 + 16 * ((4 * t + g) ^ ((n >> 1) & 7));
  const int xbase = wm * 16 * TM * 128, wbase = G::XB + wn * 16 * TN * 128;
  const int xsb = G::XS + wm * TM * 128 + 4 * lane, wsb = G::WS + wn * TN * 128 + 4 * lane;
  auto frag = [&](int stage, int base, int k, int t) {
    return *reinterpret_cast<const u32x4*>(smem + stage * STB + base + k * 2048 + roff[t]);
  };
  auto scale = [&](int stage, int base, int k) {  // of tiles 2 k and 2 k + 1
    return *reinterpret_cast<const int*>(smem + stage * STB + base + k * 256);
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{};
  u32x4 fx[TM], fw[2][TN];
  int ex[2][TM / 2], ew[2][TN / 2];

  // the adapter's operands: one block of 16 ranks goes to LDS ahead of everything (tiles
  // past the matrix read zeros)
  const int mt = (mrows + 15) >> 4, nt = (nrows + 15) >> 4;
  if constexpr (ONE) {
    const rsrc_t ru = make_rs(su + m0 * 32, (uint32_t)(mt * 1024));
    const rsrc_t rb = make_rs(bo + n0 * 16, (uint32_t)(nt * 512));
#pragma unroll
    for (int k = 0; k < BM / 16 / G::WAVES; ++k) {
      const int q = BM / 16 / G::WAVES * wave + k;
      dma16(ru, (uint32_t)(1024 * q + 16 * lane), 0, smem + G::LDS_V + 1024 * q);
    }
#pragma unroll
    for (int k = 0; k < (BN / 32 + G::WAVES - 1) / G::WAVES; ++k) {
      const int q = (k * G::WAVES + wave) % (BN / 32);  // (again where waves are more)
      dma16(rb, (uint32_t)(1024 * q + 16 * lane), 0, smem + G::LDS_L + 1024 * q);
    }
  }
#pragma unroll
  for (int k = 0; k < NST; ++k)
#pragma unroll
    for (int q = 0; q <= LPS; ++q) load_one(q, min(k, J - 1), k);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 1) * (LPS + 1)) : "memory");
  barrier_lds();
#pragma unroll
  for (int i = 0; i < TM; ++i) fx[i] = frag(0, xbase, i, 0);
#pragma unroll
  for (int j = 0; j < TN; ++j) fw[0][j] = frag(0, wbase, j, 0);
#pragma unroll
  for (int i = 0; i < TM / 2; ++i) ex[0][i] = scale(0, xsb, i);
#pragma unroll
  for (int j = 0; j < TN / 2; ++j) ew[0][j] = scale(0, wsb, j);

  // half t of step st on stage P = st % NST.  The fragments of the next half are read while
  // this one's products run (those of W in a second set, those of x in place after their
  // row).  At the end of half 0 every wave has read the stage and step st + 1 has
  // landed; half 1 sends the loads of step st + NST into the stage.
  auto half = [&](auto p_t, auto t_t, int st) {
    constexpr int P = decltype(p_t)::value, H = decltype(t_t)::value;
    constexpr int RS = H == 0 ? P : (P + 1) % NST, RH = H ^ 1, E = P & 1;
    const int lst = min(st + NST, J - 1);
    unrolled<TM>([&](auto i_t) {
      constexpr int i = decltype(i_t)::value;
      unrolled<TN>([&](auto j_t) {
        constexpr int j = decltype(j_t)::value;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            frag4(fw[H][j]), frag4(fx[i]), acc[i][j], 4, 4, 2 * (j & 1) + H, ew[E][j / 2],
            2 * (i & 1) + H, ex[E][i / 2]);
        if (i == 0) fw[RH][j] = frag(RS, wbase, j, RH);
        if (H == 1 && i == 1 && j < TN / 2) ew[E ^ 1][j] = scale(RS, wsb, j);
        constexpr int K0 = TM == 2 ? 1 : 2;  // row of the first of x's scales
        if (H == 1 && i >= K0 && j == 0 && i - K0 < TM / 2)
          ex[E ^ 1][i - K0] = scale(RS, xsb, i - K0);
        if (H == 1 && j == TN / 2)
          for (int q = (LPS + TM) / TM * i; q < (LPS + TM) / TM * (i + 1); ++q)
            if (q <= LPS) load_one(q, lst, P);
      });
      fx[i] = frag(RS, xbase, i, RH);
      __builtin_amdgcn_sched_barrier(0);
    });
    if (H == 0) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * (LPS + 1)) : "memory");
      barrier_lds();
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  int st = 0;
  for (; st + NST <= J; st += NST)
    unrolled<NST>([&](auto p) {
      half(p, I0{}, st + (int)p);
      half(p, I1{}, st + (int)p);
    });
  unrolled<NST - 1>([&](auto p) {
    if (st < J) {
      half(p, I0{}, st);
      half(p, I1{}, st++);
    }
  });
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  barrier_lds();

  // (the lane's number anew: nothing of it has to last through the loop)
  const int l = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  // the adapter: acc += B (s u)^T, 16 ranks a product of 32: lane groups 0 and 1 carry the
  // bf16 high part of s u, 2 and 3 its remainder, against the same ranks of B
  if constexpr (ONE) {
    u32x4 lb[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j)
      lb[j] = *reinterpret_cast<const u32x4*>(smem + G::LDS_L + (TN * wn + j) * 512 +
                                              16 * (l & 31));
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(smem + G::LDS_V + (TM * wm + i) * 1024 +
                                                      16 * l);
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lb[j]),
                                                            __builtin_bit_cast(bf16x8, v),
                                                            acc[i][j], 0, 0, 0);
    }
  } else {
    // (tiles past the matrix repeat its last one: nothing of them is stored)
    const u32x4 *up[TM], *bp[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
      up[i] = reinterpret_cast<const u32x4*>(su) +
              (m0 / 16 + min(TM * wm + i, mt - 1)) * nj * 64 + l;
#pragma unroll
    for (int j = 0; j < TN; ++j)
      bp[j] = reinterpret_cast<const u32x4*>(bo) +
              (n0 / 16 + min(TN * wn + j, nt - 1)) * nj * 32 + (l & 31);
    for (int q = 0; q < nj; ++q) {
      u32x4 v[TM], lb[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) lb[j] = bp[j][32 * q];
#pragma unroll
      for (int i = 0; i < TM; ++i) v[i] = up[i][64 * q];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lb[j]),
                                                              __builtin_bit_cast(bf16x8, v[i]),
                                                              acc[i][j], 0, 0, 0);
    }
  }

  // store: lane (g, n) holds row n of tile (i, j), columns 4 g .. 4 g + 3; through the
  // wave's LDS staging tile, half the rows at a time, which leaves as rows of 32 TN bytes
  uint8_t* stg = smem + wave * G::OUTW;
  constexpr int LR = 2 * TN, RPS = 64 / LR;  // lanes of a row, rows a store
  const int lc = l % LR;
  const int64_t col = n0 + 16 * TN * wn + 8 * lc;
  const bool whole = (N & 7) == 0;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int i = 0; i < TM / 2; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const f32x4 c = acc[p * TM / 2 + i][j];
        *reinterpret_cast<u32x2*>(stg + (16 * i + (l & 15)) * G::OUTP + 2 * (16 * j + 4 * (l >> 4))) =
            u32x2{pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
      }
    // (a wave's LDS accesses execute in order)
    const int64_t row0 = m0 + 16 * TM * wm + 8 * TM * p;
    if (whole) {
#pragma unroll
      for (int q = 0; q < 8 * TM / RPS; ++q) {
        const int rl = RPS * q + l / LR;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stg + rl * G::OUTP + 16 * lc);
        if (row0 + rl < M && col < N)
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y + (row0 + rl) * N + col));
      }
    } else {  // rows of y on any element
      for (int q = 0; q < 8 * TM / RPS; ++q) {
        const int rl = RPS * q + l / LR;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stg + rl * G::OUTP + 16 * lc);
        if (row0 + rl >= M || col >= N) continue;
        uint16_t* dst = y + (row0 + rl) * N + col;
        if (col + 8 <= N)
          *reinterpret_cast<u32x4_any*>(dst) = v;
        else
          for (int k = 0; col + k < N; ++k) dst[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
}

// ---- The product of few rows: W is read once, straight into registers.  A workgroup
// takes 16 NT rows of W and all of x's 16 MT, its waves the steps in turn; their sums meet
// in LDS.  u comes whole or in S slices, which every workgroup adds (u_out: the first
// one writes the sum); its loads and those of B go out ahead of W's.  Bound by W from
// memory and by the latency of one pass: 1x14336x4096 8.9 us (31.8 MB, 3.6 TB/s),
// 16x4096x14336 10.6 (34.4 MB).  Four steps' loads at once instead of two: slower; 16 slices
// of u instead of 8: x's pass wins what this one loses.
constexpr int kFewSlices = 8;
// ranks j .. j + 15 of a row of B (zero past r)
__device__ __forceinline__ void load_ranks(const uint16_t* row, int j, int r, float v[16]) {
  if ((r & 7) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(row + min(j + 8 * h, r - 8));
      const bool in = j + 8 * h < r;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[8 * h + 2 * q] = in ? bf16_lo(w[q]) : 0.f;
        v[8 * h + 2 * q + 1] = in ? bf16_hi(w[q]) : 0.f;
      }
    }
  } else {
    uint16_t w[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) w[q] = row[min(j + q, r - 1)];
#pragma unroll
    for (int q = 0; q < 16; ++q) v[q] = j + q < r ? as_f32((uint32_t)w[q] << 16) : 0.f;
  }
}
template <int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx4_rows(
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs, int M, int64_t N, int J,
    const float* __restrict__ u, const float* __restrict__ upart, int S, float* __restrict__ u_out,
    const uint16_t* __restrict__ B, int r, float s, uint16_t* __restrict__ y) {
  constexpr int ROWS = 16 * NT, PITCH = ROWS + 4, THREADS = 64 * WAVES;
  __shared__ __attribute__((aligned(16))) float sums[WAVES][16 * MT][PITCH];
  extern __shared__ __attribute__((aligned(16))) float us[];  // u, rows of 16 ceil(r / 16)
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * ROWS;
  const uint8_t *wp[NT], *xp[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) wp[i] = wc + min(n0 + 16 * i + n, N - 1) * 128 * J + 16 * g;
#pragma unroll
  for (int i = 0; i < MT; ++i) xp[i] = xc + (int64_t)min(16 * i + n, M - 1) * 128 * J + 16 * g;
  // (16 rows of W: their half of the 32 rows' scales)
  const uint8_t* wsp = ws + n0 / 32 * J * 256 + 4 * lane + (NT == 1 ? 2 * ((n0 >> 4) & 1) : 0);
  const uint32_t* xsp = reinterpret_cast<const uint32_t*>(xs) + lane;
  // this thread's column of y, its row of B, its first element of u
  const int c = tid % ROWS, rp = (r + 15) & ~15, mr = M * r;
  const uint16_t* bp = B + min(n0 + c, N - 1) * r;
  float bv[16], uv[kFewSlices];
  if (r > 0) {
#pragma unroll
    for (int k = 0; k < kFewSlices; ++k)
      uv[k] = S > 1 ? upart[min(k, S - 1) * (int64_t)mr + min(tid, mr - 1)]
                    : u[min(tid, mr - 1)];
    load_ranks(bp, 0, r, bv);
  }
  f32x4 acc[NT][MT] = {};
  constexpr int U = 2;  // steps whose loads go out together
  for (int j0 = wave; j0 < J; j0 += U * WAVES) {
    u32x4 a[U][NT][2], b[U][MT][2];
    int sa[U], sb[U][(MT + 1) / 2];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int64_t j = min(j0 + q * WAVES, J - 1);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          a[q][i][t] = *reinterpret_cast<const u32x4*>(wp[i] + 128 * j + 64 * t);
      sa[q] = NT == 1 ? (int)*reinterpret_cast<const uint16_t*>(wsp + 256 * j)
                      : *reinterpret_cast<const int*>(wsp + 256 * j);
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int64_t j = min(j0 + q * WAVES, J - 1);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          b[q][i][t] = *reinterpret_cast<const u32x4*>(xp[i] + 128 * j + 64 * t);
#pragma unroll
      for (int i = 0; i < (MT + 1) / 2; ++i)  // (past M's groups: the last one's)
        sb[q][i] = (int)xsp[(min(i, (M - 1) >> 5) * (int64_t)J + j) * 64];
    }
    unrolled<U>([&](auto q_t) {
      constexpr int q = decltype(q_t)::value;
      if (j0 + q * WAVES < J)
        unrolled<2 * NT * MT>([&](auto k_t) {
          constexpr int k = decltype(k_t)::value, t = k & 1, i = (k >> 1) % NT, m = (k >> 1) / NT;
          acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              frag4(a[q][i][t]), frag4(b[q][m][t]), acc[i][m], 4, 4, 2 * i + t, sa[q],
              2 * (m & 1) + t, sb[q][m >> 1]);
        });
    });
  }
  for (int e = tid; e < mr; e += THREADS) {
    float t = uv[0];
    if (e == tid) {
#pragma unroll
      for (int k = 1; k < kFewSlices; ++k)
        if (k < S) t += uv[k];
    } else {
      t = S > 1 ? slice_sum(upart, (int64_t)mr, S, e) : u[e];
    }
    us[e / r * rp + e % r] = t;
    if (u_out && blockIdx.x == 0) u_out[e] = t;
  }
  // lane: row 16 m + n of y, columns 16 i + 4 g + 0 .. 3
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      *reinterpret_cast<f32x4*>(&sums[wave][16 * m + n][16 * i + 4 * g]) = acc[i][m];
  __syncthreads();
  for (int m = tid / ROWS; m < M; m += THREADS / ROWS) {
    float t = sums[0][m][c], low = 0.f;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) t += sums[w][m][c];
    for (int j = 0; j < r; j += 16) {
      if (r > 16) load_ranks(bp, j, r, bv);
      const float* um = us + m * rp + j;
#pragma unroll
      for (int q = 0; q < 16; ++q) low += j + q < r ? um[q] * bv[q] : 0.f;
    }
    if (n0 + c < N) y[(int64_t)m * N + n0 + c] = to_bf16(t + s * low);
  }
}

// The same from x itself, in one launch, without an adapter: every workgroup rounds all
// of x, from the second level cache.  Lane (g, n) takes all 32 columns of its block of
// row n, so that the block's largest magnitude needs no exchange.  Against a pass of its
// own for x: 14336x4096 10.2 us a call instead of 12.2 for one row and 11.8 instead of 12.7
// for eight (four rounds of x's bytes for one of W's: 14.4 and 13.9 for sixteen),
// 4096x4096 4.7 and 7.1, 5.8 and 7.5.  With u formed in every workgroup as well (r = 16)
// 17.5 instead of 14.5: A is more bytes than the workgroup's rows of W.
template <int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx4_token(
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
    const uint16_t* __restrict__ x, int M, int64_t N, int64_t K, int J,
    uint16_t* __restrict__ y) {
  constexpr int ROWS = 16 * NT, PITCH = ROWS + 4, THREADS = 64 * WAVES;
  __shared__ __attribute__((aligned(16))) float sums[WAVES][16][PITCH];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * ROWS;
  const uint8_t* wp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) wp[i] = wc + min(n0 + 16 * i + n, N - 1) * 128 * J + 16 * g;
  const uint8_t* wsp = ws + n0 / 32 * J * 256 + 4 * lane + (NT == 1 ? 2 * ((n0 >> 4) & 1) : 0);
  const uint16_t* xp = x + (int64_t)min(n, M - 1) * K;
  f32x4 acc[NT] = {};
  for (int j = wave; j < J; j += WAVES) {
    u32x4 a[NT][2], xv[2][4], b[2];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        a[i][t] = *reinterpret_cast<const u32x4*>(wp[i] + 128 * (int64_t)j + 64 * t);
    const int sa = NT == 1 ? (int)*reinterpret_cast<const uint16_t*>(wsp + 256 * (int64_t)j)
                           : *reinterpret_cast<const int*>(wsp + 256 * (int64_t)j);
    bool in[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {  // past the row (K is a multiple of 32): its first columns
      const int64_t col = (int64_t)j * kMx4Step + 32 * (4 * t + g);
      in[t] = col < K;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        xv[t][q] = *reinterpret_cast<const u32x4*>(xp + (in[t] ? col : 0) + 8 * q);
    }
    int sb = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t top = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (!in[t]) xv[t][q] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = pk_max(top, xv[t][q][e] & 0x7fff7fffu);
      }
      const uint32_t E = mx4_exp(max(top << 16, top & 0xffff0000u));
      b[t] = u32x4{encode8(xv[t][0], E), encode8(xv[t][1], E), encode8(xv[t][2], E),
                   encode8(xv[t][3], E)};
      sb |= (int)(E << (8 * t));
    }
    unrolled<2 * NT>([&](auto k_t) {
      constexpr int k = decltype(k_t)::value, t = k & 1, i = k >> 1;
      acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag4(a[i][t]), frag4(b[t]), acc[i],
                                                                4, 4, 2 * i + t, sa, t, sb);
    });
  }
  // lane: row n of y, columns 16 i + 4 g + 0 .. 3
#pragma unroll
  for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(&sums[wave][n][16 * i + 4 * g]) = acc[i];
  __syncthreads();
  const int c = tid % ROWS;
  for (int m = tid / ROWS; m < M; m += THREADS / ROWS) {
    float t = sums[0][m][c];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) t += sums[w][m][c];
    if (n0 + c < N) y[(int64_t)m * N + n0 + c] = to_bf16(t);
  }
}

// ---- The backward's W: out[k][n] = W[n][k] as bf16 (exact: a level has two significant bits),
// row length ldt (zero for rows <= n < ldt).  dX is a bf16 product on it: dY is not rounded
// to 4 bits.  4096x4096 with A^T, B's operands and u's parts in spare workgroups 11.4 us
// (44.5 MB, 3.9 TB/s; the write goes to the memory-side cache, where the product
// reads it).  A workgroup
// takes 128 rows x 128 columns through LDS: thread (q, l) = (t / 64, t % 64) the block q
// of rows 2 l and 2 l + 1, whose columns leave as pairs of rows, a word each.
constexpr int kDtRows = 128, kDtPitch = 2 * kDtRows + 16;
__global__ __launch_bounds__(kThreads) void k_mx4_dequant_t(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
    int64_t K, int J, uint16_t* __restrict__ out, int64_t ldt, BwdAux aux, int aux_wgs, int gx) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kDtPitch];
  const int t = threadIdx.x;
  if ((int)blockIdx.x < aux_wgs) {  // one job per thread
    const int64_t i = (int64_t)blockIdx.x * kThreads + t;
    if (i < bwd_aux_count(aux)) bwd_aux_at(aux, i);
    return;
  }
  const int64_t d = (int64_t)blockIdx.x - aux_wgs, kh = d / gx;
  const int64_t n0 = (d - kh * gx) * kDtRows, k0 = kh * 128;
  const int q = t >> 6, l = t & 63, j = (int)(kh >> 1), b = 4 * (int)(kh & 1) + q;
  u32x4 c[2];
  float s[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = n0 + 2 * l + i, rr = min(row, rows - 1);
    c[i] = *reinterpret_cast<const u32x4*>(codes + rr * 128 * J + 128 * j + 16 * b);
    s[i] = mx4_scale(scales[((rr >> 5) * J + j) * 256 + mx4_scale_at((int)(rr & 31), b)]);
    if (row >= rows) {
      c[i] = u32x4{0u, 0u, 0u, 0u};
      s[i] = 1.f;
    }
  }
  uint8_t* trow = tile + 32 * q * kDtPitch + 4 * l;
  unrolled<4>([&](auto w_t) {
    constexpr int w = decltype(w_t)::value;
    const uint32_t ca = c[0][w], cb = c[1][w];
    unrolled<4>([&](auto p_t) {  // columns 8 w + 2 p, + 1
      constexpr int p = decltype(p_t)::value;
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ca, 1.f, p);
      const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cb, 1.f, p);
      const float a0 = a[0], a1 = a[1], e0 = e[0], e1 = e[1];
      *reinterpret_cast<uint32_t*>(trow + (8 * w + 2 * p) * kDtPitch) =
          pack_bf16x2(a0 * s[0], e0 * s[1]);
      *reinterpret_cast<uint32_t*>(trow + (8 * w + 2 * p + 1) * kDtPitch) =
          pack_bf16x2(a1 * s[0], e1 * s[1]);
    });
  });
  __syncthreads();
  // 128 rows of 256 bytes: pass h, thread t -> row 16 h + t / 16, chunk t % 16
  const int64_t col = n0 + 8 * (t & 15);
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    const int k = 16 * h + (t >> 4);
    const u32x4 v = *reinterpret_cast<const u32x4*>(tile + k * kDtPitch + 16 * (t & 15));
    if (col < ldt && k0 + k < K) *reinterpret_cast<u32x4*>(out + (k0 + k) * ldt + col) = v;
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
  const int64_t wgs = (bwd_aux_count(aux) + kThreads - 1) / kThreads;
  const int64_t gx = (ldt + kDtRows - 1) / kDtRows, gk = (w.cols + 127) / 128;
  hipLaunchKernelGGL(k_mx4_dequant_t, dim3((unsigned)(wgs + gx * gk)), dim3(kThreads), 0, st,
                     w.codes, w.scales, w.rows, w.cols, (int)mx4_steps(w.cols), out, ldt, aux,
                     (int)wgs, (int)gx);
  return hipGetLastError();
}

namespace {
template <int WVM, int WVN, int TM, int TN, int NST>
hipError_t launch_tiles(const Mx4& w, const Mx4X& x, uint16_t* y, hipStream_t st) {
  using G = MxGeo<WVM, WVN, TM, TN, NST>;
  const int64_t tm = (x.M + G::BM - 1) / G::BM, tn = (w.rows + G::BN - 1) / G::BN;
  const int J = (int)mx4_steps(w.cols), nj = (x.r + 15) / 16, lds = nj == 1 ? G::LDS_BYTES : G::LDS_MAIN;
  const auto kernel = nj == 1 ? k_mx4_gemm<WVM, WVN, TM, TN, NST, true>
                              : k_mx4_gemm<WVM, WVN, TM, TN, NST, false>;
  // (the attribute is the current device's)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(G::THREADS), lds, st, w.codes, w.scales,
                     x.codes, x.scales, x.M, w.rows, J, x.su, x.bo, nj, y, (int)tm, (int)tn);
  return hipGetLastError();
}

template <int MT, int NT, int WAVES>
hipError_t launch_rows(const Mx4& w, const Mx4X& x, const uint16_t* B, float s, uint16_t* y,
                       hipStream_t st) {
  const dim3 grid((unsigned)((w.rows + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((k_mx4_rows<MT, NT, WAVES>), grid, dim3(64 * WAVES),
                     (size_t)x.M * ((x.r + 15) / 16 * 16) * sizeof(float), st, w.codes, w.scales, x.codes,
                     x.scales,
                     (int)x.M, w.rows, (int)mx4_steps(w.cols), x.u, x.upart, x.S,
                     x.S > 1 ? x.u : nullptr, B, x.r, s, y);
  return hipGetLastError();
}

template <int RT, int NJ, int WAVES>
hipError_t launch_x(const uint16_t* x, int64_t K, const Mx4X& o, const Drop& d, const uint16_t* A,
                    const uint16_t* B, int64_t N, float s, hipStream_t st) {
  const int J = (int)mx4_steps(K);
  const int64_t b_wgs = o.bo ? ((N + 15) / 16 * NJ * 32 + 64 * WAVES - 1) / (64 * WAVES) : 0;
  const dim3 grid((unsigned)(b_wgs + (o.M + 16 * RT - 1) / (16 * RT) * o.S));
  if (d.on)
    hipLaunchKernelGGL((k_mx4_x<RT, NJ, true, WAVES>), grid, dim3(64 * WAVES), 0, st, x, o.M, K, J,
                       o.S, d, A, B, N, o.r, s, o.codes, o.scales, o.u, o.upart, o.su, o.bo,
                       (int)b_wgs);
  else
    hipLaunchKernelGGL((k_mx4_x<RT, NJ, false, WAVES>), grid, dim3(64 * WAVES), 0, st, x, o.M, K, J,
                       o.S, d, A, B, N, o.r, s, o.codes, o.scales, o.u, o.upart, o.su, o.bo,
                       (int)b_wgs);
  return hipGetLastError();
}
template <int RT, int WAVES>
hipError_t launch_x(const uint16_t* x, int64_t K, const Mx4X& o, const Drop& d, const uint16_t* A,
                    const uint16_t* B, int64_t N, float s, hipStream_t st) {
  switch ((o.r + 15) / 16) {
    case 1: return launch_x<RT, 1, WAVES>(x, K, o, d, A, B, N, s, st);
    case 2: return launch_x<RT, 2, WAVES>(x, K, o, d, A, B, N, s, st);
    case 3: return launch_x<RT, 3, WAVES>(x, K, o, d, A, B, N, s, st);
    default: return launch_x<RT, 4, WAVES>(x, K, o, d, A, B, N, s, st);
  }
}
}  // namespace

namespace {
int64_t compute_units() {
  static const int n = [] {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return 256;
    return cus > 0 ? cus : 256;
  }();
  return n;
}
}  // namespace

int mx4_x_slices(int64_t M, int64_t K, int r) {
  const int64_t J = mx4_steps(K), most = std::min<int64_t>(J, kFewSlices);
  if (mx4_few_rows(M, r)) return (int)most;
  // More rows in slices where one workgroup's walk takes longer than the launch that adds
  // them (pass, sum and product at 4096 columns 14.4 us instead of 17.8 for 128 rows and 16
  // ranks, at 14336 25.2 instead of 45.2, with 64 ranks 34.0 instead of 83.7; at 2048 with 16
  // ranks 12.3 and 12.8, with 64 17.0 and 20.4, at 1024 11.2 and 10.3), as many as leave a
  // workgroup to a compute unit
  if (J * ((r + 15) / 16 + 2) < 48) return 1;
  return (int)std::max<int64_t>(1, std::min(most, 256 / ((M + 15) / 16)));
}

hipError_t launch_mx4_x(const uint16_t* x, int64_t K, const Mx4X& o, const Drop& d,
                        const uint16_t* A, const uint16_t* B, int64_t N, float s, hipStream_t st) {
  if (o.r == 0) return launch_mx4_quant(x, false, o.M, K, o.codes, o.scales, st);
  // (up to 16 ranks 16 waves fit beside each other: long rows 26 -> 24 us at 8192x4096 with
  // dropout, 81 -> 71 at 4608x14336; 1024 columns are eight waves' work)
  if (o.M > 4096)
    return o.r <= 16 && mx4_steps(K) >= 16 ? launch_x<2, 1, 16>(x, K, o, d, A, B, N, s, st)
                                           : launch_x<2, 8>(x, K, o, d, A, B, N, s, st);
  if (mx4_few_rows(o.M, o.r)) return launch_x<1, 8>(x, K, o, d, A, B, N, s, st);
  if (o.S > 1) {
    Mx4X part = o;
    part.su = nullptr;
    const hipError_t e = launch_x<1, 8>(x, K, part, d, A, B, N, s, st);
    const int nj = (o.r + 15) / 16;
    const int64_t n = (o.M + 15) / 16 * nj * 32;
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_mx4_u, dim3((unsigned)((n + kThreadsU - 1) / kThreadsU)), dim3(kThreadsU),
                       0, st, o.upart, o.S, o.M, o.r, nj, s, o.u, o.su, n);
    return hipGetLastError();
  }
  return launch_x<1, 16>(x, K, o, d, A, B, N, s, st);
}

namespace {
template <int NT, int WAVES>
hipError_t launch_token(const Mx4& w, const uint16_t* x, int64_t M, uint16_t* y, hipStream_t st) {
  const dim3 grid((unsigned)((w.rows + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((k_mx4_token<NT, WAVES>), grid, dim3(64 * WAVES), 0, st, w.codes, w.scales, x,
                     (int)M, w.rows, w.cols, (int)mx4_steps(w.cols), y);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_mx4_token(const Mx4& w, const uint16_t* x, int64_t M, uint16_t* y,
                            hipStream_t st) {
  if (!mx4_one_launch(M, w.cols, 0)) return hipErrorInvalidValue;
  return w.rows >= 16 * 512 ? launch_token<2, 8>(w, x, M, y, st)
                            : launch_token<1, 16>(w, x, M, y, st);
}

hipError_t launch_mx4_mm(const Mx4& w, const Mx4X& x, const uint16_t* B, float s, uint16_t* y,
                         hipStream_t st) {
  if (mx4_few_rows(x.M, x.r)) {
    const bool wide = w.rows >= 16 * 512;
    if (x.M <= 16)
      return wide ? launch_rows<1, 2, 8>(w, x, B, s, y, st)
                  : launch_rows<1, 1, 16>(w, x, B, s, y, st);
    return launch_rows<2, 2, 8>(w, x, B, s, y, st);
  }
  const int64_t cu = compute_units();
  const auto tiles = [&](int64_t tm, int64_t tn) {
    return (x.M + tm - 1) / tm * ((w.rows + tn - 1) / tn);
  };
  // Few tiles: the smallest that still go one to a compute unit, four stages deep (a
  // unit's loads in flight bound it: 128x4096x14336 by 64 x 64 tiles 14.2 us, by 64 x 128
  // 18.8, by 128 x 128 26.2; 300x4096x4096, 320 of the first kind, 10.9, 8.7 and 12.4;
  // 1000x4096x4096 19.7, 17.8 and 13.8).
  if (tiles(64, 64) <= cu) return launch_tiles<2, 2, 2, 2, 4>(w, x, y, st);
  if (tiles(64, 128) <= cu) return launch_tiles<2, 2, 2, 4, 4>(w, x, y, st);
  if (tiles(128, 128) <= cu) return launch_tiles<2, 4, 4, 2, 4>(w, x, y, st);
  // Many: 256 x 256, one a compute unit, or 128 x 128, two, two stages deep.  A round of the
  // small ones takes 0.57 of a round of the large ones (8192x4096x4096: 84 us in 4 against
  // 74 in 2), so the large ones where they need no more than 0.6 as many
  // (301x50021x1000, 2 rounds and 3: 28.9 us and 23.8; 4096x14336x4096, 4 and 7: 134
  // and 155).
  const auto rounds = [&](int64_t t, int64_t at_once) {
    return (tiles(t, t) + at_once - 1) / at_once;
  };
  if (10 * rounds(256, cu) <= 6 * rounds(128, 2 * cu))
    return launch_tiles<2, 4, 8, 4, 2>(w, x, y, st);
  return launch_tiles<2, 2, 4, 4, 2>(w, x, y, st);
}

}  // namespace qn
