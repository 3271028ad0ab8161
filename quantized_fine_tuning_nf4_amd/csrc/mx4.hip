// MXFP4: matrices in 4 bits with a power-of-two scale for every 32 columns of a row
// (format in the header), into the format and back, and the linear's product on two
// of them with the adapter term.
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

// ---- The product of many rows.  Workgroup tile BM x BN (rows of x, rows of W), WVM x WVN
// waves of TM x TN tiles of v_mfma_scale_f32_16x16x128_f8f6f4.  A step is 256 columns:
// rows of 128 bytes of codes and 256 scale bytes per 32 rows go from global memory
// straight into LDS, two stages deep.  Chunk c (16 bytes, a block) of row y sits at unit
// c ^ ((y >> 1) & 7), so that 16 rows of a fragment read sit on distinct banks.  In
// half t of a step lane (g, n) = (l / 16, l % 16) takes row n's block 4 t + g, whose scale
// is byte 2 (tile % 2) + t of the lane's four.
template <int WVM, int WVN, int TM, int TN>
struct MxGeo {
  static constexpr int WAVES = WVM * WVN, THREADS = 64 * WAVES;
  static constexpr int BM = 16 * TM * WVM, BN = 16 * TN * WVN;
  static constexpr int XB = BM * 128, WB = BN * 128;   // codes of a stage
  static constexpr int XS = XB + WB, WS = XS + BM * 8;  // its scales
  static constexpr int STB = WS + BN * 8;              // bytes of a stage
  // output staging of a wave: half its rows at a time
  static constexpr int OUTP = 32 * TN + 16, OUTW = 8 * TM * OUTP;
  static constexpr int LDS_MAIN = 2 * STB > WAVES * OUTW ? 2 * STB : WAVES * OUTW;
  static constexpr int LDS_V = LDS_MAIN, LDS_L = LDS_V + BM * 64;  // r == 16: u and B of the tile
  static constexpr int LDS_BYTES = LDS_L + BN * 32;
  static constexpr int XL = BM / 8 / WAVES, WL = BN / 8 / WAVES;   // loads of a wave and step ...
  static constexpr int SL = (BM + BN) / 128;                       // ... and of all, of scales
  static_assert(LDS_BYTES <= 160 * 1024 && WAVES % SL == 0, "LDS");
};

typedef __attribute__((address_space(3))) void lds_void;
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

// f(0), f(1), .. f(N - 1), each with its index as a constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}

template <int WVM, int WVN, int TM, int TN, bool LORA16>
__global__ __launch_bounds__(64 * WVM * WVN, 2) void k_mx4_gemm(
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs, int64_t M, int64_t N, int J,
    const float* __restrict__ V, const uint16_t* __restrict__ L, int r, float s,
    uint16_t* __restrict__ y, int tiles_m, int tiles_n) {
  using G = MxGeo<WVM, WVN, TM, TN>;
  constexpr int BM = G::BM, BN = G::BN, STB = G::STB, XL = G::XL, WL = G::WL, LPS = XL + WL;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WVN, wn = wave % WVN;

  // tile order: each XCD (they take workgroups round robin) a contiguous run of the
  // tiles, four tile rows at a time across the columns
  int bid = blockIdx.x;
  const int ntiles = tiles_m * tiles_n;
  if (ntiles % 8 == 0) bid = (bid & 7) * (ntiles >> 3) + (bid >> 3);
  int tm, tn;
  if (tiles_m % 4 == 0) {
    const int grp = bid / (4 * tiles_n), in = bid % (4 * tiles_n);
    tm = 4 * grp + (in & 3);
    tn = in >> 2;
  } else {
    tm = bid / tiles_n;
    tn = bid % tiles_n;
  }
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
  // scales: 1 KB (four groups of 32 rows) a wave, those of x first; there are twice as
  // many waves, and the upper ones load the same again
  const int sq = wave % G::SL;
  const bool sx = sq < BM / 128;
  const int sg = 4 * (sx ? sq : sq - BM / 128) + (lane >> 4);  // group of the tile
  const int sgroups = ((sx ? mrows : nrows) + 31) >> 5;
  const rsrc_t rs = make_rs(sx ? xs + m0 / 32 * J * 256 : ws + n0 / 32 * J * 256,
                            (uint32_t)(sgroups * J * 256));
  const uint32_t soff = (uint32_t)(min(sg, sgroups - 1) * J * 256 + 16 * (lane & 15));
  // load q (0 .. LPS) of step st
  auto load_one = [&](int q, int st, int stage) {
    uint8_t* base = smem + stage * STB;
    const uint32_t so = (uint32_t)st * 128;
    if (q < XL)
      dma16(rx, xoff[q], so, base + 1024 * (XL * wave + q));
    else if (q < LPS)
      dma16(rw, woff[q - XL], so, base + G::XB + 1024 * (WL * wave + q - XL));
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

  if constexpr (LORA16) {  // u and B of the tile (rows past it read zeros)
    const rsrc_t rv = make_rs(V + m0 * 16, (uint32_t)(mrows * 64));
    const rsrc_t rl = make_rs(L + n0 * 16, (uint32_t)(nrows * 32));
#pragma unroll
    for (int k = 0; k < BM / 16 / G::WAVES; ++k) {
      const int q = BM / 16 / G::WAVES * wave + k;
      dma16(rv, (uint32_t)(1024 * q + 16 * lane), 0, smem + G::LDS_V + 1024 * q);
    }
#pragma unroll
    for (int k = 0; k < BN / 32 / G::WAVES; ++k) {
      const int q = BN / 32 / G::WAVES * wave + k;
      dma16(rl, (uint32_t)(1024 * q + 16 * lane), 0, smem + G::LDS_L + 1024 * q);
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int q = 0; q <= LPS; ++q) load_one(q, min(k, J - 1), k);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LPS + 1) : "memory");
  barrier_lds();
#pragma unroll
  for (int i = 0; i < TM; ++i) fx[i] = frag(0, xbase, i, 0);
#pragma unroll
  for (int j = 0; j < TN; ++j) fw[0][j] = frag(0, wbase, j, 0);
#pragma unroll
  for (int i = 0; i < TM / 2; ++i) ex[0][i] = scale(0, xsb, i);
#pragma unroll
  for (int j = 0; j < TN / 2; ++j) ew[0][j] = scale(0, wsb, j);

  // half t of step st on stage P = st % 2.  The fragments of the next half are read while
  // this one's products run (those of W in a second set, those of x in place after their
  // row).  At the end of half 0 every wave has read the stage and step st + 1 has
  // landed; half 1 sends the loads of step st + 2 into the stage.
  auto half = [&](auto p_t, auto t_t, int st) {
    constexpr int P = decltype(p_t)::value, H = decltype(t_t)::value;
    constexpr int RS = H == 0 ? P : P ^ 1, RH = H ^ 1;
    const int lst = min(st + 2, J - 1);
    unrolled<TM>([&](auto i_t) {
      constexpr int i = decltype(i_t)::value;
      unrolled<TN>([&](auto j_t) {
        constexpr int j = decltype(j_t)::value;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            frag4(fw[H][j]), frag4(fx[i]), acc[i][j], 4, 4, 2 * (j & 1) + H, ew[P][j / 2],
            2 * (i & 1) + H, ex[P][i / 2]);
        if (i == 0) fw[RH][j] = frag(RS, wbase, j, RH);
        if (H == 1 && i == 1 && j < TN / 2) ew[P ^ 1][j] = scale(RS, wsb, j);
        if (H == 1 && i >= 2 && j == 0 && i - 2 < TM / 2) ex[P ^ 1][i - 2] = scale(RS, xsb, i - 2);
        if (H == 1 && j == TN / 2)
          for (int q = (LPS + TM) / TM * i; q < (LPS + TM) / TM * (i + 1); ++q)
            if (q <= LPS) load_one(q, lst, P);
      });
      fx[i] = frag(RS, xbase, i, RH);
      __builtin_amdgcn_sched_barrier(0);
    });
    if (H == 0) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      barrier_lds();
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  int st = 0;
  for (; st + 2 <= J; st += 2) {
    half(I0{}, I0{}, st);
    half(I0{}, I1{}, st);
    half(I1{}, I0{}, st + 1);
    half(I1{}, I1{}, st + 1);
  }
  if (st < J) {
    half(I0{}, I0{}, st);
    half(I0{}, I1{}, st);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  barrier_lds();

  // the adapter: acc += B (s u)^T, 16 ranks a product of 32: lane groups 0 and 1 carry the
  // bf16 high part of s u, 2 and 3 its remainder, against the same ranks of B
  for (int j0 = 0; j0 < r; j0 += 16) {
    const int jl = j0 + 8 * (g & 1);
    bf16x8 lb[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int row = 16 * (TN * wn + j) + n;
      if constexpr (LORA16) {
        lb[j] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
            smem + G::LDS_L + row * 32 + 16 * (g & 1)));
      } else {
        const uint16_t* lp = L + min(n0 + row, N - 1) * r;
        uint32_t e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = jl + q < r ? lp[min(jl + q, r - 1)] : 0u;
        lb[j] = __builtin_bit_cast(bf16x8, u32x4{e[0] | (e[1] << 16), e[2] | (e[3] << 16),
                                                 e[4] | (e[5] << 16), e[6] | (e[7] << 16)});
      }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = 16 * (TM * wm + i) + n;
      float v[8];
      if constexpr (LORA16) {
        const uint8_t* vp = smem + G::LDS_V + row * 64 + 32 * (g & 1);
        const f32x4 a = *reinterpret_cast<const f32x4*>(vp);
        const f32x4 b = *reinterpret_cast<const f32x4*>(vp + 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = a[q];
          v[4 + q] = b[q];
        }
      } else {
        const float* vp = V + min(m0 + row, M - 1) * r;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = jl + q < r ? vp[min(jl + q, r - 1)] : 0.f;
      }
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float a = s * v[2 * q], b = s * v[2 * q + 1];
        const uint32_t hi = pack_bf16x2(a, b);
        w[q] = g >= 2 ? pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi)) : hi;
      }
      const bf16x8 vh = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lb[j], vh, acc[i][j], 0, 0, 0);
    }
  }

  // store: lane (g, n) holds row n of tile (i, j), columns 4 g .. 4 g + 3; through the
  // wave's LDS staging tile, half the rows at a time, which leaves as rows of 32 TN bytes
  uint8_t* stg = smem + wave * G::OUTW;
  constexpr int LR = 2 * TN, RPS = 64 / LR;  // lanes of a row, rows a store
  const int lc = lane % LR;
  const int64_t col = n0 + 16 * TN * wn + 8 * lc;
  const bool whole = (N & 7) == 0;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int i = 0; i < TM / 2; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const f32x4 c = acc[p * TM / 2 + i][j];
        *reinterpret_cast<u32x2*>(stg + (16 * i + n) * G::OUTP + 2 * (16 * j + 4 * g)) =
            u32x2{pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
      }
    // (a wave's LDS accesses execute in order)
    const int64_t row0 = m0 + 16 * TM * wm + 8 * TM * p;
    if (whole) {
#pragma unroll
      for (int q = 0; q < 8 * TM / RPS; ++q) {
        const int rl = RPS * q + lane / LR;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stg + rl * G::OUTP + 16 * lc);
        if (row0 + rl < M && col < N)
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y + (row0 + rl) * N + col));
      }
    } else {  // rows of y on any element
      for (int q = 0; q < 8 * TM / RPS; ++q) {
        const int rl = RPS * q + lane / LR;
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

namespace {
template <int WVM, int WVN, int TM, int TN>
hipError_t launch_tiles(const Mx4& w, const uint8_t* xc, const uint8_t* xs, int64_t M,
                        const float* u, const uint16_t* B, int r, float s, uint16_t* y,
                        hipStream_t st) {
  using G = MxGeo<WVM, WVN, TM, TN>;
  static const hipError_t attr = [] {
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(k_mx4_gemm<WVM, WVN, TM, TN, true>),
        hipFuncAttributeMaxDynamicSharedMemorySize, G::LDS_BYTES);
    return e != hipSuccess
               ? e
               : hipFuncSetAttribute(
                     reinterpret_cast<const void*>(k_mx4_gemm<WVM, WVN, TM, TN, false>),
                     hipFuncAttributeMaxDynamicSharedMemorySize, G::LDS_MAIN);
  }();
  if (attr != hipSuccess) return attr;
  const int64_t tm = (M + G::BM - 1) / G::BM, tn = (w.rows + G::BN - 1) / G::BN;
  const dim3 grid((unsigned)(tm * tn)), block(G::THREADS);
  const int J = (int)mx4_steps(w.cols);
  if (r == 16)
    hipLaunchKernelGGL((k_mx4_gemm<WVM, WVN, TM, TN, true>), grid, block, G::LDS_BYTES, st, w.codes,
                       w.scales, xc, xs, M, w.rows, J, u, B, r, s, y, (int)tm, (int)tn);
  else
    hipLaunchKernelGGL((k_mx4_gemm<WVM, WVN, TM, TN, false>), grid, block, G::LDS_MAIN, st, w.codes,
                       w.scales, xc, xs, M, w.rows, J, u, B, r, s, y, (int)tm, (int)tn);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_mx4_mm(const Mx4& w, const uint8_t* xc, const uint8_t* xs, int64_t M,
                         const float* u, const uint16_t* B, int r, float s, uint16_t* y,
                         hipStream_t st) {
  if (M > 64) {
    if ((M + 255) / 256 * ((w.rows + 255) / 256) >= 240)
      return launch_tiles<2, 4, 8, 4>(w, xc, xs, M, u, B, r, s, y, st);
    return launch_tiles<2, 2, 4, 4>(w, xc, xs, M, u, B, r, s, y, st);
  }
  const uint32_t cols_wgs = (uint32_t)((w.rows + 127) / 128);
  const dim3 grid(cols_wgs * (uint32_t)((M + 31) / 32));  // (at most 2^31)
  hipLaunchKernelGGL(k_mx4_mm, grid, dim3(kThreads), 0, st, w.codes, w.scales, xc, xs, M, w.rows,
                     (int)mx4_steps(w.cols), u, B, r, s, y, cols_wgs);
  return hipGetLastError();
}

}  // namespace qn
