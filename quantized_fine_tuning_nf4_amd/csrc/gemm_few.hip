// bf16 products of small outputs with the adapter term:
//
//   C[M, Nc] (bf16) = A[M, R] Bm[Nc, R]^T + s V[M, r] L[Nc, r]^T (.) mask
//
// the same as gemm_bf16.hip's, where that kernel's 128 x 128 tiles are too few to fill the
// chip (M = 1, Nc = 5112, R = 2688: 40 workgroups walk 42 steps).  Two kernels:
// k_gemm_few splits the reduction over a workgroup's waves, k_gemm_tiles takes small
// LDS tiles; launch_gemm_any chooses.
#include <type_traits>

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

// s V's eight ranks as bf16: the high parts, or what they leave
__device__ __forceinline__ bf16x8 split(const f32x4 v[2], float s, bool rest) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float x = s * v[q >> 1][2 * (q & 1)], z = s * v[q >> 1][2 * (q & 1) + 1];
    const uint32_t hi = pack_bf16x2(x, z);
    w[q] = rest ? pack_bf16x2(x - bf16_lo(hi), z - bf16_hi(hi)) : hi;
  }
  return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
}

// ---- 16 MT rows of A and 16 of Bm a workgroup, straight into registers: its eight waves
// take the steps of 32 in turn, their loads out together, and a block of 16 ranks each;
// their sums meet in LDS.  Bound by the latency of one pass over the operands, so
// worth it where every workgroup has a compute unit of its own (M = 100, Nc = R = 1024
// 6.1 us by 256 workgroups; M = 1, 4096 and 4096 8.1, 34 MB of Bm).
template <int MT>
__global__ __launch_bounds__(64 * kWaves) void k_gemm_few(
    const uint16_t* __restrict__ A, int64_t lda, int64_t R, const uint16_t* __restrict__ Bm,
    int64_t ldb, int M, int64_t Nc, const float* __restrict__ V, const uint16_t* __restrict__ L,
    int r, float s, uint16_t* __restrict__ C, const uint8_t* __restrict__ mask, int col_wgs) {
  constexpr int PITCH = 16 + 4, THREADS = 64 * kWaves;
  constexpr int U = 8;  // steps whose loads go out together
  __shared__ __attribute__((aligned(16))) float sums[kWaves][16 * MT][PITCH];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mb = (int)blockIdx.x / col_wgs;  // block of 16 MT rows
  const int64_t c0 = (int64_t)((int)blockIdx.x - mb * col_wgs) * 16;
  A += (int64_t)mb * 16 * MT * lda;
  V += (int64_t)mb * 16 * MT * r;
  C += (int64_t)mb * 16 * MT * Nc;
  if (mask) mask += (int64_t)mb * 16 * MT * Nc / 8;
  M = min(M - mb * 16 * MT, 16 * MT);
  const uint16_t* ap[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) ap[i] = A + (int64_t)min(16 * i + n, M - 1) * lda + 8 * g;
  const uint16_t* bp = Bm + min(c0 + n, Nc - 1) * ldb + 8 * g;
  const int64_t lim = R - 8 * g;  // columns left for this lane's chunk (R % 8 == 0)
  const int steps = (int)((R + 31) / 32);
  // a block of 16 ranks is a wave's: its operands and keep bits go out first
  const int jl = 16 * wave + 8 * (g & 1);
  const bool share = 16 * wave < r;
  u32x4 lb;
  f32x4 va[MT][2];
  uint32_t kb[MT];
  if (share) {
    lb = ranks(L + min(c0 + n, Nc - 1) * r, jl, r);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = min(16 * m + n, M - 1);
      ranks(V + row * r, jl, r, va[m]);
      if (mask)  // (Nc % 64 == 0: a byte is half a tile's columns)
        kb[m] = mask[((row * Nc + c0) >> 3) + (g >> 1)] >> (4 * (g & 1));
    }
  }
  f32x4 acc[MT] = {};
  for (int s0 = wave * U; s0 < steps; s0 += U * kWaves) {
    u32x4 a[U][MT], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t off = 32 * (int64_t)(s0 + u);
      const bool in = off < lim;  // past the row: its first columns, zero in both operands
      b[u] = *reinterpret_cast<const u32x4*>(bp + (in ? off : -8 * g));
#pragma unroll
      for (int i = 0; i < MT; ++i)
        a[u][i] = *reinterpret_cast<const u32x4*>(ap[i] + (in ? off : -8 * g));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = 32 * (int64_t)(s0 + u) < lim;
      if (!in) b[u] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (!in) a[u][m] = u32x4{0u, 0u, 0u, 0u};
        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[u]),
                                                         __builtin_bit_cast(bf16x8, a[u][m]),
                                                         acc[m], 0, 0, 0);
      }
    }
  }
  // the wave's ranks of the adapter term: lane groups 0 and 1 carry the bf16 high part of
  // s V, 2 and 3 its remainder; what is dropped counts as zero
  if (share) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const f32x4 low = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(bf16x8, lb), split(va[m], s, g >= 2), f32x4{}, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (!mask || ((kb[m] >> q) & 1)) acc[m][q] += low[q];
    }
  }
  // lane: row 16 m + n of C, columns 4 g + 0 .. 3
#pragma unroll
  for (int m = 0; m < MT; ++m)
    *reinterpret_cast<f32x4*>(&sums[wave][16 * m + n][4 * g]) = acc[m];
  __syncthreads();
  const int c = tid % 16;
  if (c0 + c >= Nc) return;
  for (int m = tid / 16; m < M; m += THREADS / 16) {
    float t = sums[0][m][c];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t += sums[w][m][c];
    C[(int64_t)m * Nc + c0 + c] = to_bf16(t);
  }
}

// ---- A few tiles: the product by LDS tiles BM x BN, WVM x WVN waves of TM x TN tiles of
// v_mfma_f32_16x16x32_bf16, four stages of 64 columns deep.  Where tiles are fewer than
// compute units, loads in flight bound a unit: four stages of small tiles on many units
// instead of gemm_bf16.hip's 128 x 128 (M = 128, 4096 x 4096: the product 15 us).  Rows of
// 128 bytes go from global memory straight into LDS; chunk c (16 bytes) of row y
// sits at unit c ^ ((y >> 1) & 7); lane (g, n) takes row n's chunk 4 t + g in half t.  The
// fragments of the next half are read while this one's products run; at the end of
// half 0 every wave has read the stage and the next step has landed, and half 1 sends the
// step four ahead into it.
typedef __attribute__((address_space(3))) void lds_void;
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rs(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(lo | (hi << 32)), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
// past every buffer made here (128 rows of 2^20 bf16): such a load gives zero
constexpr uint32_t kPastBuffer = 0x7ffffff0u;
__device__ __forceinline__ void dma16(rsrc_t rs, uint32_t voff, uint32_t soff, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void barrier_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}

template <int WVM, int WVN, int TM, int TN>
struct TileGeo {
  static constexpr int WAVES = WVM * WVN, NST = 4;
  static constexpr int BM = 16 * TM * WVM, BN = 16 * TN * WVN;
  static constexpr int AB = BM * 128, STB = AB + BN * 128;          // bytes of A, of a stage
  static constexpr int OUTP = 32 * TN + 16, OUTW = 16 * TM * OUTP;  // output staging of a wave
  static constexpr int LDS = NST * STB;
  static constexpr int AL = BM / 8 / WAVES, BL = BN / 8 / WAVES;    // loads of a wave and step
  static_assert(WAVES * OUTW <= LDS && LDS <= 160 * 1024, "LDS");
};

template <int WVM, int WVN, int TM, int TN>
__global__ __launch_bounds__(64 * WVM * WVN) void k_gemm_tiles(
    const uint16_t* __restrict__ A, int64_t lda, int64_t R, const uint16_t* __restrict__ Bm,
    int64_t ldb, int64_t M, int64_t Nc, const float* __restrict__ V,
    const uint16_t* __restrict__ L, int r, float s, uint16_t* __restrict__ C,
    const uint8_t* __restrict__ mask, int tiles_m) {
  using G = TileGeo<WVM, WVN, TM, TN>;
  constexpr int BM = G::BM, BN = G::BN, NST = G::NST, AL = G::AL, BL = G::BL, LPS = AL + BL;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WVN, wn = wave % WVN;
  // neighbouring tiles on one XCD (a workgroup's is its index mod 8): Bm's rows come into
  // one second level cache only
  const int per = (int)gridDim.x / 8, more = (int)gridDim.x % 8, xcd = (int)blockIdx.x % 8;
  const int tile = xcd * per + min(xcd, more) + (int)blockIdx.x / 8;
  const int tn = tile / tiles_m, tm = tile - tn * tiles_m;
  const int64_t m0 = (int64_t)tm * BM, c0 = (int64_t)tn * BN;
  const int mrows = (int)min((int64_t)BM, M - m0), ncols = (int)min((int64_t)BN, Nc - c0);
  const int steps = (int)((R + 63) / 64);

  // load i of wave w: rows 8 (AL w + i) + l / 8 (past the matrix: its last row)
  const rsrc_t ra = make_rs(A + m0 * lda, (uint32_t)(mrows * lda * 2));
  const rsrc_t rb = make_rs(Bm + c0 * ldb, (uint32_t)(ncols * ldb * 2));
  uint32_t aoff[AL], alast[AL], boff[BL];
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    const int row = 8 * (AL * wave + i) + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
    aoff[i] = (uint32_t)((min(row, mrows - 1) * lda + 8 * chunk) * 2);
    // a chunk of the last step past R: past the buffer, which reads as zero, as its
    // partner in Bm is (the row's own values there would make an infinity of the row a NaN)
    alast[i] = (int64_t)(steps - 1) * 64 + 8 * chunk >= R ? kPastBuffer : aoff[i];
  }
#pragma unroll
  for (int i = 0; i < BL; ++i) {
    const int row = 8 * (BL * wave + i) + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
    boff[i] = (uint32_t)((min(row, ncols - 1) * ldb + 8 * chunk) * 2);
  }
  auto load_one = [&](int q, int st, int stage) {
    uint8_t* base = smem + stage * G::STB;
    const uint32_t so = (uint32_t)st * 128;
    if (q < AL)
      dma16(ra, st == steps - 1 ? alast[q] : aoff[q], so, base + 1024 * (AL * wave + q));
    else
      dma16(rb, boff[q - AL], so, base + G::AB + 1024 * (BL * wave + q - AL));
  };
  int roff[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) roff[t] = n * 128 + 16 * ((4 * t + g) ^ ((n >> 1) & 7));
  const int abase = wm * 16 * TM * 128, bbase = G::AB + wn * 16 * TN * 128;
  auto frag = [&](int stage, int base, int k, int t) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
                                          smem + stage * G::STB + base + k * 2048 + roff[t]));
  };
  f32x4 acc[TM][TN] = {};
  bf16x8 fa[TM], fb[2][TN];
#pragma unroll
  for (int k = 0; k < NST; ++k)
#pragma unroll
    for (int q = 0; q < LPS; ++q) load_one(q, min(k, steps - 1), k);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 1) * LPS) : "memory");
  barrier_lds();
#pragma unroll
  for (int i = 0; i < TM; ++i) fa[i] = frag(0, abase, i, 0);
#pragma unroll
  for (int j = 0; j < TN; ++j) fb[0][j] = frag(0, bbase, j, 0);

  auto half = [&](auto p_t, auto t_t, int st) {
    constexpr int P = decltype(p_t)::value, H = decltype(t_t)::value;
    constexpr int RS = H == 0 ? P : (P + 1) % NST, RH = H ^ 1, PER = (LPS + TM - 1) / TM;
    const int lst = min(st + NST, steps - 1);
    unrolled<TM>([&](auto i_t) {
      constexpr int i = decltype(i_t)::value;
      unrolled<TN>([&](auto j_t) {
        constexpr int j = decltype(j_t)::value;
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[H][j], fa[i], acc[i][j], 0, 0, 0);
        if (i == 0) fb[RH][j] = frag(RS, bbase, j, RH);
        if (H == 1 && j == TN / 2)
          for (int q = PER * i; q < PER * (i + 1); ++q)
            if (q < LPS) load_one(q, lst, P);
      });
      fa[i] = frag(RS, abase, i, RH);
      __builtin_amdgcn_sched_barrier(0);
    });
    if (H == 0) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * LPS) : "memory");
      barrier_lds();
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  int st = 0;
  for (; st + NST <= steps; st += NST)
    unrolled<NST>([&](auto p) {
      half(p, I0{}, st + (int)p);
      half(p, I1{}, st + (int)p);
    });
  unrolled<NST - 1>([&](auto p) {
    if (st < steps) {
      half(p, I0{}, st);
      half(p, I1{}, st++);
    }
  });
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  barrier_lds();

  // the adapter term, as in k_gemm_few, in accumulators of its own for the mask's sake
  f32x4 low[TM][TN] = {};
  for (int j0 = 0; j0 < r; j0 += 16) {
    const int jl = j0 + 8 * (g & 1);
    u32x4 lb[TN];
    f32x4 va[TM][2];
#pragma unroll
    for (int j = 0; j < TN; ++j)
      lb[j] = ranks(L + min(c0 + 16 * (TN * wn + j) + n, Nc - 1) * r, jl, r);
#pragma unroll
    for (int i = 0; i < TM; ++i) ranks(V + min(m0 + 16 * (TM * wm + i) + n, M - 1) * r, jl, r, va[i]);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const bf16x8 v = split(va[i], s, g >= 2);
#pragma unroll
      for (int j = 0; j < TN; ++j)
        low[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lb[j]), v,
                                                            low[i][j], 0, 0, 0);
    }
  }
  // lane: row n of tile (i, j), columns 4 g .. 4 g + 3; through the wave's LDS staging tile,
  // which leaves as rows of 32 TN bytes
  uint8_t* stg = smem + wave * G::OUTW;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = min(m0 + 16 * (TM * wm + i) + n, M - 1);
    uint32_t kb[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j)  // (Nc % 64 == 0 with a mask: a byte is half a tile's columns)
      kb[j] = !mask ? 15u
                    : mask[((row * Nc + min(c0 + 16 * (TN * wn + j), Nc - 16)) >> 3) + (g >> 1)] >>
                          (4 * (g & 1));
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      f32x4 c = acc[i][j];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((kb[j] >> q) & 1) c[q] += low[i][j][q];
      *reinterpret_cast<u32x2*>(stg + (16 * i + n) * G::OUTP + 2 * (16 * j + 4 * g)) =
          u32x2{pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
    }
  }
  // (a wave's LDS accesses execute in order)
  constexpr int LR = 2 * TN, RPS = 64 / LR;  // lanes of a row, rows a store
  const int lc = lane % LR;
  const int64_t col = c0 + 16 * TN * wn + 8 * lc, row0 = m0 + 16 * TM * wm;
#pragma unroll
  for (int q = 0; q < 16 * TM / RPS; ++q) {
    const int rl = RPS * q + lane / LR;
    const u32x4 v = *reinterpret_cast<const u32x4*>(stg + rl * G::OUTP + 16 * lc);
    if (row0 + rl < M && col < Nc) *reinterpret_cast<u32x4*>(C + (row0 + rl) * Nc + col) = v;
  }
}

template <int WVM, int WVN, int TM, int TN>
hipError_t launch_tiles(const uint16_t* A, int64_t lda, int64_t R, const uint16_t* Bm, int64_t ldb,
                        int64_t M, int64_t Nc, const float* V, const uint16_t* L, int r, float s,
                        uint16_t* C, const uint8_t* mask, hipStream_t st) {
  using G = TileGeo<WVM, WVN, TM, TN>;
  // (the attribute is the current device's)
  const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(k_gemm_tiles<WVM, WVN, TM, TN>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, G::LDS);
  if (attr != hipSuccess) return attr;
  const int64_t tm = (M + G::BM - 1) / G::BM, tn = (Nc + G::BN - 1) / G::BN;
  hipLaunchKernelGGL((k_gemm_tiles<WVM, WVN, TM, TN>), dim3((unsigned)(tm * tn)),
                     dim3(64 * G::WAVES), G::LDS, st, A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, mask,
                     (int)tm);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_few(const uint16_t* A, int64_t lda, int64_t R, const uint16_t* Bm, int64_t ldb,
                      int64_t M, int64_t Nc, const float* V, const uint16_t* L, int r, float s,
                      uint16_t* C, const uint8_t* mask, hipStream_t st) {
  const int64_t col_wgs = (Nc + 15) / 16, row_wgs = (M + 16 * MT - 1) / (16 * MT);
  hipLaunchKernelGGL(k_gemm_few<MT>, dim3((unsigned)(col_wgs * row_wgs)), dim3(64 * kWaves), 0, st, A,
                     lda, R, Bm, ldb, (int)M, Nc, V, L, r, s, C, mask, (int)col_wgs);
  return hipGetLastError();
}

}  // namespace

static int64_t compute_units() {
  static const int n = [] {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return 256;
    return cus > 0 ? cus : 256;
  }();
  return n;
}

hipError_t launch_gemm_any(const uint16_t* A, int64_t lda, int64_t R, const uint16_t* Bm,
                           int64_t ldb, int64_t M, int64_t Nc, const float* V, const uint16_t* L,
                           int r, float s, uint16_t* C, hipStream_t st, const uint8_t* mask) {
  if (M <= 0) return hipSuccess;
  if (r > 64 || (mask && Nc % 64 != 0) || R < 8 || R % 8 != 0 || ldb % 64 != 0 || R > ldb ||
      Nc % 8 != 0)
    return hipErrorInvalidValue;
  const int64_t cu = compute_units();
  const auto tiles = [&](int64_t tm, int64_t tn) { return (M + tm - 1) / tm * ((Nc + tn - 1) / tn); };
  // The smallest that still go one to a compute unit.  The reduction split over a
  // workgroup's waves against 64 x 64 tiles: M = 64, 1024 and 1024 4.8 and 6.7 us, M = 128,
  // 1024 and 4096 (two blocks of rows a workgroup) 13.7 and 14.2, M = 64, 2048 and 2048 8.4
  // and 9.2; with two workgroups a unit and more M = 128, 2048 and 2048 16.8, by four blocks
  // of rows 12.6, tiles 9.4.  Small tiles against gemm_bf16.hip's (the whole call): M = 128,
  // 4096 and 4096 37.4 and 48.2 us, M = 65, 10560 and 4768 64 and 88; 64 x 128 tiles M = 512,
  // 14336 and 4096 108 and 116, M = 126, 12896 and 12672 260 and 295; 128 x 128 tiles four
  // stages deep lose: M = 1024, 4096 and 4096 52.5 and 48.4.
  if (tiles(16, 16) <= cu) return launch_few<1>(A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, mask, st);
  if (tiles(32, 16) <= cu) return launch_few<2>(A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, mask, st);
  if (tiles(64, 64) <= cu)
    return launch_tiles<2, 2, 2, 2>(A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, mask, st);
  if (tiles(64, 128) <= cu)
    return launch_tiles<2, 2, 2, 4>(A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, mask, st);
  return launch_gemm_nt(A, lda, R, Bm, ldb, M, Nc, V, L, r, s, C, st, mask);
}

}  // namespace qn
