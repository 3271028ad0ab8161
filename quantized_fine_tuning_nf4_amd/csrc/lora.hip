// Rank-r adapter products of the QLoRA linear (page "QLoRA: NF4 storage,
// gradients and local integration", paragraph after the teaching listing):
//   u = X A^T and v = G B          -- "thin NT" products, reduction along a
//                                     row of both operands;
//   dB = s G^T u and dA = s v^T X  -- "thin TN" products, reduction over the
//                                     M rows, split in slices whose partial
//                                     sums are added in slice order.
// All use v_mfma_f32_16x16x32_bf16; fp32 operands (u, v) enter the MFMA as a
// bf16 high part plus a bf16 remainder, so they keep ~16 significant bits (or,
// in the backward from an 8-bit checkpoint, as three parts: all 24).
#include <algorithm>
#include <type_traits>

#include "qn_device.h"
#include "qn_internal.h"

namespace qn {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// 8 consecutive bf16 of a row at column p (zero past the row end P).
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t p, int64_t P) {
  if (p + 8 <= P) return *reinterpret_cast<const u32x4*>(row + p);
  uint32_t w[4];
  for (int h = 0; h < 4; ++h) {
    uint32_t lo = p + 2 * h < P ? row[p + 2 * h] : 0u;
    uint32_t hi = p + 2 * h + 1 < P ? row[p + 2 * h + 1] : 0u;
    w[h] = lo | (hi << 16);
  }
  return u32x4{w[0], w[1], w[2], w[3]};
}

// 8 bf16 values with the dropped ones zeroed: mb holds their 8 mask bits
// (the masks are bit-packed over the elements, bit e % 8 of byte e / 8 set:
// kept, so 8 elements starting at a multiple of 8 share one byte).
__device__ __forceinline__ u32x4 keep8(u32x4 v, uint32_t mb) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v[q] &= (((mb >> (2 * q)) & 1u) * 0xffffu) | (((mb >> (2 * q + 1)) & 1u) * 0xffff0000u);
  return v;
}

// The first workgroup of a launch zeroes clr.n words at clr.p (the arrival
// counters a later kernel of the same call counts on).
__device__ __forceinline__ void clear_words(const Clear& clr) {
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < clr.n; i += blockDim.x) clr.p[i] = 0u;
}

}  // namespace

// out[M, r] = Z[M, P] T[r, P]^T over column slice s.  Workgroup (mt, s):
// rows 64mt .. 64mt+63, wave w rows 16w .. +15, all columns of the slice.
// MFMA lane l holds row l%16 and the eight columns 8(l/16).. of each 32-wide
// step of both operands (rows of Z and of T are contiguous along the
// reduction).  U steps' loads are issued before their MFMAs.  Columns past
// the slice count as zero in both operands, and a lane whose chunk lies there
// loads the slice's first columns instead (P is a multiple of 8): past the row
// there may be the buffer's end, or, in a workspace, a NaN.  NJ = ceil(r/16).
template <int NJ>
__global__ __launch_bounds__(kThreads) void k_thin_nt(const uint16_t* __restrict__ Z,
                                                      const uint16_t* __restrict__ T, int64_t M,
                                                      int64_t P, int r, int64_t slice,
                                                      float* __restrict__ out, Clear clr,
                                                      const uint8_t* __restrict__ zmask) {
  constexpr int U = NJ <= 2 ? 8 : 4;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  clear_words(clr);
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t mw = (int64_t)blockIdx.x * 64 + 16 * wave;  // first row of the wave
  const int64_t m = min(mw + l16, M - 1);
  const int64_t pb = (int64_t)blockIdx.y * slice, pe = min(pb + slice, P);
  const int steps = (int)((pe - pb + 31) / 32);
  const uint16_t* zp = Z + m * P + pb + 8 * g;
  const uint16_t* tp[NJ];
#pragma unroll
  for (int jt = 0; jt < NJ; ++jt) tp[jt] = T + (int64_t)min(16 * jt + l16, r - 1) * P + pb + 8 * g;
  const int64_t lim = pe - pb - 8 * g;  // in-slice columns left for this lane's chunk
  f32x4 acc[NJ] = {};
  for (int s0 = 0; s0 < steps; s0 += U) {
    u32x4 za[U], tb[U][NJ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t off = 32 * (int64_t)(s0 + u);
      const bool ok = off < lim;
      const int64_t o = ok ? off : -8 * g;
      za[u] = *reinterpret_cast<const u32x4*>(zp + o);
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt) tb[u][jt] = *reinterpret_cast<const u32x4*>(tp[jt] + o);
      if (zmask) za[u] = keep8(za[u], zmask[(m * P + pb + 8 * g + o) >> 3]);
      if (!ok) za[u] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt) {
        u32x4 b = tb[u][jt];
        if (16 * jt + l16 >= r || 32 * (int64_t)(s0 + u) >= lim) b = u32x4{0u, 0u, 0u, 0u};
        acc[jt] = mfma16(as_bf16x8(za[u]), as_bf16x8(b), acc[jt]);
      }
  }
  // lane l: column j = 16jt + l%16, rows mw + 4(l/16) + i
  float* dst = out + (int64_t)blockIdx.y * M * r;
#pragma unroll
  for (int jt = 0; jt < NJ; ++jt) {
    const int j = 16 * jt + l16;
    if (j >= r) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = mw + 4 * g + i;
      if (row < M) dst[row * r + j] = acc[jt][i];
    }
  }
}

// v[M, r] = G[M, N] B[N, r] whole, and with it (s v)^T in three bf16 parts as
// the transposed product takes it (up to row Mp, zero past r and M).
// Workgroup: 16 RT rows; its eight waves take U steps of 32 columns in turn, with
// the operands as in k_thin_nt, and their sums meet in LDS, added in wave order.
// So v is never in slices: with k_thin_nt's column slices and a launch that adds and
// splits them the whole backward without dX takes 39.4 us for 4096x1024x4096 at
// r = 64 (29.7 here), 85 for 8192x4096x4096 at r = 64 (59), 51 at r = 8 (37).  Bound
// by the rows of G from HBM where r is small, else by B from the L2, which every
// workgroup reads whole: in the order of the operands a wave's load is 1 KB in a
// row.  From the rows of B^T (64 bytes of 16 rows a load) the three took 31.9, 79
// and 49 us; 32 rows a workgroup, half the bytes of B, 33.0 and 61, since twice
// the workgroups hide more of the latency.
constexpr int kVWaves = 8;
template <int NJ>
__global__ __launch_bounds__(64 * kVWaves) void k_thin_v(const uint16_t* __restrict__ G,
                                                         const uint16_t* __restrict__ Bf,
                                                         int64_t M, int64_t N, int r,
                                                         float* __restrict__ v,
                                                         uint16_t* __restrict__ sv, int64_t Mp,
                                                         float s, Clear clr) {
  constexpr int U = 4, PITCH = 16 + 4;
  __shared__ __attribute__((aligned(16))) float sums[kVWaves][16 * NJ][PITCH];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  clear_words(clr);
  const int64_t m0 = 16 * (int64_t)blockIdx.x;
  const int64_t steps = (N + 31) / 32;
  const uint16_t* gp = G + min(m0 + l16, M - 1) * N + 8 * g;
  const int64_t lim = N - 8 * g;  // columns left for this lane's chunk
  f32x4 acc[NJ] = {};
  for (int64_t s0 = U * wave; s0 < steps; s0 += U * kVWaves) {
    u32x4 za[U], tb[U][NJ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t off = 32 * (s0 + u);
      // past the row: its first columns
      za[u] = *reinterpret_cast<const u32x4*>(gp + (off < lim ? off : -8 * g));
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt)
        tb[u][jt] = *reinterpret_cast<const u32x4*>(
            Bf + ((min(s0 + u, steps - 1) * NJ + jt) * 64 + lane) * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool ok = 32 * (s0 + u) < lim;
      if (!ok) za[u] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt) {
        u32x4 b = tb[u][jt];
        if (!ok) b = u32x4{0u, 0u, 0u, 0u};
        acc[jt] = mfma16(as_bf16x8(za[u]), as_bf16x8(b), acc[jt]);
      }
    }
  }
  // lane: column j = 16jt + l%16, rows 4(l/16) + i
#pragma unroll
  for (int jt = 0; jt < NJ; ++jt)
    *reinterpret_cast<f32x4*>(&sums[wave][16 * jt + l16][4 * g]) = acc[jt];
  __syncthreads();
  // four rows of one column a thread
  if (tid < 64 * NJ) {
    const int j = tid >> 2, q = tid & 3;
    f32x4 x = *reinterpret_cast<const f32x4*>(&sums[0][j][4 * q]);
#pragma unroll
    for (int w = 1; w < kVWaves; ++w) x += *reinterpret_cast<const f32x4*>(&sums[w][j][4 * q]);
    const int64_t m = m0 + 4 * q;
    u32x2 part[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = j < r && m + i < M;
      if (in) v[(m + i) * r + j] = x[i];
      float rest = in ? s * x[i] : 0.f;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t h = pack_bf16x2(rest, 0.f) & 0xffffu;
        part[k][i >> 1] = i & 1 ? part[k][i >> 1] | (h << 16) : h;
        rest -= bf16_lo(h);
      }
    }
    if (m < Mp)
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<u32x2*>(sv + (((m >> 5) * 3 + k) * 16 * NJ + j) * 32 + (m & 31)) =
            part[k];
  }
}

hipError_t launch_thin_v(const uint16_t* G, const uint16_t* Bf, int64_t M, int64_t N, int r,
                         float* v, uint16_t* sv, int64_t Mp, float s, hipStream_t st, Clear clr) {
#define QN_V(NJ)                                                                              \
  hipLaunchKernelGGL(k_thin_v<NJ>, dim3((unsigned)((Mp + 15) / 16)), dim3(64 * kVWaves), 0, st, G, \
                     Bf, M, N, r, v, sv, Mp, s, clr)
  switch ((r + 15) / 16) {
    case 1: QN_V(1); break;
    case 2: QN_V(2); break;
    case 3: QN_V(3); break;
    default: QN_V(4); break;
  }
#undef QN_V
  return hipGetLastError();
}

// r <= 16: the same product with T's slice (rows 0..15, zero past r)
// staged in LDS once per workgroup (row pitch 64 steps + 16 bytes, so the
// 16-byte reads of 8 consecutive rows fall in distinct bank groups), and Z
// streamed through registers two batches of TN1_U steps deep: the loads of
// batch b + 1 are in flight while batch b is multiplied.  Columns past the
// slice read as zero (selected at use, so no load waits at a branch).
constexpr int TN1_U = 4;
constexpr int64_t kThinNt1MaxSlice = 2048;
template <int TMODE>
__global__ __launch_bounds__(kThreads) void k_thin_nt1(const uint16_t* __restrict__ Z,
                                                       const uint16_t* __restrict__ T, int64_t M,
                                                       int64_t P, int r, int64_t slice,
                                                       float* __restrict__ out, Clear clr,
                                                       const uint8_t* __restrict__ zmask) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  clear_words(clr);
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t mw = (int64_t)blockIdx.x * 64 + 16 * wave;
  const int64_t m = min(mw + l16, M - 1);
  const int64_t pb = (int64_t)blockIdx.y * slice, pe = min(pb + slice, P);
  const int64_t width = pe - pb;
  const int steps = (int)((width + 31) / 32);
  const int nb = (steps + TN1_U - 1) / TN1_U;
  const int pitch = steps * 64 + 16;
  const uint16_t* zp = Z + m * P + pb + 8 * g;
  const int64_t lim = width - 8 * g;  // in-slice columns left for this lane's chunk
  u32x4 za[2][TN1_U];
  // the batch's mask bytes (dropout on Z), loaded beside it: row m's 16
  // bytes for the batch's 128 columns as two 8-byte halves (two steps each;
  // P % 64 == 0 and the slice starts on 128 columns, so each half is aligned
  // and lies in the row when its first column is in the slice; a half past
  // the slice reads the slice's first one instead, for steps zeroed at use)
  static_assert(TN1_U == 4, "two steps per 8-byte half of a batch's mask bytes");
  uint2 zk[2][2];
  auto load_batch = [&](int buf, int b) {
#pragma unroll
    for (int u = 0; u < TN1_U; ++u) {
      const int64_t off = 32 * (int64_t)(TN1_U * b + u);
      // (past the slice: its first columns, never past the row)
      za[buf][u] = *reinterpret_cast<const u32x4*>(zp + (off < lim ? off : -8 * g));
    }
    if (zmask) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = 128 * (int64_t)b + 64 * h;
        zk[buf][h] = *reinterpret_cast<const uint2*>(zmask + ((m * P + pb + (c < width ? c : 0)) >> 3));
      }
    }
  };
  if constexpr (TMODE == 0) {
    // stage T: eight 16-byte chunks per thread per pass, every load issued
    // before the first is used (clamped addresses; zero selected at the LDS
    // write for rows past r and columns past the slice); the first Z batch
    // goes out behind the first pass
    const int cpr = steps * 4;  // 16-byte chunks per staged row
    const int total = 16 * cpr;
    for (int e0 = 0; e0 < total; e0 += 8 * kThreads) {
      u32x4 tv[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int e = min(e0 + q * kThreads + tid, total - 1);
        const int j = e / cpr, c = e - j * cpr;
        const int64_t col = min(8 * (int64_t)c, width - 8);
        tv[q] = *reinterpret_cast<const u32x4*>(T + (int64_t)min(j, r - 1) * P + pb + col);
      }
      if (e0 == 0) load_batch(0, 0);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int e = e0 + q * kThreads + tid;
        if (e < total) {
          const int j = e / cpr, c = e - j * cpr;
          const bool ok = j < r && 8 * (int64_t)c < width;
          *reinterpret_cast<u32x4*>(smem + j * pitch + 16 * c) = ok ? tv[q] : u32x4{0u, 0u, 0u, 0u};
        }
      }
    }
  } else {
    // stage T given as its transpose Tr [P, r] (the adapter B as stored): a
    // thread takes a pair of columns (two rows of Tr, r <= 16 values each),
    // loads them (unconditional, clamped), sends the first Z batch, then
    // writes one word per rank (the pair's two values) to LDS; zero for
    // ranks >= r and columns past the slice
    const int pairs = steps * 16;
    for (int p0 = 0; p0 < pairs; p0 += 4 * kThreads) {
      uint32_t v[4][16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int pp = min(p0 + k * kThreads + tid, pairs - 1);
        const int64_t c0 = min(pb + 2 * (int64_t)pp, P - 1), c1 = min(c0 + 1, P - 1);
        if constexpr (TMODE == 1) {
          const u32x4* s0 = reinterpret_cast<const u32x4*>(T + c0 * 16);
          const u32x4* s1 = reinterpret_cast<const u32x4*>(T + c1 * 16);
          const u32x4 a0 = s0[0], a1 = s0[1], b0 = s1[0], b1 = s1[1];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[k][2 * q] = (a0[q] & 0xffffu) | (b0[q] << 16);
            v[k][2 * q + 1] = (a0[q] >> 16) | (b0[q] & 0xffff0000u);
            v[k][8 + 2 * q] = (a1[q] & 0xffffu) | (b1[q] << 16);
            v[k][8 + 2 * q + 1] = (a1[q] >> 16) | (b1[q] & 0xffff0000u);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int jj = min(j, r - 1);
            v[k][j] = (uint32_t)T[c0 * r + jj] | ((uint32_t)T[c1 * r + jj] << 16);
          }
        }
      }
      if (p0 == 0) load_batch(0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int pp = p0 + k * kThreads + tid;
        if (pp < pairs) {
          const int64_t col = 2 * (int64_t)pp;
          const uint32_t keep = (col < width ? 0xffffu : 0u) | (col + 1 < width ? 0xffff0000u : 0u);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            *reinterpret_cast<uint32_t*>(smem + j * pitch + 4 * pp) = j < r ? (v[k][j] & keep) : 0u;
        }
      }
    }
  }
  // LDS-only barrier: the first Z batch stays in flight
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const uint8_t* trow = smem + l16 * pitch + 16 * g;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto compute_batch = [&](int buf, int b) {
#pragma unroll
    for (int u = 0; u < TN1_U; ++u) {
      const int st = TN1_U * b + u;
      if (st < steps) {
        u32x4 z = 32 * (int64_t)st < lim ? za[buf][u] : u32x4{0u, 0u, 0u, 0u};
        if (zmask) {  // byte g of the step's four: this lane's eight columns
          const uint32_t w = (u & 1) ? zk[buf][u >> 1].y : zk[buf][u >> 1].x;
          z = keep8(z, (w >> (8 * g)) & 0xffu);
        }
        const u32x4 t = *reinterpret_cast<const u32x4*>(trow + 64 * st);
        acc = mfma16(as_bf16x8(z), as_bf16x8(t), acc);
      }
    }
  };
  for (int b = 0; b < nb; b += 2) {
    if (b + 1 < nb) load_batch(1, b + 1);
    compute_batch(0, b);
    if (b + 1 < nb) {
      if (b + 2 < nb) load_batch(0, b + 2);
      compute_batch(1, b + 1);
    }
  }
  // lane l: column j = l%16, rows mw + 4(l/16) + i
  float* dst = out + (int64_t)blockIdx.y * M * r;
  if (l16 < r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = mw + 4 * g + i;
      if (row < M) dst[row * r + l16] = acc[i];
    }
  }
}

// out[i] = sum over s of part[s][i], added in slice order.
__global__ void k_sum_slices(const float* __restrict__ part, int64_t count, int S,
                             float* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < count) out[i] = slice_sum(part, count, S, i);
}

// Column slice of launch_thin_nt (a multiple of 128).
int64_t thin_nt_slice(int64_t P, int S) {
  const int64_t slice = (P + S - 1) / S;
  return (slice + 127) / 128 * 128;
}

// Whether launch_thin_nt takes T as its transpose [P, r] for this shape.
bool thin_nt_rows_ok(int64_t M, int64_t P, int r) {
  return r <= 16 && thin_nt_slice(P, thin_nt_slices(M, P)) <= kThinNt1MaxSlice;
}

// Column slices (multiples of 128 columns) so that about 512 workgroups run.
int thin_nt_slices(int64_t M, int64_t P) {
  const int64_t mt = M > 0 ? (M + 63) / 64 : 1;
  int64_t S = (512 + mt - 1) / mt;
  const int64_t smax = (P + 127) / 128;
  if (S > smax) S = smax;
  if (S < 1) S = 1;
  return (int)S;
}

hipError_t launch_thin_nt(const uint16_t* Z, const uint16_t* T, int64_t M, int64_t P, int r,
                          float* out, float* part, int S, hipStream_t st, bool sum, bool t_rows,
                          Clear clr, const uint8_t* zmask) {
  const int64_t slice = thin_nt_slice(P, S);
  const dim3 grid((unsigned)((M + 63) / 64), (unsigned)S);
  float* dst = S > 1 ? part : out;
  if (r <= 16 && slice <= kThinNt1MaxSlice) {
    const int mode = !t_rows ? 0 : r == 16 ? 1 : 2;
    static const hipError_t attr[3] = {
        hipFuncSetAttribute(reinterpret_cast<const void*>(k_thin_nt1<0>),
                            hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)(16 * (kThinNt1MaxSlice * 2 + 16))),
        hipFuncSetAttribute(reinterpret_cast<const void*>(k_thin_nt1<1>),
                            hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)(16 * (kThinNt1MaxSlice * 2 + 16))),
        hipFuncSetAttribute(reinterpret_cast<const void*>(k_thin_nt1<2>),
                            hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)(16 * (kThinNt1MaxSlice * 2 + 16)))};
    if (attr[mode] != hipSuccess) return attr[mode];
    const int steps = (int)((slice + 31) / 32);
    const size_t lds = (size_t)16 * (steps * 64 + 16);
    if (mode == 0)
      hipLaunchKernelGGL(k_thin_nt1<0>, grid, dim3(kThreads), lds, st, Z, T, M, P, r, slice, dst, clr, zmask);
    else if (mode == 1)
      hipLaunchKernelGGL(k_thin_nt1<1>, grid, dim3(kThreads), lds, st, Z, T, M, P, r, slice, dst, clr, zmask);
    else
      hipLaunchKernelGGL(k_thin_nt1<2>, grid, dim3(kThreads), lds, st, Z, T, M, P, r, slice, dst, clr, zmask);
  } else {
    if (t_rows) return hipErrorInvalidValue;  // the general kernel takes T as [r, P]
  switch ((r + 15) / 16) {
    case 1: hipLaunchKernelGGL(k_thin_nt<1>, grid, dim3(kThreads), 0, st, Z, T, M, P, r, slice, dst, clr, zmask); break;
    case 2: hipLaunchKernelGGL(k_thin_nt<2>, grid, dim3(kThreads), 0, st, Z, T, M, P, r, slice, dst, clr, zmask); break;
    case 3: hipLaunchKernelGGL(k_thin_nt<3>, grid, dim3(kThreads), 0, st, Z, T, M, P, r, slice, dst, clr, zmask); break;
    default: hipLaunchKernelGGL(k_thin_nt<4>, grid, dim3(kThreads), 0, st, Z, T, M, P, r, slice, dst, clr, zmask); break;
  }
  }
  if (S > 1 && sum) {
    const int64_t count = M * r;
    hipLaunchKernelGGL(k_sum_slices, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, st,
                       part, count, S, out);
  }
  return hipGetLastError();
}

__global__ void k_fill_zero(float* __restrict__ p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t st) {
  if (n <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_fill_zero, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p, n);
  return hipGetLastError();
}

__global__ void k_bwd_aux(BwdAux a) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < bwd_aux_count(a)) bwd_aux_at(a, i);
}

hipError_t launch_bwd_aux(const BwdAux& a, hipStream_t st) {
  const int64_t count = bwd_aux_count(a);
  if (count == 0) return hipSuccess;
  hipLaunchKernelGGL(k_bwd_aux, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}

namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef short v4s __attribute__((ext_vector_type(4)));

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

constexpr int TN_COLS = 128;             // columns of Z per workgroup
constexpr int TN_ROWB = TN_COLS * 2;     // 256 B per staged Z row
// Stages (two steps in flight; three: 1.5 us slower per backward, and 46 us
// against 39 for 4096x1024x4096 at r = 64 from an 8-bit checkpoint, whose LDS then
// holds one workgroup a CU).
constexpr int TN_NST = 3;

}  // namespace

// part[z][p][j] = sum over the rows m of slice z of Z[m, p] * (s V)[m, j]
// (a transposed product: the reduction runs down the columns of Z).  Two
// independent products (dB and dA of one backward) share the launch (the order
// of their workgroups: tn_per_xcd).  Workgroup (pt, z): columns 128 pt .. +127,
// wave w: 32w .. 32w+31 (two 16-column MFMA tiles).  A step is 32 rows: their
// Z (8 KB) and their (s V)^T parts (SP x 16 NJ rows of 64 B) go global -> LDS by
// 16-byte-per-lane buffer loads into one stage, three stages deep.  A 16-byte unit
// c of (s V)^T row y sits at c ^ ((y >> 2) & 3), so that the 16 lanes that read one
// unit of 16 rows touch 256 different bytes.
// Z row y's 16-byte chunk c sits at unit c ^ 2(y & 3); the A operand (16
// columns x 32 rows) is read transposed with ds_read_b64_tr_b16, lane t of a
// 16-lane group addressing row 4h + t/4, columns 4(t%4)..+3, so that lane t
// receives column t, four consecutive rows.  NJ = ceil(r/16); SP: the parts of
// (s V)^T.
struct TnJob {
  const uint16_t* Z;   // [M, P] bf16 ...
  const int8_t* codes; // ... or an 8-bit checkpoint of it: codes [M, P]
  const uint8_t* exps; // and exponents [M, ceil(P / 64)]
  const uint16_t* vt;  // (s V)^T in parts, 32 rows [SP][16 NJ][32] after another
  int64_t P;
  int64_t slice;       // rows per slice, a multiple of 32
  int S;               // slices
  int tiles;           // column tiles of 128
  float* part;         // [S, P, r]
  float* out;          // [P, r], or [r, P] when transposed
  int transposed;
  const uint8_t* zmask;  // keep bits of Z (dropout on x), or null
};

// With an 8-bit checkpoint (one-dimensional grid): workgroups of a job per XCD.
// The XCDs take workgroups round robin; each takes a run of each job's
// workgroups, ordered slice by slice, so that an XCD's L2 holds the (s V)^T of its
// own slices alone (an eighth of it) rather than all of it, and every XCD has the
// same share of both jobs (8192x4096x4096, r = 16 with dropout: 47.2 -> 42.9 us;
// 4096x1024x4096, r = 64: 40.6 -> 39.4).  With bf16 rows, whose slices are added
// by the tiles' last workgroups, that order is slower (r = 64: 48.2 -> 51.4): there
// grid x runs over the column tiles of job 0, then job 1's, and y over the slices.
__host__ __device__ inline int tn_per_xcd(const TnJob& j) { return (j.tiles * j.S + 7) / 8; }

// Arrival counters of the column tiles of one launch (both jobs' tiles in
// grid order) sit in the caller's workspace: zero when the launch starts,
// left at zero by the workgroup that finishes a tile.
constexpr int kTnMaxTiles = kArrivalWords;
constexpr int kDeviceScope = 16;  // sc1: the level every XCD shares

// With arrivals != null the slices are also added here: each workgroup
// stores its slice with device-coherent stores, and the last of a column
// tile's S workgroups to arrive (an arrival counter per tile) adds the S
// slices of the tile in slice order with device-coherent loads and writes
// the output.
// vmcnt wait for the given count (an immediate of the instruction).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 3 && N <= 63, "counts of k_thin_tn's steps");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// MASK: a job may carry keep bits of Z (dropout on the adapter branch's
// input, for dA): the step's 32 rows x 16 bytes of bits go global -> LDS
// beside Z (one 4-byte-per-lane load in waves 0 and 1: rows 16w .. 16w+15;
// the direct-to-LDS path writes one dword per lane), word by word, so that a
// lane's eight rows of its wave's word are 32 bytes in a row, and the dropped
// values are zeroed in the A operand after the transposed reads.
//
// Z8: the second job's Z is an 8-bit checkpoint.  Its 32 rows of 128 codes are
// half the bytes of bf16 rows: one 16-byte-per-lane load per wave (8 rows each;
// row y's 16-byte chunk c at unit c ^ ((y >> 1) & 7), so that the 16 rows of a
// transposed read fill 256 bytes of banks), read as columns by
// ds_read_b64_tr_b8 (lane t of a 16-lane group addresses row t / 2, columns
// 8 (t % 2) .. + 7 and receives column t, eight rows: a lane's whole part of the
// A operand).  A lane loads one of its group's eight rows' exponents into a
// register, two steps ahead; the rows' scales reach the 16 lanes by DPP, and
// code times scale is a bf16 number exactly, so the MFMA sees the checkpoint's
// values.
// f(0), f(1), .. f(N - 1), each with its index as a constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}
template <int Q>
__device__ __forceinline__ float row_scale(float scale) {
  return as_f32(dpp<0x150 + Q>(as_u32(scale)));  // row_newbcast: lane Q of each 16
}
template <int NJ, bool MASK, int SP, bool Z8>
__global__ __launch_bounds__(kThreads) void k_thin_tn(TnJob j0, TnJob j1, int64_t M, int r,
                                                      unsigned* __restrict__ arrivals) {
  constexpr int ZB = 32 * TN_ROWB;             // Z bytes per stage
  constexpr int VB = SP * 16 * NJ * 64;        // (sV)^T bytes per stage
  constexpr int KB = MASK ? 32 * 16 : 0;       // keep bits per stage
  constexpr int SB = ZB + VB + KB;
  constexpr int NST = TN_NST;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  // this workgroup's job, column tile and slice
  bool second;
  int pt_wg, z_wg;
  if constexpr (Z8) {
    const int xcd = (int)blockIdx.x & 7, n0 = tn_per_xcd(j0), ci = (int)blockIdx.x >> 3;
    second = ci >= n0;
    const int wi = second ? xcd * tn_per_xcd(j1) + ci - n0 : xcd * n0 + ci;
    const int tiles = second ? j1.tiles : j0.tiles;
    pt_wg = wi % tiles;
    z_wg = wi / tiles;
  } else {
    second = (int)blockIdx.x >= j0.tiles;
    pt_wg = (int)blockIdx.x - (second ? j0.tiles : 0);
    z_wg = (int)blockIdx.y;
  }
  const uint16_t* Z = second ? j1.Z : j0.Z;
  const uint16_t* vt = second ? j1.vt : j0.vt;
  const int64_t P = second ? j1.P : j0.P;
  const int64_t slice = second ? j1.slice : j0.slice;
  const int S = second ? j1.S : j0.S;
  float* part = second ? j1.part : j0.part;
  const uint8_t* zmask = MASK ? (second ? j1.zmask : j0.zmask) : nullptr;
  const bool hm = MASK && zmask != nullptr;  // workgroup-uniform
  const bool z8 = Z8 && second;              // workgroup-uniform
  if (z_wg >= S) return;  // past the job's workgroups
  const int64_t p0 = (int64_t)pt_wg * TN_COLS;
  const int64_t mb = (int64_t)z_wg * slice;
  const int64_t me = min(mb + slice, M);
  const int steps = (int)((me - mb + 31) / 32);

  // ---- Z loads: instruction i (0..7) of a step covers rows 4i..4i+3; wave w
  // issues i = 2w, 2w+1; lane l -> row 4i + l/16, unit l%16, source chunk
  // (l%16) ^ 2(row & 3).  Rows past M repeat row M-1 (their sV is zero);
  // columns past P repeat the last chunk (their outputs are not stored).
  // (sV)^T loads: 16 of its 64-byte rows per instruction (lane l: row 16q + l/4,
  // bytes 16 (l%4)), instruction q = VL w + k of the step; where SP NJ is no
  // multiple of four, the last waves load the last rows again (the same bytes
  // to the same place), so that every wave counts the same loads.
  // descriptors start at the slice's first row, so that only one slice's
  // bytes (below 2^31, thin_tn_slice_rows) are ever addressed by an offset
  const rsrc_t rz = make_rs(z8 ? reinterpret_cast<const void*>(j1.codes + mb * P)
                               : reinterpret_cast<const void*>(Z + mb * P),
                            (uint32_t)((me - mb) * P * (z8 ? 1 : 2)));
  const rsrc_t rv = make_rs(vt + SP * 16 * NJ * mb, (uint32_t)(slice * SP * 16 * NJ * 2));
  // keep bits from the slice's first row (P % 64 == 0: rows start on a byte);
  // bytes past the slice read as zero (columns past P are not stored)
  const rsrc_t rk = make_rs(hm ? zmask + mb * P / 8 : reinterpret_cast<const uint8_t*>(vt),
                            hm ? (uint32_t)((me - mb) * P / 8) : 0u);
  // the checkpoint's exponents from the slice's first row, this wave's block of
  // columns
  const int64_t nb = (P + kAct8Block - 1) / kAct8Block;
  const rsrc_t re = make_rs(z8 ? j1.exps + mb * nb : reinterpret_cast<const uint8_t*>(vt),
                            z8 ? (uint32_t)((me - mb) * nb) : 0u);
  const uint32_t eoff = (uint32_t)min((p0 + 32 * wave) / kAct8Block, nb - 1);
  uint32_t zoff[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 2 * wave + h, row = 4 * i + (lane >> 4);
    const int chunk = (lane & 15) ^ (2 * (row & 3));
    const int64_t col = min(p0 + 8 * chunk, P - 8);
    zoff[h] = (uint32_t)(col * 2);
  }
  constexpr int VL = (SP * NJ + 3) / 4;
  uint32_t voff[VL];
  int vdst[VL];
#pragma unroll
  for (int k = 0; k < VL; ++k) {
    const int q = min(VL * wave + k, SP * NJ - 1), row = 16 * q + (lane >> 2);
    voff[k] = (uint32_t)(row * 64 + 16 * ((lane & 3) ^ (lane >> 4)));
    vdst[k] = ZB + 1024 * q;
  }
  // the steps, on codes or on bf16
  const int g = lane >> 4, t = lane & 15;
  f32x4 acc[2][NJ] = {};
  auto run = [&](auto q8_t) {
    constexpr bool Q8 = decltype(q8_t)::value;
    uint32_t ex[NST] = {};  // per stage: the exponent of row 8 (l / 16) + l % 8
    auto load_step = [&](int st, auto stage_t) {
      constexpr int stage = decltype(stage_t)::value;
      uint8_t* base = smem + stage * SB;
      if constexpr (Q8) {  // row 8w + l/8, unit l%8
        const int row = 8 * wave + (lane >> 3);
        const int chunk = (lane & 7) ^ ((row >> 1) & 7);
        const int64_t mm = min(mb + 32 * (int64_t)st + row, M - 1);
        dma16(rz, (uint32_t)((mm - mb) * P + min(p0 + 16 * chunk, P - 16)), 0, base + 1024 * wave);
        const int64_t me8 = min(mb + 32 * (int64_t)st + 8 * (lane >> 4) + (lane & 7), M - 1);
        ex[stage] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
            re, (uint32_t)((me8 - mb) * nb) + eoff, 0, 0);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 2 * wave + h, row = 4 * i + (lane >> 4);
          const int64_t mm = min(mb + 32 * (int64_t)st + row, M - 1);
          dma16(rz, zoff[h] + (uint32_t)((mm - mb) * P * 2), 0, base + 1024 * i);
        }
      }
#pragma unroll
      for (int k = 0; k < VL; ++k)
        dma16(rv, voff[k] + (uint32_t)(VB * st), 0, base + vdst[k]);
      if constexpr (MASK) {
        if (hm && wave < 2) {  // lane l: row 16w + l%16, bytes 4(l/16) .. +3 of the tile's 16
          const int row = 16 * wave + (lane & 15);
          const int64_t mm = min(mb + 32 * (int64_t)st + row, M - 1);
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              rk, (lds_void*)(base + ZB + VB + 256 * wave), 4,
              (uint32_t)((((mm - mb) * P + p0) >> 3) + 4 * (lane >> 4)), 0, 0, 0);
        }
      }
    };
    // all but the newest step's loads (2 + VL per wave: Z or the codes and
    // their exponents, then (sV)^T) have landed (one more in waves 0 and 1 when
    // the keep bits come along)
    auto wait_step = [&]() {
      if (MASK && hm && wave < 2)
        wait_vm<(NST - 2) * (2 + VL + (MASK ? 1 : 0))>();
      else
        wait_vm<(NST - 2) * (2 + VL)>();
    };
    unrolled<NST - 1>([&](auto i) { load_step(min((int)i, steps - 1), i); });
    wait_step();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

    // transposed-read addresses: lane l, group g = l/16, t = l%16; p-tile pt,
    // half h: row 8g + 4h + t/4, column 32w + 16pt + 4(t%4)
    int aoff[2][2];
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 8 * g + 4 * h + (t >> 2);
        const int col = 32 * wave + 16 * pt + 4 * (t & 3);
        aoff[pt][h] = row * TN_ROWB + 16 * ((col >> 3) ^ (2 * (row & 3))) + 2 * (col & 7);
      }
    // the same for codes: p-tile pt, row 8g + t/2, columns 32w + 16pt + 8(t%2)
    int aoff8[2];
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) {
      const int row = 8 * g + (t >> 1);
      aoff8[pt] = row * TN_COLS + 16 * ((2 * wave + pt) ^ ((row >> 1) & 7)) + 8 * (t & 1);
    }
    // one step on stage P (a constant, so that the compiler sees the loads of
    // the newest step and this step's LDS reads touch different stages)
    auto body = [&](auto p_t, int st) {
      constexpr int P = decltype(p_t)::value;
      load_step(min(st + NST - 1, steps - 1),
                std::integral_constant<int, (P + NST - 1) % NST>{});
      const uint8_t* zs = smem + P * SB;
      // the four transposed reads in one block that also waits for them (the
      // compiler would otherwise treat them as possibly overlapping the loads
      // in flight to the other stages and wait for all of those first)
      const uint32_t zb = (uint32_t)reinterpret_cast<uintptr_t>(zs);
      u32x4 za[2];
      if constexpr (Q8) {
        u32x2 c[2];
        asm volatile(
            "ds_read_b64_tr_b8 %0, %2\n\t"
            "ds_read_b64_tr_b8 %1, %3\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(c[0]), "=&v"(c[1])
            : "v"(zb + aoff8[0]), "v"(zb + aoff8[1])
            : "memory");
        const float scale = act8_scale(ex[P]);
        const float rs[8] = {row_scale<0>(scale), row_scale<1>(scale), row_scale<2>(scale),
                             row_scale<3>(scale), row_scale<4>(scale), row_scale<5>(scale),
                             row_scale<6>(scale), row_scale<7>(scale)};
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w = c[pt][i >> 1] >> (16 * (i & 1));
            za[pt][i] = pack_bf16x2((float)(int8_t)w * rs[2 * i],
                                    (float)(int8_t)(w >> 8) * rs[2 * i + 1]);
          }
      } else {
        u32x2 x00, x01, x10, x11;
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4\n\t"
            "ds_read_b64_tr_b16 %1, %5\n\t"
            "ds_read_b64_tr_b16 %2, %6\n\t"
            "ds_read_b64_tr_b16 %3, %7\n\t"
            "s_waitcnt lgkmcnt(0)"
            // early-clobber: a result must not share a register with an address
            // that a later read of the block still has to issue with
            : "=&v"(x00), "=&v"(x01), "=&v"(x10), "=&v"(x11)
            : "v"(zb + aoff[0][0]), "v"(zb + aoff[0][1]), "v"(zb + aoff[1][0]), "v"(zb + aoff[1][1])
            : "memory");
        za[0] = u32x4{x00[0], x00[1], x01[0], x01[1]};
        za[1] = u32x4{x10[0], x10[1], x11[0], x11[1]};
      }
      if constexpr (MASK) {
        if (hm) {
          // word i of za[pt] holds rows 8g + 2i, 8g + 2i + 1 of column
          // 32w + 16pt + t, whose keep bits are bit 16pt + t of this wave's
          // words of the two rows
          const u32x4* ks = reinterpret_cast<const u32x4*>(zs + ZB + VB + 256 * (g >> 1) +
                                                           64 * wave + 32 * (g & 1));
          const u32x4 kw[2] = {ks[0], ks[1]};
#pragma unroll
          for (int pt = 0; pt < 2; ++pt) {
            const int sh = 16 * pt + t;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // a bit as all ones or zeros, in each half
              const uint32_t lo = (uint32_t)__builtin_amdgcn_sbfe(kw[i >> 1][2 * (i & 1)], sh, 1);
              const uint32_t hi =
                  (uint32_t)__builtin_amdgcn_sbfe(kw[i >> 1][2 * (i & 1) + 1], sh, 1);
              za[pt][i] &= __builtin_amdgcn_perm(hi, lo, 0x05040100u);
            }
          }
        }
      }
      bf16x8 a[2];
      a[0] = as_bf16x8(za[0]);
      a[1] = as_bf16x8(za[1]);
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt) {
        // B operand: column j = 16jt + l%16, rows 8g..8g+7 of the step
        const uint8_t* vs = zs + ZB + (16 * jt + t) * 64 + 16 * (g ^ (t >> 2));
        bf16x8 b[SP];
#pragma unroll
        for (int q = 0; q < SP; ++q)
          b[q] = as_bf16x8(*reinterpret_cast<const u32x4*>(vs + q * 16 * NJ * 64));
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int q = 0; q < SP; ++q) acc[pt][jt] = mfma16(a[pt], b[q], acc[pt][jt]);
      }
      // step st+1's loads (issued NST - 1 steps ago) have landed everywhere before
      // anyone reads them or overwrites this stage
      wait_step();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    int st = 0;
    for (; st + NST <= steps; st += NST) unrolled<NST>([&](auto i) { body(i, st + (int)i); });
    unrolled<NST - 1>([&](auto i) {
      if (st + (int)i < steps) body(i, st + (int)i);
    });
  };
  if constexpr (Z8) {
    if (z8)
      run(std::true_type{});
    else
      run(std::false_type{});
  } else {
    run(std::false_type{});
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  // lane: column j = 16jt + l%16, rows p = 16pt + 4(l/16) + i of the wave
  const int S_ = S;
  // (all slices, below 2^32 bytes, where this launch adds them, else this one alone)
  const rsrc_t rp = make_rs(arrivals ? part : part + (int64_t)z_wg * P * r,
                            (uint32_t)((int64_t)(arrivals ? S_ : 1) * P * r * 4));
  const int64_t sl_off = arrivals ? (int64_t)z_wg * P * r : 0;
#pragma unroll
  for (int jt = 0; jt < NJ; ++jt) {
    const int j = 16 * jt + t;
    if (j >= r) continue;
    if (Z8 && !arrivals && (second ? j1.transposed : j0.transposed)) {
      // as the output lies: four columns of one rank
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) {
        const int64_t p = p0 + 32 * wave + 16 * pt + 4 * g;
        if (p < P)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[pt][jt]), rp,
                                                 (uint32_t)((sl_off + j * P + p) * 4), 0, 0);
      }
      continue;
    }
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t p = p0 + 32 * wave + 16 * pt + 4 * g + i;
        if (p < P)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[pt][jt][i]), rp,
                                                (uint32_t)((sl_off + p * r + j) * 4), 0,
                                                kDeviceScope);
      }
  }
  if (!arrivals) return;
  // ---- arrival: every wave's stores have completed before the barrier, so
  // they precede the count; the last workgroup reads them after it
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  __shared__ int s_last;
  unsigned* ctr = arrivals + (second ? j0.tiles : 0) + pt_wg;
  if (tid == 0)
    s_last = __hip_atomic_fetch_add(ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             (unsigned)(S_ - 1);
  __syncthreads();
  if (!s_last) return;
  // ---- the tile's columns p0 .. p0 + np - 1: slice z holds them as np r
  // contiguous floats at (z P + p0) r; elements e, in chunks of 2048 (eight
  // per thread, every load of a chunk issued before the first add)
  const int np = (int)min((int64_t)TN_COLS, P - p0);
  const int cnt = np * r;
  const bool tr = second ? j1.transposed : j0.transposed;
  float* out = second ? j1.out : j0.out;
  const bool vec = (r % 4) == 0 && (P * r) % 4 == 0;
  const uint32_t zst = (uint32_t)((int64_t)P * r * 4);  // bytes between slices
  for (int c0 = 0; c0 < cnt; c0 += 8 * kThreads) {
    // a[q]: element c0 + 4 ((q / 4) kThreads + tid) + q % 4
    float a[8];
    if (vec) {
      uint32_t o[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o[h] = (uint32_t)(((int64_t)p0 * r + min(c0 + 4 * (h * kThreads + tid), cnt - 4)) * 4);
      f32x4 v[2];
      // one half at a time (registers), sixteen slices' loads in flight
      // (clamped: the extra ones are not added)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        for (int z0 = 0; z0 < S_; z0 += 16) {
          f32x4 w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[k] = __builtin_bit_cast(
                f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           rp, o[h] + (uint32_t)min(z0 + k, S_ - 1) * zst, 0, kDeviceScope));
          if (z0 == 0) v[h] = w[0];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if ((z0 > 0 || k > 0) && z0 + k < S_) v[h] += w[k];
        }
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] = v[q >> 2][q & 3];
    } else {
      uint32_t o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        o[q] = (uint32_t)(((int64_t)p0 * r +
                           min(c0 + 4 * ((q >> 2) * kThreads + tid) + (q & 3), cnt - 1)) * 4);
      for (int z0 = 0; z0 < S_; z0 += 8) {
        float w[8][8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            w[q][k] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                rp, o[q] + (uint32_t)min(z0 + k, S_ - 1) * zst, 0, kDeviceScope));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (z0 == 0) a[q] = w[q][0];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if ((z0 > 0 || k > 0) && z0 + k < S_) a[q] += w[q][k];
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int e = c0 + 4 * ((q >> 2) * kThreads + tid) + (q & 3);
      if (e >= cnt) continue;
      const int64_t p = p0 + e / r;
      const int j = e % r;
      if (tr)
        out[(int64_t)j * P + p] = a[q];
      else
        out[p * r + j] = a[q];
    }
  }
  if (tid == 0)  // every slice has arrived: ready for the next call
    __hip_atomic_store(ctr, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// out = sum over slices of part, added in slice order (loads issued eight
// at a time), for the two products of one launch: threads 0 .. P0 r - 1
// produce job 0's output, the rest job 1's.  transposed: out[j][p], thread
// index running along p.
struct TnSum {
  const float* part;
  int64_t P;
  int S;
  bool transposed;
  float* out;
};
__global__ void k_sum_slices_tn(TnSum a, TnSum b, int r) {
  int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t count_a = a.P * r;
  const bool second = t >= count_a;
  const TnSum& J = second ? b : a;
  if (second) t -= count_a;
  const int64_t count = J.P * r;
  if (t >= count) return;
  // element index into part[s] ([P][r]) and into out
  const int64_t i = J.transposed ? (t % J.P) * r + t / J.P : t;
  J.out[t] = slice_sum(J.part, count, J.S, i);
}

// out[i] = sum over the slices of part[s][i], in slice order, for the two
// products of one launch whose slices lie as their outputs do; four elements a
// thread (counts are multiples of 8).
__global__ void k_sum_parts(TnSum a, TnSum b, int r) {
  int64_t i = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  const int64_t count_a = a.P * r;
  const bool second = i >= count_a;
  const TnSum& J = second ? b : a;
  if (second) i -= count_a;
  const int64_t count = J.P * r;
  if (i >= count) return;
  f32x4 acc = *reinterpret_cast<const f32x4*>(J.part + i);
  for (int s0 = 1; s0 < J.S; s0 += 8) {
    f32x4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = *reinterpret_cast<const f32x4*>(J.part + (int64_t)min(s0 + k, J.S - 1) * count + i);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k < J.S) acc += v[k];
  }
  *reinterpret_cast<f32x4*>(J.out + i) = acc;
}

// Slices of the M rows for the transposed products: enough workgroups to
// fill the chip (about 512 per product), a multiple of 32 rows each, and
// small enough that a slice of Z or of the (s V)^T parts (384 bytes a row at most)
// spans less than 2^31 bytes (the kernel addresses one slice through a 32-bit
// buffer offset).
// Rows per slice: about 512 workgroups per job, but at most 16 slices per
// column tile: the tile's last workgroup adds the slices, and with 64 of them
// (a 1024-column dB at M = 4096) that sum took longer than the products
// (the k_proj backward's dA/dB launch: 24 us).
// With x in 8 bits (act8) at most 8: a slice's partial sums weigh as much
// against half the bytes of x, and the sums are nearer (4096x1024x4096, r = 64:
// 48.4 -> 45.8 us; 8192x4096x4096, r = 16: 45.0 -> 43.1).
int64_t thin_tn_slice_rows(int64_t M, int64_t P, bool act8) {
  const int64_t pt = (P + TN_COLS - 1) / TN_COLS;
  const int64_t S = std::min<int64_t>((512 + pt - 1) / pt, act8 ? 8 : 16);
  int64_t slice = (M + S - 1) / S;
  slice = (slice + 31) / 32 * 32;
  const int64_t cap = ((((int64_t)1 << 31) - 1) / std::max<int64_t>(2 * P, 384)) / 32 * 32;
  if (slice > cap) slice = cap;
  if (slice < 32) slice = 32;
  return slice;
}

int thin_tn_slices(int64_t M, int64_t P, bool act8) {
  const int64_t slice = thin_tn_slice_rows(M, P, act8);
  return (int)((M + slice - 1) / slice);
}

// Row length of the staged (sV)^T: every slice's rows exist (zero past M).
int64_t thin_tn_rows_padded(int64_t M, int64_t P, bool act8) {
  return (int64_t)thin_tn_slices(M, P, act8) * thin_tn_slice_rows(M, P, act8);
}

hipError_t launch_thin_tn2(const ThinTn& a, const ThinTn& b, int64_t M, int r,
                           unsigned* arrivals, hipStream_t st) {
  const int nj = (r + 15) / 16;
  const bool z8 = b.codes != nullptr;
  TnJob job[2];
  const ThinTn* in[2] = {&a, &b};
  int s_max = 1;
  for (int k = 0; k < 2; ++k) {
    const ThinTn& x = *in[k];
    TnJob& j = job[k];
    j.Z = x.Z;
    j.codes = x.codes;
    j.exps = x.exps;
    j.vt = x.vt;
    j.P = x.P;
    j.slice = thin_tn_slice_rows(M, x.P, z8);
    j.S = thin_tn_slices(M, x.P, z8);
    j.tiles = x.Z || x.codes ? (int)((x.P + TN_COLS - 1) / TN_COLS) : 0;
    j.part = x.part;
    j.out = x.out;
    j.transposed = x.transposed ? 1 : 0;
    j.zmask = x.zmask;
    if (j.tiles > 0) s_max = std::max(s_max, j.S);
  }
  const int tiles = job[0].tiles + job[1].tiles;
  if (tiles == 0) return hipSuccess;
  // slices added by the last workgroup of each tile (one arrival counter per
  // tile, a job's slices through 32-bit offsets), else by a second launch
  bool here = tiles <= kTnMaxTiles;
  for (const TnJob& j : job) here = here && (int64_t)j.S * j.P * r < (int64_t)1 << 30;
  unsigned* ctr = here ? arrivals : nullptr;
  const bool mask = (job[0].tiles > 0 && job[0].zmask) || (job[1].tiles > 0 && job[1].zmask);
  if (a.codes) return hipErrorInvalidValue;  // a checkpoint is the second job's
  const size_t lds =
      (size_t)TN_NST * (32 * TN_ROWB + (z8 ? 3 : 2) * 16 * nj * 64 + (mask ? 32 * 16 : 0));
  const dim3 grid = z8 ? dim3(8u * (unsigned)(tn_per_xcd(job[0]) + tn_per_xcd(job[1])))
                       : dim3((unsigned)tiles, (unsigned)s_max);
#define QN_TN2(NJ, MASK, SP, Z8)                                                           \
  hipLaunchKernelGGL((k_thin_tn<NJ, MASK, SP, Z8>), grid, dim3(kThreads), lds, st, job[0], job[1], \
                     M, r, ctr)
#define QN_TN(NJ)                      \
  if (z8 && mask)                      \
    QN_TN2(NJ, true, 3, true);         \
  else if (z8)                         \
    QN_TN2(NJ, false, 3, true);        \
  else if (mask)                       \
    QN_TN2(NJ, true, 2, false);        \
  else                                 \
    QN_TN2(NJ, false, 2, false)
  switch (nj) {
    case 1: QN_TN(1); break;
    case 2: QN_TN(2); break;
    case 3: QN_TN(3); break;
    default: QN_TN(4); break;
  }
#undef QN_TN
#undef QN_TN2
  if (ctr) return hipGetLastError();
  TnSum sum[2];
  int64_t count = 0;
  for (int k = 0; k < 2; ++k) {
    const ThinTn& x = *in[k];
    sum[k] = TnSum{x.part, job[k].tiles > 0 ? x.P : 0, job[k].S, x.transposed, x.out};
    count += sum[k].P * r;
  }
  if (z8)
    hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)((count / 4 + 255) / 256)), dim3(256), 0, st,
                       sum[0], sum[1], r);
  else
    hipLaunchKernelGGL(k_sum_slices_tn, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, st,
                       sum[0], sum[1], r);
  return hipGetLastError();
}

}  // namespace qn
