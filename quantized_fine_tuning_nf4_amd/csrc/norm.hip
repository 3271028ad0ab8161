// Norms before and after a block, fused with its gate and residual scale
// (formulas in the header), and their gradients.
//
// Backward, with n = h' r2, q = o r1 (r1, r2 the reciprocal root mean squares):
//   dn = dy w_pre            dh = dh' + r2 (dn - n mean(dn n))
//   a  = scale gate dh       dgate = scale p dh (summed to the gate's shape)
//   dq = a w_post            do = r1 (dq - q mean(dq q))
//   dw_pre = sum_m dy n      dw_post = sum_m a q
// r1 and r2 come from o and h' again: their sums of squares ride along with
// the sums the gradients need anyway, so no statistics are kept.
//
// Both directions are bound by HBM: a row's values are read once, stay in
// registers through its two dependent reductions, and leave once.  A row
// belongs to TPR threads (a wave, or a workgroup of 256 to 1024), each holding
// NV vectors of 8 values.
#include <algorithm>
#include <type_traits>

#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

struct NormArgs {
  int64_t M;
  int D;
  const void *w_pre, *w_post, *gate;
  bool w32;
  int gate_kind;
  float scale, eps;
};

enum { kGateNone = 0, kGateChannel = 1, kGateRow = 2, kGateElement = 3 };

// Eight values of a row as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 v = {0u, 0u, 0u, 0u};
  __device__ __forceinline__ float get(int j) const {
    return (j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
  }
  __device__ __forceinline__ void put(int j, float x) {
    const uint32_t b = to_bf16(x);
    v[j >> 1] = (j & 1) ? (v[j >> 1] & 0xffffu) | (b << 16) : (v[j >> 1] & 0xffff0000u) | b;
  }
};
template <>
struct Raw8<float> {
  f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ float get(int j) const { return j < 4 ? a[j & 3] : b[j & 3]; }
};

// Column of value j of vector v of thread t.  VEC (D a multiple of 8, so that
// every row starts on 16 bytes): eight neighbours, a 16-byte access; otherwise
// one column per thread and value, neighbouring threads side by side.
template <int TPR, bool VEC>
__device__ __forceinline__ int column(int v, int j, int t) {
  return VEC ? (v * TPR + t) * 8 + j : (v * 8 + j) * TPR + t;
}

// The values are zero past the row's end.
template <int TPR, bool VEC>
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* row, int v, int t, int D) {
  Raw8<uint16_t> r;
  if constexpr (VEC) {
    const int c = column<TPR, VEC>(v, 0, t);
    if (c < D) r.v = *reinterpret_cast<const u32x4*>(row + c);
  } else {
    uint32_t x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<TPR, VEC>(v, j, t);
      x[j] = c < D ? row[c] : 0u;
    }
    r.v = u32x4{x[0] | (x[1] << 16), x[2] | (x[3] << 16), x[4] | (x[5] << 16), x[6] | (x[7] << 16)};
  }
  return r;
}
template <int TPR, bool VEC>
__device__ __forceinline__ Raw8<float> load8(const float* row, int v, int t, int D) {
  Raw8<float> r;
  if constexpr (VEC) {
    const int c = column<TPR, VEC>(v, 0, t);
    if (c < D) {
      r.a = *reinterpret_cast<const f32x4*>(row + c);
      r.b = *reinterpret_cast<const f32x4*>(row + c + 4);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<TPR, VEC>(v, j, t);
      const float x = c < D ? row[c] : 0.f;
      if (j < 4)
        r.a[j & 3] = x;
      else
        r.b[j & 3] = x;
    }
  }
  return r;
}

template <int TPR, bool VEC>
__device__ __forceinline__ void store8(uint16_t* row, int v, int t, int D, const float (&x)[8]) {
  if constexpr (VEC) {
    const int c = column<TPR, VEC>(v, 0, t);
    if (c < D)
      *reinterpret_cast<u32x4*>(row + c) = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                 pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<TPR, VEC>(v, j, t);
      if (c < D) row[c] = to_bf16(x[j]);
    }
  }
}
template <int TPR, bool VEC>
__device__ __forceinline__ void store8(float* row, int v, int t, int D, const float (&x)[8]) {
  if constexpr (VEC) {
    const int c = column<TPR, VEC>(v, 0, t);
    if (c < D) {
      *reinterpret_cast<f32x4*>(row + c) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(row + c + 4) = f32x4{x[4], x[5], x[6], x[7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<TPR, VEC>(v, j, t);
      if (c < D) row[c] = x[j];
    }
  }
}

// Eight values of a [D] parameter, bf16 or fp32: both forms' bits are loaded
// and told apart where they are used, so that no load is waited for at a
// branch.
struct Param8 {
  Raw8<uint16_t> h;
  Raw8<float> f;
  __device__ __forceinline__ float get(bool w32, int j) const { return w32 ? f.get(j) : h.get(j); }
};
template <int TPR, bool VEC>
__device__ __forceinline__ Param8 load_param(const void* w, bool w32, int v, int t, int D) {
  Param8 p;
  if (w32)
    p.f = load8<TPR, VEC>(static_cast<const float*>(w), v, t, D);
  else
    p.h = load8<TPR, VEC>(static_cast<const uint16_t*>(w), v, t, D);
  return p;
}

// N sums over the TPR threads of a row, the same in each of them.  s: LDS of
// N floats per wave; the caller alternates two of them between reductions, so
// one barrier each is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float* s) {
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = wave_sum(x[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) s[k * W + (threadIdx.x >> 6)] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) x[k] += s[k * W + w];
    }
  }
}

constexpr int group_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int TPR, int NV, bool VEC, typename R>
__global__ __launch_bounds__(group_threads(TPR)) void k_norm_fwd(
    NormArgs n, const R* __restrict__ h, const uint16_t* __restrict__ o, R* __restrict__ hn,
    uint16_t* __restrict__ y, int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  __shared__ float s[2][TPR / 64];
  const int t = threadIdx.x % TPR, D = n.D;
  const int64_t m = (int64_t)blockIdx.x * (group_threads(TPR) / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && m >= n.M) return;  // whole wave; no barrier follows
  const int64_t row = m * D;
  Raw8<R> hv[NV];
  Raw8<uint16_t> ov[NV], gv[NV];
  Param8 w1[NV], w2[NV], gc[NV];
  float gr = n.scale;
#pragma unroll
  for (int v = 0; v < NV; ++v) hv[v] = load8<TPR, VEC>(h + row, v, t, D);
  if (o) {
#pragma unroll
    for (int v = 0; v < NV; ++v) ov[v] = load8<TPR, VEC>(o + row, v, t, D);
    if (n.w_post) {
#pragma unroll
      for (int v = 0; v < NV; ++v) w1[v] = load_param<TPR, VEC>(n.w_post, n.w32, v, t, D);
    }
    if (n.gate_kind == kGateChannel) {
#pragma unroll
      for (int v = 0; v < NV; ++v) gc[v] = load_param<TPR, VEC>(n.gate, n.w32, v, t, D);
    } else if (n.gate_kind == kGateElement) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        gv[v] = load8<TPR, VEC>(static_cast<const uint16_t*>(n.gate) + row, v, t, D);
    } else if (n.gate_kind == kGateRow) {
      gr *= load_f32(static_cast<const uint16_t*>(n.gate) + m);
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) w2[v] = load_param<TPR, VEC>(n.w_pre, n.w32, v, t, D);

  float x[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) x[v][j] = hv[v].get(j);
  if (o) {
    float r1 = 1.f;
    if (n.w_post) {
      float q[1] = {0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) q[0] = __builtin_fmaf(ov[v].get(j), ov[v].get(j), q[0]);
      row_sums<TPR, 1>(q, s[0]);
      r1 = 1.f / __builtin_sqrtf(q[0] / (float)D + n.eps);
    }
    const float k = gr * r1;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float out[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float p = ov[v].get(j) * k;
        if (n.w_post) p *= w1[v].get(n.w32, j);
        if (n.gate_kind == kGateChannel) p *= gc[v].get(n.w32, j);
        if (n.gate_kind == kGateElement) p *= gv[v].get(j);
        out[j] = x[v][j] = x[v][j] + p;
      }
      store8<TPR, VEC>(hn + row, v, t, D, out);
    }
  }
  float q[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) q[0] = __builtin_fmaf(x[v][j], x[v][j], q[0]);
  row_sums<TPR, 1>(q, s[1]);
  const float r2 = 1.f / __builtin_sqrtf(q[0] / (float)D + n.eps);
  const int nb = (D + kAct8Block - 1) / kAct8Block;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = x[v][j] * r2 * w2[v].get(n.w32, j);
    store8<TPR, VEC>(y + row, v, t, D, out);
    if (!codes) continue;
    // the checkpoint of y as it is stored; values past the row's end are zero
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = to_bf16(out[j]);
    if constexpr (VEC) {  // a block of 64 columns is 8 lanes' vectors
      uint32_t top = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, b[j] & 0x7fffu);
      top = max_of_8_lanes(top);
      const uint32_t E = act8_exp(top);
      const float inv = act8_inv(E);
      const int c = column<TPR, VEC>(v, 0, t);
      if (c < D) {
        u32x2 w = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j >> 2] |= ((uint32_t)act8_code(as_f32(b[j] << 16), inv) & 0xffu) << (8 * (j & 3));
        if (E == kAct8NaN) w = u32x2{0u, 0u};
        *reinterpret_cast<u32x2*>(codes + row + c) = w;
        if ((t & 7) == 0) exps[m * nb + c / kAct8Block] = (uint8_t)E;
      }
    } else {  // a block is one value of each of a wave's lanes
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = column<TPR, VEC>(v, j, t);
        const uint32_t E = act8_exp(wave_max_u32(b[j] & 0x7fffu));
        if (c < D) {
          codes[row + c] =
              E == kAct8NaN ? 0 : (int8_t)act8_code(as_f32(b[j] << 16), act8_inv(E));
          if ((t & 63) == 0) exps[m * nb + c / kAct8Block] = (uint8_t)E;
        }
      }
    }
  }
}

// Row group z takes rows z, z + groups, ...  With SUMS a thread keeps its
// columns' sums over those rows in registers; a workgroup's groups meet in
// LDS and leave part [workgroup][3][D] (dw_pre, dw_post, channel dgate).  The
// next row's loads go out before the current row's reductions.
template <int TPR, int NV, bool VEC, bool SUMS, typename R>
__global__ __launch_bounds__(group_threads(TPR)) void k_norm_bwd(
    NormArgs n, const uint16_t* __restrict__ dy, const R* __restrict__ dhn,
    const R* __restrict__ hn, const uint16_t* __restrict__ o, R* __restrict__ dh,
    uint16_t* __restrict__ dout, void* __restrict__ dgate, float* __restrict__ part) {
  constexpr int G = group_threads(TPR) / TPR;  // row groups of a workgroup
  constexpr int W = TPR / 64;
  __shared__ float s[2][2][3 * W];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, D = n.D;
  const float rD = 1.f / (float)D;
  const bool post = n.w_post != nullptr, chan = n.gate_kind == kGateChannel,
             elem = n.gate_kind == kGateElement, rowg = n.gate_kind == kGateRow;
  float sp[NV][8] = {}, so[NV][8] = {}, sg[NV][8] = {};
  Param8 w1[NV], w2[NV], gc[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    w2[v] = load_param<TPR, VEC>(n.w_pre, n.w32, v, t, D);
    if (post) w1[v] = load_param<TPR, VEC>(n.w_post, n.w32, v, t, D);
    if (chan) gc[v] = load_param<TPR, VEC>(n.gate, n.w32, v, t, D);
  }
  Raw8<R> hv[NV], dv[NV];
  Raw8<uint16_t> yv[NV], ov[NV], gv[NV];
  auto load_row = [&](int64_t m) {
    const int64_t row = m * D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      hv[v] = load8<TPR, VEC>(hn + row, v, t, D);
      yv[v] = load8<TPR, VEC>(dy + row, v, t, D);
      if (o) ov[v] = load8<TPR, VEC>(o + row, v, t, D);
      if (dhn) dv[v] = load8<TPR, VEC>(dhn + row, v, t, D);
      if (elem) gv[v] = load8<TPR, VEC>(static_cast<const uint16_t*>(n.gate) + row, v, t, D);
    }
  };
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t m = (int64_t)blockIdx.x * G + grp;
  if (m < n.M) load_row(m);
  int par = 0;
  // the rows of a group that is a whole workgroup are the same for all its
  // threads; a wave's own rows need no barrier
  for (; m < n.M; m += step, par ^= 1) {
    const int64_t row = m * D;
    Raw8<R> h_[NV], d_[NV];
    Raw8<uint16_t> y_[NV], o_[NV], g_[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h_[v] = hv[v];
      d_[v] = dv[v];
      y_[v] = yv[v];
      o_[v] = ov[v];
      g_[v] = gv[v];
    }
    const float grow = rowg ? n.scale * load_f32(static_cast<const uint16_t*>(n.gate) + m) : n.scale;
    if (SUMS && m + step < n.M) load_row(m + step);
    float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = h_[v].get(j);
        q[0] = __builtin_fmaf(x, x, q[0]);
        q[1] = __builtin_fmaf(y_[v].get(j) * w2[v].get(n.w32, j), x, q[1]);
        if (post) q[2] = __builtin_fmaf(o_[v].get(j), o_[v].get(j), q[2]);
      }
    row_sums<TPR, 3>(q, s[par][0]);
    const float r2 = 1.f / __builtin_sqrtf(q[0] * rD + n.eps);
    const float c2 = q[1] * r2 * rD * r2;  // r2 mean(dn n)
    const float r1 = post ? 1.f / __builtin_sqrtf(q[2] * rD + n.eps) : 1.f;
    float d[NV][8], e[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float out[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = h_[v].get(j), g = y_[v].get(j);
        const float dn = g * w2[v].get(n.w32, j);
        out[j] = d[v][j] = __builtin_fmaf(r2, dn - x * c2, d_[v].get(j));
        if (SUMS) sp[v][j] = __builtin_fmaf(g, x * r2, sp[v][j]);
      }
      store8<TPR, VEC>(dh + row, v, t, D, out);
    }
    if (!o) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // d becomes dq (or a, without a post norm)
        const float x = o_[v].get(j) * r1, wp = post ? w1[v].get(n.w32, j) : 1.f;
        const float base = d[v][j];
        float a = base * grow;
        if (chan) a *= gc[v].get(n.w32, j);
        if (elem) a *= g_[v].get(j);
        d[v][j] = a * wp;
        e[0] = __builtin_fmaf(a * wp, x, e[0]);
        if (rowg) e[1] = __builtin_fmaf(base * n.scale, x * wp, e[1]);
        if (SUMS) {
          so[v][j] = __builtin_fmaf(a, x, so[v][j]);
          if (chan) sg[v][j] = __builtin_fmaf(base * n.scale, x * wp, sg[v][j]);
        }
        if (elem) g_[v].put(j, base * n.scale * (x * wp));
      }
    if (post || rowg) row_sums<TPR, 2>(e, s[par][1]);
    if (rowg && dgate && t == 0) static_cast<float*>(dgate)[m] = e[1];
    const float c1 = e[0] * rD * r1;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float out[8], dg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        out[j] = post ? r1 * (d[v][j] - o_[v].get(j) * c1) : d[v][j];
        dg[j] = g_[v].get(j);
      }
      store8<TPR, VEC>(dout + row, v, t, D, out);
      if (elem && dgate) store8<TPR, VEC>(static_cast<uint16_t*>(dgate) + row, v, t, D, dg);
    }
  }
  if constexpr (SUMS) {
    float* dst = part + (int64_t)blockIdx.x * 3 * D;
    if constexpr (G == 1) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        store8<TPR, VEC>(dst, v, t, D, sp[v]);
        store8<TPR, VEC>(dst + D, v, t, D, so[v]);
        store8<TPR, VEC>(dst + 2 * D, v, t, D, sg[v]);
      }
    } else {
      __shared__ float acc[G][3 * NV * 8 * TPR];
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = (v * 8 + j) * TPR + t;
          acc[grp][i] = sp[v][j];
          acc[grp][NV * 8 * TPR + i] = so[v][j];
          acc[grp][2 * NV * 8 * TPR + i] = sg[v][j];
        }
      __syncthreads();
      for (int i = threadIdx.x; i < 3 * NV * 8 * TPR; i += group_threads(TPR)) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < G; ++k) x += acc[k][i];
        const int which = i / (NV * 8 * TPR), l = i % (NV * 8 * TPR);
        const int c = column<TPR, VEC>(l / TPR / 8, l / TPR % 8, l % TPR);
        if (c < D) dst[which * D + c] = x;
      }
    }
  }
}

// out_j[c] = sum over the S slices of part[z][j][c]: a workgroup takes 64
// columns, thread group k the slices k, k + 16, ... in order, and the sixteen
// sums are added in order.
constexpr int kSumGroups = 16;
__global__ __launch_bounds__(64 * kSumGroups) void k_norm_sums(const float* __restrict__ part,
                                                               int S, int D, float* __restrict__ o0,
                                                               float* __restrict__ o1,
                                                               float* __restrict__ o2) {
  __shared__ float s[kSumGroups][64];
  const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + c;  // column of the 3 D
  float x = 0.f;
  if (i < 3 * D) {
    for (int z0 = k; z0 < S; z0 += 8 * kSumGroups) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int z = z0 + q * kSumGroups;
        v[q] = z < S ? part[(int64_t)z * 3 * D + i] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) x += v[q];
    }
  }
  s[k][c] = x;
  __syncthreads();
  if (k == 0 && i < 3 * D) {
    float* out = i < D ? o0 : i < 2 * D ? o1 : o2;
    if (out) {
      x = 0.f;
#pragma unroll
      for (int q = 0; q < kSumGroups; ++q) x += s[q][c];
      out[i % D] = x;
    }
  }
}

NormArgs args_of(const BlockNorm& n) {
  return NormArgs{n.M, (int)n.D, n.w_pre, n.w_post, n.gate, n.w32, n.gate_kind, n.scale, n.eps};
}

// Threads of a row: a wave up to 1024 columns, then the fewest of 256, 512 and
// 1024 that hold the row in few vectors each.
int row_threads(int64_t D) { return D <= 1024 ? 64 : D <= 2048 ? 256 : D <= 8192 ? 512 : 1024; }

// Calls f<TPR, NV>() for the row length D.
template <typename F>
hipError_t by_columns(int64_t D, F&& f) {
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  using T64 = std::integral_constant<int, 64>;
  using T256 = std::integral_constant<int, 256>;
  using T512 = std::integral_constant<int, 512>;
  using T1024 = std::integral_constant<int, 1024>;
  if (D <= 512) return f(T64{}, I1{});
  if (D <= 1024) return f(T64{}, I2{});
  if (D <= 2048) return f(T256{}, I1{});
  if (D <= 4096) return f(T512{}, I1{});
  if (D <= 8192) return f(T512{}, I2{});
  if (D <= 16384) return f(T1024{}, I2{});
  return f(T1024{}, I4{});
}

template <typename R>
hipError_t norm_fwd(const BlockNorm& n, const void* h, const uint16_t* o, void* h_new, uint16_t* y,
                    int8_t* codes, uint8_t* exps, hipStream_t st) {
  return by_columns(n.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int T = group_threads(TPR), G = T / TPR;
    const dim3 grid((unsigned)((n.M + G - 1) / G));
    const NormArgs a = args_of(n);
    const R* hp = static_cast<const R*>(h);
    R* hn = static_cast<R*>(h_new);
    if (n.D % 8 == 0)
      hipLaunchKernelGGL((k_norm_fwd<TPR, NV, true, R>), grid, dim3(T), 0, st, a, hp, o, hn, y,
                         codes, exps);
    else
      hipLaunchKernelGGL((k_norm_fwd<TPR, NV, false, R>), grid, dim3(T), 0, st, a, hp, o, hn, y,
                         codes, exps);
    return hipGetLastError();
  });
}

template <typename R, bool SUMS>
hipError_t norm_bwd(const BlockNorm& n, const uint16_t* dy, const void* dh_new, const void* h_new,
                    const uint16_t* o, void* dh, uint16_t* dout, void* dgate, float* part,
                    hipStream_t st) {
  return by_columns(n.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int T = group_threads(TPR), G = T / TPR;
    const dim3 grid((unsigned)(SUMS ? block_norm_slices(n.M, n.D) : (n.M + G - 1) / G));
    const NormArgs a = args_of(n);
    const R *dp = static_cast<const R*>(dh_new), *hp = static_cast<const R*>(h_new);
    R* out = static_cast<R*>(dh);
    if (n.D % 8 == 0)
      hipLaunchKernelGGL((k_norm_bwd<TPR, NV, true, SUMS, R>), grid, dim3(T), 0, st, a, dy, dp, hp,
                         o, out, dout, dgate, part);
    else
      hipLaunchKernelGGL((k_norm_bwd<TPR, NV, false, SUMS, R>), grid, dim3(T), 0, st, a, dy, dp,
                         hp, o, out, dout, dgate, part);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNorm& n, const void* h, const uint16_t* o, void* h_new,
                                 uint16_t* y, int8_t* codes, uint8_t* exps, hipStream_t st) {
  if (n.M == 0) return hipSuccess;
  return n.res32 ? norm_fwd<float>(n, h, o, h_new, y, codes, exps, st)
                 : norm_fwd<uint16_t>(n, h, o, h_new, y, codes, exps, st);
}

// Workgroups of a backward that sums over rows: two for each of 256 compute
// units, as many as stay resident, unless the rows are fewer.
int block_norm_slices(int64_t M, int64_t D) {
  const int64_t G = group_threads(row_threads(D)) / row_threads(D);
  return (int)std::min<int64_t>((M + G - 1) / G, 512);
}

hipError_t launch_block_norm_bwd(const BlockNorm& n, const uint16_t* dy, const void* dh_new,
                                 const void* h_new, const uint16_t* o, void* dh, uint16_t* dout,
                                 void* dgate, float* dw_post, float* dw_pre, float* part,
                                 hipStream_t st) {
  if (n.M == 0) return hipSuccess;
  hipError_t e;
  if (!part)
    return n.res32 ? norm_bwd<float, false>(n, dy, dh_new, h_new, o, dh, dout, dgate, part, st)
                   : norm_bwd<uint16_t, false>(n, dy, dh_new, h_new, o, dh, dout, dgate, part, st);
  e = n.res32 ? norm_bwd<float, true>(n, dy, dh_new, h_new, o, dh, dout, dgate, part, st)
              : norm_bwd<uint16_t, true>(n, dy, dh_new, h_new, o, dh, dout, dgate, part, st);
  if (e != hipSuccess) return e;
  float* dg = n.gate_kind == kGateChannel ? static_cast<float*>(dgate) : nullptr;
  hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)((3 * n.D + 63) / 64)), dim3(64 * kSumGroups), 0,
                     st, part, block_norm_slices(n.M, n.D), (int)n.D, dw_pre, dw_post, dg);
  return hipGetLastError();
}

}  // namespace qn
