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
// belongs to TPR threads (a wave, or a workgroup of up to 1024), each holding NV
// vectors of 8 values.
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

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

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

// Vector v of thread t holds the columns from here on.  Rows of odd lengths
// (TAIL: D no multiple of 8) start on any element -- vector accesses need no
// alignment on this target -- and end inside a vector: its thread loads the
// row's last eight values instead, and in_place moves them where they belong
// once they are here (a branch that only the row's last wave takes).
template <int TPR>
__device__ __forceinline__ int column(int v, int t) {
  return (v * TPR + t) * 8;
}

// Values past the row's end are zero (with TAIL: after in_place).
template <int TPR, bool TAIL>
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* row, int v, int t, int D) {
  Raw8<uint16_t> r;
  const int c = column<TPR>(v, t);
  if (!TAIL || D >= 8) {
    if (c < D) r.v = *reinterpret_cast<const u32x4_any*>(row + (TAIL ? min(c, D - 8) : c));
  } else if (c == 0) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < D) r.v[j >> 1] |= (uint32_t)row[j] << (16 * (j & 1));
  }
  return r;
}
template <int TPR, bool TAIL>
__device__ __forceinline__ Raw8<float> load8(const float* row, int v, int t, int D) {
  Raw8<float> r;
  const int c = column<TPR>(v, t);
  if (!TAIL || D >= 8) {
    if (c < D) {
      const float* p = row + (TAIL ? min(c, D - 8) : c);
      r.a = *reinterpret_cast<const f32x4_any*>(p);
      r.b = *reinterpret_cast<const f32x4_any*>(p + 4);
    }
  } else if (c == 0) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < D) (j < 4 ? r.a : r.b)[j & 3] = row[j];
  }
  return r;
}

template <int TPR, bool TAIL>
__device__ __forceinline__ void in_place(Raw8<uint16_t>& r, int v, int t, int D) {
  if constexpr (TAIL) {
    const int by = column<TPR>(v, t) + 8 - D;  // values that lie past the row's end
    if (D < 8 || !__any(by > 0 && by < 8)) return;
    if (by <= 0 || by >= 8) return;
    const uint64_t lo = (uint64_t)r.v[0] | ((uint64_t)r.v[1] << 32);
    const uint64_t hi = (uint64_t)r.v[2] | ((uint64_t)r.v[3] << 32);
    const int bits = 16 * by;
    const uint64_t a = bits < 64 ? (lo >> bits) | (hi << (64 - bits)) : hi >> (bits - 64);
    const uint64_t b = bits < 64 ? hi >> bits : 0;
    r.v = u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
  }
}
template <int TPR, bool TAIL>
__device__ __forceinline__ void in_place(Raw8<float>& r, int v, int t, int D) {
  if constexpr (TAIL) {
    const int by = column<TPR>(v, t) + 8 - D;
    if (D < 8 || !__any(by > 0 && by < 8)) return;
    if (by <= 0 || by >= 8) return;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = r.get(j);
#pragma unroll
    for (int k = 4; k >= 1; k >>= 1)
      if (by & k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j + k < 8 ? x[(j + k) & 7] : 0.f;
      }
    r.a = f32x4{x[0], x[1], x[2], x[3]};
    r.b = f32x4{x[4], x[5], x[6], x[7]};
  }
}

template <int TPR, bool TAIL>
__device__ __forceinline__ void store8(uint16_t* row, int v, int t, int D, const float (&x)[8]) {
  const int c = column<TPR>(v, t);
  const u32x4 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7])};
  if (TAIL ? c + 8 <= D : c < D) {
    *reinterpret_cast<u32x4_any*>(row + c) = w;
  } else if (TAIL) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (c + j < D) row[c + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}
template <int TPR, bool TAIL>
__device__ __forceinline__ void store8(float* row, int v, int t, int D, const float (&x)[8]) {
  const int c = column<TPR>(v, t);
  if (TAIL ? c + 8 <= D : c < D) {
    *reinterpret_cast<f32x4_any*>(row + c) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4_any*>(row + c + 4) = f32x4{x[4], x[5], x[6], x[7]};
  } else if (TAIL) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (c + j < D) row[c + j] = x[j];
  }
}

// Keeps the loaded form from here on: without it the compiler holds the
// values it has unpacked for one pass over the row until the next one.
__device__ __forceinline__ void as_loaded(Raw8<uint16_t>& r) { asm volatile("" : "+v"(r.v)); }
__device__ __forceinline__ void as_loaded(Raw8<float>&) {}

// Eight values of a [D] parameter, bf16 or fp32: the loaded bits, told apart
// where they are used, so that no load is waited for at a branch.
struct Param8 {
  u32x4 lo = {0u, 0u, 0u, 0u}, hi = {0u, 0u, 0u, 0u};  // fp32: values 0-3, 4-7; bf16: all in lo
  __device__ __forceinline__ float get(bool w32, int j) const {
    const uint32_t f = j < 4 ? lo[j & 3] : hi[j & 3];
    const uint32_t h = (j & 1) ? lo[j >> 1] & 0xffff0000u : lo[j >> 1] << 16;
    return as_f32(w32 ? f : h);
  }
};
template <int TPR, bool TAIL>
__device__ __forceinline__ Param8 load_param(const void* w, bool w32, int v, int t, int D) {
  Param8 p;
  if (w32) {
    Raw8<float> f = load8<TPR, TAIL>(static_cast<const float*>(w), v, t, D);
    in_place<TPR, TAIL>(f, v, t, D);
    p.lo = __builtin_bit_cast(u32x4, f.a);
    p.hi = __builtin_bit_cast(u32x4, f.b);
  } else {
    Raw8<uint16_t> h = load8<TPR, TAIL>(static_cast<const uint16_t*>(w), v, t, D);
    in_place<TPR, TAIL>(h, v, t, D);
    p.lo = h.v;
  }
  return p;
}

// N sums over the threads of a row, the same in each of them.  s: LDS of
// N floats for each of TPR / 64 waves; the caller alternates two of them between
// reductions, so one barrier each is enough, and has cleared those of waves
// that are not there (clear_sums).
template <int COUNT>
__device__ __forceinline__ void clear_sums(float* s) {
  for (int i = threadIdx.x; i < COUNT; i += blockDim.x) s[i] = 0.f;
  __syncthreads();
}
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
    // every group of W lanes adds the W waves' sums
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float v = s[k * W + (threadIdx.x & (W - 1))];
      v += as_f32(dpp<kDppXor1>(as_u32(v)));
      if (W >= 4) v += as_f32(dpp<kDppXor2>(as_u32(v)));
      if (W >= 8) v += as_f32(dpp<kDppMirror8>(as_u32(v)));
      if (W >= 16) v += as_f32(dpp<kDppMirror16>(as_u32(v)));
      x[k] = v;
    }
  }
}

// 1 / sqrt(x), x normal, infinite or NaN: the instruction's estimate and one
// Newton step, off by 2^-23.
__device__ __forceinline__ float inv_sqrt(float x) {
  const float y = __builtin_amdgcn_rsqf(x);
  const float z = __builtin_fmaf(0.5f * y, __builtin_fmaf(-x * y, y, 1.f), y);
  return y == 0.f ? 0.f : z;  // squares past fp32
}

// Most threads of a workgroup: four rows' waves, or one row's threads (no more
// waves than hold the row).
constexpr int group_threads(int tpr) { return tpr == 64 ? 256 : tpr; }
// A thread's row group in its workgroup (a wave's, in a scalar register).
template <int TPR>
__device__ __forceinline__ int row_group() {
  return TPR > 64 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// Where a row's threads have the [D] parameters (w_pre, w_post, the channel
// gate) and, in the backward, the column sums of their gradients, from row to
// row: in registers with one vector a thread in up to 512 threads, else in LDS,
// every thread its own values, as far as that goes, else the parameters come
// from L2 again for every row and the sums from k_norm_columns.
constexpr bool keeps(int tpr, int nv) { return nv == 1 && tpr < 1024; }
// Whether the next row's loads go out ahead of the current row's reductions.
constexpr bool prefetches(int nv) { return nv == 1; }

// Slots of 16 bytes a vector and thread: the first of each parameter and each
// sum (fp32 values take two), or -1.
struct Slots {
  int par[3], sum[3], count;
};
constexpr size_t kSlotBytes = 144 * 1024;  // of 160 KB a compute unit
// keep: parameters in registers.  sums: which of them go to LDS.
Slots slots_of(const BlockNorm& n, bool keep, const bool (&sums)[3], int threads, int nv) {
  Slots s{{-1, -1, -1}, {-1, -1, -1}, 0};
  const int most = (int)(kSlotBytes / ((size_t)16 * threads * nv));
  auto take = [&](int& slot, int need) {
    if (s.count + need > most) return;
    slot = s.count;
    s.count += need;
  };
  for (int k = 0; k < 3; ++k)
    if (sums[k]) take(s.sum[k], 2);
  const bool there[3] = {true, n.w_post != nullptr, n.gate_kind == kGateChannel};
  for (int k = 0; k < 3; ++k)
    if (!keep && there[k]) take(s.par[k], n.w32 ? 2 : 1);
  return s;
}

template <int TPR, int NV, bool TAIL>
struct Lds {
  u32x4* base;
  const Slots& s;
  int t;
  __device__ __forceinline__ u32x4& at(int slot, int v) const {
    return base[(slot * NV + v) * (int)blockDim.x + t];
  }
  __device__ __forceinline__ void stage(const NormArgs& n, int which, const void* w) const {
    if (s.par[which] < 0) return;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const Param8 p = load_param<TPR, TAIL>(w, n.w32, v, t, n.D);
      at(s.par[which], v) = p.lo;
      if (n.w32) at(s.par[which] + 1, v) = p.hi;
    }
  }
  __device__ __forceinline__ Param8 param(const NormArgs& n, int which, const void* w, int v) const {
    if (s.par[which] < 0) {
      asm volatile("" : "+s"(w) : : "memory");  // loaded here, no earlier
      return load_param<TPR, TAIL>(w, n.w32, v, t, n.D);
    }
    Param8 p;
    p.lo = at(s.par[which], v);
    if (n.w32) p.hi = at(s.par[which] + 1, v);
    return p;
  }
  __device__ __forceinline__ void clear(int which) const {
    if (s.sum[which] >= 0)
      at(s.sum[which], 0) = at(s.sum[which] + 1, 0) = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void add(int which, const float (&x)[8]) const {
    if (s.sum[which] < 0) return;
    f32x4* lo = reinterpret_cast<f32x4*>(&at(s.sum[which], 0));
    f32x4* hi = reinterpret_cast<f32x4*>(&at(s.sum[which] + 1, 0));
    *lo += f32x4{x[0], x[1], x[2], x[3]};
    *hi += f32x4{x[4], x[5], x[6], x[7]};
  }
  __device__ __forceinline__ void store(int which, float* row, int D) const {
    float x[8] = {};
    if (s.sum[which] >= 0) {
      const f32x4 lo = __builtin_bit_cast(f32x4, at(s.sum[which], 0));
      const f32x4 hi = __builtin_bit_cast(f32x4, at(s.sum[which] + 1, 0));
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = j < 4 ? lo[j & 3] : hi[j & 3];
    }
    store8<TPR, TAIL>(row, 0, t, D, x);
  }
};
extern __shared__ u32x4 slots_lds[];

// Measured: 4096 x 4096, h fp32, post norm and checkpoint (218 MB) 40.8 us, 5.3
// TB/s, a large copy's rate; 8192 x 4096 in bf16 with fp32 parameters 52.1 us (5.2
// TB/s; without the next row's loads ahead 67.7); 4096 x 8192 bf16, 1024 threads a
// row with the parameters in LDS, 51 us; one row of 4096 3.0 us, a launch and two
// reductions.
template <int TPR, int NV, bool TAIL, typename R>
__global__ __launch_bounds__(group_threads(TPR)) void k_norm_fwd(
    NormArgs n, Slots slots, const R* __restrict__ h, const uint16_t* __restrict__ o,
    R* __restrict__ hn, uint16_t* __restrict__ y, int8_t* __restrict__ codes,
    uint8_t* __restrict__ exps) {
  constexpr bool KEEP = keeps(TPR, NV);
  constexpr int G = group_threads(TPR) / TPR;
  __shared__ float s[2][2][TPR / 64];
  if (TPR > 64) clear_sums<4 * (TPR / 64)>(&s[0][0][0]);
  const int t = threadIdx.x % TPR, D = n.D;
  const int nb = (D + kAct8Block - 1) / kAct8Block;
  const bool post = n.w_post != nullptr, chan = n.gate_kind == kGateChannel,
             elem = n.gate_kind == kGateElement, rowg = n.gate_kind == kGateRow;
  Param8 w1, w2, gc;  // of vector 0, with KEEP
  const Lds<TPR, NV, TAIL> lds{slots_lds, slots, t};
  Raw8<R> hv[NV];
  Raw8<uint16_t> ov[NV], gv[NV];
  auto load_row = [&](int64_t m) {
    const int64_t row = m * D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      hv[v] = load8<TPR, TAIL>(h + row, v, t, D);
      if (o) ov[v] = load8<TPR, TAIL>(o + row, v, t, D);
      if (elem) gv[v] = load8<TPR, TAIL>(static_cast<const uint16_t*>(n.gate) + row, v, t, D);
    }
  };
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t m = (int64_t)blockIdx.x * G + row_group<TPR>();
  if (prefetches(NV) && m < n.M) load_row(m);
  if (KEEP) {
    if (post) w1 = load_param<TPR, TAIL>(n.w_post, n.w32, 0, t, D);
    if (chan) gc = load_param<TPR, TAIL>(n.gate, n.w32, 0, t, D);
    w2 = load_param<TPR, TAIL>(n.w_pre, n.w32, 0, t, D);
  } else {
    lds.stage(n, 0, n.w_pre);
    lds.stage(n, 1, n.w_post);
    lds.stage(n, 2, n.gate);
  }
  // a group that is a whole workgroup runs the same rows in all its threads; a
  // wave's own rows need no barrier
  for (int par = 0; m < n.M; m += step, par ^= 1) {
    const int64_t row = m * D;
    if (!prefetches(NV)) load_row(m);
    Raw8<uint16_t> o_[NV], g_[NV];
    float x[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      in_place<TPR, TAIL>(hv[v], v, t, D);
      if (o) in_place<TPR, TAIL>(ov[v], v, t, D);
      if (elem) in_place<TPR, TAIL>(gv[v], v, t, D);
      o_[v] = ov[v];
      g_[v] = gv[v];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = hv[v].get(j);
    }
    float k = n.scale;
    if (rowg) k *= load_f32(static_cast<const uint16_t*>(n.gate) + m);
    if (prefetches(NV) && m + step < n.M) load_row(m + step);
    if (o) {
      if (post) {
        float q[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) q[0] = __builtin_fmaf(o_[v].get(j), o_[v].get(j), q[0]);
        row_sums<TPR, 1>(q, s[par][0]);
        k *= inv_sqrt(q[0] / (float)D + n.eps);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float out[8];
        if (!KEEP && post) w1 = lds.param(n, 1, n.w_post, v);
        if (!KEEP && chan) gc = lds.param(n, 2, n.gate, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float p = o_[v].get(j) * k;
          if (post) p *= w1.get(n.w32, j);
          if (chan) p *= gc.get(n.w32, j);
          if (elem) p *= g_[v].get(j);
          out[j] = x[v][j] = x[v][j] + p;
        }
        store8<TPR, TAIL>(hn + row, v, t, D, out);
      }
    }
    float q[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[0] = __builtin_fmaf(x[v][j], x[v][j], q[0]);
    row_sums<TPR, 1>(q, s[par][1]);
    const float r2 = inv_sqrt(q[0] / (float)D + n.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float out[8];
      if (!KEEP) w2 = lds.param(n, 0, n.w_pre, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = x[v][j] * r2 * w2.get(n.w32, j);
      store8<TPR, TAIL>(y + row, v, t, D, out);
      if (!codes) continue;
      // the checkpoint of y as it is stored, a block of 64 columns in 8 lanes'
      // vectors; values past the row's end are zero
      uint32_t b[8], top = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        b[j] = to_bf16(out[j]);
        top = max(top, b[j] & 0x7fffu);
      }
      top = max_of_8_lanes(top);
      const uint32_t E = act8_exp(top);
      const float inv = act8_inv(E);
      const int c = column<TPR>(v, t);
      u32x2 w = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j >> 2] |= ((uint32_t)act8_code(as_f32(b[j] << 16), inv) & 0xffu) << (8 * (j & 3));
      if (E == kAct8NaN) w = u32x2{0u, 0u};
      if (TAIL ? c + 8 <= D : c < D) {
        *reinterpret_cast<u32x2_any*>(codes + row + c) = w;
      } else if (TAIL) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (c + j < D) codes[row + c + j] = (int8_t)(w[j >> 2] >> (8 * (j & 3)));
      }
      if (c < D && (t & 7) == 0) exps[m * nb + c / kAct8Block] = (uint8_t)E;
    }
  }
}

// Row group z takes rows z, z + groups, ...  A thread keeps its columns' sums
// over those rows in registers (kSumsRegs; a workgroup's groups meet in LDS) or
// LDS (kSumsLds); a workgroup leaves part [workgroup][3][D] (dw_pre, dw_post,
// channel dgate).
// Measured: 8192 x 4096 bf16, post norm, channel gate and every gradient (403 MB)
// 75.4 us and 4.8 for k_norm_sums, 5.0 TB/s; with the column sums in LDS instead
// 89 us, in twice the workgroups 97, in registers of 1024 threads, which spill,
// 255.  1003 x 1001 (rows on odd bytes, row gate) 6.4 us.
enum { kSumsNone = 0, kSumsRegs = 1, kSumsLds = 2 };
template <int TPR, int NV, bool TAIL, int SUMS, typename R>
__global__ __launch_bounds__(group_threads(TPR)) void k_norm_bwd(
    NormArgs n, Slots slots, const uint16_t* __restrict__ dy, const R* __restrict__ dhn,
    const R* __restrict__ hn, const uint16_t* __restrict__ o, R* __restrict__ dh,
    uint16_t* __restrict__ dout, void* __restrict__ dgate, float* __restrict__ part,
    f32x4* __restrict__ stats) {
  constexpr bool REGS = SUMS == kSumsRegs;
  constexpr int G = group_threads(TPR) / TPR;  // row groups of a workgroup
  constexpr int W = TPR / 64;
  constexpr bool KEEP = keeps(TPR, NV);
  __shared__ float s[2][2][3 * W];
  if (TPR > 64) clear_sums<12 * W>(&s[0][0][0]);
  const int t = threadIdx.x % TPR, grp = row_group<TPR>(), D = n.D;
  const float rD = 1.f / (float)D;
  const bool post = n.w_post != nullptr, chan = n.gate_kind == kGateChannel,
             elem = n.gate_kind == kGateElement, rowg = n.gate_kind == kGateRow;
  float sp[NV][8] = {}, so[NV][8] = {}, sg[NV][8] = {};
  Param8 w1, w2, gc;  // of vector 0, with KEEP
  const Lds<TPR, NV, TAIL> lds{slots_lds, slots, t};
  if (KEEP) {
    w2 = load_param<TPR, TAIL>(n.w_pre, n.w32, 0, t, D);
    if (post) w1 = load_param<TPR, TAIL>(n.w_post, n.w32, 0, t, D);
    if (chan) gc = load_param<TPR, TAIL>(n.gate, n.w32, 0, t, D);
  } else {
    lds.stage(n, 0, n.w_pre);
    lds.stage(n, 1, n.w_post);
    lds.stage(n, 2, n.gate);
  }
  if (SUMS == kSumsLds) {
#pragma unroll
    for (int k = 0; k < 3; ++k) lds.clear(k);
  }
  Raw8<R> hv[NV], dv[NV];
  Raw8<uint16_t> yv[NV], ov[NV], gv[NV];
  auto load_row = [&](int64_t m) {
    const int64_t row = m * D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      hv[v] = load8<TPR, TAIL>(hn + row, v, t, D);
      yv[v] = load8<TPR, TAIL>(dy + row, v, t, D);
      if (o) ov[v] = load8<TPR, TAIL>(o + row, v, t, D);
      if (dhn) dv[v] = load8<TPR, TAIL>(dhn + row, v, t, D);
      if (elem) gv[v] = load8<TPR, TAIL>(static_cast<const uint16_t*>(n.gate) + row, v, t, D);
    }
  };
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t m = (int64_t)blockIdx.x * G + grp;
  if (prefetches(NV) && m < n.M) load_row(m);
  int par = 0;
  // the rows of a group that is a whole workgroup are the same for all its
  // threads; a wave's own rows need no barrier
  for (; m < n.M; m += step, par ^= 1) {
    const int64_t row = m * D;
    if (!prefetches(NV)) load_row(m);
    Raw8<R> h_[NV], d_[NV];
    Raw8<uint16_t> y_[NV], o_[NV], g_[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      in_place<TPR, TAIL>(hv[v], v, t, D);
      in_place<TPR, TAIL>(yv[v], v, t, D);
      if (dhn) in_place<TPR, TAIL>(dv[v], v, t, D);
      if (o) in_place<TPR, TAIL>(ov[v], v, t, D);
      if (elem) in_place<TPR, TAIL>(gv[v], v, t, D);
      h_[v] = hv[v];
      d_[v] = dv[v];
      y_[v] = yv[v];
      o_[v] = ov[v];
      g_[v] = gv[v];
    }
    const float grow = rowg ? n.scale * load_f32(static_cast<const uint16_t*>(n.gate) + m) : n.scale;
    if (prefetches(NV) && m + step < n.M) load_row(m + step);
    float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!KEEP) w2 = lds.param(n, 0, n.w_pre, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = h_[v].get(j);
        q[0] = __builtin_fmaf(x, x, q[0]);
        q[1] = __builtin_fmaf(y_[v].get(j) * w2.get(n.w32, j), x, q[1]);
        if (post) q[2] = __builtin_fmaf(o_[v].get(j), o_[v].get(j), q[2]);
      }
    }
    row_sums<TPR, 3>(q, s[par][0]);
    if (!KEEP) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        as_loaded(h_[v]);
        as_loaded(y_[v]);
        as_loaded(o_[v]);
      }
    }
    const float r2 = inv_sqrt(q[0] * rD + n.eps);
    const float c2 = q[1] * r2 * rD * r2;  // r2 mean(dn n)
    const float r1 = post ? inv_sqrt(q[2] * rD + n.eps) : 1.f;
    if (SUMS == kSumsNone && stats && t == 0) stats[m] = f32x4{r2, c2, r1, grow};
    float d[NV][8], e[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float out[8];
      if (!KEEP) w2 = lds.param(n, 0, n.w_pre, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = h_[v].get(j), g = y_[v].get(j);
        const float dn = g * w2.get(n.w32, j);
        out[j] = d[v][j] = __builtin_fmaf(r2, dn - x * c2, d_[v].get(j));
        if (REGS) sp[v][j] = __builtin_fmaf(g, x * r2, sp[v][j]);
        if (SUMS == kSumsLds) sp[v][j] = g * (x * r2);
      }
      if (SUMS == kSumsLds) lds.add(0, sp[v]);
      store8<TPR, TAIL>(dh + row, v, t, D, out);
    }
    if (!o) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!KEEP && post) w1 = lds.param(n, 1, n.w_post, v);
      if (!KEEP && chan) gc = lds.param(n, 2, n.gate, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // d becomes dq (or a, without a post norm)
        const float x = o_[v].get(j) * r1, wp = post ? w1.get(n.w32, j) : 1.f;
        const float base = d[v][j];
        float a = base * grow;
        if (chan) a *= gc.get(n.w32, j);
        if (elem) a *= g_[v].get(j);
        d[v][j] = a * wp;
        e[0] = __builtin_fmaf(a * wp, x, e[0]);
        if (rowg) e[1] = __builtin_fmaf(base * n.scale, x * wp, e[1]);
        if (REGS) {
          so[v][j] = __builtin_fmaf(a, x, so[v][j]);
          if (chan) sg[v][j] = __builtin_fmaf(base * n.scale, x * wp, sg[v][j]);
        }
        if (SUMS == kSumsLds) {
          so[v][j] = a * x;
          if (chan) sg[v][j] = base * n.scale * (x * wp);
        }
        if (elem) g_[v].put(j, base * n.scale * (x * wp));
      }
      if (SUMS == kSumsLds) {
        lds.add(1, so[v]);
        if (chan) lds.add(2, sg[v]);
      }
    }
    if (post || rowg) row_sums<TPR, 2>(e, s[par][1]);
    if (!KEEP) {
#pragma unroll
      for (int v = 0; v < NV; ++v) as_loaded(o_[v]);
    }
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
      store8<TPR, TAIL>(dout + row, v, t, D, out);
      if (elem && dgate) store8<TPR, TAIL>(static_cast<uint16_t*>(dgate) + row, v, t, D, dg);
    }
  }
  if constexpr (SUMS == kSumsLds) {
    float* dst = part + (int64_t)blockIdx.x * 3 * D;
#pragma unroll
    for (int k = 0; k < 3; ++k) lds.store(k, dst + k * D, D);
  }
  if constexpr (REGS) {
    float* dst = part + (int64_t)blockIdx.x * 3 * D;
    if constexpr (G == 1) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        store8<TPR, TAIL>(dst, v, t, D, sp[v]);
        store8<TPR, TAIL>(dst + D, v, t, D, so[v]);
        store8<TPR, TAIL>(dst + 2 * D, v, t, D, sg[v]);
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
        const int c = column<TPR>(l / TPR / 8, l % TPR) + l / TPR % 8;
        if (c < D) dst[which * D + c] = x;
      }
    }
  }
}

// The column sums of rows past kSumCols columns, whose threads have no
// registers to keep them beside a row: from the rows again and their stats
// (r2, r2 mean(dn n), r1, scale times the row's gate).  Workgroup (x, z):
// columns 8 (256 x + thread) .. + 7, rows z, z + S, ...; part as above.  It reads
// everything a second time: 2048 x 16384 with every gradient takes 269 us (3.0
// TB/s of what both passes move); with the sums beside the rows in spilled
// registers 618.  Up to 8192 columns LDS holds them (4096 x 8192: 113 us, in this
// pass 170).
template <bool TAIL, typename R>
__global__ __launch_bounds__(256) void k_norm_columns(
    NormArgs n, const uint16_t* __restrict__ dy, const R* __restrict__ dhn,
    const R* __restrict__ hn, const uint16_t* __restrict__ o, const f32x4* __restrict__ stats,
    float* __restrict__ part) {
  const int t = blockIdx.x * 256 + threadIdx.x, D = n.D;
  const bool post = n.w_post != nullptr, chan = n.gate_kind == kGateChannel,
             elem = n.gate_kind == kGateElement;
  auto param = [&](const void* w) { return load_param<1, TAIL>(w, n.w32, 0, t, D); };
  Param8 w1, w2 = param(n.w_pre), gc;
  if (post) w1 = param(n.w_post);
  if (chan) gc = param(n.gate);
  float sp[8] = {}, so[8] = {}, sg[8] = {};
  for (int64_t m = blockIdx.y; m < n.M; m += gridDim.y) {
    const int64_t row = m * D;
    const f32x4 st = stats[m];
    Raw8<R> h = load8<1, TAIL>(hn + row, 0, t, D);
    Raw8<uint16_t> y = load8<1, TAIL>(dy + row, 0, t, D);
    Raw8<R> d;
    Raw8<uint16_t> ov, g;
    if (dhn) d = load8<1, TAIL>(dhn + row, 0, t, D);
    if (o) ov = load8<1, TAIL>(o + row, 0, t, D);
    if (elem) g = load8<1, TAIL>(static_cast<const uint16_t*>(n.gate) + row, 0, t, D);
    in_place<1, TAIL>(h, 0, t, D);
    in_place<1, TAIL>(y, 0, t, D);
    in_place<1, TAIL>(d, 0, t, D);
    in_place<1, TAIL>(ov, 0, t, D);
    in_place<1, TAIL>(g, 0, t, D);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = h.get(j), dn = y.get(j) * w2.get(n.w32, j);
      const float base = __builtin_fmaf(st[0], dn - x * st[1], d.get(j));
      sp[j] = __builtin_fmaf(y.get(j), x * st[0], sp[j]);
      if (!o) continue;
      const float q = ov.get(j) * st[2];
      float a = base * st[3];
      if (chan) a *= gc.get(n.w32, j);
      if (elem) a *= g.get(j);
      so[j] = __builtin_fmaf(a, q, so[j]);
      if (chan) sg[j] = __builtin_fmaf(base * n.scale, post ? q * w1.get(n.w32, j) : q, sg[j]);
    }
  }
  float* dst = part + (int64_t)blockIdx.y * 3 * D;
  store8<1, TAIL>(dst, 0, t, D, sp);
  store8<1, TAIL>(dst + D, 0, t, D, so);
  store8<1, TAIL>(dst + 2 * D, 0, t, D, sg);
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

// Workgroups that stay resident on 256 compute units when their registers leave
// room for `waves` waves on each: 20 in the forward, 16 in the backward, 12 with
// column sums (10 taken: fewer partial sums).  A launch takes no other number,
// or the last ones run alone: 8192 x 2560 with 409 workgroups 78 us, with 512
// 66.
int64_t resident(int waves, int threads) {
  return 256 * std::max(1, waves / (threads / 64));
}
constexpr int kFwdWaves = 20, kBwdWaves = 16, kSumWaves = 10;
// Columns up to which a row's threads keep the column sums.
constexpr int64_t kSumCols = 8192;
constexpr int kColumnSlices = 64;

NormArgs args_of(const BlockNorm& n) {
  return NormArgs{n.M, (int)n.D, n.w_pre, n.w_post, n.gate, n.w32, n.gate_kind, n.scale, n.eps};
}

// Threads of a row: as many as hold it in one vector each; two past 8192
// columns.
int row_threads(int64_t D) {
  int t = 64;
  while (t < 1024 && 8 * t < D) t *= 2;
  return t;
}

// Calls f<TPR, NV>() for the row length D.
template <typename F>
hipError_t by_columns(int64_t D, F&& f) {
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  switch (row_threads(D)) {
    case 64: return f(std::integral_constant<int, 64>{}, I1{});
    case 128: return f(std::integral_constant<int, 128>{}, I1{});
    case 256: return f(std::integral_constant<int, 256>{}, I1{});
    case 512: return f(std::integral_constant<int, 512>{}, I1{});
  }
  using T1024 = std::integral_constant<int, 1024>;
  return D <= 8192 ? f(T1024{}, I1{}) : f(T1024{}, I2{});
}

// Launches a kernel with that much LDS beside its own.
template <typename... P, typename... A>
hipError_t run(void (*f)(P...), dim3 grid, int threads, size_t lds, hipStream_t st, A... args) {
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kSlotBytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(f, grid, dim3(threads), lds, st, args...);
  return hipGetLastError();
}

// Threads of a workgroup for the row length D.
template <int TPR, int NV>
int threads_of(int64_t D) {
  return TPR == 64 || NV > 1 ? group_threads(TPR) : (int)((D + 511) / 512 * 64);
}

template <typename R>
hipError_t norm_fwd(const BlockNorm& n, const void* h, const uint16_t* o, void* h_new, uint16_t* y,
                    int8_t* codes, uint8_t* exps, hipStream_t st) {
  return by_columns(n.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int G = group_threads(TPR) / TPR;
    const int T = threads_of<TPR, NV>(n.D);
    const int64_t groups = (n.M + G - 1) / G;
    // (two rounds of them run as fast, and end more evenly)
    const int64_t wgs = resident(kFwdWaves, T) * (T > 512 ? 1 : 2);
    const dim3 grid((unsigned)std::min(groups, wgs));
    const NormArgs a = args_of(n);
    const Slots slots = slots_of(n, keeps(TPR, NV), {false, false, false}, T, NV);
    const size_t lds = (size_t)slots.count * 16 * T * NV;
    const R* hp = static_cast<const R*>(h);
    R* hn = static_cast<R*>(h_new);
    hipError_t e;
    if (n.D % 8 == 0)
      e = run(k_norm_fwd<TPR, NV, false, R>, grid, T, lds, st, a, slots, hp, o, hn, y, codes, exps);
    else
      e = run(k_norm_fwd<TPR, NV, true, R>, grid, T, lds, st, a, slots, hp, o, hn, y, codes, exps);
    return e;
  });
}

template <typename R>
hipError_t norm_bwd(const BlockNorm& n, const uint16_t* dy, const void* dh_new, const void* h_new,
                    const uint16_t* o, void* dh, uint16_t* dout, void* dgate, float* part,
                    void* stats, hipStream_t st) {
  const NormArgs a = args_of(n);
  const R *dp = static_cast<const R*>(dh_new), *hp = static_cast<const R*>(h_new);
  R* out = static_cast<R*>(dh);
  f32x4* rows = static_cast<f32x4*>(stats);
  hipError_t e = by_columns(n.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int G = group_threads(TPR) / TPR;
    const int T = threads_of<TPR, NV>(n.D);
    const int64_t groups = (n.M + G - 1) / G;
    auto launch = [&](auto sums, int64_t blocks) {
      constexpr int SUMS = decltype(sums)::value;
      const dim3 grid((unsigned)blocks);
      constexpr bool in_lds = SUMS == kSumsLds;
      const Slots slots =
          slots_of(n, keeps(TPR, NV), {in_lds, in_lds && n.w_post, in_lds && n.gate_kind == kGateChannel},
                   T, NV);
      const size_t lds = (size_t)slots.count * 16 * T * NV;
      return n.D % 8 == 0 ? run(k_norm_bwd<TPR, NV, false, SUMS, R>, grid, T, lds, st, a, slots, dy,
                                dp, hp, o, out, dout, dgate, part, rows)
                          : run(k_norm_bwd<TPR, NV, true, SUMS, R>, grid, T, lds, st, a, slots, dy,
                                dp, hp, o, out, dout, dgate, part, rows);
    };
    using Regs = std::integral_constant<int, kSumsRegs>;
    using InLds = std::integral_constant<int, kSumsLds>;
    if constexpr (NV == 1) {
      if (part)
        return launch(std::conditional_t<(TPR < 1024), Regs, InLds>{}, block_norm_slices(n.M, n.D));
    }
    return launch(std::integral_constant<int, kSumsNone>{},
                  std::min(groups, resident(kBwdWaves, T)));
  });
  if (e != hipSuccess || !part || n.D <= kSumCols) return e;
  const dim3 grid((unsigned)((n.D + 2047) / 2048), (unsigned)block_norm_slices(n.M, n.D));
  if (n.D % 8 == 0)
    hipLaunchKernelGGL((k_norm_columns<false, R>), grid, dim3(256), 0, st, a, dy, dp, hp, o, rows,
                       part);
  else
    hipLaunchKernelGGL((k_norm_columns<true, R>), grid, dim3(256), 0, st, a, dy, dp, hp, o, rows,
                       part);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNorm& n, const void* h, const uint16_t* o, void* h_new,
                                 uint16_t* y, int8_t* codes, uint8_t* exps, hipStream_t st) {
  if (n.M == 0) return hipSuccess;
  return n.res32 ? norm_fwd<float>(n, h, o, h_new, y, codes, exps, st)
                 : norm_fwd<uint16_t>(n, h, o, h_new, y, codes, exps, st);
}

int block_norm_slices(int64_t M, int64_t D) {
  if (D > kSumCols)
    return (int)std::min<int64_t>(M, kColumnSlices * 16384 / (2048 * ((D + 2047) / 2048)));
  const int64_t T = D <= 512 ? 256 : (D + 511) / 512 * 64, G = D <= 512 ? 4 : 1;
  return (int)std::min<int64_t>((M + G - 1) / G, resident(kSumWaves, (int)T));
}
int64_t block_norm_stats(int64_t M, int64_t D) { return D > kSumCols ? 4 * M : 0; }

hipError_t launch_block_norm_bwd(const BlockNorm& n, const uint16_t* dy, const void* dh_new,
                                 const void* h_new, const uint16_t* o, void* dh, uint16_t* dout,
                                 void* dgate, float* dw_post, float* dw_pre, float* part,
                                 float* stats, hipStream_t st) {
  if (n.M == 0) return hipSuccess;
  hipError_t e =
      n.res32 ? norm_bwd<float>(n, dy, dh_new, h_new, o, dh, dout, dgate, part, stats, st)
              : norm_bwd<uint16_t>(n, dy, dh_new, h_new, o, dh, dout, dgate, part, stats, st);
  if (e != hipSuccess || !part) return e;
  float* dg = n.gate_kind == kGateChannel ? static_cast<float*>(dgate) : nullptr;
  hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)((3 * n.D + 63) / 64)), dim3(64 * kSumGroups), 0,
                     st, part, block_norm_slices(n.M, n.D), (int)n.D, dw_pre, dw_post, dg);
  return hipGetLastError();
}

}  // namespace qn
