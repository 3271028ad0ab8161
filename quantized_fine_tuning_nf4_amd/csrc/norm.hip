// Norms before and after a block, fused with its gate and residual scale
// (formulas in the header), and their gradients.
//
// Backward, with n = h' r2, q = o r1 (r1, r2 the reciprocal root mean squares):
//   dn = dy w_pre            dh = dh' + r2 (dn - n mean(dn n))
//   a  = scale gate dh       dgate = scale p dh (summed to the gate's shape)
//   dq = a w_post            do = r1 (dq - q mean(dq q))
//   dw_pre = sum_m dy n      dw_post = sum_m a q
#include <algorithm>

#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

constexpr int kThreads = 256;

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ float group_sum(float x, float* s) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  x = s[0] + s[1] + s[2] + s[3];
  __syncthreads();
  return x;
}

struct NormArgs {
  int64_t M, D;
  const void *w_pre, *w_post, *gate;
  bool w32;
  int gate_kind;
  float scale, eps;
};

__device__ __forceinline__ float weight_at(const void* w, bool w32, int64_t c) {
  return w32 ? static_cast<const float*>(w)[c] : load_f32(static_cast<const uint16_t*>(w) + c);
}
__device__ __forceinline__ float gate_at(const NormArgs& n, int64_t m, int64_t c) {
  if (n.gate_kind == 0) return 1.f;
  if (n.gate_kind == 1) return weight_at(n.gate, n.w32, c);
  return load_f32(static_cast<const uint16_t*>(n.gate) + (n.gate_kind == 2 ? m : m * n.D + c));
}

// One workgroup per row, its values read again for every pass.
template <typename R>
__global__ __launch_bounds__(kThreads) void k_norm_fwd(NormArgs n, const R* __restrict__ h,
                                                       const uint16_t* __restrict__ o,
                                                       R* __restrict__ hn, uint16_t* __restrict__ y) {
  __shared__ float s[4];
  const int64_t m = blockIdx.x, D = n.D, row = m * D;
  float r1 = 1.f;
  if (n.w_post) {
    float q = 0.f;
    for (int64_t c = threadIdx.x; c < D; c += kThreads) {
      const float v = load_f32(o + row + c);
      q = __builtin_fmaf(v, v, q);
    }
    r1 = 1.f / __builtin_sqrtf(group_sum(q, s) / (float)D + n.eps);
  }
  auto value = [&](int64_t c) {
    float v = load_f32(h + row + c);
    if (o) {
      float p = load_f32(o + row + c);
      if (n.w_post) p = p * r1 * weight_at(n.w_post, n.w32, c);
      v += n.scale * (gate_at(n, m, c) * p);
    }
    return v;
  };
  float q = 0.f;
  for (int64_t c = threadIdx.x; c < D; c += kThreads) {
    const float v = value(c);
    q = __builtin_fmaf(v, v, q);
  }
  const float r2 = 1.f / __builtin_sqrtf(group_sum(q, s) / (float)D + n.eps);
  for (int64_t c = threadIdx.x; c < D; c += kThreads) {
    const float v = value(c);
    if (o) store_f32(hn + row + c, v);
    y[row + c] = to_bf16(v * r2 * weight_at(n.w_pre, n.w32, c));
  }
}

// Workgroup z: rows z, z + S, ...; a thread keeps its columns' sums in its
// own places of part [S][3][D] (dw_pre, dw_post, channel dgate).
template <typename R>
__global__ __launch_bounds__(kThreads) void k_norm_bwd(
    NormArgs n, const uint16_t* __restrict__ dy, const R* __restrict__ dhn,
    const R* __restrict__ hn, const uint16_t* __restrict__ o, R* __restrict__ dh,
    uint16_t* __restrict__ dout, void* __restrict__ dgate, float* __restrict__ part) {
  __shared__ float s[4];
  const int64_t D = n.D;
  float* pp = part ? part + (int64_t)blockIdx.x * 3 * D : nullptr;
  if (pp)
    for (int64_t c = threadIdx.x; c < D; c += kThreads) pp[c] = pp[D + c] = pp[2 * D + c] = 0.f;
  for (int64_t m = blockIdx.x; m < n.M; m += gridDim.x) {
    const int64_t row = m * D;
    float q2 = 0.f, d2 = 0.f, q1 = 0.f;
    for (int64_t c = threadIdx.x; c < D; c += kThreads) {
      const float v = load_f32(hn + row + c);
      q2 = __builtin_fmaf(v, v, q2);
      d2 = __builtin_fmaf(load_f32(dy + row + c) * weight_at(n.w_pre, n.w32, c), v, d2);
      if (n.w_post) {
        const float w = load_f32(o + row + c);
        q1 = __builtin_fmaf(w, w, q1);
      }
    }
    const float r2 = 1.f / __builtin_sqrtf(group_sum(q2, s) / (float)D + n.eps);
    const float k2 = group_sum(d2, s) * r2 / (float)D;  // mean(dn n)
    const float r1 = n.w_post ? 1.f / __builtin_sqrtf(group_sum(q1, s) / (float)D + n.eps) : 1.f;
    auto dh_at = [&](int64_t c) {
      const float v = load_f32(hn + row + c);
      const float dn = load_f32(dy + row + c) * weight_at(n.w_pre, n.w32, c);
      return (dhn ? load_f32(dhn + row + c) : 0.f) + r2 * (dn - v * r2 * k2);
    };
    float k1 = 0.f, gr = 0.f;
    if (o) {
      float d1 = 0.f, dg = 0.f;
      for (int64_t c = threadIdx.x; c < D; c += kThreads) {
        const float g = dh_at(c) * n.scale, w = load_f32(o + row + c);
        const float wp = n.w_post ? weight_at(n.w_post, n.w32, c) : 1.f;
        d1 = __builtin_fmaf(g * gate_at(n, m, c) * wp, w, d1);
        dg = __builtin_fmaf(g * wp, w * r1, dg);
      }
      k1 = group_sum(d1, s) * r1 / (float)D;  // mean(dq q)
      gr = group_sum(dg, s);
      if (dgate && n.gate_kind == 2 && threadIdx.x == 0) static_cast<float*>(dgate)[m] = gr;
    }
    for (int64_t c = threadIdx.x; c < D; c += kThreads) {
      const float d = dh_at(c);
      if (pp) pp[c] = __builtin_fmaf(load_f32(dy + row + c), load_f32(hn + row + c) * r2, pp[c]);
      if (o) {
        const float qv = load_f32(o + row + c) * r1, ga = gate_at(n, m, c);
        const float wp = n.w_post ? weight_at(n.w_post, n.w32, c) : 1.f;
        const float a = n.scale * d * ga;
        float w = a;
        if (n.w_post) w = r1 * (a * wp - qv * k1);
        dout[row + c] = to_bf16(w);
        const float dg = n.scale * d * qv * wp;
        if (dgate && n.gate_kind == 3) static_cast<uint16_t*>(dgate)[row + c] = to_bf16(dg);
        if (pp) {
          pp[D + c] = __builtin_fmaf(a, qv, pp[D + c]);
          pp[2 * D + c] += dg;
        }
      }
      store_f32(dh + row + c, d);
    }
  }
}

// out_j[c] = sum over the slices of part[z][j][c], in slice order.
__global__ __launch_bounds__(kThreads) void k_norm_sums(const float* __restrict__ part, int S,
                                                        int64_t D, float* __restrict__ o0,
                                                        float* __restrict__ o1,
                                                        float* __restrict__ o2) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= 3 * D) return;
  float* out = i < D ? o0 : i < 2 * D ? o1 : o2;
  if (!out) return;
  out[i % D] = slice_sum(part, 3 * D, S, i);
}

NormArgs args_of(const BlockNorm& n) {
  return NormArgs{n.M, n.D, n.w_pre, n.w_post, n.gate, n.w32, n.gate_kind, n.scale, n.eps};
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNorm& n, const void* h, const uint16_t* o, void* h_new,
                                 uint16_t* y, int8_t* codes, uint8_t* exps, hipStream_t st) {
  if (n.M == 0) return hipSuccess;
  const dim3 grid((unsigned)n.M);
  if (n.res32)
    hipLaunchKernelGGL(k_norm_fwd<float>, grid, dim3(kThreads), 0, st, args_of(n),
                       static_cast<const float*>(h), o, static_cast<float*>(h_new), y);
  else
    hipLaunchKernelGGL(k_norm_fwd<uint16_t>, grid, dim3(kThreads), 0, st, args_of(n),
                       static_cast<const uint16_t*>(h), o, static_cast<uint16_t*>(h_new), y);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && codes) e = launch_act8_pack(y, n.M, n.D, codes, exps, st);
  return e;
}

int block_norm_slices(int64_t M, int64_t D) {
  (void)D;
  return (int)std::min<int64_t>(std::max<int64_t>(M, 1), 512);
}

hipError_t launch_block_norm_bwd(const BlockNorm& n, const uint16_t* dy, const void* dh_new,
                                 const void* h_new, const uint16_t* o, void* dh, uint16_t* dout,
                                 void* dgate, float* dw_post, float* dw_pre, float* part,
                                 hipStream_t st) {
  const int S = part ? block_norm_slices(n.M, n.D) : (int)std::min<int64_t>(n.M, 4096);
  if (n.M > 0) {
    if (n.res32)
      hipLaunchKernelGGL(k_norm_bwd<float>, dim3(S), dim3(kThreads), 0, st, args_of(n), dy,
                         static_cast<const float*>(dh_new), static_cast<const float*>(h_new), o,
                         static_cast<float*>(dh), dout, dgate, part);
    else
      hipLaunchKernelGGL(k_norm_bwd<uint16_t>, dim3(S), dim3(kThreads), 0, st, args_of(n), dy,
                         static_cast<const uint16_t*>(dh_new), static_cast<const uint16_t*>(h_new),
                         o, static_cast<uint16_t*>(dh), dout, dgate, part);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part) return e;
  float* dg = n.gate_kind == 1 ? static_cast<float*>(dgate) : nullptr;
  hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)((3 * n.D + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, st, part, S, n.D, dw_pre, dw_post, dg);
  return hipGetLastError();
}

}  // namespace qn
