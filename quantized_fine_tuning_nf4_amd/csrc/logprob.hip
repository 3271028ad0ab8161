// Log probabilities of given tokens with entropy and top alternatives, and
// their gradient (formulas in the header).
//
// With t_i = scale (x_i - m) <= 0, S = sum e^t_i and W = sum e^t_i t_i:
//   ln p_i = t_i - ln S,   H = ln S - W / S.
#include <cfloat>

#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// e^t (t <= 0; -inf gives 0)
__device__ __forceinline__ float exp_of(float t) { return __builtin_amdgcn_exp2f(t * kLog2e); }
// ln s (0 gives -inf)
__device__ __forceinline__ float ln_of(float s) { return __builtin_amdgcn_logf(s) * kLn2; }

__device__ __forceinline__ float group_sum(float x, float* s) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  x = s[0] + s[1] + s[2] + s[3];
  __syncthreads();
  return x;
}

// One workgroup per row: the maximum, then the sums, then one pass per
// alternative (the largest logit below the last one taken).
template <typename L>
__global__ __launch_bounds__(kThreads) void k_logprobs_fwd(
    const L* __restrict__ x, int64_t V, int64_t ld, const int64_t* __restrict__ targets,
    float scale, int k, float* __restrict__ logp, float* __restrict__ entropy,
    float* __restrict__ stats, float* __restrict__ top_logp, int32_t* __restrict__ top_ids) {
  __shared__ float s[4];
  __shared__ float sv[kThreads];
  __shared__ int si[kThreads];
  const int64_t row = blockIdx.x;
  const L* p = x + row * ld;
  const int tid = threadIdx.x;
  float m = -FLT_MAX;
  for (int64_t i = tid; i < V; i += kThreads) m = fmaxf(m, load_f32(p + i));
  sv[tid] = m;
  __syncthreads();
  for (int o = kThreads / 2; o >= 1; o >>= 1) {
    if (tid < o) sv[tid] = fmaxf(sv[tid], sv[tid + o]);
    __syncthreads();
  }
  m = sv[0];
  __syncthreads();
  float S = 0.f, W = 0.f;
  for (int64_t i = tid; i < V; i += kThreads) {
    const float t = (load_f32(p + i) - m) * scale, e = exp_of(t);
    S += e;
    W = __builtin_fmaf(e, fmaxf(t, -1e30f), W);
  }
  S = group_sum(S, s);
  W = group_sum(W, s);
  const float lnS = ln_of(S);
  if (tid == 0) {
    entropy[row] = S == 0.f ? 0.f : lnS - W / S;
    stats[2 * row] = m;
    stats[2 * row + 1] = lnS;
    if (logp) {
      const int64_t t = targets[row];
      float v = 0.f;
      if (t >= V)
        v = __builtin_nanf("");
      else if (t >= 0)
        v = S == 0.f ? -__builtin_inff() : (load_f32(p + t) - m) * scale - lnS;
      logp[row] = v;
    }
  }
  float lv = __builtin_inff();
  int li = -1;
  for (int j = 0; j < k; ++j) {
    float bv = -__builtin_inff();
    int bi = -1;
    for (int64_t i = tid; i < V; i += kThreads) {
      const float v = load_f32(p + i);
      if ((v < lv || (v == lv && (int)i > li)) && v > bv) {
        bv = v;
        bi = (int)i;
      }
    }
    sv[tid] = bv;
    si[tid] = bi;
    __syncthreads();
    for (int o = kThreads / 2; o >= 1; o >>= 1) {
      if (tid < o) {
        const float v = sv[tid + o];
        const int i = si[tid + o];
        if (i >= 0 && (si[tid] < 0 || v > sv[tid] || (v == sv[tid] && i < si[tid]))) {
          sv[tid] = v;
          si[tid] = i;
        }
      }
      __syncthreads();
    }
    lv = sv[0];
    li = si[0];
    __syncthreads();
    if (tid == 0) {
      top_ids[row * k + j] = li;
      top_logp[row * k + j] = li < 0 ? lv : (lv - m) * scale - lnS;
    }
  }
}

template <typename L>
__global__ __launch_bounds__(kThreads) void k_logprobs_bwd(
    const L* x, int64_t T, int64_t V, int64_t ld, const int64_t* __restrict__ targets, float scale,
    const float* __restrict__ stats, const float* __restrict__ entropy,
    const float* __restrict__ dlogp, const float* __restrict__ dent, L* dx, int64_t ldd) {
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x) {
    const float m = stats[2 * row], lnS = stats[2 * row + 1];
    const int64_t t = targets ? targets[row] : -1;
    const float g = dlogp && t >= 0 && t < V ? dlogp[row] : 0.f;
    const float d = dent ? dent[row] : 0.f, H = dent ? entropy[row] : 0.f;
    for (int64_t i = threadIdx.x; i < V; i += kThreads) {
      float v = 0.f;
      if (lnS != -__builtin_inff()) {
        const float lp = (load_f32(x + row * ld + i) - m) * scale - lnS, q = exp_of(lp);
        v = (i == t ? g : 0.f) - g * q;
        v -= d * q * (fmaxf(lp, -1e30f) + H);
      }
      store_f32(dx + row * ldd + i, v * scale);
    }
  }
}

}  // namespace

hipError_t launch_logprobs_fwd(const void* x, bool f32, int64_t T, int64_t V, int64_t ld,
                               const int64_t* targets, float scale, int k, float* logp,
                               float* entropy, float* stats, float* top_logp, int32_t* top_ids,
                               hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (f32)
    hipLaunchKernelGGL(k_logprobs_fwd<float>, dim3((unsigned)T), dim3(kThreads), 0, st,
                       static_cast<const float*>(x), V, ld, targets, scale, k, logp, entropy,
                       stats, top_logp, top_ids);
  else
    hipLaunchKernelGGL(k_logprobs_fwd<uint16_t>, dim3((unsigned)T), dim3(kThreads), 0, st,
                       static_cast<const uint16_t*>(x), V, ld, targets, scale, k, logp, entropy,
                       stats, top_logp, top_ids);
  return hipGetLastError();
}

hipError_t launch_logprobs_bwd(const void* x, bool f32, int64_t T, int64_t V, int64_t ld,
                               const int64_t* targets, float scale, const float* stats,
                               const float* entropy, const float* dlogp, const float* dent,
                               void* dx, int64_t ldd, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const dim3 grid((unsigned)(T < 65536 ? T : 65536));
  if (f32)
    hipLaunchKernelGGL(k_logprobs_bwd<float>, grid, dim3(kThreads), 0, st,
                       static_cast<const float*>(x), T, V, ld, targets, scale, stats, entropy,
                       dlogp, dent, static_cast<float*>(dx), ldd);
  else
    hipLaunchKernelGGL(k_logprobs_bwd<uint16_t>, grid, dim3(kThreads), 0, st,
                       static_cast<const uint16_t*>(x), T, V, ld, targets, scale, stats, entropy,
                       dlogp, dent, static_cast<uint16_t*>(dx), ldd);
  return hipGetLastError();
}

}  // namespace qn
