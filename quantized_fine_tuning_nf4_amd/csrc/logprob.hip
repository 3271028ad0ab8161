// Log probabilities of given tokens with entropy and top alternatives, and
// their gradient (formulas in the header).
//
// With t_i = scale (x_i - m) log2 e <= 0, S = sum 2^t_i and W = sum 2^t_i t_i:
//   log2 p_i = t_i - log2 S,   H = (log2 S - W / S) ln 2.
// A row is read once: every lane keeps a running maximum m of what it has
// seen and S and W with respect to it; where m moves by d <= 0 (in the same
// units), W becomes 2^d (W + S d) and S becomes 2^d S.  Lanes, waves and
// slices of a row are joined by the same rule.
//
// Alternatives are ordered by one 64-bit number each: the logit as an ordered
// whole number above the complement of its index, so that of equal logits the
// lower index is the larger.  A wave keeps its best ones sorted across its
// lanes.  A logit that is no better than the last of them is dismissed with
// one comparison for each lane's vector; what remains (k + k ln(n / k) of n
// logits in random order) is inserted by a count and a shift across lanes.
// Sorted lists of 32 are joined by bitonic merges.
#include <algorithm>
#include <cfloat>

#include "launch_rows.h"
#include "qn_device.h"
#include "qn_internal.h"

namespace qn {
namespace {

constexpr int kThreads = 256;
constexpr int kU = 4;     // vectors of a thread in flight
constexpr int kList = 32; // alternatives of a list
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
// below any t whose 2^t is not zero, and finite: 0 times it is 0
constexpr float kFarBelow = -1e4f;

// scale log2 e, finite for every scale: 0 times it, a largest logit's, is 0
__device__ __forceinline__ float base2_scale(float scale) {
  return fminf(scale * kLog2e, FLT_MAX);
}
__device__ __forceinline__ float exp2_of(float t) { return __builtin_amdgcn_exp2f(t); }
__device__ __forceinline__ float log2_of(float s) { return __builtin_amdgcn_logf(s); }

// 16 bytes of logits, at any element.
template <typename L>
struct Vec;
template <>
struct Vec<uint16_t> {
  typedef u32x4 any __attribute__((aligned(2)));
  static constexpr int N = 8;
  u32x4 v;
  __device__ __forceinline__ float get(int j) const {
    return (j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
  }
  __device__ __forceinline__ void none() {  // -inf
    v = u32x4{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
  }
  __device__ __forceinline__ void put(int j, uint16_t x) {
    v[j >> 1] = (j & 1) ? (v[j >> 1] & 0xffffu) | ((uint32_t)x << 16)
                        : (v[j >> 1] & 0xffff0000u) | x;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    v = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
              pack_bf16x2(x[6], x[7])};
  }
  __device__ __forceinline__ uint16_t raw(int j) const {
    return (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
  }
};
template <>
struct Vec<float> {
  typedef f32x4 any __attribute__((aligned(4)));
  static constexpr int N = 4;
  f32x4 v;
  __device__ __forceinline__ float get(int j) const { return v[j]; }
  __device__ __forceinline__ void none() {
    const float x = -__builtin_inff();
    v = f32x4{x, x, x, x};
  }
  __device__ __forceinline__ void put(int j, float x) { v[j] = x; }
  __device__ __forceinline__ void set(const float (&x)[4]) { v = f32x4{x[0], x[1], x[2], x[3]}; }
  __device__ __forceinline__ float raw(int j) const { return v[j]; }
};

// Logits i .. of a row, -inf from `end` on.
template <typename L>
__device__ __forceinline__ Vec<L> load_part(const L* p, int64_t i, int64_t end) {
  Vec<L> r;
  r.none();
  if (i + Vec<L>::N <= end) {
    r.v = *reinterpret_cast<const typename Vec<L>::any*>(p + i);
  } else {
#pragma unroll
    for (int j = 0; j < Vec<L>::N - 1; ++j)
      if (i + j < end) r.put(j, p[i + j]);
  }
  return r;
}

// What a lane, wave, workgroup or slice knows of a row.
struct Stat {
  float m, S, W;
};
// The same with respect to a maximum mx >= a.m.
__device__ __forceinline__ void rebase(Stat& a, float mx, float k2) {
  const float d = fmaxf((a.m - mx) * k2, kFarBelow), f = exp2_of(d);
  a.W = a.S > 0.f ? f * __builtin_fmaf(a.S, d, a.W) : 0.f;
  a.S *= f;
  a.m = mx;
}

__device__ __forceinline__ float wave_max(float x) {
  return as_f32(reduce_wave(as_u32(x), [](uint32_t a, uint32_t b) {
    return as_u32(fmaxf(as_f32(a), as_f32(b)));
  }));
}
__device__ __forceinline__ void wave_join(Stat& a, float k2) {
  rebase(a, wave_max(a.m), k2);
  a.S = wave_sum(a.S);
  a.W = wave_sum(a.W);
}

// ---- alternatives
typedef unsigned long long Key;  // 0: none
constexpr Key kNoKey = ((Key)0x007fffffu << 32) | 0xffffffffu;  // above every key of -inf

__device__ __forceinline__ uint32_t ordered(float x) {
  // -0 counts as 0, a NaN as -inf: none of the best, whatever the order in which
  // the waves' bars reach each other
  const uint32_t b = as_u32(fmaxf(x + 0.f, -__builtin_inff()));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ Key key_of(float x, uint32_t i) {
  return ((Key)ordered(x) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return as_f32((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ int key_index(Key k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint32_t read_lane(uint32_t x, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}
__device__ __forceinline__ Key read_lane(Key x, int lane) {
  return (Key)read_lane((uint32_t)x, lane) | ((Key)read_lane((uint32_t)(x >> 32), lane) << 32);
}

// A wave's sorted list (lane l: its l-th best) and the key that a logit has to
// pass to be one of its first k.
struct Best {
  Key mine = 0, bar = kNoKey;
  float bar_value = -__builtin_inff();

  __device__ __forceinline__ void raise(Key k) {
    bar = k;
    bar_value = key_value(k);
  }
  // One key for each lane.
  __device__ __forceinline__ void offer(Key x, int k) {
    uint64_t todo = __ballot(x > bar);
    while (todo) {
      const int from = __builtin_ctzll(todo);
      const Key c = read_lane(x, from);
      const int at = __builtin_popcountll(__ballot(mine > c));
      const int lane = threadIdx.x & 63;
      const Key up = (Key)dpp<0x138>((uint32_t)mine) |  // wave_shr:1
                     ((Key)dpp<0x138>((uint32_t)(mine >> 32)) << 32);
      mine = lane < at ? mine : lane == at ? c : up;
      const Key last = read_lane(mine, k - 1);
      if (last > bar) raise(last);
      todo &= todo - 1;
      todo &= __ballot(x > bar);
    }
  }
  // Before anything was offered: tops holds the best of a few logits of each
  // lane of the workgroup's W waves, as ordered numbers.  The k-th largest of
  // 256 of them (each the best of W / 4 lanes) bounds the k-th best logit from
  // below; its leading 16 bits are enough (and all of a bf16), found bit by bit
  // from how many reach them.
  template <int W>
  __device__ __forceinline__ void start(const uint32_t* tops, int k) {
    uint32_t u[4] = {}, low = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) u[w & 3] = max(u[w & 3], tops[64 * w + (threadIdx.x & 63)]);
#pragma unroll
    for (int b = 31; b >= 16; --b) {
      const uint32_t c = low | (1u << b);
      int n = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) n += __builtin_popcountll(__ballot(u[w] >= c));
      if (n >= k) low = c;
    }
    at_least(low);
  }
  // k logits at least as large (as ordered numbers) are known.
  __device__ __forceinline__ void at_least(uint32_t low) {
    const Key b = (Key)low << 32;  // below every key of that value
    if (b > bar) raise(b);
  }
  __device__ __forceinline__ uint32_t known() const { return (uint32_t)(bar >> 32); }
};

// The value of the lane at distance D (lane ^ D), without a trip through LDS.
template <int D>
__device__ __forceinline__ uint32_t xor_lanes(uint32_t x) {
  if constexpr (D == 1) return dpp<kDppXor1>(x);
  if constexpr (D == 2) return dpp<kDppXor2>(x);
  if constexpr (D == 4) return dpp<0x1b>(dpp<kDppMirror8>(x));  // (i ^ 7) ^ 3
  if constexpr (D == 8) return dpp<0x128>(x);                   // row_ror:8
  if constexpr (D == 16) {
    auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return (threadIdx.x & 16) ? s[0] : s[1];
  }
  auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return (threadIdx.x & 32) ? s[0] : s[1];
}
template <int D>
__device__ __forceinline__ void merge_step(Key& x) {
  const Key y = (Key)xor_lanes<D>((uint32_t)x) | ((Key)xor_lanes<D>((uint32_t)(x >> 32)) << 32);
  const bool upper = (threadIdx.x & D) != 0;
  x = (y > x) != upper ? y : x;
}
// Two lists of 32, descending in lanes 0 .. 31 and ascending in 32 .. 63: all
// 64 in descending order.  (Equal keys, both "none", may go either way.)
__device__ __forceinline__ void merge_lists(Key& x) {
  merge_step<32>(x);
  merge_step<16>(x);
  merge_step<8>(x);
  merge_step<4>(x);
  merge_step<2>(x);
  merge_step<1>(x);
}
// The lists of N waves (a power of two), joined pairwise through LDS; the
// result is in wave 0's lanes 0 .. 31.
template <int N>
__device__ __forceinline__ void join_lists(Key& mine, Key (*s)[kList]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int h = N / 2; h >= 1; h /= 2) {
    if (wave >= h && wave < 2 * h && lane < kList) s[wave - h][lane] = mine;
    __syncthreads();
    if (wave < h) {
      if (lane >= kList) mine = s[wave][63 - lane];
      merge_lists(mine);
    }
    __syncthreads();
  }
}

struct RowOut {
  const int64_t* targets;
  float *logp, *entropy, *stats, *top_logp;
  int32_t* top_ids;
  int k;
  float scale;
};
// A row's results from its joined Stat, by the lanes of one wave; xt: the
// target's logit (read where 0 <= t < V).
__device__ __forceinline__ void write_row(const RowOut& r, int64_t row, const Stat& a, int64_t t,
                                          int64_t V, float xt, Key mine) {
  const int lane = threadIdx.x & 63;
  const float log2S = log2_of(a.S), lnS = log2S * kLn2;
  if (lane == 0) {
    r.entropy[row] = a.S == 0.f ? 0.f : (log2S - a.W / a.S) * kLn2;
    r.stats[2 * row] = a.m;
    r.stats[2 * row + 1] = lnS;
    if (r.logp) {
      float v = 0.f;
      if (t >= V)
        v = __builtin_nanf("");
      else if (t >= 0)
        v = a.S == 0.f ? -__builtin_inff() : (xt - a.m) * r.scale - lnS;
      r.logp[row] = v;
    }
  }
  if (lane < r.k) {
    const bool none = mine == 0;
    r.top_ids[row * r.k + lane] = none ? -1 : key_index(mine);
    r.top_logp[row * r.k + lane] =
        none ? -__builtin_inff() : (key_value(mine) - a.m) * r.scale - lnS;
  }
}

// Workgroup b of W waves: slice b % S of row b / S, U vectors a thread in flight.
// A slice's results go to parts and lists, or, when S is 1, straight to the
// outputs.
// Bound by HBM for many rows (8192 x 32000 bf16, 524 MB: 95.6 us, 5.5 TB/s, with
// the vector units at work nine tenths of the time; two passes over the row took
// 447 us), with alternatives by their bookkeeping (the same with top 20: 136 us)
// and for few rows by latency: one row of 131072 fp32 with top 20 takes 6.3 us and
// 3.5 in the join, 301 rows of 50021 fp32 with top 5 17.5 us (3.4 TB/s) and 4.0.
template <typename L, bool TOP, int W, int U>
__global__ __launch_bounds__(64 * W) void k_logprobs_fwd(const L* __restrict__ x, int64_t V,
                                                           int64_t ld, int S, int64_t slice,
                                                           RowOut out, Stat* __restrict__ parts,
                                                           Key* __restrict__ lists) {
  constexpr int N = Vec<L>::N;
  constexpr int64_t kStep = 64 * W * N;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t row = S == 1 ? (int64_t)blockIdx.x : (int64_t)(blockIdx.x / (unsigned)S);
  const int64_t z = blockIdx.x - row * S;
  const L* p = x + row * ld;
  const int64_t begin = z * slice, end = min(begin + slice, V);
  const float k2 = base2_scale(out.scale);
  int64_t t = -1;
  float xt = 0.f;
  if (S == 1 && out.logp) {
    t = out.targets[row];
    if (t >= 0 && t < V) xt = load_f32(p + t);
  }
  Stat a{-FLT_MAX, 0.f, 0.f};
  Best best;
  // what each wave's bar is by now: a logit below any of them is none of the
  // row's best.  Read and written without order: an old value only lets more
  // through.
  __shared__ uint32_t bars[W], tops[TOP ? 64 * W : 1];
  if constexpr (TOP) {
    if (tid < W) bars[tid] = 0u;
    __syncthreads();
  }
  auto take = [&](Vec<L>(&v)[U], int64_t i, bool first) {
    float top[U], mx;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      top[u] = v[u].get(0);
#pragma unroll
      for (int j = 1; j < N; ++j) top[u] = fmaxf(top[u], v[u].get(j));
    }
    mx = top[0];
#pragma unroll
    for (int u = 1; u < U; ++u) mx = fmaxf(mx, top[u]);
    if (__any(mx > a.m)) rebase(a, fmaxf(a.m, mx), k2);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float d = (v[u].get(j) - a.m) * k2, e = exp2_of(d);
        a.S += e;
        a.W = __builtin_fmaf(e, fmaxf(d, kFarBelow), a.W);
      }
    if constexpr (TOP) {
      if (first) {
        tops[tid] = ordered(mx);
        __syncthreads();
        best.template start<W>(tops, out.k);
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w)
          best.at_least(__builtin_amdgcn_readfirstlane(__hip_atomic_load(
              &bars[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)));
      }
      if (__any(mx >= best.bar_value)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (__any(top[u] >= best.bar_value)) {
#pragma unroll
            for (int j = 0; j < N; ++j)
              best.offer(key_of(v[u].get(j), (uint32_t)(i + u * kStep + j)), out.k);
          }
      }
      if (lane == 0)
        __hip_atomic_store(&bars[wave], best.known(), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  };
  int64_t i = begin + (int64_t)tid * N;
  for (int64_t b = begin; b < end; b += U * kStep, i += U * kStep) {
    Vec<L> v[U];
    if (b + U * kStep <= end) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u].v = *reinterpret_cast<const typename Vec<L>::any*>(p + i + u * kStep);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = load_part<L>(p, i + u * kStep, end);
    }
    take(v, i, b == begin);
  }
  wave_join(a, k2);
  __shared__ Stat s[W];
  __shared__ Key sk[TOP ? W / 2 : 1][kList];
  if (lane == 0) s[wave] = a;
  if constexpr (TOP) join_lists<W>(best.mine, sk);
  __syncthreads();
  if (wave != 0) return;
  a = lane < W ? s[lane] : Stat{-FLT_MAX, 0.f, 0.f};
  wave_join(a, k2);
  if (S == 1) {
    write_row(out, row, a, t, V, xt, best.mine);
    return;
  }
  if (lane == 0) parts[blockIdx.x] = a;
  if (TOP && lane < kList) lists[(int64_t)blockIdx.x * kList + lane] = best.mine;
}

// Joins the S slices of a row (S <= 64): workgroup of 64 W threads per row.
template <typename L, int W>
__global__ __launch_bounds__(64 * W) void k_logprobs_join(const L* __restrict__ x, int64_t V,
                                                          int64_t ld, int S, RowOut out,
                                                          const Stat* __restrict__ parts,
                                                          const Key* __restrict__ lists) {
  const int64_t row = blockIdx.x;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int64_t t = -1;
  float xt = 0.f;
  Stat a{-FLT_MAX, 0.f, 0.f};
  if (wave == 0) {
    if (lane < S) a = parts[row * S + lane];
    if (out.logp) {
      t = out.targets[row];
      if (t >= 0 && t < V) xt = load_f32(x + row * ld + t);
    }
  }
  Key mine = 0;
  if constexpr (W > 1) {
    __shared__ Key sk[W / 2][kList];
    // this wave's slices, two lists at a time
    const Key* l = lists + row * S * kList;
    for (int z = wave; z < S; z += W) {
      if (z == wave) {
        if (lane < kList) mine = l[z * kList + lane];
      } else {
        if (lane >= kList) mine = l[z * kList + 63 - lane];
        merge_lists(mine);
      }
    }
    join_lists<W>(mine, sk);
  }
  if (wave != 0) return;
  wave_join(a, base2_scale(out.scale));
  write_row(out, row, a, t, V, xt, mine);
}

// Workgroup b: chunk b % chunks of row b / chunks, kU vectors a thread, all
// loaded before the first is stored (the gradient may take the logits' place).
// Bound by HBM: 4096 x 131072 bf16, 2.15 GB, 368 us, 5.8 TB/s.
template <typename L>
__global__ __launch_bounds__(kThreads) void k_logprobs_bwd(
    const L* x, int64_t V, int64_t ld, unsigned chunks, const int64_t* __restrict__ targets,
    float scale, const float* __restrict__ stats, const float* __restrict__ entropy,
    const float* __restrict__ dlogp, const float* __restrict__ dent, L* dx, int64_t ldd) {
  constexpr int N = Vec<L>::N;
  const int64_t row = blockIdx.x / chunks;
  const int64_t begin = (int64_t)(blockIdx.x - (unsigned)row * chunks) * (kThreads * N * kU);
  const float m = stats[2 * row], lnS = stats[2 * row + 1];
  const int64_t t = targets ? targets[row] : -1;
  const float g = dlogp && t >= 0 && t < V ? dlogp[row] : 0.f;
  const float d = dent ? dent[row] : 0.f, H = dent ? entropy[row] : 0.f;
  const bool empty = lnS == -__builtin_inff();
  // scale p (-(g + d H) - d ln p)
  const float c0 = -scale * __builtin_fmaf(d, H, g), c1 = -scale * d;
  const L* p = x + row * ld;
  L* q = dx + row * ldd;
  const int64_t i0 = begin + (int64_t)threadIdx.x * N;
  Vec<L> v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) v[u] = load_part<L>(p, i0 + u * kThreads * N, V);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = i0 + u * kThreads * N;
    float o[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float lp = __builtin_fmaf(v[u].get(j) - m, scale, -lnS);
      const float pr = exp2_of(lp * kLog2e);
      o[j] = empty ? 0.f : pr * __builtin_fmaf(c1, fmaxf(lp, kFarBelow), c0);
    }
    if ((uint64_t)(t - i) < (uint64_t)N && !empty) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (i + j == t) o[j] += scale * g;
    }
    Vec<L> w;
    w.set(o);
    if (i + N <= V) {
      *reinterpret_cast<typename Vec<L>::any*>(q + i) = w.v;
    } else {
#pragma unroll
      for (int j = 0; j < N - 1; ++j)
        if (i + j < V) q[i + j] = w.raw(j);
    }
  }
}

// How a call reads its rows.  Many rows, or short ones: a workgroup of four
// waves each.  Up to 256 rows of up to 128 KB: a workgroup of 16 waves each (128
// rows of 32000 bf16 logits 5.4 us, in slices 8.0; but one row of 131072 fp32 10.8
// us, in slices 4.4: one compute unit reads no faster).  Other few rows: cut in
// slices that leave every thread of a small workgroup two vectors, at most 64,
// joined by a second launch.
constexpr int64_t kWideBytes = 128 * 1024;
constexpr int64_t kWideRows = 256;
constexpr int64_t kLeastSlice = 2 * kThreads * 8;
bool wide(int64_t T, int64_t V, bool f32) {
  return T <= kWideRows && V >= 2 * kLeastSlice && V * (f32 ? 4 : 2) <= kWideBytes;
}
int64_t slice_length(int64_t T, int64_t V, bool f32) {
  int64_t S = std::min<int64_t>((1024 + T - 1) / T, 64);
  S = std::min<int64_t>(S, V / kLeastSlice);
  if (S <= 1 || wide(T, V, f32)) return V;
  return ((V + S - 1) / S + 511) / 512 * 512;
}

template <typename L>
hipError_t logprobs_fwd(const L* x, int64_t T, int64_t V, int64_t ld, const RowOut& out, void* ws,
                        hipStream_t st) {
  constexpr bool f32 = sizeof(L) == 4;
  const int64_t slice = slice_length(T, V, f32);
  const int S = logprob_slices(T, V, f32);
  Stat* parts = static_cast<Stat*>(ws);
  Key* lists = reinterpret_cast<Key*>(static_cast<char*>(ws) + logprob_parts_bytes(T, S));
  const dim3 grid((unsigned)(T * S));
  auto launch = [&](auto f, int threads) {
    hipLaunchKernelGGL(f, grid, dim3(threads), 0, st, x, V, ld, S, slice, out, parts, lists);
    return hipGetLastError();
  };
  if (wide(T, V, f32))
    return out.k > 0 ? launch(k_logprobs_fwd<L, true, 16, kU>, 1024)
                     : launch(k_logprobs_fwd<L, false, 16, kU>, 1024);
  const hipError_t e = out.k > 0 ? launch(k_logprobs_fwd<L, true, 4, kU>, kThreads)
                                 : launch(k_logprobs_fwd<L, false, 4, kU>, kThreads);
  if (e != hipSuccess || S == 1) return e;
  if (out.k == 0)
    hipLaunchKernelGGL((k_logprobs_join<L, 1>), dim3((unsigned)T), dim3(64), 0, st, x, V, ld, S, out,
                       parts, lists);
  else if (S <= 4)
    hipLaunchKernelGGL((k_logprobs_join<L, 4>), dim3((unsigned)T), dim3(256), 0, st, x, V, ld, S,
                       out, parts, lists);
  else
    hipLaunchKernelGGL((k_logprobs_join<L, 16>), dim3((unsigned)T), dim3(1024), 0, st, x, V, ld, S,
                       out, parts, lists);
  return hipGetLastError();
}

}  // namespace

int logprob_slices(int64_t T, int64_t V, bool f32) {
  const int64_t slice = slice_length(T, V, f32);
  return (int)((V + slice - 1) / slice);
}
size_t logprob_parts_bytes(int64_t T, int S) { return ((size_t)T * S * sizeof(Stat) + 15) / 16 * 16; }
size_t logprob_workspace(int64_t T, int64_t V, bool f32, int k) {
  const int S = logprob_slices(T, V, f32);
  if (S == 1) return 0;
  return logprob_parts_bytes(T, S) + (k > 0 ? (size_t)T * S * kList * sizeof(Key) : 0);
}

hipError_t launch_logprobs_fwd(const void* x, bool f32, int64_t T, int64_t V, int64_t ld,
                               const int64_t* targets, float scale, int k, float* logp,
                               float* entropy, float* stats, float* top_logp, int32_t* top_ids,
                               void* ws, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const RowOut out{targets, logp, entropy, stats, top_logp, top_ids, k, scale};
  return f32 ? logprobs_fwd(static_cast<const float*>(x), T, V, ld, out, ws, st)
             : logprobs_fwd(static_cast<const uint16_t*>(x), T, V, ld, out, ws, st);
}

hipError_t launch_logprobs_bwd(const void* x, bool f32, int64_t T, int64_t V, int64_t ld,
                               const int64_t* targets, float scale, const float* stats,
                               const float* entropy, const float* dlogp, const float* dent,
                               void* dx, int64_t ldd, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const int64_t per = (int64_t)kThreads * kU * (f32 ? 4 : 8), chunks = (V + per - 1) / per;
  // rows whose work items a launch can count
  const int64_t most = rows_per_launch(chunks, kThreads);
  for (int64_t r = 0; r < T; r += most) {
    const dim3 grid((unsigned)(std::min<int64_t>(most, T - r) * chunks));
    const int64_t* tg = targets ? targets + r : nullptr;
    const float *en = entropy ? entropy + r : nullptr, *dl = dlogp ? dlogp + r : nullptr,
                *de = dent ? dent + r : nullptr;
    if (f32)
      hipLaunchKernelGGL(k_logprobs_bwd<float>, grid, dim3(kThreads), 0, st,
                         static_cast<const float*>(x) + r * ld, V, ld, (unsigned)chunks, tg, scale,
                         stats + 2 * r, en, dl, de, static_cast<float*>(dx) + r * ldd, ldd);
    else
      hipLaunchKernelGGL(k_logprobs_bwd<uint16_t>, grid, dim3(kThreads), 0, st,
                         static_cast<const uint16_t*>(x) + r * ld, V, ld, (unsigned)chunks, tg,
                         scale, stats + 2 * r, en, dl, de, static_cast<uint16_t*>(dx) + r * ldd,
                         ldd);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qn
