// C ABI of the QLoRA NF4 library: argument checks, workspace layout and
// launch order.  Every call checks its arguments on the host first and
// launches nothing on error.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/qlora_nf4.h"
#include "qn_device.h"
#include "qn_internal.h"

namespace {

using namespace qn;

// Carves 256-byte aligned pieces out of a caller workspace; with a null
// base it only measures.
struct Carver {
  char* base;
  size_t used = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(size_t count) {
    used = (used + 255) & ~size_t(255);
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += count * sizeof(T);
    return p;
  }
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Rows of `cols` elements end to end: where their starts do not keep 16-byte
// boundaries (cols % 8 != 0) the kernels take them on any element of `size` bytes,
// so that a slice of rows is as good a buffer as the whole.
bool aligned_rows(const void* p, int64_t cols, unsigned size) {
  return (reinterpret_cast<uintptr_t>(p) & (cols % 8 == 0 ? 15u : size - 1u)) == 0;
}
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }
int64_t groups_of(int64_t nb) { return (nb + kGroup - 1) / kGroup; }
int64_t pow2_at_least(int64_t v) {
  int64_t p = 1;
  while (p < v) p *= 2;
  return p;
}

qn_status from_hip(hipError_t e) { return e == hipSuccess ? QN_OK : QN_EDEVICE; }

struct QuantWs {
  float* absmax;
  double* part;
  int64_t part_len;
  int* bad;   // [ng] per-group flags
  int* flag;  // the synchronous call's flag
  float* mean;  // the mean of a call without double quantization (unused)
};

QuantWs carve_quant(Carver& c, int64_t n) {
  const int64_t nb = blocks_of(n), ng = groups_of(nb);
  QuantWs w;
  c.take<unsigned>(kArrivalWords);  // left alone: a workspace may be shared with linear calls
  w.absmax = c.take<float>(nb);
  w.part_len = pow2_at_least(ng);
  w.part = c.take<double>(w.part_len);
  w.bad = c.take<int>(ng);
  w.flag = c.take<int>(1);
  w.mean = c.take<float>(1);
  return w;
}

qn_status check_state(const qn_nf4dq* w) {
  if (!w || !w->packed) return QN_EINVAL;
  if (w->codebook != QN_CODE_NF4 && w->codebook != QN_CODE_FP4) return QN_EINVAL;
  if (!w->absmax && (!w->qscale || !w->scale2 || !w->offset)) return QN_EINVAL;
  if (w->rows < 1 || w->cols < 1) return QN_EINVAL;
  if (w->rows > (INT64_MAX / 2) / w->cols) return QN_EINVAL;
  if (!aligned16(w->packed)) return QN_EALIGN;
  if (w->absmax ? !aligned16(w->absmax)
                : (!aligned16(w->qscale) || !aligned16(w->scale2) || !aligned16(w->offset)))
    return QN_EALIGN;
  return QN_OK;
}


// Largest M and weight dimension the linear calls take: the kernels address
// buffers through 32-bit offsets from a row or slice base, which these
// bounds keep below 2^31 bytes.
constexpr int64_t kMaxRowsM = (int64_t)1 << 23;
constexpr int64_t kMaxDim = (int64_t)1 << 20;

qn_status check_linear(const qn_nf4dq* w, int64_t M, int r) {
  qn_status s = check_state(w);
  if (s != QN_OK) return s;
  if (w->cols % kBlock != 0 || w->rows % 8 != 0) return QN_EINVAL;
  if (w->rows > kMaxDim || w->cols > kMaxDim) return QN_EINVAL;
  if (r < 1 || r > 64) return QN_EINVAL;
  if (M < 0 || M > kMaxRowsM) return QN_EINVAL;
  return QN_OK;
}

WState to_state(const qn_nf4dq* w) {
  return WState{w->packed, w->qscale, w->scale2, w->offset, w->rows, w->cols, w->absmax,
                w->codebook};
}

// Large batches (enough 128 x 128 output tiles to fill the chip) take the
// weight through a bf16 copy in the workspace and a plain bf16 GEMM (256 x 256
// tiles where there are enough of those, else 128 x 128); smaller ones
// dequantize inside the GEMM.  At the decoder layer's k_proj shape (M = 4096,
// 1024 x 4096) the dequantizing GEMM re-read its operands 6.5 times and ran
// at a tenth of the bf16 peak.
bool dense_path(int64_t M, int64_t out_cols) {
  return M > 0 && ((M + 127) / 128) * ((out_cols + 127) / 128) >= 240;
}
int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

struct FwdWs {
  unsigned* arrivals;  // [kArrivalWords] arrival counters (zero between calls)
  float* u;      // [M, r] when the caller gives no u_out
  float* upart;  // [S, M, r] when S > 1
  int S;
  uint16_t* wd;  // [rows, cols] bf16 Qhat(W) (dense path)
  float* dpart;  // [dS, M, rows] decode partial sums (decode path)
  float* dupart; // [dS, M, r] decode partials of u
  int dS;
  DecodeTiles dt;  // one-kernel decode tiling (dt.rgt == 0: not used)
  float* tpart;    // [dt.S, M, rows] its partial sums
  float* tupart;   // [dt.bands, dt.S, 256] its partials of u
  int dbr;         // rows per band of the whole-row decode kernel (0: not used)
};

// dropout: the adapter branch reads a masked x, which the decode kernels
// (one set of x fragments for both products) do not take; such forwards use
// the GEMM routes.  Every route takes every state format.
FwdWs carve_fwd(Carver& c, int64_t M, int64_t rows, int64_t cols, int r, bool need_u,
                bool counters = true, bool dropout = false) {
  FwdWs f;
  f.arrivals = counters ? c.take<unsigned>(kArrivalWords) : nullptr;
  const bool dec = rows > 0 && !dropout;
  f.dbr = dec ? decode_rows_band(M, rows, cols, r) : 0;
  f.dt = dec && f.dbr == 0 ? decode_tiles(M, rows, cols, r) : DecodeTiles{0, 0, 0};
  f.dS = dec && f.dbr == 0 && f.dt.rgt == 0 ? decode_slices(M, rows, cols) : 0;
  const bool decode = f.dbr > 0 || f.dt.rgt > 0 || f.dS > 0;  // u from the decode kernels
  f.S = thin_nt_slices(M, cols);
  f.u = need_u ? c.take<float>((size_t)M * r) : nullptr;
  f.upart = f.S > 1 && !decode ? c.take<float>((size_t)f.S * M * r) : nullptr;
  f.wd = rows > 0 && M > 0 && !decode && dense_path(M, rows)
             ? c.take<uint16_t>((size_t)rows * cols)
             : nullptr;
  f.dpart = f.dS > 0 ? c.take<float>((size_t)f.dS * M * rows) : nullptr;
  f.dupart = f.dS > 0 ? c.take<float>((size_t)f.dS * M * r) : nullptr;
  f.tpart = f.dt.rgt > 0 ? c.take<float>((size_t)f.dt.S * M * round_up(rows, 4)) : nullptr;
  f.tupart = f.dt.rgt > 0 ? c.take<float>((size_t)f.dt.bands * f.dt.S * 256) : nullptr;
  return f;
}

struct BwdWs {
  unsigned* arrivals;  // [kArrivalWords] arrival counters
  FwdWs fu;      // recomputed u (if not saved)
  uint16_t* Bt;  // [r, rows]; x in 8 bits: B in launch_thin_v's order, [rp, rows up to 32]
  float* v;      // [M, r]
  float* vpart;  // [Sv, M, r]
  int Sv;
  float* dBpart;  // [Sb, rows, r]
  int Sb;
  uint16_t* su;   // [2][rp][Mpb] (s u)^T high and remainder parts ([3]: x in 8 bits)
  float* dApart;  // [Sa, cols, r]
  int Sa;
  uint16_t* sv;   // [2][rp][Mpa] (s v)^T
  uint16_t* wt;   // [cols, ldt] bf16 Qhat(W)^T (dense path)
  int64_t ldt;
  uint16_t* At;   // [cols, r] A^T (dense path)
};

BwdWs carve_bwd(Carver& c, int64_t M, int64_t rows, int64_t cols, int r, bool need_u,
                bool act8 = false, bool need_dx = true) {
  BwdWs b;
  b.arrivals = c.take<unsigned>(kArrivalWords);
  if (need_u) {
    b.fu = carve_fwd(c, M, 0, cols, r, true, false);
  } else {
    b.fu = FwdWs{};
    b.fu.S = 1;
  }
  const int64_t rp = 16 * ((r + 15) / 16);
  b.Bt = c.take<uint16_t>((size_t)(act8 ? rp * round_up(rows, 32) : r * rows));
  b.Sv = thin_nt_slices(M, rows);
  b.v = c.take<float>((size_t)M * r);
  b.vpart = b.Sv > 1 && !act8 ? c.take<float>((size_t)b.Sv * M * r) : nullptr;
  b.Sb = thin_tn_slices(M, rows, act8);
  b.dBpart = c.take<float>((size_t)b.Sb * rows * r);
  const size_t parts = act8 ? 3 : 2;
  b.su = c.take<uint16_t>(parts * rp * thin_tn_rows_padded(M, rows, act8));
  b.Sa = thin_tn_slices(M, cols, act8);
  b.dApart = c.take<float>((size_t)b.Sa * cols * r);
  b.sv = c.take<uint16_t>(parts * rp * thin_tn_rows_padded(M, cols, act8));
  b.ldt = round_up(rows, 64);
  // with x in 8 bits at every size: a weight read once and a product of few tiles
  // beat the dequantizing product, whose tiles walk the rows of W at 57 us per
  // 1024 (M = 300, 4096x4096: 285 us with it, 55 from the copy; M = 1, 1024x4096:
  // 64 and 30; even at 64 rows, 24 us)
  const bool dense = M > 0 && (act8 ? need_dx : dense_path(M, cols));
  b.wt = dense ? c.take<uint16_t>((size_t)cols * b.ldt) : nullptr;
  b.At = dense ? c.take<uint16_t>((size_t)cols * r) : nullptr;
  return b;
}

// The adapter branch's options (nullable: alpha / r, no dropout).
struct Lora {
  float s;               // branch scale
  const uint8_t* mask;   // dropout keep mask (nullable)
};

qn_status lora_options(const qn_lora_opts* o, float alpha, int r, Lora* out) {
  out->s = alpha / (float)r;
  out->mask = nullptr;
  if (!o) return QN_OK;
  if (o->rslora != 0 && o->rslora != 1) return QN_EINVAL;
  // rsLoRA: alpha / sqrt(r) (sqrtf is correctly rounded)
  if (o->rslora) out->s = alpha / sqrtf((float)r);
  if (o->dropout_mask) {
    const float p = o->dropout_p;
    if (!(p >= 0.f && p < 1.f)) return QN_EINVAL;
    if (!aligned16(o->dropout_mask)) return QN_EALIGN;  // read in 8- and 16-byte pieces
    out->mask = o->dropout_mask;
    out->s = out->s / (1.f - p);  // inverted dropout, folded into the scale
  } else if (o->dropout_p != 0.f) {
    return QN_EINVAL;
  }
  return QN_OK;
}

// The forward, on a workspace of ws_bytes at ws; clear: zero the arrival
// counters with a kernel before the launch that counts on them.
qn_status forward(const qn_nf4dq* w, const uint16_t* x, int64_t M, const uint16_t* A,
                  const uint16_t* B, int r, const Lora& lo, uint16_t* y, float* u_out,
                  void* workspace, size_t workspace_bytes, void* stream, bool clear) {
  qn_status s = check_linear(w, M, r);
  if (s != QN_OK) return s;
  if (M == 0) return QN_OK;
  if (!x || !A || !B || !y) return QN_EINVAL;
  if (!aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned16(y) ||
      (u_out && !aligned16(u_out)))
    return QN_EALIGN;
  Carver probe(nullptr);
  const bool drop = lo.mask != nullptr;
  carve_fwd(probe, M, w->rows, w->cols, r, u_out == nullptr, true, drop);
  if (probe.used > 0) {
    if (!workspace) return QN_EINVAL;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return QN_EALIGN;
    if (workspace_bytes < probe.used) return QN_EWORKSPACE;
  }
  Carver c(workspace);
  FwdWs f = carve_fwd(c, M, w->rows, w->cols, r, u_out == nullptr, true, drop);
  float* u = u_out ? u_out : f.u;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const float scale = lo.s;
  const int64_t N = w->rows, K = w->cols;
  if (f.dbr > 0)  // decode-sized batch, whole rows per workgroup
    return from_hip(launch_decode_rows(to_state(w), x, M, A, B, r, scale, y, u, f.dbr, st));
  if (f.dt.rgt > 0) {  // decode-sized batch, one kernel over column slices
    hipError_t e = hipSuccess;
    if (clear) e = launch_fill_zero(reinterpret_cast<float*>(f.arrivals), kArrivalWords, st);
    if (e == hipSuccess)
      e = launch_decode_tile(to_state(w), x, M, A, B, r, scale, y, u, f.dt, f.arrivals, f.tpart,
                             f.tupart, st);
    return from_hip(e);
  }
  if (f.dpart)  // decode-sized batch: u and the product in two kernels
    return from_hip(launch_decode_fwd(to_state(w), x, M, A, B, r, scale, y, u, f.dpart,
                                      f.dupart, f.dS, st));
  // dense path: the slices of u are added by spare workgroups of the
  // dequantization launch that follows
  const bool fold = f.wd && f.S > 1;
  hipError_t e = launch_thin_nt(x, A, M, K, r, u, f.upart, f.S, st, !fold, false,
                                Clear{nullptr, 0}, lo.mask);
  if (f.wd) {
    if (e == hipSuccess)
      e = launch_dequant(w->packed, w->qscale, w->scale2, w->offset, N * K, true, f.wd, st,
                         fold ? SliceSum{f.upart, M * (int64_t)r, f.S, u} : SliceSum{},
                         w->codebook, w->absmax);
    if (e == hipSuccess) e = launch_gemm_nt(x, K, K, f.wd, K, M, N, u, B, r, scale, y, st);
  } else if (e == hipSuccess) {
    e = launch_qgemm_fwd(to_state(w), x, M, u, B, r, scale, y, st);
  }
  return from_hip(e);
}

qn_status check_act8_shape(int64_t M, int64_t cols) {
  if (M < 0 || M > kMaxRowsM || cols < 1 || cols > kMaxDim) return QN_EINVAL;
  return QN_OK;
}

qn_status check_norm(const qn_block_norm* n, BlockNorm* out) {
  if (!n || n->M < 0 || n->M > kMaxRowsM || n->D < 1 || n->D > QN_NORM_MAX_COLS) return QN_EINVAL;
  if (n->res_dtype != QN_F32 && n->res_dtype != QN_BF16) return QN_EINVAL;
  if (n->w_dtype != QN_F32 && n->w_dtype != QN_BF16) return QN_EINVAL;
  if (n->gate_kind < QN_GATE_NONE || n->gate_kind > QN_GATE_ELEMENT) return QN_EINVAL;
  if (!std::isfinite(n->scale) || !std::isfinite(n->eps) || !(n->eps >= FLT_MIN))
    return QN_EINVAL;
  if (!n->w_pre) return QN_EINVAL;
  // no element gate has storage for an empty batch
  if ((n->gate_kind == QN_GATE_NONE) != (n->gate == nullptr) && n->M > 0) return QN_EINVAL;
  if (!aligned16(n->w_pre) || !aligned16(n->w_post)) return QN_EALIGN;
  // (a row's gate is read by itself)
  if (n->gate_kind == QN_GATE_ROW ? reinterpret_cast<uintptr_t>(n->gate) & 1u
      : n->gate_kind == QN_GATE_ELEMENT ? !aligned_rows(n->gate, n->D, 2)
                                        : !aligned16(n->gate))
    return QN_EALIGN;
  *out = BlockNorm{n->M, n->D, n->w_pre, n->w_post, n->gate, n->res_dtype == QN_F32,
                   n->w_dtype == QN_F32, n->gate_kind, n->scale, n->eps};
  return QN_OK;
}

// Logits rows are addressed from their own start (64-bit), elements of a row
// by 32-bit numbers.
constexpr int64_t kMaxVocab = (int64_t)1 << 28;
constexpr int64_t kMaxLd = (int64_t)1 << 40;
qn_status check_logits(const void* x, qn_dtype dtype, int64_t T, int64_t V, int64_t ld,
                       float scale) {
  if (dtype != QN_F32 && dtype != QN_BF16) return QN_EINVAL;
  if (T < 0 || T > kMaxRowsM || V < 1 || V > kMaxVocab || ld < V || ld > kMaxLd) return QN_EINVAL;
  if (!std::isfinite(scale) || !(scale > 0.f)) return QN_EINVAL;
  if (T == 0) return QN_OK;
  if (!x) return QN_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) & (dtype == QN_F32 ? 3u : 1u)) return QN_EALIGN;
  return QN_OK;
}

// The backward; the forward's input comes as x (bf16) or as x8 (an 8-bit
// checkpoint, with u_saved).
qn_status backward(const qn_nf4dq* w, const uint16_t* x, const qn_act8* x8, const uint16_t* dY,
                   int64_t M, const uint16_t* A, const uint16_t* B, int r, float alpha,
                   const qn_lora_opts* opts, const float* u_saved, uint16_t* dX, float* dA,
                   float* dB, void* workspace, size_t workspace_bytes, void* stream) {
  qn_status s = check_linear(w, M, r);
  if (s != QN_OK) return s;
  Lora lo;
  s = lora_options(opts, alpha, r, &lo);
  if (s != QN_OK) return s;
  if (!A || !B || !dA || !dB) return QN_EINVAL;
  if (M > 0 && !dY) return QN_EINVAL;
  if (M > 0 && (x8 ? (!x8->codes || !x8->exps || !u_saved) : !x)) return QN_EINVAL;
  if (x8 && (!aligned16(x8->codes) || !aligned16(x8->exps))) return QN_EALIGN;
  if (!aligned16(x) || !aligned16(dY) || !aligned16(A) || !aligned16(B) || !aligned16(dA) ||
      !aligned16(dB) || (dX && !aligned16(dX)) || (u_saved && !aligned16(u_saved)))
    return QN_EALIGN;
  const int64_t N = w->rows, K = w->cols;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 0) {
    // empty batch: the gradients of the adapters are zero
    hipError_t e = launch_fill_zero(dA, (int64_t)r * K, st);
    if (e == hipSuccess) e = launch_fill_zero(dB, N * (int64_t)r, st);
    return from_hip(e);
  }
  Carver probe(nullptr);
  carve_bwd(probe, M, N, K, r, u_saved == nullptr, x8 != nullptr, dX != nullptr);
  if (!workspace) return QN_EINVAL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return QN_EALIGN;
  if (workspace_bytes < probe.used) return QN_EWORKSPACE;
  Carver c(workspace);
  BwdWs b = carve_bwd(c, M, N, K, r, u_saved == nullptr, x8 != nullptr, dX != nullptr);
  const float scale = lo.s;
  hipError_t e = hipSuccess;
  const float* u = u_saved;
  // an early launch of the call zeroes the arrival counters the adapter
  // gradients' launch counts on, so the backward never depends on what the
  // workspace held before.  With x in 8 bits the slices of those gradients are
  // added by a launch of their own instead, unless the call is so short that it
  // waits for its launches: without dX 8192x4096x4096 at r = 16 40.3 -> 38.0 us,
  // 4096x4096x2048 at r = 8 25.8 -> 23.6, but 1024x1024x2048 17.3 -> 21.6; past 16
  // ranks a tile's last workgroup has too many values to add (4096x1024x4096 at
  // r = 64: 66 us for what takes 30)
  const bool few_launches = r <= 16 && M * (N + K) < (int64_t)1 << 24;
  unsigned* arrivals = x8 && !few_launches ? nullptr : b.arrivals;
  Clear clr{arrivals, arrivals ? kArrivalWords : 0};
  if (!u && e == hipSuccess) {
    e = launch_thin_nt(x, A, M, K, r, b.fu.u, b.fu.upart, b.fu.S, st, true, false, clr, lo.mask);
    clr = Clear{nullptr, 0};
    u = b.fu.u;
  }
  // v = G B.  With x in 8 bits: whole, and (s v)^T with it, from B in the order of
  // the product's operands, made first (and with that (s u)^T, and A^T for the dense
  // dX product; in spare workgroups of the transposed dequantization when there is
  // one).  Else in slices
  // (added below); the product takes B as stored when it can, else B^T made first.
  const bool b_rows = thin_nt_rows_ok(M, N, r);
  const bool dense_dx = dX && b.wt;
  if (e == hipSuccess && x8) {
    BwdAux t{};
    t.B = B;
    t.Bf = b.Bt;
    t.N = N;
    t.u = u;
    t.su = b.su;
    t.Mpu = thin_tn_rows_padded(M, N, true);
    t.M = M;
    t.r = r;
    t.s = scale;
    t.three_parts = true;
    t.A = A;
    t.At = dense_dx ? b.At : nullptr;
    t.K = K;
    if (dense_dx)
      e = launch_dequant_t(w->packed, w->qscale, w->scale2, w->offset, N, K, b.wt, b.ldt, t, st,
                           w->codebook, w->absmax);
    else
      e = launch_bwd_aux(t, st);
    if (e == hipSuccess)
      e = launch_thin_v(dY, b.Bt, M, N, r, b.v, b.sv, thin_tn_rows_padded(M, K, true), scale, st,
                        clr);
  }
  if (e == hipSuccess && !x8 && !b_rows) {
    if (clr.n) {  // (no earlier launch: a kernel, not a memset, for graph capture)
      e = launch_fill_zero(reinterpret_cast<float*>(clr.p), clr.n, st);
      clr = Clear{nullptr, 0};
    }
    BwdAux t{};
    t.B = B;
    t.Bt = b.Bt;
    t.N = N;
    t.r = r;
    e = launch_bwd_aux(t, st);
  }
  if (e == hipSuccess && !x8)
    e = launch_thin_nt(dY, b_rows ? B : b.Bt, M, N, r, b.v, b.vpart, b.Sv, st, false, b_rows,
                       clr);
  // the small jobs: v's slice sum, (s u)^T and (s v)^T split for the
  // transposed products, A^T for the dense dX product; in spare workgroups of
  // the transposed dequantization when there is one
  if (e == hipSuccess && !x8) {
    BwdAux aux{};
    aux.A = A;
    aux.At = dense_dx ? b.At : nullptr;
    aux.K = K;
    aux.u = u;
    aux.su = b.su;
    aux.Mpu = thin_tn_rows_padded(M, N, false);
    aux.vpart = b.vpart;
    aux.Sv = b.Sv;
    aux.v = b.v;
    aux.sv = b.sv;
    aux.Mpv = thin_tn_rows_padded(M, K, false);
    aux.M = M;
    aux.r = r;
    aux.s = scale;
    if (dense_dx)
      e = launch_dequant_t(w->packed, w->qscale, w->scale2, w->offset, N, K, b.wt, b.ldt, aux,
                           st, w->codebook, w->absmax);
    else
      e = launch_bwd_aux(aux, st);
  }
  if (e == hipSuccess && dX) {
    if (dense_dx)
      e = launch_gemm_nt(dY, N, N, b.wt, b.ldt, M, K, b.v, b.At, r, scale, dX, st, lo.mask);
    else
      e = launch_qgemm_dx(to_state(w), dY, M, b.v, A, r, scale, dX, st, lo.mask);
  }
  // dB = s G^T u and dA = s v^T X in one launch (and their slice sums in one)
  if (e == hipSuccess)
    e = launch_thin_tn2(ThinTn{dY, b.su, N, dB, false, b.dBpart},
                        ThinTn{x, b.sv, K, dA, true, b.dApart, lo.mask, x8 ? x8->codes : nullptr,
                               x8 ? x8->exps : nullptr},
                        M, r, arrivals, st);
  return from_hip(e);
}

// Scratch of qlora_linear_fwd_noalloc: a file-scope device array, one copy
// per GPU, held until the process ends.  Host code never passes its name to
// a kernel (on the host it is only a stand-in for the symbol): it uses the
// device address hipGetSymbolAddress returns for the current device.
constexpr size_t kStaticScratchBytes = QN_STATIC_SCRATCH_BYTES;
__device__ __align__(256) unsigned char scratch[kStaticScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// This device's address of the scratch array (looked up once per device).
qn_status static_scratch(void** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return QN_EDEVICE;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return QN_EDEVICE;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return QN_OK;
}

}  // namespace

extern "C" {

static_assert(QN_ARRIVAL_BYTES == 4 * kArrivalWords, "arrival counter page");

int qn_abi_version(void) { return QN_ABI_VERSION; }

const char* qn_status_str(qn_status s) {
  switch (s) {
    case QN_OK: return "ok";
    case QN_EINVAL: return "invalid argument";
    case QN_ENONFINITE: return "non-finite value in the weight";
    case QN_EALIGN: return "pointer not 16-byte aligned";
    case QN_EWORKSPACE: return "workspace too small";
    case QN_EDEVICE: return "HIP runtime error";
  }
  return "unknown status";
}

void qn_nf4_codebook(float out[16]) {
  for (int k = 0; k < 16; ++k) {
    uint32_t b = kNF4Bits[k];
    std::memcpy(&out[k], &b, 4);
  }
}

void qn_fp4_codebook(float out[16]) {
  for (int k = 0; k < 16; ++k) {
    uint32_t b = kFP4Bits[k];
    std::memcpy(&out[k], &b, 4);
  }
}

size_t nf4_quantize_dq_workspace(int64_t rows, int64_t cols) {
  if (rows < 1 || cols < 1 || rows > INT64_MAX / 2 / cols) return 0;
  Carver c(nullptr);
  carve_quant(c, rows * cols);
  return c.used;
}

qn_status nf4_quantize_dq(const float* W, int64_t rows, int64_t cols, uint8_t* packed,
                          uint8_t* qscale, float* scale2, float* offset, int* nonfinite,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return qn_quantize(W, rows, cols, QN_CODE_NF4, 1, packed, qscale, scale2, offset, nullptr,
                     nonfinite, workspace, workspace_bytes, stream);
}

qn_status qn_quantize(const float* W, int64_t rows, int64_t cols, int codebook,
                      int double_quant, uint8_t* packed, uint8_t* qscale, float* scale2,
                      float* offset, float* absmax, int* nonfinite, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (codebook != QN_CODE_NF4 && codebook != QN_CODE_FP4) return QN_EINVAL;
  if (!W || !packed || !workspace) return QN_EINVAL;
  if (double_quant ? (!qscale || !scale2 || !offset) : !absmax) return QN_EINVAL;
  if (rows < 1 || cols < 1 || rows > INT64_MAX / 2 / cols) return QN_EINVAL;
  if (!aligned16(W) || !aligned16(packed) || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      (reinterpret_cast<uintptr_t>(nonfinite) & 3u))
    return QN_EALIGN;
  if (double_quant ? (!aligned16(qscale) || !aligned16(scale2) || !aligned16(offset))
                   : !aligned16(absmax))
    return QN_EALIGN;
  const int64_t n = rows * cols;
  if (workspace_bytes < nf4_quantize_dq_workspace(rows, cols)) return QN_EWORKSPACE;
  Carver c(workspace);
  QuantWs ws = carve_quant(c, n);
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = launch_quantize(W, n, packed, qscale, scale2, offset, ws.absmax, ws.part,
                                 ws.part_len, ws.bad, nonfinite ? nonfinite : ws.flag, st,
                                 codebook, double_quant ? nullptr : absmax, ws.mean);
  if (e != hipSuccess) return QN_EDEVICE;
  if (nonfinite) return QN_OK;  // asynchronous: the caller reads the flag
  int bad = 0;
  e = hipMemcpyAsync(&bad, ws.flag, sizeof(int), hipMemcpyDeviceToHost, st);
  if (e != hipSuccess) return QN_EDEVICE;
  e = hipStreamSynchronize(st);
  if (e != hipSuccess) return QN_EDEVICE;
  return bad ? QN_ENONFINITE : QN_OK;
}

qn_status nf4_dequantize(const qn_nf4dq* w, qn_dtype out_dtype, void* out, void* stream) {
  qn_status s = check_state(w);
  if (s != QN_OK) return s;
  if (!out || (out_dtype != QN_F32 && out_dtype != QN_BF16)) return QN_EINVAL;
  if (!aligned16(out)) return QN_EALIGN;
  return from_hip(launch_dequant(w->packed, w->qscale, w->scale2, w->offset, w->rows * w->cols,
                                 out_dtype == QN_BF16, out, static_cast<hipStream_t>(stream),
                                 SliceSum{}, w->codebook, w->absmax, /*nt=*/true));
}

size_t qlora_linear_workspace_ex(int64_t M, int64_t rows, int64_t cols, int r, int backward,
                                 const qn_lora_opts* opts) {
  if (M < 0 || rows < 1 || cols < 1 || r < 1 || r > 64) return 0;
  const bool drop = opts && opts->dropout_mask;
  Carver c(nullptr);
  if (backward)
    carve_bwd(c, M, rows, cols, r, true);
  else
    carve_fwd(c, M, rows, cols, r, true, true, drop);
  return c.used;
}

size_t qlora_linear_workspace(int64_t M, int64_t rows, int64_t cols, int r, int backward) {
  return qlora_linear_workspace_ex(M, rows, cols, r, backward, nullptr);
}

size_t qlora_linear_workspace_state(const qn_nf4dq* w, int64_t M, int r, int backward,
                                    const qn_lora_opts* opts) {
  if (!w || M < 0 || w->rows < 1 || w->cols < 1 || r < 1 || r > 64) return 0;
  const bool drop = opts && opts->dropout_mask;
  Carver c(nullptr);
  if (backward)
    carve_bwd(c, M, w->rows, w->cols, r, true);
  else
    carve_fwd(c, M, w->rows, w->cols, r, true, true, drop);
  return c.used;
}

qn_status qlora_linear_fwd(const qn_nf4dq* w, const uint16_t* x, int64_t M, const uint16_t* A,
                           const uint16_t* B, int r, float alpha, uint16_t* y, float* u_out,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return qlora_linear_fwd_ex(w, x, M, A, B, r, alpha, nullptr, y, u_out, workspace,
                             workspace_bytes, stream);
}

qn_status qlora_linear_fwd_ex(const qn_nf4dq* w, const uint16_t* x, int64_t M, const uint16_t* A,
                              const uint16_t* B, int r, float alpha, const qn_lora_opts* opts,
                              uint16_t* y, float* u_out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (r < 1 || r > 64) return QN_EINVAL;
  Lora lo;
  qn_status s = lora_options(opts, alpha, r, &lo);
  if (s != QN_OK) return s;
  return forward(w, x, M, A, B, r, lo, y, u_out, workspace, workspace_bytes, stream, false);
}

qn_status qlora_linear_fwd_noalloc(const qn_nf4dq* w, const uint16_t* x, int64_t M,
                                   const uint16_t* A, const uint16_t* B, int r, float alpha,
                                   uint16_t* y, float* u_out, void* stream) {
  qn_status s = check_linear(w, M, r);
  if (s != QN_OK) return s;
  if (M == 0) return QN_OK;
  Carver probe(nullptr);
  carve_fwd(probe, M, w->rows, w->cols, r, u_out == nullptr);
  if (probe.used > kStaticScratchBytes) return QN_EWORKSPACE;
  void* ptr = nullptr;
  s = static_scratch(&ptr);
  if (s != QN_OK) return s;
  // the array keeps what the last call left in it: its counters are cleared
  // by a kernel before the launch that counts on them
  return forward(w, x, M, A, B, r, Lora{alpha / (float)r, nullptr}, y, u_out, ptr,
                 kStaticScratchBytes, stream, true);
}



qn_status qlora_linear_bwd(const qn_nf4dq* w, const uint16_t* x, const uint16_t* dY, int64_t M,
                           const uint16_t* A, const uint16_t* B, int r, float alpha,
                           const float* u_saved, uint16_t* dX, float* dA, float* dB,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return qlora_linear_bwd_ex(w, x, dY, M, A, B, r, alpha, nullptr, u_saved, dX, dA, dB,
                             workspace, workspace_bytes, stream);
}

qn_status qlora_linear_bwd_ex(const qn_nf4dq* w, const uint16_t* x, const uint16_t* dY,
                              int64_t M, const uint16_t* A, const uint16_t* B, int r, float alpha,
                              const qn_lora_opts* opts, const float* u_saved, uint16_t* dX,
                              float* dA, float* dB, void* workspace, size_t workspace_bytes,
                              void* stream) {
  return backward(w, x, nullptr, dY, M, A, B, r, alpha, opts, u_saved, dX, dA, dB, workspace,
                  workspace_bytes, stream);
}

qn_status nf4_merge_lora(const qn_nf4dq* w, const uint16_t* A, const uint16_t* B, int r,
                         float alpha, float* out, void* stream) {
  qn_status s = check_state(w);
  if (s != QN_OK) return s;
  if (r < 1 || r > 64 || w->rows > kMaxDim * 64 || w->cols > kMaxDim * 64) return QN_EINVAL;
  if (!A || !B || !out) return QN_EINVAL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(out)) return QN_EALIGN;
  return from_hip(launch_merge(to_state(w), A, B, r, alpha / (float)r, out,
                               static_cast<hipStream_t>(stream), w->codebook, w->absmax));
}

qn_status adamw8_step(float* p, const float* g, int64_t n, uint8_t* m_codes, float* m_scales,
                      uint8_t* v_codes, float* v_scales, uint16_t* p_bf16,
                      const qn_adamw_hparams* h, void* stream) {
  if (n < 0 || !h || h->step < 1) return QN_EINVAL;
  if (n == 0) return QN_OK;
  if (!p || !g || !m_codes || !m_scales || !v_codes || !v_scales) return QN_EINVAL;
  if (!aligned16(p) || !aligned16(g) || !aligned16(m_codes) || !aligned16(v_codes) ||
      !aligned16(m_scales) || !aligned16(v_scales) || (p_bf16 && !aligned16(p_bf16)))
    return QN_EALIGN;
  if (!(h->beta1 >= 0.f && h->beta1 < 1.f && h->beta2 >= 0.f && h->beta2 < 1.f)) return QN_EINVAL;
  // the derived scalars in fp64 from the fp32 hyperparameters, rounded once
  const double b1 = h->beta1, b2 = h->beta2, t = (double)h->step;
  AdamScalars s;
  s.lr = h->lr;
  s.b1 = h->beta1;
  s.b2 = h->beta2;
  s.omb1 = (float)(1.0 - b1);
  s.omb2 = (float)(1.0 - b2);
  s.eps = h->eps;
  s.c1 = (float)(1.0 - std::pow(b1, t));
  s.c2 = (float)(1.0 - std::pow(b2, t));
  s.decay = (float)(1.0 - (double)h->lr * (double)h->weight_decay);
  return from_hip(launch_adamw8(p, g, n, m_codes, m_scales, v_codes, v_scales, p_bf16, s,
                                static_cast<hipStream_t>(stream)));
}

int qlora_linear_route(int64_t M, int64_t rows, int64_t cols, int r, int backward) {
  if (M < 1 || M > kMaxRowsM || rows < 8 || cols < kBlock || rows % 8 != 0 ||
      cols % kBlock != 0 || rows > kMaxDim || cols > kMaxDim || r < 1 || r > 64)
    return -1;
  const int64_t out_cols = backward ? cols : rows;
  if (!backward) {
    if (decode_rows_band(M, rows, cols, r) > 0) return QN_ROUTE_DECODE_ROWS;
    if (decode_tiles(M, rows, cols, r).rgt > 0) return QN_ROUTE_DECODE_TILES;
    if (decode_slices(M, rows, cols) > 0) return QN_ROUTE_DECODE_SPLIT;
  }
  if (dense_path(M, out_cols)) return QN_ROUTE_DENSE;
  return M <= 32 ? QN_ROUTE_FUSED_SMALL : QN_ROUTE_FUSED;
}

qn_status lora_linear_bf16(const uint16_t* x, int64_t M, const uint16_t* W, int64_t rows,
                           int64_t cols, const float* V, const uint16_t* L, int r, float alpha,
                           uint16_t* y, void* stream) {
  if (rows < 1 || cols < 1 || M < 0 || r < 1 || r > 64) return QN_EINVAL;
  if (cols % kBlock != 0 || rows % 8 != 0) return QN_EINVAL;
  if (M == 0) return QN_OK;
  if (!x || !W || !V || !L || !y) return QN_EINVAL;
  if (!aligned16(x) || !aligned16(W) || !aligned16(V) || !aligned16(L) || !aligned16(y))
    return QN_EALIGN;
  return from_hip(launch_gemm_nt(x, cols, cols, W, cols, M, rows, V, L, r, alpha / (float)r, y,
                                 static_cast<hipStream_t>(stream)));
}

qn_status act8_pack(const uint16_t* x, int64_t M, int64_t cols, int8_t* codes, uint8_t* exps,
                    void* stream) {
  qn_status s = check_act8_shape(M, cols);
  if (s != QN_OK || M == 0) return s;
  if (!x || !codes || !exps) return QN_EINVAL;
  if (!aligned_rows(x, cols, 2) || !aligned_rows(codes, cols, 1) || !aligned_rows(exps, cols, 1))
    return QN_EALIGN;
  return from_hip(launch_act8_pack(x, M, cols, codes, exps, static_cast<hipStream_t>(stream)));
}

qn_status act8_unpack(const qn_act8* x8, int64_t M, int64_t cols, uint16_t* out, void* stream) {
  qn_status s = check_act8_shape(M, cols);
  if (s != QN_OK || M == 0) return s;
  if (!x8 || !x8->codes || !x8->exps || !out) return QN_EINVAL;
  if (!aligned_rows(x8->codes, cols, 1) || !aligned_rows(x8->exps, cols, 1) ||
      !aligned_rows(out, cols, 2))
    return QN_EALIGN;
  return from_hip(launch_act8_unpack(x8->codes, x8->exps, M, cols, out,
                                     static_cast<hipStream_t>(stream)));
}

size_t qlora_linear_bwd_act8_workspace(int64_t M, int64_t rows, int64_t cols, int r, int need_dx) {
  if (M < 0 || rows < 1 || cols < 1 || r < 1 || r > 64) return 0;
  Carver c(nullptr);
  carve_bwd(c, M, rows, cols, r, false, true, need_dx != 0);
  return c.used;
}

qn_status qlora_linear_bwd_act8(const qn_nf4dq* w, const qn_act8* x8, const uint16_t* dY,
                                int64_t M, const uint16_t* A, const uint16_t* B, int r,
                                float alpha, const qn_lora_opts* opts, const float* u,
                                uint16_t* dX, float* dA, float* dB, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!x8 && M != 0) return QN_EINVAL;
  return backward(w, nullptr, x8, dY, M, A, B, r, alpha, opts, u, dX, dA, dB, workspace,
                  workspace_bytes, stream);
}

qn_status block_norm_fwd(const qn_block_norm* n, const void* h, const uint16_t* o, void* h_new,
                         uint16_t* y, int8_t* codes, uint8_t* exps, void* stream) {
  BlockNorm b;
  qn_status s = check_norm(n, &b);
  if (s != QN_OK) return s;
  if ((codes == nullptr) != (exps == nullptr)) return QN_EINVAL;
  if (n->M == 0) return QN_OK;
  if (!o && (n->w_post || n->gate || h_new)) return QN_EINVAL;
  if (!h || !y || (o && !h_new)) return QN_EINVAL;
  const int64_t D = n->D;
  const unsigned res = b.res32 ? 4 : 2;
  if (!aligned_rows(h, D, res) || !aligned_rows(o, D, 2) || !aligned_rows(h_new, D, res) ||
      !aligned_rows(y, D, 2) || !aligned_rows(codes, D, 1) || !aligned_rows(exps, D, 1))
    return QN_EALIGN;
  return from_hip(launch_block_norm_fwd(b, h, o, h_new, y, codes, exps,
                                        static_cast<hipStream_t>(stream)));
}

size_t block_norm_bwd_workspace(const qn_block_norm* n, int need_weights, int need_gate) {
  if (!n || n->M < 0 || n->D < 1 || n->D > QN_NORM_MAX_COLS) return 0;
  if (!need_weights && !(need_gate && n->gate_kind == QN_GATE_CHANNEL)) return 0;
  Carver c(nullptr);
  c.take<unsigned>(kArrivalWords);  // left alone, as above
  c.take<float>((size_t)block_norm_slices(n->M, n->D) * 3 * n->D);
  c.take<float>((size_t)block_norm_stats(n->M, n->D));
  return c.used;
}

qn_status block_norm_bwd(const qn_block_norm* n, const uint16_t* dy, const void* dh_new,
                         const void* h_new, const uint16_t* o, void* dh, uint16_t* dout,
                         void* dgate, float* dw_post, float* dw_pre, void* workspace,
                         size_t workspace_bytes, void* stream) {
  BlockNorm b;
  qn_status s = check_norm(n, &b);
  if (s != QN_OK) return s;
  if ((o == nullptr) != (dout == nullptr) && n->M > 0) return QN_EINVAL;
  if (n->M > 0 && !o && (n->w_post || n->gate)) return QN_EINVAL;
  if ((dw_post && !n->w_post) || (dgate && !n->gate)) return QN_EINVAL;
  if (n->M > 0 && (!dy || !h_new || !dh)) return QN_EINVAL;
  const int64_t D = n->D;
  const unsigned res = b.res32 ? 4 : 2;
  if (!aligned_rows(dy, D, 2) || !aligned_rows(dh_new, D, res) || !aligned_rows(h_new, D, res) ||
      !aligned_rows(o, D, 2) || !aligned_rows(dh, D, res) || !aligned_rows(dout, D, 2) ||
      (n->gate_kind == QN_GATE_ELEMENT ? !aligned_rows(dgate, D, 2) : !aligned16(dgate)) ||
      !aligned16(dw_post) || !aligned16(dw_pre))
    return QN_EALIGN;
  const bool chan = dgate && n->gate_kind == QN_GATE_CHANNEL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n->M == 0) {  // sums over no rows
    hipError_t e = hipSuccess;
    if (dw_pre) e = launch_fill_zero(dw_pre, n->D, st);
    if (e == hipSuccess && dw_post) e = launch_fill_zero(dw_post, n->D, st);
    if (e == hipSuccess && chan) e = launch_fill_zero(static_cast<float*>(dgate), n->D, st);
    return from_hip(e);
  }
  float *part = nullptr, *stats = nullptr;
  if (dw_pre || dw_post || chan) {
    if (!workspace) return QN_EINVAL;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return QN_EALIGN;
    if (workspace_bytes < block_norm_bwd_workspace(n, dw_pre || dw_post, chan)) return QN_EWORKSPACE;
    Carver c(workspace);
    c.take<unsigned>(kArrivalWords);
    part = c.take<float>((size_t)block_norm_slices(n->M, n->D) * 3 * n->D);
    stats = c.take<float>((size_t)block_norm_stats(n->M, n->D));
  }
  return from_hip(launch_block_norm_bwd(b, dy, dh_new, h_new, o, dh, dout, dgate, dw_post, dw_pre,
                                        part, stats, st));
}

size_t token_logprobs_workspace(int64_t T, int64_t V, qn_dtype dtype, int top_k) {
  if (T < 1 || T > kMaxRowsM || V < 1 || V > kMaxVocab || top_k < 0) return 0;
  const size_t used = logprob_workspace(T, V, dtype == QN_F32, top_k);
  return used ? QN_ARRIVAL_BYTES + used : 0;  // (the counters left alone, as above)
}

qn_status token_logprobs_fwd(const void* logits, qn_dtype dtype, int64_t T, int64_t V, int64_t ld,
                             const int64_t* targets, float scale, int top_k, float* logp,
                             float* entropy, float* stats, float* top_logp, int32_t* top_ids,
                             void* workspace, size_t workspace_bytes, void* stream) {
  qn_status s = check_logits(logits, dtype, T, V, ld, scale);
  if (s != QN_OK) return s;
  if (top_k < 0 || top_k > QN_LOGPROB_MAX_TOP || top_k > V) return QN_EINVAL;
  if ((targets == nullptr) != (logp == nullptr) && T > 0) return QN_EINVAL;
  if (T == 0) return QN_OK;
  if (!entropy || !stats || (top_k > 0 && (!top_logp || !top_ids))) return QN_EINVAL;
  if (!aligned8(targets) || !aligned16(logp) || !aligned16(entropy) || !aligned16(stats) ||
      !aligned16(top_logp) || !aligned16(top_ids))
    return QN_EALIGN;
  const size_t need = token_logprobs_workspace(T, V, dtype, top_k);
  if (need > 0) {
    if (!workspace) return QN_EINVAL;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return QN_EALIGN;
    if (workspace_bytes < need) return QN_EWORKSPACE;
  }
  return from_hip(launch_logprobs_fwd(logits, dtype == QN_F32, T, V, ld, targets, scale, top_k,
                                      logp, entropy, stats, top_logp, top_ids,
                                      need ? static_cast<char*>(workspace) + QN_ARRIVAL_BYTES
                                           : nullptr,
                                      static_cast<hipStream_t>(stream)));
}

qn_status token_logprobs_bwd(const void* logits, qn_dtype dtype, int64_t T, int64_t V, int64_t ld,
                             const int64_t* targets, float scale, const float* stats,
                             const float* entropy, const float* dlogp, const float* dentropy,
                             void* dlogits, int64_t ldd, void* stream) {
  qn_status s = check_logits(logits, dtype, T, V, ld, scale);
  if (s != QN_OK) return s;
  if (ldd < V || ldd > kMaxLd) return QN_EINVAL;
  if (T == 0) return QN_OK;
  if (!stats || !dlogits || (!dlogp && !dentropy) || (dlogp && !targets) || (dentropy && !entropy))
    return QN_EINVAL;
  if (dlogits == logits && ldd != ld) return QN_EINVAL;
  if (!aligned8(targets) || !aligned16(stats) || !aligned16(entropy) || !aligned16(dlogp) ||
      !aligned16(dentropy) || (reinterpret_cast<uintptr_t>(dlogits) & (dtype == QN_F32 ? 3u : 1u)))
    return QN_EALIGN;
  return from_hip(launch_logprobs_bwd(logits, dtype == QN_F32, T, V, ld, targets, scale, stats,
                                      entropy, dlogp, dentropy, dlogits, ldd,
                                      static_cast<hipStream_t>(stream)));
}

}  // extern "C"
