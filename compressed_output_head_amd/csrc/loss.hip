// Losses on rows of logits with their gradient: the clipped policy loss with
// a KL term (archead_policy_loss) and the preference loss over pairs of
// sequences (archead_preference_loss).
//
// With z = s y (s the inverse temperature) both need of a row its label's
// log-probability, log p = z_label - max z - log sum exp(z - max z), and both
// leave the same kind of gradient, coef s (one-hot(label) - softmax(z)), with
// a coefficient per row.  With k = s log2 e as an fp32 pair (one fp32 number
// alone would shift every log p of a call by a few 1e-7, the same way for all
// rows) and M = max y
//   e_j = 2^(k (y_j - M)),  S = sum_j e_j,  log p = s (y_label - M) - ln S,
// where the last line and all per-row arithmetic after it are fp64 (a loss
// is a sum of terms of both signs, and one row is one thread's work).  The
// difference is taken first: a fused k y - k M would save an instruction, but
// overflows where every logit of a piece is the type's lowest value.  S is
// summed in fp32 by thousands of partial sums of at most a few hundred terms.
// The label's element of the gradient is -coef s expm1(log p), which keeps
// its digits where p is close to 1.
//
// A row is cut into pieces so that few rows still fill the GPU:
//   row_pieces_kernel   (M, S) of every piece, and the label's logit
//   pair_kernel         preference loss only: sequence sums, the pairs'
//                       losses and every row's coefficient
//   row_gradient_kernel the gradient, piece by piece; for the policy loss
//                       each workgroup first merges its row's pieces and works
//                       the coefficient out; one more workgroup adds up the loss
// Rows of weight zero are neither read nor counted; their gradient is zero.
// Every sum has a fixed order, so results do not depend on scheduling.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "device_common.h"
#include "internal.h"

namespace archead {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;        // 16-byte loads in flight per thread
constexpr int kSumThreads = 1024;
constexpr int64_t kMaxPieces = 64;

// What the gradient of a row needs: dY_j = neg 2^(k (y_j - M)), label_g at the label.
struct RowGrad {
  float neg, M, label_g;
  uint32_t on;  // 0: the gradient is zero
};

// s log2 e = hi + lo
struct Scale {
  float hi, lo;
};

struct RowArgs {
  const void* Y;
  void* dY;
  int64_t N, V, y_stride, dy_stride;
  int64_t width;  // columns of a piece
  int pieces;
  Scale k;
  float s;
  const int32_t* labels;
  const float* weight;
  // workspace
  float2* part;    // [N][pieces] (M, S)
  float* ylab;     // [N]
  RowGrad* grad;   // [N], preference loss
  double* pair_loss;  // [B], preference loss
  // policy loss
  const float *old_logp, *ref_logp, *advantage;
  float clip_low, clip_high, kl_coef;
  // preference loss
  const int32_t* offsets;
  int64_t B;
  const float* pair_weight;
  float beta, smoothing;
  int kind;
  // outputs (each may be null)
  float *loss, *logp, *row_loss, *chosen, *rejected;
};

// 16 bytes that start at any element: rows of an odd length have every alignment.
typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {  // bf16
  static constexpr int kPer16 = 8;
  static constexpr uint32_t kNegInf2 = 0xff80ff80u;
  static __device__ __forceinline__ float at(const u4& v, int j) {
    return __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16);
  }
  static __device__ __forceinline__ float one(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t from(float f) { return f32_to_bf16(f); }
};
template <>
struct Elem<float> {
  static constexpr int kPer16 = 4;
  static constexpr uint32_t kNegInf2 = 0xff800000u;
  static __device__ __forceinline__ float at(const u4& v, int j) { return __uint_as_float(v[j]); }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ float from(float f) { return f; }
};

// n = 4 or 8 values to consecutive elements, 16 or 8 bytes a store.
template <int n>
__device__ __forceinline__ void store_run(uint16_t* p, const float* g) {
  if constexpr (n == 8) {
    const u2 a = pack_bf16x4(g[0], g[1], g[2], g[3]), b = pack_bf16x4(g[4], g[5], g[6], g[7]);
    *reinterpret_cast<u4_any*>(p) = u4{a[0], a[1], b[0], b[1]};
  } else {
    *reinterpret_cast<u2_any*>(p) = pack_bf16x4(g[0], g[1], g[2], g[3]);
  }
}
template <int n>
__device__ __forceinline__ void store_run(float* p, const float* g) {
#pragma unroll
  for (int i = 0; i < n; i += 4) {
    const f4 v = {g[i], g[i + 1], g[i + 2], g[i + 3]};
    *reinterpret_cast<u4_any*>(p + i) = __builtin_bit_cast(u4, v);
  }
}

// 2^(k d)
__device__ __forceinline__ float exp_at(float d, Scale k) {
  return __builtin_amdgcn_exp2f(fmaf(d, k.hi, d * k.lo));
}

// What is subtracted from logits of maximum M: nothing where all are -inf.
__device__ __forceinline__ float shift_of(float M) { return M == -INFINITY ? 0.0f : M; }

// Two (M, S) pieces as one.
__device__ __forceinline__ float2 merge(float2 a, float2 b, Scale k) {
  const float M = fmaxf(a.x, b.x), M0 = shift_of(M);
  return float2{M, a.y * exp_at(a.x - M0, k) + b.y * exp_at(b.x - M0, k)};
}

template <int kThreads>
__device__ __forceinline__ float2 block_merge(float2 v, Scale k, float2* buf) {
  for (int o = 32; o > 0; o >>= 1) v = merge(v, float2{__shfl_xor(v.x, o), __shfl_xor(v.y, o)}, k);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < kThreads / 64; ++w) v = merge(v, buf[w], k);
  return v;
}

template <int kThreads>
__device__ __forceinline__ double block_sum(double v, double* buf) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < kThreads / 64; ++w) v += buf[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ float weight_of(const RowArgs& a, int64_t n) { return a.weight ? a.weight[n] : 1.0f; }

// Rows [first, last) that belong to a sequence of a pair.
__device__ __forceinline__ bool in_pairs(const RowArgs& a, int64_t n) {
  return n >= a.offsets[0] && n < a.offsets[2 * a.B];
}

// (M, S) of the elements [0, len) at p, one thread's share.
template <typename T>
__device__ __forceinline__ float2 thread_stats(const T* p, int64_t len, Scale k) {
  using E = Elem<T>;
  const int64_t full = len / E::kPer16;
  float M = -INFINITY, M0 = 0.0f, S = 0.0f;
  auto rise = [&](float top) {  // of the running maximum
    if (top > M) {
      S *= exp_at(M - top, k);
      M = M0 = top;
    }
  };
  for (int64_t c0 = threadIdx.x; c0 < full; c0 += kRowThreads * kRowUnroll) {
    u4 v[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int64_t c = c0 + u * kRowThreads;
      v[u] = c < full ? u4(*reinterpret_cast<const u4_any*>(p + c * E::kPer16))
                      : u4{E::kNegInf2, E::kNegInf2, E::kNegInf2, E::kNegInf2};
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u)
#pragma unroll
      for (int j = 0; j < E::kPer16; ++j) top = fmaxf(top, E::at(v[u], j));
    rise(top);
    float add = 0.0f;
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u)
#pragma unroll
      for (int j = 0; j < E::kPer16; ++j) add += exp_at(E::at(v[u], j) - M0, k);
    S += add;
  }
  const int64_t i = full * E::kPer16 + threadIdx.x;  // fewer than 8 elements are left
  if (i < len) {
    const float y = E::one(p[i]);
    rise(y);
    S += exp_at(y - M0, k);
  }
  return float2{M, S};
}

template <typename T, bool kPairs>
__global__ __launch_bounds__(kRowThreads) void row_pieces_kernel(const RowArgs a) {
  __shared__ float2 buf[kRowThreads / 64];
  const int64_t n = blockIdx.x / a.pieces;
  const int p = (int)(blockIdx.x % a.pieces);
  const bool on = weight_of(a, n) != 0.0f && (!kPairs || in_pairs(a, n));
  if (p == 0 && threadIdx.x == 0) {
    // what stays of a row that does not count (or that no sequence of descending offsets holds)
    if (a.logp) a.logp[n] = 0.0f;
    if (a.row_loss) a.row_loss[n] = 0.0f;
    if (kPairs) a.grad[n] = RowGrad{0.0f, 0.0f, 0.0f, 0u};
  }
  if (!on) return;
  const T* row = static_cast<const T*>(a.Y) + n * a.y_stride;
  const int64_t c0 = p * a.width, c1 = c0 + a.width < a.V ? c0 + a.width : a.V;
  const int64_t label = a.labels[n];
  const bool valid = label >= 0 && label < a.V;
  // in its own launch: the gradient may be written over Y
  if (threadIdx.x == 0 && (valid ? label >= c0 && label < c1 : p == 0))
    a.ylab[n] = valid ? Elem<T>::one(row[label]) : __builtin_nanf("");
  const float2 r = block_merge<kRowThreads>(thread_stats(row + c0, c1 - c0, a.k), a.k, buf);
  if (threadIdx.x == 0) a.part[n * a.pieces + p] = r;
}

// The row's pieces in order.
__device__ __forceinline__ float2 merged(const RowArgs& a, int64_t n) {
  float2 r = a.part[n * a.pieces];
  for (int p = 1; p < a.pieces; ++p) r = merge(r, a.part[n * a.pieces + p], a.k);
  return r;
}

__device__ __forceinline__ double row_logp(const RowArgs& a, int64_t n, float2 r) {
  return (double)a.s * ((double)a.ylab[n] - (double)r.x) - log((double)r.y);
}

__device__ __forceinline__ RowGrad row_grad(const RowArgs& a, double coef, double logp, float2 r) {
  const double c = coef * (double)a.s;
  return RowGrad{(float)(-c / (double)r.y), r.x, (float)(-c * expm1(logp)), coef != 0.0 ? 1u : 0u};
}

// The policy loss of one row and its derivative in the log-probability.
__device__ __forceinline__ void policy_row(const RowArgs& a, int64_t n, double logp, double& loss, double& slope) {
  const double A = a.advantage[n];
  const double ratio = a.old_logp ? exp(logp - (double)a.old_logp[n]) : exp(logp - logp);
  const double lo = 1.0 - (double)a.clip_low, hi = 1.0 + (double)a.clip_high;
  const double kept = ratio < lo ? lo : ratio > hi ? hi : ratio;  // NaN stays NaN
  const bool plain = !(kept * A < ratio * A);  // the unclipped term is the smaller one
  loss = plain ? -(ratio * A) : -(kept * A);
  slope = plain ? -(ratio * A) : 0.0;
  if (a.kl_coef != 0.0f) {
    const double d = (double)a.ref_logp[n] - logp, e = expm1(d);
    loss += (double)a.kl_coef * (e - d);
    slope -= (double)a.kl_coef * e;
  }
}

// Workgroup i: pair i.  Threads take the rows of a sequence in turn.
__global__ __launch_bounds__(kRowThreads) void pair_kernel(const RowArgs a) {
  __shared__ double buf[kRowThreads / 64];
  const int64_t i = blockIdx.x;
  auto bound = [&](int64_t q) {  // offsets outside [0, N] end at its borders
    const int64_t o = a.offsets[q];
    return o < 0 ? (int64_t)0 : o > a.N ? a.N : o;
  };
  const int64_t b[3] = {bound(2 * i), bound(2 * i + 1), bound(2 * i + 2)};
  double sum[2];
  for (int side = 0; side < 2; ++side) {
    double part = 0.0;
    for (int64_t n = b[side] + threadIdx.x; n < b[side + 1]; n += kRowThreads) {
      const float w = weight_of(a, n);
      if (w == 0.0f || !in_pairs(a, n)) continue;
      const double logp = row_logp(a, n, merged(a, n));
      if (a.logp) a.logp[n] = (float)logp;
      part += (double)w * (logp - (a.ref_logp ? (double)a.ref_logp[n] : 0.0));
    }
    sum[side] = block_sum<kRowThreads>(part, buf);
  }
  const double h = sum[0] - sum[1], beta = a.beta, eps = a.smoothing;
  double loss, slope;  // of the pair, and its derivative in h
  if (a.kind == ARCHEAD_PREF_SIGMOID) {
    const double x = beta * h, t = log1p(exp(-fabs(x)));  // softplus(x) = max(x, 0) + t
    loss = (1.0 - eps) * ((x < 0.0 ? -x : 0.0) + t) + eps * ((x > 0.0 ? x : 0.0) + t);
    slope = beta * (eps - 1.0 / (1.0 + exp(x)));
  } else {
    const double u = h - 0.5 / beta;
    loss = u * u;
    slope = 2.0 * u;
  }
  const double pw = a.pair_weight ? (double)a.pair_weight[i] : 1.0;
  // a pair of weight zero is left out, whatever its rows hold
  loss = pw != 0.0 ? pw * loss : 0.0;
  slope = pw != 0.0 ? pw * slope : 0.0;
  if (threadIdx.x == 0) {
    a.pair_loss[i] = loss;
    if (a.chosen) a.chosen[i] = (float)(beta * sum[0]);
    if (a.rejected) a.rejected[i] = (float)(beta * sum[1]);
  }
  for (int side = 0; side < 2; ++side)
    for (int64_t n = b[side] + threadIdx.x; n < b[side + 1]; n += kRowThreads) {
      const float w = weight_of(a, n);
      if (w == 0.0f || !in_pairs(a, n)) continue;
      const float2 r = merged(a, n);
      a.grad[n] = row_grad(a, (side ? -slope : slope) * (double)w, row_logp(a, n, r), r);
    }
}

// The elements [0, len) of a gradient row; `label` is the label's place in them, or no place.
template <typename T, typename G>
__device__ __forceinline__ void thread_gradient(const T* y, G* dy, int64_t len, int64_t label, Scale k, RowGrad r) {
  using E = Elem<T>;
  constexpr int n = E::kPer16;
  const int64_t full = len / n;
  for (int64_t c0 = threadIdx.x; c0 < full; c0 += kRowThreads * kRowUnroll) {
    u4 v[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int64_t c = c0 + u * kRowThreads;
      if (r.on && c < full) v[u] = *reinterpret_cast<const u4_any*>(y + c * n);
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int64_t c = c0 + u * kRowThreads;
      if (c >= full) break;
      float g[n];
#pragma unroll
      for (int j = 0; j < n; ++j) g[j] = r.on ? r.neg * exp_at(E::at(v[u], j) - r.M, k) : 0.0f;
      const int64_t at = label - c * n;
      if (at >= 0 && at < n && r.on) {
#pragma unroll
        for (int j = 0; j < n; ++j) g[j] = at == j ? r.label_g : g[j];
      }
      store_run<n>(dy + c * n, g);
    }
  }
  const int64_t i = full * n + threadIdx.x;
  if (i < len) {
    const float g = !r.on ? 0.0f : i == label ? r.label_g : r.neg * exp_at(E::one(y[i]) - r.M, k);
    dy[i] = Elem<G>::from(g);
  }
}

// Workgroup n pieces + p: piece p of row n; the last workgroup: the loss.
template <typename T, typename G, bool kPairs>
__global__ __launch_bounds__(kRowThreads) void row_gradient_kernel(const RowArgs a) {
  const int64_t n = blockIdx.x / a.pieces;
  const int p = (int)(blockIdx.x % a.pieces);
  RowGrad r{0.0f, 0.0f, 0.0f, 0u};
  if constexpr (kPairs) {
    r = a.grad[n];
  } else {
    const float w = weight_of(a, n);
    if (w != 0.0f) {
      const float2 st = merged(a, n);
      const double logp = row_logp(a, n, st);
      double loss, slope;
      policy_row(a, n, logp, loss, slope);
      r = row_grad(a, (double)w * slope, logp, st);
    }
  }
  const int64_t c0 = p * a.width, c1 = c0 + a.width < a.V ? c0 + a.width : a.V;
  thread_gradient(static_cast<const T*>(a.Y) + n * a.y_stride + c0, static_cast<G*>(a.dY) + n * a.dy_stride + c0,
                  c1 - c0, (int64_t)a.labels[n] - c0, a.k, r);
}

// One workgroup: the policy loss's per-row outputs and the sum of either loss.
template <bool kPairs>
__global__ __launch_bounds__(kSumThreads) void loss_sum_kernel(const RowArgs a) {
  __shared__ double buf[kSumThreads / 64];
  double sum = 0.0;
  if constexpr (kPairs) {
    for (int64_t i = threadIdx.x; i < a.B; i += kSumThreads) sum += a.pair_loss[i];
  } else {
    for (int64_t n = threadIdx.x; n < a.N; n += kSumThreads) {
      const float w = weight_of(a, n);
      if (w == 0.0f) continue;
      const double logp = row_logp(a, n, merged(a, n));
      double loss, slope;
      policy_row(a, n, logp, loss, slope);
      if (a.logp) a.logp[n] = (float)logp;
      if (a.row_loss) a.row_loss[n] = (float)loss;
      sum += (double)w * loss;
    }
  }
  sum = block_sum<kSumThreads>(sum, buf);
  if (threadIdx.x == 0 && a.loss) *a.loss = (float)sum;
}

// ------------------------------------------------------------------- host ---

// Pieces a row is cut into: about 16384 workgroups in all (8 rounds of the
// GPU's 2048 resident ones), none under 2048 columns.
int64_t row_pieces(int64_t N, int64_t V) {
  const int64_t most = std::min<int64_t>(kMaxPieces, (V + 2047) / 2048);
  return std::max<int64_t>(1, std::min<int64_t>(most, 16384 / std::max<int64_t>(N, 1)));
}

struct LossWorkspace {
  uint64_t part, ylab, grad, pair_loss, total;
};

LossWorkspace loss_workspace(int64_t N, int64_t V, int64_t B) {
  LossWorkspace w{};
  auto take = [&](uint64_t bytes) {
    const uint64_t at = w.total;
    w.total += round_up(bytes, ARCHEAD_ALIGNMENT);
    return at;
  };
  w.part = take((uint64_t)N * (uint64_t)row_pieces(N, V) * sizeof(float2));
  w.ylab = take((uint64_t)N * 4);
  w.grad = take(B > 0 ? (uint64_t)N * sizeof(RowGrad) : 0);
  w.pair_loss = take((uint64_t)B * 8);
  return w;
}

int check_shape(int64_t N, int64_t V) {
  if (N < 0 || V < 1) return ARCHEAD_E_SHAPE;
  if (N > (int64_t(1) << 22) || V > (int64_t(1) << 31) - 1) return ARCHEAD_E_UNSUPPORTED;
  return ARCHEAD_OK;
}

int elem_size(int32_t dtype) { return dtype == ARCHEAD_F32 ? 4 : dtype == ARCHEAD_BF16 ? 2 : 0; }

// Whether two tensors of the same rows and columns share bytes: their spans
// meet, and they are not two column windows of rows of the same stride.
bool overlap(const archead_tensor* x, int xs, const archead_tensor* y, int ys) {
  const uint64_t a = (uint64_t)x->data, b = (uint64_t)y->data;
  const uint64_t sa = (uint64_t)x->row_stride * xs, sb = (uint64_t)y->row_stride * ys;
  const uint64_t ra = (uint64_t)x->cols * xs, rb = (uint64_t)y->cols * ys, rows = (uint64_t)x->rows;
  if (a + (rows - 1) * sa + ra <= b || b + (rows - 1) * sb + rb <= a) return false;
  if (sa != sb) return true;
  const uint64_t off = (b >= a ? b - a : sa - (a - b) % sa) % sa;
  return !(off >= ra && off + rb <= sa);
}

int check_rows(const archead_tensor* Y, const archead_tensor* dY, float s) {
  const int ys = elem_size(Y->dtype);
  if (!ys || (dY && !elem_size(dY->dtype))) return ARCHEAD_E_DTYPE;
  if (int rc = check_shape(Y->rows, Y->cols)) return rc;
  if (Y->row_stride < Y->cols) return ARCHEAD_E_SHAPE;
  if (dY && (dY->rows != Y->rows || dY->cols != Y->cols || dY->row_stride < dY->cols)) return ARCHEAD_E_SHAPE;
  if (!(s > 0.0f) || !isfinite(s)) return ARCHEAD_E_VALUE;
  return ARCHEAD_OK;
}

int check_row_pointers(const archead_tensor* Y, const archead_tensor* dY) {
  if (!Y->data || (dY && !dY->data)) return ARCHEAD_E_NULL;
  const int ys = elem_size(Y->dtype), gs = dY ? elem_size(dY->dtype) : 1;
  if ((uintptr_t)Y->data % ys || (dY && (uintptr_t)dY->data % gs)) return ARCHEAD_E_ALIGN;
  if (dY) {
    const bool in_place = dY->data == Y->data && dY->dtype == Y->dtype && dY->row_stride == Y->row_stride;
    if (!in_place && overlap(Y, ys, dY, gs)) return ARCHEAD_E_SHAPE;
  }
  return ARCHEAD_OK;
}

int check_words(std::initializer_list<const void*> pointers) {
  for (const void* p : pointers)
    if ((uintptr_t)p % 4) return ARCHEAD_E_ALIGN;
  return ARCHEAD_OK;
}

int check_workspace(const void* ws, uint64_t bytes, uint64_t need) {
  if (!ws) return ARCHEAD_E_NULL;
  if ((uintptr_t)ws % ARCHEAD_ALIGNMENT) return ARCHEAD_E_ALIGN;
  return bytes < need ? ARCHEAD_E_WORKSPACE : ARCHEAD_OK;
}

RowArgs row_args(const archead_tensor* Y, const archead_tensor* dY, float s, void* workspace, const LossWorkspace& W) {
  RowArgs a{};
  a.Y = Y->data;
  a.N = Y->rows;
  a.V = Y->cols;
  a.y_stride = Y->row_stride;
  if (dY) {
    a.dY = dY->data;
    a.dy_stride = dY->row_stride;
  }
  a.pieces = (int)row_pieces(a.N, a.V);
  a.width = (int64_t)round_up((uint64_t)((a.V + a.pieces - 1) / a.pieces), 8);
  a.s = s;
  const double k = (double)s * 1.44269504088896340736;
  a.k.hi = (float)k;
  a.k.lo = (float)(k - (double)a.k.hi);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part = reinterpret_cast<float2*>(ws + W.part);
  a.ylab = reinterpret_cast<float*>(ws + W.ylab);
  a.grad = reinterpret_cast<RowGrad*>(ws + W.grad);
  a.pair_loss = reinterpret_cast<double*>(ws + W.pair_loss);
  return a;
}

template <typename T, bool kPairs>
hipError_t launch_loss(const RowArgs& a, const archead_tensor* dY, hipStream_t s) {
  const dim3 grid((unsigned)(a.N * a.pieces)), block(kRowThreads);
  (void)hipGetLastError();  // start from a clean error state
  if (a.N > 0) hipLaunchKernelGGL((row_pieces_kernel<T, kPairs>), grid, block, 0, s, a);
  if constexpr (kPairs) {
    if (a.B > 0) hipLaunchKernelGGL(pair_kernel, dim3((unsigned)a.B), block, 0, s, a);
  }
  if (a.loss || a.logp || a.row_loss)
    hipLaunchKernelGGL(loss_sum_kernel<kPairs>, dim3(1), dim3(kSumThreads), 0, s, a);
  if (!dY || a.N == 0) return hipGetLastError();
  if (dY->dtype == ARCHEAD_BF16)
    hipLaunchKernelGGL((row_gradient_kernel<T, uint16_t, kPairs>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((row_gradient_kernel<T, float, kPairs>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <bool kPairs>
int run_loss(const RowArgs& a, const archead_tensor* Y, const archead_tensor* dY, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = Y->dtype == ARCHEAD_BF16 ? launch_loss<uint16_t, kPairs>(a, dY, s)
                                                : launch_loss<float, kPairs>(a, dY, s);
  return e == hipSuccess ? ARCHEAD_OK : ARCHEAD_E_HIP;
}

}  // namespace
}  // namespace archead

using namespace archead;

extern "C" {

int archead_loss_workspace_bytes(int64_t n_rows, int64_t V, int64_t n_pairs, uint64_t* bytes) {
  if (!bytes) return ARCHEAD_E_NULL;
  if (int rc = check_shape(n_rows, V)) return rc;
  if (n_pairs < 0) return ARCHEAD_E_SHAPE;
  if (n_pairs > (int64_t(1) << 22)) return ARCHEAD_E_UNSUPPORTED;
  *bytes = loss_workspace(n_rows, V, n_pairs).total;
  return ARCHEAD_OK;
}

int archead_policy_loss(const archead_tensor* Y, const archead_policy_inputs* in, const archead_policy_outputs* out,
                        void* workspace, uint64_t workspace_bytes, void* stream) {
  if (!Y || !in || !out) return ARCHEAD_E_NULL;
  if (int rc = check_rows(Y, out->dY, in->inv_temperature)) return rc;
  if (!(in->clip_low >= 0.0f) || !(in->clip_high >= 0.0f) || !(in->kl_coef >= 0.0f) || isinf(in->kl_coef))
    return ARCHEAD_E_VALUE;
  if (Y->rows > 0) {
    if (!in->labels || !in->advantage || (in->kl_coef != 0.0f && !in->ref_logp)) return ARCHEAD_E_NULL;
    if (int rc = check_row_pointers(Y, out->dY)) return rc;
  }
  if (int rc = check_words({in->labels, in->weight, in->old_logp, in->ref_logp, in->advantage, out->loss, out->logp,
                            out->row_loss}))
    return rc;
  const LossWorkspace W = loss_workspace(Y->rows, Y->cols, 0);
  if (W.total > 0)
    if (int rc = check_workspace(workspace, workspace_bytes, W.total)) return rc;
  if (Y->rows == 0 && !out->loss) return ARCHEAD_OK;
  RowArgs a = row_args(Y, out->dY, in->inv_temperature, workspace, W);
  a.labels = in->labels;
  a.weight = in->weight;
  a.old_logp = in->old_logp;
  a.ref_logp = in->ref_logp;
  a.advantage = in->advantage;
  a.clip_low = in->clip_low;
  a.clip_high = in->clip_high;
  a.kl_coef = in->kl_coef;
  a.loss = out->loss;
  a.logp = out->logp;
  a.row_loss = out->row_loss;
  return run_loss<false>(a, Y, out->dY, stream);
}

int archead_preference_loss(const archead_tensor* Y, const archead_preference_inputs* in,
                            const archead_preference_outputs* out, void* workspace, uint64_t workspace_bytes,
                            void* stream) {
  if (!Y || !in || !out) return ARCHEAD_E_NULL;
  if (int rc = check_rows(Y, out->dY, in->inv_temperature)) return rc;
  if (in->n_pairs < 0) return ARCHEAD_E_SHAPE;
  if (in->n_pairs > (int64_t(1) << 22) || (in->kind != ARCHEAD_PREF_SIGMOID && in->kind != ARCHEAD_PREF_SQUARED))
    return ARCHEAD_E_UNSUPPORTED;
  if (!(in->beta > 0.0f) || isinf(in->beta) || !(in->label_smoothing >= 0.0f) || !(in->label_smoothing < 0.5f))
    return ARCHEAD_E_VALUE;
  if (!in->offsets) return ARCHEAD_E_NULL;
  if (Y->rows > 0) {
    if (!in->labels) return ARCHEAD_E_NULL;
    if (int rc = check_row_pointers(Y, out->dY)) return rc;
  }
  if (int rc = check_words({in->labels, in->weight, in->ref_logp, in->offsets, in->pair_weight, out->loss, out->logp,
                            out->chosen_reward, out->rejected_reward}))
    return rc;
  const LossWorkspace W = loss_workspace(Y->rows, Y->cols, in->n_pairs);
  if (W.total > 0)
    if (int rc = check_workspace(workspace, workspace_bytes, W.total)) return rc;
  if (Y->rows == 0 && in->n_pairs == 0 && !out->loss) return ARCHEAD_OK;
  RowArgs a = row_args(Y, out->dY, in->inv_temperature, workspace, W);
  a.labels = in->labels;
  a.weight = in->weight;
  a.ref_logp = in->ref_logp;
  a.offsets = in->offsets;
  a.B = in->n_pairs;
  a.pair_weight = in->pair_weight;
  a.beta = in->beta;
  a.smoothing = in->label_smoothing;
  a.kind = in->kind;
  a.loss = out->loss;
  a.logp = out->logp;
  a.chosen = out->chosen_reward;
  a.rejected = out->rejected_reward;
  return run_loss<true>(a, Y, out->dY, stream);
}

}  // extern "C"
