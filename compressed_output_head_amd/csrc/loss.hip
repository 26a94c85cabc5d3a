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
//   e_j = 2^(k (y_j - M)),  S = sum of e_j but the label's,  E = exp(s (y_label - M)),
//   log p = -ln(1 + S / E) where S < E, else s (y_label - M) - ln(S + E),
// M being the maximum without the label too.  The last two and all per-row
// arithmetic after them are fp64 (a loss is a sum of terms of both signs, and
// one row is one thread's work).  With the label's own term in S, a row with p
// close to 1 would lose log p in its rounding, as 1 + S rounds S's digits off;
// so S / E keeps them, and so does the label's element of the gradient,
// -coef s expm1(log p).  The difference y - M is taken before the product: a
// fused k y - k M would save an instruction, but overflows where every logit
// of a piece is the type's lowest value.  S is summed in fp32 trees of 8 to 32
// terms, and in fp64 from there.
//
// A row is cut into pieces so that few rows still fill the GPU:
//   row_pieces_kernel   (M, S) of every piece without the label, and the label's logit
//   rows_kernel         a row's pieces merged, its loss and its coefficient
//   pair_kernel         preference loss only: the sequences' sums, the pair's
//                       loss and its slope for every row
//   row_gradient_kernel the gradient, piece by piece; one more workgroup adds
//                       up the loss
// which reads the logits twice, as the coefficient of a row needs all of it (of
// a pair, all of the pair).  Many rows of a policy loss take another way, that
// reads most of them once:
//   row_order_kernel, policy_fused_kernel, loss_total_kernel
// and so do calls whose launches take longer than their work:
//   small_loss_kernel                          a few short rows
//   row_pieces_kernel, few_gradient_kernel     a few long ones
// Rows of weight zero are neither read nor counted; their gradient is zero.
// Every sum has a fixed order, so results do not depend on scheduling.
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <limits>

#include "device_common.h"
#include "internal.h"

namespace archead {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;        // 16-byte loads in flight per thread
constexpr int kPairThreads = 1024;
constexpr int kFusedThreads = 1024;
constexpr int kOrderThreads = 1024;
constexpr int kSmallThreads = 1024;
constexpr int kSmallRows = 64;       // and pairs, of small_loss_kernel
constexpr int kFewRows = 16;         // of few_gradient_kernel
constexpr int kHeldChunks = 12;      // of 16 bytes, in registers
constexpr int64_t kFusedLeastRows = 256;   // one per CU
constexpr int64_t kMaxPieces = 64;
constexpr int64_t kTargetGroups = 12288, kLeastWidth = 2048;

// What the gradient of a row needs: dY_j = neg 2^(k (y_j - M)), label_g at the label.
struct RowGrad {
  float neg, M, label_g;
  uint32_t on;  // 0: the gradient is zero
};

// s log2 e = hi + lo, both above zero
struct Scale {
  float hi, lo;
};

// The maximum M of some logits and the sum S of 2^(k (y - M)).
struct Stat {
  double S;
  float M;
};

struct RowArgs {
  const void* Y;
  void* dY;
  int64_t N, V, y_stride, dy_stride;
  int64_t width;  // columns of a piece
  int pieces;
  int lanes;      // that merge a row's pieces
  Scale k;
  float s;
  const int32_t* labels;
  const float* weight;
  // workspace
  Stat* part;      // [N][pieces]
  float* ylab;     // [N]
  RowGrad* grad;   // [N]
  double* term;    // [N] weighted, of the loss (policy) or of the sequence's sum (preference)
  float* row_slope;   // [N], preference loss: of the pair's loss in the row's log-probability; else null
  double* pair_loss;  // [B]
  int32_t* order;     // [N + 1], policy loss
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

// n = 4 or 8 values to consecutive elements, 16 or 8 bytes a store.  Gradients
// are written once and too large to wait for their reader in the cache; stores
// that say so leave it to the logits, which are read twice (480 rows of a
// preference loss took 74 us with them and 83 without, 4096 rows 513 and 537).
template <int n>
__device__ __forceinline__ void store_run(uint16_t* p, const float* g) {
  if constexpr (n == 8) {
    const u2 a = pack_bf16x4(g[0], g[1], g[2], g[3]), b = pack_bf16x4(g[4], g[5], g[6], g[7]);
    __builtin_nontemporal_store(u4_any(u4{a[0], a[1], b[0], b[1]}), reinterpret_cast<u4_any*>(p));
  } else {
    __builtin_nontemporal_store(u2_any(pack_bf16x4(g[0], g[1], g[2], g[3])), reinterpret_cast<u2_any*>(p));
  }
}
template <int n>
__device__ __forceinline__ void store_run(float* p, const float* g) {
#pragma unroll
  for (int i = 0; i < n; i += 4) {
    const f4 v = {g[i], g[i + 1], g[i + 2], g[i + 3]};
    __builtin_nontemporal_store(u4_any(__builtin_bit_cast(u4, v)), reinterpret_cast<u4_any*>(p + i));
  }
}

// 2^(k d).  d is -inf where a logit or a running maximum is: both products are
// -inf then and the result 0, as neither part of k is negative or zero.
__device__ __forceinline__ float exp_at(float d, Scale k) {
  return __builtin_amdgcn_exp2f(fmaf(d, k.hi, d * k.lo));
}

// What is subtracted from logits of maximum M: nothing where all are -inf.
__device__ __forceinline__ float shift_of(float M) { return M == -INFINITY ? 0.0f : M; }

// Two (M, S) pieces as one.
__device__ __forceinline__ Stat merge(Stat a, Stat b, Scale k) {
  const float M = fmaxf(a.M, b.M), M0 = shift_of(M);
  return Stat{a.S * (double)exp_at(a.M - M0, k) + b.S * (double)exp_at(b.M - M0, k), M};
}

__device__ __forceinline__ Stat lane_xor(Stat v, int o) { return Stat{__shfl_xor(v.S, o), __shfl_xor(v.M, o)}; }

__device__ __forceinline__ Stat wave_merge(Stat v, Scale k) {
  for (int o = 32; o > 0; o >>= 1) v = merge(v, lane_xor(v, o), k);
  return v;
}

template <int kThreads>
__device__ __forceinline__ Stat block_merge(Stat v, Scale k, Stat* buf) {
  v = wave_merge(v, k);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < kThreads / 64; ++w) v = merge(v, buf[w], k);
  return v;
}

__device__ __forceinline__ double wave_sum(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int kThreads>
__device__ __forceinline__ double block_sum(double v, double* buf) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < kThreads / 64; ++w) v += buf[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ float weight_of(const RowArgs& a, int64_t n) { return a.weight ? a.weight[n] : 1.0f; }

// Whether row n counts: its weight, and for pairs a place in a sequence.
template <bool kPairs>
__device__ __forceinline__ bool row_counts(const RowArgs& a, int64_t n) {
  if (kPairs && !(n >= a.offsets[0] && n < a.offsets[2 * a.B])) return false;
  return weight_of(a, n) != 0.0f;
}

// The sum of 2^(k (y - M0)) over a chunk, as a tree: one large term does not
// round with every small one.
template <typename T>
__device__ __forceinline__ float chunk_sum(const u4& v, float M0, Scale k) {
  using E = Elem<T>;
  float e[E::kPer16];
#pragma unroll
  for (int j = 0; j < E::kPer16; ++j) e[j] = exp_at(E::at(v, j) - M0, k);
#pragma unroll
  for (int w = E::kPer16 / 2; w > 0; w >>= 1)
#pragma unroll
    for (int j = 0; j < w; ++j) e[j] += e[j + w];
  return e[0];
}

// A chunk whose element j is -inf.
template <typename T>
__device__ __forceinline__ u4 without(u4 v, int j) {
  constexpr int n = Elem<T>::kPer16 / 4;  // elements of a word
  const uint32_t keep = n == 1 ? 0u : 0xffff0000u >> (16 * (j & 1));
#pragma unroll
  for (int w = 0; w < 4; ++w) v[w] = w == j / n ? (v[w] & keep) | (Elem<T>::kNegInf2 & ~keep) : v[w];
  return v;
}

// The largest logit of a chunk; NaN is passed over (it is in the sum).
template <typename T>
__device__ __forceinline__ float chunk_max(const u4& v) {
  float top = Elem<T>::at(v, 0);
#pragma unroll
  for (int j = 1; j < Elem<T>::kPer16; ++j) top = fmaxf(top, Elem<T>::at(v, j));
  return top;
}

// (M, S) of the elements [0, len) at p but that at `label` (none where it is
// negative), the share of thread tid of kThreads.
template <typename T, int kThreads>
__device__ __forceinline__ Stat thread_stats(const T* p, int64_t len, int64_t label, Scale k, int tid) {
  using E = Elem<T>;
  const int64_t full = len / E::kPer16;
  const int64_t label_chunk = label >= 0 && label / E::kPer16 % kThreads == tid ? label / E::kPer16 : -1;
  float M = -INFINITY, M0 = 0.0f;
  double S = 0.0;
  auto rise = [&](float top) {  // of the running maximum
    if (top > M) {
      S *= (double)exp_at(M - top, k);
      M = M0 = top;
    }
  };
  for (int64_t c0 = tid; c0 < full; c0 += kThreads * kRowUnroll) {
    u4 v[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int64_t c = c0 + u * kThreads;
      v[u] = c < full ? u4(*reinterpret_cast<const u4_any*>(p + c * E::kPer16))
                      : u4{E::kNegInf2, E::kNegInf2, E::kNegInf2, E::kNegInf2};
    }
    if (label_chunk >= c0 && label_chunk < c0 + kThreads * kRowUnroll) {
#pragma unroll
      for (int u = 0; u < kRowUnroll; ++u)
        if (c0 + u * kThreads == label_chunk) v[u] = without<T>(v[u], (int)(label % E::kPer16));
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) top = fmaxf(top, chunk_max<T>(v[u]));
    rise(top);
    float add[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) add[u] = chunk_sum<T>(v[u], M0, k);
    S += (double)((add[0] + add[1]) + (add[2] + add[3]));
  }
  const int64_t i = full * E::kPer16 + tid;  // fewer than 8 elements are left
  if (i < len && i != label) {
    const float y = E::one(p[i]);
    rise(y);
    S += (double)exp_at(y - M0, k);
  }
  return Stat{S, M};
}

template <typename T, bool kPairs>
__global__ __launch_bounds__(kRowThreads) void row_pieces_kernel(const RowArgs a) {
  __shared__ Stat buf[kRowThreads / 64];
  const int64_t n = blockIdx.x / a.pieces;
  const int p = (int)(blockIdx.x % a.pieces);
  if (!row_counts<kPairs>(a, n)) return;
  const T* row = static_cast<const T*>(a.Y) + n * a.y_stride;
  const int64_t c0 = p * a.width, c1 = c0 + a.width < a.V ? c0 + a.width : a.V;
  const int64_t label = a.labels[n];
  const bool valid = label >= 0 && label < a.V;
  // read here, before any launch that may write the gradient over Y
  if (threadIdx.x == 0 && (valid ? label >= c0 && label < c1 : p == 0))
    a.ylab[n] = valid ? Elem<T>::one(row[label]) : __builtin_nanf("");
  const int64_t place = valid && label < c1 ? label - c0 : -1;  // negative in a later piece too
  const Stat r =
      block_merge<kRowThreads>(thread_stats<T, kRowThreads>(row + c0, c1 - c0, place, a.k, threadIdx.x), a.k, buf);
  if (threadIdx.x == 0) a.part[n * a.pieces + p] = r;
}

// (M, S) of row n, merged by a.lanes neighbouring lanes (a power of two that
// divides 64), of which this is number `lane`; all of them return it.
__device__ __forceinline__ Stat merged(const RowArgs& a, int64_t n, int lane) {
  Stat r = lane < a.pieces ? a.part[n * a.pieces + lane] : Stat{0.0, -INFINITY};
  for (int p = lane + a.lanes; p < a.pieces; p += a.lanes) r = merge(r, a.part[n * a.pieces + p], a.k);
  for (int o = a.lanes >> 1; o > 0; o >>= 1) r = merge(r, lane_xor(r, o), a.k);
  return r;
}

// What the policy loss has of one row, and what comes of it.
struct PolicyRow {
  double S;
  float y_label, M, advantage, old_logp, ref_logp, weight;
};
struct PolicyResult {
  double loss, term;  // term = weight loss
  float logp;
  RowGrad grad;
};
struct PolicyScalars {
  float s, clip_low, clip_high, kl_coef;
  uint32_t own_ratio;  // 1: the policy that sampled is this one
};

// A row's log-probability, its S with the label's term, and the M that S is by.
struct RowLogp {
  double logp, S;
  float M;
};
__device__ __forceinline__ RowLogp row_logp(const PolicyRow& x, double s) {
  // NaN and +inf have no log p; neither has a row with nothing above -inf, where the difference is NaN
  const double y = x.y_label < INFINITY ? (double)x.y_label : __builtin_nan("");
  const float M = x.M == -INFINITY ? x.y_label : x.M;  // the label is all there is
  const double t = s * (y - (double)M), E = exp(t), S = x.S + E;
  return RowLogp{x.S < E ? 0.0 - log1p(x.S / E) : t - log(S), S, M};
}

// Not inlined: in a loop, the compiler would hold every constant of the fp64
// functions in registers that the row needs.
__device__ __attribute__((noinline)) PolicyResult policy_row(PolicyRow x, PolicyScalars p) {
  const double s = p.s, w = x.weight, A = x.advantage;
  const RowLogp row = row_logp(x, s);
  const double logp = row.logp;
  // this policy's own ratio is 1 at a log p of -inf too
  const double ratio = !p.own_ratio ? exp(logp - (double)x.old_logp) : logp == logp ? 1.0 : logp;
  const double lo = 1.0 - (double)p.clip_low, hi = 1.0 + (double)p.clip_high;
  const double kept = ratio < lo ? lo : ratio > hi ? hi : ratio;  // NaN stays NaN
  const bool plain = !(kept * A < ratio * A);  // the unclipped term is the smaller one
  double loss = plain ? -(ratio * A) : -(kept * A);
  double slope = plain ? -(ratio * A) : 0.0;  // the loss's derivative in logp
  if (p.kl_coef != 0.0f) {
    const double d = (double)x.ref_logp - logp, e = expm1(d);
    loss += (double)p.kl_coef * (e - d);
    slope -= (double)p.kl_coef * e;
  }
  const double c = w * slope * s;
  return PolicyResult{loss, w * loss, (float)logp,
                      RowGrad{(float)(-c / row.S), row.M, (float)(-c * expm1(logp)), c != 0.0 ? 1u : 0u}};
}

__device__ __forceinline__ PolicyScalars policy_scalars(const RowArgs& a) {
  return PolicyScalars{a.s, a.clip_low, a.clip_high, a.kl_coef, a.old_logp ? 0u : 1u};
}

// A row of a pair: its term of the sequence's sum, and its gradient but for
// the slope of the pair's loss.
__device__ __forceinline__ PolicyResult pair_row(const PolicyRow& x, float s) {
  const RowLogp row = row_logp(x, s);
  const double w = x.weight, c = w * (double)s;
  return PolicyResult{0.0, w * (row.logp - (double)x.ref_logp), (float)row.logp,
                      RowGrad{(float)(-c / row.S), row.M, (float)(-c * expm1(row.logp)), 1u}};
}

template <bool kPairs>
__device__ __forceinline__ PolicyRow row_inputs(const RowArgs& a, int64_t n) {
  PolicyRow x{};
  x.ref_logp = a.ref_logp ? a.ref_logp[n] : 0.0f;
  x.weight = weight_of(a, n);
  if constexpr (!kPairs) {
    x.advantage = a.advantage[n];
    x.old_logp = a.old_logp ? a.old_logp[n] : 0.0f;
  }
  return x;
}

template <bool kPairs>
__device__ __forceinline__ PolicyResult row_result(const RowArgs& a, const PolicyRow& x) {
  if constexpr (kPairs)
    return pair_row(x, a.s);
  else
    return policy_row(x, policy_scalars(a));
}

__device__ __forceinline__ void write_row(const RowArgs& a, int64_t n, const PolicyResult& r) {
  if (a.logp) a.logp[n] = r.logp;
  if (a.row_loss) a.row_loss[n] = (float)r.loss;
}

// a.lanes lanes a row: its log-probability, its term of the loss (or of its
// sequence's sum) and what its gradient needs, for pairs still to be
// multiplied by the slope of the pair's loss.  (The fp64 functions here take
// about as many instructions as a thread's share of a short row, so no
// gradient workgroup repeats them.)
template <bool kPairs>
__global__ __launch_bounds__(kRowThreads) void rows_kernel(const RowArgs a) {
  const int64_t t = (int64_t)blockIdx.x * kRowThreads + threadIdx.x, n = t / a.lanes;
  const int lane = (int)(t % a.lanes);
  if (n >= a.N) return;
  PolicyResult r{};
  if (row_counts<kPairs>(a, n)) {
    PolicyRow x = row_inputs<kPairs>(a, n);
    const Stat st = merged(a, n, lane);
    x.y_label = a.ylab[n];
    x.M = st.M;
    x.S = st.S;
    r = row_result<kPairs>(a, x);
  }
  if (lane != 0) return;
  a.grad[n] = r.grad;
  a.term[n] = r.term;
  if (kPairs) a.row_slope[n] = 0.0f;
  write_row(a, n, r);
}

// Rows [first, last) of sequence q; offsets outside [0, N] end at its borders.
__device__ __forceinline__ int64_t sequence_start(const RowArgs& a, int64_t q) {
  const int64_t o = a.offsets[q];
  return o < 0 ? (int64_t)0 : o > a.N ? a.N : o;
}

// Pair i from its sequences' sums: its outputs, its loss and the loss's
// derivative in h = sum[0] - sum[1], both weighted.
struct PairResult {
  double loss, slope;
};
__device__ __forceinline__ PairResult pair_result(const RowArgs& a, int64_t i, double sum0, double sum1, bool writes) {
  const double pw = a.pair_weight ? (double)a.pair_weight[i] : 1.0;
  const double h = sum0 - sum1, beta = a.beta, eps = a.smoothing;
  double loss, slope;
  if (a.kind == ARCHEAD_PREF_SIGMOID) {
    const double x = beta * h, e = exp(-fabs(x)), t = log1p(e);  // softplus(x) = max(x, 0) + t
    loss = (1.0 - eps) * ((x < 0.0 ? -x : 0.0) + t) + eps * ((x > 0.0 ? x : 0.0) + t);
    slope = beta * (eps - (x < 0.0 ? 1.0 : e) / (1.0 + e));
  } else {
    const double u = h - 0.5 / beta;
    loss = u * u;
    slope = 2.0 * u;
  }
  if (writes) {
    if (a.chosen) a.chosen[i] = (float)(beta * sum0);
    if (a.rejected) a.rejected[i] = (float)(beta * sum1);
  }
  // a pair of weight zero is left out, whatever its rows hold
  return pw != 0.0 ? PairResult{pw * loss, pw * slope} : PairResult{0.0, 0.0};
}

// Workgroup i: pair i.  Its sequences are neighbours, so one walk over their
// rows takes both.
__global__ __launch_bounds__(kPairThreads) void pair_kernel(const RowArgs a) {
  __shared__ double buf[2][kPairThreads / 64];
  const int64_t i = blockIdx.x;
  const int64_t b0 = sequence_start(a, 2 * i), b1 = sequence_start(a, 2 * i + 1), b2 = sequence_start(a, 2 * i + 2);
  double sum[2] = {0.0, 0.0};
  for (int64_t n = b0 + threadIdx.x; n < b1; n += kPairThreads) sum[0] += a.term[n];
  for (int64_t n = b1 + threadIdx.x; n < b2; n += kPairThreads) sum[1] += a.term[n];
  for (int side = 0; side < 2; ++side) sum[side] = block_sum<kPairThreads>(sum[side], buf[side]);
  const PairResult r = pair_result(a, i, sum[0], sum[1], threadIdx.x == 0);
  if (threadIdx.x == 0) a.pair_loss[i] = r.loss;
  for (int64_t n = b0 + threadIdx.x; n < b1; n += kPairThreads) a.row_slope[n] = (float)r.slope;
  for (int64_t n = b1 + threadIdx.x; n < b2; n += kPairThreads) a.row_slope[n] = (float)-r.slope;
}

// The elements [0, len) of a gradient row, the share of thread tid of kThreads;
// `label` is the label's place in them, or no place.
template <typename T, typename G, int kThreads>
__device__ __forceinline__ void thread_gradient(const T* y, G* dy, int64_t len, int64_t label, Scale k, RowGrad r,
                                                int tid) {
  using E = Elem<T>;
  constexpr int n = E::kPer16;
  const int64_t full = len / n;
  for (int64_t c0 = tid; c0 < full; c0 += kThreads * kRowUnroll) {
    u4 v[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int64_t c = c0 + u * kThreads;
      if (r.on && c < full) v[u] = *reinterpret_cast<const u4_any*>(y + c * n);
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int64_t c = c0 + u * kThreads;
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
  const int64_t i = full * n + tid;
  if (i < len) {
    const float g = !r.on ? 0.0f : i == label ? r.label_g : r.neg * exp_at(E::one(y[i]) - r.M, k);
    dy[i] = Elem<G>::from(g);
  }
}

// The loss from its rows' or pairs' parts, by one workgroup.
__device__ __forceinline__ void loss_total(const RowArgs& a) {
  __shared__ double buf[kRowThreads / 64];
  double sum = 0.0;
  const double* parts = a.row_slope ? a.pair_loss : a.term;
  const int64_t count = a.row_slope ? a.B : a.N;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < count; i += kRowThreads) sum += parts[i];
  sum = block_sum<kRowThreads>(sum, buf);
  if (threadIdx.x == 0 && a.loss) *a.loss = (float)sum;
}

__global__ __launch_bounds__(kRowThreads) void loss_total_kernel(const RowArgs a) { loss_total(a); }

template <typename T, typename G>
__device__ __forceinline__ void piece_gradient(const RowArgs& a, int64_t n, int p, const RowGrad& r) {
  const int64_t c0 = p * a.width, c1 = c0 + a.width < a.V ? c0 + a.width : a.V;
  thread_gradient<T, G, kRowThreads>(static_cast<const T*>(a.Y) + n * a.y_stride + c0,
                                     static_cast<G*>(a.dY) + n * a.dy_stride + c0, c1 - c0,
                                     (int64_t)a.labels[n] - c0, a.k, r, threadIdx.x);
}

__device__ __forceinline__ RowGrad with_slope(RowGrad r, float slope) {
  r.neg *= slope;
  r.label_g *= slope;
  r.on = r.on && slope != 0.0f;
  return r;
}

// Workgroup n pieces + p: piece p of row N - 1 - n; one more: the loss.  (The
// last rows that row_pieces_kernel read come first, while they are cached:
// 4096 rows of a preference loss take 499 us, and 523 in the other order.)
template <typename T, typename G>
__global__ __launch_bounds__(kRowThreads) void row_gradient_kernel(const RowArgs a) {
  const int p = (int)(blockIdx.x % a.pieces);
  if (blockIdx.x / a.pieces >= a.N) return loss_total(a);
  const int64_t n = a.N - 1 - blockIdx.x / a.pieces;
  RowGrad r = a.grad[n];
  if (a.row_slope) r = with_slope(r, a.row_slope[n]);
  piece_gradient<T, G>(a, n, p, r);
}

// The same for a policy loss of so few rows that one launch less is worth
// working a row's numbers out in each of its workgroups (a.lanes is 64).
template <typename T, typename G>
__global__ __launch_bounds__(kRowThreads) void few_gradient_kernel(const RowArgs a) {
  __shared__ RowGrad grad;
  __shared__ double terms[kFewRows];
  const int64_t n = blockIdx.x / a.pieces;
  const int p = (int)(blockIdx.x % a.pieces);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto result = [&](int64_t row) {
    if (!row_counts<false>(a, row)) return PolicyResult{};
    PolicyRow x = row_inputs<false>(a, row);
    const Stat st = merged(a, row, lane);
    x.y_label = a.ylab[row];
    x.M = st.M;
    x.S = st.S;
    return row_result<false>(a, x);
  };
  if (n >= a.N) {
    for (int64_t row = wave; row < a.N; row += kRowThreads / 64) {
      const PolicyResult r = result(row);
      if (lane != 0) continue;
      terms[row] = r.term;
      write_row(a, row, r);
    }
    __syncthreads();
    double sum = 0.0;
    for (int64_t row = 0; row < a.N; ++row) sum += terms[row];
    if (threadIdx.x == 0 && a.loss) *a.loss = (float)sum;
    return;
  }
  if (wave == 0) {
    const PolicyResult r = result(n);
    if (lane == 0) grad = r.grad;
  }
  __syncthreads();
  piece_gradient<T, G>(a, n, p, grad);
}

// Either loss of a few short rows in one launch of one workgroup: a wave a
// row, what rows and pairs tell each other in LDS.
template <typename T, typename G, bool kPairs>
__global__ __launch_bounds__(kSmallThreads) void small_loss_kernel(const RowArgs a) {
  constexpr int kWaves = kSmallThreads / 64;
  __shared__ RowGrad grad[kSmallRows];
  __shared__ double term[kSmallRows], pair_loss[kSmallRows];
  __shared__ float slope[kSmallRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto row_of = [&](int64_t n) { return static_cast<const T*>(a.Y) + n * a.y_stride; };
  for (int n = wave; n < a.N; n += kWaves) {
    PolicyResult r{};
    if (row_counts<kPairs>(a, n)) {
      PolicyRow x = row_inputs<kPairs>(a, n);
      const int64_t label = a.labels[n];
      const bool valid = label >= 0 && label < a.V;
      x.y_label = valid ? Elem<T>::one(row_of(n)[label]) : __builtin_nanf("");
      const Stat st = wave_merge(thread_stats<T, 64>(row_of(n), a.V, valid ? label : -1, a.k, lane), a.k);
      x.M = st.M;
      x.S = st.S;
      r = row_result<kPairs>(a, x);
    }
    if (lane != 0) continue;
    grad[n] = r.grad;
    term[n] = r.term;
    slope[n] = kPairs ? 0.0f : 1.0f;
    write_row(a, n, r);
  }
  __syncthreads();
  if constexpr (kPairs) {
    for (int i = wave; i < a.B; i += kWaves) {
      const int64_t b0 = sequence_start(a, 2 * i), b1 = sequence_start(a, 2 * i + 1), b2 = sequence_start(a, 2 * i + 2);
      const double sum0 = wave_sum(b0 + lane < b1 ? term[b0 + lane] : 0.0);  // at most 64 rows
      const double sum1 = wave_sum(b1 + lane < b2 ? term[b1 + lane] : 0.0);
      const PairResult r = pair_result(a, i, sum0, sum1, lane == 0);
      if (lane == 0) pair_loss[i] = r.loss;
      if (b0 + lane < b1) slope[b0 + lane] = (float)r.slope;
      if (b1 + lane < b2) slope[b1 + lane] = (float)-r.slope;
    }
    __syncthreads();
  }
  if (wave == 0) {
    const double* parts = kPairs ? pair_loss : term;
    const double sum = wave_sum(lane < (kPairs ? a.B : a.N) ? parts[lane] : 0.0);
    if (lane == 0 && a.loss) *a.loss = (float)sum;
  }
  if (!a.dY) return;
  for (int n = wave; n < a.N; n += kWaves)
    thread_gradient<T, G, 64>(row_of(n), static_cast<G*>(a.dY) + n * a.dy_stride, a.V, a.labels[n], a.k,
                              with_slope(grad[n], slope[n]), lane);
}

// The rows in the order policy_fused_kernel takes them: those that count from
// the front, the others from the back, so that every workgroup gets the same
// number of each to within one.
__global__ __launch_bounds__(kOrderThreads) void row_order_kernel(const RowArgs a) {
  constexpr int kWaves = kOrderThreads / 64;
  __shared__ int count[2][kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t front = 0, back = 0;  // rows placed so far
  int turn = 0;
  auto counts = [&](int64_t n) { return n < a.N && row_counts<false>(a, n); };
  bool later = counts(threadIdx.x);
  for (int64_t n0 = 0; n0 < a.N; n0 += kOrderThreads, turn ^= 1) {
    const int64_t n = n0 + threadIdx.x;
    const bool in = n < a.N, on = later;
    later = counts(n + kOrderThreads);  // the next rows' weights are on their way meanwhile
    const uint64_t ons = __ballot(on);
    if (lane == 0) count[turn][wave] = __popcll(ons);
    __syncthreads();  // the other turn's counts are read before the next one's are written
    int before = 0, all = 0;
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? count[turn][w] : 0;
      all += count[turn][w];
    }
    const int rank = before + __popcll(ons & ((1ull << lane) - 1));  // rows that count before this one
    const int64_t here = a.N - n0 < kOrderThreads ? a.N - n0 : kOrderThreads;
    if (on) a.order[front + rank] = (int32_t)n;
    if (in && !on) a.order[a.N - 1 - (back + (threadIdx.x - rank))] = (int32_t)n;
    front += all;
    back += here - all;
  }
  if (threadIdx.x == 0) a.order[a.N] = (int32_t)front;
}

// The policy loss of many rows in one launch: a workgroup of 16 waves takes
// the first kHeldChunks 16-byte chunks a thread of a row into its registers
// and reads them once, for the sum and for the gradient; the next row's are
// loaded into the registers that the gradient's stores free.  The rest of a
// row is read again from the cache.  On 4096 rows of 151936 bf16 logits (a
// tenth of them left out), 0.52 ms: 4.5 TB/s of the bytes it cannot do
// without, against 0.63 ms for the kernels above, which read all rows twice.
// Holding the whole row (18 chunks) took 0.54 to 0.59 ms, and so did summing a
// row's chunks between the stores of the row before it; two workgroups a CU
// with half the registers each took 0.64 ms or more.
//
// What is subtracted in the exponents is the maximum without the label of two
// rounds of chunks, the first and one further on (a vocabulary may have its
// first columns masked): S >= 1 as those chunks are in it.  A row whose S
// passes 2^20 (logits about as many octaves above them), or which is -inf
// there, is summed again by its own maximum: the coefficient over S has to stay
// a normal number for the gradient's other elements, and the exponential of
// many octaves has fewer digits.  (By its own maximum in the first place, a
// pass more over the registers, the rows above take 0.57 ms.)
// A bf16 gradient leaves the low part of k out, 2^-23 of the exponent at most.
template <typename T, typename G>
__global__ __launch_bounds__(kFusedThreads) void policy_fused_kernel(const RowArgs a) {
  using E = Elem<T>;
  constexpr int n16 = E::kPer16, kWaves = kFusedThreads / 64, kHeld = kHeldChunks;
  __shared__ float top_buf[kWaves];
  __shared__ double sum_buf[kWaves];
  __shared__ Stat pair_buf[kWaves];
  __shared__ RowGrad grad;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int full = (int)(a.V / n16), rest = (int)(a.V % n16);
  const int64_t count = a.order[a.N];  // rows that count
  u4 v[kHeld];
  float y_rest = -INFINITY, y_label = 0.0f;
  auto row_of = [&](int64_t n) { return static_cast<const T*>(a.Y) + n * a.y_stride; };
  // a uniform address and one small offset for all chunks: no address takes registers
  const uint32_t y_off = (uint32_t)tid * 16, dy_off = (uint32_t)(tid * n16 * sizeof(G));
  auto load = [&](const T* row, int c, int end) {
    v[c] = u4{E::kNegInf2, E::kNegInf2, E::kNegInf2, E::kNegInf2};
    if (tid < end - c * kFusedThreads)
      v[c] = __builtin_nontemporal_load(
          reinterpret_cast<const u4_any*>(reinterpret_cast<const char*>(row + c * kFusedThreads * n16) + y_off));
  };
  auto load_ends = [&](const T* row, int64_t n) {
    const int64_t label = a.labels[n];
    y_rest = tid < rest ? E::one(row[(int64_t)full * n16 + tid]) : -INFINITY;
    y_label = label >= 0 && label < a.V ? E::one(row[label]) : __builtin_nanf("");
  };
  int64_t place = blockIdx.x;
  if (place < count) {
    const int64_t n = a.order[place];
#pragma unroll
    for (int c = 0; c < kHeld; ++c) load(row_of(n), c, full);
    load_ends(row_of(n), n);
  }
  for (; place < count; place += gridDim.x) {
    const int64_t n = a.order[place];
    const T* row = row_of(n);
    G* out = static_cast<G*>(a.dY) + n * a.dy_stride;
    const bool more = place + gridDim.x < count;
    const int64_t next = more ? a.order[place + gridDim.x] : n;
    PolicyRow x = row_inputs<false>(a, n);
    x.y_label = y_label;
    // the label out of its chunk, or out of the row's last elements (its gradient is written for itself)
    const int label = __builtin_amdgcn_readfirstlane(a.labels[n]);
    const bool valid = label >= 0 && label < a.V;
    const int label_chunk = valid ? label / n16 : -1, label_at = label % n16;
    if (valid && label_chunk % kFusedThreads / 64 == wave) {
#pragma unroll
      for (int c = 0; c < kHeld; ++c)
        if (label_chunk / kFusedThreads == c && label_chunk % kFusedThreads == tid) v[c] = without<T>(v[c], label_at);
    }
    if (label_chunk == full && tid == label_at) y_rest = -INFINITY;
    float top = fmaxf(chunk_max<T>(v[0]), chunk_max<T>(v[kHeld / 2 - 1]));  // every row has these
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) top_buf[wave] = top;
    __syncthreads();
    top = top_buf[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, top_buf[w]);
    const float shift = shift_of(top);
    double S = tid < rest ? exp_at(y_rest - shift, a.k) : 0.0f;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
      S += (double)chunk_sum<T>(v[c], shift, a.k);
      // the gradient converts the chunk anew: kept, the converted logits
      // would take twice the registers that a row has
      asm volatile("" : "+v"(v[c]));
    }
    auto tail_chunk = [&](int64_t c) {
      const u4 y = u4(*reinterpret_cast<const u4_any*>(row + c * n16));
      return c == label_chunk ? without<T>(y, label_at) : y;
    };
    for (int64_t c = kHeld * kFusedThreads + tid; c < full; c += kFusedThreads)
      S += (double)chunk_sum<T>(tail_chunk(c), shift, a.k);
    for (int o = 32; o > 0; o >>= 1) S += __shfl_xor(S, o);
    if (lane == 0) sum_buf[wave] = S;
    __syncthreads();
    S = sum_buf[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) S += sum_buf[w];
    x.M = shift;
    x.S = S;
    if (!(S >= 0.5 && S <= 0x1p20)) {  // the same decision in every thread
      Stat st{0.0, y_rest};
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        st.M = fmaxf(st.M, chunk_max<T>(v[c]));
        asm volatile("" : "+v"(v[c]));
      }
      float shift = shift_of(st.M);
      st.S = exp_at(y_rest - shift, a.k);
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        st.S += (double)chunk_sum<T>(v[c], shift, a.k);
        asm volatile("" : "+v"(v[c]));
      }
      for (int64_t c = kHeld * kFusedThreads + tid; c < full; c += kFusedThreads) {
        const u4 y = tail_chunk(c);
        const float top = chunk_max<T>(y);
        if (top > st.M) {
          st.S *= (double)exp_at(st.M - top, a.k);
          st.M = shift = top;
        }
        st.S += (double)chunk_sum<T>(y, shift, a.k);
      }
      st = block_merge<kFusedThreads>(st, a.k, pair_buf);
      x.M = st.M;
      x.S = st.S;
    }
    if (wave == 0) {
      const PolicyResult r = policy_row(x, policy_scalars(a));
      if (lane == 0) {
        grad = r.grad;
        a.term[n] = r.term;
        write_row(a, n, r);
      }
    }
    __syncthreads();
    const RowGrad g = grad;
    auto put = [&](const u4& y, G* at_chunk) {
      float r[n16];
#pragma unroll
      for (int j = 0; j < n16; ++j) {
        const float d = E::at(y, j) - g.M;
        r[j] = g.neg * (sizeof(G) == 2 ? __builtin_amdgcn_exp2f(d * a.k.hi) : exp_at(d, a.k));
      }
      store_run<n16>(reinterpret_cast<G*>(reinterpret_cast<char*>(at_chunk) + dy_off), r);
    };
    const T* next_row = row_of(next);
    const int next_full = more ? full : 0;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
      if (tid < full - c * kFusedThreads) put(v[c], out + c * kFusedThreads * n16);
      load(next_row, c, next_full);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int64_t c = kHeld * kFusedThreads; c + tid < full; c += kFusedThreads)
      put(u4(*reinterpret_cast<const u4_any*>(row + (c + tid) * n16)), out + c * n16);
    if (tid < rest) out[(int64_t)full * n16 + tid] = Elem<G>::from(g.neg * exp_at(y_rest - g.M, a.k));
    // the label's element, by the thread that wrote it
    if (valid && tid == (label_chunk < full ? label_chunk % kFusedThreads : label_at)) out[label] = Elem<G>::from(g.label_g);
    if (more) load_ends(next_row, next);
  }
  // the rows that do not count
  for (; place < a.N; place += gridDim.x) {
    const int64_t n = a.order[place];
    G* out = static_cast<G*>(a.dY) + n * a.dy_stride;
    const float zero[n16] = {};
    for (int64_t c = tid; c < full; c += kFusedThreads) store_run<n16>(out + c * n16, zero);
    if (tid < rest) out[(int64_t)full * n16 + tid] = Elem<G>::from(0.0f);
    if (tid == 0) {
      a.term[n] = 0.0;
      if (a.logp) a.logp[n] = 0.0f;
      if (a.row_loss) a.row_loss[n] = 0.0f;
    }
  }
}

// ------------------------------------------------------------------- host ---

// Pieces a row is cut into: about 12288 workgroups in all (six rounds of the
// GPU's 2048 resident ones), none under 2048 columns.  With 4096 in all, 4096
// rows of a preference loss took 4% longer, with 16384 the 257 rows of an odd
// vocabulary 15%.
int64_t row_pieces(int64_t N, int64_t V) {
  const int64_t most = std::min<int64_t>(kMaxPieces, (V + kLeastWidth - 1) / kLeastWidth);
  return std::max<int64_t>(1, std::min<int64_t>(most, kTargetGroups / std::max<int64_t>(N, 1)));
}

// Whether small_loss_kernel takes a call: its one workgroup takes 5 us for 4
// rows of 1024 logits, where three launches take 11, and about as long as
// those for 64 such rows.
bool small_takes(int64_t N, int64_t V, int64_t B) {
  return N <= kSmallRows && N * V <= 65536 && B <= kSmallRows;
}

struct LossWorkspace {
  uint64_t part, ylab, grad, term, row_words, pair_loss, total;
};

LossWorkspace loss_workspace(int64_t N, int64_t V, int64_t B) {
  LossWorkspace w{};
  if (small_takes(N, V, B)) return w;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = w.total;
    w.total += round_up(bytes, ARCHEAD_ALIGNMENT);
    return at;
  };
  w.part = take((uint64_t)N * (uint64_t)row_pieces(N, V) * sizeof(Stat));
  w.ylab = take((uint64_t)N * 4);
  w.grad = take((uint64_t)N * sizeof(RowGrad));
  w.term = take((uint64_t)N * 8);
  w.row_words = take(N > 0 ? (uint64_t)(N + 1) * 4 : 0);  // the order of rows (policy) or their slopes (preference)
  w.pair_loss = take((uint64_t)B * 8);
  return w;
}

int check_shape(int64_t N, int64_t V) {
  if (N < 0 || V < 1) return ARCHEAD_E_SHAPE;
  if (N > (int64_t(1) << 22) || V > (int64_t(1) << 31) - 1) return ARCHEAD_E_UNSUPPORTED;
  return ARCHEAD_OK;
}

int elem_size(int32_t dtype) { return dtype == ARCHEAD_F32 ? 4 : dtype == ARCHEAD_BF16 ? 2 : 0; }

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

// A vector of n words; null or without words it meets nothing.
struct Words {
  const void* p;
  int64_t n;
};
bool meet(uint64_t a, uint64_t a_bytes, uint64_t b, uint64_t b_bytes) { return a < b + b_bytes && b < a + a_bytes; }
bool meet(Words x, const void* p, uint64_t bytes) {
  return x.p && p && x.n > 0 && bytes > 0 && meet((uint64_t)x.p, 4 * (uint64_t)x.n, (uint64_t)p, bytes);
}
// ... some row of a tensor
bool meet(Words x, const archead_tensor* t) {
  if (!t || !x.p || x.n <= 0 || t->rows <= 0) return false;
  const uint64_t size = elem_size(t->dtype), row = (uint64_t)t->cols * size, stride = (uint64_t)t->row_stride * size;
  const uint64_t first = (uint64_t)t->data, at = (uint64_t)x.p;
  const uint64_t i = at < first + row ? 0 : (at - first - row) / stride + 1;  // the first row that ends behind its start
  return i < (uint64_t)t->rows && meet(at, 4 * (uint64_t)x.n, first + i * stride, row);
}

// Kernels read the vectors while others write: no output may share bytes with
// another vector or the logits, and no vector with the gradient or the workspace.
int check_apart(const archead_tensor* Y, const archead_tensor* dY, std::initializer_list<Words> in,
                std::initializer_list<Words> out, const void* ws, uint64_t ws_bytes) {
  for (const Words* x = out.begin(); x != out.end(); ++x) {
    for (const Words& y : in)
      if (meet(*x, y.p, 4 * (uint64_t)y.n)) return ARCHEAD_E_SHAPE;
    for (const Words* y = out.begin(); y != x; ++y)
      if (meet(*x, y->p, 4 * (uint64_t)y->n)) return ARCHEAD_E_SHAPE;
    if (meet(*x, Y) || meet(*x, dY) || meet(*x, ws, ws_bytes)) return ARCHEAD_E_SHAPE;
  }
  for (const Words& x : in)
    if (meet(x, dY) || meet(x, ws, ws_bytes)) return ARCHEAD_E_SHAPE;
  return ARCHEAD_OK;
}

int check_workspace(const void* ws, uint64_t bytes, uint64_t need) {
  if (!ws) return ARCHEAD_E_NULL;
  if ((uintptr_t)ws % ARCHEAD_ALIGNMENT) return ARCHEAD_E_ALIGN;
  return bytes < need ? ARCHEAD_E_WORKSPACE : ARCHEAD_OK;
}

// The scale's two parts.  hi is s log2 e to nearest where that lies below it,
// else the number before that, so that lo is above zero as well; where s is at
// the end of fp32's range they stay in it.
Scale scale_of(float s) {
  constexpr float kLeast = std::numeric_limits<float>::denorm_min(), kMost = std::numeric_limits<float>::max();
  const double k = (double)s * 1.44269504088896340736;
  float hi = (float)std::min(k, (double)kMost);
  if ((double)hi >= k) hi = nextafterf(hi, 0.0f);
  return Scale{std::max(hi, kLeast), std::max((float)(k - (double)hi), kLeast)};
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
  // Where pieces abound, they end where a workgroup's round of loads does: a part of a
  // round takes as long as a whole one.  (480 rows of a preference loss on 151936 bf16
  // logits: 65 us, in 25 pieces a row 70; 4096 rows the same either way.)
  const int64_t round = kRowThreads * kRowUnroll * 16 / elem_size(Y->dtype);
  if (a.N * ((a.V + round - 1) / round) >= 2048) {
    a.width = (int64_t)round_up((uint64_t)a.width, (uint64_t)round);
    a.pieces = (int)((a.V + a.width - 1) / a.width);
  }
  a.s = s;
  a.k = scale_of(s);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part = reinterpret_cast<Stat*>(ws + W.part);
  a.ylab = reinterpret_cast<float*>(ws + W.ylab);
  a.grad = reinterpret_cast<RowGrad*>(ws + W.grad);
  a.term = reinterpret_cast<double*>(ws + W.term);
  a.order = reinterpret_cast<int32_t*>(ws + W.row_words);
  a.lanes = 1;
  while (a.lanes < a.pieces && a.lanes < 16) a.lanes *= 2;
  return a;
}

template <typename T>
hipError_t launch_gradient(const RowArgs& a, const archead_tensor* dY, hipStream_t s) {
  const dim3 grid((unsigned)(a.N * a.pieces + 1)), block(kRowThreads);
  if (!dY) {
    if (a.loss) hipLaunchKernelGGL(loss_total_kernel, dim3(1), block, 0, s, a);
  } else if (dY->dtype == ARCHEAD_BF16) {
    hipLaunchKernelGGL((row_gradient_kernel<T, uint16_t>), grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((row_gradient_kernel<T, float>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

// The fused kernel: a row for every CU, and rows that fill half of the chunks
// held.  Of bf16 rows in between one round of the CUs and eight it would leave
// part of them idle in the last round, and the split kernels' second read comes
// from the cache.  How full the last round is goes by the rows that count,
// which the host does not know; the rule is the one for 3/4 of them.
// (Microseconds of the fused and of the split kernels there, 151936 bf16
// logits: 256 rows 40 and 46, 320 45 and 52, 400 74 and 63, 512 82 and 76, 640
// 87 and 93, 768 115 and 103, 1024 123 and 129, 1280 160 and 165, 1536 198 and
// 198, 2048 237 and 269, 4096 460 and 567; 100003 fp32 logits: 256 rows 42 and
// 44, 320 50 and 50, 400 76 and 61, 512 82 and 77, 640 92 and 93, 768 120 and
// 108, 1024 133 and 144, 1536 213 and 228, 2048 266 and 314, 4096 514 and 665.
// So the rule is 5% off at 640, 1024 and 1280 bf16 rows, and 7 to 25% at 400 to
// 768 fp32 rows but 640.  All rows counting: 300 rows 69 and 57, 512 85 and 90,
// 1024 154 and 157; half of them: 512 55 and 62, 1024 105 and 112.)
bool fused_takes(const RowArgs& a, int64_t size) {
  if (size == 2 && a.N > kFusedLeastRows * 5 / 4 && a.N < kFusedLeastRows * 8) return false;
  return a.N >= kFusedLeastRows && a.V * size >= kHeldChunks / 2 * kFusedThreads * 16 && a.V < (int64_t(1) << 30);
}

template <typename T, bool kPairs>
hipError_t launch_loss(const RowArgs& a, const archead_tensor* dY, hipStream_t s) {
  (void)hipGetLastError();  // start from a clean error state
  const bool bf16 = dY && dY->dtype == ARCHEAD_BF16;
  if (small_takes(a.N, a.V, a.B)) {
    if (bf16)
      hipLaunchKernelGGL((small_loss_kernel<T, uint16_t, kPairs>), dim3(1), dim3(kSmallThreads), 0, s, a);
    else
      hipLaunchKernelGGL((small_loss_kernel<T, float, kPairs>), dim3(1), dim3(kSmallThreads), 0, s, a);
    return hipGetLastError();
  }
  if constexpr (!kPairs) {
    if (dY && a.N > 0 && a.N <= kFewRows) {
      RowArgs f = a;
      f.lanes = 64;
      const dim3 grid((unsigned)(a.N * a.pieces)), block(kRowThreads);
      hipLaunchKernelGGL((row_pieces_kernel<T, kPairs>), grid, block, 0, s, f);
      if (bf16)
        hipLaunchKernelGGL((few_gradient_kernel<T, uint16_t>), dim3(grid.x + 1), block, 0, s, f);
      else
        hipLaunchKernelGGL((few_gradient_kernel<T, float>), dim3(grid.x + 1), block, 0, s, f);
      return hipGetLastError();
    }
    if (dY && fused_takes(a, sizeof(T))) {
      int device = 0, cus = 0;
      if (hipGetDevice(&device) != hipSuccess ||
          hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess)
        return hipErrorUnknown;
      const dim3 grid((unsigned)std::min<int64_t>(a.N, cus)), block(kFusedThreads);
      hipLaunchKernelGGL(row_order_kernel, dim3(1), dim3(kOrderThreads), 0, s, a);
      if (dY->dtype == ARCHEAD_BF16)
        hipLaunchKernelGGL((policy_fused_kernel<T, uint16_t>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((policy_fused_kernel<T, float>), grid, block, 0, s, a);
      if (a.loss) hipLaunchKernelGGL(loss_total_kernel, dim3(1), dim3(kRowThreads), 0, s, a);
      return hipGetLastError();
    }
  }
  if (a.N > 0) {
    const int64_t rows = kRowThreads / a.lanes;
    hipLaunchKernelGGL((row_pieces_kernel<T, kPairs>), dim3((unsigned)(a.N * a.pieces)), dim3(kRowThreads), 0, s, a);
    hipLaunchKernelGGL(rows_kernel<kPairs>, dim3((unsigned)((a.N + rows - 1) / rows)), dim3(kRowThreads), 0, s, a);
  }
  if constexpr (kPairs) {
    if (a.B > 0) hipLaunchKernelGGL(pair_kernel, dim3((unsigned)a.B), dim3(kPairThreads), 0, s, a);
  }
  return launch_gradient<T>(a, dY, s);
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
  const int64_t N = Y->rows;
  const LossWorkspace W = loss_workspace(N, Y->cols, 0);
  if (int rc = check_apart(Y, out->dY,
                           {{in->labels, N}, {in->advantage, N}, {in->old_logp, N}, {in->ref_logp, N}, {in->weight, N}},
                           {{out->loss, 1}, {out->logp, N}, {out->row_loss, N}}, workspace, W.total))
    return rc;
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
  const int64_t N = Y->rows, B = in->n_pairs;
  const LossWorkspace W = loss_workspace(N, Y->cols, B);
  if (int rc = check_apart(
          Y, out->dY,
          {{in->labels, N}, {in->offsets, 2 * B + 1}, {in->ref_logp, N}, {in->weight, N}, {in->pair_weight, B}},
          {{out->loss, 1}, {out->logp, N}, {out->chosen_reward, B}, {out->rejected_reward, B}}, workspace, W.total))
    return rc;
  if (W.total > 0)
    if (int rc = check_workspace(workspace, workspace_bytes, W.total)) return rc;
  if (Y->rows == 0 && in->n_pairs == 0 && !out->loss) return ARCHEAD_OK;
  RowArgs a = row_args(Y, out->dY, in->inv_temperature, workspace, W);
  a.labels = in->labels;
  a.weight = in->weight;
  a.ref_logp = in->ref_logp;
  a.offsets = in->offsets;
  a.B = in->n_pairs;
  a.row_slope = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + W.row_words);
  a.pair_loss = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + W.pair_loss);
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
