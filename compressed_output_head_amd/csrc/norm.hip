// The norm in front of the head, and its gradient (archead_rmsnorm,
// archead_rmsnorm_backward).  With s = bf16(x + residual), the sum that the
// residual stream keeps, and inv = 1 / sqrt(sum_d s_d^2 / D + eps),
//   h_d = s_d inv w_d,
// in bf16, or in 8 bits with a scale for the row:
//   code_d = rint(127 t_d / m), scale = m inv / 127,  t = s w, m = max_d |t_d|.
// The factor inv cancels in the codes, and t is exact in fp32 (8 bits times 8
// bits).  The quotient rounded to fp32 decides as the exact one does: with
// t = T 2^a and m = M 2^b (T, M below 2^16) it misses a border (2k + 1) / 2,
// where it does not meet it, by 1 / (2^(b-a+1) M) at least, and a quotient of
// 1/2 or more has 2^(b-a) M <= 254 T: 1 / (508 T) > 2^-25, half a step of fp32
// there (both grow alike from 1/2 up).
//
// One pass: a row is read once, held in registers from the sums to the
// outputs (a row whose t leaves fp32 again for h).  Bound by HBM where rows are
// many, by the launch where they are few: 16384 rows of 4096 with a residual, sum
// and codes 81 us, 5.8 TB/s of what is read and written (rows that start at odd
// elements or leave threads idle 4.6 to 5.0), to bf16 with the factor 95 us, 5.6
// TB/s, without a residual 50, 5.3; their gradient 108 us, 5.0 TB/s; one row 3.1
// us.
#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace archead {

namespace {

constexpr int64_t kNormMaxRows = int64_t(1) << 22;
constexpr int64_t kNormMaxCols = 32768;

typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(1)));

struct NormArgs {
  int64_t N, D;
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* residual;  // or null
  int64_t r_stride;
  const uint16_t* weight;    // or null
  float eps;
  uint16_t* sum;             // outputs, each or null
  int64_t sum_stride;
  uint16_t* h;
  int64_t h_stride;
  int8_t* codes;
  int64_t c_stride;
  float* scale;
  float* inv_rms;
};

struct NormBwdArgs {
  int64_t N, D;
  const uint16_t* dh;
  int64_t dh_stride;
  const uint16_t* sum;
  int64_t sum_stride;
  const float* inv_rms;
  const uint16_t* weight;  // or null
  const uint16_t* dsum;    // or null
  int64_t ds_stride;
  uint16_t* dx;            // or null
  int64_t dx_stride;
  float* part;             // [parts][D], or null
  float* dweight;
  int parts;
};

// Elements v .. v + 8 of a row that starts at any element, zeros from `end` on.
__device__ __forceinline__ u4 load8(const uint16_t* row, int64_t v, int64_t end) {
  u4 x = {};
  if (v + 8 <= end) {
    x = *reinterpret_cast<const u4_any*>(row + v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (v + j < end) x[j >> 1] |= (uint32_t)row[v + j] << (16 * (j & 1));
  }
  return x;
}
__device__ __forceinline__ void store8(uint16_t* row, int64_t v, int64_t end, u4 x) {
  if (v + 8 <= end) {
    *reinterpret_cast<u4_any*>(row + v) = x;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (v + j < end) row[v + j] = (uint16_t)(x[j >> 1] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ float at(const u4& x, int j) {
  return __uint_as_float(j & 1 ? x[j >> 1] & 0xffff0000u : x[j >> 1] << 16);
}
__device__ __forceinline__ u4 pack8(const float (&y)[8]) {
  const u2 lo = pack_bf16x4(y[0], y[1], y[2], y[3]), hi = pack_bf16x4(y[4], y[5], y[6], y[7]);
  return u4{lo[0], lo[1], hi[0], hi[1]};
}
// x + r, rounded to bf16
__device__ __forceinline__ u4 add8(u4 x, u4 r) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = at(x, j) + at(r, j);
  return pack8(y);
}
constexpr uint32_t kOnes = 0x3f803f80u;  // two bf16 ones

// Sum (in a fixed order) and largest of a row's threads, given to all of them.
template <int T>
__device__ __forceinline__ void row_reduce(double& sum, uint32_t& top) {
#pragma unroll
  for (int o = std::min(T, 64) / 2; o > 0; o >>= 1) {
    sum += __shfl_xor(sum, o);
    top = std::max(top, (uint32_t)__shfl_xor((int)top, o));
  }
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    __shared__ double sSum[W];
    __shared__ uint32_t sTop[W];
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      sSum[wave] = sum;
      sTop[wave] = top;
    }
    __syncthreads();
    sum = sSum[0];
    top = sTop[0];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      sum += sSum[w];
      top = std::max(top, sTop[w]);
    }
  }
}

constexpr int norm_threads(int T) { return T < 256 ? 256 : T; }

// T threads a row, K octets of columns each; kH: h is wanted.  (Calls for codes
// alone in a kernel of their own: beside h they take 4% longer, 4096 rows of 8192.)
template <int T, int K, bool kH>
__global__ __launch_bounds__(norm_threads(T)) void rmsnorm_kernel(const NormArgs a) {
  constexpr int kRows = norm_threads(T) / T;
  const int t0 = threadIdx.x % T;
  const int64_t n = (int64_t)blockIdx.x * kRows + threadIdx.x / T;
  if (n >= a.N) return;  // all threads of a row, and of T > 64 whole workgroups
  u4 s[K], w[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t v = 8 * (int64_t)(t0 + T * k);
    s[k] = load8(a.x + n * a.x_stride, v, a.D);
    w[k] = a.weight ? load8(a.weight, v, a.D) : u4{kOnes, kOnes, kOnes, kOnes};
  }
  if (a.residual) {
    u4 r[K];
#pragma unroll
    for (int k = 0; k < K; ++k) r[k] = load8(a.residual + n * a.r_stride, 8 * (int64_t)(t0 + T * k), a.D);
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = add8(s[k], r[k]);
  }
  if (a.sum) {
#pragma unroll
    for (int k = 0; k < K; ++k) store8(a.sum + n * a.sum_stride, 8 * (int64_t)(t0 + T * k), a.D, s[k]);
  }
  // squares and their sum in fp64: neither overflows for any bf16 row.  The
  // largest by its bits, which puts a NaN above everything.
  double sum = 0.0;
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double y = (double)at(s[k], j);
      sum = fma(y, y, sum);
      top = std::max(top, __float_as_uint(at(s[k], j) * at(w[k], j)) & 0x7fffffffu);
    }
  row_reduce<T>(sum, top);
  const double inv = 1.0 / sqrt(sum / (double)a.D + (double)a.eps);
  const float m = __uint_as_float(top), inv32 = (float)inv;
  const bool finite = top < 0x7f800000u && sum < (double)__builtin_huge_valf();
  if (t0 == 0) {
    if (a.inv_rms) a.inv_rms[n] = inv32;
    if (a.scale) a.scale[n] = finite ? (float)((double)m * inv / 127.0) : __builtin_nanf("");
  }
  if (a.codes) {
    const double step = finite && m > 0.0f ? 127.0 / (double)m : 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t v = 8 * (int64_t)(t0 + T * k);
      u2 c = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // 1.5 2^23 + q rounds q to a whole number, half to even, in the sum's low bits
        const float q = (float)((double)(at(s[k], j) * at(w[k], j)) * step);
        c[j >> 2] |= (__float_as_uint(q + 12582912.0f) & 0xffu) << (8 * (j & 3));
      }
      if (!finite) c = u2{};
      int8_t* row = a.codes + n * a.c_stride;
      if (v + 8 <= a.D) {
        *reinterpret_cast<u2_any*>(row + v) = c;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v + j < a.D) row[v + j] = (int8_t)(c[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
  if constexpr (!kH) return;
  if (top < 0x7f800000u && inv <= 32768.0) {
    // (a product below 2^-126 is off by 2^-150, and h by 2^-135: nothing)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = at(s[k], j) * at(w[k], j) * inv32;
      store8(a.h + n * a.h_stride, 8 * (int64_t)(t0 + T * k), a.D, pack8(y));
    }
  } else {
    // s w leaves fp32 where h may not: (s 2^e w) (inv 2^-e), the factor in [1, 2),
    // leaves it where h does.  (s 2^e is exact: where it is subnormal s is 2^-126
    // of the row's mean.)  The row is read again, from the sum where that may
    // stand in the place of x or the residual by now, so that rows as above need
    // not hold s and w beside their products.  inv is 0 or NaN of a row that is
    // not finite.
    int e = 0;
    float power = inv32, factor = 1.0f;
    if (inv > 0.0) {
      factor = (float)(2.0 * frexp(inv, &e));
      power = ldexpf(1.0f, e - 1);
    }
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
      const int64_t v = 8 * (int64_t)(t0 + T * k);
      u4 x = a.sum ? load8(a.sum + n * a.sum_stride, v, a.D) : load8(a.x + n * a.x_stride, v, a.D);
      if (a.residual && !a.sum) x = add8(x, load8(a.residual + n * a.r_stride, v, a.D));
      const u4 g = a.weight ? load8(a.weight, v, a.D) : u4{kOnes, kOnes, kOnes, kOnes};
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = at(x, j) * power * at(g, j) * factor;
      store8(a.h + n * a.h_stride, v, a.D, pack8(y));
    }
  }
}

// An octet of a row's operands of the gradient.
struct GradOctet {
  u4 s, d, e;
  __device__ __forceinline__ void load(const NormBwdArgs& a, int64_t n, int64_t v) {
    s = load8(a.sum + n * a.sum_stride, v, a.D);
    d = load8(a.dh + n * a.dh_stride, v, a.D);
    e = a.dsum ? load8(a.dsum + n * a.ds_stride, v, a.D) : u4{};
  }
  // sum of g s inv: s inv is at most sqrt(D), where s may be at the end of fp32
  __device__ __forceinline__ float dot(const u4& w, float inv) const {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(at(d, j) * at(w, j), at(s, j) * inv, sum);
    return sum;
  }
  // dx, with c the row's mean of g s inv, and what the octet adds to dweight
  __device__ __forceinline__ u4 apply(const u4& w, float inv, float c, float (&dw)[8]) const {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float unit = at(s, j) * inv;
      y[j] = fmaf(inv, at(d, j) * at(w, j) - unit * c, at(e, j));
      dw[j] = fmaf(at(d, j), unit, dw[j]);
    }
    return pack8(y);
  }
};

// dx = dsum + inv (g - u sum_d(g u) / D), g = w dh, u = s inv, and part p of
// dweight = sum_n dh u: row slot p takes the rows p, p + parts, ..., its
// threads the same columns of all of them.  The next row is on its way while
// one is worked on; rows too long for that (K > 2) are read again for dx, from
// the cache, and their threads hold the sums of dweight in LDS.
template <int T, int K>
__global__ __launch_bounds__(norm_threads(T)) void rmsnorm_backward_kernel(const NormBwdArgs a) {
  constexpr int kSlots = norm_threads(T) / T;
  constexpr bool kHeld = K <= 2;
  const int t0 = threadIdx.x % T;
  const int p = (int)blockIdx.x * kSlots + threadIdx.x / T;
  if (p >= a.parts) return;
  auto column = [&](int k) { return 8 * (int64_t)(t0 + T * k); };
  auto weight = [&](int k) { return a.weight ? load8(a.weight, column(k), a.D) : u4{kOnes, kOnes, kOnes, kOnes}; };
  auto finish = [&](double dot) {
    uint32_t none = 0;
    if constexpr (T > 64) __syncthreads();  // the row before is done with the reduction's memory
    row_reduce<T>(dot, none);
    return (float)(dot / (double)a.D);
  };
  if constexpr (kHeld) {
    u4 w[K];
    float dw[K][8] = {};
    GradOctet next[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k] = weight(k);
      next[k].load(a, p, column(k));
    }
    float next_inv = a.inv_rms[p];
    for (int64_t n = p; n < a.N; n += a.parts) {
      GradOctet row[K];
      const float inv = next_inv;
#pragma unroll
      for (int k = 0; k < K; ++k) row[k] = next[k];
      if (n + a.parts < a.N) {
#pragma unroll
        for (int k = 0; k < K; ++k) next[k].load(a, n + a.parts, column(k));
        next_inv = a.inv_rms[n + a.parts];
      }
      double dot = 0.0;
#pragma unroll
      for (int k = 0; k < K; ++k) dot += (double)row[k].dot(w[k], inv);
      const float c = finish(dot);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        // new values to the compiler: it would keep the products and the
        // unpacked elements of the sum above, three times the registers
        asm("" : "+v"(row[k].s), "+v"(row[k].d), "+v"(w[k]));
        const u4 y = row[k].apply(w[k], inv, c, dw[k]);
        if (a.dx) store8(a.dx + n * a.dx_stride, column(k), a.D, y);
      }
    }
    if (!a.part) return;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (column(k) + j < a.D) a.part[p * a.D + column(k) + j] = dw[k][j];
  } else {
    extern __shared__ f4 sDw[];  // [2 K][T], each thread's own
    f4* mine = sDw + t0;
    for (int i = 0; i < 2 * K; ++i) mine[i * T] = f4{};
    for (int64_t n = p; n < a.N; n += a.parts) {
      const float inv = a.inv_rms[n];
      double dot = 0.0;
#pragma unroll 2
      for (int k = 0; k < K; ++k) {
        GradOctet x;
        x.load(a, n, column(k));
        dot += (double)x.dot(weight(k), inv);
      }
      const float c = finish(dot);
#pragma unroll 1
      for (int k = 0; k < K; ++k) {
        GradOctet x;
        x.load(a, n, column(k));
        float dw[8];
        *reinterpret_cast<f4*>(dw) = mine[2 * k * T];
        *reinterpret_cast<f4*>(dw + 4) = mine[(2 * k + 1) * T];
        const u4 y = x.apply(weight(k), inv, c, dw);
        mine[2 * k * T] = *reinterpret_cast<f4*>(dw);
        mine[(2 * k + 1) * T] = *reinterpret_cast<f4*>(dw + 4);
        if (a.dx) store8(a.dx + n * a.dx_stride, column(k), a.D, y);
      }
    }
    if (!a.part) return;
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (column(k) + j < a.D) a.part[p * a.D + column(k) + j] = mine[(2 * k + j / 4) * T][j % 4];
  }
}

// kSumCols columns of dweight: kDeal threads a column add its parts, in fp64.
constexpr int kSumCols = 16, kDeal = 64;
__global__ __launch_bounds__(kSumCols * kDeal) void rmsnorm_dweight_kernel(const NormBwdArgs a) {
  __shared__ double buf[kDeal][kSumCols];
  const int c = threadIdx.x % kSumCols, deal = threadIdx.x / kSumCols;
  const int64_t v = kSumCols * (int64_t)blockIdx.x + c;
  double sum = 0.0;
  if (v < a.D)
#pragma unroll 4
    for (int p = deal; p < a.parts; p += kDeal) sum += (double)a.part[p * a.D + v];
  buf[deal][c] = sum;
  __syncthreads();
  if (deal == 0 && v < a.D) {
#pragma unroll
    for (int i = 1; i < kDeal; ++i) sum += buf[i][c];
    a.dweight[v] = (float)sum;
  }
}

// ------------------------------------------------------------------- host ---

// Threads of a row, and octets of columns that each takes.
template <int T_, int K_>
struct Width {
  static constexpr int T = T_, K = K_;
};
template <class F>
auto norm_width(int64_t D, F&& f) {
  return D <= 128    ? f(Width<16, 1>{})
         : D <= 256  ? f(Width<32, 1>{})
         : D <= 512  ? f(Width<64, 1>{})
         : D <= 1024 ? f(Width<64, 2>{})
         : D <= 2048 ? f(Width<64, 4>{})
         : D <= 4096 ? f(Width<256, 2>{})
         : D <= 8192 ? f(Width<256, 4>{})
         : D <= 16384 ? f(Width<256, 8>{})
                      : f(Width<1024, 4>{});
}
// The gradient holds the sums of dweight too, and a second row: two octets at
// most, where the norm has up to eight.  (8192 rows of 8192: 105 us with 1024
// threads of one octet, 114 with 512 of two.)
template <class F>
auto backward_width(int64_t D, F&& f) {
  return D <= 128    ? f(Width<16, 1>{})
         : D <= 256  ? f(Width<32, 1>{})
         : D <= 512  ? f(Width<64, 1>{})
         : D <= 1024 ? f(Width<64, 2>{})
         : D <= 2048 ? f(Width<256, 1>{})
         : D <= 4096 ? f(Width<512, 1>{})
         : D <= 8192 ? f(Width<1024, 1>{})
         : D <= 16384 ? f(Width<1024, 2>{})
                      : f(Width<1024, 4>{});
}

// Rows that are worked on at the same time: parts of dweight.  More of them
// hide more latency, and are more to write and to add up: with 2^17 and 2^18
// threads in all, 131072 rows of 512 take 99 and 113 us, 32768 of 2048 101 and
// 108, 8192 of 8192 165 and 105, 2048 of 32768 206 and 156.
int norm_parts(int64_t N, int64_t D) {
  const int64_t threads = backward_width(D, [](auto w) { return (int64_t)decltype(w)::T; });
  return (int)std::min(N, (int64_t(1) << (D <= 2048 ? 17 : 18)) / threads);
}

// A bf16 (or int8) tensor of N rows and D columns.
int check_rows(const archead_tensor* t, int64_t N, int64_t D, int dtype) {
  if (t->dtype != dtype) return ARCHEAD_E_DTYPE;
  if (t->rows != N || t->cols != D || t->row_stride < D) return ARCHEAD_E_SHAPE;
  return ARCHEAD_OK;
}
int size_of(const archead_tensor* t) { return t->dtype == ARCHEAD_I8 ? 1 : 2; }
bool misaligned(const archead_tensor* t) { return t && (uintptr_t)t->data % size_of(t) != 0; }
// The rows of `in` that `out` replaces as they are.
bool same_rows(const archead_tensor* in, const archead_tensor* out) {
  return in->data == out->data && in->row_stride == out->row_stride && in->dtype == out->dtype;
}
// A vector's bytes, as one row.
archead_tensor bytes_of(const void* p, int64_t n) { return archead_tensor{const_cast<void*>(p), 1, n, n, ARCHEAD_I8}; }
bool meets(const archead_tensor* x, const archead_tensor* y) {
  if (x->rows == 0 || y->rows == 0) return false;
  if (x->rows == y->rows) return overlap(x, size_of(x), y, size_of(y));
  // a vector and a tensor: by their spans
  const uint64_t a = (uint64_t)x->data, b = (uint64_t)y->data;
  return a < b + ((uint64_t)(y->rows - 1) * y->row_stride + y->cols) * size_of(y) &&
         b < a + ((uint64_t)(x->rows - 1) * x->row_stride + x->cols) * size_of(x);
}

}  // namespace
}  // namespace archead

using namespace archead;

extern "C" {

int archead_rmsnorm(const archead_rmsnorm_inputs* in, const archead_rmsnorm_outputs* out, void* stream) {
  if (!in || !out || !in->x) return ARCHEAD_E_NULL;
  const archead_tensor* x = in->x;
  const int64_t N = x->rows, D = x->cols;
  if (N < 0 || D < 1) return ARCHEAD_E_SHAPE;
  if (int rc = check_rows(x, N, D, ARCHEAD_BF16)) return rc;
  if (in->residual)
    if (int rc = check_rows(in->residual, N, D, ARCHEAD_BF16)) return rc;
  const archead_tensor* outs[] = {out->sum, out->h, out->codes};
  for (const archead_tensor* t : outs)
    if (t)
      if (int rc = check_rows(t, N, D, t == out->codes ? ARCHEAD_I8 : ARCHEAD_BF16)) return rc;
  if (!(in->eps > 0.0f) || !(in->eps < __builtin_huge_valf())) return ARCHEAD_E_VALUE;
  if (N > kNormMaxRows || D > kNormMaxCols) return ARCHEAD_E_UNSUPPORTED;
  if (N == 0) return ARCHEAD_OK;
  if ((out->codes != nullptr) != (out->scale != nullptr)) return ARCHEAD_E_NULL;
  if (!x->data || (in->residual && !in->residual->data)) return ARCHEAD_E_NULL;
  for (const archead_tensor* t : outs)
    if (t && !t->data) return ARCHEAD_E_NULL;
  if (misaligned(x) || misaligned(in->residual) || misaligned(out->sum) || misaligned(out->h)) return ARCHEAD_E_ALIGN;
  if ((uintptr_t)in->weight % 2 || (uintptr_t)out->scale % 4 || (uintptr_t)out->inv_rms % 4) return ARCHEAD_E_ALIGN;
  // outputs meet no input, but that a row may be replaced by the sum or h of itself, and no other output
  const archead_tensor weight = bytes_of(in->weight, 2 * D), scale = bytes_of(out->scale, 4 * N),
                       inv = bytes_of(out->inv_rms, 4 * N);
  const archead_tensor* all_out[] = {out->sum, out->h, out->codes, out->scale ? &scale : nullptr,
                                     out->inv_rms ? &inv : nullptr};
  const archead_tensor* all_in[] = {x, in->residual, in->weight ? &weight : nullptr};
  for (int i = 0; i < 5; ++i) {
    if (!all_out[i]) continue;
    for (const archead_tensor* t : all_in)
      if (t && !(i < 2 && same_rows(t, all_out[i])) && meets(t, all_out[i])) return ARCHEAD_E_SHAPE;
    for (int j = 0; j < i; ++j)
      if (all_out[j] && meets(all_out[i], all_out[j])) return ARCHEAD_E_SHAPE;
  }
  if (!out->sum && !out->h && !out->codes && !out->inv_rms) return ARCHEAD_OK;
  NormArgs a{};
  a.N = N;
  a.D = D;
  a.x = static_cast<const uint16_t*>(x->data);
  a.x_stride = x->row_stride;
  if (in->residual) {
    a.residual = static_cast<const uint16_t*>(in->residual->data);
    a.r_stride = in->residual->row_stride;
  }
  a.weight = static_cast<const uint16_t*>(in->weight);
  a.eps = in->eps;
  if (out->sum) {
    a.sum = static_cast<uint16_t*>(out->sum->data);
    a.sum_stride = out->sum->row_stride;
  }
  if (out->h) {
    a.h = static_cast<uint16_t*>(out->h->data);
    a.h_stride = out->h->row_stride;
  }
  if (out->codes) {
    a.codes = static_cast<int8_t*>(out->codes->data);
    a.c_stride = out->codes->row_stride;
  }
  a.scale = out->scale;
  a.inv_rms = out->inv_rms;
  (void)hipGetLastError();  // start from a clean error state
  norm_width(D, [&](auto w) {
    constexpr int T = decltype(w)::T, K = decltype(w)::K, kRows = norm_threads(T) / T;
    const dim3 grid((unsigned)((N + kRows - 1) / kRows)), block(norm_threads(T));
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.h)
      hipLaunchKernelGGL((rmsnorm_kernel<T, K, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((rmsnorm_kernel<T, K, false>), grid, block, 0, s, a);
  });
  return hipGetLastError() == hipSuccess ? ARCHEAD_OK : ARCHEAD_E_HIP;
}

int archead_rmsnorm_backward_workspace_bytes(int64_t n_rows, int64_t D, uint64_t* bytes) {
  if (!bytes) return ARCHEAD_E_NULL;
  if (n_rows < 0 || D < 1) return ARCHEAD_E_SHAPE;
  if (n_rows > kNormMaxRows || D > kNormMaxCols) return ARCHEAD_E_UNSUPPORTED;
  *bytes = round_up((uint64_t)norm_parts(n_rows, D) * (uint64_t)D * 4, ARCHEAD_ALIGNMENT);
  return ARCHEAD_OK;
}

int archead_rmsnorm_backward(const archead_rmsnorm_grad_inputs* in, const archead_rmsnorm_grad_outputs* out,
                             void* workspace, uint64_t workspace_bytes, void* stream) {
  if (!in || !out || !in->dh || !in->sum) return ARCHEAD_E_NULL;
  const int64_t N = in->dh->rows, D = in->dh->cols;
  if (N < 0 || D < 1) return ARCHEAD_E_SHAPE;
  for (const archead_tensor* t : {in->dh, in->sum, in->dsum, out->dx})
    if (t)
      if (int rc = check_rows(t, N, D, ARCHEAD_BF16)) return rc;
  if (N > kNormMaxRows || D > kNormMaxCols) return ARCHEAD_E_UNSUPPORTED;
  if (!out->dx && !out->dweight) return ARCHEAD_OK;
  for (const archead_tensor* t : {in->dh, in->sum, in->dsum, out->dx})
    if (t && N > 0 && !t->data) return ARCHEAD_E_NULL;
  if (N > 0 && !in->inv_rms) return ARCHEAD_E_NULL;
  for (const archead_tensor* t : {in->dh, in->sum, in->dsum, out->dx})
    if (misaligned(t)) return ARCHEAD_E_ALIGN;
  if ((uintptr_t)in->weight % 2 || (uintptr_t)in->inv_rms % 4 || (uintptr_t)out->dweight % 4) return ARCHEAD_E_ALIGN;
  const uint64_t need = out->dweight ? round_up((uint64_t)norm_parts(N, D) * (uint64_t)D * 4, ARCHEAD_ALIGNMENT) : 0;
  if (need && !workspace) return ARCHEAD_E_NULL;
  if (need && (uintptr_t)workspace % ARCHEAD_ALIGNMENT) return ARCHEAD_E_ALIGN;
  if (workspace_bytes < need) return ARCHEAD_E_WORKSPACE;
  const archead_tensor weight = bytes_of(in->weight, 2 * D), inv = bytes_of(in->inv_rms, 4 * N),
                       dw = bytes_of(out->dweight, 4 * D), ws = bytes_of(workspace, (int64_t)need);
  const archead_tensor* all_out[] = {out->dx, out->dweight ? &dw : nullptr, need ? &ws : nullptr};
  const archead_tensor* all_in[] = {in->dh, in->dsum, in->sum, in->weight ? &weight : nullptr, N > 0 ? &inv : nullptr};
  for (int i = 0; i < 3; ++i) {
    if (!all_out[i]) continue;
    for (int j = 0; j < 5; ++j)
      if (all_in[j] && !(i == 0 && j < 3 && same_rows(all_in[j], all_out[i])) && meets(all_in[j], all_out[i]))
        return ARCHEAD_E_SHAPE;
    for (int j = 0; j < i; ++j)
      if (all_out[j] && meets(all_out[i], all_out[j])) return ARCHEAD_E_SHAPE;
  }
  NormBwdArgs a{};
  a.N = N;
  a.D = D;
  a.dh = static_cast<const uint16_t*>(in->dh->data);
  a.dh_stride = in->dh->row_stride;
  a.sum = static_cast<const uint16_t*>(in->sum->data);
  a.sum_stride = in->sum->row_stride;
  a.inv_rms = in->inv_rms;
  a.weight = static_cast<const uint16_t*>(in->weight);
  if (in->dsum) {
    a.dsum = static_cast<const uint16_t*>(in->dsum->data);
    a.ds_stride = in->dsum->row_stride;
  }
  if (out->dx) {
    a.dx = static_cast<uint16_t*>(out->dx->data);
    a.dx_stride = out->dx->row_stride;
  }
  a.part = out->dweight ? static_cast<float*>(workspace) : nullptr;
  a.dweight = out->dweight;
  a.parts = norm_parts(N, D);
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // start from a clean error state
  if (N > 0)
    backward_width(D, [&](auto w) {
      constexpr int T = decltype(w)::T, K = decltype(w)::K, kSlots = norm_threads(T) / T;
      constexpr size_t lds = K > 2 ? (size_t)32 * K * T : 0;
      const auto kernel = rmsnorm_backward_kernel<T, K>;
      if (lds > 64 * 1024)  // more is opted into per kernel
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      hipLaunchKernelGGL(kernel, dim3((unsigned)((a.parts + kSlots - 1) / kSlots)), dim3(norm_threads(T)), lds, s, a);
    });
  // no rows: a gradient of zeros
  if (out->dweight) hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((unsigned)((D + kSumCols - 1) / kSumCols)), dim3(kSumCols * kDeal), 0, s, a);
  return hipGetLastError() == hipSuccess ? ARCHEAD_OK : ARCHEAD_E_HIP;
}

}  // extern "C"
