// Cross entropy of labels through the packed head with the hidden states'
// gradient, without the logits of more than a piece (archead_cross_entropy).
// With z = tau y and the label l apart from the others,
//   m = max_{v != l} z_v,  e_v = exp(z_v - m),  S = sum_{v != l} e_v,
//   d = m + ln S - z_l,  log p = -ln(1 + exp d),  q = 1 - p = 1 / (1 + exp -d),
//   dH = w tau q ((sum_{v != l} e_v W_v) / S - W_l):
// a mean of the other rows of W_hat less the label's row, times what is left
// of the probability.  Nothing cancels in a row that is sure of its label, and
// the sum can be taken piece by piece of the vocabulary under a running
// maximum, whose exponentials are then multiplied with the head in place of a
// gradient of logits.
//
// Few rows (up to 32 at a time): the decode kernels' logits in fp32, then
//   xent_pieces_kernel      maxima and sums of pieces of a row's logits
//   xent_operand_kernel     e s_R, e s_Ac, e s_Aw as fp16 operands; log p
//   bwd_few_kernel, bwd_few16_kernel (backward.hip)
//   xent_finish_few_kernel  the splits' sums, Z B and the label's row to dH
#include <algorithm>

#include "backward_main.h"
#include "device_common.h"
#include "internal.h"

namespace archead {

namespace {

constexpr int64_t kXentMaxRows = int64_t(1) << 22;
constexpr int64_t kXentMaxVocab = int64_t(1) << 24;
constexpr int kPieceThreads = 256;
constexpr int64_t kPieceCols = 8 * kPieceThreads;
constexpr int kMaxPieces = 128;
constexpr int kFinishThreads = 256;

// What a row's pieces leave, relative to the piece's maximum.
struct Piece {
  float m, s, top[3];  // maximum of y; sum of exponentials; largest e s_R, e s_Ac, e s_Aw
};

// What the last kernel needs of a row.
struct RowOut {
  float mean, label;  // factors of the others' sum and of the label's row: w tau q / S, w tau q
};

struct XentArgs {
  BwdArgs b;  // the head, the product's operands and sums; N rows from row n0 of the call
  const float* Y;
  int64_t y_stride;
  const int32_t* labels;
  const float* weight;
  float tau, c_hi, c_lo;  // log2(e) tau = c_hi + c_lo
  float* logp;            // or null
  uint16_t* dH;           // or null
  int64_t dh_stride;
  Piece* piece;           // [N][pieces]
  RowOut* row;            // [N]
  double* terms;          // [N] -w log p
  int pieces;
  int64_t width;          // columns of a piece
};

__device__ __forceinline__ bool counts(const XentArgs& a, int64_t n) { return !a.weight || a.weight[n] != 0.0f; }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// exp(z - m) of a logit: differences before the scale, so that nothing overflows
__device__ __forceinline__ float exp_of(const XentArgs& a, float y, float m) {
  const float d = y - m;
  return __builtin_amdgcn_exp2f(fmaf(d, a.c_hi, d * a.c_lo));
}

// The scales of vocabulary row v: s_R, and s_Ac, s_Aw of the parts that there are.
__device__ __forceinline__ void scales_of(const BwdArgs& b, int64_t v, float (&s)[3]) {
  s[0] = f16_to_f32(b.r_rowscale[v]);
  s[1] = b.r_c ? f16_to_f32(b.a_scales[v * b.nA]) : 0.0f;
  s[2] = b.r_r ? f16_to_f32(b.a_scales[v * b.nA + b.nA - 1]) : 0.0f;
}

// Workgroup n pieces + p: piece p of row n.  The workgroups behind those lay
// the group codes out for the product.
__global__ __launch_bounds__(kPieceThreads) void xent_pieces_kernel(const XentArgs a) {
  constexpr int kWaves = kPieceThreads / 64;
  __shared__ float buf[kWaves][4];
  const int64_t items = a.b.N * a.pieces;
  if ((int64_t)blockIdx.x >= items) {
    arrange_groups(a.b, ((int64_t)blockIdx.x - items) * kPieceThreads + threadIdx.x);
    return;
  }
  const int64_t n = blockIdx.x / a.pieces;
  const int p = (int)(blockIdx.x % a.pieces);
  if (!counts(a, n)) return;
  const int64_t v0 = p * a.width, v1 = std::min(v0 + a.width, a.b.V), label = a.labels[n];
  const float* y = a.Y + n * a.y_stride;
  const float infinity = __builtin_huge_valf();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  // logits v .. v + 4, the label and what is past the piece at -inf (rows are 16-byte aligned)
  auto load4 = [&](int64_t v) {
    f4 x = v < v1 ? *reinterpret_cast<const f4*>(y + v) : f4{-infinity, -infinity, -infinity, -infinity};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v + j == label || v + j >= v1) x[j] = -infinity;
    return x;
  };
  float m = -infinity;
  for (int64_t v = v0 + 4 * threadIdx.x; v < v1; v += 4 * kPieceThreads) {
    const f4 x = load4(v);
    m = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
  }
  m = wave_max(m);
  if (lane == 0) buf[wave][0] = m;
  __syncthreads();
  m = fmaxf(fmaxf(buf[0][0], buf[1][0]), fmaxf(buf[2][0], buf[3][0]));
  __syncthreads();
  float sum = 0.0f, top[3] = {};
  for (int64_t v = v0 + 4 * threadIdx.x; v < v1; v += 4 * kPieceThreads) {
    const f4 x = load4(v);
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (v + j >= v1 || v + j == label) continue;
      const float e = exp_of(a, x[j], m);
      float s[3];
      scales_of(a.b, v + j, s);
      part += e;
#pragma unroll
      for (int q = 0; q < 3; ++q) top[q] = fmaxf(top[q], e * fabsf(s[q]));
    }
    sum += part;
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int q = 0; q < 3; ++q) top[q] = wave_max(top[q]);
  if (lane == 0) {
    buf[wave][0] = sum;
#pragma unroll
    for (int q = 0; q < 3; ++q) buf[wave][1 + q] = top[q];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Piece out{m, buf[0][0], {buf[0][1], buf[0][2], buf[0][3]}};
    for (int w = 1; w < kWaves; ++w) {
      out.s += buf[w][0];
      for (int q = 0; q < 3; ++q) out.top[q] = fmaxf(out.top[q], buf[w][1 + q]);
    }
    a.piece[n * a.pieces + p] = out;
  }
}

// Run blockIdx.x of 128 columns of all rows as operands, thread t octet t % 16
// of rows t / 16 and t / 16 + 16; the rows' pieces are merged by every
// workgroup, and the first one writes what is known of the rows then.
constexpr int kOperandThreads = 256;
__global__ __launch_bounds__(kOperandThreads) void xent_operand_kernel(const XentArgs a) {
  __shared__ float sM[32], sP[3][32];
  const int tid = threadIdx.x, N = (int)a.b.N;
  const float infinity = __builtin_huge_valf();
  {  // eight lanes a row
    const int n = tid >> 3, lane = tid & 7;
    const bool on = n < N && counts(a, n);
    const Piece* piece = a.piece + (int64_t)n * a.pieces;
    float m = -infinity, top[3] = {};
    double s = 0.0;
    if (on)
      for (int p = lane; p < a.pieces; p += 8) m = fmaxf(m, piece[p].m);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (on)
      for (int p = lane; p < a.pieces; p += 8) {
        if (piece[p].m == -infinity && m != -infinity) {  // no entry, or none above -inf
          s += (double)piece[p].s;
          continue;
        }
        const float f = m == -infinity ? 1.0f : exp_of(a, piece[p].m, m);
        s += (double)piece[p].s * (double)f;
#pragma unroll
        for (int q = 0; q < 3; ++q) top[q] = fmaxf(top[q], piece[p].top[q] * f);
      }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      s += __shfl_xor(s, o);
#pragma unroll
      for (int q = 0; q < 3; ++q) top[q] = fmaxf(top[q], __shfl_xor(top[q], o));
    }
    if (lane == 0) {
      sM[n] = m;
#pragma unroll
      for (int q = 0; q < 3; ++q) sP[q][n] = ldexpf(1.0f, std::min(row_exponent(top[q]), 126));
      if (blockIdx.x == 0 && n < N) {
        double logp = 0.0;
        RowOut out{0.0f, 0.0f};
        if (on) {
          const int64_t label = a.labels[n];
          const double w = a.weight ? (double)a.weight[n] : 1.0;
          const float yl = label >= 0 && label < a.b.V ? a.Y[n * a.y_stride + label] : infinity;
          if (!(fabsf(yl) < infinity)) {
            logp = out.mean = out.label = __builtin_nanf("");
          } else {
            const double z = (double)a.tau * ((double)m - (double)yl);
            double q = 0.0;
            if (s != 0.0) {  // (a vocabulary of one entry: p = 1)
              const double d = z + log(s);
              logp = d == d ? -(fmax(d, 0.0) + log1p(exp(-fabs(d)))) : d;
              q = 1.0 / (1.0 + exp(-d));
              out.mean = (float)(w * (double)a.tau * q / s);
            }
            out.label = (float)(w * (double)a.tau * q);
          }
          a.terms[n] = -w * logp;
        } else {
          a.terms[n] = 0.0;
        }
        a.row[n] = out;
        if (a.logp) a.logp[n] = (float)logp;
        if (a.dH)
#pragma unroll
          for (int q = 0; q < 3; ++q) a.b.rscale[3 * n + q] = ldexpf(1.0f, -std::min(row_exponent(top[q]), 126));
      }
    }
  }
  if (!a.dH) return;
  __syncthreads();
  const int oct = tid & 15, run = blockIdx.x;
  const int64_t v = 128 * (int64_t)run + 8 * oct, V16 = 16 * a.b.nb;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = (tid >> 4) + 16 * i;
    if (n >= N) continue;
    h8 f[3] = {};
    if (counts(a, n) && v < V16) {
      const float m = sM[n];
      const int64_t label = a.labels[n];
      const float* y = a.Y + n * a.y_stride + v;
      f4 x[2] = {};
      if (v < a.b.V) x[0] = *reinterpret_cast<const f4*>(y);
      if (v + 4 < a.b.V) x[1] = *reinterpret_cast<const f4*>(y + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (v + j >= a.b.V || v + j == label) continue;
        const float e = exp_of(a, x[j >> 2][j & 3], m);
        float s[3];
        scales_of(a.b, v + j, s);
#pragma unroll
        for (int q = 0; q < 3; ++q) f[q][j] = (_Float16)(fmaf(e, s[q], 0.0f) * sP[q][n]);
      }
    }
    const int64_t step = 8 * (int64_t)run + (oct >> 1);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      reinterpret_cast<h8*>(a.b.hf)[(2 * ((int64_t)q * a.b.ksteps + step) + (oct & 1)) * N + n] = f[q];
  }
}

// Row blockIdx.x x 256 columns of dH, four columns a lane; the waves take a
// quarter each of the splits and of the ranks.
__global__ __launch_bounds__(kFinishThreads) void xent_finish_few_kernel(const XentArgs a) {
  constexpr int kWaves = kFinishThreads / 64;
  extern __shared__ __align__(16) float sZ[];  // [r] factors of B's rows
  __shared__ f4 red[kWaves][64];
  const BwdArgs& b = a.b;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = b.r_c + b.r_r;
  const int64_t n = blockIdx.x, d = 256 * (int64_t)blockIdx.y + 4 * lane, dd = d < b.D ? d : 0, group = dd / b.g;
  const bool on = counts(a, n);
  const int64_t label = on ? a.labels[n] : 0, l = label >= 0 && label < b.V ? label : 0;
  const RowOut out = a.row[n];
  for (int j = tid; j < r; j += kFinishThreads) {
    float z = 0.0f;
#pragma unroll 8
    for (int p = 0; p < b.splits; ++p) z += b.zpart[((int64_t)p * b.n32 + n) * r + j];
    const bool in_c = j < b.r_c;
    const float al = (float)b.a_codes[l * r + j] * f16_to_f32(b.a_scales[l * b.nA + (in_c ? 0 : b.nA - 1)]);
    sZ[j] = out.mean * (z * b.rscale[n * 3 + (in_c ? 1 : 2)]) - out.label * al;
  }
  f4 acc = {};
#pragma unroll 4
  for (int p = wave; p < b.splits; p += kWaves) acc += *reinterpret_cast<const f4*>(b.part + ((int64_t)p * b.N + n) * b.D + dd);
  acc *= b.rscale[n * 3] * out.mean;
  if (wave == 0) {  // the label's row of the residual
    const int64_t kt = dd / kKTile;
    const int k = (int)(dd % kKTile);
    const uint8_t* tile = b.r_codes + (kt * b.nb + l / 16) * kTileBytes;
    const uint32_t w = *reinterpret_cast<const uint16_t*>(tile + 16 * (l % 16 + 16 * (k % 32 / 8)) + 4 * (k / 32) + k % 8 / 2);
    const float s = out.label * ((float)b.r_gcodes[l * b.ng + group] * f16_to_f32(b.r_rowscale[l]));
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(-s, (float)((int32_t)(w << (28 - 4 * e)) >> 28), acc[e]);
  }
  __syncthreads();
#pragma unroll 8
  for (int j = wave; j < r; j += kWaves) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(b.b_codes + (int64_t)j * b.D + dd);
    const float z = sZ[j] * f16_to_f32(b.b_scales[(int64_t)j * b.ng + group]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(z, (float)(int8_t)(c >> (8 * e)), acc[e]);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && d < b.D) {
    for (int w = 1; w < kWaves; ++w) acc += red[w][lane];
    if (!on) acc = f4{};
    typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
    *reinterpret_cast<u2_any*>(a.dH + n * a.dh_stride + d) = pack_bf16x4(acc[0], acc[1], acc[2], acc[3]);
  }
}

// The loss: the rows' terms in fp64, in a fixed order.
constexpr int kTotalThreads = 1024;
__global__ __launch_bounds__(kTotalThreads) void xent_total_kernel(const double* terms, int64_t N, float* loss) {
  __shared__ double buf[kTotalThreads / 64];
  double s = 0.0;
  for (int64_t n = threadIdx.x; n < N; n += kTotalThreads) s += terms[n];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kTotalThreads / 64; ++w) s += buf[w];
    *loss = (float)s;
  }
}

// ------------------------------------------------------------------- host ---

int64_t y_stride_of(const archead_dims* d) { return (int64_t)round_up((uint64_t)d->V, 64); }

struct XentLayout {
  int64_t n32, ksteps, width;
  int pieces, splits;
  uint64_t terms, y, fwd, fwd_bytes, piece, row, rscale, hf, gt, zpart, part, total;
};

// Of a pass of `rows` rows in a call of N.
XentLayout xent_layout(const archead_dims* d, int64_t N, int64_t rows) {
  XentLayout L{};
  if (N <= 0 || rows <= 0) return L;
  const uint64_t V128 = round_up((uint64_t)d->V, 128);
  const int64_t r = d->r_c + d->r_r;
  L.n32 = 32;
  L.ksteps = (int64_t)V128 / 16;
  L.width = (int64_t)round_up((uint64_t)((d->V + kMaxPieces - 1) / kMaxPieces), (uint64_t)kPieceCols);
  L.pieces = (int)((d->V + L.width - 1) / L.width);
  L.splits = main_splits(rows, d->D, (d->r_c + 31) / 32 + (d->r_r + 31) / 32, L.ksteps / 4);
  auto take = [&](uint64_t bytes) {
    const uint64_t at = L.total;
    L.total += round_up(bytes, ARCHEAD_ALIGNMENT);
    return at;
  };
  L.terms = take((uint64_t)N * 8);
  L.y = take((uint64_t)rows * (uint64_t)y_stride_of(d) * 4);
  L.fwd_bytes = workspace_layout(d, rows).total;
  L.fwd = take(L.fwd_bytes);
  L.piece = take((uint64_t)rows * (uint64_t)L.pieces * sizeof(Piece));
  L.row = take((uint64_t)rows * sizeof(RowOut));
  L.rscale = take((uint64_t)rows * 12);
  L.hf = take(V128 * 2 * 3 * (uint64_t)rows);
  L.gt = take(round_up((uint64_t)d->V, 16) * (uint64_t)(d->D / d->g));
  L.zpart = take((uint64_t)L.splits * (uint64_t)L.n32 * (uint64_t)r * 4);
  L.part = take((uint64_t)L.splits * (uint64_t)rows * (uint64_t)d->D * 4);
  return L;
}

uint64_t xent_bytes(const archead_dims* d, int64_t N) {
  return std::max(xent_layout(d, N, std::min(N, kFewTokens)).total, xent_layout(d, N, N % kFewTokens).total);
}

int check_xent_dims(const archead_dims* d) {
  if (int rc = check_kernel_dims(d)) return rc;
  if (int rc = check_archead_format(d)) return rc;
  if (d->V > kXentMaxVocab || d->r_c + d->r_r > kMaxRank) return ARCHEAD_E_UNSUPPORTED;
  return ARCHEAD_OK;
}

// A pass of few rows, from row n0 of the call on.
int launch_few_rows(const archead_tensor* H, const archead_packed_head* head, const archead_cross_entropy_inputs* in,
                    const archead_cross_entropy_outputs* out, int64_t n0, int64_t rows, hipStream_t s) {
  const archead_dims* d = &head->dims;
  const XentLayout L = xent_layout(d, H->rows, rows);
  archead_layout P;
  compute_layout(d, &P);
  const uint8_t* buf = static_cast<const uint8_t*>(head->buffer);
  uint8_t* ws = static_cast<uint8_t*>(head->workspace);
  archead_tensor h = *H;
  h.data = static_cast<uint16_t*>(H->data) + n0 * H->row_stride;
  h.rows = rows;
  archead_tensor y{ws + L.y, rows, d->V, y_stride_of(d), ARCHEAD_F32};
  archead_packed_head p = *head;
  p.workspace = ws + L.fwd;
  p.workspace_bytes = L.fwd_bytes;
  if (int rc = archead_logits(&h, &p, &y, s)) return rc;
  XentArgs a{};
  BwdArgs& b = a.b;
  b.V = d->V;
  b.D = d->D;
  b.N = rows;
  b.n32 = L.n32;
  b.nb = P.padded_rows / 16;
  b.r_c = d->r_c;
  b.r_r = d->r_r;
  b.g = d->g;
  b.ng = (int)(d->D / d->g);
  b.nkt = (int)(d->D / kKTile);
  b.nA = (d->r_c > 0) + (d->r_r > 0);
  b.nct = (d->r_c + 31) / 32;
  b.nwt = (d->r_r + 31) / 32;
  b.r_codes = buf + P.r_codes.offset;
  b.r_gcodes = buf + P.r_gcodes.offset;
  b.r_rowscale = reinterpret_cast<const uint16_t*>(buf + P.r_rowscale.offset);
  b.a_codes = reinterpret_cast<const int8_t*>(buf + P.a_codes.offset);
  b.a_scales = reinterpret_cast<const uint16_t*>(buf + P.a_scales.offset);
  b.b_codes = reinterpret_cast<const int8_t*>(buf + P.b_codes.offset);
  b.b_scales = reinterpret_cast<const uint16_t*>(buf + P.b_scales.offset);
  b.rscale = reinterpret_cast<float*>(ws + L.rscale);
  b.hf = reinterpret_cast<_Float16*>(ws + L.hf);
  b.gt = ws + L.gt;
  b.zpart = reinterpret_cast<float*>(ws + L.zpart);
  b.part = reinterpret_cast<float*>(ws + L.part);
  b.zparts = b.splits = L.splits;
  b.ksteps = (int)L.ksteps;
  a.Y = reinterpret_cast<const float*>(ws + L.y);
  a.y_stride = y.row_stride;
  a.labels = in->labels + n0;
  a.weight = in->weight ? in->weight + n0 : nullptr;
  a.tau = in->inv_temperature;
  const double c = 1.4426950408889634 * (double)in->inv_temperature;
  a.c_hi = (float)c;
  a.c_lo = (float)(c - (double)a.c_hi);
  a.logp = out->logp ? out->logp + n0 : nullptr;
  if (out->dH) {
    a.dH = static_cast<uint16_t*>(out->dH->data) + n0 * out->dH->row_stride;
    a.dh_stride = out->dH->row_stride;
  }
  a.piece = reinterpret_cast<Piece*>(ws + L.piece);
  a.row = reinterpret_cast<RowOut*>(ws + L.row);
  a.terms = reinterpret_cast<double*>(ws + L.terms) + n0;
  a.pieces = L.pieces;
  a.width = L.width;
  const int64_t arrange = a.dH ? b.nb * b.ng / std::max(1, kKTile / b.g) : 0;
  hipLaunchKernelGGL(xent_pieces_kernel, dim3((unsigned)(rows * L.pieces + (arrange + kPieceThreads - 1) / kPieceThreads)),
                     dim3(kPieceThreads), 0, s, a);
  hipLaunchKernelGGL(xent_operand_kernel, dim3(a.dH ? (unsigned)(L.ksteps / 8) : 1u), dim3(kOperandThreads), 0, s, a);
  if (hipGetLastError() != hipSuccess) return ARCHEAD_E_HIP;
  if (!a.dH) return ARCHEAD_OK;
  if (launch_bwd_few(b, s) != hipSuccess) return ARCHEAD_E_HIP;
  hipLaunchKernelGGL(xent_finish_few_kernel, dim3((unsigned)rows, (unsigned)((b.D + 255) / 256)), dim3(kFinishThreads),
                     (size_t)(b.r_c + b.r_r) * 4, s, a);
  return hipGetLastError() == hipSuccess ? ARCHEAD_OK : ARCHEAD_E_HIP;
}

}  // namespace
}  // namespace archead

using namespace archead;

extern "C" {

int archead_cross_entropy_workspace_bytes(const archead_dims* d, int64_t n_tokens, uint64_t* bytes) {
  if (!d || !bytes) return ARCHEAD_E_NULL;
  if (int rc = check_xent_dims(d)) return rc;
  if (n_tokens < 0) return ARCHEAD_E_SHAPE;
  if (n_tokens > kXentMaxRows) return ARCHEAD_E_UNSUPPORTED;
  *bytes = xent_bytes(d, n_tokens);
  return ARCHEAD_OK;
}

int archead_cross_entropy(const archead_tensor* H, const archead_packed_head* head,
                          const archead_cross_entropy_inputs* in, const archead_cross_entropy_outputs* out, void* stream) {
  if (!H || !head || !in || !out) return ARCHEAD_E_NULL;
  const archead_dims* d = &head->dims;
  if (int rc = check_xent_dims(d)) return rc;
  const archead_tensor* dH = out->dH;
  if (H->dtype != ARCHEAD_BF16 || (dH && dH->dtype != ARCHEAD_BF16)) return ARCHEAD_E_DTYPE;
  const int64_t N = H->rows;
  if (N < 0 || H->cols != d->D || H->row_stride < d->D) return ARCHEAD_E_SHAPE;
  if (dH && (dH->rows != N || dH->cols != d->D || dH->row_stride < d->D)) return ARCHEAD_E_SHAPE;
  if (N > kXentMaxRows) return ARCHEAD_E_UNSUPPORTED;
  if (!(in->inv_temperature > 0.0f) || !(in->inv_temperature < __builtin_huge_valf())) return ARCHEAD_E_VALUE;
  if ((uintptr_t)out->loss % 4 || (uintptr_t)out->logp % 4 || (uintptr_t)in->labels % 4 || (uintptr_t)in->weight % 4)
    return ARCHEAD_E_ALIGN;
  if (N > 0) {
    if (!H->data || !head->buffer || !head->workspace || !in->labels || (dH && !dH->data)) return ARCHEAD_E_NULL;
    if ((uintptr_t)H->data % 16 || (H->row_stride * 2) % 16 || (dH && (uintptr_t)dH->data % 2)) return ARCHEAD_E_ALIGN;
    if ((uintptr_t)head->buffer % ARCHEAD_ALIGNMENT || (uintptr_t)head->workspace % ARCHEAD_ALIGNMENT) return ARCHEAD_E_ALIGN;
    archead_layout P;
    compute_layout(d, &P);
    if (head->buffer_bytes < P.total_bytes) return ARCHEAD_E_SIZE;
    const uint64_t need = xent_bytes(d, N);
    if (head->workspace_bytes < need) return ARCHEAD_E_WORKSPACE;
    if (!forward_takes(d, std::min(N, kFewTokens)) || (N % kFewTokens && !forward_takes(d, N % kFewTokens)))
      return ARCHEAD_E_UNSUPPORTED;
    if (dH && overlap(H, 2, dH, 2)) return ARCHEAD_E_SHAPE;
    // what the call writes shares bytes with nothing else
    struct Span {
      uint64_t at, bytes;
    };
    auto tensor = [&](const archead_tensor* t) { return Span{(uint64_t)t->data, ((uint64_t)(N - 1) * (uint64_t)t->row_stride + (uint64_t)t->cols) * 2}; };
    const Span written[] = {{(uint64_t)out->loss, out->loss ? 4u : 0u}, {(uint64_t)out->logp, out->logp ? 4 * (uint64_t)N : 0},
                            {(uint64_t)head->workspace, need}, dH ? tensor(dH) : Span{0, 0}};
    const Span read[] = {{(uint64_t)in->labels, 4 * (uint64_t)N}, {(uint64_t)in->weight, in->weight ? 4 * (uint64_t)N : 0},
                         {(uint64_t)head->buffer, P.total_bytes}, tensor(H)};
    auto meet = [](const Span& x, const Span& y) { return x.bytes && y.bytes && x.at < y.at + y.bytes && y.at < x.at + x.bytes; };
    for (int i = 0; i < 4; ++i) {
      for (int j = 0; j < 4; ++j)
        if (!(i == 3 && j == 3) && meet(written[i], read[j])) return ARCHEAD_E_SHAPE;  // (dH and H: above)
      for (int j = 0; j < i; ++j)
        if (meet(written[i], written[j])) return ARCHEAD_E_SHAPE;
    }
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // start from a clean error state
  for (int64_t n0 = 0; n0 < N; n0 += kFewTokens)
    if (int rc = launch_few_rows(H, head, in, out, n0, std::min(kFewTokens, N - n0), s)) return rc;
  if (out->loss) {
    hipLaunchKernelGGL(xent_total_kernel, dim3(1), dim3(kTotalThreads), 0, s, static_cast<const double*>(head->workspace), N, out->loss);
    if (hipGetLastError() != hipSuccess) return ARCHEAD_E_HIP;
  }
  return ARCHEAD_OK;
}

}  // extern "C"
