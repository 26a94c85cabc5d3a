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
//   xent_operand_kernel     e s_R, e s_Ac, e s_Aw as fp16 operands; log p, loss
//   bwd_few_kernel, bwd_few16_kernel (backward.hip)
//   xent_finish_few_kernel  the splits' sums, Z B and the label's row to dH
// More rows, those that count gathered, up to 4096 at a time; for every piece
//   tile32_exp_kernel       the exponentials as fp16 operands, with an exponent
//                           and a sum for each row and 32 entries
//   xent_merge_kernel       the rows' running exponent and sum, and what brings
//                           the sums before the piece to that exponent
//   xent_move_kernel        operands at other exponents than their row's
//   xent_z_kernel           (e s_A) code added to Z
//   xent_main_kernel        e (s_R q4 c8) added to the sums
// and at the end xent_rows_kernel (log p, Z), xent_finish_kernel (dH).
//
// Few rows are bound by the head's bytes, which are read twice, for the logits
// and for dH: one row of a 151936 x 4096 head 150 us, of it 57 and 67 of the
// two readings and 29 of the launches around them; the loss alone 70.  Both ways
// at the border, calls of at most 32 rows each and the other one: 33 rows of a
// 151936 x 4096 head 394 and 341 us, 64 rows 493 and 361; of 32000 x 2048 124 and
// 133, 148 and 135; of 1024 x 256 82 and 72, 95 and 72.  32 rows in one call take
// 245, 75 and 48, and as much as 33 the other way.
//
// Many rows are bound by the MFMAs under the power limit, two products of the
// head with the rows: 4096 rows, nine in ten of which count, 9.1 to 9.3 ms, 4.8 in
// tile32_exp_kernel (0.96 PFLOP/s) and 3.9 to 4.1 in xent_main_kernel (1.13), 0.7
// in what joins the pieces; 4096 rows that all count 10.1 ms, their loss alone 5.0
// (bf16 logits of them 4.6).
#include <algorithm>
#include <limits>

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

// What the last kernel needs of a row: dH is `all` times the others' sum over S
// less the label's row.  `all` comes last, since q and with it what it
// multiplies may be below 2^-126.
struct RowOut {
  float mean, all;  // 1 / S, w tau q
};

struct XentArgs {
  BwdArgs b;  // the head, the product's operands and sums; N rows from row n0 of the call
  const float* Y;
  int64_t y_stride;
  const int32_t* labels;
  const float* weight;
  float tau, c_hi, c_lo;  // log2(e) tau = c_hi + c_lo, both above zero
  float* logp;            // or null
  uint16_t* dH;           // or null
  int64_t dh_stride;
  Piece* piece;           // [N][pieces]
  RowOut* row;            // [N]
  float* loss;            // or null
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

// exp(z - m) of a logit: differences before the scale, so that nothing
// overflows.  The difference is -inf of a logit that is: both products are -inf
// then and the result 0, as neither part of the scale is negative or zero.
__device__ __forceinline__ float exp_of(const XentArgs& a, float y, float m) {
  const float d = y - m;
  return __builtin_amdgcn_exp2f(fmaf(d, a.c_hi, d * a.c_lo));
}

// What exponentials are taken relative to where the maximum is m: of no logit
// above -inf any number, so that they are 0 (and NaN of a NaN).
__device__ __forceinline__ float base_of(float m) { return m == -__builtin_huge_valf() ? 0.0f : m; }

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
  const float base = base_of(m);
  float sum = 0.0f, top[3] = {};
  for (int64_t v = v0 + 4 * threadIdx.x; v < v1; v += 4 * kPieceThreads) {
    const f4 x = load4(v);
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (v + j >= v1 || v + j == label) continue;
      const float e = exp_of(a, x[j], base);
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

constexpr int kOperandThreads = 256;
// Run blockIdx.x of 128 columns of all rows as operands, thread t octet t % 16
// of rows t / 16 and t / 16 + 16; the rows' pieces are merged by every
// workgroup, and the first one writes what is known of the rows then, and the
// loss.
__global__ __launch_bounds__(kOperandThreads) void xent_operand_kernel(const XentArgs a) {
  __shared__ float sM[32], sP[3][32];
  __shared__ double sTerm[32];
  const int tid = threadIdx.x, N = (int)a.b.N;
  const float infinity = __builtin_huge_valf();
  {  // eight lanes a row; a wave a row where its pieces take eight lanes many rounds
     // (75 pieces of one row: 8.0 us, with eight lanes 10.8; one piece of four rows: 8.5 and 6.7)
    const int bits = N <= 4 && a.pieces > 16 ? 6 : 3, lanes = 1 << bits, n = tid >> bits, lane = tid & (lanes - 1);
    const bool on = n < N && counts(a, n);
    const Piece* piece = a.piece + (int64_t)n * a.pieces;
    float m = -infinity, top[3] = {};
    double s = 0.0;
    if (on)
      for (int p = lane; p < a.pieces; p += lanes) m = fmaxf(m, piece[p].m);
    for (int o = lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (on)
      for (int p = lane; p < a.pieces; p += lanes) {
        if (piece[p].m == -infinity) {  // no entry, or none above -inf
          s += (double)piece[p].s;
          continue;
        }
        const float f = exp_of(a, piece[p].m, m);
        s += (double)piece[p].s * (double)f;
#pragma unroll
        for (int q = 0; q < 3; ++q) top[q] = fmaxf(top[q], piece[p].top[q] * f);
      }
    for (int o = lanes / 2; o > 0; o >>= 1) {
      s += __shfl_xor(s, o);
#pragma unroll
      for (int q = 0; q < 3; ++q) top[q] = fmaxf(top[q], __shfl_xor(top[q], o));
    }
    if (lane == 0) {
      sM[n] = base_of(m);
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
            logp = out.all = __builtin_nanf("");
          } else {
            const double z = (double)a.tau * ((double)m - (double)yl);
            double q = 0.0;
            if (s != 0.0) {  // (a vocabulary of one entry: p = 1)
              const double d = z + log(s);
              logp = d == d ? -(fmax(d, 0.0) + log1p(exp(-fabs(d)))) : d;
              q = 1.0 / (1.0 + exp(-d));
              out.mean = (float)(1.0 / s);
            }
            out.all = (float)(w * (double)a.tau * q);
          }
          sTerm[n] = -w * logp;
        } else {
          sTerm[n] = 0.0;
        }
        a.row[n] = out;
        if (a.logp) a.logp[n] = (float)logp;
        if (a.dH)
#pragma unroll
          for (int q = 0; q < 3; ++q) a.b.rscale[3 * n + q] = ldexpf(1.0f, -std::min(row_exponent(top[q]), 126));
      }
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0 && a.loss) {
    double loss = 0.0;
    for (int n = 0; n < N; ++n) loss += sTerm[n];
    *a.loss = (float)loss;
  }
  if (!a.dH) return;
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
    sZ[j] = out.mean * (z * b.rscale[n * 3 + (in_c ? 1 : 2)]) - al;
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
    const float s = (float)b.r_gcodes[l * b.ng + group] * f16_to_f32(b.r_rowscale[l]);
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
    acc = on ? acc * out.all : f4{};
    typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
    *reinterpret_cast<u2_any*>(a.dH + n * a.dh_stride + d) = pack_bf16x4(acc[0], acc[1], acc[2], acc[3]);
  }
}

// ------------------------------------------------------------ many rows ---

constexpr int64_t kChunkRows = 4096;                // rows that count, a pass
// Of a piece's operands.  Every piece adds to the partial sums of all before, so
// fewer are better until they outgrow the last cache: 4096 rows of 151936 x 4096
// take 9.97 ms with 64 MiB, 9.64 with 128, 9.52 with 192, 9.34 with 256 and with
// 384, 9.35 with 512.
constexpr uint64_t kPieceBytes = 256ull << 20;
// Where 512 workgroups of 2 row tiles (two a CU) do the tiles of the first
// product, they get 2, and the launches for other numbers are left out: 200 rows
// of 8192 x 1024 take 126 us in place of 156, 250 of 32000 x 2048 194 (206), 4096
// of 1024 x 2048 166 (193); with up to 1536 workgroups, 250 of 65536 x 2048 take
// 287 in place of 256, 130 of 65536 x 4096 350 (286).
constexpr int64_t kSmall = 512;
constexpr int kHeadParts = 64, kHeadThreads = 256;
constexpr int kMergeRows = 8, kMergeSlices = 128;
constexpr int kZThreads = 512, kZTiles = 4;         // rank tiles of a workgroup

struct ManyArgs {
  BwdArgs b;               // of a pass: N its most rows; hf the piece's operands e, ksteps its steps
  int64_t rows;            // of the call
  const uint16_t* H;
  int64_t h_stride;
  const int32_t* labels;   // of the call, by row
  const float* weight;
  float tau;
  float* logp;
  uint16_t* dH;
  int64_t dh_stride;
  float* head_max;         // [kHeadParts][3]
  float* scale;            // [4] the power of two that s_R are taken with; what undoes those of the sums, Z_c, Z_w
  _Float16* scale_a;       // [2][16 vtiles of V][16] s_Ac, s_Aw times powers of two
  int32_t* map;            // [rows] rows that count, in order
  int32_t* label;          // [rows] their labels
  int32_t* plan;           // [passes][4] rows that count, row tiles of a workgroup, parts of a piece's product
  double* terms;           // [rows] -w log p by row of the call
  uint16_t* Hc;            // [n32][D] gathered H
  float* stat;             // [blocks][n32][2]
  float* alpha;            // [n32]
  float* ref;              // [n32] running exponent
  int32_t* moved;          // [n32/kMergeRows] whether operands of these rows are at others
  double* sum;             // [n32] running sum
  float* z_label;          // [n32] log2(e) tau times the label's logit
  RowOut* row;             // [n32]
  int64_t asteps;          // steps of the whole vocabulary
  int row_tiles;           // of a workgroup for any number of rows that count, or 0: by that number
  int pass, passes, blocks, first, step0, steps;
  int64_t part_rows;       // room for partial sums
  int64_t main_steps;      // steps of a whole piece
};

// Workgroups of the product's launches, for any number of rows that count.
__host__ __device__ inline int64_t main_groups(int64_t rows, int64_t D, int tt) {
  return std::max<int64_t>((rows + 32 * tt - 1) / (32 * tt) * ((D + 255) / 256), tt == 2 ? 1024 : 512);
}

// The rows that count, in order, by one workgroup, and how the kernels that
// multiply with the head cut each pass.
__device__ __forceinline__ void order_rows(const ManyArgs& a) {
  constexpr int kRows = 4, kWaves = kHeadThreads / 64;  // rows of a thread at a time
  __shared__ int sCount[kRows][kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t total = 0;
  for (int64_t n0 = 0; n0 < a.rows; n0 += kRows * kHeadThreads) {
    uint64_t on[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t n = n0 + kHeadThreads * i + tid;
      on[i] = __ballot(n < a.rows && (!a.weight || a.weight[n] != 0.0f));
      if (lane == 0) sCount[i][wave] = __popcll(on[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t n = n0 + kHeadThreads * i + tid;
      int64_t at = total + __popcll(on[i] & ((1ull << lane) - 1));
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? sCount[i][w] : 0;
        total += sCount[i][w];
      }
      if (on[i] >> lane & 1) {
        a.map[at] = (int32_t)n;
        a.label[at] = a.labels[n];
      } else if (n < a.rows) {
        a.terms[n] = 0.0;
        if (a.logp) a.logp[n] = 0.0f;
      }
    }
    __syncthreads();
  }
  for (int p = tid; p < a.passes; p += kHeadThreads) {
    const int64_t count = std::max<int64_t>(0, std::min(total - p * kChunkRows, kChunkRows));
    const int tt = a.row_tiles ? a.row_tiles : exp_tiles((count + 31) / 32, a.b.D >= 256);
    const int64_t tiles = std::max<int64_t>(1, (count + 32 * tt - 1) / (32 * tt) * ((a.b.D + 255) / 256));
    const int64_t most = std::min(std::min<int64_t>(kMaxSplits, a.main_steps / 4),
                                  std::min(main_groups(a.b.N, a.b.D, tt) / tiles, a.part_rows / std::max<int64_t>(count, 1)));
    a.plan[4 * p] = (int32_t)count;
    a.plan[4 * p + 1] = tt;
    a.plan[4 * p + 2] = best_parts(count, a.b.D, a.main_steps / 4, tt, most);
  }
}

// What waits for nothing.  Workgroup 0: order_rows.  The next kHeadParts: largest
// |s_R|, |s_Ac|, |s_Aw| of a part of the vocabulary.  The next `arrange`: the A
// codes in the order of the product along the vocabulary.  Those behind, for
// rows that do not count: their gradient.
__global__ __launch_bounds__(kHeadThreads) void xent_head_kernel(const ManyArgs a, int64_t arrange) {
  __shared__ float buf[kHeadThreads / 64][3];
  if (blockIdx.x == 0) return order_rows(a);
  const int64_t part = (int64_t)blockIdx.x - 1;
  if (part >= kHeadParts) {
    const int64_t i = part - kHeadParts, n = i - arrange;
    if (n < 0)
      arrange_codes(a.b, i * kHeadThreads + threadIdx.x);
    else if (a.weight[n] == 0.0f)
      for (int64_t d = threadIdx.x; d < a.b.D; d += kHeadThreads) a.dH[n * a.dh_stride + d] = 0;
    return;
  }
  float m[3] = {};
  for (int64_t v = part * kHeadThreads + threadIdx.x; v < a.b.V; v += kHeadParts * kHeadThreads) {
    float s[3];
    scales_of(a.b, v, s);
#pragma unroll
    for (int q = 0; q < 3; ++q) m[q] = fmaxf(m[q], fabsf(s[q]));
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    m[q] = wave_max(m[q]);
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6][q] = m[q];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = buf[0][threadIdx.x];
    for (int w = 1; w < kHeadThreads / 64; ++w) t = fmaxf(t, buf[w][threadIdx.x]);
    a.head_max[3 * part + threadIdx.x] = t;
  }
}

// What the head's scales give: powers of two that bring the largest |q4 c8 s_R|
// (2040 at most before s_R) and the largest |s_A| to [2^14, 2^15) and [1/2, 1),
// and s_A times theirs, of entry i.  Nothing is lost by that where the largest s_R
// is below 16 and the largest s_A below 1, as a power of 1 and more makes no fp16
// number subnormal; else an s_R below 2^-17 (s_A: 2^-13) of the largest loses digits,
// half a step being 2^-28 (2^-24) of the largest at most.  The product (q4 c8) s_R
// is rounded to fp16 in any case, 2^-11 of itself or 2^-39 of the largest weight,
// and so is e s_A, 2^-11 or, beside a row's largest e, 2^-34 of the largest s_A.
__device__ __forceinline__ void head_scales(const ManyArgs& a, int64_t i) {
  static_assert(kHeadParts == 64, "a part for each lane");
  int k[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const float m = wave_max(a.head_max[3 * (threadIdx.x & 63) + q]);
    k[q] = std::max(-100, std::min(q == 0 ? row_exponent(2040.0f * m) : row_exponent(m) - 15, 100));
  }
  if (i < 4) a.scale[i] = ldexpf(1.0f, i == 0 ? k[0] : -k[i - 1]);
  if (i < 16 * a.asteps)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float s[3] = {};
      if (i < a.b.V) scales_of(a.b, i, s);
      a.scale_a[q * 16 * a.asteps + i] = (_Float16)ldexpf(s[1 + q], k[1 + q]);
    }
}

// Row blockIdx.x of the pass: its H (zeros behind the last one that counts),
// and no sums.  Workgroups behind the rows: head_scales.
__global__ __launch_bounds__(256) void xent_gather_kernel(const ManyArgs a) {
  const int64_t i = blockIdx.x, count = a.plan[4 * a.pass];
  if (i >= a.b.n32) return head_scales(a, (i - a.b.n32) * 256 + threadIdx.x);
  if (threadIdx.x == 0) {
    a.ref[i] = -__builtin_huge_valf();
    a.sum[i] = 0.0;
    a.z_label[i] = __builtin_nanf("");  // stays where the label is outside the vocabulary
  }
  const u4* src = reinterpret_cast<const u4*>(a.H + (i < count ? (int64_t)a.map[a.pass * kChunkRows + i] : 0) * a.h_stride);
  u4* dst = reinterpret_cast<u4*>(a.Hc + i * a.b.D);
  for (int64_t c = threadIdx.x; c < a.b.D / 8; c += 256) dst[c] = i < count ? src[c] : u4{};
}

// kMergeRows rows a workgroup, kMergeSlices threads each: the sum of the piece's blocks
// and of those before, and the running exponent, which is moved only where a
// block has one above it: to kHeadroom above the largest, so that few pieces
// move it.  (With 32 rows a workgroup, 8 of them read 8 MB: 34 us, now 20.)
constexpr float kHeadroom = 3.0f;
__global__ __launch_bounds__(kMergeRows * kMergeSlices) void xent_merge_kernel(const ManyArgs a) {
  constexpr int kWaves = kMergeRows * kMergeSlices / 64;
  __shared__ float sTop[kWaves][kMergeRows];
  __shared__ double sSum[kWaves][kMergeRows];
  constexpr int kBatch = 16;  // loads in flight: their latency is what a round takes
  const int c = threadIdx.x % kMergeRows, slice = threadIdx.x / kMergeRows;
  const int64_t n = kMergeRows * (int64_t)blockIdx.x + c;
  if (n / 32 * 32 >= a.plan[4 * a.pass]) return;
  const float infinity = __builtin_huge_valf();
  const u2* stat = reinterpret_cast<const u2*>(a.stat) + n;
  // sum s at exponent m moved to m + j (j whole and not below 0, or not finite
  // where there is no entry or the row is not finite, which shows in s)
  auto moved = [](double s, float j) { return j <= 1000.0f ? ldexp(s, -(int)j) : s == s ? 0.0 : s; };
  float m = -infinity;
  double s = 0.0;
  for (int k0 = slice; k0 < a.blocks; k0 += kBatch * kMergeSlices) {
    u2 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) x[i] = stat[(int64_t)std::min(k0 + i * kMergeSlices, a.blocks - 1) * a.b.n32];
    float t = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) t = fmaxf(t, __uint_as_float(x[i][0]));
    s = moved(s, t - m);
    m = t;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (k0 + i * kMergeSlices < a.blocks) {  // (2^-149 is nothing beside the largest, 2^-8 at least)
        const float y = __uint_as_float(x[i][1]), j = m - __uint_as_float(x[i][0]);
        s += (double)(j <= 1000.0f ? ldexpf(y, -(int)j) : y == y ? 0.0f : y);
      }
  }
  auto join = [&](float m1, double s1) {
    const float t = fmaxf(m, m1);
    s = moved(s, t - m) + moved(s1, t - m1);
    m = t;
  };
#pragma unroll
  for (int o = kMergeRows; o < 64; o *= 2) join(__shfl_xor(m, o), __shfl_xor(s, o));
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) < kMergeRows) {
    sTop[wave][c] = m;
    sSum[wave][c] = s;
  }
  __syncthreads();
  if (slice == 0) {
    for (int k = 1; k < kWaves; ++k) join(sTop[k][c], sSum[k][c]);
    const float old = a.ref[n];
    float t = fmaxf(old, m);
    const bool raised = t > old;
    if (raised) t += kHeadroom;
    a.sum[n] = moved(a.sum[n], t - old) + moved(s, t - m);
    a.ref[n] = t;
    a.alpha[n] = t - old <= 1000.0f ? ldexpf(1.0f, -(int)(t - old)) : 0.0f;
    const bool any = __any(raised);
    if (c == 0) a.moved[blockIdx.x] = any;
  }
}

// Operands times 2^t, t whole and below 0 (times 0 where it is not a number),
// in two steps, as fp16's least power is 2^-24 and operands reach 2^15.
__device__ __forceinline__ h8 times_power(h8 x, float t) {
  t = fmaxf(t, -100.0f);
  const float lo = fmaxf(t, -20.0f);
  const _Float16 a = (_Float16)ldexpf(1.0f, (int)lo), b = (_Float16)ldexpf(1.0f, (int)(t - lo));
  x = x * h8{a, a, a, a, a, a, a, a};
  return x * h8{b, b, b, b, b, b, b, b};
}

// The operands of rows whose exponent this piece moved, brought there in place:
// exactly, but for what ends below 2^-14.  Row tiles without such rows are left
// alone, and of the others the rows.  (In the product, which reads every operand
// once for 256 columns, the same takes 9% of all its time.)  Wave: every
// gridDim.y kMoveWaves-th block of row tile blockIdx.x.
constexpr int kMoveWaves = 4;
__global__ __launch_bounds__(64 * kMoveWaves) void xent_move_kernel(const ManyArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t tile = blockIdx.x, n = 32 * tile + (lane & 31);
  if (32 * tile >= a.plan[4 * a.pass]) return;
  int any = 0;
#pragma unroll
  for (int i = 0; i < 32 / kMergeRows; ++i) any |= a.moved[32 / kMergeRows * tile + i];
  if (!any) return;
  constexpr int kBatch = 4;
  const float ref = a.ref[n];
  h8* e = reinterpret_cast<h8*>(a.b.hf) + tile * a.steps * 64 + lane;
  const int first = (int)blockIdx.y * kMoveWaves + (threadIdx.x >> 6), stride = kMoveWaves * gridDim.y;
  for (int k0 = first; k0 < a.blocks; k0 += kBatch * stride) {
    float t[kBatch];
    h8 x[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)  // past the last block: nothing
      t[i] = k0 + i * stride < a.blocks ? a.stat[2 * ((int64_t)(k0 + i * stride) * a.b.n32 + n)] - ref : 0.0f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (t[i] != 0.0f)
#pragma unroll
        for (int h = 0; h < 2; ++h) x[i][h] = e[(2 * (int64_t)(k0 + i * stride) + h) * 64];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (t[i] != 0.0f)
#pragma unroll
        for (int h = 0; h < 2; ++h) e[(2 * (int64_t)(k0 + i * stride) + h) * 64] = times_power(x[i][h], t[i]);
  }
}

// 64 rows x kZTiles rank tiles (half of them of each part of the ranks) a
// workgroup over part blockIdx.y of the piece's steps, dealt to the waves; e s_A
// is formed in registers (rounded to fp16 once more), the codes are exact.  The
// waves' sums are added up in order and then to the part's sums of the pieces
// before.  Bound by the operands' bytes (250 MB a full piece, 84 us).
__global__ __launch_bounds__(kZThreads, 2) void xent_z_kernel(const ManyArgs a) {
  constexpr int kWaves = kZThreads / 64, kDepth = 3;
  __shared__ float red[kWaves / 2][kZTiles][16][64];
  const BwdArgs& b = a.b;
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t count = a.plan[4 * a.pass], ntiles = (count + 31) / 32, tile0 = 2 * (int64_t)blockIdx.x;
  if (tile0 >= ntiles) return;
  const int parts = gridDim.y, r = b.r_c + b.r_r;
  // rank tile of slot t: of part c (0) or w (1), its place in the part
  auto part_of = [](int t) { return t / (kZTiles / 2); };
  auto place_of = [&](int t) { return kZTiles / 2 * (int)blockIdx.z + t % (kZTiles / 2); };
  const int k0 = (int)((int64_t)blockIdx.y * b.ksteps / parts), k1 = (int)((int64_t)(blockIdx.y + 1) * b.ksteps / parts);
  // row tiles start at different steps, so that they are not all at the same memory channels
  const int turn = k1 > k0 ? (int)(blockIdx.x * 5 * kWaves % (unsigned)(k1 - k0)) : 0;
  const h8* e[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    e[i] = reinterpret_cast<const h8*>(b.hf) + std::min(tile0 + i, ntiles - 1) * a.steps * 64 + lane;
  const u2* codes[kZTiles];
#pragma unroll
  for (int t = 0; t < kZTiles; ++t)  // past a part's last tile: another, not stored
    codes[t] = reinterpret_cast<const u2*>(b.af) +
               ((int64_t)std::min(place_of(t) + (part_of(t) ? b.nct : 0), b.nct + b.nwt - 1) * a.asteps + a.step0) * 64 + lane;
  const h8* scale[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) scale[q] = reinterpret_cast<const h8*>(a.scale_a) + 2 * (q * a.asteps + a.step0) + half;
  f16x acc[2][kZTiles] = {};
  h8 x[kDepth][2], s[kDepth][2];
  u2 y[kDepth][kZTiles];
  auto load = [&](int k, auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
    k = std::min(k, k1 - 1) + turn;  // past the end: a step that is not used
    k -= k >= k1 ? k1 - k0 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) x[slot][i] = e[i][(int64_t)k * 64];
#pragma unroll
    for (int q = 0; q < 2; ++q) s[slot][q] = scale[q][2 * (int64_t)k];
#pragma unroll
    for (int t = 0; t < kZTiles; ++t) y[slot][t] = codes[t][(int64_t)k * 64];
    __builtin_amdgcn_sched_barrier(0);
  };
  auto use = [&](auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const h8 part[2] = {x[slot][i] * s[slot][0], x[slot][i] * s[slot][1]};
#pragma unroll
      for (int t = 0; t < kZTiles; ++t) acc[i][t] = mfma32(part[part_of(t)], unpack_u8x8(y[slot][t]), acc[i][t]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  if (k0 + wave < k1) {
    static_for<0, kDepth>([&](auto i) { load(k0 + wave + kWaves * decltype(i)::value, i); });
    int g0 = k0 + wave;
    for (; g0 + kWaves * (kDepth - 1) < k1; g0 += kWaves * kDepth)
      static_for<0, kDepth>([&](auto i) {
        use(i);
        load(g0 + kWaves * (decltype(i)::value + kDepth), i);
      });
    static_for<0, kDepth - 1>([&](auto i) {
      if (g0 + kWaves * decltype(i)::value < k1) use(i);
    });
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int h = kWaves / 2; h > 0; h >>= 1) {
      __syncthreads();
      if (wave >= h && wave < 2 * h) {
#pragma unroll
        for (int t = 0; t < kZTiles; ++t)
#pragma unroll
          for (int v = 0; v < 16; ++v) red[wave - h][t][v][lane] = acc[i][t][v];
      }
      __syncthreads();
      if (wave < h) {
#pragma unroll
        for (int t = 0; t < kZTiles; ++t)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][t][v] += red[wave][t][v][lane];
      }
    }
    if (wave != 0 || tile0 + i >= ntiles) continue;
    float alpha[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) alpha[v] = a.alpha[32 * (tile0 + i) + 8 * (v >> 2) + 4 * half + (v & 3)];
#pragma unroll
    for (int t = 0; t < kZTiles; ++t) {
      const bool in_c = part_of(t) == 0;
      const int j = 32 * place_of(t) + c32;
      if (j >= (in_c ? b.r_c : b.r_r)) continue;
      // (rows of a tile past the last one that counts have a place, too)
      float* z = b.zpart + ((int64_t)blockIdx.y * b.n32 + 32 * (tile0 + i) + 4 * half) * r + (in_c ? 0 : b.r_c) + j;
      if (!a.first) {
        float old[16];
#pragma unroll
        for (int v = 0; v < 16; ++v) old[v] = z[(8 * (v >> 2) + (v & 3)) * r];
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][t][v] = fmaf(alpha[v], old[v], acc[i][t][v]);
      }
#pragma unroll
      for (int v = 0; v < 16; ++v) z[(8 * (v >> 2) + (v & 3)) * r] = acc[i][t][v];
    }
  }
}

template <int TT, int kCodes>
__global__ __launch_bounds__(kMainThreads, 2) void xent_main_kernel(const BwdArgs a, const MainExp ex) {
  bwd_main_body<TT, kCodes, true>(a, ex);
}

// Row blockIdx.x of the pass: log p and its term of the loss, the factors of
// its sums, and Z less the label's A, with those factors.
__global__ __launch_bounds__(256) void xent_rows_kernel(const ManyArgs a) {
  __shared__ RowOut sOut;
  const BwdArgs& b = a.b;
  const int64_t i = blockIdx.x;
  if (i >= a.plan[4 * a.pass]) return;
  const int64_t at = a.pass * kChunkRows + i, label = a.label[at], l = label >= 0 && label < b.V ? label : 0;
  if (threadIdx.x == 0) {
    const int64_t n = a.map[at];
    const double w = a.weight ? (double)a.weight[n] : 1.0, s = a.sum[i];
    const float zl = a.z_label[i];
    double logp = 0.0, q = 0.0;
    RowOut out{0.0f, 0.0f};
    if (!(fabsf(zl) < __builtin_huge_valf())) {
      logp = q = __builtin_nan("");
    } else if (s != 0.0) {  // (a vocabulary of one entry: p = 1)
      const double d = log(s) + ((double)a.ref[i] - (double)zl) * 0.6931471805599453;
      logp = d == d ? -(fmax(d, 0.0) + log1p(exp(-fabs(d)))) : d;
      q = 1.0 / (1.0 + exp(-d));
      out.mean = (float)(1.0 / s);
    }
    out.all = (float)(w * (double)a.tau * q);
    a.terms[n] = -w * logp;
    if (a.logp) a.logp[n] = (float)logp;
    a.row[i] = sOut = out;
  }
  if (!a.dH) return;
  __syncthreads();
  const int r = b.r_c + b.r_r;
  for (int j = threadIdx.x; j < r; j += 256) {
    float z = 0.0f;
#pragma unroll 8
    for (int p = 0; p < b.zparts; ++p) z += b.zpart[((int64_t)p * b.n32 + i) * r + j];
    const bool in_c = j < b.r_c;
    const float al = (float)b.a_codes[l * r + j] * f16_to_f32(b.a_scales[l * b.nA + (in_c ? 0 : b.nA - 1)]);
    b.z[i * r + j] = sOut.mean * (z * a.scale[in_c ? 2 : 3]) - al;
  }
}

// 32 rows x 128 columns of dH a wave: the splits' sums, the label's row of the
// residual, and Z B on the bf16 MFMA with Z and B as pairs of bf16 numbers (three
// products, 2^-15 of |Z| |B| at most).  Tile c of four holds the columns 4 i +
// c, so that a lane has four neighbouring ones of a row.
template <bool kShare>
__global__ __launch_bounds__(kFinishThreads, 2) void xent_finish_kernel(const ManyArgs a) {
  constexpr int kWaves = kFinishThreads / 64;
  const BwdArgs& b = a.b;
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = b.r_c + b.r_r;
  const int first = kShare ? wave : 0, waves = kShare ? kWaves : 1;  // of the splits and of the ranks
  const int64_t n0 = 32 * (int64_t)blockIdx.x, kt = kShare ? (int64_t)blockIdx.y : (int64_t)blockIdx.y * kWaves + wave;
  const int64_t count = a.plan[4 * a.pass];
  if (n0 >= count || kt >= b.nkt) return;
  const int64_t d = kKTile * kt + 4 * c32, group = d / b.g;
  // row of element v of a result tile; past the last row that one
  auto row = [&](int v) { return std::min<int64_t>(n0 + 8 * (v >> 2) + 4 * half + (v & 3), count - 1); };
  const int splits = a.plan[4 * a.pass + 2];
  f16x acc[4] = {};
  for (int p = first; p < splits; p += waves) {
    f4 y[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) y[v] = *reinterpret_cast<const f4*>(b.part + ((int64_t)p * count + row(v)) * b.D + d);
#pragma unroll
    for (int v = 0; v < 16; ++v)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c][v] += y[v][c];
  }
  const float undo = a.scale[1];
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int64_t label = a.label[a.pass * kChunkRows + row(v)], l = label >= 0 && label < b.V ? label : 0;
    const uint8_t* tile = b.r_codes + (kt * b.nb + l / 16) * kTileBytes;
    const uint32_t w = *reinterpret_cast<const uint16_t*>(tile + 16 * (l % 16 + 16 * (c32 % 8 / 2)) + 4 * (c32 / 8) + 2 * (c32 % 2));
    const float s = (float)b.r_gcodes[l * b.ng + group] * f16_to_f32(b.r_rowscale[l]);
    const float f = undo * a.row[row(v)].mean;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c][v] = fmaf(first == 0 ? -s : 0.0f, (float)((int32_t)(w << (28 - 4 * c)) >> 28), acc[c][v] * f);
  }
  const float* zrow = b.z + std::min<int64_t>(n0 + c32, count - 1) * r;
  for (int j0 = 16 * first; j0 < r; j0 += 16 * waves) {
    const bool in = j0 + 8 * half < r;  // ranks come in eights
    const int j = in ? j0 + 8 * half : j0;
    uint32_t code[8];
    float z[8], s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      code[k] = *reinterpret_cast<const uint32_t*>(b.b_codes + (int64_t)(j + k) * b.D + d);
      s[k] = f16_to_f32(b.b_scales[(int64_t)(j + k) * b.ng + group]);
      z[k] = zrow[j + k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = in ? z[k] : 0.0f;
    const Bf16Pair zp = split_bf16(z);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = s[k] * (float)(int8_t)(code[k] >> (8 * c));
      const Bf16Pair bp = split_bf16(x);
      acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zp.hi, bp.lo, acc[c], 0, 0, 0);
      acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zp.lo, bp.hi, acc[c], 0, 0, 0);
      acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zp.hi, bp.hi, acc[c], 0, 0, 0);
    }
  }
  if constexpr (kShare) {
    __shared__ f16x red[kWaves - 1][4][64];
    if (wave > 0)
#pragma unroll
      for (int c = 0; c < 4; ++c) red[wave - 1][c][lane] = acc[c];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] += red[w][c][lane];
  }
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int64_t i = n0 + 8 * (v >> 2) + 4 * half + (v & 3);
    if (i >= count) continue;
    const float f = a.row[i].all;
    typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
    *reinterpret_cast<u2_any*>(a.dH + (int64_t)a.map[a.pass * kChunkRows + i] * a.dh_stride + d) =
        pack_bf16x4(acc[0][v] * f, acc[1][v] * f, acc[2][v] * f, acc[3][v] * f);
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
  uint64_t y, fwd, fwd_bytes, piece, row, rscale, hf, gt, zpart, part, total;
};

XentLayout xent_layout(const archead_dims* d, int64_t rows) {
  XentLayout L{};
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


int check_xent_dims(const archead_dims* d) {
  if (int rc = check_kernel_dims(d)) return rc;
  if (int rc = check_archead_format(d)) return rc;
  if (d->V > kXentMaxVocab || d->r_c + d->r_r > kMaxRank) return ARCHEAD_E_UNSUPPORTED;
  return ARCHEAD_OK;
}

void set_head(const archead_packed_head* head, BwdArgs& b) {
  const archead_dims* d = &head->dims;
  archead_layout P;
  compute_layout(d, &P);
  const uint8_t* buf = static_cast<const uint8_t*>(head->buffer);
  b.V = d->V;
  b.D = d->D;
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
}

// log2(e) tau as a pair of fp32 numbers.  The first is the nearest one where
// that lies below, else the one before it, so that the second is above zero as
// well; at the ends of fp32's range both stay in it.
void set_exponent(float tau, float& hi, float& lo) {
  constexpr float kLeast = std::numeric_limits<float>::denorm_min(), kMost = std::numeric_limits<float>::max();
  const double c = 1.4426950408889634 * (double)tau;
  hi = (float)std::min(c, (double)kMost);
  if ((double)hi >= c) hi = nextafterf(hi, 0.0f);
  hi = std::max(hi, kLeast);
  lo = std::max((float)(c - (double)hi), kLeast);
}

int launch_few_rows(const archead_tensor* H, const archead_packed_head* head, const archead_cross_entropy_inputs* in,
                    const archead_cross_entropy_outputs* out, hipStream_t s) {
  const archead_dims* d = &head->dims;
  const int64_t rows = H->rows;
  const XentLayout L = xent_layout(d, rows);
  uint8_t* ws = static_cast<uint8_t*>(head->workspace);
  archead_tensor y{ws + L.y, rows, d->V, y_stride_of(d), ARCHEAD_F32};
  archead_packed_head p = *head;
  p.workspace = ws + L.fwd;
  p.workspace_bytes = L.fwd_bytes;
  if (int rc = archead_logits(H, &p, &y, s)) return rc;
  XentArgs a{};
  BwdArgs& b = a.b;
  set_head(head, b);
  b.N = rows;
  b.n32 = L.n32;
  b.rscale = reinterpret_cast<float*>(ws + L.rscale);
  b.hf = reinterpret_cast<_Float16*>(ws + L.hf);
  b.gt = ws + L.gt;
  b.zpart = reinterpret_cast<float*>(ws + L.zpart);
  b.part = reinterpret_cast<float*>(ws + L.part);
  b.zparts = b.splits = L.splits;
  b.ksteps = (int)L.ksteps;
  a.Y = reinterpret_cast<const float*>(ws + L.y);
  a.y_stride = y.row_stride;
  a.labels = in->labels;
  a.weight = in->weight;
  a.tau = in->inv_temperature;
  set_exponent(a.tau, a.c_hi, a.c_lo);
  a.logp = out->logp;
  if (out->dH) {
    a.dH = static_cast<uint16_t*>(out->dH->data);
    a.dh_stride = out->dH->row_stride;
  }
  a.piece = reinterpret_cast<Piece*>(ws + L.piece);
  a.row = reinterpret_cast<RowOut*>(ws + L.row);
  a.loss = out->loss;
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

// ---- many rows

struct ManyLayout {
  int64_t rows, n32, vtiles, piece;  // rows of a pass; 256-row tiles of the vocabulary, of a piece
  int zparts, passes;
  int64_t part_rows;
  uint64_t terms, head_max, scale, scale_a, map, label, plan, fwd, fwd_bytes, Hc, e, stat,
      alpha, ref, moved, sum, z_label, row, af, zpart, z, part, total;
};

// Workgroups of xent_z_kernel side by side for the ranks.
int z_groups(const archead_dims* d) { return (std::max(d->r_c, d->r_r) + 16 * kZTiles - 1) / (16 * kZTiles); }

// Steps of a row tile of a piece's operands: a few more than there are, as row
// tiles that are a power of two apart meet in the same memory channels.
int64_t piece_steps(int64_t vtiles) { return 16 * vtiles + 5; }

ManyLayout many_layout(const archead_dims* d, int64_t N) {
  ManyLayout L{};
  L.rows = std::min(N, kChunkRows);
  L.passes = (int)((N + kChunkRows - 1) / kChunkRows);
  L.n32 = (int64_t)round_up((uint64_t)L.rows, 32);
  L.vtiles = (d->V + 255) / 256;
  // whole rounds of 256 workgroups of 256 rows where there are several pieces
  const int64_t most = std::max<int64_t>(1, (int64_t)(kPieceBytes / ((uint64_t)L.n32 * 512)));
  const int64_t pieces = (L.vtiles + most - 1) / most;
  L.piece = (L.vtiles + pieces - 1) / pieces;
  if (pieces > 1) L.piece = std::min((int64_t)round_up((uint64_t)L.piece, 16), std::max<int64_t>(most / 16 * 16, 1));
  // partial sums: what all the rows take in as many parts as are best for them, or
  // 64 MiB for fewer rows in more parts
  const int64_t stages = 4 * L.piece;
  L.part_rows = std::max(L.rows * best_parts(L.rows, d->D, stages, main_tiles(L.rows), std::min<int64_t>(kMaxSplits, stages)),
                         std::min(L.rows * std::min<int64_t>(kMaxSplits, stages), (int64_t)(16 << 20) / d->D));
  const int64_t r = d->r_c + d->r_r, tiles = (d->r_c + 31) / 32 + (d->r_r + 31) / 32;
  const int64_t groups = (L.n32 + 63) / 64 * std::max(1, z_groups(d));
  L.zparts = (int)std::max<int64_t>(1, std::min<int64_t>({(256 + groups - 1) / groups, L.piece, 64}));
  auto take = [&](uint64_t bytes) {
    const uint64_t at = L.total;
    L.total += round_up(bytes, ARCHEAD_ALIGNMENT);
    return at;
  };
  const uint64_t n32 = (uint64_t)L.n32, blocks = 8 * (uint64_t)L.piece;
  L.terms = take((uint64_t)N * 8);
  L.head_max = take(kHeadParts * 12);
  L.scale = take(16);
  L.scale_a = take(2 * 256 * (uint64_t)L.vtiles * 2);
  L.map = take((uint64_t)N * 4);
  L.label = take((uint64_t)std::max(N, L.passes * L.rows) * 4);  // whole passes are read
  L.plan = take((uint64_t)L.passes * 16);
  L.fwd_bytes = workspace_layout(d, L.rows, false, 0, false).total;
  L.fwd = take(L.fwd_bytes);
  L.Hc = take(n32 * (uint64_t)d->D * 2);
  L.e = take(n32 / 32 * (uint64_t)piece_steps(L.piece) * 1024);
  L.stat = take(blocks * n32 * 8);
  L.alpha = take(n32 * 4);
  L.ref = take(n32 * 4);
  L.moved = take(n32 / kMergeRows * 4);
  L.sum = take(n32 * 8);
  L.z_label = take(n32 * 4);
  L.row = take(n32 * sizeof(RowOut));
  L.af = take((uint64_t)tiles * (uint64_t)L.vtiles * 16 * 512);
  L.zpart = take((uint64_t)L.zparts * n32 * (uint64_t)r * 4);
  L.z = take(n32 * (uint64_t)r * 4);
  L.part = take((uint64_t)L.part_rows * (uint64_t)d->D * 4);
  return L;
}

uint64_t xent_bytes(const archead_dims* d, int64_t N) {
  return N == 0 ? 0 : N <= kFewTokens ? xent_layout(d, N).total : many_layout(d, N).total;
}

template <int TT>
void launch_xent_main(const BwdArgs& b, const MainExp& ex, hipStream_t s) {
  const dim3 grid((unsigned)main_groups(b.N, b.D, TT)), block(kMainThreads);
  if (b.g == 32)
    hipLaunchKernelGGL((xent_main_kernel<TT, 4>), grid, block, 0, s, b, ex);
  else if (b.g == 64)
    hipLaunchKernelGGL((xent_main_kernel<TT, 2>), grid, block, 0, s, b, ex);
  else
    hipLaunchKernelGGL((xent_main_kernel<TT, 1>), grid, block, 0, s, b, ex);
}

int launch_many_rows(const archead_tensor* H, const archead_packed_head* head, const archead_cross_entropy_inputs* in,
                     const archead_cross_entropy_outputs* out, hipStream_t s) {
  const archead_dims* d = &head->dims;
  const int64_t N = H->rows;
  const ManyLayout L = many_layout(d, N);
  uint8_t* ws = static_cast<uint8_t*>(head->workspace);
  ManyArgs a{};
  set_head(head, a.b);
  BwdArgs& b = a.b;
  b.N = L.rows;
  b.n32 = L.n32;
  b.hf = reinterpret_cast<_Float16*>(ws + L.e);
  b.af = ws + L.af;
  b.zpart = reinterpret_cast<float*>(ws + L.zpart);
  b.z = reinterpret_cast<float*>(ws + L.z);
  b.part = reinterpret_cast<float*>(ws + L.part);
  b.zparts = L.zparts;
  a.rows = N;
  a.H = static_cast<const uint16_t*>(H->data);
  a.h_stride = H->row_stride;
  a.labels = in->labels;
  a.weight = in->weight;
  a.tau = in->inv_temperature;
  a.logp = out->logp;
  if (out->dH) {
    a.dH = static_cast<uint16_t*>(out->dH->data);
    a.dh_stride = out->dH->row_stride;
  }
  a.head_max = reinterpret_cast<float*>(ws + L.head_max);
  a.scale = reinterpret_cast<float*>(ws + L.scale);
  a.scale_a = reinterpret_cast<_Float16*>(ws + L.scale_a);
  a.map = reinterpret_cast<int32_t*>(ws + L.map);
  a.label = reinterpret_cast<int32_t*>(ws + L.label);
  a.plan = reinterpret_cast<int32_t*>(ws + L.plan);
  a.terms = reinterpret_cast<double*>(ws + L.terms);
  a.Hc = reinterpret_cast<uint16_t*>(ws + L.Hc);
  a.stat = reinterpret_cast<float*>(ws + L.stat);
  a.alpha = reinterpret_cast<float*>(ws + L.alpha);
  a.ref = reinterpret_cast<float*>(ws + L.ref);
  a.moved = reinterpret_cast<int32_t*>(ws + L.moved);
  a.part_rows = L.part_rows;
  a.sum = reinterpret_cast<double*>(ws + L.sum);
  a.z_label = reinterpret_cast<float*>(ws + L.z_label);
  a.steps = (int)piece_steps(L.piece);
  a.row = reinterpret_cast<RowOut*>(ws + L.row);
  a.asteps = 16 * L.vtiles;
  // the tile path's arguments, for the gathered rows
  archead_tensor h{a.Hc, L.rows, d->D, d->D, ARCHEAD_BF16};
  archead_packed_head p = *head;
  p.workspace = ws + L.fwd;
  p.workspace_bytes = L.fwd_bytes;
  FwdArgs f;
  if (int rc = tile_args(&h, &p, f)) return rc;
  const int tiles = b.nct + b.nwt;
  (void)hipGetLastError();  // start from a clean error state
  const int64_t arrange = a.dH ? (tiles * a.asteps * 16 + kHeadThreads - 1) / kHeadThreads : 0;
  // the launches that some number of rows that count may need (without weights it
  // is known): for each of 2, 4, 6 and 8 row tiles
  bool may[5] = {};
  a.row_tiles = d->D >= 256 && L.vtiles * ((L.n32 + 63) / 64) <= kSmall ? 2 : L.rows > kExpFewRows ? 8 : 0;
  if (a.row_tiles)
    may[a.row_tiles / 2] = true;
  else
    for (int64_t t = a.weight ? 1 : L.n32 / 32; t <= L.n32 / 32; ++t) may[exp_tiles(t, d->D >= 256) / 2] = true;
  a.passes = L.passes;
  a.main_steps = 16 * L.piece;
  b.ksteps = (int)a.asteps;
  hipLaunchKernelGGL(xent_head_kernel, dim3((unsigned)(1 + kHeadParts + arrange + (a.dH && a.weight ? N : 0))), dim3(kHeadThreads), 0, s, a, arrange);
  for (int pass = 0; pass < L.passes; ++pass) {
    a.pass = pass;
    hipLaunchKernelGGL(xent_gather_kernel, dim3((unsigned)(L.n32 + (pass == 0 ? (16 * a.asteps + 255) / 256 : 0))), dim3(256), 0, s, a);
    if (launch_prep(f, s) != hipSuccess) return ARCHEAD_E_HIP;
    for (int64_t vt = 0; vt < L.vtiles; vt += L.piece) {
      const int64_t vn = std::min(L.piece, L.vtiles - vt);
      T32Exp ex{};
      ex.plan = a.plan + 4 * pass;
      ex.ref = a.ref;
      ex.labels = a.label + pass * kChunkRows;
      ex.c = 1.4426950408889634 * (double)in->inv_temperature;
      ex.vt0 = (int)vt;
      ex.vtiles = (int)vn;
      ex.e = a.dH ? b.hf : nullptr;
      ex.steps = a.steps;
      ex.stat = a.stat;
      ex.z_label = a.z_label;
      for (int t = 1; t <= 4; ++t)
        if (may[t] && launch_tile_exp(f, ex, 2 * t, s) != hipSuccess) return ARCHEAD_E_HIP;
      a.blocks = (int)(8 * vn);
      a.first = vt == 0;
      a.step0 = (int)(16 * vt);
      b.ksteps = (int)(16 * vn);
      hipLaunchKernelGGL(xent_merge_kernel, dim3((unsigned)(L.n32 / kMergeRows)), dim3(kMergeRows * kMergeSlices), 0, s, a);
      if (!a.dH) continue;
      const int64_t row_tiles = L.n32 / 32;
      // (2048 workgroups where there are row tiles enough, and a block for every wave)
      hipLaunchKernelGGL(xent_move_kernel, dim3((unsigned)row_tiles, (unsigned)std::max<int64_t>(1, std::min((2048 + row_tiles - 1) / row_tiles, 2 * vn))),
                         dim3(64 * kMoveWaves), 0, s, a);
      if (tiles)
        hipLaunchKernelGGL(xent_z_kernel, dim3((unsigned)((L.n32 + 63) / 64), (unsigned)L.zparts, (unsigned)z_groups(d)),
                           dim3(kZThreads), 0, s, a);
      const MainExp me{a.plan + 4 * pass, a.alpha, a.scale, a.steps, a.first, (int)(4 * vt)};
      if (may[1]) launch_xent_main<2>(b, me, s);
      if (may[2]) launch_xent_main<4>(b, me, s);
      if (may[3]) launch_xent_main<6>(b, me, s);
      if (may[4]) launch_xent_main<8>(b, me, s);
    }
    hipLaunchKernelGGL(xent_rows_kernel, dim3((unsigned)L.rows), dim3(256), 0, s, a);
    if (a.dH) {
      // where tiles are few, four waves share one: 64, 500, 1000 and 2000 rows of 4096
      // columns take 14, 20, 34 and 49 us, with a wave each 26, 23, 27 and 39
      if (L.n32 / 32 * b.nkt < 1024)
        hipLaunchKernelGGL(xent_finish_kernel<true>, dim3((unsigned)(L.n32 / 32), (unsigned)b.nkt), dim3(kFinishThreads), 0, s, a);
      else
        hipLaunchKernelGGL(xent_finish_kernel<false>, dim3((unsigned)(L.n32 / 32), (unsigned)((b.nkt + 3) / 4)), dim3(kFinishThreads), 0, s, a);
    }
    if (hipGetLastError() != hipSuccess) return ARCHEAD_E_HIP;
  }
  return ARCHEAD_OK;
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
    if (N <= kFewTokens && !forward_takes(d, N)) return ARCHEAD_E_UNSUPPORTED;
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
  if (N > 0)
    if (int rc = N <= kFewTokens ? launch_few_rows(H, head, in, out, s) : launch_many_rows(H, head, in, out, s)) return rc;
  if (out->loss && (N == 0 || N > kFewTokens)) {
    hipLaunchKernelGGL(xent_total_kernel, dim3(1), dim3(kTotalThreads), 0, s, static_cast<const double*>(head->workspace), N, out->loss);
    if (hipGetLastError() != hipSuccess) return ARCHEAD_E_HIP;
  }
  return ARCHEAD_OK;
}

}  // extern "C"
