// The hidden states' gradient through the packed head,
//   dH[n, d] = sum_v dY[n, v] W_hat[v, d],  W_hat = R + A_c B_c + A_w B_w,
// for a head that stays as it is (archead_logits_backward).  With the stored
// codes, R[v, d] = s_R[v] (q4 c8)[v, d] and A[v, j] = s_A[v] code[v, j], so
//   dH = (dY s_R) (q4 c8) + Z_c B_c + Z_w B_w,  Z = (dY s_A) code:
// the row scales go to the gradient's side, and the integers q4 c8 (below
// 2048) and the INT8 codes are exact fp16 operands of the 32 x 32 x 16 MFMA.
// dY s is rounded to fp16 after scaling its row by a power of two that brings
// the row's largest product to [2^14, 2^15): 2^-11 of an element at most, an
// eighth of the half step of the bf16 result, and independent from one
// vocabulary entry to the next.  (A pair of fp16 numbers would keep 22 bits,
// for twice the MFMAs and fragments.)  The scale is taken from the products
// themselves, so a gradient that sits on vocabulary entries of tiny scales keeps its digits.
//
//   bwd_max_kernel     per row: the largest |dY s_R|, |dY s_Ac|, |dY s_Aw|;
//                      beside that, the A codes in operand order (few
//                      tokens: the group codes by k-tile)
//   bwd_prep_kernel    dY s_R as fp16 operand fragments; parts of Z
//   bwd_zsum_kernel    Z in fp32
//   bwd_main_kernel    the product with the packed residual, the vocabulary
//                      split over several workgroups where tiles are few
//   bwd_finish_kernel  the splits' sums and Z B to dH (many rows:
//                      bwd_finish_many_kernel)
// Up to 32 tokens: bwd_few_kernel or (up to 16) bwd_few16_kernel in place of
// zsum and main, and bwd_finish_few_kernel.
// The packed residual is never expanded in memory: a stage of 64 vocabulary
// rows (few tokens: 16) is unpacked to fp16 in LDS, and the MFMA's operand, which runs along
// the vocabulary, is read from there by transposing LDS reads.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace archead {

namespace {

constexpr int64_t kBwdChunkRows = 4096;  // rows of dY a pass takes
constexpr int kMaxThreads = 256;
constexpr int kMaxRows = 4;
constexpr int kPrepWaves = 4;       // and 32-rank tiles of Z that a workgroup forms
constexpr int kZsumThreads = 512, kZsumRanks = 64;
constexpr int kMainThreads = 512;
constexpr int kFinishThreads = 256;
constexpr int kFinishRows = 8;
constexpr int kMaxMaxPieces = 128;
constexpr int kXcds = 8;
constexpr int kMaxSplits = 64;
constexpr int64_t kFewTokens = 32;  // of bwd_few_kernel
// Where kOwnRounds rounds of loads reach all of dY, every workgroup of
// bwd_prep_kernel finds the rows' maxima itself: a call of 4 rows of a 1024 x
// 256 head takes 20 us, with a launch for them 24; sixteen rounds 25 and 24,
// 32 rounds 36 and 25.
constexpr int64_t kOwnRounds = 8;

// Lanes a row then: as many as there are, a wave at most.
__host__ __device__ constexpr int own_lanes(int64_t N) {
  int lanes = 64;
  while (lanes * N > 64 * kPrepWaves) lanes /= 2;
  return lanes;
}

struct BwdArgs {
  int64_t V, D, N, n32, nb;
  int r_c, r_r, g, ng, nkt, nA;
  int nct, nwt;                    // 32-rank tiles of the two parts
  const void* dY;
  int64_t dy_stride;
  uint16_t* dH;
  int64_t dh_stride;
  const uint8_t* r_codes;
  const uint8_t* r_gcodes;
  const uint16_t* r_rowscale;
  const int8_t* a_codes;
  const uint16_t* a_scales;
  const int8_t* b_codes;
  const uint16_t* b_scales;
  // workspace
  float* pmax;      // [N][3][pieces]
  float* rscale;    // [n32][3] powers of two that undo the rows' scales
  _Float16* hf;     // [n32/32][ksteps][64][8]; few tokens: [s_R, s_Ac, s_Aw][ksteps][2][N][8]
  uint8_t* af;      // A codes, [32-rank tiles][ksteps][64][8]
  uint8_t* gt;      // few tokens: group codes, [D / 128 or D / g][16 nb][128 / g or 1]
  float* zpart;     // [zparts][n32][r_c + r_r]
  float* z;         // [n32][r_c + r_r]; few tokens: not used, bwd_finish_few_kernel sums the parts
  float* part;      // [splits][N][D]
  int pieces, zparts, splits, ksteps;  // pieces 0: bwd_prep_kernel finds the maxima itself
  int64_t width;    // columns of a piece of bwd_max_kernel
};

typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements of a row as they are stored; a row may start at any element.
template <typename T>
struct Raw8 {
  u4 w[sizeof(T) / 2];
};
__device__ __forceinline__ uint32_t raw_bits(const uint16_t* p) { return *p; }
__device__ __forceinline__ uint32_t raw_bits(const float* p) { return __float_as_uint(*p); }
// Elements v .. v + 8 of a row, zeros from `end` on.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* row, int64_t v, int64_t end) {
  Raw8<T> x = {};
  if (v + 8 <= end) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h)
      x.w[h] = __builtin_nontemporal_load(reinterpret_cast<const u4_any*>(reinterpret_cast<const char*>(row + v) + 16 * h));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (v + j < end) {
        if constexpr (sizeof(T) == 2)
          x.w[0][j >> 1] |= raw_bits(row + v + j) << (16 * (j & 1));
        else
          x.w[j >> 2][j & 3] = raw_bits(row + v + j);
      }
  }
  return x;
}
__device__ __forceinline__ float at(const Raw8<uint16_t>& x, int j) {
  return __uint_as_float(j & 1 ? x.w[0][j >> 1] & 0xffff0000u : x.w[0][j >> 1] << 16);
}
__device__ __forceinline__ float at(const Raw8<float>& x, int j) { return __uint_as_float(x.w[j >> 2][j & 3]); }

// The fp16 scales of eight vocabulary rows (v a multiple of 8 below V16) as
// they are stored: s_R, and s_Ac, s_Aw of the parts that there are.
struct Scales8 {
  u4 R, A[2];
};
// (without a branch: a load behind one is waited for with all others in flight)
__device__ __forceinline__ Scales8 scales8(const BwdArgs& a, int64_t v) {
  Scales8 s;
  s.R = *reinterpret_cast<const u4*>(a.r_rowscale + v);
  const uint16_t* p = (a.nA ? a.a_scales : a.r_rowscale) + (a.nA == 2 ? 2 * v : v);
  s.A[0] = *reinterpret_cast<const u4*>(p);
  s.A[1] = *reinterpret_cast<const u4*>(p + (a.nA == 2 ? 8 : 0));
  return s;
}
__device__ __forceinline__ float scale_R(const Scales8& s, int j) {
  return f16_to_f32((uint16_t)(s.R[j >> 1] >> (16 * (j & 1))));
}
// s_Ac (part 0) or s_Aw (part 1); of a head with one part, that one's for both
__device__ __forceinline__ float scale_A(const Scales8& s, int nA, int part, int j) {
  return nA == 2 ? f16_to_f32((uint16_t)(s.A[j >> 2][j & 3] >> (16 * part)))
                 : f16_to_f32((uint16_t)(s.A[0][j >> 1] >> (16 * (j & 1))));
}

// The layout of the A codes: rank tile t, vocabulary step, lane (rank lane % 32,
// rows 16 step + 8 (lane / 32) .. + 8) hold the rows' 8 codes + 128.  Thread i
// takes four ranks: eight words of the stored rows, transposed byte by byte.
__device__ __forceinline__ void arrange_codes(const BwdArgs& a, int64_t i) {
  const int quad = (int)(i & 7), half = (int)(i >> 3) & 1;
  const int64_t step = (i >> 4) % a.ksteps, t = (i >> 4) / a.ksteps;
  if (t >= a.nct + a.nwt) return;
  const bool in_c = t < a.nct;
  const int j = 32 * (int)(in_c ? t : t - a.nct) + 4 * quad, r = a.r_c + a.r_r;
  const bool valid = j < (in_c ? a.r_c : a.r_r);  // ranks come in eights
  const int64_t v = 16 * step + 8 * half;
  const int8_t* codes = a.a_codes + v * r + (in_c ? 0 : a.r_c) + j;
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    w[k] = valid && v < 16 * a.nb ? *reinterpret_cast<const uint32_t*>(codes + (int64_t)k * r) : 0u;
  u2* out = reinterpret_cast<u2*>(a.af) + ((t * a.ksteps + step) * 64 + 32 * half + 4 * quad);
#pragma unroll
  for (int b = 0; b < 4; ++b) {  // byte b of the eight rows
    u2 x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sel = 0x0c0c0000u | (uint32_t)(4 + b) << 8 | (uint32_t)b;
      const uint32_t lo = __builtin_amdgcn_perm(w[4 * h + 1], w[4 * h], sel);
      const uint32_t hi = __builtin_amdgcn_perm(w[4 * h + 3], w[4 * h + 2], sel);
      x[h] = (lo | hi << 16) ^ 0x80808080u;
    }
    out[b] = x;
  }
}

// The group codes of 16 vocabulary rows by k-tile, for bwd_few_kernel: thread i
// takes those of one k-tile (or of the two that share a code of 256 columns).
// As they are stored, a k-tile's wave finds the 16 bytes that it needs in 16
// sectors, which took 11 us on one token of a 151936 x 4096 head; this, beside
// the maxima, takes 2.
template <typename C>
__device__ __forceinline__ void arrange_groups(const BwdArgs& a, int64_t i) {
  const int columns = a.ng / (int)sizeof(C);
  const int64_t kk = i % columns, b = i / columns;
  if (b >= a.nb) return;
  const C* src = reinterpret_cast<const C*>(a.r_gcodes) + 16 * b * columns + kk;
  C c[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) c[k] = src[k * columns];
  u4* out = reinterpret_cast<u4*>(a.gt) + (kk * a.nb + b) * (int64_t)sizeof(C);
#pragma unroll
  for (int k = 0; k < (int)sizeof(C); ++k) {
    u4 x;
    __builtin_memcpy(&x, c + k * 16 / sizeof(C), 16);
    out[k] = x;
  }
}

__device__ __forceinline__ void arrange_groups(const BwdArgs& a, int64_t i) {
  if (a.g == 32)
    arrange_groups<uint32_t>(a, i);
  else if (a.g == 64)
    arrange_groups<uint16_t>(a, i);
  else
    arrange_groups<uint8_t>(a, i);
}

// Eight of them as fp16: byte u under the byte 0x64 is 1024 + u, exactly.
__device__ __forceinline__ h8 unpack_u8x8(u2 c) {
  const h2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
  u4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = __builtin_amdgcn_perm(c[i >> 1], 0x64646464u, i & 1 ? 0x00070006u : 0x00050004u);
    x[i] = h2_bits(bits_h2(pair) - bias);
  }
  return __builtin_bit_cast(h8, x);
}

// Workgroup q pieces + p: the largest products of piece p of rows kMaxRows q
// .. + kMaxRows, which share the scales they are multiplied with.  The
// workgroups behind those lay the A codes out for bwd_prep_kernel, or the
// group codes for bwd_few_kernel, which the rows do not wait for.
template <typename T>
__global__ __launch_bounds__(kMaxThreads) void bwd_max_kernel(const BwdArgs a) {
  constexpr int kWaves = kMaxThreads / 64;
  __shared__ float buf[kWaves][kMaxRows][3];
  const int64_t groups = (a.N + kMaxRows - 1) / kMaxRows;
  if ((int64_t)blockIdx.x >= groups * a.pieces) {
    const int64_t i = ((int64_t)blockIdx.x - groups * a.pieces) * kMaxThreads + threadIdx.x;
    if (a.gt)
      arrange_groups(a, i);
    else
      arrange_codes(a, i);
    return;
  }
  const int64_t n0 = blockIdx.x / a.pieces * kMaxRows;
  const int p = (int)(blockIdx.x % a.pieces);
  const int64_t end = (p + 1) * a.width < a.V ? (p + 1) * a.width : a.V;
  float m[kMaxRows][3] = {};
  for (int64_t v = p * a.width + 8 * threadIdx.x; v < end; v += 8 * kMaxThreads) {
    Raw8<T> x[kMaxRows];
#pragma unroll
    for (int i = 0; i < kMaxRows; ++i)  // rows past the end: the last one again
      x[i] = load8(static_cast<const T*>(a.dY) + (n0 + i < a.N ? n0 + i : a.N - 1) * a.dy_stride, v, end);
    const Scales8 s = scales8(a, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float R = scale_R(s, j), c = scale_A(s, a.nA, 0, j), w = scale_A(s, a.nA, 1, j);
#pragma unroll
      for (int i = 0; i < kMaxRows; ++i) {
        const float y = at(x[i], j);
        m[i][0] = fmaxf(m[i][0], fabsf(y * R));
        m[i][1] = fmaxf(m[i][1], fabsf(y * c));
        m[i][2] = fmaxf(m[i][2], fabsf(y * w));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMaxRows; ++i)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      for (int o = 32; o > 0; o >>= 1) m[i][q] = fmaxf(m[i][q], __shfl_xor(m[i][q], o));
      if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6][i][q] = m[i][q];
    }
  __syncthreads();
  const int i = threadIdx.x / 3, q = threadIdx.x % 3;
  if (i < kMaxRows && n0 + i < a.N) {
    float t = buf[0][i][q];
    for (int w = 1; w < kWaves; ++w) t = fmaxf(t, buf[w][i][q]);
    a.pmax[((n0 + i) * 3 + q) * a.pieces + p] = t;
  }
}

// Grid (32-row tiles, parts of the vocabulary, groups of kPrepWaves rank
// tiles).  A run of 128 columns of the 32 rows is read as whole 256-byte
// pieces of rows (512 of fp32), multiplied with each of the three scales,
// rounded to fp16 and put in LDS in the MFMA operand's order (lane l: row
// l % 32, columns 16 step + 8 (l / 32) .. + 8).  From there dY s_R goes to
// memory, 1 KB a store, and wave w multiplies dY s_A of its rank tile with
// the codes that arrange_codes laid out; without kZ all three go to memory,
// for bwd_few_kernel, without the rows that there are not.  Of few columns
// (kOwn) its workgroups find the rows' maxima themselves, and others beside
// them lay the group codes out: a launch less.
// (4096 rows of 151936, 128 ranks: 0.57 ms, 4.4 TB/s of dY and the fragments,
// the vector ALUs busy 60% of the time.  Loads behind branches, which the
// compiler cannot count, took 0.62; three waves a SIMD instead of four the
// same, five and their spills 1.46.)
template <typename T, bool kZ, bool kOwn>
__global__ __launch_bounds__(64 * kPrepWaves, 4) void bwd_prep_kernel(const BwdArgs a) {
  __shared__ float sMax[3][32];
  __shared__ h8 frag[3][8][66];  // steps two octets apart, so that a wave's writes meet no bank twice
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if constexpr (kOwn) {
    if (blockIdx.x == 1) {
      for (int64_t i = (int64_t)blockIdx.y * 64 * kPrepWaves + tid; i < a.nb * a.ng; i += (int64_t)gridDim.y * 64 * kPrepWaves)
        arrange_groups(a, i);
      return;
    }
  }
  const int64_t tile = blockIdx.x;
  const int part = blockIdx.y;
  const bool first = blockIdx.z == 0;
  // this thread's rows and columns of a run: octet tid % 16 of rows tid / 16 and + 16
  const int oct = tid & 15;
  float P[2][3];
  const T* row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)  // past the last row: that one, whose results nobody reads
    row[i] = static_cast<const T*>(a.dY) + std::min<int64_t>(32 * tile + (tid >> 4) + 16 * i, a.N - 1) * a.dy_stride;
  const int64_t V16 = 16 * a.nb;
  const int r = a.r_c + a.r_r, tiles = a.nct + a.nwt;
  const int t = kZ ? kPrepWaves * (int)blockIdx.z + wave : tiles;  // this wave's rank tile
  const bool in_c = t < a.nct;
  const int runs = a.ksteps / 8;
  const int run0 = (int)((int64_t)part * runs / gridDim.y), run1 = (int)((int64_t)(part + 1) * runs / gridDim.y);
  // (waves without a rank tile load some other's: a load behind a branch would be waited for)
  const u2* codes = reinterpret_cast<const u2*>(tiles ? a.af : reinterpret_cast<uint8_t*>(a.hf)) +
                    (int64_t)(t < tiles ? t : 0) * a.ksteps * 64 + lane;
  f16x acc = {};
  // the next run's loads are in flight while this one is stored and multiplied
  Raw8<T> x[2] = {};
  Scales8 s;
  u2 b[8];
  auto load = [&](int run) {
    const int64_t v = 128 * (int64_t)run + 8 * oct;
    if (128 * (int64_t)(run + 1) <= a.V) {
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] = load8(row[i], v, v + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] = load8(row[i], v, a.V);
    }
    s = scales8(a, v < V16 ? v : V16 - 8);  // past V16 dY is zero
  };
  auto load_codes = [&](int run) {
    if constexpr (kZ) {
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = codes[(8 * run + k) * 64];
    }
  };
  if (run0 < run1) load(run0);
  if constexpr (kOwn) {
    const int lanes = own_lanes(a.N), rr = tid / lanes;
    float m[3] = {};
    if (rr < a.N) {
      const T* src = static_cast<const T*>(a.dY) + rr * a.dy_stride;
      for (int64_t v = 8 * (tid % lanes); v < a.V; v += 8 * lanes) {
        const Raw8<T> y8 = load8(src, v, a.V);
        const Scales8 s8 = scales8(a, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = at(y8, j);
          m[0] = fmaxf(m[0], fabsf(y * scale_R(s8, j)));
          m[1] = fmaxf(m[1], fabsf(y * scale_A(s8, a.nA, 0, j)));
          m[2] = fmaxf(m[2], fabsf(y * scale_A(s8, a.nA, 1, j)));
        }
      }
    }
    for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int q = 0; q < 3; ++q) m[q] = fmaxf(m[q], __shfl_xor(m[q], o));
    if (tid < 96) sMax[tid / 32][tid % 32] = 0.0f;
    __syncthreads();
    if (rr < a.N && tid % lanes == 0)
#pragma unroll
      for (int q = 0; q < 3; ++q) sMax[q][rr] = m[q];
  } else {
    // the tile's maxima from the pieces', eight lanes each
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int i = tid / 8 + 32 * k, rr = i / 3;
      float m = 0.0f;
      if (32 * tile + rr < a.N) {
        const float* src = a.pmax + (96 * tile + i) * a.pieces;
#pragma unroll 4
        for (int p = tid & 7; p < a.pieces; p += 8) m = fmaxf(m, src[p]);
      }
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
      if ((tid & 7) == 0) sMax[i % 3][rr] = m;
    }
  }
  __syncthreads();
  // at most 126: the power and its inverse are normal fp32
  auto exponent = [&](int q, int rr) { return std::min(row_exponent(sMax[q][rr]), 126); };
  if (tid < 96 && part == 0 && first)
    a.rscale[(32 * tile + tid % 32) * 3 + tid / 32] = ldexpf(1.0f, -exponent(tid / 32, tid % 32));
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 3; ++q) P[i][q] = ldexpf(1.0f, exponent(q, (tid >> 4) + 16 * i));
  auto all_runs = [&](auto store_) __attribute__((always_inline)) {
    for (int run = run0; run < run1; ++run) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h8 f[3];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // the product first, as the maximum was taken: times the power it is below 2^15,
          // also for a large y of an entry of scale 0; what the power adds is exact
          const float y = at(x[i], j);
          f[0][j] = (_Float16)(fmaf(y, scale_R(s, j), 0.0f) * P[i][0]);
          f[1][j] = (_Float16)(fmaf(y, scale_A(s, a.nA, 0, j), 0.0f) * P[i][1]);
          f[2][j] = (_Float16)(fmaf(y, scale_A(s, a.nA, 1, j), 0.0f) * P[i][2]);
        }
        const int at_ = 32 * (oct & 1) + (tid >> 4) + 16 * i;
#pragma unroll
        for (int q = 0; q < 3; ++q) frag[q][oct >> 1][at_] = f[q];
      }
      load_codes(run);
      load(std::min(run + 1, run1 - 1));
      __syncthreads();
      if constexpr (decltype(store_)::value) {
#pragma unroll
        for (int q = 0; q < (kZ ? 1 : 3); ++q)
#pragma unroll
          for (int i = 0; i < 8 / kPrepWaves; ++i) {
            const int k = wave + kPrepWaves * i;
            const int64_t step = (int64_t)q * a.ksteps + 8 * run + k;
            if (!kZ && c32 >= a.N) continue;
            h8* out = reinterpret_cast<h8*>(a.hf) + (kZ ? (tile * a.ksteps + step) * 64 + lane : (2 * step + half) * a.N + c32);
            *out = frag[q][k][lane];
          }
      }
      if (t < tiles) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          acc = mfma32(frag[in_c ? 1 : 2][k][lane], unpack_u8x8(b[k]), acc);
      }
      __syncthreads();
    }
  };
  if (first)
    all_runs(std::true_type{});
  else
    all_runs(std::false_type{});
  if (t >= tiles) return;
  const int j = 32 * (in_c ? t : t - a.nct) + c32;
  if (j >= (in_c ? a.r_c : a.r_r)) return;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int i = 8 * (v >> 2) + 4 * half + (v & 3);
    a.zpart[((int64_t)part * a.n32 + 32 * tile + i) * r + (in_c ? 0 : a.r_c) + j] = acc[v];
  }
}

// Row blockIdx.x of Z from its parts of the vocabulary, with the row's scales
// undone: kZsumRanks ranks at a time, the parts dealt to the threads of a rank
// and their sums added in order.
__global__ __launch_bounds__(kZsumThreads) void bwd_zsum_kernel(const BwdArgs a) {
  constexpr int kDeal = kZsumThreads / kZsumRanks;
  __shared__ float buf[kDeal][kZsumRanks];
  const int r = a.r_c + a.r_r, jj = threadIdx.x % kZsumRanks, deal = threadIdx.x / kZsumRanks;
  const int64_t n = blockIdx.x;
  for (int j0 = 0; j0 < r; j0 += kZsumRanks) {
    const int j = j0 + jj;
    float z = 0.0f;
    if (j < r) {
#pragma unroll 8
      for (int p = deal; p < a.zparts; p += kDeal) z += a.zpart[((int64_t)p * a.n32 + n) * r + j];
    }
    buf[deal][jj] = z;
    __syncthreads();
    if (deal == 0 && j < r) {
#pragma unroll
      for (int d = 1; d < kDeal; ++d) z += buf[d][jj];
      a.z[n * r + j] = z * a.rscale[n * 3 + (j < a.r_c ? 1 : 2)];
    }
    __syncthreads();
  }
}

// f(integral_constant<I>) for I = B .. E-1, unrolled at compile time
template <int B, int E, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

// Place of 16-byte octet o (8 columns) of row k in a stage's fp16 tile of 64
// rows x 256 columns: both the 16 rows that a wave writes at one octet and the
// 4 rows x 4 octets that 32 lanes read at a time fall in different banks.
__device__ __forceinline__ int tile_octet(int k, int o) {
  return 32 * k + (o ^ (((k & 3) << 2) | ((k >> 1) & 3)));
}

typedef short s4 __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
// Transposing read: of 16 lanes that point at 4 rows x 4 runs of 4 columns
// (lane q at row q / 4, run q % 4), lane i receives column i of the 4 rows.
__device__ __forceinline__ h4 read_tr(const _Float16* p) {
  return __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)p));
}

// 32 TT tokens x 256 columns of dH per workgroup over a share of the
// vocabulary, in stages of 64 vocabulary rows (4 MFMA steps).  The operands
// come from LDS, 6 KB a wave and step for eight MFMAs, and the fragments of dY
// and the unpacked tile are written there, 16 KB a step: 64% of the cycles
// that the MFMAs take, so the two run side by side.
// 4096 rows of 151936 x 4096: 4.1 ms, 1.25 PFLOP/s, MFMAs busy in 70% of the
// cycles of a clock that the power limit holds at 1.64 GHz; a dense bf16
// product of these sizes by the library, 3.6 to 4.1 ms.  (Four waves of 128 x
// 128 read a third less from LDS, but one wave a SIMD waits for itself: 2%
// slower.  Three workgroups' worth of registers do not exist at TT = 8.)
template <int TT>
struct MainShape {
  static constexpr int WM = TT >= 4 ? 2 : 1, WN = 8 / WM;  // eight waves in WM rows
  static constexpr int MT = TT / WM, NT = 8 / WN;          // 32 x 32 tiles of a wave
  static constexpr int kFrags = 4 * TT;                    // 1 KB dY fragments of a stage
  static constexpr int kLoads = kFrags / 8;                // of those, per wave
  static_assert(kFrags % 8 == 0, "TT must be even");
  static constexpr int kDepth = TT == 2 ? 4 : TT == 4 ? 2 : 1;  // stages whose loads are in flight
};

// kCodes: group codes of 128 columns of a row: 4 for g = 32, 2 for 64, else 1.
template <int TT, int kCodes>
__global__ __launch_bounds__(kMainThreads, TT >= 8 ? 2 : 4) void bwd_main_kernel(const BwdArgs a) {
  using S = MainShape<TT>;
  constexpr int kDepth = S::kDepth;
  __shared__ h8 sA[2][S::kFrags][64];
  __shared__ h8 sB[2][64 * 32];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int CB = (int)((a.D + 255) / 256), ntiles = (int)(a.n32 / 32), TB = (ntiles + TT - 1) / TT;
  // Workgroups are dealt to the XCDs round robin: each XCD gets a contiguous
  // range of (split, token block, column block), so that those in one L2 share
  // few streams of dY fragments, the larger of the two operands.
  const int per = gridDim.x / kXcds, rem = gridDim.x % kXcds, x = blockIdx.x % kXcds;
  const int item = x * per + std::min(x, rem) + blockIdx.x / kXcds;
  const int cb = item % CB, tb = item / CB % TB, split = item / CB / TB;
  const int stages = a.ksteps / 4;
  const int s0 = (int)((int64_t)split * stages / a.splits), s1 = (int)((int64_t)(split + 1) * stages / a.splits);

  // this wave's share of unpacking: one packed tile, 16 rows x 128 columns
  const int blk = wave & 3, kth = wave >> 2;
  const int kt = std::min(2 * cb + kth, a.nkt - 1);
  const uint8_t* wsrc = a.r_codes + (int64_t)kt * a.nb * 1024 + lane * 16;
  const uint8_t* csrc = a.r_gcodes + (lane & 15) * a.ng + kKTile * kt / a.g;
  u4 w[kDepth];
  uint32_t code[kDepth];
  h8 av[kDepth][S::kLoads];
  auto load = [&](int s, auto slot_) {
    constexpr int slot = decltype(slot_)::value;
    s = std::min(s, s1 - 1);  // past the end: a stage that is cached, never used
    const int64_t b = std::min<int64_t>(4 * (int64_t)s + blk, a.nb - 1);  // past the last rows dY is zero
    w[slot] = *reinterpret_cast<const u4*>(wsrc + b * 1024);
    const uint8_t* c = csrc + 16 * b * a.ng;
    code[slot] = kCodes == 4   ? *reinterpret_cast<const uint32_t*>(c)
                 : kCodes == 2 ? *reinterpret_cast<const uint16_t*>(c)
                               : *c;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int f = 8 * i + wave;
      const int64_t tile = std::min(tb * TT + f / 4, ntiles - 1);
      av[slot][i] = *reinterpret_cast<const h8*>(a.hf + ((tile * a.ksteps + 4 * s + f % 4) * 64 + lane) * 8);
    }
  };
  // columns 32 d .. + 32 of the packed tile in a register slot to the LDS tile
  auto unpack = [&](auto buf_, auto slot_, int d) {
    constexpr int buf = decltype(buf_)::value, slot = decltype(slot_)::value;
    const uint32_t c = kCodes == 4 ? (code[slot] >> (8 * d)) & 0xffu
                       : kCodes == 2 ? (code[slot] >> (8 * (d >> 1))) & 0xffu
                                     : code[slot];
    sB[buf][tile_octet(16 * blk + (lane & 15), 16 * kth + 4 * d + (lane >> 4))] =
        unpack_q4_scaled(w[slot][d], (_Float16)(float)c);
  };
  auto put_fragments = [&](auto buf_, auto slot_) {
    constexpr int buf = decltype(buf_)::value, slot = decltype(slot_)::value;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) sA[buf][8 * i + wave][lane] = av[slot][i];
  };

  f16x acc[S::MT][S::NT] = {};
  const int q = lane & 15, colhalf = (lane >> 4) & 1, khalf = lane >> 5;
  // operands of an MFMA step, fetched while the step before it runs
  h8 fa[2][S::MT], fb[2][S::NT];
  auto fetch = [&](auto buf_, auto t_) {
    constexpr int buf = decltype(buf_)::value, t = decltype(t_)::value, P = t & 1;
    const _Float16* B = reinterpret_cast<const _Float16*>(sB[buf]);
#pragma unroll
    for (int c = 0; c < S::NT; ++c) {
      const int ct = wn * S::NT + c;
      h4 x[2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int k = 16 * t + 8 * khalf + 4 * rr + q / 4;
        x[rr] = read_tr(B + 8 * tile_octet(k, 4 * ct + 2 * colhalf + (q & 3) / 2) + 4 * (q & 1));
      }
      fb[P][c] = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
#pragma unroll
    for (int m = 0; m < S::MT; ++m) fa[P][m] = sA[buf][4 * (wm * S::MT + m) + t][lane];
  };
  auto multiply = [&](auto t_) {
    constexpr int P = decltype(t_)::value & 1;
#pragma unroll
    for (int m = 0; m < S::MT; ++m)
#pragma unroll
      for (int c = 0; c < S::NT; ++c) acc[m][c] = mfma32(fa[P][m], fb[P][c], acc[m][c]);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  if (s0 < s1) {
    constexpr int kUnroll = kDepth < 2 ? 2 : kDepth;
    static_for<0, kDepth>([&](auto i) { load(s0 + decltype(i)::value, i); });
    for (int d = 0; d < 4; ++d) unpack(I0{}, I0{}, d);
    put_fragments(I0{}, I0{});
    load(s0 + kDepth, I0{});
    __syncthreads();
    fetch(I0{}, I0{});
    // A step's MFMAs, with what is around them dealt out between them: an LDS
    // read, a little arithmetic and an LDS write behind each.  (4096 rows of
    // 151936 x 4096: 2.5% of a call less than in the compiler's own order; with
    // two or five instructions 1.5%, with the LDS read first 2.5% more.)
    auto interleave = [] {
      static_for<0, S::MT * S::NT>([](auto) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);  // VALU
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // LDS write
      });
      __builtin_amdgcn_sched_barrier(0);
    };
    // One stage from LDS tile i & 1: each step's operands are fetched, and the
    // next stage unpacked to the other tile, while the step before multiplies;
    // its last step multiplies behind the barrier that opens the other tile.
    auto stage = [&](auto i_, int s) __attribute__((always_inline)) {
      constexpr int i = decltype(i_)::value;
      constexpr std::integral_constant<int, i & 1> buf{};
      constexpr std::integral_constant<int, (i + 1) & 1> other{};
      constexpr std::integral_constant<int, (i + 1) % kDepth> slot{};
      fetch(buf, I1{});
      unpack(other, slot, 0);
      unpack(other, slot, 1);
      multiply(I0{});
      interleave();
      fetch(buf, I2{});
      unpack(other, slot, 2);
      unpack(other, slot, 3);
      multiply(I1{});
      interleave();
      fetch(buf, I3{});
      put_fragments(other, slot);
      load(s + 1 + kDepth, slot);
      multiply(I2{});
      interleave();
      __syncthreads();
      fetch(other, I0{});
      multiply(I3{});
      interleave();
    };
    // whole rounds without an exit inside (an exit costs 2%), then the rest
    int g0 = s0;
    for (; g0 + kUnroll <= s1; g0 += kUnroll)
      static_for<0, kUnroll>([&](auto i) { stage(i, g0 + decltype(i)::value); });
    static_for<0, kUnroll - 1>([&](auto i) {
      if (g0 + decltype(i)::value < s1) stage(i, g0 + decltype(i)::value);
    });
  }
  // columns sit in the tile in the order the unpacking gives them
  const int c32 = lane & 31;
#pragma unroll
  for (int m = 0; m < S::MT; ++m)
#pragma unroll
    for (int c = 0; c < S::NT; ++c) {
      const int64_t d = 256 * (int64_t)cb + 32 * (wn * S::NT + c) + 8 * (c32 >> 3) + k_order_h(c32 & 7);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t n = 32 * (int64_t)(tb * TT + wm * S::MT + m) + 8 * (v >> 2) + 4 * khalf + (v & 3);
        if (n < a.N && d < a.D) a.part[((int64_t)split * a.N + n) * a.D + d] = acc[m][c][v];
      }
    }
}

constexpr int kFewWaves = kMainThreads / 64;

// 16-byte octets from a row of a wave's tile (128 columns) to the next: the four
// rows that 16 lanes read fall in different banks, and every address is one
// register and a constant, which tile_octet's are not.
constexpr int kFewPitch = 21;

// What the waves of bwd_few_kernel keep in LDS: a tile each, and at the end
// half of the waves' sums.
union FewShared {
  h8 tile[kFewWaves][16 * kFewPitch];
  float sum[kFewWaves / 2][4][16][64];
};

// The waves' sums of kCols result tiles added up in wave 0: the upper half of
// the waves to LDS, added by the lower half, three times.  Elements 4 i .. + 4
// of a result are rows 8 i .. + 8.
template <int kCols>
__device__ __forceinline__ void few_reduce(FewShared& sm, f16x (&acc)[kCols], int64_t N, int wave, int lane) {
#pragma unroll
  for (int half = kFewWaves / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (8 * i >= N) break;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int v = 4 * i; v < 4 * i + 4; ++v) sm.sum[wave - half][c][v][lane] = acc[c][v];
      }
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (8 * i >= N) break;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int v = 4 * i; v < 4 * i + 4; ++v) acc[c][v] += sm.sum[wave][c][v][lane];
      }
    }
  }
}

// A lane's place in a wave's tile, and the operand of an MFMA step of columns
// 32 c .. + 32 from there (rows along the step).
__device__ __forceinline__ const _Float16* few_operand(const h8* tile, int lane) {
  const int q = lane & 15, colhalf = (lane >> 4) & 1, khalf = lane >> 5;
  return reinterpret_cast<const _Float16*>(tile) + 8 * (kFewPitch * (8 * khalf + q / 4) + 2 * colhalf) + 4 * (q & 3);
}
__device__ __forceinline__ h8 few_read(const _Float16* at, int c) {
  return __builtin_shufflevector(read_tr(at + 32 * c), read_tr(at + 32 * c + 32 * kFewPitch), 0, 1, 2, 3, 4, 5, 6, 7);
}

// Rank tile t of Z over blocks [b0, b1) of 16 vocabulary rows.
__device__ __forceinline__ void few_ranks(const BwdArgs& a, FewShared& sm, int t, int split, int b0, int b1, int wave,
                                          int lane) {
  const bool in_c = t < a.nct;
  constexpr int kDepth = 8;
  const int part = in_c ? a.r_c : a.r_r, r = a.r_c + a.r_r, j0 = 32 * (in_c ? t : t - a.nct);
  const uint8_t* fsrc = reinterpret_cast<const uint8_t*>(a.hf) + (int64_t)(in_c ? 1 : 2) * a.ksteps * 32 * a.N;
  // lane: eight ranks (they come in eights; past the last ones those again) of row lane / 4
  const uint8_t* codes = reinterpret_cast<const uint8_t*>(a.a_codes) + (in_c ? 0 : a.r_c) + j0;
  const uint32_t at_code = (uint32_t)((lane >> 2) * r + std::min(8 * (lane & 3), part - j0 - 8));
  const uint32_t at_row = 16 * (uint32_t)((lane >> 5) * a.N + std::min<int64_t>(lane & 31, a.N - 1));
  f16x acc[1] = {};
  u2 c[kDepth];
  h8 f[kDepth];
  auto load = [&](int b, auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
    b = std::min(b, b1 - 1);
    c[slot] = *reinterpret_cast<const u2*>(codes + (int64_t)b * 16 * r + at_code);
    f[slot] = *reinterpret_cast<const h8*>(fsrc + (int64_t)b * 32 * a.N + at_row);
    __builtin_amdgcn_sched_barrier(0);
  };
  h8* put = sm.tile[wave] + kFewPitch * (lane >> 2) + (lane & 3);
  const _Float16* get = few_operand(sm.tile[wave], lane);
  auto use = [&](auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
    *put = unpack_i8x8(c[slot][0], c[slot][1]);
    __builtin_amdgcn_sched_barrier(0);
    acc[0] = mfma32(f[slot], few_read(get, 0), acc[0]);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (b0 + wave < b1) {  // as the ring of bwd_few_kernel
    static_for<0, kDepth>([&](auto i) { load(b0 + wave + kFewWaves * decltype(i)::value, i); });
    int g0 = b0 + wave;
    for (; g0 + kFewWaves * (kDepth - 1) < b1; g0 += kFewWaves * kDepth)
      static_for<0, kDepth>([&](auto i) {
        use(i);
        load(g0 + kFewWaves * (decltype(i)::value + kDepth), i);
      });
    static_for<0, kDepth - 1>([&](auto i) {
      if (g0 + kFewWaves * decltype(i)::value < b1) use(i);
    });
  }
  few_reduce(sm, acc, a.N, wave, lane);
  // ranks sit in the tile in the order the unpacking gives them
  const int c32 = lane & 31, j = j0 + 8 * (c32 >> 3) + (c32 & 4) + 2 * (c32 & 1) + (c32 >> 1 & 1);
  if (wave != 0 || j >= part) return;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int64_t n = 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
    if (n < a.N) a.zpart[((int64_t)split * a.n32 + n) * r + (in_c ? 0 : a.r_c) + j] = acc[0][v];
  }
}

// 17 to 32 tokens: one 128-column k-tile per workgroup over a share of the
// vocabulary, or one 32-rank tile of Z.  Each of the eight waves streams
// packed tiles of its own (16 vocabulary rows, one MFMA step) and the step's
// dY fragment, turns them in 4 KB of LDS that no other wave reads, and keeps
// the sums of all the tokens and columns; the waves' sums are added at the
// end.  A rank tile's codes are read as they are stored and turned the same way.
// 32 tokens of a 151936 x 4096 head: 84 us; the accumulators leave registers
// for four tiles in flight a wave, and none for operands that wait while the
// next tile is unpacked.  The group codes as stored cost 11 us more, a ring
// whose waits the compiler could not count 10 to 20.
template <int kCodes>
__global__ __launch_bounds__(kMainThreads, 4) void bwd_few_kernel(const BwdArgs a) {
  constexpr int kDepth = kCodes == 4 ? 3 : 4;  // without spills
  __shared__ __align__(16) FewShared sm;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = a.nkt + a.nct + a.nwt, kt = blockIdx.x % tiles, split = blockIdx.x / tiles, nb = (int)a.nb;
  const int b0 = (int)((int64_t)split * nb / a.splits), b1 = (int)((int64_t)(split + 1) * nb / a.splits);
  if (kt >= a.nkt) return few_ranks(a, sm, kt - a.nkt, split, b0, b1, wave, lane);
  // addresses: of the block (uniform), and the lane's place in it; lanes
  // without a token read the last one's row, and their sums are not used
  const uint8_t* wsrc = a.r_codes + (int64_t)kt * a.nb * 1024;
  const uint8_t* csrc = a.gt + (int64_t)(kCodes > 1 ? kt : kKTile * kt / a.g) * a.nb * 16 * kCodes;
  const uint32_t at_lane = (uint32_t)lane * 16, at_code = (uint32_t)(lane & 15) * kCodes;
  const uint32_t at_row = 16 * (uint32_t)((lane >> 5) * a.N + std::min<int64_t>(lane & 31, a.N - 1));
  const uint32_t f_step = 32 * (uint32_t)a.N;
  u4 w[kDepth];
  uint32_t code[kDepth];
  h8 f[kDepth];
  auto load = [&](int b, auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
    b = std::min(b, b1 - 1);  // past the end: a tile that is cached, never used
    w[slot] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(wsrc + (int64_t)b * 1024 + at_lane));
    const uint8_t* c = csrc + (int64_t)b * 16 * kCodes + at_code;
    code[slot] = kCodes == 4   ? *reinterpret_cast<const uint32_t*>(c)
                 : kCodes == 2 ? *reinterpret_cast<const uint16_t*>(c)
                               : *c;
    f[slot] = *reinterpret_cast<const h8*>(reinterpret_cast<const uint8_t*>(a.hf) + (int64_t)b * f_step + at_row);
  };
  f16x acc[4] = {};
  h8* put = sm.tile[wave] + kFewPitch * (lane & 15) + (lane >> 4);
  const _Float16* get = few_operand(sm.tile[wave], lane);
  auto use = [&](auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t c = kCodes == 4   ? (code[slot] >> (8 * d)) & 0xffu
                         : kCodes == 2 ? (code[slot] >> (8 * (d >> 1))) & 0xffu
                                       : code[slot];
      put[4 * d] = unpack_q4_scaled(w[slot][d], (_Float16)(float)c);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = mfma32(f[slot], few_read(get, c), acc[c]);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (b0 + wave < b1) {
    // Loads stay in the order of their use, and whole rounds have no exit
    // inside: the waits then count loads exactly, and the others stay in flight.
    static_for<0, kDepth>([&](auto i) {
      load(b0 + wave + kFewWaves * decltype(i)::value, i);
      __builtin_amdgcn_sched_barrier(0);
    });
    int g0 = b0 + wave;
    for (; g0 + kFewWaves * (kDepth - 1) < b1; g0 += kFewWaves * kDepth)
      static_for<0, kDepth>([&](auto i) {
        use(i);
        load(g0 + kFewWaves * (decltype(i)::value + kDepth), i);
        __builtin_amdgcn_sched_barrier(0);
      });
    static_for<0, kDepth - 1>([&](auto i) {
      if (g0 + kFewWaves * decltype(i)::value < b1) use(i);
    });
  }
  few_reduce(sm, acc, a.N, wave, lane);
  if (wave != 0) return;
  const int c32 = lane & 31, khalf = lane >> 5;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int64_t d = 128 * (int64_t)kt + 32 * c + 8 * (c32 >> 3) + k_order_h(c32 & 7);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t n = 8 * (v >> 2) + 4 * khalf + (v & 3);
      if (n < a.N) a.part[((int64_t)split * a.N + n) * a.D + d] = acc[c][v];
    }
  }
}

constexpr int kFew16Pitch = 9;  // octets a row of half a tile

// Up to 16 tokens: as bwd_few_kernel, on the 16 x 16 x 32 MFMA.  A step is two
// packed tiles, 32 vocabulary rows, turned in LDS one half of the columns at a
// time; the sums take half the registers, which go to a ring of six tiles a
// wave and to operands that are read ahead: while they come, the next half is
// unpacked over theirs (a wave's LDS accesses keep their order).  The
// workgroups of a k-tile take steps in turn, so that they read one part of
// memory together (1% over parts of their own).
// One token of a 151936 x 4096 head: 67 us, 4.9 TB/s of the packed bytes;
// bwd_few_kernel takes 77.  The packed tiles' loads alone take 51, all loads
// 58; 480 of 512 places hold k-tiles, as the ranks' tiles need some.  A ring
// of eight tiles takes the same.
template <int kCodes>
__global__ __launch_bounds__(kMainThreads, 4) void bwd_few16_kernel(const BwdArgs a) {
  constexpr int kDepth = 3;
  __shared__ __align__(16) FewShared sm;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = a.nkt + a.nct + a.nwt, kt = blockIdx.x % tiles, split = blockIdx.x / tiles, nb = (int)a.nb;
  if (kt >= a.nkt)
    return few_ranks(a, sm, kt - a.nkt, split, (int)((int64_t)split * nb / a.splits),
                     (int)((int64_t)(split + 1) * nb / a.splits), wave, lane);
  const int first = split * kFewWaves + wave, stride = kFewWaves * a.splits, end = (nb + 1) / 2;
  const uint8_t* wsrc = a.r_codes + (int64_t)kt * a.nb * 1024;
  const uint8_t* csrc = a.gt + (int64_t)(kCodes > 1 ? kt : kKTile * kt / a.g) * a.nb * 16 * kCodes;
  const uint32_t at_lane = (uint32_t)lane * 16, at_code = (uint32_t)(lane & 15) * kCodes;
  const uint32_t at_row = 16 * (uint32_t)((lane >> 4) * a.N + std::min<int64_t>(lane & 15, a.N - 1));
  const uint32_t f_step = 64 * (uint32_t)a.N;
  u4 w[kDepth][2];
  uint32_t code[kDepth][2];
  h8 f[kDepth];
  auto load = [&](int step, auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
    step = std::min(step, end - 1);  // past the end: tiles that are cached, never used
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int b = std::min(2 * step + j, nb - 1);  // past the last tile dY is zero
      w[slot][j] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(wsrc + (int64_t)b * 1024 + at_lane));
      const uint8_t* c = csrc + (int64_t)b * 16 * kCodes + at_code;
      code[slot][j] = kCodes == 4   ? *reinterpret_cast<const uint32_t*>(c)
                      : kCodes == 2 ? *reinterpret_cast<const uint16_t*>(c)
                                    : *c;
    }
    f[slot] = *reinterpret_cast<const h8*>(reinterpret_cast<const uint8_t*>(a.hf) + (int64_t)step * f_step + at_row);
    __builtin_amdgcn_sched_barrier(0);
  };
  h8* put = sm.tile[wave] + kFew16Pitch * (lane & 15) + (lane >> 4);
  auto unpack = [&](auto slot_, int half) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = 2 * half + e;
        const uint32_t c = kCodes == 4   ? (code[slot][j] >> (8 * d)) & 0xffu
                           : kCodes == 2 ? (code[slot][j] >> (8 * half)) & 0xffu
                                         : code[slot][j];
        put[16 * kFew16Pitch * j + 4 * e] = unpack_q4_scaled(w[slot][j][d], (_Float16)(float)c);
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  const int q = lane & 15;
  const _Float16* get = reinterpret_cast<const _Float16*>(sm.tile[wave]) +
                        8 * kFew16Pitch * (8 * (lane >> 4) + q / 4) + 4 * (q & 3);
  h8 x[4];
  auto fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      x[c] = __builtin_shufflevector(read_tr(get + 16 * c), read_tr(get + 16 * c + 32 * kFew16Pitch), 0, 1, 2, 3, 4, 5,
                                     6, 7);
    __builtin_amdgcn_sched_barrier(0);
  };
  f4 acc[8] = {};
  auto multiply = [&](auto slot_, int half) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      acc[4 * half + c] = mfma16(f[slot], x[c], acc[4 * half + c]);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (first < end) {
    // as in bwd_few_kernel: loads in the order of their use, rounds without an exit
    static_for<0, kDepth>([&](auto i) { load(first + stride * decltype(i)::value, i); });
    unpack(std::integral_constant<int, 0>{}, 0);
    fetch();
    auto step = [&](auto i) __attribute__((always_inline)) {
      unpack(i, 1);
      multiply(i, 0);
      fetch();
      unpack(std::integral_constant<int, (decltype(i)::value + 1) % kDepth>{}, 0);
      multiply(i, 1);
      fetch();
    };
    int g0 = first;
    for (; g0 + stride * (kDepth - 1) < end; g0 += stride * kDepth)
      static_for<0, kDepth>([&](auto i) __attribute__((always_inline)) {
        step(i);
        load(g0 + stride * (decltype(i)::value + kDepth), i);
      });
    static_for<0, kDepth - 1>([&](auto i) __attribute__((always_inline)) {
      if (g0 + stride * decltype(i)::value < end) step(i);
    });
  }
  // the waves' sums, halving the waves
#pragma unroll
  for (int half = kFewWaves / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) sm.sum[wave - half][c >> 2][4 * (c & 3) + v][lane] = acc[c][v];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[c][v] += sm.sum[wave][c >> 2][4 * (c & 3) + v][lane];
    }
  }
  if (wave != 0) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int64_t d = 128 * (int64_t)kt + 16 * c + (q & 8) + k_order_h(q & 7);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t n = 4 * (lane >> 4) + v;
      if (n < a.N) a.part[((int64_t)split * a.N + n) * a.D + d] = acc[c][v];
    }
  }
}

// Four columns of row n of dH.
__device__ __forceinline__ void write_dh(const BwdArgs& a, int64_t n, int64_t d, f4 y) {
  typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
  *reinterpret_cast<u2_any*>(a.dH + n * a.dh_stride + d) = pack_bf16x4(y[0], y[1], y[2], y[3]);
}

// Up to 32 tokens: one row x 256 columns of dH, four columns a lane; the waves
// take a quarter each of the splits and of the ranks.  Latency is all it
// takes: the sums of Z's parts (four lanes a rank), the splits' sums and the
// first ranks' B are loaded before any of them is waited for.  (One row of
// 4096, 15 parts, 64 ranks: 5.7 us; as bwd_finish_kernel does it 9.6.)
__global__ __launch_bounds__(kFinishThreads) void bwd_finish_few_kernel(const BwdArgs a) {
  constexpr int kWaves = kFinishThreads / 64, kParts = 8, kB = 16;
  extern __shared__ __align__(16) float sZ[];  // [r]
  __shared__ f4 red[kWaves][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = a.r_c + a.r_r;
  const int64_t n = blockIdx.x, d = 256 * (int64_t)blockIdx.y + 4 * lane, dd = d < a.D ? d : 0, group = dd / a.g;
  auto part = [&](int p) {  // past the last one: that one again
    return *reinterpret_cast<const f4*>(a.part + ((int64_t)std::min(p, a.splits - 1) * a.N + n) * a.D + dd);
  };
  f4 y[kParts];
#pragma unroll
  for (int k = 0; k < kParts; ++k) y[k] = part(wave + kWaves * k);
  uint32_t c[kB];
  uint16_t s[kB];
  auto load_b = [&](int j, int k) {
    j = std::min(j, r - 1);
    c[k] = *reinterpret_cast<const uint32_t*>(a.b_codes + (int64_t)j * a.D + dd);
    s[k] = a.b_scales[(int64_t)j * a.ng + group];
  };
  if (r > 0) {
#pragma unroll
    for (int k = 0; k < kB; ++k) load_b(wave + kWaves * k, k);
  }
  for (int e = tid; e < 4 * r; e += kFinishThreads) {  // r is a multiple of 8: whole groups of four lanes
    const int j = e >> 2;
    const float* src = a.zpart + n * r + j;
    float z = 0.0f;
    for (int p = e & 3; p < a.zparts; p += 4 * kParts) {
      float x[kParts];
#pragma unroll
      for (int k = 0; k < kParts; ++k) x[k] = src[(int64_t)std::min(p + 4 * k, a.zparts - 1) * a.n32 * r];
#pragma unroll
      for (int k = 0; k < kParts; ++k) z += p + 4 * k < a.zparts ? x[k] : 0.0f;
    }
    z += __shfl_xor(z, 1);
    z += __shfl_xor(z, 2);
    if ((e & 3) == 0) sZ[j] = z * a.rscale[n * 3 + (j < a.r_c ? 1 : 2)];
  }
  const float scale = a.rscale[n * 3];
  f4 acc = {};
  for (int p = wave; p < a.splits; p += kParts * kWaves) {
    if (p != wave) {
#pragma unroll
      for (int k = 0; k < kParts; ++k) y[k] = part(p + kWaves * k);
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      if (p + kWaves * k < a.splits) acc += y[k];
  }
  acc *= scale;
  __syncthreads();
  for (int j0 = wave; j0 < r; j0 += kB * kWaves) {
    if (j0 != wave) {
#pragma unroll
      for (int k = 0; k < kB; ++k) load_b(j0 + kWaves * k, k);
    }
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      const int j = j0 + kWaves * k;
      const float z = j < r ? sZ[j] * f16_to_f32(s[k]) : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(z, (float)(int8_t)(c[k] >> (8 * e)), acc[e]);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && d < a.D) {
    for (int w = 1; w < kWaves; ++w) acc += red[w][lane];
    write_dh(a, n, d, acc);
  }
}

// kFinishRows rows x 256 columns of dH, four columns a lane: the splits' sums
// and Z B, in fp32.  The four waves of a workgroup take a quarter each of the
// splits and of the ranks, and their sums are added in order.
__global__ __launch_bounds__(kFinishThreads) void bwd_finish_kernel(const BwdArgs a) {
  constexpr int kWaves = kFinishThreads / 64, kRows = kFinishRows;
  extern __shared__ __align__(16) float Z[];  // [r][kRows]
  __shared__ f4 red[kWaves][kRows][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = a.r_c + a.r_r;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  const int64_t d = 256 * (int64_t)blockIdx.y + 4 * lane;
  const int rows = (int)std::min<int64_t>(kRows, a.N - n0);
  for (int e = tid; e < kRows * r; e += kFinishThreads) {
    const int i = e / r, j = e % r;
    Z[j * kRows + i] = i < rows ? a.z[(n0 + i) * r + j] : 0.0f;
  }
  __syncthreads();
  f4 acc[kRows] = {};
  if (d < a.D) {
    for (int p = wave; p < a.splits; p += kWaves) {
      f4 y[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i)  // past the last row: that one again
        y[i] = *reinterpret_cast<const f4*>(a.part + ((int64_t)p * a.N + n0 + std::min(i, rows - 1)) * a.D + d);
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[i] += y[i];
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) acc[i] *= a.rscale[(n0 + std::min(i, rows - 1)) * 3];
    const int64_t group = d / a.g;
#pragma unroll 8
    for (int j = wave; j < r; j += kWaves) {
      const uint32_t c = *reinterpret_cast<const uint32_t*>(a.b_codes + (int64_t)j * a.D + d);
      const float s = f16_to_f32(a.b_scales[(int64_t)j * a.ng + group]);
      float b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = s * (float)(int8_t)(c >> (8 * e));
#pragma unroll
      for (int i = 0; i < kRows; i += 4) {
        const f4 z = *reinterpret_cast<const f4*>(Z + j * kRows + i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i + k][e] = fmaf(z[k], b[e], acc[i + k][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < rows; i += kWaves) {
    f4 y = red[0][i][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) y += red[w][i][lane];
    if (d < a.D) write_dh(a, n0 + i, d, y);
  }
}

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
// v as the sum of two bf16 numbers, to 2^-17 of it: v in [2^e, 2^(e+1)) leaves
// at most 2^(e-8) to lo, whose own half step is 2^(e-17) below that.
struct Bf16Pair {
  bf8 hi, lo;
};
__device__ __forceinline__ Bf16Pair split_bf16(const float (&v)[8]) {
  Bf16Pair p;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p.hi[i] = (__bf16)v[i];
    p.lo[i] = (__bf16)(v[i] - (float)p.hi[i]);
  }
  return p;
}

// Many rows: 32 rows x 128 columns of dH a wave, Z B on the bf16 MFMA with Z
// and B as pairs of bf16 numbers (three products; bf16 has fp32's range, so
// neither needs a scale).  What the pairs and the fourth product, of two lo's,
// leave out is 2^-17 + 2^-17 + 2^-16 = 2^-15 of |Z| |B| at most, a sixteenth of
// what Z has from dY's fp16.  Tile c of four holds the columns 4 i + c, so that
// a lane has four neighbouring ones of a row: whole lines of the parts, of B
// and of dH.  (4096 rows of 4096 columns, 128 ranks: 47 us, and 107 with fp32
// products; 256 rows of 8192 columns, 8 parts: 22 and 25.)
__global__ __launch_bounds__(kFinishThreads, 2) void bwd_finish_many_kernel(const BwdArgs a) {
  constexpr int kWaves = kFinishThreads / 64;
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = a.r_c + a.r_r;
  const int64_t n0 = 32 * (int64_t)blockIdx.x, d0 = kKTile * ((int64_t)blockIdx.y * kWaves + wave);
  if (d0 >= a.D) return;
  const int64_t d = d0 + 4 * c32, group = d / a.g;
  // row of element v of a result tile; past the last row that one
  auto row = [&](int v) { return std::min<int64_t>(n0 + 8 * (v >> 2) + 4 * half + (v & 3), a.N - 1); };
  f16x acc[4] = {};
  for (int p = 0; p < a.splits; ++p) {
    f4 y[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) y[v] = *reinterpret_cast<const f4*>(a.part + ((int64_t)p * a.N + row(v)) * a.D + d);
#pragma unroll
    for (int v = 0; v < 16; ++v)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c][v] += y[v][c];
  }
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const float s = a.rscale[row(v) * 3];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c][v] *= s;
  }
  const float* zrow = a.z + std::min<int64_t>(n0 + c32, a.N - 1) * r;
  for (int j0 = 0; j0 < r; j0 += 16) {
    const bool in = j0 + 8 * half < r;  // ranks come in eights
    const int j = in ? j0 + 8 * half : j0;
    uint32_t code[8];
    float z[8], s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      code[k] = *reinterpret_cast<const uint32_t*>(a.b_codes + (int64_t)(j + k) * a.D + d);
      s[k] = f16_to_f32(a.b_scales[(int64_t)(j + k) * a.ng + group]);
      z[k] = zrow[j + k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = in ? z[k] : 0.0f;
    const Bf16Pair zp = split_bf16(z);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = s[k] * (float)(int8_t)(code[k] >> (8 * c));
      const Bf16Pair bp = split_bf16(b);
      acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zp.hi, bp.lo, acc[c], 0, 0, 0);
      acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zp.lo, bp.hi, acc[c], 0, 0, 0);
      acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zp.hi, bp.hi, acc[c], 0, 0, 0);
    }
  }
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int64_t n = n0 + 8 * (v >> 2) + 4 * half + (v & 3);
    if (n < a.N) write_dh(a, n, d, f4{acc[0][v], acc[1][v], acc[2][v], acc[3][v]});
  }
}

// ------------------------------------------------------------------- host ---

int main_tiles(int64_t N) { return N <= 64 ? 2 : N <= 128 ? 4 : 8; }

// Parts of the vocabulary for the main kernel: the count that a model of its
// time likes best, workgroups in rounds of the resident ones (two a CU for
// 64-token tiles, else one) of kRoundUs plus a stage's measured
// time for every stage, and the partial sums written and read at 4 TB/s.
int main_splits(int64_t N, int64_t D, int64_t ranks, int64_t stages) {
  constexpr double kRoundUs = 4.0;
  if (N <= kFewTokens)  // two workgroups a CU; a packed tile for each wave at least
    return (int)std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, 512 / (D / kKTile + ranks), (stages + 1) / 2}));
  const int tt = main_tiles(N);
  const int64_t tiles = (N + 32 * tt - 1) / (32 * tt) * ((D + 255) / 256), slots = tt == 2 ? 512 : 256;
  const double stage_us = tt == 8 ? 1.75 : tt == 4 ? 1.15 : 1.4;
  double best = 1e30;
  int pick = 1;
  for (int64_t p = 1; p <= std::min<int64_t>(kMaxSplits, stages); ++p) {
    const double us = (double)((tiles * p + slots - 1) / slots) * (kRoundUs + stage_us * (double)((stages + p - 1) / p)) +
                      (double)(p * N * D) * 8.0 / 4e6;
    if (us < best) {
      best = us;
      pick = (int)p;
    }
  }
  return pick;
}

struct BwdLayout {
  int64_t rows, n32, ksteps, width;
  int pieces, zparts, splits;
  uint64_t pmax, rscale, hf, af, gt, zpart, z, part, total;
};

BwdLayout bwd_layout(const archead_dims* d, int64_t n_tokens) {
  BwdLayout L{};
  L.rows = std::min(n_tokens, kBwdChunkRows);
  if (L.rows <= 0) return L;
  const int64_t V128 = (int64_t)round_up((uint64_t)d->V, 128), r = d->r_c + d->r_r;
  L.n32 = (int64_t)round_up((uint64_t)L.rows, 32);
  L.ksteps = V128 / 16;  // whole runs of bwd_prep_kernel
  L.pieces = (int)std::max<int64_t>(
      1, std::min<int64_t>({(int64_t)kMaxMaxPieces, (d->V + 2047) / 2048, 2048 * kMaxRows / L.rows}));
  if (L.rows <= kFewTokens && d->V <= 8 * kOwnRounds * own_lanes(L.rows)) L.pieces = 0;
  L.width = L.pieces == 0 ? 0 : (int64_t)round_up((uint64_t)((d->V + L.pieces - 1) / L.pieces), 8);
  L.splits = main_splits(L.rows, d->D, (d->r_c + 31) / 32 + (d->r_r + 31) / 32, L.ksteps / 4);
  L.zparts = L.rows <= kFewTokens
                 ? L.splits
                 : (int)std::max<int64_t>(1, std::min<int64_t>({256, L.ksteps / 8, 1024 * 32 / L.n32}));
  auto take = [&](uint64_t bytes) {
    const uint64_t at = L.total;
    L.total += round_up(bytes, ARCHEAD_ALIGNMENT);
    return at;
  };
  L.pmax = take((uint64_t)L.rows * L.pieces * 12);
  L.rscale = take((uint64_t)L.n32 * 12);
  const bool few = L.rows <= kFewTokens;
  L.hf = take((uint64_t)V128 * 2 * (few ? 3 * L.rows : L.n32));
  L.af = take(few ? 0 : (uint64_t)((d->r_c + 31) / 32 + (d->r_r + 31) / 32) * L.ksteps * 512);
  L.gt = take(few ? round_up((uint64_t)d->V, 16) * (uint64_t)(d->D / d->g) : 0);
  L.zpart = take((uint64_t)L.zparts * L.n32 * r * 4);
  L.z = take((uint64_t)L.n32 * r * 4);
  L.part = take((uint64_t)L.splits * L.rows * d->D * 4);
  return L;
}

// Workspace of a call: of its chunks of kBwdChunkRows rows, or of the last, smaller one.
uint64_t bwd_bytes(const archead_dims* d, int64_t n_tokens) {
  return std::max(bwd_layout(d, n_tokens).total, bwd_layout(d, n_tokens % kBwdChunkRows).total);
}

template <int TT>
void launch_main_tt(const BwdArgs& a, hipStream_t s) {
  const int64_t tb = (a.n32 / 32 + TT - 1) / TT, cb = (a.D + 255) / 256;
  const dim3 grid((unsigned)(tb * cb * a.splits)), block(kMainThreads);
  if (a.g == 32)
    hipLaunchKernelGGL((bwd_main_kernel<TT, 4>), grid, block, 0, s, a);
  else if (a.g == 64)
    hipLaunchKernelGGL((bwd_main_kernel<TT, 2>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((bwd_main_kernel<TT, 1>), grid, block, 0, s, a);
}

template <int kCodes>
void launch_few_codes(const BwdArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.nkt + a.nct + a.nwt) * a.splits)), block(kMainThreads);
  if (a.N <= 16)  // tokens of its operands
    hipLaunchKernelGGL(bwd_few16_kernel<kCodes>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(bwd_few_kernel<kCodes>, grid, block, 0, s, a);
}

void launch_few(const BwdArgs& a, hipStream_t s) {
  if (a.g == 32)
    launch_few_codes<4>(a, s);
  else if (a.g == 64)
    launch_few_codes<2>(a, s);
  else
    launch_few_codes<1>(a, s);
}

template <typename T>
hipError_t launch_backward(const BwdArgs& a, hipStream_t s) {
  const int64_t ranks = a.nct + a.nwt, max_groups = (a.N + kMaxRows - 1) / kMaxRows * a.pieces;
  const int64_t arrange = a.gt ? a.nb * a.ng / std::max(1, kKTile / a.g) : ranks * a.ksteps * 16;  // threads
  if (a.pieces > 0)
    hipLaunchKernelGGL(bwd_max_kernel<T>, dim3((unsigned)(max_groups + (arrange + kMaxThreads - 1) / kMaxThreads)),
                     dim3(kMaxThreads), 0, s, a);
  const int tt = main_tiles(a.N);
  if (a.N <= kFewTokens) {
    const unsigned runs = (unsigned)(a.ksteps / 8);
    if (a.pieces > 0)
      hipLaunchKernelGGL((bwd_prep_kernel<T, false, false>), dim3(1, std::min(runs, 1024u)), dim3(64 * kPrepWaves), 0, s, a);
    else
      hipLaunchKernelGGL((bwd_prep_kernel<T, false, true>), dim3(2, runs), dim3(64 * kPrepWaves), 0, s, a);
    launch_few(a, s);
  } else {
    hipLaunchKernelGGL((bwd_prep_kernel<T, true, false>),
                       dim3((unsigned)(a.n32 / 32), (unsigned)a.zparts, (unsigned)std::max<int64_t>(1, (ranks + kPrepWaves - 1) / kPrepWaves)),
                       dim3(64 * kPrepWaves), 0, s, a);
    if (ranks > 0) hipLaunchKernelGGL(bwd_zsum_kernel, dim3((unsigned)a.N), dim3(kZsumThreads), 0, s, a);
    if (tt == 2)
      launch_main_tt<2>(a, s);
    else if (tt == 4)
      launch_main_tt<4>(a, s);
    else
      launch_main_tt<8>(a, s);
  }
  const size_t lds = (size_t)(a.r_c + a.r_r) * 4;
  const unsigned columns = (unsigned)((a.D + 255) / 256), waves = kFinishThreads / 64;
  // bwd_finish_many_kernel where its tiles give every CU two waves: with fewer, one wave
  // for all parts of a tile is the longer way
  if (a.N <= kFewTokens)
    hipLaunchKernelGGL(bwd_finish_few_kernel, dim3((unsigned)a.N, columns), dim3(kFinishThreads), lds, s, a);
  else if (a.n32 / 32 * a.nkt < 512)
    hipLaunchKernelGGL(bwd_finish_kernel, dim3((unsigned)((a.N + kFinishRows - 1) / kFinishRows), columns),
                       dim3(kFinishThreads), lds * kFinishRows, s, a);
  else
    hipLaunchKernelGGL(bwd_finish_many_kernel, dim3((unsigned)(a.n32 / 32), (unsigned)((a.nkt + waves - 1) / waves)),
                       dim3(kFinishThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace archead

using namespace archead;

extern "C" {

int archead_logits_backward_workspace_bytes(const archead_dims* d, int64_t n_tokens, uint64_t* bytes) {
  if (!d || !bytes) return ARCHEAD_E_NULL;
  if (int rc = check_dims(d)) return rc;
  if (int rc = check_archead_format(d)) return rc;
  if (n_tokens < 0) return ARCHEAD_E_SHAPE;
  *bytes = bwd_bytes(d, n_tokens);
  return ARCHEAD_OK;
}

int archead_logits_backward(const archead_tensor* dY, const archead_packed_head* head, archead_tensor* dH,
                            void* stream) {
  if (!dY || !head || !dH) return ARCHEAD_E_NULL;
  const archead_dims* d = &head->dims;
  if (int rc = check_kernel_dims(d)) return rc;
  if (int rc = check_archead_format(d)) return rc;
  if ((dY->dtype != ARCHEAD_BF16 && dY->dtype != ARCHEAD_F32) || dH->dtype != ARCHEAD_BF16) return ARCHEAD_E_DTYPE;
  const int64_t N = dY->rows;
  if (N < 0 || dY->cols != d->V || dY->row_stride < d->V) return ARCHEAD_E_SHAPE;
  if (dH->rows != N || dH->cols != d->D || dH->row_stride < d->D) return ARCHEAD_E_SHAPE;
  // 32-bit row, fragment and work-item counts; Z of kFinishRows rows in LDS
  if (N > (int64_t(1) << 22) || d->V > (int64_t(1) << 26) || d->r_c + d->r_r > kMaxRank) return ARCHEAD_E_UNSUPPORTED;
  if (N == 0) return ARCHEAD_OK;
  if (!dY->data || !dH->data || !head->buffer || !head->workspace) return ARCHEAD_E_NULL;
  const int size = dY->dtype == ARCHEAD_F32 ? 4 : 2;
  if ((uintptr_t)dY->data % size || (uintptr_t)dH->data % 2) return ARCHEAD_E_ALIGN;
  if (overlap(dY, size, dH, 2)) return ARCHEAD_E_SHAPE;  // later rows are read after earlier ones are written
  if ((uintptr_t)head->buffer % ARCHEAD_ALIGNMENT || (uintptr_t)head->workspace % ARCHEAD_ALIGNMENT)
    return ARCHEAD_E_ALIGN;
  archead_layout P;
  compute_layout(d, &P);
  if (head->buffer_bytes < P.total_bytes) return ARCHEAD_E_SIZE;
  if (head->workspace_bytes < bwd_bytes(d, N)) return ARCHEAD_E_WORKSPACE;
  const uint8_t* buf = static_cast<const uint8_t*>(head->buffer);
  uint8_t* ws = static_cast<uint8_t*>(head->workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // start from a clean error state
  for (int64_t n0 = 0; n0 < N; n0 += kBwdChunkRows) {
    const BwdLayout L = bwd_layout(d, std::min(kBwdChunkRows, N - n0));
    BwdArgs a{};
    a.V = d->V;
    a.D = d->D;
    a.N = L.rows;
    a.n32 = L.n32;
    a.nb = P.padded_rows / 16;
    a.r_c = d->r_c;
    a.r_r = d->r_r;
    a.g = d->g;
    a.ng = (int)(d->D / d->g);
    a.nkt = (int)(d->D / kKTile);
    a.nA = (d->r_c > 0) + (d->r_r > 0);
    a.nct = (d->r_c + 31) / 32;
    a.nwt = (d->r_r + 31) / 32;
    a.dY = static_cast<const uint8_t*>(dY->data) + (uint64_t)n0 * (uint64_t)dY->row_stride * size;
    a.dy_stride = dY->row_stride;
    a.dH = static_cast<uint16_t*>(dH->data) + n0 * dH->row_stride;
    a.dh_stride = dH->row_stride;
    a.r_codes = buf + P.r_codes.offset;
    a.r_gcodes = buf + P.r_gcodes.offset;
    a.r_rowscale = reinterpret_cast<const uint16_t*>(buf + P.r_rowscale.offset);
    a.a_codes = reinterpret_cast<const int8_t*>(buf + P.a_codes.offset);
    a.a_scales = reinterpret_cast<const uint16_t*>(buf + P.a_scales.offset);
    a.b_codes = reinterpret_cast<const int8_t*>(buf + P.b_codes.offset);
    a.b_scales = reinterpret_cast<const uint16_t*>(buf + P.b_scales.offset);
    a.pmax = reinterpret_cast<float*>(ws + L.pmax);
    a.rscale = reinterpret_cast<float*>(ws + L.rscale);
    a.hf = reinterpret_cast<_Float16*>(ws + L.hf);
    a.af = ws + L.af;
    a.gt = L.rows <= kFewTokens ? ws + L.gt : nullptr;
    a.zpart = reinterpret_cast<float*>(ws + L.zpart);
    a.z = L.rows <= kFewTokens ? nullptr : reinterpret_cast<float*>(ws + L.z);
    a.part = reinterpret_cast<float*>(ws + L.part);
    a.pieces = L.pieces;
    a.zparts = L.zparts;
    a.splits = L.splits;
    a.ksteps = (int)L.ksteps;
    a.width = L.width;
    const hipError_t e = size == 4 ? launch_backward<float>(a, s) : launch_backward<uint16_t>(a, s);
    if (e != hipSuccess) return ARCHEAD_E_HIP;
  }
  return ARCHEAD_OK;
}

}  // extern "C"
