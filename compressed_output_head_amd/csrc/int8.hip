// Logits of INT8 hidden states through a row-INT8 head (archead_logits_int8):
//   Y[n, v] = (sum_k X[n, k] q8[v, k]) s[v] scale[n],
// on the 8-bit integer MFMA: products and sums are exact (|sum| <= 2^14 D, D
// up to 65536), and only the scales round: the row's first, as a sum times an fp16
// number stays within 2^-24 and 2^46, where two scales alone may leave fp32.
//
// The head is stored for fp16 operands (tile (b, kt), lane l: row l % 16,
// columns 32 s + 8 (l / 16) + P[p], byte 8 s + p).  A sum may take its terms in
// any order, so the codes are used as they lie, and X is brought to their
// order: P swaps the middle pairs of every eight columns.
//
//   i8_few_kernel      up to 8 tokens: streams the head once
//   i8_arrange_kernel  X in operand order
//   i8_tile_kernel     32 TT tokens x 32 WN WCB rows of the vocabulary a workgroup
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace archead {

namespace {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i16x __attribute__((ext_vector_type(16)));

constexpr int64_t kI8ChunkRows = 16384;  // rows of X whose operands the workspace holds
constexpr int64_t kI8MaxCols = 65536;    // 2^14 D below 2^30
constexpr int64_t kI8MaxRows = int64_t(1) << 22;
constexpr int kI8Tile = 2048;            // bytes of a tile of 16 rows x 128 columns
constexpr uint32_t kFewLds = 128 * 1024;
constexpr int kXcds = 8;

struct I8Args {
  int64_t V, D, N, nb;
  int nkt, ntiles;          // 128-column tiles; 32-token tiles
  const int8_t* X;
  int64_t x_stride;
  const float* scale;
  const uint8_t* codes;
  const uint16_t* rowscale;
  u4* xf;                   // [ntiles][nkt][4][64] operands
  void* Y;
  int64_t y_stride;
  int y_bf16;
};

__device__ __forceinline__ i4 as_i4(u4 x) { return __builtin_bit_cast(i4, x); }

// Eight columns in the order of the stored codes: 0 1 4 5 2 3 6 7.
__device__ __forceinline__ u2 code_order(u2 x) {
  return u2{__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[1], x[0], 0x07060302u)};
}
// The operand bytes of a token's row at tile kt, of steps 2 h and 2 h + 1 and run q.
__device__ __forceinline__ u4 operand(const int8_t* row, int kt, int q, int h) {
  const u2 lo = code_order(*reinterpret_cast<const u2*>(row + 128 * kt + 64 * h + 8 * q));
  const u2 hi = code_order(*reinterpret_cast<const u2*>(row + 128 * kt + 64 * h + 32 + 8 * q));
  return u4{lo[0], lo[1], hi[0], hi[1]};
}

__device__ __forceinline__ void put(const I8Args& a, int64_t n, int64_t v, float y) {
  if (a.y_bf16)
    static_cast<uint16_t*>(a.Y)[n * a.y_stride + v] = f32_to_bf16(y);
  else
    static_cast<float*>(a.Y)[n * a.y_stride + v] = y;
}

// Few tokens: bound by the head's bytes, 622 MB of a 151936 x 4096 head in 106
// us, 5.9 TB/s (the 16 columns of an MFMA cost nothing beside that, and one
// workgroup of 16 waves a CU reads as fast as two of eight).  The tokens'
// operands come from LDS for every 16 rows: 1, 8 and 16 tokens take 108, 116
// and 130 us, in a tile of 64 tokens, whose waves take 32 rows, 115, 119 and 122.
// So up to 8, where they fit LDS.  Every wave takes blocks of 16 rows of the vocabulary, a
// grid's waves apart, over all columns, with kRing packed tiles in flight
// across the blocks' borders; X in operand order in LDS (tile, step pair h, run
// q, token).  Tiles past the last column meet operands of zero.
constexpr int kFewTokens = 8;
constexpr int kFewThreads = 1024;
constexpr int kRing = 4;
__global__ __launch_bounds__(kFewThreads, 4) void i8_few_kernel(const I8Args a) {
  extern __shared__ __align__(16) u4 sX[];  // [nkt rounded up to kRing][2][4][N]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = (int)a.N, groups = (a.nkt + kRing - 1) / kRing;
  const int64_t first = (int64_t)wave * gridDim.x + blockIdx.x, waves = (int64_t)gridDim.x * (kFewThreads / 64);
  const uint8_t* const src = a.codes + 32 * lane;
  const int64_t tstride = a.nb * kI8Tile;
  u4 w[kRing][2];
  auto load = [&](int64_t b, int kt, auto i_) __attribute__((always_inline)) {
    constexpr int i = decltype(i_)::value;
    const uint8_t* p = src + b * kI8Tile + std::min(kt, a.nkt - 1) * tstride;
    w[i][0] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(p));
    w[i][1] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(p + 16));
  };
  // (past the last block: tiles of that one, which are cached and not used)
  static_for<0, kRing>([&](auto i) { load(std::min(first, a.nb - 1), decltype(i)::value, i); });
  for (int e = tid; e < groups * kRing * 8 * N; e += kFewThreads) {
    const int n = e % N, hq = e / N % 8, kt = e / N / 8;
    sX[e] = kt < a.nkt ? operand(a.X + n * a.x_stride, kt, hq & 3, hq >> 2) : u4{};
  }
  __syncthreads();
  const int t = lane & 15, q = lane >> 4;
  const u4* const sx = sX + q * N + std::min(t, N - 1);  // columns without a token: not stored
  const float ts = a.scale[std::min(t, N - 1)];
  for (int64_t b = first; b < a.nb; b += waves) {
    i4 acc = {};
    const int64_t next = std::min(b + waves, a.nb - 1);
    for (int g = 0; g < groups; ++g) {
      const bool last = g + 1 == groups;
      static_for<0, kRing>([&](auto i_) __attribute__((always_inline)) {
        constexpr int i = decltype(i_)::value;
        const u4* x = sx + (int64_t)(kRing * g + i) * 8 * N;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(as_i4(w[i][h]), as_i4(x[4 * h * N]), acc, 0, 0, 0);
        load(last ? next : b, last ? i : kRing * (g + 1) + i, i_);
      });
    }
    // lane: rows 4 q + e of the block, token t
    const int64_t v0 = 16 * b + 4 * q;
    if (t < N) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v0 + e < a.V) put(a, t, v0 + e, (float)acc[e] * f16_to_f32(a.rowscale[v0 + e]) * ts);
    }
  }
}

// X in operand order, a fragment of 64 lanes for each 32 tokens, tile and run
// q: lane l holds token l % 32, steps 2 (l / 32) and the next.  Rows past the
// last one are zero.
__global__ __launch_bounds__(256) void i8_arrange_kernel(const I8Args a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lane = (int)(i & 63), q = (int)(i >> 6) & 3;
  const int64_t rest = i >> 8;
  const int kt = (int)(rest % a.nkt);
  const int64_t tile = rest / a.nkt, n = 32 * tile + (lane & 31);
  if (tile >= a.ntiles) return;
  a.xf[i] = n < a.N ? operand(a.X + n * a.x_stride, kt, q, lane >> 5) : u4{};
}

// TT token tiles of 32, WM x WN waves, each MT = TT / WM token tiles and WCB
// blocks of 32 rows of the vocabulary.  A stage is one 128-column tile, four
// MFMA steps: the tokens' fragments by copies straight to an LDS ring of four
// stages, the head's codes to registers of the wave that uses them, AHEAD
// stages before; a step's registers are loaded again as soon as it is
// multiplied.  256 tokens x 256 rows have every code fetched for 128 tokens and
// every token's for 64 rows: 4096 tokens of a 151936 x 4096 head 2.75 ms, 1.86
// POP/s (a large library product of 8-bit integers: 1.94), bound by the MFMAs
// under the power limit; 16 to 64 tokens are bound by the head's bytes.
template <int TT, int WM, int WN, int WCB>
struct I8Shape {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves, MT = TT / WM;
  static constexpr int kAhead = WCB == 1 ? 4 : 2;
  static constexpr int kRows = 32 * WN * WCB;        // of the vocabulary
  static constexpr int kHOps = 4 * TT / kWaves, kWOps = 4 * WCB;  // loads of a wave and stage
  static_assert(kHOps * kWaves == 4 * TT && MT * WM == TT, "whole shares");
  // Operations of a wave behind the copies that a stage's barrier waits for:
  // the copies of the two stages after, and the codes loaded since, which are
  // fewest in the first stages.
  static constexpr int kBehind = 2 * kHOps + (kAhead == 4 ? 3 * kWOps : kWOps + 3 * WCB);
  static constexpr int kBehindFirst = 3 * kHOps + kAhead * kWOps;
  static_assert(kBehind < 64 && kBehindFirst < 64, "the counter's range");
};

#define I8_SLOT(S) (*((S) == 0 ? &sH0 : (S) == 1 ? &sH1 : (S) == 2 ? &sH2 : &sH3))

template <int TT, int WM, int WN, int WCB>
__global__ __launch_bounds__(64 * WM * WN, WCB == 2 ? 2 : 4) void i8_tile_kernel(const I8Args a) {
  using S_ = I8Shape<TT, WM, WN, WCB>;
  constexpr int MT = S_::MT, kAhead = S_::kAhead, kHOps = S_::kHOps, kWaves = S_::kWaves;
  // an array for each slot, chosen at compile time, so that reads of one are
  // not taken to wait for copies to another
  __shared__ u4 sH0[4 * TT][64], sH1[4 * TT][64], sH2[4 * TT][64], sH3[4 * TT][64];
  __shared__ float sTok[32 * TT];
  const int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int ttiles = (a.ntiles + TT - 1) / TT;
  const int vtiles = (int)((a.V + S_::kRows - 1) / S_::kRows);
  // Each XCD gets a contiguous range of the walk, in which groups of four
  // token tiles go through the vocabulary together.
  constexpr int kGroup = 4;
  const int per = gridDim.x / kXcds, rem = gridDim.x % kXcds, x = blockIdx.x % kXcds;
  const int item = x * per + std::min(x, rem) + blockIdx.x / kXcds;
  const int whole = ttiles / kGroup * kGroup * vtiles;
  const int width = item < whole ? kGroup : ttiles % kGroup;
  const int at = item < whole ? item % (kGroup * vtiles) : item - whole;
  const int vt = at / width, tt = (item < whole ? item / (kGroup * vtiles) * kGroup : ttiles / kGroup * kGroup) + at % width;
  const int tile0 = tt * TT;
  const int64_t v0 = (int64_t)vt * S_::kRows;
  const int nS = a.nkt;

  const __amdgpu_buffer_rsrc_t hrs = buffer_rsrc(a.xf, (uint32_t)a.ntiles * (uint32_t)a.nkt * 4096u);
  const uint32_t lane16 = 16u * (uint32_t)lane;
  uint32_t hoff[kHOps];
#pragma unroll
  for (int i = 0; i < kHOps; ++i) {  // fragment kWaves i + wave: token tile f / 4, run f % 4
    const int f = kWaves * i + wave;
    hoff[i] = (uint32_t)std::min(tile0 + f / 4, a.ntiles - 1) * (uint32_t)a.nkt * 4096u + (uint32_t)(f % 4) * 1024u;
  }
  auto load_h = [&](int ks, auto slot_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
#pragma unroll
    for (int i = 0; i < kHOps; ++i)
      lds_copy16(hrs, &I8_SLOT(slot)[kWaves * i + wave][0], lane16, hoff[i] + (uint32_t)std::min(ks, nS - 1) * 4096u);
  };
  // codes: row c32 of block cb, the step's run in the tile's order; blocks past
  // the last one read that one, and are not stored
  const int64_t b0 = v0 / 16, tstride = a.nb * kI8Tile;
  const uint8_t* const wsrc = a.codes + b0 * kI8Tile;
  uint32_t woff[WCB];
#pragma unroll
  for (int cb = 0; cb < WCB; ++cb) {
    const int64_t b = std::min<int64_t>(b0 + 2 * (wn * WCB + cb) + (c32 >> 4), a.nb - 1);
    woff[cb] = (uint32_t)(b - b0) * kI8Tile + 32u * (uint32_t)(c32 & 15) + 16u * (uint32_t)half;
  }
  u4 w[kAhead][4][WCB];
  auto load_w = [&](int ks, auto slot_, auto step_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value, step = decltype(step_)::value;
    const uint8_t* p = wsrc + std::min(ks, nS - 1) * tstride + 512 * step;
#pragma unroll
    for (int cb = 0; cb < WCB; ++cb) w[slot][step][cb] = *reinterpret_cast<const u4*>(p + woff[cb]);
  };
  auto load_w4 = [&](int ks, auto slot) { static_for<0, 4>([&](auto t) { load_w(ks, slot, t); }); };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  // in this order, which the first barrier's count is of
  load_h(0, I0{});
  __builtin_amdgcn_sched_barrier(0);
  load_w4(0, I0{});
  load_h(1, I1{});
  load_w4(1, I1{});
  load_h(2, I2{});
  if constexpr (kAhead == 4) load_w4(2, I2{});
  load_h(3, I3{});
  if constexpr (kAhead == 4) load_w4(3, I3{});
  if (tid < 32 * TT) sTok[tid] = a.scale[std::min<int64_t>(32 * (int64_t)tile0 + tid, a.N - 1)];

  i16x acc[MT][WCB] = {};
  u4 av[2][MT];
  auto fetch = [&](auto slot_, auto step_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value, step = decltype(step_)::value;
#pragma unroll
    for (int m = 0; m < MT; ++m) av[step & 1][m] = I8_SLOT(slot)[4 * (MT * wm + m) + step][lane];
  };
  auto multiply = [&](auto slot_, auto step_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value % kAhead, step = decltype(step_)::value;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int cb = 0; cb < WCB; ++cb)
        acc[m][cb] = __builtin_amdgcn_mfma_i32_32x32x32_i8(as_i4(av[step & 1][m]), as_i4(w[slot][step][cb]), acc[m][cb], 0, 0, 0);
  };
  ring_barrier<S_::kBehindFirst>();
  fetch(I0{}, I0{});
  // (of the last stages the codes loaded ahead are used by none, and the compiler
  // drops such loads: only the copies are sure to be behind)
  auto stage = [&](int ks, auto slot_, auto last_) __attribute__((always_inline)) {
    constexpr int slot = decltype(slot_)::value;
    constexpr int behind = decltype(last_)::value ? 2 * kHOps : S_::kBehind;
    constexpr std::integral_constant<int, slot> here{};
    constexpr std::integral_constant<int, (slot + 1) & 3> there{};
    constexpr std::integral_constant<int, slot % kAhead> ring{};
    static_for<0, 3>([&](auto t_) __attribute__((always_inline)) {
      constexpr int t = decltype(t_)::value;
      fetch(here, std::integral_constant<int, t + 1>{});
      multiply(here, t_);
      load_w(ks + kAhead, ring, t_);
      __builtin_amdgcn_sched_barrier(0);
    });
    ring_barrier<behind>();
    load_h(ks + 4, here);
    fetch(there, I0{});  // past the last stage: not used
    multiply(here, I3{});
    load_w(ks + kAhead, ring, I3{});
    __builtin_amdgcn_sched_barrier(0);
  };
  int ks = 0;
  for (; ks + 4 <= nS; ks += 4) {
    stage(ks, I0{}, std::false_type{});
    stage(ks + 1, I1{}, std::false_type{});
    stage(ks + 2, I2{}, std::false_type{});
    stage(ks + 3, I3{}, std::false_type{});
  }
  if (ks < nS) stage(ks, I0{}, std::true_type{});
  if (ks + 1 < nS) stage(ks + 1, I1{}, std::true_type{});
  if (ks + 2 < nS) stage(ks + 2, I2{}, std::true_type{});
  __builtin_amdgcn_s_waitcnt(0);

  // lane: row c32 of each block, tokens 8 (e / 4) + 4 half + e % 4 of each tile
#pragma unroll
  for (int cb = 0; cb < WCB; ++cb) {
    const int64_t v = v0 + 32 * (wn * WCB + cb) + c32;
    const float s = v < a.V ? f16_to_f32(a.rowscale[v]) : 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int tl = 32 * (MT * wm + m) + 8 * (e >> 2) + 4 * half + (e & 3);
        const int64_t n = 32 * (int64_t)tile0 + tl;
        if (n < a.N && v < a.V) put(a, n, v, (float)acc[m][cb][e] * s * sTok[tl]);
      }
  }
}

#undef I8_SLOT

// ------------------------------------------------------------------- host ---

uint32_t few_lds(int64_t N, int64_t D) { return (uint32_t)(round_up((uint64_t)D / kKTile, kRing) * 128 * (uint64_t)N); }

bool few_fits(int64_t N, int64_t D) { return N <= kFewTokens && few_lds(N, D) <= kFewLds; }

uint64_t i8_workspace(const archead_dims* d, int64_t N) {
  if (N == 0 || few_fits(N, d->D)) return 0;
  return round_up((uint64_t)std::min(N, kI8ChunkRows), 32) * (uint64_t)d->D;
}

int check_int8_head(const archead_dims* d) {
  if (int rc = check_dims(d)) return rc;
  if (d->format != ARCHEAD_FMT_ROW_INT8 || d->D > kI8MaxCols) return ARCHEAD_E_UNSUPPORTED;
  return ARCHEAD_OK;
}

hipError_t launch_i8_few(const I8Args& a, hipStream_t s) {
  const uint32_t lds = few_lds(a.N, a.D);
  const int64_t blocks = std::min<int64_t>(a.nb, 256);  // one a CU
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)&i8_few_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(i8_few_kernel, dim3((unsigned)blocks), dim3(kFewThreads), lds, s, a);
  return hipGetLastError();
}

template <int TT, int WM, int WN, int WCB>
hipError_t launch_i8_tile(const I8Args& a, hipStream_t s) {
  using S_ = I8Shape<TT, WM, WN, WCB>;
  const int64_t groups = (int64_t)((a.ntiles + TT - 1) / TT) * ((a.V + S_::kRows - 1) / S_::kRows);
  hipLaunchKernelGGL((i8_tile_kernel<TT, WM, WN, WCB>), dim3((unsigned)groups), dim3(S_::kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_i8(const I8Args& a, hipStream_t s) {
  if (few_fits(a.N, a.D)) return launch_i8_few(a, s);
  const int64_t pieces = (int64_t)a.ntiles * a.nkt * 256;
  hipLaunchKernelGGL(i8_arrange_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, a);
  if (const hipError_t e = hipGetLastError()) return e;
  // 64 tokens x 128 rows, 128 x 256 and 256 x 256: 64 tokens of a 151936 x 4096
  // head take 136, 170 us (with the first and the second), 128 take 183 and 216
  // (second, third), 256 take 232 and 264 (third, second)
  if (a.N <= 64) return launch_i8_tile<2, 1, 4, 1>(a, s);
  if (a.N <= 128) return launch_i8_tile<4, 2, 4, 2>(a, s);
  return launch_i8_tile<8, 2, 4, 2>(a, s);
}

}  // namespace
}  // namespace archead

using namespace archead;

extern "C" {

int archead_logits_int8_workspace_bytes(const archead_dims* d, int64_t n_tokens, uint64_t* bytes) {
  if (!d || !bytes) return ARCHEAD_E_NULL;
  if (int rc = check_int8_head(d)) return rc;
  if (n_tokens < 0) return ARCHEAD_E_SHAPE;
  if (n_tokens > kI8MaxRows) return ARCHEAD_E_UNSUPPORTED;
  *bytes = i8_workspace(d, n_tokens);
  return ARCHEAD_OK;
}

int archead_logits_int8(const archead_tensor* X, const float* scale, const archead_packed_head* head,
                        const archead_tensor* Y, void* stream) {
  if (!X || !head || !Y) return ARCHEAD_E_NULL;
  const archead_dims* d = &head->dims;
  if (int rc = check_int8_head(d)) return rc;
  if (X->dtype != ARCHEAD_I8 || (Y->dtype != ARCHEAD_F32 && Y->dtype != ARCHEAD_BF16)) return ARCHEAD_E_DTYPE;
  const int64_t N = X->rows;
  if (N < 0 || X->cols != d->D || X->row_stride < d->D) return ARCHEAD_E_SHAPE;
  if (Y->rows != N || Y->cols != d->V || Y->row_stride < d->V) return ARCHEAD_E_SHAPE;
  if (N > kI8MaxRows) return ARCHEAD_E_UNSUPPORTED;
  if (N == 0) return ARCHEAD_OK;
  const uint64_t need = i8_workspace(d, N);
  if (!X->data || !Y->data || !scale || !head->buffer || (need && !head->workspace)) return ARCHEAD_E_NULL;
  const int size = Y->dtype == ARCHEAD_F32 ? 4 : 2;
  if ((uintptr_t)X->data % 16 || X->row_stride % 16 || (uintptr_t)scale % 4 || (uintptr_t)Y->data % size)
    return ARCHEAD_E_ALIGN;
  if ((uintptr_t)head->buffer % ARCHEAD_ALIGNMENT || (need && (uintptr_t)head->workspace % ARCHEAD_ALIGNMENT))
    return ARCHEAD_E_ALIGN;
  archead_layout L;
  compute_layout(d, &L);
  if (head->buffer_bytes < L.total_bytes) return ARCHEAD_E_SIZE;
  if (head->workspace_bytes < need) return ARCHEAD_E_WORKSPACE;
  // Y's bytes belong to nothing that the call reads
  const uint64_t y0 = (uint64_t)Y->data, y1 = y0 + ((uint64_t)(N - 1) * (uint64_t)Y->row_stride + (uint64_t)d->V) * size;
  auto in_y = [&](const void* p, uint64_t bytes) { return (uint64_t)p < y1 && y0 < (uint64_t)p + bytes; };
  if (overlap(X, 1, Y, size) || in_y(scale, 4 * (uint64_t)N) || in_y(head->buffer, L.total_bytes) ||
      (need && in_y(head->workspace, need)))
    return ARCHEAD_E_SHAPE;
  const uint8_t* buf = static_cast<const uint8_t*>(head->buffer);
  I8Args a{};
  a.V = d->V;
  a.D = d->D;
  a.nb = L.padded_rows / 16;
  a.nkt = (int)(d->D / kKTile);
  a.x_stride = X->row_stride;
  a.codes = buf + L.r_codes.offset;
  a.rowscale = reinterpret_cast<const uint16_t*>(buf + L.r_rowscale.offset);
  a.xf = static_cast<u4*>(head->workspace);
  a.y_stride = Y->row_stride;
  a.y_bf16 = Y->dtype == ARCHEAD_BF16;
  // 32-bit counts of workgroups: at least 128 rows of the vocabulary and 32 tokens each
  if ((uint64_t)((std::min(N, kI8ChunkRows) + 31) / 32) * (uint64_t)((d->V + 127) / 128) >= (1ull << 31))
    return ARCHEAD_E_UNSUPPORTED;
  (void)hipGetLastError();  // start from a clean error state
  for (int64_t n0 = 0; n0 < N; n0 += kI8ChunkRows) {
    a.N = std::min(kI8ChunkRows, N - n0);
    a.ntiles = (int)((a.N + 31) / 32);
    a.X = static_cast<const int8_t*>(X->data) + n0 * X->row_stride;
    a.scale = scale + n0;
    a.Y = static_cast<uint8_t*>(Y->data) + (uint64_t)n0 * (uint64_t)Y->row_stride * size;
    if (launch_i8(a, static_cast<hipStream_t>(stream)) != hipSuccess) return ARCHEAD_E_HIP;
  }
  return ARCHEAD_OK;
}

}  // extern "C"
