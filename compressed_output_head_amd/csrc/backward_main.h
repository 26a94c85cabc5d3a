// The product with the packed residual along the vocabulary, sum_v x[n, v]
// (q4 c8)[v, d], shared by the translation units that instantiate it
// (archead_logits_backward and archead_cross_entropy), and what they hand to
// the kernels of few rows.
#pragma once

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace archead {

constexpr int64_t kFewTokens = 32;  // of bwd_few_kernel: as many as its operands' tile holds

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

// The kernels of up to kFewTokens rows on operands that are in place: a.part
// and a.zpart from a.hf and a.gt (backward.hip).
hipError_t launch_bwd_few(const BwdArgs& a, hipStream_t s);
constexpr int kMaxSplits = 64;
// Parts of the vocabulary for the main kernel, at most `most`: the count that a
// model of its time likes best, workgroups in rounds of the resident ones (two
// a CU for 64-row tiles, else one) of kRoundUs plus a stage's measured time for
// every stage, and the partial sums written and read at 4 TB/s.
__host__ __device__ inline int best_parts(int64_t N, int64_t D, int64_t stages, int tt, int64_t most) {
  constexpr double kRoundUs = 4.0;
  // (32 bits: a kernel does this too, one thread, whose wide divisions would take 10 us)
  const uint32_t tiles = (uint32_t)((N + 32 * tt - 1) / (32 * tt) * ((D + 255) / 256)), slots = tt == 2 ? 512 : 256;
  const uint32_t steps = (uint32_t)stages, top = (uint32_t)std::max<int64_t>(most, 0);
  const double stage_us = tt == 8 ? 1.75 : tt == 6 ? 1.45 : tt == 4 ? 1.15 : 1.4;
  double best = 1e30;
  int pick = 1;
  for (uint32_t p = 1; p <= top; ++p) {
    const double us = (double)((tiles * p + slots - 1) / slots) * (kRoundUs + stage_us * (double)((steps + p - 1) / p)) +
                      (double)((int64_t)p * N * D) * 8.0 / 4e6;
    if (us < best) {
      best = us;
      pick = (int)p;
    }
  }
  return pick;
}
// Parts of the vocabulary for `ranks` tiles of 32 ranks (of few rows).
int main_splits(int64_t N, int64_t D, int64_t ranks, int64_t stages);
inline int main_tiles(int64_t N) { return N <= 64 ? 2 : N <= 128 ? 4 : 8; }

namespace {

constexpr int kMainThreads = 512;
constexpr int kMainXcds = 8;

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

// The product of a piece's exponentials (tile32_exp_kernel's operands, a.hf)
// with the residual, added to the sums of the pieces before it.
struct MainExp {
  const int32_t* plan;     // {rows that count, row tiles of a workgroup, parts of the piece}; sums are
                           // [parts][rows that count][D]
  const float* alpha;      // [n32] what brings the sums so far to the operands' exponents, a power of two
  const float* scale;      // [1] the power of two that the row scales s_R are taken with
  int steps;               // of a row tile in a.hf
  int first;               // no sums yet
  int stage0;              // first stage of the piece in the vocabulary
};

// kCodes: group codes of 128 columns of a row: 4 for g = 32, 2 for 64, else 1.
// EX: a.hf and a.ksteps are of the piece of `ex`, and the residual's operand is
// (q4 c8) s_R, rounded to fp16 (2^-11).  (With s_R in a second set of fragments
// from the kernel that makes them, that kernel takes 12% longer; here it takes 4%.)
template <int TT, int kCodes, bool EX>
__device__ __forceinline__ void bwd_main_body(const BwdArgs& a, const MainExp& ex) {
  using S = MainShape<TT>;
  constexpr int kDepth = S::kDepth;
  __shared__ h8 sA[2][S::kFrags][64];
  __shared__ h8 sB[2][64 * 32];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  if (EX && ex.plan[1] != TT) return;
  const int64_t rows = EX ? ex.plan[0] : a.N;
  const int CB = (int)((a.D + 255) / 256), ntiles = (int)((EX ? rows + 31 : a.n32) / 32), TB = (ntiles + TT - 1) / TT;
  const int splits = EX ? ex.plan[2] : a.splits, items = EX ? CB * TB * splits : gridDim.x;
  if (EX && (int)blockIdx.x >= items) return;
  // Workgroups are dealt to the XCDs round robin: each XCD gets a contiguous
  // range of (split, token block, column block), so that those in one L2 share
  // few streams of dY fragments, the larger of the two operands.
  const int per = items / kMainXcds, rem = items % kMainXcds, x = blockIdx.x % kMainXcds;
  const int item = x * per + std::min(x, rem) + blockIdx.x / kMainXcds;
  const int cb = item % CB, tb = item / CB % TB, split = item / CB / TB;
  const int stages = a.ksteps / 4;
  const int s0 = (int)((int64_t)split * stages / splits), s1 = (int)((int64_t)(split + 1) * stages / splits);

  // this wave's share of unpacking: one packed tile, 16 rows x 128 columns
  const int blk = wave & 3, kth = wave >> 2;
  const int kt = std::min(2 * cb + kth, a.nkt - 1);
  const uint8_t* wsrc = a.r_codes + (int64_t)kt * a.nb * 1024 + lane * 16;
  const uint8_t* csrc = a.r_gcodes + (lane & 15) * a.ng + kKTile * kt / a.g;
  u4 w[kDepth];
  uint32_t code[kDepth];
  h8 av[kDepth][S::kLoads];
  uint16_t rs[EX ? kDepth : 1];  // EX: the row's s_R
  const float scale = EX ? *ex.scale : 1.0f;
  auto load = [&](int s, auto slot_) {
    constexpr int slot = decltype(slot_)::value;
    s = std::min(s, s1 - 1);  // past the end: a stage that is cached, never used
    // past the last rows dY is zero
    const int64_t b = std::min<int64_t>(4 * (int64_t)(EX ? s + ex.stage0 : s) + blk, a.nb - 1);
    w[slot] = *reinterpret_cast<const u4*>(wsrc + b * 1024);
    const uint8_t* c = csrc + 16 * b * a.ng;
    code[slot] = kCodes == 4   ? *reinterpret_cast<const uint32_t*>(c)
                 : kCodes == 2 ? *reinterpret_cast<const uint16_t*>(c)
                               : *c;
    if constexpr (EX) rs[slot] = a.r_rowscale[16 * b + (lane & 15)];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int f = 8 * i + wave;
      const int64_t tile = std::min(tb * TT + f / 4, ntiles - 1);
      av[slot][i] = *reinterpret_cast<const h8*>(a.hf + ((tile * (EX ? ex.steps : a.ksteps) + 4 * s + f % 4) * 64 + lane) * 8);
    }
  };
  // columns 32 d .. + 32 of the packed tile in a register slot to the LDS tile
  auto unpack = [&](auto buf_, auto slot_, int d) {
    constexpr int buf = decltype(buf_)::value, slot = decltype(slot_)::value;
    const uint32_t c = kCodes == 4 ? (code[slot] >> (8 * d)) & 0xffu
                       : kCodes == 2 ? (code[slot] >> (8 * (d >> 1))) & 0xffu
                                     : code[slot];
    h8 x = unpack_q4_scaled(w[slot][d], (_Float16)(float)c);
    if constexpr (EX) {
      const _Float16 r = (_Float16)(f16_to_f32(rs[slot]) * scale);
      x = x * h8{r, r, r, r, r, r, r, r};
    }
    sB[buf][tile_octet(16 * blk + (lane & 15), 16 * kth + 4 * d + (lane >> 4))] = x;
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
  for (int m = 0; m < S::MT; ++m) {
    auto column = [&](int c) { return 256 * (int64_t)cb + 32 * (wn * S::NT + c) + 8 * (c32 >> 3) + k_order_h(c32 & 7); };
    auto row = [&](int v) { return 32 * (int64_t)(tb * TT + wm * S::MT + m) + 8 * (v >> 2) + 4 * khalf + (v & 3); };
    if constexpr (EX) {
      if (!ex.first) {  // all loads of a row tile in flight together
        float old[S::NT][16], al[16];
#pragma unroll
        for (int v = 0; v < 16; ++v) {  // rows and columns past the last: those, not stored
          const int64_t n = std::min(row(v), rows - 1);
          al[v] = ex.alpha[n];
#pragma unroll
          for (int c = 0; c < S::NT; ++c) old[c][v] = a.part[((int64_t)split * rows + n) * a.D + std::min(column(c), a.D - 1)];
        }
#pragma unroll
        for (int c = 0; c < S::NT; ++c)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[m][c][v] = fmaf(al[v], old[c][v], acc[m][c][v]);
      }
    }
#pragma unroll
    for (int c = 0; c < S::NT; ++c)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (row(v) < rows && column(c) < a.D) a.part[((int64_t)split * rows + row(v)) * a.D + column(c)] = acc[m][c][v];
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

template <int TT, int kCodes>
__global__ __launch_bounds__(kMainThreads, TT >= 8 ? 2 : 4) void bwd_main_kernel(const BwdArgs a) {
  bwd_main_body<TT, kCodes, false>(a, MainExp{});
}

}  // namespace
}  // namespace archead
