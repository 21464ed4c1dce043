// The dense product beside the experts, with bias, activation and residual in its epilogue,
// and its gradients, on gfx950:
//   z = x w^T + b, y = act(z) + residual        x [M, K], w [N, K]   (bqm_linear_fwd)
//   dx = (dz w) act'(zx) + add                  dz [M, N]            (bqm_linear_dgrad)
//   dw = dz^T x, db = sum_m dz                                       (bqm_linear_wgrad)
//   dz = dy act'(z)                                                  (bqm_act_grad)
//
// All three products are C[i, j] = sum_c A(i, c) B(j, c) of bf16 operands on the 16x16x32
// MFMA with FP32 accumulators.  They differ in how an operand lies in memory: with its
// contraction contiguous (x and w in the forward, dz in the input gradient) or as rows of the
// contraction (w in the input gradient, dz and x in the weight gradient); the latter is read
// from LDS transposed.  No transposed copy of a tensor is made.
//
// What bounds it.  Large products: the power the matrix unit draws (69% busy at a clock of 2.0
// GHz); 16384 x 4096 x 6144 takes 555 us forward, 570 for the input's and 590 for the weight's
// gradient, 1.4 to 1.5 PFLOP/s.  The 16x16x32 instruction draws less than the 32x32x16 of the
// same rate.  Small ones: 4 to 7 us of launch, first copies and epilogue, and steps in which the
// copies take about as long as the fragment reads and products beside them: 1111 x 2848 x 2080, one
// round of 128 x 128 tiles, takes 21.0 us, without its copies 19.0, without its products 20.1, without
// both (fragment reads, waits, barriers) 13.0; where rows start on 128 bytes (2048 in place of 2080) the
// copies are hidden, 17.9 us in all.  64 x 64 tiles: a CU's copies, 85 GB/s (16 KB of a step in 0.19
// us); 203 x 768 x 2048 8.7 us.  Few rows: the weights' bytes.
#include "common.h"
#include "linear_plan.h"

#include <type_traits>

namespace bqm {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;

constexpr int NTHR = 256;  // four waves, one per SIMD

enum Mode { FWD, DGRAD, WGRAD };

struct LinParams {
  const uint8_t *a, *b;  // operands
  int64_t I, J;          // rows and columns of the result
  int64_t lda, ldb;      // bytes per row of an operand as it is stored
  int C, nk;             // contraction, and its steps
  int NI, NJ;            // tiles
  int full, rem;         // tiles computed whole, and those behind them
  int S, per;            // which are split into S parts of per steps
  int grid;              // workgroups that walk tiles
  int mode, act, accumulate;
  const uint16_t *bias, *add, *zx;
  uint16_t *out, *z;
  float *dw, *part;
};

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
__device__ __forceinline__ float sigmoid_f(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// tanh-GELU as v s(2 u), u = sqrt(2/pi) (v + 0.044715 v^3), from (1 + tanh(u)) / 2 = s(2 u)
constexpr float kGelu = 1.5957691216057308f;  // 2 sqrt(2/pi)

__device__ __forceinline__ float act_f(int act, float v) {
  if (act == BQM_ACT_RELU) return v < 0.0f ? 0.0f : v;  // NaN stays
  if (act == BQM_ACT_SILU) return v * sigmoid_f(v);
  return v * sigmoid_f(kGelu * (v + 0.044715f * v * v * v));
}

// d act'(v).  ReLU chooses: where it is off, nothing of d passes, NaN or infinite as it may be;
// a NaN in v does not hide (d passes).
__device__ __forceinline__ float through_act(int act, float d, float v) {
  if (act == BQM_ACT_RELU) return v <= 0.0f ? 0.0f : d;
  if (act == BQM_ACT_SILU) {
    const float s = sigmoid_f(v);
    return d * (s * (1.0f + v * (1.0f - s)));
  }
  // past |v| = 16 the sigmoid is 0 or 1 in FP32 and so is the derivative; v^2 need not be formed.
  // Comparisons, as the minimum and maximum of the machine would make a number of a NaN.
  const float t = v > 16.0f ? 16.0f : v < -16.0f ? -16.0f : v, q = t * t;
  const float s = sigmoid_f(kGelu * t * (1.0f + 0.044715f * q));
  return d * (s * (1.0f + t * (1.0f - s) * kGelu * (1.0f + 0.134145f * q)));
}

// ---------------------------------------------------------------------------
// what becomes of 8 sums of a row
// ---------------------------------------------------------------------------
__device__ __forceinline__ float unpack(const u32x4 &v, int i) { return i & 1 ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]); }
__device__ __forceinline__ u32x4 pack(const float *v) {
  return u32x4{pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3]), pack_bf16_rne(v[4], v[5]), pack_bf16_rne(v[6], v[7])};
}
__device__ __forceinline__ u32x4 load8(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

struct Extra {
  u32x4 add, zx;
};
__device__ __forceinline__ Extra load_extra(const LinParams &p, int64_t at) {
  Extra x = {};
  if (p.mode != WGRAD && p.add) x.add = load8(p.add + at);
  if (p.mode == DGRAD && p.act != BQM_ACT_NONE) x.zx = load8(p.zx + at);
  return x;
}

// at: element offset of the first of the 8 in the output
__device__ __forceinline__ void finish(const LinParams &p, int64_t at, float *v, const u32x4 &bias, const Extra &x) {
  if (p.mode == WGRAD) {
    f32x4 *o = reinterpret_cast<f32x4 *>(p.dw + at);
    f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    if (p.accumulate) lo += o[0], hi += o[1];
    o[0] = lo;
    o[1] = hi;
    return;
  }
  if (p.mode == FWD) {
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += unpack(bias, i);
    }
    if (p.z) *reinterpret_cast<u32x4 *>(p.z + at) = pack(v);
    if (p.act != BQM_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_f(p.act, v[i]);
    }
  } else if (p.act != BQM_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = through_act(p.act, v[i], unpack(x.zx, i));
  }
  if (p.add) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += unpack(x.add, i);
  }
  *reinterpret_cast<u32x4 *>(p.out + at) = pack(v);
}

// ---------------------------------------------------------------------------
// copies and waits
// ---------------------------------------------------------------------------
__device__ __forceinline__ const uint8_t *uniform(const void *q) {
  const uint64_t v = reinterpret_cast<uint64_t>(q);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t *>(((uint64_t)hi << 32) | lo);
}
// Direct-to-LDS copies: lane i's 16 bytes land at lds + 16 i.  Inline assembly, so that the
// compiler's wait counts do not drain every LDS read before each use of an LDS result; the
// copies are waited for with wait_vm before their stage is read.
__device__ __forceinline__ void dma_b128(const void *g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(g), "s"(lds) : "memory", "m0");
}
// The same with a scalar base and a lane's byte offset; lane i's 16 bytes land at lds + AT + 16 i.
template <int AT>
__device__ __forceinline__ void dma_b128(const void *base, uint32_t off, uint32_t lds) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(uniform(base)), "s"(__builtin_amdgcn_readfirstlane(lds)), "n"(AT)
               : "memory", "m0", "scc");
}
__device__ __forceinline__ void barrier_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void *p) { return (uint32_t)(uintptr_t)(const lds_void *)p; }
__device__ __align__(16) const uint32_t c_zeros[4] = {0u, 0u, 0u, 0u};

#define LIN_PIN() __builtin_amdgcn_sched_barrier(0)

// ---------------------------------------------------------------------------
// one operand of a tile
// ---------------------------------------------------------------------------
// R result rows (or columns) of it by KS of the contraction per stage.
// T = false: [row][KS], the 16-byte chunk c of a row at c ^ ((row >> 1) & (chunks - 1)), so that
// a fragment read (one chunk of 16 rows) falls on different banks.
// T = true: for each 64 result columns [contraction row][128 bytes], chunk c of row r at
// c ^ 2 ((r & 3) ^ (r / 8 & 1)): a transposing read takes 32 bytes of rows 0..3 and 8..11 per
// 32 lanes.
// Stages are filled by direct copies of 1 KB per wave: 512 / KS rows, or 8 of the 128-byte rows.
template <int R, bool T, bool FAST>
struct Operand {
  static constexpr int kCopies = R * KS / 2048;  // per wave and step
  static constexpr int CPR = KS / 8;             // chunks per row
  const uint8_t *base;
  int64_t ld;
  uint32_t off[kCopies];
  int C;
  int lane, w;

  // row (of the result, or with T of the contraction) and result column of copy j of this lane
  __device__ __forceinline__ int row(int j) const {
    const int n = kCopies * w + j;
    return T ? 8 * (n % CPR) + (lane >> 3) : 512 / KS * n + lane / CPR;
  }
  __device__ __forceinline__ int chunk(int j) const {
    const int r = row(j);
    return T ? (lane & 7) ^ turn(r) : (lane & (CPR - 1)) ^ ((r >> 1) & (CPR - 1));
  }

  // T: what a row's chunks are XORed with
  __device__ __forceinline__ static int turn(int r) { return 2 * ((r & 3) ^ ((r >> 3) & 1)); }

  // rows: of the whole operand; r0: the tile's first
  __device__ __forceinline__ void setup(const uint8_t *q, int64_t ld_, int C_, int64_t rows, int64_t r0, int lane_, int w_) {
    ld = ld_, C = C_, lane = lane_, w = w_;
    base = uniform(T ? q + 2 * r0 : q + r0 * ld);
    const int most = (int)min(rows - r0, (int64_t)R);
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      if constexpr (T)  // columns past the last are the last 8 again (their results are dropped)
        off[j] = (uint32_t)row(j) * (uint32_t)ld + 2 * min(64 * ((kCopies * w + j) / CPR) + 8 * chunk(j), most - 8);
      else
        off[j] = (uint32_t)min(row(j), most - 1) * (uint32_t)ld + 16 * chunk(j);
    }
  }

  // copy J of step ks.  FAST: a contraction of at least one whole step; the last step, where
  // it is not whole, takes the last KS of the contraction (and zeroes in registers what the
  // step before had).  Otherwise the one step there is takes zeros past the end.
  template <int J>
  __device__ __forceinline__ void copy(int ks, uint8_t *stage) const {
    const uint32_t to = lds_addr(stage) + 1024 * kCopies * w;
    if constexpr (FAST) {
      const int at = min(KS * ks, C - KS);
      dma_b128<1024 * J>(base + (T ? at * ld : (int64_t)(2 * at)), off[J], to);
    } else {
      const bool in = T ? row(J) < C : 8 * chunk(J) < C;
      dma_b128(in ? base + off[J] : reinterpret_cast<const uint8_t *>(c_zeros), to + 1024 * J);
    }
  }

  // Fragment of 16 rows from row c0 + c on (c0: the wave's), slice kk: lane l holds row l % 16,
  // contraction 32 kk + 8 (l / 16) + 0..7.  Its address is one of a few that depend on the
  // lane (kept in registers, one addition per stage), and a constant.
  static constexpr int kVariants = T ? 4 : 2;  // by c / 16 % 4, by kk
  uint32_t lane_at[kVariants];
  __device__ __forceinline__ void setup_fragments(int c0) {
#pragma unroll
    for (int v = 0; v < kVariants; ++v) {
      if constexpr (T) {
        const int g = lane >> 4, s = lane & 15, c = c0 + 16 * v;
        lane_at[v] = (c >> 6) * (KS * 128) + (8 * g + (s >> 2)) * 128 +
                     16 * (((c & 63) / 8 + ((s & 3) >> 1)) ^ turn(8 * g + (s >> 2))) + 8 * (s & 1);
      } else {
        const int r = c0 + (lane & 15);
        lane_at[v] = r * (2 * KS) + 16 * ((4 * v + (lane >> 4)) ^ ((r >> 1) & (CPR - 1)));
      }
    }
  }
  // the fragments' addresses in a stage; opaque, or the compiler adds the constants to the
  // stage first, and then the lane's part to each of the sums
  uint32_t at[kVariants];
  __device__ __forceinline__ void enter(uint32_t stage) {
#pragma unroll
    for (int v = 0; v < kVariants; ++v) {
      at[v] = stage + lane_at[v];
      asm("" : "+v"(at[v]));
    }
  }
  // c: a multiple of 16, known when compiled
  __device__ __forceinline__ i32x4 fragment(int c, int kk) const {
    if constexpr (T) {
      const uint32_t q = at[c / 16 % 4] + (c >> 6) * (KS * 128) + kk * (32 * 128);
      const s16x4 h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(q));
      const s16x4 h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(q + 4 * 128));
      const s16x8 v = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
      return __builtin_bit_cast(i32x4, v);
    } else {
      return *(const lds_i32x4 *)(uintptr_t)(at[kk] + c * (2 * KS));
    }
  }
};

// OUT: bytes of the epilogue for each wave; 0: it takes the stages
template <int BM, int BN, int NSA, int NSB, int OUT>
struct Smem {
  uint8_t a[NSA][BM * 2 * KS];
  uint8_t b[NSB][BN * 2 * KS];
  uint8_t out[4][OUT];
};
template <int BM, int BN, int NSA, int NSB>
struct Smem<BM, BN, NSA, NSB, 0> {
  uint8_t a[NSA][BM * 2 * KS];
  uint8_t b[NSB][BN * 2 * KS];
};

// row and column tile of tile L: groups of about G row tiles, column by column, so that the tiles
// in flight on an XCD are about as many rows as columns (G = 1, 16384 x 4096 x 6144: forward 571
// against 555 us, gradients 598 and 611 against 571 and 590)
template <int G>
__device__ __forceinline__ int2 tile_at(const LinParams &p, int L) {
  const int n_g = max((p.NI + G / 2) / G, 1), g = (p.NI + n_g - 1) / n_g;
  const int m_first = L / (g * p.NJ) * g, gm = min(g, p.NI - m_first), in_g = L - m_first * p.NJ;
  return make_int2(m_first + in_g % gm, in_g / gm);
}

// ---------------------------------------------------------------------------
// a tile
// ---------------------------------------------------------------------------
// A workgroup of four waves (WM x WN) computes BM = 32 WM TM rows by BN = 32 WN TN columns;
// wave (wm, wn) owns the 32-row tiles WM tm + wm (interleaved, so that a partly filled tile
// leaves all rows of waves the same work) of 32 TN columns.  The contraction goes in steps of
// KS through NS LDS stages; a step is KS / 32 slices of 2 VT x 2 TN MFMAs.  One wave per SIMD (the
// accumulators of the largest tile take half the register file) has no other wave to hide its
// waits behind, so a step is written out in issue order: each MFMA is followed by its share of
// the fragment reads of the next slice and of the copies of a later step, held there by
// scheduling barriers.  The step's one barrier sits inside its last slice, whose fragments are
// in registers by then; the copies of step ks + NS start behind it, into the stage just read.
// Stages: as many as LDS holds.  Of the largest tile's three of A and two of B against two of
// both: 16384 x 4096 x 6144 555 against 619 us.  128 x 128 columns, four against two: 1111 x 2848
// x 2080 21.0 against 28.4; 64 x 64, four, three, two: 37 x 6144 x 2048 8.9, 11.2, 17.8 us.  Two
// groups of four waves that share the steps of one 64 x 64 tile gain nothing (8.8 us): the CU's
// copies are at their rate.
//
// Accumulators hold the product transposed (B x A): register v of lane L of a 16 x 16 block is
// row L % 16 and column 4 (L / 16) + v.
template <int WM, int TM, int TN, bool AT, bool BT, bool FAST, int NSA, int NSB>
struct Tile {
  static constexpr int WN = 4 / WM, BM = 32 * WM * TM, BN = 32 * WN * TN;
  using OpA = Operand<BM, AT, FAST>;
  using OpB = Operand<BN, BT, FAST>;
  static constexpr int CA = OpA::kCopies, CB = OpB::kCopies, kCopies = CA + CB;
  static constexpr int NSL = KS / 32;  // slices per step
  static constexpr bool WHOLE = TM * TN == 1;  // fragments of a whole step in registers, twice
  static constexpr int RM = 2 * TM, RN = 2 * TN;    // fragments of 16 rows, of 16 columns
  // sets of fragments; WHOLE: set NSL q + kk for slice kk of a step of parity q
  static constexpr int SETS_A = WHOLE ? 2 * NSL : 1, SETS_B = WHOLE ? 2 * NSL : 2;
  static_assert(WHOLE ? NSA == NSB : NSL == 2 && (NSA == NSB || NSA == NSB + 1), "stages");
  static constexpr int UN = TN < 2 ? 1 : 2;  // column tiles of a unit of the epilogue
  static constexpr int CH = 8 * UN, LPR = 4 * UN, RP = 64 / LPR, NP = 32 / RP;
  using Mem = Smem<BM, BN, NSA, NSB, WHOLE ? 32 * CH * 16 : 0>;
  static constexpr int NS = NSB;  // WHOLE: of both
  const LinParams &p;
  Mem &sm;
  int lane, w, wm, wn;
  OpA a;
  OpB b;
  int over;  // of the last step, the leading part that the step before had
  i32x4 af[SETS_A][RM], bf[SETS_B][RN];
  f32x4 acc[RM][RN];
  // where a lane's share of the result goes
  struct Out {
    int64_t first;      // element offset of the wave's first row and column in the result
    uint32_t off;       // of this lane's from there
    int rows, cols;     // of the result from this lane's first on
    bool whole;         // all of the tile exists
    float *part;
    const uint16_t *bias;
  };

  __device__ __forceinline__ Tile(const LinParams &p_, Mem &sm_) : p(p_), sm(sm_) {
    lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = WM == 2 ? w >> 1 : 0;
    wn = WM == 2 ? w & 1 : w;
  }

  __device__ __forceinline__ static int stage_a(int ks) { return (int)((unsigned)ks % NSA); }
  __device__ __forceinline__ static int stage_b(int ks) { return (int)((unsigned)ks % NSB); }
  template <int J>
  __device__ __forceinline__ void copy_a(int ks) {
    a.template copy<J>(ks, sm.a[stage_a(ks)]);
  }
  template <int J>
  __device__ __forceinline__ void copy_b(int ks) {
    b.template copy<J>(ks, sm.b[stage_b(ks)]);
  }
  template <int J = 0>
  __device__ __forceinline__ void copy_step(int ks) {  // B, then A
    if constexpr (J < CB)
      copy_b<J>(ks);
    else
      copy_a<J - CB>(ks);
    if constexpr (J + 1 < kCopies) copy_step<J + 1>(ks);
  }
  // fragments are read from the stages of step ks from here on
  __device__ __forceinline__ void enter(int ks) {
    a.enter(lds_addr(sm.a[0]) + stage_a(ks) * (uint32_t)sizeof(sm.a[0]));
    b.enter(lds_addr(sm.b[0]) + stage_b(ks) * (uint32_t)sizeof(sm.b[0]));
  }
  // a wave's 32-row tiles are 32 WM rows apart
  __device__ __forceinline__ void read_a(int k, int m, int kk) { af[k][m] = a.fragment(32 * WM * (m / 2) + 16 * (m % 2), kk); }
  __device__ __forceinline__ void read_b(int k, int n, int kk) { bf[k][n] = b.fragment(16 * n, kk); }
  // the q-th of a slice's MFMAs
  __device__ __forceinline__ void mfma(int ka, int kb, int q) {
    const int m = q / RN, n = q % RN;
    acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bf[kb][n]),
                                                        __builtin_bit_cast(bf16x8, af[ka][m]), acc[m][n], 0, 0, 0);
  }

  // zeros in place of what the step before the last had, in both operands (0 times an
  // infinity would be NaN)
  template <int VT>
  __device__ __forceinline__ void drop_overlap(int ka, int kb, int kk) {
    if (over <= 32 * kk) return;
    int mask[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = over - (32 * kk + 8 * (lane >> 4) + 2 * i);
      mask[i] = d <= 0 ? -1 : d == 1 ? (int)0xFFFF0000 : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int m = 0; m < 2 * VT; ++m) af[ka][m][i] &= mask[i];
#pragma unroll
      for (int n = 0; n < RN; ++n) bf[kb][n][i] &= mask[i];
    }
  }

  // Large tiles: a slice is 2 VT x RN MFMAs, row of fragments by row.  Beside them go, evenly
  // spread, the fragment reads of the next slice.  A row's fragment is read into the place of
  // the one just used, the last one at the start of its slice; B has two sets (two sets of both
  // leave too few registers).  Slice 1 has the step's barrier behind its first row, from where
  // on this step's stages are filled anew: with B for step ks + NSB, then A for ks + NSA, which
  // goes on in slice 0 of the next step.  The copies are kGap MFMAs apart: the four waves' take
  // 64 cycles on their way, and closer ones hold up the MFMAs (one MFMA apart, 16384 x 4096 x
  // 6144: forward 581 against 555 us, gradients 589 and 610 against 571 and 590); B, with fewer
  // stages, comes first as it has the least time.
  static constexpr int kGap = 5;
  // MFMAs between the barrier and copy j of a step
  template <int VT>
  __device__ __forceinline__ static constexpr int copy_at(int j) {
    constexpr int all = 3 * VT * RN + (VT - 1) * RN, gap = kGap * kCopies < all ? kGap : 0;
    if (!gap) return j * all / kCopies;
    return j < CB ? gap * j : gap * CB + (j - CB) * (all - gap * CB) / CA;
  }
  template <int VT, int J>
  __device__ __forceinline__ void copies_at(int at, int s) {
    if (copy_at<VT>(J) == at) {
      if constexpr (J < CB)
        copy_b<J>(s + NSB);
      else
        copy_a<J - CB>(s + NSA);
    }
    if constexpr (J + 1 < kCopies) copies_at<VT, J + 1>(at, s);
  }
  // of A's copies of a step, those from J on that come before the next step's slice 0
  template <int VT, int J = 0>
  __device__ __forceinline__ void first_copies_a(int ks) {
    if constexpr (J < CA) {
      if constexpr (copy_at<VT>(CB + J) < (2 * VT - 1) * RN) copy_a<J>(ks);
      first_copies_a<VT, J + 1>(ks);
    }
  }
  template <int VT>
  static constexpr int count_first() {
    int n = 0;
    for (int j = 0; j < CA; ++j) n += copy_at<VT>(CB + j) < (2 * VT - 1) * RN;
    return n;
  }
  template <int J = 0>
  __device__ __forceinline__ void copies_b(int ks) {
    copy_b<J>(ks);
    if constexpr (J + 1 < CB) copies_b<J + 1>(ks);
  }
  template <int VT, int KK, bool LAST>
  __device__ __forceinline__ void slice(int ks) {
    constexpr int R = 2 * VT, NP = R * RN, QB = RN, NR = LAST && KK == 1 ? 0 : RN + R - 1, Q0 = KK == 1 ? QB : 0;
    read_a(0, R - 1, KK);
    if constexpr (FAST && LAST) drop_overlap<VT>(0, KK, KK);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      mfma(0, KK, q);
      if constexpr (KK == 1 && !LAST) {
        if (q == QB - 1) {
          // every wave is done reading this step's stages, and the next are whole
          LIN_PIN();
          wait_vm<(NSB - 2) * kCopies + (NSA > NSB ? CA : 0)>();
          barrier_lds();
          enter(ks + 1);
          LIN_PIN();
        }
      }
      if (q >= QB) {  // a row's fragment has been used
#pragma unroll
        for (int i = (q - QB) * NR / (NP - QB); i < (q - QB + 1) * NR / (NP - QB); ++i) {
          if (i < RN)
            read_b(KK ^ 1, i, KK ^ 1);
          else
            read_a(0, i - RN, KK ^ 1);
        }
      }
      if (!LAST && q >= Q0) copies_at<VT, 0>(KK == 1 ? q - QB : NP - QB + q, KK == 1 ? ks : ks - 1);
      LIN_PIN();
    }
  }

  // zeros as products of zeros: short code
  template <int VT>
  __device__ __forceinline__ void clear() {
    bf16x8 z = {};
    asm volatile("" : "+v"(z));
#pragma unroll
    for (int m = 0; m < 2 * VT; ++m)
#pragma unroll
      for (int n = 0; n < RN; ++n) acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z, z, f32x4{}, 0, 0, 0);
  }

  // Small tiles: a slice's few MFMAs are shorter than a fragment read takes, so all of the next
  // step's fragments are read while this step's are multiplied.
  template <int VT>
  __device__ __forceinline__ void read_step(int ks, int par) {
    enter(ks);
#pragma unroll
    for (int kk = 0; kk < NSL; ++kk) {
#pragma unroll
      for (int i = 0; i < RN; ++i) read_b(NSL * par + kk, i, kk);
#pragma unroll
      for (int i = 0; i < 2 * VT; ++i) read_a(NSL * par + kk, i, kk);
    }
  }
  template <int VT>
  __device__ __forceinline__ void mfma_step(int par) {
#pragma unroll
    for (int kk = 0; kk < NSL; ++kk)
#pragma unroll
      for (int q = 0; q < 2 * VT * RN; ++q) mfma(NSL * par + kk, NSL * par + kk, q);
  }
  // waits until at most min(n, N) steps' copies are in flight
  template <int N>
  __device__ __forceinline__ static void wait_steps(int n) {
    if (N == 0 || n >= N)
      wait_vm<N * kCopies>();
    else if constexpr (N > 0)
      wait_steps<N - 1>(n);
  }
  // MORE: at least NS steps follow
  template <int VT, int PAR, bool MORE>
  __device__ __forceinline__ void whole_step(int ks, int last) {
    wait_steps<NS - 2>(MORE ? NS : last - ks - 1);
    barrier_lds();  // the next step's stage is whole, and every wave has this step's fragments
    read_step<VT>(ks + 1, PAR ^ 1);
    if (MORE || ks + NS <= last) copy_step(ks + NS);
    mfma_step<VT>(PAR);
  }
  template <int VT, int PAR>
  __device__ __forceinline__ void last_step() {
    if constexpr (FAST) {
#pragma unroll
      for (int kk = 0; kk < NSL; ++kk) drop_overlap<VT>(NSL * PAR + kk, NSL * PAR + kk, kk);
    }
    mfma_step<VT>(PAR);
  }
  template <int VT>
  __device__ __forceinline__ void run_whole(int k0, int last) {
#pragma unroll
    for (int q = 0; q < NS; ++q)
      if (k0 + q <= last) copy_step(k0 + q);
    clear<VT>();
    wait_steps<NS - 1>(last - k0);
    barrier_lds();
    read_step<VT>(k0, 0);
    int ks = k0;
    for (; ks + NS + 1 <= last; ks += 2) {
      whole_step<VT, 0, true>(ks, last);
      whole_step<VT, 1, true>(ks + 1, last);
    }
    for (; ks + 2 <= last; ks += 2) {
      whole_step<VT, 0, false>(ks, last);
      whole_step<VT, 1, false>(ks + 1, last);
    }
    if (ks < last) {
      whole_step<VT, 0, false>(ks, last);
      last_step<VT, 1>();
    } else {
      last_step<VT, 0>();
    }
  }

  // steps [k0, k1) of the tile, of which VT row tiles per wave hold rows
  template <int VT>
  __device__ __forceinline__ void run(int k0, int k1) {
    over = FAST && k1 == p.nk ? KS * p.nk - p.C : 0;
    if constexpr (WHOLE)
      run_whole<VT>(k0, k1 - 1);
    else
      run_sliced<VT>(k0, k1 - 1);
  }

  // The copies run up to NSA steps past the last (where FAST has them end within the operand)
  // and are not used: one loop body for all steps but the last keeps the code that a workgroup
  // executes short, and its first pass over it is bound by the instruction fetch.
  template <int VT>
  __device__ __forceinline__ void run_sliced(int k0, int last) {
    // in the order of the loop; its first slice 0 has the rest
#pragma unroll
    for (int q = 0; q < NSB; ++q) {
      if (q < NSA - 1) {
        copy_step(k0 + q);
      } else {
        copies_b(k0 + q);
        first_copies_a<VT>(k0 + q);
      }
    }
    if constexpr (NSA > NSB) first_copies_a<VT>(k0 + NSB);
    constexpr int rest = NSA > NSB ? NSB : NSA - 1;  // whole steps of A, of which one is needed
    clear<VT>();
    wait_vm<(NSB - 1) * CB + (rest - 1) * CA + count_first<VT>()>();
    barrier_lds();
    enter(k0);
#pragma unroll
    for (int i = 0; i < RN; ++i) read_b(0, i, 0);
#pragma unroll
    for (int i = 0; i < 2 * VT - 1; ++i) read_a(0, i, 0);
    for (int ks = k0; ks < last; ++ks) {
      slice<VT, 0, false>(ks);
      slice<VT, 1, false>(ks);
    }
    slice<VT, 0, true>(last);
    slice<VT, 1, true>(last);
    // the epilogue takes the stages: no copy lands there, no wave reads them any more
    wait_vm<0>();
    barrier_lds();
  }

  // The accumulators hold 4 columns of 16 rows a lane quarter.  They pass through LDS in FP32 in
  // units of 32 rows by UN column tiles of a wave, so that a lane finishes 8 consecutive columns
  // of NP rows and reads and writes 16 bytes at a time (chunk c of row r at c ^ (r & (CH - 1))).
  // One wave per SIMD means that every instruction here counts: addresses are a scalar base
  // and a lane offset that stays, choices are made once for all of a lane's values, and what
  // the epilogue reads (residual, pre-activation) is loaded one unit ahead.
  static constexpr int MODE = AT ? WGRAD : BT ? DGRAD : FWD;
  static constexpr int UC = TN / UN;  // units per 32 rows

  template <int TMX, int U>
  __device__ __forceinline__ void put(uint8_t *t) const {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = 16 * m + (lane & 15);
#pragma unroll
      for (int n = 0; n < 2 * UN; ++n)
        *reinterpret_cast<f32x4 *>(t + 16 * (r * CH + ((4 * n + (lane >> 4)) ^ (r & (CH - 1))))) = acc[2 * TMX + m][2 * UN * U + n];
    }
    // an end of its own for each: with one end in common the compiler addresses the
    // accumulators by a variable, and so keeps them in memory
    asm volatile("; unit %0" ::"n"(TMX * UC + U));
  }
  template <int U>
  __device__ __forceinline__ void put_unit(int tm, uint8_t *t) const {
    if (TM == 1 || tm == 0)
      put<0, U>(t);
    else if (TM == 2 || tm == 1)
      put<TM < 2 ? 0 : 1, U>(t);
    else if (tm == 2)
      put<TM < 4 ? 0 : 2, U>(t);
    else
      put<TM < 4 ? 0 : 3, U>(t);
  }

  __device__ __forceinline__ Out out_of(int64_t i0, int64_t j0, float *part) const {
    Out o;
    const int lr = lane / LPR, c = lane % LPR;
    o.first = (i0 + 32 * wm) * p.J + j0 + 32 * TN * wn;
    o.off = (uint32_t)lr * (uint32_t)p.J + 8 * c;
    o.rows = (int)min(p.I - i0, (int64_t)BM) - 32 * wm - lr;
    o.cols = (int)min(p.J - j0, (int64_t)BN) - 32 * TN * wn - 8 * c;
    o.whole = p.I - i0 >= BM && p.J - j0 >= BN;
    o.part = part;
    o.bias = p.bias + j0 + 32 * TN * wn;
    return o;
  }
  // element (32 WM tm, 32 UN u) from the wave's first on
  __device__ __forceinline__ int64_t unit_at(int tm, int u) const { return (int64_t)(32 * WM * tm) * p.J + 32 * UN * u; }
  __device__ __forceinline__ static bool inside(const Out &o, int tm, int u, int q) {
    return 32 * WM * tm + RP * q < o.rows && 32 * UN * u < o.cols;
  }

  // what lies outside the result is read from src's first elements instead (and not used)
  __device__ __forceinline__ void load_rows(const Out &o, const uint16_t *src, int tm, int u, u32x4 *x) const {
    const uint8_t *base = uniform(src + o.first + unit_at(tm, u));
    const int64_t pass = (int64_t)RP * p.J * 2;
    if (o.whole) {
#pragma unroll
      for (int q = 0; q < NP; ++q) x[q] = *reinterpret_cast<const u32x4 *>(base + q * pass + 2 * o.off);
    } else {
#pragma unroll
      for (int q = 0; q < NP; ++q)
        x[q] = load8(inside(o, tm, u, q) ? reinterpret_cast<const uint16_t *>(base + q * pass + 2 * o.off) : src);
    }
  }
  // ADD, ZX: whether there is something to add, and an activation's argument
  template <bool ADD, bool ZX>
  struct Extras {
    u32x4 add[ADD ? NP : 1], zx[ZX ? NP : 1];
  };
  template <bool ADD, bool ZX>
  __device__ __forceinline__ void load_extras(const Out &o, int tm, int u, Extras<ADD, ZX> &x) const {
    if constexpr (ADD) load_rows(o, p.add, tm, u, x.add);
    if constexpr (ZX) load_rows(o, p.zx, tm, u, x.zx);
  }
  __device__ __forceinline__ void store_rows(const Out &o, uint16_t *dst, int tm, int u, const u32x4 *x) const {
    uint8_t *base = const_cast<uint8_t *>(uniform(dst + o.first + unit_at(tm, u)));
    const int64_t pass = (int64_t)RP * p.J * 2;
    if (o.whole) {
#pragma unroll
      for (int q = 0; q < NP; ++q) *reinterpret_cast<u32x4 *>(base + q * pass + 2 * o.off) = x[q];
    } else {
#pragma unroll
      for (int q = 0; q < NP; ++q)
        if (inside(o, tm, u, q)) *reinterpret_cast<u32x4 *>(base + q * pass + 2 * o.off) = x[q];
    }
  }

  template <int U, bool ADD, bool ZX>
  __device__ __forceinline__ void finish_unit(const Out &o, int tm, const Extras<ADD, ZX> &x) {
    uint8_t *t;
    if constexpr (WHOLE)
      t = sm.out[w];
    else
      t = sm.a[0] + w * (32 * CH * 16);
    const int lr = lane / LPR, c = lane % LPR;
    put_unit<U>(tm, t);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    f32x4 v[NP][2];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int rr = q * RP + lr;
#pragma unroll
      for (int h = 0; h < 2; ++h) v[q][h] = *reinterpret_cast<const f32x4 *>(t + 16 * (rr * CH + ((2 * c + h) ^ (rr & (CH - 1)))));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (MODE == WGRAD || o.part) {
      float *dst = o.part ? o.part + (32 * wm + 32 * WM * tm) * BN + 32 * TN * wn + 32 * UN * U : p.dw + o.first + unit_at(tm, U);
      const int64_t ld = o.part ? BN : p.J;
      uint8_t *base = const_cast<uint8_t *>(uniform(dst));
      const uint32_t off = 4 * (o.part ? (uint32_t)(lr * BN + 8 * c) : o.off);
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        f32x4 *d = reinterpret_cast<f32x4 *>(base + q * (RP * ld * 4) + off);
        if (o.whole || inside(o, tm, U, q)) {
          if (MODE == WGRAD && p.accumulate && !o.part) v[q][0] += d[0], v[q][1] += d[1];
          d[0] = v[q][0];
          d[1] = v[q][1];
        }
      }
      return;
    }
    auto each = [&](auto f) {
#pragma unroll
      for (int q = 0; q < NP; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[q][i >> 2][i & 3] = f(q, i, v[q][i >> 2][i & 3]);
    };
    u32x4 r[NP];
    auto packed = [&] {
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const float f[8] = {v[q][0][0], v[q][0][1], v[q][0][2], v[q][0][3], v[q][1][0], v[q][1][1], v[q][1][2], v[q][1][3]};
        r[q] = pack(f);
      }
    };
    if constexpr (MODE == FWD) {
      if (p.bias) {
        const u32x4 b = load8(o.cols > 32 * UN * U ? o.bias + 32 * UN * U + 8 * c : p.bias);
        each([&](int, int i, float f) { return f + unpack(b, i); });
      }
      if (p.z) {
        packed();
        store_rows(o, p.z, tm, U, r);
      }
      if (p.act == BQM_ACT_RELU)
        each([](int, int, float f) { return act_f(BQM_ACT_RELU, f); });
      else if (p.act == BQM_ACT_SILU)
        each([](int, int, float f) { return act_f(BQM_ACT_SILU, f); });
      else if (p.act == BQM_ACT_GELU_TANH)
        each([](int, int, float f) { return act_f(BQM_ACT_GELU_TANH, f); });
    } else if constexpr (ZX) {
      if (p.act == BQM_ACT_RELU)
        each([&](int q, int i, float f) { return through_act(BQM_ACT_RELU, f, unpack(x.zx[q], i)); });
      else if (p.act == BQM_ACT_SILU)
        each([&](int q, int i, float f) { return through_act(BQM_ACT_SILU, f, unpack(x.zx[q], i)); });
      else
        each([&](int q, int i, float f) { return through_act(BQM_ACT_GELU_TANH, f, unpack(x.zx[q], i)); });
    }
    if constexpr (ADD) each([&](int q, int i, float f) { return f + unpack(x.add[q], i); });
    packed();
    store_rows(o, p.out, tm, U, r);
  }

  template <int VT, bool ADD, bool ZX>
  __device__ __forceinline__ void store(const Out &o) {
    Extras<ADD, ZX> x0, x1;
    load_extras(o, 0, 0, x0);
#pragma unroll 1
    for (int tm = 0; tm < VT; ++tm) {
      const int next = tm + 1 < VT ? tm + 1 : tm;
      if constexpr (UC == 2) {
        load_extras(o, tm, 1, x1);
        finish_unit<0>(o, tm, x0);
        load_extras(o, next, 0, x0);
        finish_unit<1>(o, tm, x1);
      } else {
        load_extras(o, next, 0, x1);
        finish_unit<0>(o, tm, x0);
        x0 = x1;
      }
    }
  }
  template <int VT>
  __device__ __forceinline__ void store(const Out &o) {
    const bool add = MODE != WGRAD && !o.part && p.add, zx = MODE == DGRAD && !o.part && p.act != BQM_ACT_NONE;
    constexpr bool A = MODE != WGRAD, Z = MODE == DGRAD;
    if (add)
      zx ? store<VT, A, Z>(o) : store<VT, A, false>(o);
    else
      zx ? store<VT, false, Z>(o) : store<VT, false, false>(o);
  }
  template <int VT>
  __device__ __forceinline__ void run_and_store(const Out &o, int k0, int k1) {
    run<VT>(k0, k1);
    store<VT>(o);
  }

  __device__ __forceinline__ void tile(int L, int k0, int k1, float *part) {
    // what follows from the lane is computed anew for each tile: kept across tiles it is
    // spilled, and the wait for its reload lands inside the loop
    asm volatile("" : "+v"(lane));
    const int2 at = tile_at<GM>(p, L);
    const int64_t i0 = (int64_t)at.x * BM, j0 = (int64_t)at.y * BN;
    a.setup(p.a, p.lda, p.C, p.I, i0, lane, w);
    b.setup(p.b, p.ldb, p.C, p.J, j0, lane, w);
    a.setup_fragments(32 * wm);
    b.setup_fragments(32 * TN * wn);
    const int rows = (int)min(p.I - i0, (int64_t)BM), vt = (rows + 32 * WM - 1) / (32 * WM);
    const Out o = out_of(i0, j0, part);
    if (TM == 4 && vt > 3)
      run_and_store<TM>(o, k0, k1);
    else if (TM == 4 && vt > 2)
      run_and_store<TM == 4 ? 3 : TM>(o, k0, k1);
    else if (TM >= 2 && vt > 1)
      run_and_store<TM >= 2 ? 2 : TM>(o, k0, k1);
    else
      run_and_store<1>(o, k0, k1);
    // no copy of this tile lands, and no wave reads a stage, when the next tile's copies begin
    wait_vm<0>();
    barrier_lds();
  }

  static constexpr int GM = TM == 4 ? 4 : 8;
};

// ---------------------------------------------------------------------------
// column sums (the bias gradient)
// ---------------------------------------------------------------------------
// Workgroup n sums rows [y rows, (y + 1) rows) of 64 columns, y = n / (N / 64): 8 lanes of 8
// columns, 32 rows at a time; the 32 partial sums are added in order through LDS.  One part per
// y, or the gradient itself where there is one.
struct ColSums {
  const uint16_t *dz;
  int64_t M, N, rows;
  float *out;
  int accumulate;
};
__device__ __forceinline__ void col_sums(const ColSums &p, int n, float (*s)[65]) {
  const int nx = (int)((p.N + 63) / 64), y = n / nx, x = n - y * nx;
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int64_t col = (int64_t)x * 64 + 8 * c;
  const int64_t r0 = y * p.rows, r1 = min(r0 + p.rows, p.M);
  float v[8] = {};
  if (col < p.N) {
#pragma unroll 8
    for (int64_t r = r0 + g; r < r1; r += 32) {
      const u32x4 d = load8(p.dz + r * p.N + col);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += unpack(d, i);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[g][8 * c + i] = v[i];
  __syncthreads();
  const int64_t at = (int64_t)x * 64 + threadIdx.x;
  if (threadIdx.x < 64 && at < p.N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    float *o = p.out + y * p.N + at;
    *o = p.accumulate ? *o + t : t;
  }
}

// Workgroups b % 8 are one XCD: each walks a contiguous range of tiles, so that the tiles in
// flight there share rows and columns in its L2.  First whole rounds of tiles, one for every
// workgroup; the tiles left over are split along the contraction into S parts, whose FP32 sums
// go to part and are joined by join_parts.  Workgroups behind those of the tiles take the
// column sums.
template <int WM, int TM, int TN, bool AT, bool BT, bool FAST, int OCC, int NSA, int NSB>
__global__ void __launch_bounds__(NTHR, OCC) lin_tiles(LinParams p, ColSums cols) {
  using T = Tile<WM, TM, TN, AT, BT, FAST, NSA, NSB>;
  __shared__ __attribute__((aligned(16))) typename T::Mem sm;
  static_assert(sizeof(sm) >= 32 * 65 * 4, "the column sums' LDS");
  if (AT && BT && (int)blockIdx.x >= p.grid) return col_sums(cols, (int)blockIdx.x - p.grid, reinterpret_cast<float(*)[65]>(&sm));
  T t(p, sm);
  const int x = blockIdx.x & 7, q = blockIdx.x >> 3, nq = p.grid >> 3;
  const int full8 = p.full / 8, items = p.rem * p.S, per8 = (items + 7) / 8;
  for (int L = q; L < full8 + per8; L += nq) {
    int tile = x * full8 + L, s = 0;
    if (L >= full8) {
      const int it = x * per8 + L - full8;
      if (it >= items) break;
      s = it / p.rem;
      tile = p.full + it - s * p.rem;
    }
    const bool split = L >= full8 && p.S > 1;
    const int k0 = split ? s * p.per : 0, k1 = split ? min(k0 + p.per, p.nk) : p.nk;
    // (in scalar registers: the divisions that they come from are done in vector ones)
    float *part = split ? p.part + ((int64_t)(tile - p.full) * p.S + s) * (T::BM * T::BN) : nullptr;
    t.tile(__builtin_amdgcn_readfirstlane(tile), __builtin_amdgcn_readfirstlane(k0), __builtin_amdgcn_readfirstlane(k1), part);
  }
}
#undef LIN_PIN

// The split tiles' parts added in order, then what the others' epilogue does.  HBM and the
// last-level cache bound it: 128 tiles of 256 x 256 in two parts, 18 us, 5.6 TB/s.
template <int BM, int BN, int GM>
__global__ void __launch_bounds__(256) join_parts(LinParams p) {
  constexpr int U = BM * BN / 8, UR = BN / 8;  // units of 8 columns, per row
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int r = (int)(n / U), u = (int)(n % U);
  if (r >= p.rem) return;
  const int2 at = tile_at<GM>(p, p.full + r);
  const int64_t row = (int64_t)at.x * BM + u / UR, col = (int64_t)at.y * BN + 8 * (u % UR);
  if (row >= p.I || col >= p.J) return;
  const float *q = p.part + (int64_t)r * p.S * (BM * BN) + 8 * u;
  u32x4 bias = {};
  if (p.mode == FWD && p.bias) bias = load8(p.bias + col);
  const Extra x = load_extra(p, row * p.J + col);
  f32x4 lo = {}, hi = {};
#pragma unroll 4
  for (int s = 0; s < p.S; ++s, q += BM * BN) {
    lo += reinterpret_cast<const f32x4 *>(q)[0];
    hi += reinterpret_cast<const f32x4 *>(q)[1];
  }
  float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  finish(p, row * p.J + col, v, bias, x);
}

// ---------------------------------------------------------------------------
// the forward of few rows
// ---------------------------------------------------------------------------
// A few rows of x: the weights' bytes bound it, each of which is read once.  A workgroup takes
// 16 rows of w, each of its FW waves every FW-th group of 128 of the contraction, straight from
// memory into the operands of the 16x16x32 MFMA (lane l: row l % 16, elements 8 (l / 16) + 0..7
// of 32; the rows of x past the last stay zeros), with the next group's loads in flight.
// Weights are the first operand, so lane l ends with columns 4 (l / 16) + 0..3 of row l % 16 of
// the result.  The waves' sums are added in their order through LDS.
//
// The weights go through the caches, whose lines are two loads long (past them 8192 x 8192 with one
// row takes 30.8 us, 27.7 through them); lanes without a row of x load none (with all of them 4096 x
// 6144 takes 12.2 us instead of 11.6: 4.3 TB/s).
//
// 1, 4 and 8 rows, against tiles, in us, weights from HBM (copies of 600 MB in all, in turn): of 4096
// x 6144 12.0, 13.4 and 14.6 against 15.9; of 8192 x 8192 32.5, 30.7 and 32.4 against 37.5; of 6144 x
// 2048 9.1, 9.2 and 9.9 against 12.2; of 768 x 2048 5.3, 5.6 and 6.0 against 8.8; of 256 x 1024 3.8,
// 4.0 and 4.1 against 5.6; of 1024 x 4096 7.7, 8.4 and 9.0 against 9.5; with 16 rows of these 17.5,
// 38.3, 11.0, 6.7, 4.5 and 10.2.  From the last-level cache one row of 4096 x 6144 takes 9.9, and 8 of
// 6144 x 2048 9.3 where tiles take 8.7.  A workgroup's stream takes 1.0 us per 1024 of the contraction,
// so that where few of them have long rows the tiles, which split the contraction over idle CUs, are
// ahead: 1, 4 and 8 rows of 1024 x 8192 12.1, 13.3 and 14.7 against 10.8, of 2048 x 8192 14.0, 14.4
// and 15.5 against 12.8.
constexpr int FW = 8, FU = 4;  // waves; MFMA steps of 32 per group

__global__ void __launch_bounds__(64 * FW) lin_few(LinParams p) {
  __shared__ float sum[FW][16][20];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = p.C, M = (int)p.I, N = (int)p.J, n0 = blockIdx.x * 16;
  const int e = 8 * (lane >> 4);
  const uint8_t *wr = p.b + (int64_t)min(n0 + (lane & 15), N - 1) * p.ldb;
  const uint8_t *xr = p.a + (int64_t)(lane & 15) * p.lda;
  f32x4 acc = {};
  u32x4 wf[2][FU], xf[2][FU] = {};
  const bool mine = (lane & 15) < M;
  // group i into set b; what lies past the end of the rows is their last 8 elements again,
  // and zeros before it is used
  auto load = [&](int b, int i) {
#pragma unroll
    for (int u = 0; u < FU; ++u) wf[b][u] = *reinterpret_cast<const u32x4 *>(wr + 2 * min(32 * (FU * i + u) + e, K - 8));
    if (mine) {
#pragma unroll
      for (int u = 0; u < FU; ++u) xf[b][u] = *reinterpret_cast<const u32x4 *>(xr + 2 * min(32 * (FU * i + u) + e, K - 8));
    }
  };
  auto use = [&](int b, int i) {
    if (32 * FU * (i + 1) > K) {
#pragma unroll
      for (int u = 0; u < FU; ++u) {
        const uint32_t in = 32 * (FU * i + u) + e < K ? ~0u : 0u;
        wf[b][u] &= u32x4{in, in, in, in};
        xf[b][u] &= u32x4{in, in, in, in};
      }
    }
#pragma unroll
    for (int u = 0; u < FU; ++u)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wf[b][u]), __builtin_bit_cast(bf16x8, xf[b][u]),
                                                    acc, 0, 0, 0);
  };
  const int groups = (K + 32 * FU - 1) / (32 * FU);
  int i = w;
  if (i < groups) load(0, i);
  for (; i + 2 * FW < groups; i += 2 * FW) {
    load(1, i + FW);
    use(0, i);
    load(0, i + 2 * FW);
    use(1, i + FW);
  }
  if (i + FW < groups) {
    load(1, i + FW);
    use(0, i);
    use(1, i + FW);
  } else if (i < groups) {
    use(0, i);
  }
  *reinterpret_cast<f32x4 *>(&sum[w][lane & 15][4 * (lane >> 4)]) = acc;
  __syncthreads();
  if ((int)threadIdx.x < 2 * M) {
    const int row = threadIdx.x >> 1, c = 8 * (threadIdx.x & 1), col = n0 + c;
    if (col >= N) return;
    const int64_t at = (int64_t)row * N + col;
    u32x4 bias = {};
    if (p.bias) bias = load8(p.bias + col);
    const Extra x = load_extra(p, at);
    float v[8] = {};
#pragma unroll
    for (int q = 0; q < FW; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += sum[q][row][c + i];
    finish(p, at, v, bias, x);
  }
}

__global__ void __launch_bounds__(256) join_cols(const float *part, int64_t N, int parts, float *out, int accumulate) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float t = 0.0f;
#pragma unroll 8
  for (int i = 0; i < parts; ++i) t += part[i * N + n];
  out[n] = accumulate ? out[n] + t : t;
}

// where there is no contraction (no rows): zeros, or what was there
__global__ void __launch_bounds__(256) zero_f32(float *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

// ---------------------------------------------------------------------------
// the gradient through an activation alone
// ---------------------------------------------------------------------------
// 8 elements per lane, once each: HBM bounds it, 16384 x 4096 in 64 us, 6.3 TB/s; 203 x 768 2.9 us.
__global__ void __launch_bounds__(256) act_grad_rows(const uint16_t *dy, const uint16_t *z, int act, int64_t n, uint16_t *dz) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i + 8 <= n) {
    const u32x4 d = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(dy + i));
    const u32x4 q = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(z + i));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = through_act(act, unpack(d, j), unpack(q, j));
    __builtin_nontemporal_store(pack(v), reinterpret_cast<u32x4 *>(dz + i));
  } else {
    for (int64_t j = i; j < n; ++j)
      dz[j] = (uint16_t)pack_bf16_rne(through_act(act, bf16_lo(dy[j]), bf16_lo(z[j])), 0.0f);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bqm_status check_linear(const char *who, int64_t M, int64_t N, int64_t K) {
  BQM_REQUIRE(M >= 0, BQM_ERR_INVALID_ARG, "%s: M < 0", who);
  // (the weight gradient counts rows, rounded up to steps, in 32 bits)
  BQM_REQUIRE(M < ((int64_t)1 << 30), BQM_ERR_SHAPE, "%s: M=%lld reaches 2^30", who, (long long)M);
  BQM_REQUIRE(N >= 8 && N % 8 == 0 && N < (1 << 22), BQM_ERR_SHAPE, "%s: N=%lld is not a multiple of 8 in [8, 2^22)", who,
              (long long)N);
  BQM_REQUIRE(K >= 8 && K % 8 == 0 && K < (1 << 22), BQM_ERR_SHAPE, "%s: K=%lld is not a multiple of 8 in [8, 2^22)", who,
              (long long)K);
  BQM_REQUIRE(cdiv(M, 64) * cdiv(N > K ? N : K, 64) < ((int64_t)1 << 31) && cdiv(N, 64) * cdiv(K, 64) < ((int64_t)1 << 31),
              BQM_ERR_SHAPE, "%s: too many tiles", who);
  return BQM_OK;
}

template <bool AT, bool BT>
bqm_status launch_tiles(LinParams p, const Plan &plan, hipStream_t s, const char *what, const ColSums &cols = {}) {
  p.NI = plan.NI, p.NJ = plan.NJ, p.full = plan.full, p.rem = plan.rem, p.S = plan.S, p.per = plan.per, p.nk = plan.nk;
  const Shape &h = kShapes[plan.shape];
  const int64_t slots = kCUs * h.occ, tiles = (int64_t)plan.full + (int64_t)plan.rem * plan.S;
  p.grid = (int)(cdiv(tiles < slots ? tiles : slots, 8) * 8);
  const unsigned grid = (unsigned)(p.grid + (cols.out ? cdiv(cols.N, 64) * cdiv(cols.M, cols.rows) : 0));
  const unsigned joins = (unsigned)cdiv((int64_t)plan.rem * h.bm * h.bn / 8, 256);
  auto go = [&](auto WM, auto TM, auto TN, auto FAST, auto OCC, auto NSA, auto NSB) {
    lin_tiles<WM.value, TM.value, TN.value, AT, BT, FAST.value, OCC.value, NSA.value, NSB.value><<<grid, NTHR, 0, s>>>(p, cols);
    if (plan.S > 1)
      join_parts<32 * WM.value * TM.value, 32 * (4 / WM.value) * TN.value, TM.value == 4 ? 4 : 8><<<joins, 256, 0, s>>>(p);
  };
  constexpr std::integral_constant<int, 1> n1;
  constexpr std::integral_constant<int, 2> n2;
  constexpr std::integral_constant<int, 3> n3;
  constexpr std::integral_constant<int, 4> n4;
  constexpr std::true_type fast;
  constexpr std::false_type slow;
  if (p.C < 64)
    go(n2, n2, n2, slow, n1, n4, n4);
  else if (plan.shape == 0)
    go(n2, n4, n4, fast, n1, n3, n2);
  else if (plan.shape == 1)
    go(n2, n4, n2, fast, n1, n3, n3);
  else if (plan.shape == 2)
    go(n2, n2, n2, fast, n1, n4, n4);
  else
    go(n2, n1, n1, fast, n2, n4, n4);
  return launch_status(what);
}

bqm_status check_act(const char *who, int32_t act) {
  BQM_REQUIRE(act >= BQM_ACT_NONE && act <= BQM_ACT_GELU_TANH, BQM_ERR_INVALID_ARG, "%s: act=%d is no activation", who, act);
  return BQM_OK;
}

bqm_status check_ws(const char *who, const void *ws, size_t ws_bytes, size_t need) {
  if (need == 0) return BQM_OK;
  BQM_REQUIRE(ws && ws_bytes >= need, BQM_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, ws ? ws_bytes : (size_t)0,
              need);
  BQM_REQUIRE(aligned16(ws), BQM_ERR_ALIGN, "%s: ws not 16-byte aligned", who);
  return BQM_OK;
}

}  // namespace
}  // namespace bqm

using namespace bqm;

extern "C" size_t bqm_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (check_linear("bqm_linear_workspace_size", M, N, K) != BQM_OK || M == 0) return 0;
  return align256((size_t)workspace_floats(M, N, K) * 4);
}

extern "C" bqm_status bqm_linear_fwd(const uint16_t *x, const uint16_t *w, const uint16_t *bias, int32_t act,
                                     const uint16_t *residual, int64_t M, int64_t N, int64_t K, uint16_t *y, uint16_t *z,
                                     void *ws, size_t ws_bytes, void *stream) {
  const char *who = "bqm_linear_fwd";
  bqm_status st = check_linear(who, M, N, K);
  if (st == BQM_OK) st = check_act(who, act);
  if (st != BQM_OK || M == 0) return st;
  BQM_REQUIRE(x && w && y, BQM_ERR_INVALID_ARG, "%s: x, w or y is NULL", who);
  BQM_REQUIRE(aligned16(x) && aligned16(w) && aligned16(bias) && aligned16(residual) && aligned16(y) && aligned16(z),
              BQM_ERR_ALIGN, "%s: pointer not 16-byte aligned", who);
  const bool few = few_rows(M, N, K);
  const Plan plan = few ? Plan{} : plan_fwd(M, N, K);
  st = check_ws(who, ws, ws_bytes, (size_t)plan.part * 4);
  if (st != BQM_OK) return st;
  LinParams p = {};
  p.mode = FWD, p.act = act;
  p.a = reinterpret_cast<const uint8_t *>(x), p.lda = 2 * K, p.I = M;
  p.b = reinterpret_cast<const uint8_t *>(w), p.ldb = 2 * K, p.J = N;
  p.C = (int)K;
  p.bias = bias, p.add = residual, p.out = y, p.z = z, p.part = reinterpret_cast<float *>(ws);
  if (few) {
    lin_few<<<(unsigned)cdiv(N, 16), 64 * FW, 0, as_stream(stream)>>>(p);
    return launch_status(who);
  }
  return launch_tiles<false, false>(p, plan, as_stream(stream), who);
}

extern "C" bqm_status bqm_linear_dgrad(const uint16_t *dz, const uint16_t *w, const uint16_t *zx, int32_t act,
                                       const uint16_t *add, int64_t M, int64_t N, int64_t K, uint16_t *dx, void *ws,
                                       size_t ws_bytes, void *stream) {
  const char *who = "bqm_linear_dgrad";
  bqm_status st = check_linear(who, M, N, K);
  if (st == BQM_OK) st = check_act(who, act);
  if (st != BQM_OK || M == 0) return st;
  BQM_REQUIRE(dz && w && dx, BQM_ERR_INVALID_ARG, "%s: dz, w or dx is NULL", who);
  BQM_REQUIRE(zx || act == BQM_ACT_NONE, BQM_ERR_INVALID_ARG, "%s: an activation needs zx", who);
  BQM_REQUIRE(aligned16(dz) && aligned16(w) && aligned16(zx) && aligned16(add) && aligned16(dx), BQM_ERR_ALIGN,
              "%s: pointer not 16-byte aligned", who);
  const Plan plan = plan_dgrad(M, N, K);
  st = check_ws(who, ws, ws_bytes, (size_t)plan.part * 4);
  if (st != BQM_OK) return st;
  LinParams p = {};
  p.mode = DGRAD, p.act = act;
  p.a = reinterpret_cast<const uint8_t *>(dz), p.lda = 2 * N, p.I = M;
  p.b = reinterpret_cast<const uint8_t *>(w), p.ldb = 2 * K, p.J = K;
  p.C = (int)N;
  p.add = add, p.zx = zx, p.out = dx, p.part = reinterpret_cast<float *>(ws);
  return launch_tiles<false, true>(p, plan, as_stream(stream), who);
}

extern "C" bqm_status bqm_linear_wgrad(const uint16_t *dz, const uint16_t *x, int32_t accumulate, int64_t M, int64_t N,
                                       int64_t K, float *dw, float *dbias, void *ws, size_t ws_bytes, void *stream) {
  const char *who = "bqm_linear_wgrad";
  bqm_status st = check_linear(who, M, N, K);
  if (st != BQM_OK) return st;
  BQM_REQUIRE(dw, BQM_ERR_INVALID_ARG, "%s: dw is NULL", who);
  BQM_REQUIRE((dz && x) || M == 0, BQM_ERR_INVALID_ARG, "%s: dz or x is NULL", who);
  BQM_REQUIRE(aligned16(dz) && aligned16(x) && aligned16(dw) && aligned16(dbias), BQM_ERR_ALIGN,
              "%s: pointer not 16-byte aligned", who);
  const hipStream_t s = as_stream(stream);
  if (M == 0) {  // sums over nothing
    if (accumulate) return BQM_OK;
    zero_f32<<<(unsigned)(cdiv(N * K, 256) < 4096 ? cdiv(N * K, 256) : 4096), 256, 0, s>>>(dw, N * K);
    if (dbias) zero_f32<<<(unsigned)cdiv(N, 256), 256, 0, s>>>(dbias, N);
    return launch_status(who);
  }
  const Plan plan = plan_wgrad(M, N, K);
  const int parts = dbias ? col_parts(M, N) : 1;
  st = check_ws(who, ws, ws_bytes, (size_t)(plan.part + (dbias ? col_floats(M, N) : 0)) * 4);
  if (st != BQM_OK) return st;
  LinParams p = {};
  p.mode = WGRAD, p.accumulate = accumulate != 0;
  p.a = reinterpret_cast<const uint8_t *>(dz), p.lda = 2 * N, p.I = N;
  p.b = reinterpret_cast<const uint8_t *>(x), p.ldb = 2 * K, p.J = K;
  p.C = (int)M;
  p.dw = dw, p.part = reinterpret_cast<float *>(ws);
  ColSums cols = {};
  if (dbias) cols = {dz, M, N, cdiv(M, parts), parts > 1 ? p.part + plan.part : dbias, parts == 1 && p.accumulate};
  st = launch_tiles<true, true>(p, plan, s, who, cols);
  if (st != BQM_OK || parts == 1) return st;
  join_cols<<<(unsigned)cdiv(N, 256), 256, 0, s>>>(cols.out, N, (int)cdiv(M, cols.rows), dbias, p.accumulate);
  return launch_status(who);
}

extern "C" bqm_status bqm_act_grad(const uint16_t *dy, const uint16_t *z, int32_t act, int64_t n, uint16_t *dz,
                                   void *stream) {
  const char *who = "bqm_act_grad";
  bqm_status st = check_act(who, act);
  if (st != BQM_OK) return st;
  BQM_REQUIRE(n >= 0, BQM_ERR_INVALID_ARG, "%s: n < 0", who);
  BQM_REQUIRE(act != BQM_ACT_NONE, BQM_ERR_INVALID_ARG, "%s: BQM_ACT_NONE has no gradient to apply", who);
  // (a launch takes less than 2^32 threads, of 8 elements each)
  BQM_REQUIRE(n < ((int64_t)1 << 34), BQM_ERR_SHAPE, "%s: n reaches 2^34", who);
  if (n == 0) return BQM_OK;
  BQM_REQUIRE(dy && z && dz, BQM_ERR_INVALID_ARG, "%s: dy, z or dz is NULL", who);
  BQM_REQUIRE(aligned16(dy) && aligned16(z) && aligned16(dz), BQM_ERR_ALIGN, "%s: pointer not 16-byte aligned", who);
  act_grad_rows<<<(unsigned)cdiv(n, 2048), 256, 0, as_stream(stream)>>>(dy, z, act, n, dz);
  return launch_status(who);
}
