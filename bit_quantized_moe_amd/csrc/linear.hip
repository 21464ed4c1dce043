// The dense product beside the experts, with bias, activation and residual in its epilogue,
// and its gradients, on gfx950:
//   z = x w^T + b, y = act(z) + residual        x [M, K], w [N, K]   (bqm_linear_fwd)
//   dx = (dz w) act'(zx) + add                  dz [M, N]            (bqm_linear_dgrad)
//   dw = dz^T x, db = sum_m dz                                       (bqm_linear_wgrad)
//   dz = dy act'(z)                                                  (bqm_act_grad)
//
// All three products are C[i, j] = sum_c A(i, c) B(j, c) of bf16 operands on the 32x32x16
// MFMA with FP32 accumulators.  They differ in how an operand lies in memory: with its
// contraction contiguous (x and w in the forward, dz in the input gradient) or as rows of the
// contraction (w in the input gradient, dz and x in the weight gradient); the latter is read
// from LDS transposed.  No transposed copy of a tensor is made.
#include "common.h"

#include <type_traits>

namespace bqm {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int NTHR = 256;  // four waves, one per SIMD
constexpr int KS = 64;     // contraction per step: 128 bytes of a row
constexpr int kCUs = 256;

enum Mode { FWD, DGRAD, WGRAD };

struct LinParams {
  const uint8_t *a, *b;  // operands
  int64_t I, J;          // rows and columns of the result
  int64_t lda, ldb;      // bytes per row of an operand as it is stored
  int C, nk;             // contraction, and its steps
  int NI, NJ;            // tiles
  int full, rem;         // tiles computed whole, and those behind them
  int S, per;            // which are split into S parts of per steps
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
  if (act == BQM_ACT_RELU) return v > 0.0f ? v : 0.0f;
  if (act == BQM_ACT_SILU) return v * sigmoid_f(v);
  return v * sigmoid_f(kGelu * (v + 0.044715f * v * v * v));
}

__device__ __forceinline__ float act_grad_f(int act, float v) {
  if (act == BQM_ACT_RELU) return v > 0.0f ? 1.0f : 0.0f;
  if (act == BQM_ACT_SILU) {
    const float s = sigmoid_f(v);
    return s * (1.0f + v * (1.0f - s));
  }
  // past |v| = 16 the sigmoid is 0 or 1 in FP32 and so is the derivative; v^2 need not be formed
  const float t = fminf(fmaxf(v, -16.0f), 16.0f), q = t * t;
  const float s = sigmoid_f(kGelu * t * (1.0f + 0.044715f * q));
  return s * (1.0f + t * (1.0f - s) * kGelu * (1.0f + 0.134145f * q));
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
    for (int i = 0; i < 8; ++i) v[i] *= act_grad_f(p.act, unpack(x.zx, i));
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
__device__ __forceinline__ void dma_b128(const void *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(uniform(base)), "s"(lds)
               : "memory", "m0");
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
// T = false: [row][128 bytes], the 16-byte chunk c of a row at c ^ ((row >> 1) & 7), so that a
// fragment read (one chunk of 32 rows) falls on different banks.
// T = true: for each 64 result columns [contraction row][128 bytes], chunk c at c ^ 2 (row & 3):
// a transposing read takes 32 bytes of 4 rows per 16 lanes.
// Stages are filled by direct copies of 1 KB (8 of those 128-byte rows) per wave.
template <int R, bool T, bool FAST>
struct Operand {
  static constexpr int kCopies = R / 32;  // per wave and step
  const uint8_t *base;
  int64_t ld;
  uint32_t off[kCopies];
  int C;
  int lane, w;

  // rows: of the whole operand; r0: the tile's first
  __device__ __forceinline__ void setup(const uint8_t *q, int64_t ld_, int C_, int64_t rows, int64_t r0, int lane_, int w_) {
    ld = ld_, C = C_, lane = lane_, w = w_;
    base = uniform(T ? q + 2 * r0 : q + r0 * ld);
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int n = kCopies * w + j;
      if constexpr (T) {
        const int r = 8 * (n & 7) + (lane >> 3), c = 64 * (n >> 3) + 8 * ((lane & 7) ^ (2 * (r & 3)));
        // columns past the last are the last 8 again (their results are dropped)
        const int most = (int)min(rows - r0, (int64_t)R) - 8;
        off[j] = (uint32_t)r * (uint32_t)ld + 2 * min(c, most);
      } else {
        const int r = 8 * n + (lane >> 3), most = (int)min(rows - r0, (int64_t)R) - 1;
        off[j] = (uint32_t)min(r, most) * (uint32_t)ld + 16 * ((lane & 7) ^ ((r >> 1) & 7));
      }
    }
  }

  // copy j of step ks.  FAST: a contraction of at least one whole step; the last step, where
  // it is not whole, takes the last KS of the contraction (and zeroes in registers what the
  // step before had).  Otherwise the one step there is takes zeros past the end.
  __device__ __forceinline__ void copy(int j, int ks, uint8_t *stage) const {
    const uint32_t to = lds_addr(stage) + 1024 * (kCopies * w + j);
    if constexpr (FAST) {
      const int at = min(KS * ks, C - KS);
      dma_b128(base + (T ? at * ld : (int64_t)(2 * at)), off[j], to);
    } else {
      const int n = kCopies * w + j, r = 8 * n + (lane >> 3);
      const bool in = T ? (r & 63) < C : 8 * ((lane & 7) ^ ((r >> 1) & 7)) < C;
      dma_b128(in ? base + off[j] : reinterpret_cast<const uint8_t *>(c_zeros), to);
    }
  }

  // fragment of 32 rows from row c on, slice kk: lane l holds row l % 32, contraction
  // 16 kk + 8 (l / 32) + 0..7
  __device__ __forceinline__ i32x4 fragment(const uint8_t *stage, int c, int kk) const {
    if constexpr (T) {
      const int g = lane >> 4, s = lane & 15;
      const uint8_t *q = stage + (c >> 6) * (KS * 128) + (16 * kk + 8 * (g >> 1) + (s >> 2)) * 128 +
                         16 * (((c & 63) / 8 + 2 * (g & 1) + ((s & 3) >> 1)) ^ (2 * (s >> 2))) + 8 * (s & 1);
      const s16x4 h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(q));
      const s16x4 h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(q + 4 * 128));
      const s16x8 v = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
      return __builtin_bit_cast(i32x4, v);
    } else {
      const int r = c + (lane & 31);
      return *reinterpret_cast<const i32x4 *>(stage + r * 128 + 16 * ((2 * kk + (lane >> 5)) ^ ((r >> 1) & 7)));
    }
  }
};

template <int BM, int BN, int NS>
struct Smem {
  uint8_t a[NS][BM * 128];
  uint8_t b[NS][BN * 128];
};

// ---------------------------------------------------------------------------
// a tile
// ---------------------------------------------------------------------------
// A workgroup of four waves (WM x WN) computes BM = 32 WM TM rows by BN = 32 WN TN columns;
// wave (wm, wn) owns the 32-row tiles WM tm + wm (interleaved, so that a partly filled tile
// leaves all rows of waves the same work) of 32 TN columns.  The contraction goes in steps of
// KS through NS LDS stages; a step is four slices of VT x TN MFMAs.  One wave per SIMD (the
// accumulators of the largest tile take half the register file) has no other wave to hide its
// waits behind, so a step is written out in issue order: each MFMA is followed by its share of
// the fragment reads of the next slice and of the copies of a later step, held there by
// scheduling barriers.  The step's one barrier sits inside slice 3, whose fragments are in
// registers by then; the copies of step ks + NS start behind it, into the stage just read.
//
// Accumulators hold the product transposed (B x A): register v of lane L of tile (tm, tn) is
// row L % 32 and column 8 (v / 4) + 4 (L / 32) + v % 4.
template <int WM, int TM, int TN, bool AT, bool BT, bool FAST, int NS>
struct Tile {
  static constexpr int WN = 4 / WM, BM = 32 * WM * TM, BN = 32 * WN * TN;
  static constexpr int CA = BM / 32, CB = BN / 32, kCopies = CA + CB, kFirst = kCopies / 2;
  const LinParams &p;
  Smem<BM, BN, NS> &sm;
  int lane, w, wm, wn;
  Operand<BM, AT, FAST> a;
  Operand<BN, BT, FAST> b;
  int over;  // of the last step, the leading part that the step before had
  i32x4 af[2][TM], bf[2][TN];
  f32x16 acc[TM][TN];

  __device__ __forceinline__ Tile(const LinParams &p_, Smem<BM, BN, NS> &sm_) : p(p_), sm(sm_) {
    lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = WM == 2 ? w >> 1 : 0;
    wn = WM == 2 ? w & 1 : w;
  }

  __device__ __forceinline__ void copy(int j, int ks) {
    if (j < CA)
      a.copy(j, ks, sm.a[ks & (NS - 1)]);
    else
      b.copy(j - CA, ks, sm.b[ks & (NS - 1)]);
  }
  // the i-th of a slice's reads, in the order its MFMAs ask for them
  __device__ __forceinline__ void read(int k, int i, int kk, int st) {
    if (i == 0 || i > TN) {
      const int tm = i == 0 ? 0 : i - TN;
      af[k][tm] = a.fragment(sm.a[st], 32 * (WM * tm + wm), kk);
    } else {
      bf[k][i - 1] = b.fragment(sm.b[st], 32 * (wn * TN + i - 1), kk);
    }
  }
  __device__ __forceinline__ void mfma(int k, int tm, int tn) {
    acc[tm][tn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, bf[k][tn]),
                                                          __builtin_bit_cast(bf16x8, af[k][tm]), acc[tm][tn], 0, 0, 0);
  }

  // zeros in place of what the step before the last had, in both operands (0 times an
  // infinity would be NaN)
  template <int VT>
  __device__ __forceinline__ void drop_overlap(int kk) {
    if (over <= 16 * kk) return;
    int mask[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = over - (16 * kk + 8 * (lane >> 5) + 2 * i);
      mask[i] = d <= 0 ? -1 : d == 1 ? (int)0xFFFF0000 : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int tm = 0; tm < VT; ++tm) af[kk & 1][tm][i] &= mask[i];
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) bf[kk & 1][tn][i] &= mask[i];
    }
  }

  // LEFT: steps that follow, NS for that or more.
  // slices 0-2: fragment reads of the next slice; in slice 0 first the copies that slice 3 of
  // the step before has not begun
  template <int VT, int KK, int LEFT>
  __device__ __forceinline__ void slice(int ks) {
    if constexpr (FAST && LEFT == 0) drop_overlap<VT>(KK);
    constexpr int NP = VT * TN, NC = KK == 0 && LEFT >= NS - 1 ? kCopies - kFirst : 0, NI = NC + TN + VT;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      mfma(KK & 1, q / TN, q % TN);
#pragma unroll
      for (int i = q * NI / NP; i < (q + 1) * NI / NP; ++i) {
        if (i < NC)
          copy(kFirst + i, ks - 1 + NS);
        else
          read((KK + 1) & 1, i - NC, KK + 1, ks & (NS - 1));
      }
      LIN_PIN();
    }
  }
  template <int VT, int LEFT>
  __device__ __forceinline__ void slice3(int ks) {
    if constexpr (FAST && LEFT == 0) drop_overlap<VT>(3);
    constexpr int NP = VT * TN, NR = TN + VT, NC = LEFT >= NS ? kFirst : 0, NI = NR + NC;
    constexpr int both = NC < NR ? NC : NR;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      mfma(1, q / TN, q % TN);
      if constexpr (LEFT > 0) {
        if (q == 0) {
          // every wave is done reading this stage, and the next is whole
          LIN_PIN();
          wait_vm<(LEFT - 1 < NS - 2 ? LEFT - 1 : NS - 2) * kCopies>();
          barrier_lds();
          LIN_PIN();
        }
#pragma unroll
        for (int i = q * NI / NP; i < (q + 1) * NI / NP; ++i) {
          // in turn a copy and a read, as long as there are both
          const bool isc = i < 2 * both ? !(i & 1) : NC > both;
          const int j = i < 2 * both ? i >> 1 : i - both;
          if (isc)
            copy(j, ks + NS);
          else
            read(0, j, 0, (ks + 1) & (NS - 1));
        }
      }
      LIN_PIN();
    }
  }
  template <int VT, int LEFT>
  __device__ __forceinline__ void step(int ks) {
    slice<VT, 0, LEFT>(ks);
    slice<VT, 1, LEFT>(ks);
    slice<VT, 2, LEFT>(ks);
    slice3<VT, LEFT>(ks);
  }
  template <int VT, int LEFT>
  __device__ __forceinline__ void tail(int &ks, int last) {
    if (last - ks == LEFT) step<VT, LEFT>(ks++);
    if constexpr (LEFT > 0) tail<VT, LEFT - 1>(ks, last);
  }

  // steps [k0, k1) of the tile at (i0, j0), of which VT row tiles per wave hold rows
  template <int VT>
  __device__ __forceinline__ void run(int k0, int k1) {
#pragma unroll
    for (int tm = 0; tm < VT; ++tm)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[tm][tn][v] = 0.0f;
    over = FAST && k1 == p.nk ? KS * p.nk - p.C : 0;
    const int last = k1 - 1;
#pragma unroll
    for (int q = 0; q < NS - 1; ++q)
      if (k0 + q <= last) {
#pragma unroll
        for (int j = 0; j < kCopies; ++j) copy(j, k0 + q);
      }
    if (NS == 2 || last - k0 < NS - 2)
      wait_vm<0>();
    else
      wait_vm<(NS - 2) * kCopies>();
    barrier_lds();
#pragma unroll
    for (int i = 0; i < TN + VT; ++i) read(0, i, 0, k0 & (NS - 1));
    if (k0 + NS - 1 <= last) {
#pragma unroll
      for (int j = 0; j < kFirst; ++j) copy(j, k0 + NS - 1);
    }
    int ks = k0;
    for (; ks + NS <= last; ++ks) step<VT, NS>(ks);
    tail<VT, NS - 1>(ks, last);
  }

  // 32 rows of the wave to its part t of LDS
  template <int TMX>
  __device__ __forceinline__ void put(uint8_t *t) const {
    constexpr int CH = 8 * TN;
    const int r = lane & 31;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4 *>(t + 16 * (r * CH + ((8 * tn + 2 * q + (lane >> 5)) ^ (r & (CH - 1))))) =
            f32x4{acc[TMX][tn][4 * q], acc[TMX][tn][4 * q + 1], acc[TMX][tn][4 * q + 2], acc[TMX][tn][4 * q + 3]};
  }

  // The accumulators hold 4 columns of 32 rows a lane quarter.  They pass through LDS in FP32,
  // 32 rows of a wave at a time, so that a lane finishes 8 consecutive columns of a row and
  // reads and writes 16 bytes at a time (chunk c of row r at c ^ (r & its number of chunks - 1)).
  __device__ __forceinline__ void store(int vt, int64_t i0, int64_t j0, float *part) {
    constexpr int CH = 8 * TN, LPR = 4 * TN, RP = 64 / LPR, NP = 32 / RP, UN = 4;
    static_assert(sizeof(sm.a) + sizeof(sm.b) >= 4 * 32 * CH * 16, "the waves' parts fit the stages");
    uint8_t *t = sm.a[0] + w * (32 * CH * 16);
    const int lr = lane / LPR, c = lane % LPR;
    const int col = 32 * TN * wn + 8 * c;
    const bool cin = j0 + col < p.J;
    u32x4 bias = {};
    if (!part && p.mode == FWD && p.bias && cin) bias = load8(p.bias + j0 + col);
    barrier_lds();  // every wave is done with the stages
#pragma unroll 1
    for (int tm = 0; tm < vt; ++tm) {
      const int r0 = 32 * (WM * tm + wm);
      if (TM == 1 || tm == 0)
        put<0>(t);
      else if (TM == 2 || tm == 1)
        put<TM < 2 ? 0 : 1>(t);
      else if (tm == 2)
        put<TM < 4 ? 0 : 2>(t);
      else
        put<TM < 4 ? 0 : 3>(t);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
      for (int q0 = 0; q0 < NP; q0 += UN) {
        Extra x[UN];
        f32x4 lo[UN], hi[UN];
#pragma unroll
        for (int q = 0; q < UN; ++q) {
          const int64_t row = i0 + r0 + (q0 + q) * RP + lr;
          if (!part && cin && row < p.I) x[q] = load_extra(p, row * p.J + j0 + col);
        }
#pragma unroll
        for (int q = 0; q < UN; ++q) {
          const int rr = (q0 + q) * RP + lr;
          lo[q] = *reinterpret_cast<const f32x4 *>(t + 16 * (rr * CH + ((2 * c) ^ (rr & (CH - 1)))));
          hi[q] = *reinterpret_cast<const f32x4 *>(t + 16 * (rr * CH + ((2 * c + 1) ^ (rr & (CH - 1)))));
        }
#pragma unroll
        for (int q = 0; q < UN; ++q) {
          const int rr = (q0 + q) * RP + lr;
          const int64_t row = i0 + r0 + rr;
          if (cin && row < p.I) {
            if (part) {
              f32x4 *o = reinterpret_cast<f32x4 *>(part + (r0 + rr) * BN + col);
              o[0] = lo[q];
              o[1] = hi[q];
            } else {
              float v[8] = {lo[q][0], lo[q][1], lo[q][2], lo[q][3], hi[q][0], hi[q][1], hi[q][2], hi[q][3]};
              finish(p, row * p.J + j0 + col, v, bias, x[q]);
            }
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    barrier_lds();  // the stages are free for the next tile
  }

  __device__ __forceinline__ void tile(int L, int k0, int k1, float *part) {
    // what follows from the lane is computed anew for each tile: kept across tiles it is
    // spilled, and the wait for its reload lands inside the loop
    asm volatile("" : "+v"(lane));
    const int2 at = tile_at<GM>(p, L);
    const int64_t i0 = (int64_t)at.x * BM, j0 = (int64_t)at.y * BN;
    a.setup(p.a, p.lda, p.C, p.I, i0, lane, w);
    b.setup(p.b, p.ldb, p.C, p.J, j0, lane, w);
    const int rows = (int)min(p.I - i0, (int64_t)BM), vt = (rows + 32 * WM - 1) / (32 * WM);
    if (TM == 4 && vt > 3)
      run<TM>(k0, k1);
    else if (TM == 4 && vt > 2)
      run<TM == 4 ? 3 : TM>(k0, k1);
    else if (TM >= 2 && vt > 1)
      run<TM >= 2 ? 2 : TM>(k0, k1);
    else
      run<1>(k0, k1);
    store(vt, i0, j0, part);
  }

  static constexpr int GM = TM == 4 ? 4 : 8;
  // row and column tile of tile L: groups of about G row tiles, column by column
  template <int G>
  __device__ __forceinline__ static int2 tile_at(const LinParams &p, int L) {
    const int n_g = max((p.NI + G / 2) / G, 1), g = (p.NI + n_g - 1) / n_g;
    const int m_first = L / (g * p.NJ) * g, gm = min(g, p.NI - m_first), in_g = L - m_first * p.NJ;
    return make_int2(m_first + in_g % gm, in_g / gm);
  }
};

// Workgroups b % 8 are one XCD: each walks a contiguous range of tiles, so that the tiles in
// flight there share rows and columns in its L2.  First whole rounds of tiles, one for every
// workgroup; the tiles left over are split along the contraction into S parts, whose FP32 sums
// go to part and are joined by join_parts.
template <int WM, int TM, int TN, bool AT, bool BT, bool FAST, int OCC, int NS>
__global__ void __launch_bounds__(NTHR, OCC) lin_tiles(LinParams p) {
  using T = Tile<WM, TM, TN, AT, BT, FAST, NS>;
  __shared__ __attribute__((aligned(16))) Smem<T::BM, T::BN, NS> sm;
  T t(p, sm);
  const int x = blockIdx.x & 7, q = blockIdx.x >> 3, nq = gridDim.x >> 3;
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
    t.tile(tile, k0, k1, split ? p.part + ((int64_t)(tile - p.full) * p.S + s) * (T::BM * T::BN) : nullptr);
  }
}
#undef LIN_PIN

// the split tiles' parts added in order, then what the others' epilogue does
template <int BM, int BN, int GM>
__global__ void __launch_bounds__(256) join_parts(LinParams p) {
  constexpr int U = BM * BN / 8, UR = BN / 8;  // units of 8 columns, per row
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int r = (int)(n / U), u = (int)(n % U);
  if (r >= p.rem) return;
  const int2 at = Tile<2, BM / 64, BN / 64, false, false, true, 2>::template tile_at<GM>(p, p.full + r);
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
// column sums (the bias gradient)
// ---------------------------------------------------------------------------
// A workgroup sums rows [y rows, (y + 1) rows) of 64 columns: 8 lanes of 8 columns, 32 rows at
// a time; the 32 partial sums are added in order through LDS.  One part per workgroup, or the
// gradient itself where there is one.
__global__ void __launch_bounds__(256) col_sums(const uint16_t *dz, int64_t M, int64_t N, int64_t rows, float *out,
                                                int accumulate) {
  __shared__ float s[32][65];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int64_t col = (int64_t)blockIdx.x * 64 + 8 * c;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = min(r0 + rows, M);
  float v[8] = {};
  if (col < N) {
#pragma unroll 4
    for (int64_t r = r0 + g; r < r1; r += 32) {
      const u32x4 d = load8(dz + r * N + col);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += unpack(d, i);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[g][8 * c + i] = v[i];
  __syncthreads();
  const int64_t n = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x < 64 && n < N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    float *o = out + (int64_t)blockIdx.y * N + n;
    *o = accumulate ? *o + t : t;
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
__global__ void __launch_bounds__(256) act_grad_rows(const uint16_t *dy, const uint16_t *z, int act, int64_t n, uint16_t *dz) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i + 8 <= n) {
    const u32x4 d = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(dy + i));
    const u32x4 q = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(z + i));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = unpack(d, j) * act_grad_f(act, unpack(q, j));
    __builtin_nontemporal_store(pack(v), reinterpret_cast<u32x4 *>(dz + i));
  } else {
    for (int64_t j = i; j < n; ++j)
      dz[j] = (uint16_t)pack_bf16_rne(bf16_lo(dy[j]) * act_grad_f(act, bf16_lo(z[j])), 0.0f);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bqm_status check_linear(const char *who, int64_t M, int64_t N, int64_t K) {
  BQM_REQUIRE(M >= 0, BQM_ERR_INVALID_ARG, "%s: M < 0", who);
  BQM_REQUIRE(M < ((int64_t)1 << 31), BQM_ERR_SHAPE, "%s: M=%lld reaches 2^31", who, (long long)M);
  BQM_REQUIRE(N >= 8 && N % 8 == 0 && N < (1 << 22), BQM_ERR_SHAPE, "%s: N=%lld is not a multiple of 8 in [8, 2^22)", who,
              (long long)N);
  BQM_REQUIRE(K >= 8 && K % 8 == 0 && K < (1 << 22), BQM_ERR_SHAPE, "%s: K=%lld is not a multiple of 8 in [8, 2^22)", who,
              (long long)K);
  BQM_REQUIRE(cdiv(M, 64) * cdiv(N > K ? N : K, 64) < ((int64_t)1 << 31) && cdiv(N, 64) * cdiv(K, 64) < ((int64_t)1 << 31),
              BQM_ERR_SHAPE, "%s: too many tiles", who);
  return BQM_OK;
}

// A tile's size, its workgroups per CU, and what a step of it and the rest of it take (in ns,
// with every workgroup slot busy)
struct Shape {
  int bm, bn, occ;
  float step, rest;
};
constexpr Shape kShapes[3] = {{256, 256, 1, 1000, 8000}, {128, 128, 2, 800, 4000}, {64, 128, 3, 800, 4000}};

struct Plan {
  int shape, NI, NJ, full, rem, S, per, nk;
  int64_t part;  // floats of the workspace
};

Plan plan_of(int64_t I, int64_t J, int64_t C) {
  Plan best = {};
  float least = 0.0f;
  const int nk = (int)cdiv(C, KS);
  for (int h = 0; h < 3; ++h) {
    const Shape &s = kShapes[h];
    if (C < KS && h != 1) continue;
    const int64_t NI = cdiv(I, s.bm), NJ = cdiv(J, s.bn), slots = kCUs * s.occ;
    const int64_t full = NI * NJ / slots * slots, rem = NI * NJ - full;
    for (int S = 1; S <= (rem ? 32 : 1); ++S) {
      if (S > 1 && (rem * S > slots || cdiv(nk, S) < 2)) break;
      const int per = (int)cdiv(nk, S);
      if (S > 1 && (int64_t)per * (S - 1) >= nk) continue;  // a part without steps
      float t = full / slots * (nk * s.step + s.rest);
      if (rem) t += per * s.step + s.rest;
      if (S > 1) t += 5000.0f + 2.0f * rem * S * s.bm * s.bn * 4 / 4000.0f;  // a launch; 4 TB/s
      if (least == 0.0f || t < least) {
        least = t;
        best = {h, (int)NI, (int)NJ, (int)full, (int)rem, S, per, nk, S > 1 ? rem * S * s.bm * s.bn : 0};
      }
    }
  }
  return best;
}

// row parts of the column sums
int col_parts(int64_t M, int64_t N) {
  const int64_t most = 2048 / cdiv(N, 64), want = cdiv(M, 256);
  const int64_t n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n);
}

// floats of the workspace that a direction takes
int64_t wgrad_floats(int64_t M, int64_t N, int64_t K) {
  const int parts = col_parts(M, N);
  const int64_t a = plan_of(N, K, M).part, b = parts > 1 ? parts * N : 0;
  return a + b;
}
size_t ws_size(int64_t floats) { return align256((size_t)floats * 4); }

template <bool AT, bool BT>
bqm_status launch_tiles(LinParams p, const Plan &plan, hipStream_t s, const char *what) {
  p.NI = plan.NI, p.NJ = plan.NJ, p.full = plan.full, p.rem = plan.rem, p.S = plan.S, p.per = plan.per, p.nk = plan.nk;
  const Shape &h = kShapes[plan.shape];
  const int64_t slots = kCUs * h.occ, items = plan.full ? slots : (int64_t)plan.rem * plan.S;
  const unsigned grid = (unsigned)(cdiv(items < slots ? items : slots, 8) * 8);
  if (p.C < KS)
    lin_tiles<2, 2, 2, AT, BT, false, 2, 2><<<grid, NTHR, 0, s>>>(p);
  else if (plan.shape == 0)
    lin_tiles<2, 4, 4, AT, BT, true, 1, 2><<<grid, NTHR, 0, s>>>(p);
  else if (plan.shape == 1)
    lin_tiles<2, 2, 2, AT, BT, true, 2, 2><<<grid, NTHR, 0, s>>>(p);
  else
    lin_tiles<2, 1, 2, AT, BT, true, 3, 2><<<grid, NTHR, 0, s>>>(p);
  if (plan.S > 1) {
    const unsigned n = (unsigned)cdiv((int64_t)plan.rem * h.bm * h.bn / 8, 256);
    if (plan.shape == 0)
      join_parts<256, 256, 4><<<n, 256, 0, s>>>(p);
    else if (plan.shape == 1)
      join_parts<128, 128, 8><<<n, 256, 0, s>>>(p);
    else
      join_parts<64, 128, 8><<<n, 256, 0, s>>>(p);
  }
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
  int64_t most = plan_of(M, N, K).part;
  const int64_t d = plan_of(M, K, N).part, w = wgrad_floats(M, N, K);
  most = d > most ? d : most;
  return ws_size(w > most ? w : most);
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
  const Plan plan = plan_of(M, N, K);
  st = check_ws(who, ws, ws_bytes, (size_t)plan.part * 4);
  if (st != BQM_OK) return st;
  LinParams p = {};
  p.mode = FWD, p.act = act;
  p.a = reinterpret_cast<const uint8_t *>(x), p.lda = 2 * K, p.I = M;
  p.b = reinterpret_cast<const uint8_t *>(w), p.ldb = 2 * K, p.J = N;
  p.C = (int)K;
  p.bias = bias, p.add = residual, p.out = y, p.z = z, p.part = reinterpret_cast<float *>(ws);
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
  const Plan plan = plan_of(M, K, N);
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
  const Plan plan = plan_of(N, K, M);
  const int parts = dbias ? col_parts(M, N) : 1;
  st = check_ws(who, ws, ws_bytes, (size_t)(plan.part + (parts > 1 ? parts * N : 0)) * 4);
  if (st != BQM_OK) return st;
  LinParams p = {};
  p.mode = WGRAD, p.accumulate = accumulate != 0;
  p.a = reinterpret_cast<const uint8_t *>(dz), p.lda = 2 * N, p.I = N;
  p.b = reinterpret_cast<const uint8_t *>(x), p.ldb = 2 * K, p.J = K;
  p.C = (int)M;
  p.dw = dw, p.part = reinterpret_cast<float *>(ws);
  st = launch_tiles<true, true>(p, plan, s, who);
  if (st != BQM_OK || !dbias) return st;
  float *cols = parts > 1 ? p.part + plan.part : dbias;
  const dim3 grid((unsigned)cdiv(N, 64), (unsigned)parts);
  col_sums<<<grid, 256, 0, s>>>(dz, M, N, cdiv(M, parts), cols, parts == 1 && p.accumulate);
  if (parts > 1) join_cols<<<(unsigned)cdiv(N, 256), 256, 0, s>>>(cols, N, parts, dbias, p.accumulate);
  return launch_status(who);
}

extern "C" bqm_status bqm_act_grad(const uint16_t *dy, const uint16_t *z, int32_t act, int64_t n, uint16_t *dz,
                                   void *stream) {
  const char *who = "bqm_act_grad";
  bqm_status st = check_act(who, act);
  if (st != BQM_OK) return st;
  BQM_REQUIRE(n >= 0, BQM_ERR_INVALID_ARG, "%s: n < 0", who);
  BQM_REQUIRE(act != BQM_ACT_NONE, BQM_ERR_INVALID_ARG, "%s: BQM_ACT_NONE has no gradient to apply", who);
  BQM_REQUIRE(n < ((int64_t)1 << 35), BQM_ERR_SHAPE, "%s: n reaches 2^35", who);
  if (n == 0) return BQM_OK;
  BQM_REQUIRE(dy && z && dz, BQM_ERR_INVALID_ARG, "%s: dy, z or dz is NULL", who);
  BQM_REQUIRE(aligned16(dy) && aligned16(z) && aligned16(dz), BQM_ERR_ALIGN, "%s: pointer not 16-byte aligned", who);
  act_grad_rows<<<(unsigned)cdiv(n, 2048), 256, 0, as_stream(stream)>>>(dy, z, act, n, dz);
  return launch_status(who);
}
