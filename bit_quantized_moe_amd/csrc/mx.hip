// The experts' product over MXFP4 activations and MXFP4 weights, and its input gradient
// through the dequantized weights, on gfx950.
//
//   y[pos, n]  = sum_k X[row(pos), k] W[e, n, k]       (bqm_mxfp4_gemm)
//   dx[pos, k] = sum_n dY[row(pos), n] W[e, n, k]      (bqm_mxfp4_dgrad)
//
// for the routed rows pos of expert e, offsets[e] <= pos < offsets[e + 1], with row(pos) =
// perm[pos] / k or pos itself.  The forward contracts along the blocks of both operands,
// which is what the block-scaled MFMA multiplies: 32x32x64, one E8M0 scale per operand row
// and 32 of k, at four times the bf16 rate, FP32 accumulation.  The gradient contracts
// across the weight's blocks, so its weights are decoded to bf16 (exact) and multiplied
// with bf16 dY; no second, columnwise copy of the weights exists.
#include "common.h"

#include <type_traits>

namespace bqm {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kMaxE = 1024;
constexpr int NTHR = 256;  // four waves, one per SIMD

struct MxParams {
  const uint8_t *xc, *xs;  // MXFP4 activations (forward)
  const uint16_t *dy;      // bf16 output gradients (dgrad)
  int64_t xrows;
  const uint8_t *wc, *ws;  // MXFP4 weights [E, N, K]
  const int32_t *offsets, *perm;
  int E, k, N, K, NT;
  int64_t R;
  uint16_t *out;
};

// ---------------------------------------------------------------------------
// copies and waits
// ---------------------------------------------------------------------------
// Direct-to-LDS copy: lane i's 16 bytes land at lds + 16 i.  Inline assembly, so that the
// compiler's wait counts do not drain every LDS read before each use of an LDS result; the
// copies are waited for with wait_vm before their stage is read.
__device__ __forceinline__ void dma_b128(const void *g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(g), "s"(lds) : "memory", "m0");
}
// workgroup barrier that orders LDS without draining outstanding copies
__device__ __forceinline__ void barrier_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
__device__ __forceinline__ uint32_t lds_addr(const void *p) { return (uint32_t)(uintptr_t)(const lds_void *)p; }

// 16 zero bytes for the parts of a K step past the end of a row
__device__ __align__(16) const uint32_t c_zeros[4] = {0u, 0u, 0u, 0u};

// Rows of 128 bytes in LDS hold their 16-byte chunk c at c ^ ((row >> 1) & 7): the lanes
// of a fragment read (one chunk of consecutive rows) then fall on different banks.
__device__ __forceinline__ int swz(int row, int c) { return row * 128 + 16 * (c ^ ((row >> 1) & 7)); }

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// First rows of the experts' segments, clamped to [0, R] and non-decreasing
__device__ __forceinline__ int seg_at(const MxParams &p, int e) {
  const int64_t v = p.offsets[e];
  return (int)(v < 0 ? 0 : (v > p.R ? p.R : v));
}

// toff[e] = BM-row tiles of the experts before e, for e = 0 .. E; returns their total
template <int BM>
__device__ int tile_prefix(const MxParams &p, int *toff, int *wsum) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int PER = kMaxE / NTHR;
  int c[PER], run = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    int n = 0;
    if (e < p.E) n = seg_at(p, e + 1) - seg_at(p, e);
    c[i] = n > 0 ? (n + BM - 1) / BM : 0;
    run += c[i];
  }
  int inc = run;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(inc, o, 64);
    if (lane >= o) inc += t;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int q = 0; q < NTHR / 64; ++q) {
    if (q < wave) base += wsum[q];
    total += wsum[q];
  }
  int ex = base + inc - run;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e <= p.E) toff[e] = ex;
    ex += c[i];
  }
  if (p.E == kMaxE && tid == 0) toff[kMaxE] = total;
  __syncthreads();
  return total;
}

// the expert whose tiles hold row tile mt
__device__ __forceinline__ int expert_of_tile(const int *toff, int E, int mt) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (toff[mid] <= mt)
      lo = mid;
    else
      hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// source row of routed position pos, kept inside the tensor
__device__ __forceinline__ int64_t src_row(const MxParams &p, int64_t pos) {
  int64_t r = p.perm ? (int64_t)(p.perm[pos] / p.k) : pos;
  r = r < 0 ? 0 : r;
  return r < p.xrows ? r : p.xrows - 1;
}

// Accumulators hold the product transposed (weights x activations): register v of lane L of
// tile (tm, tn) is row tm * 32 + L % 32 and column tn * 32 + 8 (v / 4) + 4 (L / 32) + v % 4,
// so a lane stores 4 consecutive columns of one row at a time.
template <int TM, int TN>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[TM][TN], uint16_t *out, int64_t ld, int64_t row_base,
                                           int rows, int col_base, int ncols, int lane) {
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const int r = tm * 32 + (lane & 31);
    if (r < rows) {
      uint16_t *o = out + (row_base + r) * ld;
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = col_base + tn * 32 + 8 * q + 4 * (lane >> 5);
          if (n < ncols)
            *reinterpret_cast<uint2 *>(o + n) = make_uint2(pack_bf16_rne(acc[tm][tn][4 * q], acc[tm][tn][4 * q + 1]),
                                                           pack_bf16_rne(acc[tm][tn][4 * q + 2], acc[tm][tn][4 * q + 3]));
        }
    }
  }
}

template <int TM, int TN>
__device__ __forceinline__ void clear_acc(f32x16 (&acc)[TM][TN]) {
#pragma unroll
  for (int tm = 0; tm < TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[tm][tn][v] = 0.0f;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// A workgroup computes BM = 32 TM rows by 256 columns of one expert; each of its four waves
// all rows of 64 columns.  K steps of 256 (128 bytes of codes per row, eight MX blocks) go
// through two LDS stages filled by direct-to-LDS copies one step ahead.  The scales of two
// steps (16 bytes a row) are loaded to registers and written to LDS regrouped: for each step
// and half g of a wave, the four scales of a row's blocks g, 2 + g, 4 + g, 6 + g as one word,
// so that a lane reads one word per operand row and step and the MFMA picks its byte.
constexpr int BN = 256, BK = 256;

template <int TM>
struct FwdSmem {
  uint8_t a[2][32 * TM * 128];
  uint8_t b[2][BN * 128];
  uint32_t s[2][2][2][32 * TM + BN];  // [group parity][step of the group][half][row]
  int toff[kMaxE + 1];
  int wsum[NTHR / 64];
};

// the 16 scale bytes of blocks 16 g .. of a row with nb blocks (127 = 2^0 past its end)
__device__ __forceinline__ u32x4 load_scales(const uint8_t *row, int g, int nb) {
  const uint8_t *p = row + 16 * g;
  if ((nb & 15) == 0) return *reinterpret_cast<const u32x4 *>(p);
  u32x4 v = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
  if ((nb & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (16 * g + 4 * i < nb) v[i] = *reinterpret_cast<const uint32_t *>(p + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (16 * g + i < nb) v[i >> 2] = (v[i >> 2] & ~(0xFFu << (8 * (i & 3)))) | ((uint32_t)p[i] << (8 * (i & 3)));
  }
  return v;
}

template <int TM>
__global__ void __launch_bounds__(NTHR, 1) mx_gemm(MxParams p) {
  constexpr int BM = 32 * TM, TN = 2;
  constexpr int AR = BM / 32;  // copies of 8 rows per wave: BM / 4 waves / 8
  __shared__ __attribute__((aligned(16))) FwdSmem<TM> sm;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int total = tile_prefix<BM>(p, sm.toff, sm.wsum) * p.NT;
  // each XCD (workgroups b % 8) walks a contiguous range of tiles, so that the tiles in
  // flight there share an expert's rows and weights in its L2
  const int per = (total + 7) / 8;
  const int first = (blockIdx.x & 7) * per, last = min(first + per, total);
  const int nb = p.K / 32, nk = (p.K + BK - 1) / BK;
  for (int L = first + (int)(blockIdx.x >> 3); L < last; L += (int)(gridDim.x >> 3)) {
    const int mt = L / p.NT, nt = L % p.NT;
    const int e = expert_of_tile(sm.toff, p.E, mt);
    const int rb = seg_at(p, e), n_e = seg_at(p, e + 1) - rb;
    const int m0 = (mt - sm.toff[e]) * BM, n0 = nt * BN;
    const int rows = min(n_e - m0, BM);
    const int vt = (rows + 31) / 32;
    // copy sources at step 0
    const uint8_t *asrc[AR], *bsrc[8];
    const int lc = lane & 7;  // position of this lane's chunk in its row
    const uint8_t *wc = p.wc + (int64_t)e * p.N * (p.K / 2), *ws = p.ws + (int64_t)e * p.N * nb;
#pragma unroll
    for (int j = 0; j < AR; ++j) {
      const int r = 8 * (AR * w + j) + (lane >> 3);
      asrc[j] = p.xc + src_row(p, (int64_t)rb + min(m0 + r, n_e - 1)) * (p.K / 2);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 8 * (8 * w + j) + (lane >> 3);
      bsrc[j] = wc + (int64_t)min(n0 + r, p.N - 1) * (p.K / 2);
    }
    // the rows whose scales this thread carries: weight row tid, and activation row tid
    const uint8_t *bs = ws + (int64_t)min(n0 + tid, p.N - 1) * nb;
    const uint8_t *as = tid < BM ? p.xs + src_row(p, (int64_t)rb + min(m0 + tid, n_e - 1)) * nb : nullptr;
    auto copy = [&](int ks, int st) {
#pragma unroll
      for (int j = 0; j < AR; ++j) {
        const int r = 8 * (AR * w + j) + (lane >> 3), c = 8 * ks + (lc ^ ((r >> 1) & 7));
        dma_b128(c < nb ? asrc[j] + 16 * c : reinterpret_cast<const uint8_t *>(c_zeros),
                 lds_addr(sm.a[st]) + 1024 * (AR * w + j));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = 8 * (8 * w + j) + (lane >> 3), c = 8 * ks + (lc ^ ((r >> 1) & 7));
        dma_b128(c < nb ? bsrc[j] + 16 * c : reinterpret_cast<const uint8_t *>(c_zeros),
                 lds_addr(sm.b[st]) + 1024 * (8 * w + j));
      }
    };
    auto put_scales = [&](const u32x4 &v, int buf, int row) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sm.s[buf][h][0][row] = __builtin_amdgcn_perm(v[2 * h + 1], v[2 * h], 0x06040200u);
        sm.s[buf][h][1][row] = __builtin_amdgcn_perm(v[2 * h + 1], v[2 * h], 0x07050301u);
      }
    };
    f32x16 acc[TM][TN];
    clear_acc(acc);
    __syncthreads();  // the stages of the tile before are free
    u32x4 sa = {}, sb = load_scales(bs, 0, nb);
    if (tid < BM) sa = load_scales(as, 0, nb);
    copy(0, 0);
    put_scales(sb, 0, BM + tid);
    if (tid < BM) put_scales(sa, 0, tid);
    for (int ks = 0; ks < nk; ++ks) {
      const int st = ks & 1;
      wait_vm<0>();
      barrier_lds();
      const bool odd = ks & 1, more = ks + 1 < nk;
      if (!odd && ks + 2 < nk) {  // the next group's scales, written at the end of the odd step
        sb = load_scales(bs, (ks >> 1) + 1, nb);
        if (tid < BM) sa = load_scales(as, (ks >> 1) + 1, nb);
      }
      if (more) copy(ks + 1, st ^ 1);
      const uint32_t *sw = sm.s[(ks >> 1) & 1][ks & 1][lane >> 5];
      int ssa[TM], ssb[TN];
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) ssa[tm] = (int)sw[tm * 32 + (lane & 31)];
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) ssb[tn] = (int)sw[BM + 64 * w + tn * 32 + (lane & 31)];
      auto slice = [&](auto KK) {
        constexpr int kk = KK.value;
        const int c = 2 * kk + (lane >> 5);
        i32x4 bf[TN];
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
          bf[tn] = *reinterpret_cast<const i32x4 *>(sm.b[st] + swz(64 * w + tn * 32 + (lane & 31), c));
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
          const i32x4 af = *reinterpret_cast<const i32x4 *>(sm.a[st] + swz(tm * 32 + (lane & 31), c));
          const i32x8 a8 = {af[0], af[1], af[2], af[3], 0, 0, 0, 0};
          if (tm < vt) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn) {
              const i32x8 b8 = {bf[tn][0], bf[tn][1], bf[tn][2], bf[tn][3], 0, 0, 0, 0};
              acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[tm][tn], 4, 4, kk, ssb[tn], kk,
                                                                            ssa[tm]);
            }
          }
        }
      };
      slice(std::integral_constant<int, 0>{});
      slice(std::integral_constant<int, 1>{});
      slice(std::integral_constant<int, 2>{});
      slice(std::integral_constant<int, 3>{});
      if (odd && more) {
        put_scales(sb, ((ks >> 1) + 1) & 1, BM + tid);
        if (tid < BM) put_scales(sa, ((ks >> 1) + 1) & 1, tid);
      }
    }
    store_tile<TM, TN>(acc, p.out, p.N, (int64_t)rb + m0, rows, n0 + 64 * w, p.N, lane);
  }
}

// ---------------------------------------------------------------------------
// dgrad
// ---------------------------------------------------------------------------
// A workgroup computes BM rows by 256 columns (of k) of one expert, in steps of 64 weight
// rows n.  dY goes to LDS by direct copies one step ahead.  Each wave owns 64 columns, that
// is two MX blocks of every weight row: lane i of the wave loads row i's two blocks (32 bytes
// and two scales), decodes them to bf16 and writes them to the wave's own 64 x 64 LDS tile,
// from which the 16-bit transposing read hands every lane one column's 8 consecutive rows.
constexpr int DK = 64;   // weight rows per step
constexpr int DQS = 72;  // row stride (bf16) of the decoded tile

template <int TM>
struct DgradSmem {
  uint8_t a[2][32 * TM * 128];        // bf16 dY, 64 of n per row
  uint16_t dq[NTHR / 64][DK * DQS];
  int toff[kMaxE + 1];
  int wsum[NTHR / 64];
};

// B fragment (8 consecutive rows of one column per lane) of the decoded tile
__device__ __forceinline__ bf16x8 frag_trans(const uint16_t *t, int kbase, int nbase, int lane) {
  const int g = lane >> 4, s = lane & 15;
  const uint16_t *p = t + (kbase + 8 * (g >> 1) + (s >> 2)) * DQS + nbase + 16 * (g & 1) + 4 * (s & 3);
  const s16x4 h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
  const s16x4 h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * DQS));
  const s16x8 v = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
  return __builtin_bit_cast(bf16x8, v);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int P>
__device__ __forceinline__ uint32_t fp4_bf16(uint32_t c, float sc) {
  return __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, P));
}

// one MX block (32 codes) -> 32 bf16 at dst; sc: its E8M0 code
__device__ __forceinline__ void decode_block(const u32x4 &c, uint32_t sc, uint16_t *dst) {
  const float s = sc == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(sc ? sc << 23 : 0x00400000u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 o = {fp4_bf16<0>(c[i], s), fp4_bf16<1>(c[i], s), fp4_bf16<2>(c[i], s), fp4_bf16<3>(c[i], s)};
    *reinterpret_cast<u32x4 *>(dst + 8 * i) = o;
  }
}

template <int TM>
__global__ void __launch_bounds__(NTHR, 1) mx_dgrad(MxParams p) {
  constexpr int BM = 32 * TM, TN = 2, AR = BM / 32;
  __shared__ __attribute__((aligned(16))) DgradSmem<TM> sm;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int total = tile_prefix<BM>(p, sm.toff, sm.wsum) * p.NT;
  const int per = (total + 7) / 8;
  const int first = (blockIdx.x & 7) * per, last = min(first + per, total);
  const int nb = p.K / 32, nk = (p.N + DK - 1) / DK;
  for (int L = first + (int)(blockIdx.x >> 3); L < last; L += (int)(gridDim.x >> 3)) {
    const int mt = L / p.NT, nt = L % p.NT;
    const int e = expert_of_tile(sm.toff, p.E, mt);
    const int rb = seg_at(p, e), n_e = seg_at(p, e + 1) - rb;
    const int m0 = (mt - sm.toff[e]) * BM;
    const int rows = min(n_e - m0, BM);
    const int vt = (rows + 31) / 32;
    const uint16_t *asrc[AR];
#pragma unroll
    for (int j = 0; j < AR; ++j) {
      const int r = 8 * (AR * w + j) + (lane >> 3);
      asrc[j] = p.dy + src_row(p, (int64_t)rb + min(m0 + r, n_e - 1)) * p.N;
    }
    // the two MX blocks of this wave's 64 columns (past the row's end: its last block,
    // whose columns are dropped)
    const int b0 = min((nt * 256 + 64 * w) / 32, nb - 1), b1 = min(b0 + 1, nb - 1);
    const uint8_t *wc = p.wc + (int64_t)e * p.N * (p.K / 2), *ws = p.ws + (int64_t)e * p.N * nb;
    auto copy = [&](int ks, int st) {
#pragma unroll
      for (int j = 0; j < AR; ++j) {
        const int r = 8 * (AR * w + j) + (lane >> 3), n = DK * ks + 8 * ((lane & 7) ^ ((r >> 1) & 7));
        dma_b128(n < p.N ? reinterpret_cast<const void *>(asrc[j] + n) : reinterpret_cast<const void *>(c_zeros),
                 lds_addr(sm.a[st]) + 1024 * (AR * w + j));
      }
    };
    u32x4 wc0, wc1;
    uint32_t ws0, ws1;
    auto load_w = [&](int ks) {  // rows past N: the last row's (their dY is zero)
      const int64_t n = min(DK * ks + lane, p.N - 1);
      wc0 = *reinterpret_cast<const u32x4 *>(wc + n * (p.K / 2) + 16 * b0);
      wc1 = *reinterpret_cast<const u32x4 *>(wc + n * (p.K / 2) + 16 * b1);
      ws0 = ws[n * nb + b0];
      ws1 = ws[n * nb + b1];
    };
    f32x16 acc[TM][TN];
    clear_acc(acc);
    __syncthreads();  // the stages of the tile before are free
    uint16_t *dq = sm.dq[w];
    load_w(0);
    copy(0, 0);
    for (int ks = 0; ks < nk; ++ks) {
      const int st = ks & 1;
      wait_vm<0>();
      barrier_lds();
      decode_block(wc0, ws0, dq + lane * DQS);
      decode_block(wc1, ws1, dq + lane * DQS + 32);
      if (ks + 1 < nk) {
        load_w(ks + 1);
        copy(ks + 1, st ^ 1);
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        bf16x8 bf[TN];
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) bf[tn] = frag_trans(dq, 16 * kk, 32 * tn, lane);
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
          const bf16x8 af = *reinterpret_cast<const bf16x8 *>(sm.a[st] + swz(tm * 32 + (lane & 31), 2 * kk + (lane >> 5)));
          if (tm < vt) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
              acc[tm][tn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[tn], af, acc[tm][tn], 0, 0, 0);
          }
        }
      }
    }
    store_tile<TM, TN>(acc, p.out, p.K, (int64_t)rb + m0, rows, nt * 256 + 64 * w, p.K, lane);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bqm_status check_mx(const char *who, const bqm_qtensor *q, const char *name) {
  BQM_REQUIRE(q, BQM_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  BQM_REQUIRE(q->fmt == BQM_FMT_MXFP4, BQM_ERR_INVALID_ARG, "%s: %s->fmt must be BQM_FMT_MXFP4", who, name);
  BQM_REQUIRE(q->n_mat >= 0 && q->rows >= 0 && q->cols >= 0, BQM_ERR_INVALID_ARG, "%s: %s: negative size", who, name);
  return BQM_OK;
}

bqm_status check_data(const char *who, const bqm_qtensor *q, const char *name) {
  BQM_REQUIRE(q->codes && q->scales, BQM_ERR_INVALID_ARG, "%s: %s codes/scales pointer is NULL", who, name);
  BQM_REQUIRE(aligned16(q->codes) && aligned16(q->scales), BQM_ERR_ALIGN, "%s: %s codes/scales not 16-byte aligned",
              who, name);
  return BQM_OK;
}

// What both directions ask of the weights, the routing and the row count; rows: those of
// the activations or output gradients.
bqm_status check_routed(const char *who, const bqm_qtensor *w, const int32_t *offsets, const int32_t *perm, int32_t k,
                        int64_t R, int64_t rows) {
  bqm_status st = check_mx(who, w, "w");
  if (st != BQM_OK) return st;
  BQM_REQUIRE(w->n_mat >= 1 && w->n_mat <= kMaxE, BQM_ERR_SHAPE, "%s: E=%lld outside [1, 1024]", who,
              (long long)w->n_mat);
  BQM_REQUIRE(w->rows >= 32 && w->rows % 32 == 0 && w->rows < (1 << 24), BQM_ERR_SHAPE,
              "%s: N=%lld is not a positive multiple of 32 below 2^24", who, (long long)w->rows);
  BQM_REQUIRE(w->cols >= 32 && w->cols % 32 == 0 && w->cols < (1 << 24), BQM_ERR_SHAPE,
              "%s: K=%lld is not a positive multiple of 32 below 2^24", who, (long long)w->cols);
  BQM_REQUIRE(R >= 0 && rows >= 0, BQM_ERR_INVALID_ARG, "%s: negative size", who);
  BQM_REQUIRE(R < ((int64_t)1 << 30), BQM_ERR_SHAPE, "%s: R=%lld too large", who, (long long)R);
  if (perm) {
    BQM_REQUIRE(k >= 1, BQM_ERR_SHAPE, "%s: k=%d < 1", who, k);
    BQM_REQUIRE(rows * k == R, BQM_ERR_SHAPE, "%s: R=%lld is not %lld rows times k=%d", who, (long long)R,
                (long long)rows, k);
  } else {
    BQM_REQUIRE(rows == R, BQM_ERR_SHAPE, "%s: R=%lld, but %lld rows and no perm", who, (long long)R, (long long)rows);
  }
  BQM_REQUIRE((R / 32 + w->n_mat) * cdiv(w->rows > w->cols ? w->rows : w->cols, 32) < ((int64_t)1 << 31),
              BQM_ERR_SHAPE, "%s: too many tiles", who);
  if (R == 0) return BQM_OK;
  st = check_data(who, w, "w");
  if (st != BQM_OK) return st;
  BQM_REQUIRE(offsets, BQM_ERR_INVALID_ARG, "%s: offsets is NULL", who);
  BQM_REQUIRE(aligned16(offsets) && aligned16(perm), BQM_ERR_ALIGN, "%s: offsets or perm not 16-byte aligned", who);
  return BQM_OK;
}

constexpr int kCUs = 256;

// workgroups for at most R / bm + E row tiles of nt column tiles, one resident per CU
unsigned tile_grid(int64_t R, int E, int bm, int64_t nt) {
  const int64_t tiles = (R / bm + (E < R ? E : R)) * nt;
  const int64_t g = cdiv(tiles < kCUs ? tiles : kCUs, 8) * 8;
  return (unsigned)g;
}

}  // namespace
}  // namespace bqm

using namespace bqm;

extern "C" bqm_status bqm_mxfp4_gemm(const bqm_qtensor *x, const bqm_qtensor *w, const int32_t *offsets,
                                     const int32_t *perm, int32_t k, int64_t R, uint16_t *y, void *stream) {
  const char *who = "bqm_mxfp4_gemm";
  bqm_status st = check_mx(who, x, "x");
  if (st != BQM_OK) return st;
  BQM_REQUIRE(x->n_mat == 1, BQM_ERR_SHAPE, "%s: x must be one matrix of rows", who);
  st = check_routed(who, w, offsets, perm, k, R, x->rows);
  if (st != BQM_OK) return st;
  BQM_REQUIRE(x->cols == w->cols, BQM_ERR_SHAPE, "%s: x has K=%lld, w K=%lld", who, (long long)x->cols,
              (long long)w->cols);
  if (R == 0) return BQM_OK;
  st = check_data(who, x, "x");
  if (st != BQM_OK) return st;
  BQM_REQUIRE(y, BQM_ERR_INVALID_ARG, "%s: y is NULL", who);
  BQM_REQUIRE(aligned16(y), BQM_ERR_ALIGN, "%s: y not 16-byte aligned", who);
  MxParams p = {};
  p.xc = x->codes;
  p.xs = reinterpret_cast<const uint8_t *>(x->scales);
  p.xrows = x->rows;
  p.wc = w->codes;
  p.ws = reinterpret_cast<const uint8_t *>(w->scales);
  p.offsets = offsets;
  p.perm = perm;
  p.E = (int)w->n_mat;
  p.k = k;
  p.N = (int)w->rows;
  p.K = (int)w->cols;
  p.NT = (int)cdiv(p.N, BN);
  p.R = R;
  p.out = y;
  mx_gemm<8><<<tile_grid(R, p.E, 256, p.NT), NTHR, 0, as_stream(stream)>>>(p);
  return launch_status("mx_gemm");
}

extern "C" bqm_status bqm_mxfp4_dgrad(const bqm_qtensor *w, const uint16_t *dy, int64_t dy_rows,
                                      const int32_t *offsets, const int32_t *perm, int32_t k, int64_t R, uint16_t *dx,
                                      void *stream) {
  const char *who = "bqm_mxfp4_dgrad";
  bqm_status st = check_routed(who, w, offsets, perm, k, R, dy_rows);
  if (st != BQM_OK) return st;
  if (R == 0) return BQM_OK;
  BQM_REQUIRE(dy && dx, BQM_ERR_INVALID_ARG, "%s: dy or dx is NULL", who);
  BQM_REQUIRE(aligned16(dy) && aligned16(dx), BQM_ERR_ALIGN, "%s: dy or dx not 16-byte aligned", who);
  MxParams p = {};
  p.dy = dy;
  p.xrows = dy_rows;
  p.wc = w->codes;
  p.ws = reinterpret_cast<const uint8_t *>(w->scales);
  p.offsets = offsets;
  p.perm = perm;
  p.E = (int)w->n_mat;
  p.k = k;
  p.N = (int)w->rows;
  p.K = (int)w->cols;
  p.NT = (int)cdiv(p.K, 256);
  p.R = R;
  p.out = dx;
  mx_dgrad<8><<<tile_grid(R, p.E, 256, p.NT), NTHR, 0, as_stream(stream)>>>(p);
  return launch_status("mx_dgrad");
}
