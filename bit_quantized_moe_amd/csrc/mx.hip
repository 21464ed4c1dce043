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

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
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
// a pointer that is the same in all lanes, in scalar registers
__device__ __forceinline__ const uint8_t *uniform(const void *q) {
  const uint64_t v = reinterpret_cast<uint64_t>(q);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t *>(((uint64_t)hi << 32) | lo);
}

// Direct-to-LDS copy: lane i's 16 bytes land at lds + 16 i.  Inline assembly, so that the
// compiler's wait counts do not drain every LDS read before each use of an LDS result; the
// copies are waited for with wait_vm before their stage is read.
__device__ __forceinline__ void dma_b128(const void *g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(g), "s"(lds) : "memory", "m0");
}
// The same with a scalar base and a lane's byte offset: no vector instruction per copy.
__device__ __forceinline__ void dma_b128(const void *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(uniform(base)), "s"(lds)
               : "memory", "m0");
}
// lane i's byte, as a word, lands at lds + 4 i
__device__ __forceinline__ void dma_u8(const void *g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, off" : : "v"(g), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma_b32(const void *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(uniform(base)), "s"(lds)
               : "memory", "m0");
}
// workgroup barrier that orders LDS without draining outstanding copies
__device__ __forceinline__ void barrier_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  // the builtin, not inline assembly: the compiler then knows which loads have landed
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");  // no read of what the copies wrote before it
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
// first row of expert e's segment, clamped to [0, R]
__device__ __forceinline__ int seg_at(const MxParams &p, int e) {
  const int64_t v = p.offsets[e];
  return (int)(v < 0 ? 0 : (v > p.R ? p.R : v));
}

// Row tiles (of BM rows) in expert order.  Each thread keeps the prefix of its PER experts in
// registers; the one that owns a row tile's expert tells the others through LDS.
constexpr int PER = kMaxE / NTHR;
struct TileMap {
  int first[PER + 1];  // row tiles before expert PER tid + i

  // returns the number of row tiles, at most as many as offsets that do not fall can make:
  // falling ones give rows to many experts, and the tiles of all of them (E / 2 times R rows)
  // need not fit 32 bits, so the sums are unsigned and tiles past that number are left out
  template <int BM>
  __device__ int build(const MxParams &p, int *wsum) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int c[PER];
    uint32_t run = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid * PER + i;
      int n = 0;
      if (e < p.E) n = seg_at(p, e + 1) - seg_at(p, e);
      c[i] = n > 0 ? (n + BM - 1) / BM : 0;
      run += c[i];
    }
    uint32_t inc = run;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t t = __shfl_up(inc, o, 64);
      if (lane >= o) inc += t;
    }
    if (lane == 63) wsum[wave] = (int)inc;
    __syncthreads();
    uint32_t base = 0, total = 0;
#pragma unroll
    for (int q = 0; q < NTHR / 64; ++q) {
      if (q < wave) base += (uint32_t)wsum[q];
      total += (uint32_t)wsum[q];
    }
    base += inc - run;
    first[0] = (int)base;
#pragma unroll
    for (int i = 0; i < PER; ++i) first[i + 1] = (int)(base += c[i]);
    const int64_t most = p.R / BM + (p.E < p.R ? p.E : p.R);
    return (int)min((int64_t)total, most);
  }

  // the owner of row tile mt writes its expert, that expert's first tile and number of tiles to found
  __device__ __forceinline__ void find(int mt, int *found) const {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (first[i] <= mt && mt < first[i + 1]) {
        found[0] = (int)threadIdx.x * PER + i;
        found[1] = first[i];
        found[2] = first[i + 1] - first[i];
      }
  }
};

// source row of routed position pos, kept inside the tensor
__device__ __forceinline__ int64_t src_row(const MxParams &p, int64_t pos) {
  int64_t r = p.perm ? (int64_t)(p.perm[pos] / p.k) : pos;
  r = r < 0 ? 0 : r;
  return r < p.xrows ? r : p.xrows - 1;
}

// ---------------------------------------------------------------------------
// the tiled kernels
// ---------------------------------------------------------------------------
// A workgroup of four waves (WM x WN) computes BM = 32 WM TM rows by BN = 32 WN TN columns of
// one expert; wave (wm, wn) owns the 32-row tiles WM tm + wm (interleaved, so that a partly
// filled tile leaves all rows of waves the same work) of 32 TN columns.  The contraction goes
// in steps of 128 bytes per activation row (256 MXFP4 values or 64 bf16 values) through two
// LDS stages filled by direct-to-LDS copies one step ahead; a step is four slices of
// VT x TN MFMAs of 32x32.
//
// One wave per SIMD (the accumulators of the largest tile take half the register file) has
// no other wave to hide its waits behind, so the step is written out in issue order: after
// each MFMA comes a share of the slice's other work (the fragment reads of the next slice,
// copies of the next step, weight decode), pinned there by scheduling barriers.  The step's
// one barrier sits inside slice 3, whose fragments are in registers by then: from it on the
// next step's first fragments are read while slice 3's MFMAs run.
//
// 2 x 2 and not 1 x 4 waves: a wave of 128 x 128 reads 8 KB of fragments per 16 MFMAs, one
// of 256 x 64 10 KB; with the copies into LDS that is 94 against 109 bytes per clock of the
// LDS's 128 at the MFMA rate.
//
// Accumulators hold the product transposed (weights x activations): register v of lane L of
// tile (tm, tn) is row L % 32 and column 8 (v / 4) + 4 (L / 32) + v % 4, so a lane stores 4
// consecutive columns of one row at a time.
#define MX_PIN() __builtin_amdgcn_sched_barrier(0)

constexpr int DK = 64;   // dgrad: weight rows per step
constexpr int DQS = 72;  // dgrad: row stride (bf16) of a decoded 64-column group

template <int BM, int BN, bool FWD, int NS>
struct Smem;
template <int BM, int BN>
struct Smem<BM, BN, true, 2> {
  uint8_t a[2][BM * 128];
  uint8_t b[2][BN * 128];
  uint32_t s[2][2][2][BM + BN + 4];  // [group parity][step of the group][half][row]
  int wsum[NTHR / 64], found[3];
};
template <int BM, int BN, int NS>
struct Smem<BM, BN, false, NS> {
  uint8_t a[NS][BM * 128];
  uint16_t dq[2][BN / 64][DK * DQS];
  uint8_t c[NS][DK * 128];           // codes of a step's weight rows, 256 columns
  uint32_t cs[NS][BN / 32 * DK];     // their scales: FAST [row][4 words, of which 2 hold bytes], else [block][row]
  int wsum[NTHR / 64], found[3];
};

// The scales of blocks 16 g .. 16 g + 15 of a row of nb >= 16 blocks in one load; the last
// group's 16 bytes end at the row's end, and shift_scales moves them down once they have
// landed (by the same number of bytes for every row), filling with 127 (2^0).
__device__ __forceinline__ u32x4 load_scales(const uint8_t *row, int g, int nb) {
  u32x4 v;
  __builtin_memcpy(&v, row + min(16 * g, nb - 16), 16);  // unaligned where 4 does not divide nb
  return v;
}
__device__ __forceinline__ u32x4 shift_scales(const u32x4 &v, int g, int nb) {
  const int d = 16 * g - min(16 * g, nb - 16);  // 0 .. 15
  constexpr uint32_t f = 0x7F7F7F7Fu;
  // by 8, by 4, then by the remaining 0 to 3 bytes, without a branch
  const bool by8 = d & 8, by4 = d & 4;
  auto pick = [](bool c, uint32_t x, uint32_t y) { return c ? x : y; };
  const uint32_t a0 = pick(by8, v[2], v[0]), a1 = pick(by8, v[3], v[1]), a2 = pick(by8, f, v[2]), a3 = pick(by8, f, v[3]);
  const uint32_t b0 = pick(by4, a1, a0), b1 = pick(by4, a2, a1), b2 = pick(by4, a3, a2), b3 = pick(by4, f, a3);
  const uint32_t r = (uint32_t)d & 3u;
  return u32x4{__builtin_amdgcn_alignbyte(b1, b0, r), __builtin_amdgcn_alignbyte(b2, b1, r),
               __builtin_amdgcn_alignbyte(b3, b2, r), __builtin_amdgcn_alignbyte(f, b3, r)};
}
// the same for a row of fewer than 16 blocks: its bytes at the end of the 16
__device__ __forceinline__ u32x4 load_few_scales(const uint8_t *row, int nb) {
  u32x4 v = {};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i >= 16 - nb) v[i >> 2] |= (uint32_t)row[i - (16 - nb)] << (8 * (i & 3));
  return v;
}

// B fragment (8 consecutive rows of one column per lane) of a decoded 64-column group
__device__ __forceinline__ i32x4 frag_trans(const uint16_t *t, int kbase, int nbase, int lane) {
  const int g = lane >> 4, s = lane & 15;
  const uint16_t *p = t + (kbase + 8 * (g >> 1) + (s >> 2)) * DQS + nbase + 16 * (g & 1) + 4 * (s & 3);
  const s16x4 h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
  const s16x4 h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * DQS));
  const s16x8 v = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
  return __builtin_bit_cast(i32x4, v);
}

template <int P>
__device__ __forceinline__ uint32_t fp4_bf16(uint32_t c, float sc) {
  return __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, P));
}

__device__ __forceinline__ float e8m0(uint32_t c) {
  return c == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(c ? c << 23 : 0x00400000u);
}

// Everything a wave keeps while it works on one tile.
// FAST: the contraction has at least one whole step and every source lies within 4 GiB of a
// base, so a copy's address is a scalar base that moves with the step plus the lane's
// constant offset.  Where the last step is not whole it takes the last 128 bytes of the rows
// instead, and the fragments' share of the step before is replaced by zeros.  Without FAST
// copies take 64-bit addresses, and zeros past the end of an activation row: four to six more
// vector instructions for each (64 experts of 1024 rows, product 4096 x 6176: 1322 us so,
// 1271 us with FAST; gradient 4128 x 6144: 2985 and 2778 us).
// NS: stages.  Two: the copies of a step begin in slice 3 of the step before the last.  Four
// (the gradient with few rows, where the activation stages are small): they run three steps
// ahead, which a stream of weights from HBM needs when a step holds little else.
template <int WM, int TM, int TN, bool FWD, bool FAST, int NS>
struct Tile {
  static constexpr int WN = 4 / WM, BM = 32 * WM * TM, BN = 32 * WN * TN;
  static constexpr int CA = BM / 32, CB = BN / 32;  // copies (of 8 rows) per wave and step
  static constexpr int DB = BN / 128;  // dgrad: MX blocks a lane decodes per step
  static constexpr int kCodeOps = FWD ? 0 : DB + (FAST ? 1 : DB);  // dgrad: copies of codes and scales per step
  static_assert(FWD || BN == 256, "the gradient's code rows are 128 bytes");
  static constexpr bool DEEP = NS > 2;
  static constexpr int D = NS - 1;  // DEEP: steps the copies run ahead
  static_assert(!DEEP || !FWD, "the forward's scales are loaded one group ahead");
  const MxParams &p;
  Smem<BM, BN, FWD, NS> &sm;
  int lane, w, wm, wn, nb, nk;
  const uint8_t *asrc[FAST ? 1 : CA];  // activation rows of this lane's copies (bytes)
  const uint8_t *abase;                    // FAST: what aoff counts from
  uint32_t aoff[FAST ? CA : 1];
  int alen;                     // bytes of an activation row
  const uint8_t *zeros;
  const uint8_t *wbase;         // the expert's codes
  uint32_t boff[FWD ? CB : 1];
  const uint8_t *sa, *sb;       // forward: the scale rows this thread carries
  u32x4 va, vb;                 // their 16 bytes of the next group
  u32x4 cc[DB];                 // dgrad: codes of the next step
  uint32_t sc[DB];              // and their scales
  int q0;                       // dgrad: first block of the tile's columns
  uint32_t coff[DB], soff;      // dgrad, FAST: of codes and scales
  i32x4 af[2][TM], bf[2][TN];
  int ssa[TM], ssb[TN];         // forward: scale words of the step
  f32x16 acc[TM][TN];

  __device__ __forceinline__ Tile(const MxParams &p_, Smem<BM, BN, FWD, NS> &sm_) : p(p_), sm(sm_) {
    lane = threadIdx.x & 63;
    w = wave_id();
    wm = WM == 2 ? w >> 1 : 0;
    wn = WM == 2 ? w & 1 : w;
    nb = p.K / 32;
    nk = FWD ? (p.K + 255) / 256 : (p.N + DK - 1) / DK;
    alen = FWD ? p.K / 2 : p.N * 2;
    zeros = reinterpret_cast<const uint8_t *>(c_zeros);
  }

  // rb: the expert's first row, m0: the tile's, within n_e rows; n0: the tile's first column
  __device__ __forceinline__ void setup(int e, int rb, int m0, int n_e, int n0) {
    const int tid = threadIdx.x;
    // what follows from the lane is computed anew for each tile: kept across tiles it is
    // spilled, and the wait for its reload lands inside the K loop
    asm volatile("" : "+v"(lane));
#pragma unroll
    for (int j = 0; j < CA; ++j) {
      const int r = 8 * (CA * w + j) + (lane >> 3);
      const uint8_t *x = FWD ? p.xc : reinterpret_cast<const uint8_t *>(p.dy);
      const int64_t row = src_row(p, (int64_t)rb + min(m0 + r, n_e - 1));
      if constexpr (FAST) {
        // without perm the rows follow each other: count from the tile's first
        const int64_t row0 = p.perm ? 0 : src_row(p, (int64_t)rb + m0);
        abase = x + row0 * alen;
        aoff[j] = (uint32_t)((row - row0) * alen) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
      } else {
        asrc[j] = x + row * alen;
      }
    }
    wbase = p.wc + (int64_t)e * p.N * (p.K / 2);
    const uint8_t *ws = p.ws + (int64_t)e * p.N * nb;
    if constexpr (FWD) {
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        const int r = 8 * (CB * w + j) + (lane >> 3);
        boff[j] = (uint32_t)min(n0 + r, p.N - 1) * (p.K / 2) + (FAST ? 16 * ((lane & 7) ^ ((r >> 1) & 7)) : 0);
      }
      sb = ws + (int64_t)min(n0 + (tid < BN ? tid : 0), p.N - 1) * nb;
      sa = p.xs + src_row(p, (int64_t)rb + min(m0 + (tid < BM ? tid : 0), n_e - 1)) * nb;
    } else {
      sb = ws;
      q0 = n0 / 32;
      if constexpr (FAST) {
#pragma unroll
        for (int i = 0; i < DB; ++i)
          coff[i] = (uint32_t)code_row(i) * (p.K / 2) + 16 * min(q0 + code_chunk(i), nb - 1);
        soff = (uint32_t)(16 * w + (lane >> 2)) * nb + min(q0 + 4 * min(lane & 3, 1), nb - 4);
      }
    }
  }

  // FAST: where step ks begins in its rows, and the dgrad's weight rows (steps past the last
  // are the last again: copied for nothing, and not read)
  __device__ __forceinline__ int at_step(int ks) const { return min(128 * ks, alen - 128); }
  __device__ __forceinline__ int64_t row_at(int ks) const { return min(DK * ks, p.N - DK); }
  // the last step's 16-byte chunks that belong to the step before
  __device__ __forceinline__ int overlap() const { return FAST ? 8 * nk - alen / 16 : 0; }

  // copy j of step ks into stage st: activations (j < 2 TM; zeros past the row's end), then
  // weights (any of the row's bytes there)
  __device__ __forceinline__ void copy(int j, int ks, int st) {
    if (j < CA) {
      const uint32_t to = lds_addr(sm.a[st]) + 1024 * (CA * w + j);
      if constexpr (FAST) {
        dma_b128(abase + at_step(ks), aoff[j], to);
      } else {
        const int r = 8 * (CA * w + j) + (lane >> 3);
        const int o = 128 * ks + 16 * ((lane & 7) ^ ((r >> 1) & 7));
        dma_b128(o < alen ? asrc[j] + o : zeros, to);
      }
    } else if constexpr (FWD) {
      j -= CA;
      const uint32_t to = lds_addr(sm.b[st]) + 1024 * (CB * w + j);
      if constexpr (FAST) {
        dma_b128(wbase + at_step(ks), boff[j], to);
      } else {
        const int r = 8 * (CB * w + j) + (lane >> 3);
        const int o = 128 * ks + 16 * ((lane & 7) ^ ((r >> 1) & 7));
        dma_b128(wbase + (boff[j] + (uint32_t)(o < alen ? o : 0)), to);
      }
    }
  }

  // ---- forward: scales of a group of two steps, loaded by the thread of their row (threads
  // past the tile's rows load row 0's and drop them) ----
  __device__ __forceinline__ void get_scales(int group) {
    va = load_scales(sa, group, nb);
    vb = load_scales(sb, group, nb);
  }
  // for each step and half g of a wave: the scales of blocks g, 2 + g, 4 + g, 6 + g as one
  // word, of which the MFMA of slice kk takes byte kk
  __device__ __forceinline__ void put_words(const u32x4 &v, int group, int row) {
    const u32x4 u = shift_scales(v, group, nb);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // FAST: the last step's eight blocks are the row's last, the top half of what was loaded
      const bool last = FAST && 2 * group + h == nk - 1;
      const uint32_t lo = last ? v[2] : u[2 * h], hi = last ? v[3] : u[2 * h + 1];
      uint32_t(&s)[2][BM + BN + 4] = sm.s[group & 1][h];
      s[0][row] = __builtin_amdgcn_perm(hi, lo, 0x06040200u);
      s[1][row] = __builtin_amdgcn_perm(hi, lo, 0x07050301u);
    }
  }
  __device__ __forceinline__ void put_scales(int group) {
    // threads without a row write to a word past the rows': a branch here would let the
    // compiler move MFMAs past it, out of their order
    const int tid = threadIdx.x, none = BM + BN;
    put_words(va, group, BM == NTHR || tid < BM ? tid : none);
    put_words(vb, group, BN == NTHR || tid < BN ? BM + tid : none);
  }
  __device__ __forceinline__ const uint32_t *scale_words(int ks) const { return sm.s[(ks >> 1) & 1][ks & 1][lane >> 5]; }

  // ---- dgrad: lane i of a wave decodes DB blocks of weight row i of the step ----
  // The codes go through LDS, whole 128-byte rows like the activations', and are there one
  // step before the activations of their step, as decoding comes first.  (Copies, not loads
  // to registers: the compiler would wait for those without counting the copies in between.)
  __device__ __forceinline__ int code_row(int i) const { return 8 * (DB * w + i) + (lane >> 3); }
  __device__ __forceinline__ int code_chunk(int i) const { return (lane & 7) ^ ((code_row(i) >> 1) & 7); }
  __device__ __forceinline__ void code_op(int i, int ks) {
    const int d = ks & (NS - 1);
    if (i < DB) {
      const uint32_t to = lds_addr(sm.c[d]) + 1024 * (DB * w + i);
      if constexpr (FAST) {
        dma_b128(wbase + row_at(ks) * (p.K / 2), coff[i], to);
      } else {
        const int64_t n = min(DK * ks + code_row(i), p.N - 1);  // past the end: the last row (its dY is zero)
        const int q = min(q0 + code_chunk(i), nb - 1);          // past the end: columns that are dropped
        dma_b128(wbase + n * (p.K / 2) + 16 * q, to);
      }
    } else if constexpr (FAST) {  // 16 rows a wave, 4 words each (the last two again the second)
      dma_b32(sb + row_at(ks) * nb, soff, lds_addr(sm.cs[d]) + 256 * w);
    } else {
      const int64_t n = min(DK * ks + lane, p.N - 1);
      const int blk = w * DB + i - DB;
      dma_u8(sb + n * nb + min(q0 + blk, nb - 1), lds_addr(sm.cs[d]) + 4 * DK * blk);
    }
  }
  __device__ __forceinline__ void read_codes(int ks) {
    const int d = ks & (NS - 1);
    uint32_t two = 0;  // FAST: the scales of this lane's two blocks
    if constexpr (FAST) two = reinterpret_cast<const uint16_t *>(sm.cs[d])[8 * lane + w];
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      cc[b] = *reinterpret_cast<const u32x4 *>(sm.c[d] + swz(lane, w * DB + b));
      sc[b] = FAST ? (b ? two >> 8 : two & 0xFFu) : sm.cs[d][DK * (w * DB + b) + lane];
    }
  }
  // quarter u of the lane's blocks -> bf16 (exact) in buffer d
  __device__ __forceinline__ void decode(int u, int d) {
    const int b = u >> 2, i = u & 3, blk = w * DB + b;
    const float f = e8m0(sc[b]);
    const u32x4 o = {fp4_bf16<0>(cc[b][i], f), fp4_bf16<1>(cc[b][i], f), fp4_bf16<2>(cc[b][i], f),
                     fp4_bf16<3>(cc[b][i], f)};
    *reinterpret_cast<u32x4 *>(sm.dq[d][blk >> 1] + lane * DQS + 32 * (blk & 1) + 8 * i) = o;
  }

  // stage of the activations of step ks, of parity st
  __device__ __forceinline__ static int stage(int ks, int st) { return DEEP ? ks & (NS - 1) : st; }

  // ---- fragments of slice kk of stage st into set k ----
  __device__ __forceinline__ void read_a(int k, int tm, int kk, int st) {
    af[k][tm] = *reinterpret_cast<const i32x4 *>(sm.a[st] + swz(32 * (WM * tm + wm) + (lane & 31), 2 * kk + (lane >> 5)));
  }
  __device__ __forceinline__ void read_b(int k, int tn, int kk, int st) {
    const int c = 32 * (wn * TN + tn);
    if constexpr (FWD)
      bf[k][tn] = *reinterpret_cast<const i32x4 *>(sm.b[st] + swz(c + (lane & 31), 2 * kk + (lane >> 5)));
    else
      bf[k][tn] = frag_trans(sm.dq[st][c >> 6], 16 * kk, c & 63, lane);
  }

  // the i-th of a slice's reads, in the order its MFMAs ask for them
  __device__ __forceinline__ void read(int k, int i, int kk, int sa, int st) {
    if (i == 0)
      read_a(k, 0, kk, sa);
    else if (i <= TN)
      read_b(k, i - 1, kk, st);
    else
      read_a(k, i - TN, kk, sa);
  }

  template <int KK>
  __device__ __forceinline__ void mfma(int k, int tm, int tn) {
    const i32x4 a = af[k][tm], b = bf[k][tn];
    if constexpr (FWD) {
      const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
      acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[tm][tn], 4, 4, KK, ssb[tn], KK, ssa[tm]);
    } else {
      acc[tm][tn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a),
                                                            acc[tm][tn], 0, 0, 0);
    }
  }

  // The copies of step ks + 2 go into the stage that step ks has finished reading: the first
  // half from slice 3 of step ks on (after its barrier), the rest in slice 0 of step ks + 1.
  // LEFT: steps that follow (0, 1, or 2 for more).  PAR: the step's parity (-1: not known).
  static constexpr int kCopies = CA + (FWD ? CB : 0), kFirst = DEEP ? 0 : kCopies / 2;
  static constexpr int kOps = kCopies + kCodeOps;  // per step

  // Copies of this wave that its wait in slice 3 may leave in flight: those of later steps
  static constexpr int kInFlight = DEEP ? (D - 1) * kOps : 0;

  // other work of slices 0-2, item i: fragment reads of the next slice, copies and what
  // becomes of them.  Slice 0: the rest of the next step's copies, before the reads as they
  // have the least time (64 experts of 1024 rows, 4096 x 6144: product 1046 -> 1013 us,
  // gradient 2668 -> 2615 us), and the forward's scales of the next group (even steps).  DEEP:
  // after the reads all copies of step ks + D, whose stage was read in step ks - 1, and the
  // codes of the step after it.  Slice 1: dgrad: the next step's codes are read and half
  // decoded.  Slice 2: scales written, or the rest decoded.
  template <int VT, int KK, int LEFT, int PAR>
  static constexpr int items() {
    const int reads = TN + VT;
    if (LEFT == 0) return reads;
    if (KK == 0) return reads + (kCopies - kFirst) + (FWD ? (PAR == 0 ? 1 : 0) : (DEEP ? kCodeOps : 0));
    if (KK == 1) return reads + (FWD ? 0 : 1 + 2 * DB);
    return reads + (FWD ? 1 : 2 * DB);
  }
  template <int VT, int KK, int LEFT, int PAR>
  __device__ __forceinline__ void item(int i, int ks, int st) {
    constexpr int k = (KK + 1) & 1;
    if constexpr (KK == 0 && !DEEP && LEFT > 0) {  // copies first
      if (i < kCopies - kFirst) return copy(kFirst + i, ks + 1, st ^ 1);
      i -= kCopies - kFirst;
    }
    if (i < TN + VT) return read(k, i, KK + 1, stage(ks, st), st);
    i -= TN + VT;
    if constexpr (LEFT > 0) {
      if constexpr (KK == 0) {
        if constexpr (DEEP) {
          if (i < kCopies) return copy(i, ks + D, stage(ks + D, st));
          i -= kCopies;
        }
        if constexpr (FWD)
          get_scales(min((ks >> 1) + 1, (nb - 1) >> 4));  // the last group again: it is then not used
        else
          code_op(i, ks + D + 1);
      } else if constexpr (KK == 1) {
        if constexpr (!FWD) {
          if (i == 0)
            read_codes(ks + 1);
          else
            decode(i - 1, st ^ 1);
        }
      } else {
        if constexpr (FWD) {
          if constexpr (PAR != 0) put_scales((ks >> 1) + 1);  // (at an even step of no known parity: not read)
        } else {
          decode(2 * DB + i, st ^ 1);
        }
      }
    }
  }

  // zeros in place of the activations of slice kk of the last step that the step before had
  template <int VT>
  __device__ __forceinline__ void drop_overlap(int kk) {
    const bool drop = 2 * kk + (lane >> 5) < overlap();
#pragma unroll
    for (int tm = 0; tm < VT; ++tm)
#pragma unroll
      for (int i = 0; i < 4; ++i) af[kk & 1][tm][i] = drop ? 0 : af[kk & 1][tm][i];
  }

  template <int VT, int KK, int LEFT, int PAR>
  __device__ __forceinline__ void slice(int ks, int st) {
    if constexpr (FAST && LEFT == 0) drop_overlap<VT>(KK);
    constexpr int NP = VT * TN, NI = items<VT, KK, LEFT, PAR>();
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      mfma<KK>(KK & 1, q / TN, q % TN);
#pragma unroll
      for (int i = q * NI / NP; i < (q + 1) * NI / NP; ++i) item<VT, KK, LEFT, PAR>(i, ks, st);
      MX_PIN();
    }
  }

  // slice 3: its first MFMA, then the step's barrier, then slice 0 of the next step is read
  // and, in turn with those reads, the copies of the step after it begin (12 or all 16 of
  // them here, not 8, is no faster)
  template <int VT, int LEFT>
  __device__ __forceinline__ void slice3(int ks, int st) {
    constexpr int NP = VT * TN, NR = TN + VT, NW = FWD ? NR : 0;
    constexpr int NC = LEFT > 1 && !DEEP ? kCodeOps + kFirst : 0, NI = NR + NW + NC;
    if constexpr (FAST && LEFT == 0) drop_overlap<VT>(3);
    int na[TM], nw[TN];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      mfma<3>(1, q / TN, q % TN);
      if constexpr (LEFT > 0) {
        if (q == 0) {
          // every wave is done reading stage st, and the next stage is whole
          MX_PIN();
          wait_vm<kInFlight>();
          barrier_lds();
          MX_PIN();
        }
        const uint32_t *sw = nullptr;
        if constexpr (FWD) sw = scale_words(ks + 1);
#pragma unroll
        for (int at = q * NI / NP; at < (q + 1) * NI / NP; ++at) {
          // in turn a copy and a read, as long as there are both
          constexpr int both = NC < NR + NW ? NC : NR + NW;
          const bool isc = at < 2 * both ? !(at & 1) : NC > both;
          const int j0 = at < 2 * both ? at >> 1 : at - both;
          const int i = isc ? NR + NW + j0 : j0;
          if (i < NR) {
            read(0, i, 0, stage(ks + 1, st ^ 1), st ^ 1);
          } else if (i < NR + NW) {
            const int j = i - NR;
            if (j < TN)
              nw[j] = (int)sw[BM + 32 * (wn * TN + j) + (lane & 31)];
            else
              na[j - TN] = (int)sw[32 * (WM * (j - TN) + wm) + (lane & 31)];
          } else if (i < NR + NW + kFirst) {
            copy(i - NR - NW, ks + 2, st);
          } else {
            if constexpr (!FWD) code_op(i - NR - NW - kFirst, ks + 3);  // their place was read in slice 1
          }
        }
      }
      MX_PIN();
    }
    if constexpr (FWD && LEFT > 0) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) ssb[tn] = nw[tn];
#pragma unroll
      for (int tm = 0; tm < VT; ++tm) ssa[tm] = na[tm];
    }
  }

  template <int VT, int LEFT, int PAR>
  __device__ __forceinline__ void step(int ks, int st) {
    slice<VT, 0, LEFT, PAR>(ks, st);
    slice<VT, 1, LEFT, PAR>(ks, st);
    slice<VT, 2, LEFT, PAR>(ks, st);
    slice3<VT, LEFT>(ks, st);
  }

  // the contraction of one tile of which VT row tiles per wave hold rows
  template <int VT>
  __device__ __forceinline__ void run() {
#pragma unroll
    for (int tm = 0; tm < VT; ++tm)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[tm][tn][v] = 0.0f;
    if constexpr (FWD) {
      if (nb >= 16) {
        get_scales(0);
      } else {  // in the place where the others' loads end
        va = load_few_scales(sa, nb);
        vb = load_few_scales(sb, nb);
      }
    }
    if constexpr (!FWD) {
#pragma unroll
      for (int i = 0; i < kCodeOps; ++i) code_op(i, 0);
    }
#pragma unroll
    for (int q = 0; q < (DEEP ? D : 1); ++q) {
      if constexpr (!FWD) {
#pragma unroll
        for (int i = 0; i < kCodeOps; ++i) code_op(i, q + 1);
      }
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy(j, q, q);
    }
    if constexpr (FWD) put_scales(0);
    wait_vm<kInFlight>();
    barrier_lds();
    if constexpr (!FWD) {
      read_codes(0);
#pragma unroll
      for (int u = 0; u < 4 * DB; ++u) decode(u, 0);
      barrier_lds();
      if constexpr (!DEEP) {
#pragma unroll
        for (int i = 0; i < kCodeOps; ++i) code_op(i, 2);
      }
    }
#pragma unroll
    for (int i = 0; i < TN + VT; ++i) read(0, i, 0, 0, 0);
    if constexpr (FWD) {
      const uint32_t *sw = scale_words(0);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) ssb[tn] = (int)sw[BM + 32 * (wn * TN + tn) + (lane & 31)];
#pragma unroll
      for (int tm = 0; tm < VT; ++tm) ssa[tm] = (int)sw[32 * (WM * tm + wm) + (lane & 31)];
    }
    if (!DEEP && nk > 1) {
#pragma unroll
      for (int j = 0; j < kFirst; ++j) copy(j, 1, 1);
    }
    int ks = 0;
    for (; ks + 3 < nk; ks += 2) {
      step<VT, 2, 0>(ks, 0);
      step<VT, 2, 1>(ks + 1, 1);
    }
    if (ks + 3 == nk) step<VT, 2, 0>(ks++, 0);
    if (ks + 2 == nk) {
      step<VT, 1, -1>(ks, ks & 1);
      ++ks;
    }
    step<VT, 0, -1>(ks, ks & 1);
    // copies for steps that there are not, before the next tile's take their places
    if (DEEP || (!FWD && nk == 1)) wait_vm<0>();
  }

  // The accumulators hold 4 columns of 32 rows a lane quarter: stored as they are, an
  // instruction touches 32 rows.  They pass through the stages instead (each wave its own
  // part, 16-byte chunk c of row r at c ^ (r & its number of chunks - 1)), so that 16 bytes a
  // lane leave as whole row pieces: 64 experts of 1024 rows, product
  // 6144 x 2048 699 -> 636 us, 4096 x 6144 1037 -> 998 us.
  // rows: those of the tile that exist; ncols: columns of the output
  template <int VT>
  __device__ __forceinline__ void store(int64_t row_base, int rows, int n0, int ncols) {
    constexpr int CH = 4 * TN;  // chunks per row
    static_assert(sizeof(sm.a) + (FWD ? 2 * BN * 128 : 2 * (BN / 64) * DK * DQS * 2) >= 4 * TM * 32 * CH * 16,
                  "the waves' parts fit the stages");
    uint8_t *t = sm.a[0] + w * (TM * 32 * CH * 16);
    barrier_lds();  // every wave is done with the stages
#pragma unroll
    for (int tm = 0; tm < VT; ++tm) {
      const int r = tm * 32 + (lane & 31);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2 *>(t + 16 * (r * CH + ((4 * tn + q) ^ (r & (CH - 1)))) + 8 * (lane >> 5)) =
              make_uint2(pack_bf16_rne(acc[tm][tn][4 * q], acc[tm][tn][4 * q + 1]),
                         pack_bf16_rne(acc[tm][tn][4 * q + 2], acc[tm][tn][4 * q + 3]));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // store i takes RP rows of the wave's from RP i on; lane l holds chunk l % CH of row l / CH
    // of them.  Only lane offsets are vector arithmetic (32 rows of the output, below 2 GiB),
    // and eight reads are in flight at a time: addresses formed in full for each store, and
    // a wait for each read, cost 6 us per tile of 256 x 256.
    constexpr int RP = 64 / CH, NS8 = VT * CH / 2;
    const int lr = lane / CH, c = lane & (CH - 1);
    const uint32_t off = ((uint32_t)lr * ncols + 8 * c) * 2;
    const int n = n0 + 32 * wn * TN;  // the wave's first column
    const bool in = n + 8 * c < ncols;
    const int left = rows - 32 * wm - lr;
    const uint8_t *base = uniform(p.out + (row_base + 32 * wm) * ncols + n);
#pragma unroll
    for (int i0 = 0; i0 < NS8; i0 += 8) {
      u32x4 v[8];
#pragma unroll
      for (int j = 0; j < 8 && i0 + j < NS8; ++j) {
        const int r0 = RP * (i0 + j);
        v[j] = *reinterpret_cast<const u32x4 *>(t + 16 * CH * r0 + 16 * CH * lr +
                                                16 * (c ^ (lr & (CH - 1)) ^ (r0 & (CH - 1))));
      }
#pragma unroll
      for (int j = 0; j < 8 && i0 + j < NS8; ++j) {
        const int r0 = RP * (i0 + j), row = 32 * WM * (r0 >> 5) + (r0 & 31);
        if (in && row < left)
          *reinterpret_cast<u32x4 *>(const_cast<uint8_t *>(base + (int64_t)row * ncols * 2 + off)) = v[j];
      }
    }
  }

  template <int VT>
  __device__ __forceinline__ void run_and_store(int64_t row_base, int rows, int n0, int ncols) {
    run<VT>();
    store<VT>(row_base, rows, n0, ncols);
  }
};

template <int WM, int TM, int TN, bool FWD, bool FAST, int OCC, int NS>
__global__ void __launch_bounds__(NTHR, OCC) mx_tiles(MxParams p) {
  using T = Tile<WM, TM, TN, FWD, FAST, NS>;
  constexpr int BM = T::BM, BN = T::BN;
  __shared__ __attribute__((aligned(16))) Smem<BM, BN, FWD, NS> sm;
  const int ncols = FWD ? p.N : p.K;
  TileMap map;
  const int total = map.build<BM>(p, sm.wsum) * p.NT;
  // each XCD (workgroups b % 8) walks a contiguous range of tiles, so that the tiles in
  // flight there share an expert's rows and weights in its L2.  In the largest tile's kernels
  // an expert's row tiles are walked in groups of about GM, column tile by column tile: the 32
  // tiles that an XCD has in flight are then 4 x 8 and not 2 x 16 of them.  The groups are
  // even and end with the expert.  64 experts, 4096 x 6144, GB read and us, three kernels in
  // turn on one card (2 or 8 row tiles gain less, and the smaller tiles lose 1%):
  //                                 product          gradient
  //   1024 rows each, no groups     1.96   926       3.41  2534
  //     groups of 4 or about 4      1.30   904       2.56  2554
  //   922 to 1096 rows, no groups   3.23  1003       4.83  2788
  //     groups of 4 over experts    2.76  1004       5.21  2867
  //     even groups per expert      1.96   930       4.75  2797
  // (The gradient is bound by the matrix unit and keeps its time.)
  constexpr int GM = TM == 4 ? 4 : 1;
  const int per = (total + 7) / 8;
  const int first = (blockIdx.x & 7) * per, last = min(first + per, total);
  T t(p, sm);
  for (int L = first + (int)(blockIdx.x >> 3); L < last; L += (int)(gridDim.x >> 3)) {
    map.find(L / p.NT, sm.found);
    barrier_lds();  // also: the stages of the tile before are free
    const int e = __builtin_amdgcn_readfirstlane(sm.found[0]);
    const int rb = __builtin_amdgcn_readfirstlane(seg_at(p, e));
    const int n_e = __builtin_amdgcn_readfirstlane(seg_at(p, e + 1)) - rb;
    const int in_e = L - __builtin_amdgcn_readfirstlane(sm.found[1]) * p.NT;  // among the expert's tiles
    int mt = in_e / p.NT, nt = in_e % p.NT;
    if constexpr (GM > 1) {  // n_g groups of g row tiles, the last of them of what is left
      const int c = __builtin_amdgcn_readfirstlane(sm.found[2]), n_g = max((c + GM / 2) / GM, 1), g = (c + n_g - 1) / n_g;
      const int m_first = in_e / (g * p.NT) * g, gm = min(g, c - m_first), in_g = in_e - m_first * p.NT;
      mt = m_first + in_g % gm;
      nt = in_g / gm;
    }
    const int m0 = mt * BM, n0 = nt * BN;
    const int rows = min(n_e - m0, BM);
    const int vt = (rows + 32 * WM - 1) / (32 * WM);  // row tiles per wave that hold rows
    t.setup(e, rb, m0, n_e, n0);
    const int64_t row_base = (int64_t)rb + m0;
    if constexpr (TM == 1) {
      t.template run_and_store<1>(row_base, rows, n0, ncols);
    } else if constexpr (TM == 2) {
      if (vt == 2)
        t.template run_and_store<2>(row_base, rows, n0, ncols);
      else
        t.template run_and_store<1>(row_base, rows, n0, ncols);
    } else {
      if (vt == 4)
        t.template run_and_store<4>(row_base, rows, n0, ncols);
      else if (vt == 3)
        t.template run_and_store<3>(row_base, rows, n0, ncols);
      else if (vt == 2)
        t.template run_and_store<2>(row_base, rows, n0, ncols);
      else
        t.template run_and_store<1>(row_base, rows, n0, ncols);
    }
  }
}
#undef MX_PIN

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
    BQM_REQUIRE(rows <= R && rows * k == R, BQM_ERR_SHAPE, "%s: R=%lld is not %lld rows times k=%d", who, (long long)R,
                (long long)rows, k);
  } else {
    BQM_REQUIRE(rows == R, BQM_ERR_SHAPE, "%s: R=%lld, but %lld rows and no perm", who, (long long)R, (long long)rows);
  }
  BQM_REQUIRE(w->rows * (w->cols / 2) < ((int64_t)1 << 32), BQM_ERR_SHAPE, "%s: one expert's codes reach 4 GiB", who);
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

// The tile goes by the rows an expert has on average (the host knows R and E, not the
// offsets), one tile of rows as long as it can hold them: every further one reads the
// expert's weights again, and a tile's empty rows cost what full ones do.  Pairs that belong
// to no expert count as rows, and experts without rows as experts.  Measured in us, product
// N = 2816, K = 2048, 60 experts, gradient N = K = 2048, 64 experts; e: the same rows for
// every expert, r: every row's expert at random, s: with weights 1, 2^-0.7, 3^-0.7, ...
//   product     rows 12   24   28   32   40   56   64   96  128  160  256
//   32 x 128  e      39   40   41   41   49   51   50   65   83   98  149
//             r      38   40   41   43   49   52   58   73   87  106  158
//             s      38   43   47   46   49   57   61   77   91  108  162
//   64 x 128  e      41   42   43   43   43   45   45   63   66   86  112
//             r      41   42   42   43   43   45   53   63   74   86  125
//             s      41   42   42   43   50   52   53   63   79   90  129
//   128 x 128 e      42   43   44   44   45   46   47   54   58   74   86
//             r      42   43   43   44   44   46   49   55   63   75   98
//             s      43   46   46   48   47   50   50   58   65   73   98
//   256 x 256 e      50   50   51   51   51   52   52   58   59   67   82
//             r      50   50   50   51   51   53   54   58   62   68  104
//             s      50   52   53   54   55   61   59   63   65   82   88
//   gradient    rows 12   24   28   32   40   56   64   72   88  112  160
//   32 x 256  e      43   44   44   44   84   86   86  133  130  171  222
//             r      44   43   62   62   85  106  104  124  152  185  229
//             s      60   61   61   62   81  102  102  122  143  164  225
//   64 x 256  e      51   51   51   51   52   54   54  104  104  104  162
//             r      51   51   51   52   53   77   78  100  104  125  153
//             s      73   73   74   74   75   77   78   98  101  124  152
//   256 x 256 e      69   69   69   68   69   71   71   76   76   79   97
//             r      69   68   68   68   69   72   73   73   76   81   94
//             s      68   73   82  109  112  119  134  134  137  138  142
// The 32-row tile ends at 24 rows and not at the 32 that it can hold: with uneven rows some
// expert has more from about 28 on.  The gradient's 64-row tile ends between where it loses
// at random (about 56) and where it does with popular experts (above 112).
// Without FAST there are the middle and the largest tile.
constexpr int64_t kRows32 = 24, kRows64 = 64, kRows128 = 128, kRowsDgrad64 = 88;

template <bool FWD>
bqm_status launch_tiles(MxParams p, hipStream_t s, const char *what) {
  const int64_t ncols = FWD ? p.N : p.K, alen = FWD ? p.K / 2 : 2 * (int64_t)p.N, most = (int64_t)1 << 32;
  const bool fast = alen >= 128 && (FWD || p.K % 128 == 0) && (p.perm ? p.xrows : 256) * alen < most &&
                    (int64_t)p.N * (p.K / 2) < most;
  auto go = [&](auto WM, auto TM, auto TN, auto FAST, auto OCC, auto NS) {
    constexpr int BM = 32 * WM.value * TM.value, BN = 32 * (4 / WM.value) * TN.value;
    p.NT = (int)cdiv(ncols, BN);
    // at most R / BM + E row tiles; as many workgroups as the chip holds at once
    const int64_t tiles = (p.R / BM + (p.E < p.R ? p.E : p.R)) * p.NT, slots = (int64_t)kCUs * OCC.value;
    const unsigned grid = (unsigned)(cdiv(tiles < slots ? tiles : slots, 8) * 8);
    mx_tiles<WM.value, TM.value, TN.value, FWD, FAST.value, OCC.value, NS.value><<<grid, NTHR, 0, s>>>(p);
  };
  constexpr std::integral_constant<int, 1> one;
  constexpr std::integral_constant<int, 2> two;
  constexpr std::integral_constant<int, 3> three;
  constexpr std::integral_constant<int, 4> four;
  constexpr std::true_type yes;
  constexpr std::false_type no;
  const int64_t E = p.E;
  if constexpr (FWD) {
    if (p.R >= kRows128 * E)
      fast ? go(two, four, four, yes, one, two) : go(two, four, four, no, one, two);
    else if (!fast)
      go(two, two, two, no, two, two);
    else if (p.R >= kRows64 * E)
      go(two, two, two, yes, two, two);
    else if (p.R >= kRows32 * E)
      go(two, one, two, yes, two, two);
    else
      go(one, one, one, yes, three, two);
  } else {
    if (p.R >= kRowsDgrad64 * E)
      fast ? go(two, four, four, yes, one, two) : go(two, four, four, no, one, two);
    else if (!fast)
      go(two, one, four, no, one, four);
    else if (p.R >= kRows32 * E)
      go(two, one, four, yes, one, four);
    else
      go(one, one, two, yes, one, four);
  }
  return launch_status(what);
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
  p.R = R;
  p.out = y;
  return launch_tiles<true>(p, as_stream(stream), who);
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
  p.R = R;
  p.out = dx;
  return launch_tiles<false>(p, as_stream(stream), who);
}
