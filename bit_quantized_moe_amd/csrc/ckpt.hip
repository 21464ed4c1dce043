// SwiGLU with an 8-bit activation checkpoint: the forward writes a = silu(g) u and keeps
// h = [g, u] in 8 bits, the backward reads those 8 bits instead of h.
//
// The checkpoint holds each 32-element block of a row of h as E4M3 values times a power
// of two 2^s, the smallest with max|h| 2^-s <= 448 (so nothing saturates): 1.03 bytes per
// value where bf16 takes 2.  With g~, u~ the values it stands for, sig = 1 / (1 + e^-g~)
// and w the row's routing weight,
//   dg = w da u~ sig (1 + g~ (1 - sig)),   du = w da g~ sig,   dw = sum_i da_i g~_i sig_i u~_i.
//
// Both kernels are bound by HBM: forward 4 + 2 + 2.06 bytes per element of a, backward
// 2.06 + 2 + 4.  A lane holds 8 consecutive elements of a row's g and the same 8 of its u
// (16-byte loads and stores), so a quad of lanes shares a block of each and finds its
// maximum with two quad-permute moves.  131072 x 2048: forward 350 us, backward 355 us, 6.1
// to 6.2 TB/s; 808 x 768: 4 and 5 us, of which a launch with no work is 2.
#include "common.h"

namespace bqm {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kE8M0NaN = 255u;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x4 ld_nt(const uint16_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ void st_nt(uint16_t *p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}

__device__ __forceinline__ uint32_t quad_max_u(uint32_t v) {
  uint32_t t = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);  // quad_perm 1,0,3,2
  v = v > t ? v : t;
  t = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);  // quad_perm 2,3,0,1
  return v > t ? v : t;
}

__device__ __forceinline__ uint32_t absmax8(u32x4 v) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = v[i] & 0x7FFFu, b = (v[i] >> 16) & 0x7FFFu, c = a > b ? a : b;
    m = m > c ? m : c;
  }
  return m;
}

// E8M0 code of a block whose largest magnitude has the bf16 bits mx: with
// max = (1 + M / 128) 2^(E - 127), max 2^-s <= 448 = 1.75 2^8 asks for s = E - 135,
// or one more where M > 96, which is where M + 31 carries into the exponent
__device__ __forceinline__ uint32_t ckpt_scale(uint32_t mx) {
  if (mx >= 0x7F80u) return kE8M0NaN;
  const uint32_t c = (mx + 31u) >> 7;
  return c > 8u ? c - 8u : 0u;
}

__device__ __forceinline__ float e8m0(uint32_t c) {
  return c == kE8M0NaN ? __uint_as_float(0x7FC00000u) : __uint_as_float(c ? c << 23 : 0x00400000u);
}

// 2^-s of a scale code (codes reach 247; a block marked NaN has no use for it)
__device__ __forceinline__ float inv_scale(uint32_t c) { return __uint_as_float((254u - (c < 254u ? c : 254u)) << 23); }

// 8 bf16 values -> 8 E4M3 bytes; r = 2^-s, the products exact in FP32 and at most 448
__device__ __forceinline__ u32x2 to_e4m3(u32x4 v, float r) {
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int t = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(v[2 * i]) * r, bf16_hi(v[2 * i]) * r, 0, false);
    o[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(v[2 * i + 1]) * r, bf16_hi(v[2 * i + 1]) * r, t, true);
  }
  return o;
}

__device__ __forceinline__ float sigmoid_f(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// silu(g) u of a bf16 pair in FP32, rounded to bf16 once
__device__ __forceinline__ uint32_t swiglu_pair(uint32_t g, uint32_t u) {
  const float g0 = bf16_lo(g), g1 = bf16_hi(g);
  return pack_bf16_rne(g0 * sigmoid_f(g0) * bf16_lo(u), g1 * sigmoid_f(g1) * bf16_hi(u));
}

// 8 bf16 values -> MXFP4 codes of their block (the rule of bqm_quantize_mxfp4)
__device__ __forceinline__ uint32_t to_mxfp4(u32x4 v, uint32_t mx, uint32_t &sc) {
  if (mx >= 0x7F80u) {
    sc = kE8M0NaN;
    return 0u;
  }
  const uint32_t ex = mx >> 7;
  sc = ex > 2u ? ex - 2u : 0u;
  const float r = __uint_as_float((254u - sc) << 23);
  uint32_t c = 0u;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v[0]) * r, bf16_hi(v[0]) * r, 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v[1]) * r, bf16_hi(v[1]) * r, 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v[2]) * r, bf16_hi(v[2]) * r, 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v[3]) * r, bf16_hi(v[3]) * r, 1.0f, 3);
  return c;
}

__device__ __forceinline__ int64_t live_rows(int64_t R, const int32_t *n_rows) {
  if (!n_rows) return R;
  const int64_t n = *n_rows;
  return n < 0 ? 0 : (n < R ? n : R);
}

constexpr int kFwdIter = 2;
constexpr int kFwdUnits = kFwdIter * kThreads;

// upr: 8-element units per row of a (I / 8); a workgroup takes kFwdUnits consecutive ones
__global__ void __launch_bounds__(kThreads) swiglu_ckpt_fwd(const uint16_t *__restrict__ h, int64_t R, uint32_t upr,
                                                            const int32_t *__restrict__ n_rows,
                                                            uint8_t *__restrict__ h8, uint8_t *__restrict__ h8s,
                                                            uint16_t *__restrict__ a, uint32_t *__restrict__ aq,
                                                            uint8_t *__restrict__ aqs) {
  const int64_t total = live_rows(R, n_rows) * upr;
  const int64_t base = (int64_t)blockIdx.x * kFwdUnits;
  if (base >= total) return;
  const int64_t row0 = base / upr;
  const uint32_t rest = (uint32_t)(base - row0 * upr);
  u32x4 g[kFwdIter], u[kFwdIter];
  int64_t row[kFwdIter];
  uint32_t col[kFwdIter];
#pragma unroll
  for (int it = 0; it < kFwdIter; ++it) {
    const int64_t left = total - base - 1;
    uint32_t t = it * kThreads + threadIdx.x;
    t = t < left ? t : (uint32_t)left;
    const uint32_t o = rest + t, q = o / upr;
    row[it] = row0 + q;
    col[it] = o - q * upr;
    const uint16_t *hr = h + row[it] * 16 * upr + 8 * col[it];
    g[it] = ld_nt(hr);
    u[it] = ld_nt(hr + 8 * upr);
  }
#pragma unroll
  for (int it = 0; it < kFwdIter; ++it) {
    // total is a multiple of 4, so a quad of lanes is in range or out as one
    const bool in = base + it * kThreads + threadIdx.x < total;
    const uint32_t gs = ckpt_scale(quad_max_u(absmax8(g[it]))), us = ckpt_scale(quad_max_u(absmax8(u[it])));
    const u32x2 g8 = to_e4m3(g[it], inv_scale(gs)), u8 = to_e4m3(u[it], inv_scale(us));
    u32x4 av;
#pragma unroll
    for (int i = 0; i < 4; ++i) av[i] = swiglu_pair(g[it][i], u[it][i]);
    uint32_t as = 0u, ac = 0u;
    if (aq) ac = to_mxfp4(av, quad_max_u(absmax8(av)), as);
    if (in) {
      const int64_t at = row[it] * 16 * upr + 8 * col[it];
      __builtin_nontemporal_store(g8, reinterpret_cast<u32x2 *>(h8 + at));
      __builtin_nontemporal_store(u8, reinterpret_cast<u32x2 *>(h8 + at + 8 * upr));
      if (a) st_nt(a + row[it] * 8 * upr + 8 * col[it], av);
      if (aq) aq[row[it] * upr + col[it]] = ac;
      if ((threadIdx.x & 3) == 0) {
        const int64_t sat = (row[it] * 2 * upr + col[it]) >> 2;
        h8s[sat] = (uint8_t)gs;
        h8s[sat + (upr >> 2)] = (uint8_t)us;
        if (aq) aqs[(row[it] * upr + col[it]) >> 2] = (uint8_t)as;
      }
    }
  }
}

// pair P of 4 E4M3 bytes -> two floats
template <bool HI>
__device__ __forceinline__ f32x2 e4m3_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_pk_f32_fp8((int)w, HI);
}

// L = 2^logL lanes per row (up to 64): with few elements a wave takes 64 / L rows
__global__ void __launch_bounds__(kThreads) swiglu_ckpt_bwd(const uint8_t *__restrict__ h8,
                                                            const uint8_t *__restrict__ h8s,
                                                            const uint16_t *__restrict__ da,
                                                            const int32_t *__restrict__ perm,
                                                            const float *__restrict__ tw, int64_t R, uint32_t upr,
                                                            int logL, const int32_t *__restrict__ n_rows,
                                                            uint16_t *__restrict__ dh, float *__restrict__ dtw) {
  const int64_t live = live_rows(R, n_rows);
  const int L = 1 << logL;
  const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> logL;
  const uint32_t l = threadIdx.x & (L - 1);
  if (row >= R) return;
  // a pair's index from outside [0, R) belongs to no pair: weight 0, no gradient
  int64_t f = perm ? perm[row] : row;
  const bool fok = f >= 0 && f < R;
  if (row >= live) {
    if (dtw && l == 0 && fok) dtw[f] = 0.0f;
    return;
  }
  const float w = tw ? (fok ? tw[f] : 0.0f) : 1.0f;
  const uint8_t *hr = h8 + row * 16 * upr;
  const uint8_t *sr = h8s + row * (upr >> 1);
  const uint16_t *dr = da + row * 8 * upr;
  uint16_t *o = dh + row * 16 * upr;
  float dot = 0.0f;
  for (uint32_t c = l; c < upr; c += L) {
    const u32x2 g8 = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(hr + 8 * c));
    const u32x2 u8 = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(hr + 8 * upr + 8 * c));
    const u32x4 d = ld_nt(dr + 8 * c);
    const float gs = e8m0(sr[c >> 2]), us = e8m0(sr[(upr + c) >> 2]);
    u32x4 dg, du;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 gp = (i & 1) ? e4m3_pair<true>(g8[i >> 1]) : e4m3_pair<false>(g8[i >> 1]);
      const f32x2 up = (i & 1) ? e4m3_pair<true>(u8[i >> 1]) : e4m3_pair<false>(u8[i >> 1]);
      float dgv[2], duv[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float g = gp[j] * gs, u = up[j] * us;
        const float dv = j ? bf16_hi(d[i]) : bf16_lo(d[i]);
        const float s = sigmoid_f(g), gsg = g * s;
        dot += dv * (gsg * u);  // da times a: da silu(g) can overflow where a and the sum are finite
        const float wd = w * dv;
        dgv[j] = wd * (u * s) * (1.0f + g * (1.0f - s));
        duv[j] = wd * gsg;
      }
      dg[i] = pack_bf16_rne(dgv[0], dgv[1]);
      du[i] = pack_bf16_rne(duv[0], duv[1]);
    }
    st_nt(o + 8 * c, dg);
    st_nt(o + 8 * upr + 8 * c, du);
  }
  if (dtw) {  // the row's lanes added in a fixed butterfly
    for (int m = L >> 1; m >= 1; m >>= 1) dot += __shfl_xor(dot, m, 64);
    if (l == 0 && fok) dtw[f] = dot;
  }
}

// the sizes and the four tensors both directions share
bqm_status check_ckpt(const char *who, const void *h8, const void *h8s, int64_t R, int64_t I) {
  BQM_REQUIRE(R >= 0, BQM_ERR_INVALID_ARG, "%s: R < 0", who);
  BQM_REQUIRE(I >= 32 && I % 32 == 0, BQM_ERR_SHAPE, "%s: I=%lld is not a positive multiple of 32", who, (long long)I);
  BQM_REQUIRE(I < ((int64_t)1 << 24) && R < ((int64_t)1 << 31), BQM_ERR_SHAPE, "%s: tensor too large", who);
  if (R == 0) return BQM_OK;
  BQM_REQUIRE(h8 && h8s, BQM_ERR_INVALID_ARG, "%s: h8 or h8_scales is NULL", who);
  BQM_REQUIRE(aligned16(h8) && aligned16(h8s), BQM_ERR_ALIGN, "%s: h8 or h8_scales not 16-byte aligned", who);
  return BQM_OK;
}

}  // namespace
}  // namespace bqm

using namespace bqm;

extern "C" bqm_status bqm_swiglu_ckpt_fwd(const uint16_t *h, int64_t R, int64_t I, const int32_t *n_rows, uint8_t *h8,
                                          uint8_t *h8_scales, uint16_t *a, bqm_qtensor *aq, void *stream) {
  const char *who = "bqm_swiglu_ckpt_fwd";
  bqm_status st = check_ckpt(who, h8, h8_scales, R, I);
  if (st != BQM_OK) return st;
  if (aq) {
    BQM_REQUIRE(aq->fmt == BQM_FMT_MXFP4, BQM_ERR_INVALID_ARG, "%s: aq->fmt must be BQM_FMT_MXFP4", who);
    BQM_REQUIRE(aq->n_mat == 1 && aq->rows == R && aq->cols == I, BQM_ERR_SHAPE, "%s: aq must be [1, R, I]", who);
  }
  if (R == 0) return BQM_OK;
  BQM_REQUIRE(h, BQM_ERR_INVALID_ARG, "%s: h is NULL", who);
  BQM_REQUIRE(aligned16(h) && aligned16(a), BQM_ERR_ALIGN, "%s: h or a not 16-byte aligned", who);
  if (aq) {
    BQM_REQUIRE(aq->codes && aq->scales, BQM_ERR_INVALID_ARG, "%s: aq codes/scales pointer is NULL", who);
    BQM_REQUIRE(aligned16(aq->codes) && aligned16(aq->scales), BQM_ERR_ALIGN, "%s: aq not 16-byte aligned", who);
  }
  const int64_t grid = cdiv(R * (I / 8), kFwdUnits);
  BQM_REQUIRE(grid < ((int64_t)1 << 31), BQM_ERR_SHAPE, "%s: tensor too large", who);
  swiglu_ckpt_fwd<<<(unsigned)grid, kThreads, 0, as_stream(stream)>>>(
      h, R, (uint32_t)(I / 8), n_rows, h8, h8_scales, a, aq ? reinterpret_cast<uint32_t *>(aq->codes) : nullptr,
      aq ? reinterpret_cast<uint8_t *>(aq->scales) : nullptr);
  return launch_status("swiglu_ckpt_fwd");
}

extern "C" bqm_status bqm_swiglu_ckpt_bwd(const uint8_t *h8, const uint8_t *h8_scales, const uint16_t *da,
                                          const int32_t *perm, const float *topk_w, int64_t R, int64_t I,
                                          const int32_t *n_rows, uint16_t *dh, float *dtopk_w, void *stream) {
  const char *who = "bqm_swiglu_ckpt_bwd";
  bqm_status st = check_ckpt(who, h8, h8_scales, R, I);
  if (st != BQM_OK) return st;
  if (R == 0) return BQM_OK;
  BQM_REQUIRE(da && dh, BQM_ERR_INVALID_ARG, "%s: da or dh is NULL", who);
  BQM_REQUIRE(aligned16(da) && aligned16(dh) && aligned16(perm) && aligned16(topk_w) && aligned16(dtopk_w),
              BQM_ERR_ALIGN, "%s: pointer not 16-byte aligned", who);
  const uint32_t upr = (uint32_t)(I / 8);
  int logL = 2;
  while (logL < 6 && (1u << logL) < upr) ++logL;
  while ((R << logL) >= (int64_t)1 << 32) --logL;  // a launch has less than 2^32 threads
  const int64_t grid = cdiv(R << logL, kThreads);
  swiglu_ckpt_bwd<<<(unsigned)grid, kThreads, 0, as_stream(stream)>>>(h8, h8_scales, da, perm, topk_w, R, upr, logL,
                                                                      n_rows, dh, dtopk_w);
  return launch_status("swiglu_ckpt_bwd");
}
