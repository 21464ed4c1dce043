// Rows between token order and expert order.  Pair f = t k + j (token t, slot j) stands at
// row inv[f] of the expert-ordered tensors, as bqm_permute gives it; a pair whose place lies
// outside [0, n) (n = *n_rows, or R) has been dropped and takes no part.
//   rows[inv[f]] = x[t]                                     (bqm_dispatch)
//   out[t] = residual[t] + sum_j w[f] y[inv[f]]             (bqm_combine; without w the
//                                                            gradient of dispatch)
//   dy[inv[f]] = w[f] dout[t],  dw[f] = <dout[t], y[inv[f]]>  (bqm_combine_grad)
//
// All three go by tokens, so that a token's row is read or written once and only the k rows
// of its pairs are spread: the bytes are the least there are, T H + R H (twice R H for the
// gradient), and HBM bounds them.  A lane holds 8 consecutive elements (16-byte accesses;
// one element where H is no multiple of 8) of the token and of several of its rows at a
// time, all loaded before the first is used.  The experts' rows are read, and all results
// written, past the caches, the tokens' rows are read through them: 16384 x 8 x 6144 without
// dropped pairs, dispatch 307 us (379 with everything past them, 366 with nothing), combine with a
// residual 309 (355, 392), gradient 640 (680, 687), which are 5.9, 6.5 and 5.3 TB/s.  With 5% of the
// pairs dropped 298, 296 and 597 us, 5.8, 6.5 and 5.5 TB/s of what is then moved.  One element per
// lane: 16384 x 8 x 6145 868, 879 and 961 us, 2.1, 2.3 and 3.6 TB/s.
#include "common.h"

namespace bqm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Pairs in flight per lane, G: 8 for up to kFewTokens tokens, where a load's latency counts
// (gradient of 64 x 8 x 6144 9.1 us, 10.2 with 4), 4 for more, where the registers of 8 cost
// workgroups in flight (16384 x 2 x 768: combine 20.0 against 18.0 us, gradient 32.6 against 28.1;
// 16384 x 8 x 256 33.5 against 29.6, but 16384 x 8 x 128 16.1 against 18.7; 16384 x 8 x 6144 the
// same within 1%).
constexpr int64_t kFewTokens = 512;
// Units per row up to which a wave takes several tokens (16384 x 8 x 256 and x 64: combine 14.2
// and 7.5 us, 20.0 and 16.2 with a token per wave; gradient 29.7 and 12.8 against 39.3 and 28.1).
constexpr int kPacked = 32;
// Lanes per token: gradient of 64 x 8 x 6144 9.1 us, 11.7 with up to 256; combine of 16384 x 8 x
// 6144 308 against 324, dispatch 308 against 304.
constexpr int kMaxThreads = 1024;
constexpr int64_t kMaxBlocks = 1 << 21;  // of kMaxThreads: a launch takes less than 2^32 threads in x

struct RowsParams {
  const uint16_t *x;  // dispatch: x; combine: residual or NULL; gradient: dout
  const uint16_t *y;  // combine, gradient: expert rows
  const int32_t *inv, *n_rows;
  const float *w;
  uint16_t *out;      // dispatch: rows; combine: out; gradient: dy or NULL
  float *dw;
  int64_t T, R;
  int k;
  uint32_t upr;       // units (of V elements) per row
  uint32_t span;      // units per workgroup in y (all, for the gradient)
  int logL;           // packed: lanes per token
};

// V bf16 values of a row
template <int V>
struct Unit;
template <>
struct Unit<8> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const u32x4 *>(p); }
  __device__ __forceinline__ void load_once(const uint16_t *p) {
    v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
  }
  __device__ __forceinline__ void store(uint16_t *p) const {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
  }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]); }
  __device__ __forceinline__ void set(const float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16_rne(f[2 * i], f[2 * i + 1]);
  }
};
template <>
struct Unit<1> {
  uint16_t v;
  __device__ __forceinline__ void load(const uint16_t *p) { v = *p; }
  __device__ __forceinline__ void load_once(const uint16_t *p) { v = *p; }
  __device__ __forceinline__ void store(uint16_t *p) const { *p = v; }
  __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)v << 16); }
  __device__ __forceinline__ void set(const float *f) { v = (uint16_t)pack_bf16_rne(f[0], 0.0f); }
};

__device__ __forceinline__ int64_t live_rows(const RowsParams &p) {
  if (!p.n_rows) return p.R;
  const int64_t n = *p.n_rows;
  return n < p.R ? n : p.R;
}

// The token and the units of this lane.  PACKED: 2^logL lanes of a wave per token; otherwise a
// workgroup per token (and part of its units), its token in scalar registers.
template <bool PACKED>
struct Place {
  int64_t t;
  uint32_t c, step, end;
  __device__ __forceinline__ explicit Place(const RowsParams &p) {
    const int64_t b = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if constexpr (PACKED) {
      t = (b * blockDim.x + threadIdx.x) >> p.logL;
      c = threadIdx.x & ((1u << p.logL) - 1);
      step = 1u << p.logL;
      end = t < p.T ? p.upr : 0;
    } else {
      t = b;
      c = blockIdx.y * p.span + threadIdx.x;
      step = blockDim.x;
      end = t < p.T ? min((blockIdx.y + 1) * p.span, p.upr) : 0;
    }
  }
};

// the place of the token's pair j, or -1
__device__ __forceinline__ int64_t place(const RowsParams &p, int64_t t, int j, int64_t live) {
  if (j >= p.k) return -1;
  const int64_t at = p.inv[t * p.k + j];
  return at >= 0 && at < live ? at : -1;
}

template <int V, bool PACKED>
__global__ void __launch_bounds__(kMaxThreads) dispatch_rows(RowsParams p) {
  const Place<PACKED> at(p);
  const int64_t live = live_rows(p);
  for (uint32_t c = at.c; c < at.end; c += at.step) {
    Unit<V> u;
    u.load(p.x + (at.t * p.upr + c) * V);
    for (int j = 0; j < p.k; ++j) {
      const int64_t row = place(p, at.t, j, live);
      if (row >= 0) u.store(p.out + (row * p.upr + c) * V);
    }
  }
}

template <int V, bool PACKED, int G>
__global__ void __launch_bounds__(kMaxThreads) combine_rows(RowsParams p) {
  const Place<PACKED> at(p);
  const int64_t live = live_rows(p);
  for (uint32_t c = at.c; c < at.end; c += at.step) {
    const int64_t o = (at.t * p.upr + c) * V;
    Unit<V> r;
    if (p.x) r.load(p.x + o);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += G) {
      Unit<V> u[G];
      int64_t row[G];
      float w[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        row[j] = place(p, at.t, j0 + j, live);
        w[j] = p.w && row[j] >= 0 ? p.w[at.t * p.k + j0 + j] : 1.0f;
      }
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (row[j] >= 0) u[j].load_once(p.y + (row[j] * p.upr + c) * V);
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (row[j] >= 0) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += w[j] * u[j].get(i);
        }
    }
    if (p.x) {
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += r.get(i);
    }
    r.set(acc);
    r.store(p.out + o);
  }
}

template <int V, bool PACKED, int G>
__global__ void __launch_bounds__(kMaxThreads) combine_grad_rows(RowsParams p) {
  __shared__ float part[kMaxThreads / 64][G];
  const Place<PACKED> at(p);
  const int64_t live = live_rows(p);
  for (int j0 = 0; j0 < p.k; j0 += G) {
    int64_t row[G];
    float w[G], dot[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      row[j] = at.t < p.T ? place(p, at.t, j0 + j, live) : -1;
      w[j] = p.w && row[j] >= 0 ? p.w[at.t * p.k + j0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (uint32_t c = at.c; c < at.end; c += at.step) {
      Unit<V> d, u[G];
      d.load(p.x + (at.t * p.upr + c) * V);
      if (p.dw) {
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (row[j] >= 0) u[j].load_once(p.y + (row[j] * p.upr + c) * V);
      }
      if (p.out) {
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (row[j] >= 0) {
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = w[j] * d.get(i);
            Unit<V> o;
            o.set(f);
            o.store(p.out + (row[j] * p.upr + c) * V);
          }
      }
      if (p.dw) {
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (row[j] >= 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] += d.get(i) * u[j].get(i);
          }
      }
    }
    if (!p.dw) continue;
    // the lanes' sums in a fixed butterfly, then the waves' in order
#pragma unroll
    for (int j = 0; j < G; ++j)
      for (int m = PACKED ? 1 << p.logL >> 1 : 32; m >= 1; m >>= 1) dot[j] += __shfl_xor(dot[j], m, 64);
    if constexpr (PACKED) {
      if (at.t < p.T && at.c == 0) {
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (j0 + j < p.k) p.dw[at.t * p.k + j0 + j] = dot[j];
      }
    } else {
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int j = 0; j < G; ++j) part[threadIdx.x >> 6][j] = dot[j];
      }
      __syncthreads();
      if (at.t < p.T && threadIdx.x < G && j0 + (int)threadIdx.x < p.k) {
        float s = 0.0f;
        for (unsigned q = 0; q < blockDim.x / 64; ++q) s += part[q][threadIdx.x];
        p.dw[at.t * p.k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// sizes and the tensors that the three share
bqm_status check_rows(const char *who, const int32_t *inv, int64_t T, int64_t H, int32_t k) {
  BQM_REQUIRE(T >= 0, BQM_ERR_INVALID_ARG, "%s: T < 0", who);
  BQM_REQUIRE(k >= 1, BQM_ERR_SHAPE, "%s: k=%d < 1", who, k);
  BQM_REQUIRE(H >= 1 && H < ((int64_t)1 << 24), BQM_ERR_SHAPE, "%s: H=%lld outside [1, 2^24)", who, (long long)H);
  BQM_REQUIRE(T < ((int64_t)1 << 31) && T * k < ((int64_t)1 << 31), BQM_ERR_SHAPE, "%s: T * k reaches 2^31", who);
  if (T == 0) return BQM_OK;
  BQM_REQUIRE(inv, BQM_ERR_INVALID_ARG, "%s: inv is NULL", who);
  BQM_REQUIRE(aligned16(inv), BQM_ERR_ALIGN, "%s: inv not 16-byte aligned", who);
  return BQM_OK;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// whole: a workgroup has to see a token's whole row
template <typename Launch>
void go(RowsParams &p, int64_t H, bool whole, Launch launch) {
  const int V = H % 8 ? 1 : 8;
  p.upr = (uint32_t)(H / V);
  dim3 grid(1, 1, 1), block(256, 1, 1);
  const bool packed = p.upr <= kPacked;
  int64_t blocks = p.T;
  if (packed) {
    p.logL = 0;
    while ((1u << p.logL) < p.upr) ++p.logL;
    blocks = cdiv(p.T << p.logL, 256);
  } else {
    // parts of even width, in whole waves
    const uint32_t parts = whole ? 1 : (uint32_t)cdiv(p.upr, kMaxThreads);
    p.span = (uint32_t)cdiv(p.upr, parts);
    const uint32_t turns = (uint32_t)cdiv(p.span, kMaxThreads);
    block.x = (unsigned)(cdiv(cdiv(p.span, turns), 64) * 64);
    grid.y = parts;
  }
  grid.x = (unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
  grid.z = (unsigned)cdiv(blocks, kMaxBlocks);
  launch(V, packed, grid, block);
}

}  // namespace
}  // namespace bqm

using namespace bqm;

// kernel<V, PACKED, extra ..>
#define BQM_ROWS_LAUNCH(kernel, ...)                                                    \
  [&](int V, bool packed, dim3 grid, dim3 block) {                                      \
    const hipStream_t s = as_stream(stream);                                            \
    if (V == 8)                                                                         \
      packed ? kernel<8, true, ##__VA_ARGS__><<<grid, block, 0, s>>>(p)                 \
             : kernel<8, false, ##__VA_ARGS__><<<grid, block, 0, s>>>(p);               \
    else                                                                                \
      packed ? kernel<1, true, ##__VA_ARGS__><<<grid, block, 0, s>>>(p)                 \
             : kernel<1, false, ##__VA_ARGS__><<<grid, block, 0, s>>>(p);               \
  }

extern "C" bqm_status bqm_dispatch(const uint16_t *x, const int32_t *inv, int64_t T, int64_t H, int32_t k,
                                   const int32_t *n_rows, uint16_t *rows, void *stream) {
  const char *who = "bqm_dispatch";
  bqm_status st = check_rows(who, inv, T, H, k);
  if (st != BQM_OK || T == 0) return st;
  BQM_REQUIRE(x && rows, BQM_ERR_INVALID_ARG, "%s: x or rows is NULL", who);
  BQM_REQUIRE(aligned16(x) && aligned16(rows), BQM_ERR_ALIGN, "%s: x or rows not 16-byte aligned", who);
  BQM_REQUIRE(aligned4(n_rows), BQM_ERR_ALIGN, "%s: n_rows not 4-byte aligned", who);
  RowsParams p = {};
  p.x = x, p.inv = inv, p.n_rows = n_rows, p.out = rows, p.T = T, p.R = T * k, p.k = k;
  go(p, H, false, BQM_ROWS_LAUNCH(dispatch_rows));
  return launch_status(who);
}

extern "C" bqm_status bqm_combine(const uint16_t *y, const int32_t *inv, const float *topk_w, const uint16_t *residual,
                                  int64_t T, int64_t H, int32_t k, const int32_t *n_rows, uint16_t *out, void *stream) {
  const char *who = "bqm_combine";
  bqm_status st = check_rows(who, inv, T, H, k);
  if (st != BQM_OK || T == 0) return st;
  BQM_REQUIRE(y && out, BQM_ERR_INVALID_ARG, "%s: y or out is NULL", who);
  BQM_REQUIRE(aligned16(y) && aligned16(out) && aligned16(topk_w) && aligned16(residual), BQM_ERR_ALIGN,
              "%s: pointer not 16-byte aligned", who);
  BQM_REQUIRE(aligned4(n_rows), BQM_ERR_ALIGN, "%s: n_rows not 4-byte aligned", who);
  RowsParams p = {};
  p.x = residual, p.y = y, p.inv = inv, p.n_rows = n_rows, p.w = topk_w, p.out = out, p.T = T, p.R = T * k, p.k = k;
  if (T <= kFewTokens)
    go(p, H, false, BQM_ROWS_LAUNCH(combine_rows, 8));
  else
    go(p, H, false, BQM_ROWS_LAUNCH(combine_rows, 4));
  return launch_status(who);
}

extern "C" bqm_status bqm_combine_grad(const uint16_t *dout, const uint16_t *y, const int32_t *inv, const float *topk_w,
                                       int64_t T, int64_t H, int32_t k, const int32_t *n_rows, uint16_t *dy,
                                       float *dtopk_w, void *stream) {
  const char *who = "bqm_combine_grad";
  bqm_status st = check_rows(who, inv, T, H, k);
  if (st != BQM_OK || T == 0) return st;
  BQM_REQUIRE(dy || dtopk_w, BQM_ERR_INVALID_ARG, "%s: dy and dtopk_w are both NULL", who);
  BQM_REQUIRE(dout, BQM_ERR_INVALID_ARG, "%s: dout is NULL", who);
  BQM_REQUIRE(y || !dtopk_w, BQM_ERR_INVALID_ARG, "%s: dtopk_w needs y", who);
  BQM_REQUIRE(aligned16(dout) && aligned16(y) && aligned16(topk_w) && aligned16(dy) && aligned16(dtopk_w),
              BQM_ERR_ALIGN, "%s: pointer not 16-byte aligned", who);
  BQM_REQUIRE(aligned4(n_rows), BQM_ERR_ALIGN, "%s: n_rows not 4-byte aligned", who);
  RowsParams p = {};
  p.x = dout, p.y = y, p.inv = inv, p.n_rows = n_rows, p.w = topk_w, p.out = dy, p.dw = dtopk_w;
  p.T = T, p.R = T * k, p.k = k;
  if (T <= kFewTokens)
    go(p, H, dtopk_w != nullptr, BQM_ROWS_LAUNCH(combine_grad_rows, 8));
  else
    go(p, H, dtopk_w != nullptr, BQM_ROWS_LAUNCH(combine_grad_rows, 4));
  return launch_status(who);
}
#undef BQM_ROWS_LAUNCH
