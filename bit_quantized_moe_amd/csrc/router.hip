// The router's training: balance loss, z-loss and per-expert counts, and the gradient of
// the logits through the losses and the routing weights.
//
// Over the n tokens that count (valid[t] != 0), with p_t = softmax(l_t), c_e the routed
// pairs of expert e, f_e = c_e / (n k) and P_e = mean_t p_te:
//   L_b = E sum_e f_e P_e,    L_z = mean_t lse(l_t)^2.
// Gradient (the counts are constants), with g_b, g_z the losses' gradients, q_j = p_{t,i_j}:
//   G_e = g_b E f_e / n + sum_{j: i_j = e} dq_j,
//   dl_te = p_te (G_e - sum_e' p_te' G_e') + (2 g_z / n) lse_t p_te,
// where dq_j = dw_j, or, with weights w_j = q_j / S, S = sum_j q_j,
// dq_j = (dw_j - sum_m w_m dw_m) / S.  In that second case the routing weights' share of
// sum_e p_e G_e is zero, and their term is p_e (A_e - D m_e) / S with A_e = sum of dw_j
// over j with i_j = e, m_e their number, D = sum_e p_e A_e / S.
//
// Bound by HBM: each direction reads the T E logits once (the softmax is recomputed from
// registers in the backward rather than kept, which would cost a write and a read of the
// same size); the gradient is written once.  A token is held by 2^n lanes, 4 NV logits a
// lane, so a row is read with 16-byte loads and all its sums are moves between lanes.
#include "common.h"

#include <type_traits>

namespace bqm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxE = 1024, kMaxK = 16;

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Reductions over groups of L lanes (a power of two); every lane gets the result.  Within
// 16 lanes by DPP moves, beyond that by exchanging rows of 16 and halves of the wave: vector
// instructions all, none of which waits for the LDS crossbar as a shuffle does.
__device__ __forceinline__ void swap_rows16(float v, float &a, float &b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap_halves(float v, float &a, float &b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
template <int L, class F>
__device__ __forceinline__ float group_reduce(float v, F op) {
  if constexpr (L >= 2) v = op(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false)));
  if constexpr (L >= 4) v = op(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false)));
  if constexpr (L >= 8) v = op(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false)));
  if constexpr (L >= 16) v = op(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false)));
  float a, b;
  if constexpr (L >= 32) {
    swap_rows16(v, a, b);
    v = op(a, b);
  }
  if constexpr (L >= 64) {
    swap_halves(v, a, b);
    v = op(a, b);
  }
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// e^x for x <= 0 within about an ulp: 2^(x log2 e) with the rounding of the product put back
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;
  const float t = x * kLog2e;
  if (x < -104.0f) return 0.0f;  // also -inf, where the correction below would be NaN
  const float r = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2e, -t));
  const float y = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(y, r * kLn2, y);
}

// A token's logits in its group's registers: slot (v, c) of lane l is expert
// 4 (v L + l) + c with 16-byte loads (E % 4 == 0), else (4 v + c) L + l.
template <int L, int NV, bool VEC>
__device__ __forceinline__ int expert_of(int v, int c, int l) {
  return VEC ? 4 * (v * L + l) + c : (4 * v + c) * L + l;
}

// orders this wave's LDS accesses for the compiler (the hardware keeps their order)
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// where expert e sits in the order (v, l, c) of the lanes' vectors without 16-byte loads
template <int L, int NV>
__device__ __forceinline__ int slot_of(int e) {
  const int l = e & (L - 1), q = e / L;  // q = 4 v + c
  return 4 * ((q >> 2) * L + l) + (q & 3);
}

template <int L, int NV, bool VEC>
__device__ __forceinline__ void load_row(const float *__restrict__ row, int E, int l, bool use, f32x4 (&x)[NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (VEC) {
      const int e = expert_of<L, NV, VEC>(v, 0, l);
      x[v] = use && e < E ? *reinterpret_cast<const f32x4 *>(row + e)
                          : f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = expert_of<L, NV, VEC>(v, c, l);
        x[v][c] = use && e < E ? row[e] : -INFINITY;
      }
    }
  }
}

// x <- e^(x - base), base the row's maximum (0 for a row of nothing but -inf); returns 1 / sum
// and the row's lse (both 0 for such a row, whose sum alone is 0: a row of -inf and NaN has a
// maximum of -inf too, as fmaxf passes NaN over, and its lse is NaN)
template <int L, int NV>
__device__ __forceinline__ float softmax_row(f32x4 (&x)[NV], float &lse, float &base) {
  float m = -INFINITY;
#pragma unroll
  for (int v = 0; v < NV; ++v) m = fmaxf(m, fmaxf(fmaxf(x[v][0], x[v][1]), fmaxf(x[v][2], x[v][3])));
  m = group_max<L>(m);
  base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[v][c] = exp_neg(x[v][c] - base);
      s += x[v][c];
    }
  s = group_sum<L>(s);
  lse = s == 0.0f ? 0.0f : m + logf(s);
  return s > 0.0f ? 1.0f / s : 0.0f;
}

// ---------------------------------------------------------------------------
// losses and counts
// ---------------------------------------------------------------------------
// Workspace: per workgroup of the first kernel, E sums of p (FP32), E counts and the sum
// of lse^2 and the tokens that count; then the finishing kernel's partial losses and its
// arrival counter.
struct LossWs {
  float *psum;        // [G][E]
  int32_t *counts;    // [G][E]
  float *z;           // [G]
  int32_t *n;         // [G]
  double *part;       // [kMaxE / kFinE]
  uint32_t *arrived;  // 1
};

constexpr int kFinE = 32;  // experts per workgroup of the finishing kernel

struct LossGeom {
  int G;  // workgroups of the first kernel
  size_t bytes;
};

// lanes that hold a token's logits, 4 each up to 256 experts
int lanes_of(int E) { return E <= 16 ? 4 : E <= 32 ? 8 : E <= 64 ? 16 : E <= 128 ? 32 : 64; }

// Workgroups of 16 waves, two per CU at most: 32 waves keep enough rows in flight (with 8
// waves per CU the 131072 x 256 batch took 62 us, with 32 and the next row in flight 34 us,
// 4.0 TB/s).  One workgroup per kTokMin tokens, so that a small batch writes few partial
// sums, but no more than get a token: with 32 experts or fewer a workgroup's groups of lanes
// take 128 or 256 tokens in one turn.  A batch of at most kOneTurns tokens per group of lanes
// goes to one workgroup, which forms the losses itself and saves the finishing kernel: a turn
// takes 0.8 us, the two kernels 8.3 us at 8 experts, 9.1 at 60, 12.7 at 256 and 21.6 at 1024
// (one with 8 turns: 9.6, 10.1, 10.7 and 20.4 us), and a launch costs the host 3.3 us.
constexpr int kSumThreads = 1024, kSumWaves = kSumThreads / 64;
constexpr int64_t kTokMin = 64, kOneTurns = 8;
LossGeom loss_geom(int64_t T, int32_t E) {
  const int64_t groups = kSumThreads / lanes_of(E);
  int64_t G = T <= kOneTurns * groups ? 1 : cdiv(T, groups > kTokMin ? groups : kTokMin);
  G = G > 512 ? 512 : G;
  LossGeom g;
  g.G = (int)G;
  g.bytes = align256((size_t)G * E * 4) * 2 + align256((size_t)G * 4) * 2 + align256(kMaxE / kFinE * sizeof(double)) + 256;
  return g;
}

LossWs loss_ws(void *ws, int G, int E) {
  LossWs w;
  char *p = reinterpret_cast<char *>(ws);
  w.psum = reinterpret_cast<float *>(p);
  p += align256((size_t)G * E * 4);
  w.counts = reinterpret_cast<int32_t *>(p);
  p += align256((size_t)G * E * 4);
  w.z = reinterpret_cast<float *>(p);
  p += align256((size_t)G * 4);
  w.n = reinterpret_cast<int32_t *>(p);
  p += align256((size_t)G * 4);
  w.part = reinterpret_cast<double *>(p);
  p += align256(kMaxE / kFinE * sizeof(double));
  w.arrived = reinterpret_cast<uint32_t *>(p);
  return w;
}

// the losses from sum_e c_e P_e n and sum_t lse^2 over the n tokens that count
__device__ __forceinline__ void write_losses(int E, int k, int32_t n, double b, double z, int32_t *counts, float *loss) {
  const double nn = (double)n;
  counts[E] = n;
  loss[0] = n > 0 ? (float)((double)E * b / (nn * nn * (double)k)) : 0.0f;
  loss[1] = n > 0 ? (float)(z / nn) : 0.0f;
}

template <int L, int NV, bool VEC>
__global__ void __launch_bounds__(kSumThreads) router_sums(const float *__restrict__ logits,
                                                        const int32_t *__restrict__ idx,
                                                        const uint8_t *__restrict__ valid, int64_t T, int E, int k,
                                                        LossWs w, int32_t *__restrict__ counts,
                                                        float *__restrict__ loss) {
  constexpr int kGroups = kSumThreads / L;
  extern __shared__ float ps[];  // [kSumWaves][E]: the waves' sums
  __shared__ int32_t hist[kMaxE];
  __shared__ float zs[kSumWaves];
  __shared__ int32_t ns[kSumWaves];
  const int tid = threadIdx.x, l = tid & (L - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int grp = L == 64 ? wave : tid / L;
  for (int e = tid; e < E; e += kSumThreads) hist[e] = 0;
  if (blockIdx.x == 0 && tid == 0) *w.arrived = 0u;
  __syncthreads();
  f32x4 acc[NV] = {};
  float z = 0.0f;
  int32_t n = 0;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t t = (int64_t)blockIdx.x * kGroups + grp;
  // the next token's row, flag and index are loaded while this one's are reduced
  f32x4 x[NV], nx[NV];
  bool use = false, nuse = false;
  int ix = -1, nix = -1;
  auto fetch = [&](int64_t tt) {
    nuse = !valid || valid[tt];
    load_row<L, NV, VEC>(logits + tt * E, E, l, true, nx);
    nix = l < k ? idx[tt * k + l] : -1;
  };
  if (t < T) fetch(t);
  for (; t < T; t += step) {
    use = nuse;
    ix = nix;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[v][c] = use ? nx[v][c] : -INFINITY;
    if (t + step < T) fetch(t + step);
    if (use) {
      if ((unsigned)ix < (unsigned)E) atomicAdd(&hist[ix], 1);
      for (int j = l + L; j < k; j += L) {  // groups of fewer lanes than k
        const int e = idx[t * k + j];
        if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
      }
    }
    float lse, base;
    const float inv = softmax_row<L, NV>(x, lse, base);
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] += x[v] * inv;
    if (use && l == 0) {
      z += lse * lse;
      ++n;
    }
  }
  // the groups of a wave added in a fixed butterfly, the waves in wave order
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int m = L; m < 64; m <<= 1) acc[v][c] += __shfl_xor(acc[v][c], m, 64);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    z += __shfl_xor(z, m, 64);
    n += __shfl_xor(n, m, 64);
  }
  if (lane == 0) {
    zs[wave] = z;
    ns[wave] = n;
  }
  if (lane < L) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = expert_of<L, NV, VEC>(v, c, l);
        if (e < E) ps[wave * E + e] = acc[v][c];
      }
  }
  __syncthreads();
  const bool one = gridDim.x == 1;
  float p = 0.0f;
  if (tid < E) {  // E <= kSumThreads
#pragma unroll
    for (int q = 0; q < kSumWaves; ++q) p += ps[q * E + tid];
    if (one) {
      counts[tid] = hist[tid];
    } else {
      w.psum[(int64_t)blockIdx.x * E + tid] = p;
      w.counts[(int64_t)blockIdx.x * E + tid] = hist[tid];
    }
  }
  double b = 0.0;
  if (one) {  // sum_e c_e P_e: a butterfly in each wave, then the waves in order
    __shared__ double bs[kSumWaves];
    b = tid < E ? (double)hist[tid] * (double)p : 0.0;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) b += __shfl_xor(b, m, 64);
    if (lane == 0) bs[wave] = b;
    __syncthreads();
    b = 0.0;
    for (int q = 0; q < kSumWaves; ++q) b += bs[q];
  }
  if (tid == 0) {
    float zt = 0.0f;
    int32_t nt = 0;
    for (int q = 0; q < kSumWaves; ++q) {
      zt += zs[q];
      nt += ns[q];
    }
    if (one) {
      write_losses(E, k, nt, b, (double)zt, counts, loss);
    } else {
      w.z[blockIdx.x] = zt;
      w.n[blockIdx.x] = nt;
    }
  }
}

// Workgroup b adds the G partial sums of experts kFinE b .. in FP64 and forms their share
// sum_e c_e P_e; the workgroup that arrives last adds the shares in order.  (The counter is
// cleared by the first kernel of the same call, so a workspace needs no preparation.)
constexpr int kFinThreads = 1024, kFinParts = kFinThreads / kFinE;

__global__ void __launch_bounds__(kFinThreads) router_finish(LossWs w, int G, int E, int k, int32_t *__restrict__ counts,
                                                          float *__restrict__ loss) {
  __shared__ double ps[kFinParts][kFinE];
  __shared__ int32_t cs[kFinParts][kFinE];
  __shared__ uint32_t rank;
  const int tid = threadIdx.x, el = tid % kFinE, part = tid / kFinE;
  const int e = blockIdx.x * kFinE + el;
  double p = 0.0;
  int32_t c = 0;
  if (e < E)
#pragma unroll 4
    for (int g = part; g < G; g += kFinParts) {
      p += (double)w.psum[(int64_t)g * E + e];
      c += w.counts[(int64_t)g * E + e];
    }
  ps[part][el] = p;
  cs[part][el] = c;
  __syncthreads();
  if (tid < kFinE) {
    p = 0.0;
    c = 0;
    for (int q = 0; q < kFinParts; ++q) {
      p += ps[q][el];
      c += cs[q][el];
    }
    if (e < E) counts[e] = c;
    ps[0][el] = (double)c * p;
  }
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int q = 0; q < kFinE; ++q) s += ps[0][q];
    __hip_atomic_store(&w.part[blockIdx.x], s, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    rank = __hip_atomic_fetch_add(w.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (rank != gridDim.x - 1) return;
  // the last workgroup: tokens and lse^2 over the G partial sums, then the losses
  double z = 0.0;
  int32_t n = 0;
  for (int g = tid; g < G; g += kFinThreads) {
    z += (double)w.z[g];
    n += w.n[g];
  }
  double *zs = &ps[0][0];
  int32_t *ns = &cs[0][0];
  zs[tid] = z;
  ns[tid] = n;
  __syncthreads();
  for (int s = kFinThreads / 2; s > 0; s >>= 1) {
    if (tid < s) {
      zs[tid] += zs[tid + s];
      ns[tid] += ns[tid + s];
    }
    __syncthreads();
  }
  if (tid == 0) {
    double b = 0.0;
    for (unsigned q = 0; q < gridDim.x; ++q)
      b += __hip_atomic_load(&w.part[q], __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_AGENT);
    write_losses(E, k, ns[0], b, zs[0], counts, loss);
  }
}

// ---------------------------------------------------------------------------
// gradient of the logits
// ---------------------------------------------------------------------------
// The routing weights' part of a token, per pair j: dq_j = dw_j, or (dw_j - D) / S with
// renormalised weights (S = sum q, D = sum q dw / S), and off = sum_j q_j dq_j over all pairs
// (which is 0 with renormalised weights).
//
// More than 128 experts (a wave per token): lane j holds pair j.  Its q comes from its own
// load of the logit (in cache by then), the sums over pairs are moves within 16 lanes, and
// dq reaches the lanes that hold the experts through a zeroed row of LDS; pairs of the same
// expert are first added in the order of j, so that each of them writes the same total.
// Comparing each pair with each expert instead took 12 k NV vector instructions a lane
// (131072 x 256, k = 8: 91 us so, 65 us through LDS, 4.2 TB/s).  Fewer experts (several tokens per
// wave) have few lanes per token and compare.
template <int NV>
struct Selected {
  f32x4 a[NV];  // sum of dq over a lane's experts' pairs
  float off;
};

template <int L, int NV, bool VEC>
__global__ void __launch_bounds__(kThreads) router_grad(const float *__restrict__ logits,
                                                        const int32_t *__restrict__ idx,
                                                        const uint8_t *__restrict__ valid,
                                                        const int32_t *__restrict__ counts,
                                                        const float *__restrict__ dw, const float *__restrict__ dloss,
                                                        int64_t T, int E, int k, int renorm,
                                                        float *__restrict__ dlogits) {
  constexpr int kGroups = kThreads / L, kRow = L * 4 * NV;
  constexpr bool kScatter = L == 64;
  __shared__ __attribute__((aligned(16))) float rows[kScatter ? kGroups : 1][kScatter ? kRow : 1];
  const int tid = threadIdx.x, l = tid & (L - 1);
  const int grp = L == 64 ? __builtin_amdgcn_readfirstlane(tid >> 6) : tid / L;
  float *row = rows[kScatter ? grp : 0];
  if constexpr (kScatter) {
#pragma unroll
    for (int v = 0; v < 4 * NV; ++v) row[v * 64 + l] = 0.0f;  // this wave's own row: no barrier
    wave_fence();
  }
  // the losses' gradients per expert: g_b E f_e / n, and 2 g_z / n
  const int32_t n = counts[E];
  const float rn = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gz = dloss ? 2.0f * dloss[1] * rn : 0.0f;
  const float gb = dloss ? dloss[0] * rn * rn * (float)E / (float)k : 0.0f;
  f32x4 fe[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int e = expert_of<L, NV, VEC>(v, c, l);
      fe[v][c] = e < E ? gb * (float)counts[e] : 0.0f;
    }
  for (int64_t t = (int64_t)blockIdx.x * kGroups + grp; t < T; t += (int64_t)gridDim.x * kGroups) {
    const bool use = !valid || valid[t];
    const float *lrow = logits + t * E;
    f32x4 x[NV];
    load_row<L, NV, VEC>(lrow, E, l, use, x);
    // pair l of the token (kScatter)
    int pi = -1;
    float pd = 0.0f, pl = -INFINITY;
    if constexpr (kScatter) {
      if (dw && use && l < k) {
        pi = idx[t * k + l];
        pd = dw[t * k + l];
        if ((unsigned)pi < (unsigned)E)
          pl = lrow[pi];
        else
          pi = -1;
      }
    }
    float m, lse;
    const float inv = softmax_row<L, NV>(x, lse, m);
    Selected<NV> sel = {};
    if constexpr (kScatter) {
      if (dw) {
        const float q = pi >= 0 ? exp_neg(pl - m) * inv : 0.0f;
        pd = pi >= 0 ? pd : 0.0f;
        float qd = q * pd, qs = q;
        // over the first 16 lanes (the others hold none)
        qd = group_sum<16>(qd);
        qd = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(qd)));
        if (renorm) {
          qs = group_sum<16>(qs);
          qs = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(qs)));
          const float rs = qs > 0.0f ? 1.0f / qs : 0.0f;
          pd = (pd - qd * rs) * rs;
        } else {
          sel.off = qd;
        }
        float sum = 0.0f;
        for (int j = 0; j < k; ++j) {
          const int ij = __builtin_amdgcn_readlane(pi, j);
          const float dj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(pd), j));
          sum += ij == pi ? dj : 0.0f;
        }
        // one wave's LDS operations complete in order: write, read by all lanes, clear
        if (pi >= 0) row[VEC ? pi : slot_of<L, NV>(pi)] = sum;
        wave_fence();
#pragma unroll
        for (int v = 0; v < NV; ++v) sel.a[v] = *reinterpret_cast<const f32x4 *>(row + 4 * (v * L + l));
        wave_fence();
        if (pi >= 0) row[VEC ? pi : slot_of<L, NV>(pi)] = 0.0f;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) x[v] *= inv;
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) x[v] *= inv;
      if (dw && use) {
        f32x4 mult[NV] = {};
        for (int j = 0; j < k; ++j) {
          const int i = idx[t * k + j];
          const float d = dw[t * k + j];
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const bool hit = i == expert_of<L, NV, VEC>(v, c, l);
              sel.a[v][c] += hit ? d : 0.0f;
              mult[v][c] += hit ? 1.0f : 0.0f;
            }
        }
        float sa = 0.0f, sm = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // a dropped pair's index may name a slot past E (p 0 there); its dw can be anything
            sa += expert_of<L, NV, VEC>(v, c, l) < E ? x[v][c] * sel.a[v][c] : 0.0f;
            sm += x[v][c] * mult[v][c];
          }
        sa = group_sum<L>(sa);
        if (renorm) {
          sm = group_sum<L>(sm);
          const float rs = sm > 0.0f ? 1.0f / sm : 0.0f, d = sa * rs;
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int c = 0; c < 4; ++c) sel.a[v][c] = (sel.a[v][c] - d * mult[v][c]) * rs;
        } else {
          sel.off = sa;
        }
      }
    }
    float sf = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int c = 0; c < 4; ++c) sf += x[v][c] * fe[v][c];
    sf = group_sum<L>(sf);
    const float shift = gz * lse - sf - sel.off;
    float *out = dlogits + t * E;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      f32x4 g;
#pragma unroll
      for (int c = 0; c < 4; ++c) g[c] = x[v][c] * (fe[v][c] + sel.a[v][c] + shift);
      if constexpr (VEC) {
        const int e = expert_of<L, NV, VEC>(v, 0, l);
        if (e < E) __builtin_nontemporal_store(g, reinterpret_cast<f32x4 *>(out + e));
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int e = expert_of<L, NV, VEC>(v, c, l);
          if (e < E) out[e] = g[c];
        }
      }
    }
  }
}

bqm_status check_router(const char *who, int64_t T, int32_t E, int32_t k) {
  BQM_REQUIRE(T >= 0, BQM_ERR_INVALID_ARG, "%s: T < 0", who);
  BQM_REQUIRE(E >= 1 && E <= kMaxE, BQM_ERR_SHAPE, "%s: E=%d outside [1, 1024]", who, E);
  BQM_REQUIRE(k >= 1 && k <= E && k <= kMaxK, BQM_ERR_SHAPE, "%s: k=%d outside [1, min(E,16)]", who, k);
  // per-expert counts are 32-bit
  BQM_REQUIRE(T < ((int64_t)1 << 31) && T * k < ((int64_t)1 << 31), BQM_ERR_SHAPE, "%s: T*k too large", who);
  return BQM_OK;
}

// Calls f with the lanes per token, the 4-logit vectors per lane and the load form for E.
// Four logits a lane up to 256 experts: the lanes per token halve with E, so a wave takes
// several tokens of a small router.
template <class F>
void with_shape(int E, F f) {
  auto vec = [&](auto L, auto NV) {
    if (E % 4 == 0)
      f(L, NV, std::true_type{});
    else
      f(L, NV, std::false_type{});
  };
  using std::integral_constant;
  switch (lanes_of(E)) {
    case 4: return vec(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    case 8: return vec(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    case 16: return vec(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    case 32: return vec(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  }
  if (E <= 256)
    vec(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (E <= 512)
    vec(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else
    vec(integral_constant<int, 64>{}, integral_constant<int, 4>{});
}

}  // namespace
}  // namespace bqm

using namespace bqm;

extern "C" size_t bqm_router_loss_workspace_size(int64_t T, int32_t E) {
  if (T < 0 || E < 1 || E > kMaxE) return 0;
  return loss_geom(T, E).bytes;
}

extern "C" bqm_status bqm_router_loss(const float *logits, const int32_t *topk_idx, const uint8_t *valid, int64_t T,
                                      int32_t E, int32_t k, int32_t *counts, float *loss, void *ws, size_t ws_bytes,
                                      void *stream) {
  const char *who = "bqm_router_loss";
  bqm_status st = check_router(who, T, E, k);
  if (st != BQM_OK) return st;
  BQM_REQUIRE(counts && loss, BQM_ERR_INVALID_ARG, "%s: counts or loss is NULL", who);
  BQM_REQUIRE(T == 0 || (logits && topk_idx), BQM_ERR_INVALID_ARG, "%s: NULL pointer", who);
  BQM_REQUIRE(aligned16(logits) && aligned16(topk_idx) && aligned16(valid) && aligned16(counts) && aligned16(loss),
              BQM_ERR_ALIGN, "%s: pointer not 16-byte aligned", who);
  const LossGeom g = loss_geom(T, E);
  BQM_REQUIRE(ws && ws_bytes >= g.bytes, BQM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", who,
              g.bytes, ws_bytes);
  BQM_REQUIRE(aligned16(ws), BQM_ERR_ALIGN, "%s: ws not 16-byte aligned", who);
  const LossWs w = loss_ws(ws, g.G, E);
  hipStream_t s = as_stream(stream);
  with_shape(E, [&](auto L, auto NV, auto VEC) {
    router_sums<L.value, NV.value, VEC.value><<<g.G, kSumThreads, kSumWaves * E * sizeof(float), s>>>(
        logits, topk_idx, valid, T, E, k, w, counts, loss);
  });
  st = launch_status("router_sums");
  if (st != BQM_OK || g.G == 1) return st;
  router_finish<<<(unsigned)cdiv(E, kFinE), kFinThreads, 0, s>>>(w, g.G, E, k, counts, loss);
  return launch_status("router_finish");
}

extern "C" bqm_status bqm_router_grad(const float *logits, const int32_t *topk_idx, const uint8_t *valid,
                                      const int32_t *counts, const float *dtopk_w, const float *dloss, int64_t T,
                                      int32_t E, int32_t k, int32_t renorm, float *dlogits, void *stream) {
  const char *who = "bqm_router_grad";
  bqm_status st = check_router(who, T, E, k);
  if (st != BQM_OK) return st;
  if (T == 0) return BQM_OK;
  BQM_REQUIRE(logits && topk_idx && counts && dlogits, BQM_ERR_INVALID_ARG, "%s: NULL pointer", who);
  BQM_REQUIRE(aligned16(logits) && aligned16(topk_idx) && aligned16(valid) && aligned16(counts) &&
                  aligned16(dtopk_w) && aligned16(dloss) && aligned16(dlogits),
              BQM_ERR_ALIGN, "%s: pointer not 16-byte aligned", who);
  with_shape(E, [&](auto L, auto NV, auto VEC) {
    constexpr int kGroups = kThreads / L.value;
    const int64_t G = cdiv(T, kGroups);
    const unsigned grid = (unsigned)(G < 2048 ? G : 2048);
    router_grad<L.value, NV.value, VEC.value><<<grid, kThreads, 0, as_stream(stream)>>>(
        logits, topk_idx, valid, counts, dtopk_w, dloss, T, E, k, renorm, dlogits);
  });
  return launch_status("router_grad");
}
