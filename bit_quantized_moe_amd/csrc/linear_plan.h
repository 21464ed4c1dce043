// How the dense product is laid over the CUs: the tile, the split of its contraction and the
// workspace that this takes, by sizes alone.  Host code without HIP, so that a CPU test can evaluate
// it.
#pragma once

#include <stdint.h>

#include "sizes.h"

namespace bqm {

constexpr int kCUs = 256;
constexpr int KS = 64;  // contraction per step: 128 bytes of a row

// Rows of x up to which the weights are streamed (measured beside the kernel, lin_few).
constexpr int kFewRows = 8;
inline bool few_rows(int64_t M, int64_t N, int64_t K) { return M <= kFewRows && (K <= 4096 || 2 * N >= K); }

// The tile and its split by what they are expected to take: per round of tiles, the steps of 64
// and the rest (launch, first copies, epilogue), both measured with every CU busy, and for a split
// the parts written and read and the join's launch.  It ranks tiles rather than foretells times: the
// rest is charged to every round, launch and all, and with idle CUs a step is shorter (37 x 6144 x
// 2048 is expected at 11.8 us and takes 8.9).  Both sides, in us (tiles of 256 x 256, 256 x 128, 128 x
// 128, 64 x 64, each in the split that is best for it):
//   forward 37 x 6144 x 2048          15.0  13.0  12.3   8.9
//           300 x 2048 x 2048         26.4  20.0  15.9   9.0
//           1111 x 2848 x 2080        36.6  28.9  21.0  34.2
//           2048 x 4096 x 2048        43.6  33.5  38.7  49.1
//           4096 x 4096 x 4096         103   119   151   241
//           16384 x 4096 x 6144        567   682   885  1441
//   input gradient 203 x 2048 x 768   20.5  14.8  12.6   8.8
//   weight gradient 203 x 2048 x 768  16.4  10.5   8.1   5.9
//           16384 x 4096 x 6144        607   668   925  2537   (256 x 256 unsplit: 678)
// Rows that start off 64 bytes cost a large tile's copies least: forward 799 x 3032 x 6192, 256 x
// 256 tiles in five parts 56 us, 256 x 128 in two 69, 128 x 128 68; 600 x 4096 x 4096 41 (four
// parts), 36 (two), 35.6.  Splits pay where a round of tiles is not whole or has many steps: 64 x 1024 x 8192 takes 23.6
// us in one part, 11.9 in 16.  Tiles that leave CUs idle are split into one part per CU at most, as
// two workgroups on a CU share its copies and there are more parts to join: input gradient 72 x 3064 x
// 472 in 16 parts 8.7 us, in 24 10.7; 60 drawn sizes take 0.75 to 1.02 times as long as with two, 0.86
// in the mean.  step2 is more than two unsplit workgroups take (.31 to .40, and .51 to .55 with rows off
// 64 bytes), so it has no factor: with one, 19 drawn sizes get 128 x 128 tiles and take 0.94 to 1.26
// times as long (input gradient 345 x 776 x 3064 11.3 us, 64 x 64 tiles 9.4).
struct Shape {
  int bm, bn, occ;     // its size, workgroups per CU
  float step, rest;    // us
  float step2, rest2;  // with two workgroups per CU
  float odd;           // factor of step where an operand's rows start off 64 bytes
};
constexpr Shape kShapes[4] = {{256, 256, 1, 1.0f, 12.4f, 0, 0, 1.15f}, {256, 128, 1, .62f, 8.6f, 0, 0, 1.35f},
                              {128, 128, 1, .42f, 7.0f, 0, 0, 1.3f}, {64, 64, 2, .19f, 5.7f, .60f, 4.5f, 1.3f}};
constexpr float kJoin = 4.6f, kJoinRate = 7.5e6f;  // us of a join's launch; its bytes per us
constexpr int kMostParts = 32;
constexpr int kSlow = 2;  // the shape for contractions of less than a step

inline float step_of(const Shape &s, bool two, bool odd) { return two ? s.step2 : odd ? s.step * s.odd : s.step; }

struct Plan {
  int shape, NI, NJ, full, rem, S, per, nk;
  int64_t part;  // floats of the workspace
};

// odd: an operand's rows are no multiple of 64 bytes
inline Plan plan_of(int64_t I, int64_t J, int64_t C, bool odd) {
  Plan best = {};
  float least = 0.0f;
  for (int h = 0; h < 4; ++h) {
    const Shape &s = kShapes[h];
    if (C < 64 && h != kSlow) continue;
    const int64_t tiles = cdiv(I, s.bm) * cdiv(J, s.bn);
    const int nk = (int)cdiv(C, KS);
    const bool two = s.occ == 2 && tiles > kCUs;
    const int64_t slots = two ? 2 * kCUs : kCUs, full = tiles / slots * slots, rem = tiles - full;
    for (int S = 1; S <= kMostParts; ++S) {
      const int per = (int)cdiv(nk, S);
      if (S > 1 && (rem == 0 || rem * S > slots || per < 2)) break;
      if (S > 1 && (int64_t)per * (S - 1) >= nk) continue;  // a part without steps
      const float step = step_of(s, two, odd), rest = two ? s.rest2 : s.rest;
      float t = full / slots * (nk * step + rest);
      if (rem) t += per * step + rest;
      if (S > 1) t += kJoin + 8.0f * rem * S * s.bm * s.bn / kJoinRate;  // written and read
      if (least == 0.0f || t < least) {
        least = t;
        best = {h, (int)cdiv(I, s.bm), (int)cdiv(J, s.bn), (int)full, (int)rem, S, per, nk, S > 1 ? rem * S * s.bm * s.bn : 0};
      }
    }
  }
  return best;
}

inline bool odd_fwd(int64_t K) { return K % 32 != 0; }
inline bool odd_grad(int64_t N, int64_t K) { return N % 32 || K % 32; }
inline Plan plan_fwd(int64_t M, int64_t N, int64_t K) { return plan_of(M, N, K, odd_fwd(K)); }
inline Plan plan_dgrad(int64_t M, int64_t N, int64_t K) { return plan_of(M, K, N, odd_grad(N, K)); }
inline Plan plan_wgrad(int64_t M, int64_t N, int64_t K) { return plan_of(N, K, M, odd_grad(N, K)); }

// Row parts of the column sums: of at least 1024 rows, which take no longer than the tiles beside
// them (in a launch of their own: 203 x 2048 x 768 9.6 against 6.9 us for the weight's and the
// bias's gradients, 1111 x 2848 x 2080 31 against 27), and at most 2048 workgroups
inline int col_parts(int64_t M, int64_t N) {
  const int64_t most = 2048 / cdiv(N, 64), want = cdiv(M, 1024), n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n);
}

inline int64_t col_floats(int64_t M, int64_t N) {
  const int parts = col_parts(M, N);
  return parts > 1 ? parts * N : 0;
}

// Floats of a workspace that is enough for I, J and C and for all smaller I or C: what plan_of
// takes rises and falls with them (as whole rounds come and go), this only rises.  A split is chosen
// only where it is ahead of each shape unsplit; whole is the least of those, in a form that does not
// fall as I or C grows, and a split's own steps (two at least), rest and join leave what its parts
// may take to write and read.  Apart from that there are no more parts than workgroups of a round.
inline int64_t most_floats(int64_t I, int64_t J, int64_t C, bool odd) {
  const int64_t nk = cdiv(C, KS), most_s = (nk + 1) / 2 < kMostParts ? (nk + 1) / 2 : kMostParts;
  if (nk < 3) return 0;
  float whole = 0.0f;
  for (const Shape &s : kShapes) {
    const int64_t tiles = cdiv(I, s.bm) * cdiv(J, s.bn);
    const bool two = s.occ == 2 && tiles > kCUs;
    const float t = cdiv(tiles, two ? 2 * kCUs : kCUs) * (nk * step_of(s, two, odd) + s.rest);
    if (whole == 0.0f || t < whole) whole = t;
  }
  int64_t most = 0;
  for (const Shape &s : kShapes) {
    const float rest = s.occ == 2 && s.rest2 < s.rest ? s.rest2 : s.rest;
    const float left = 1.001f * whole - (2 * s.step + rest + kJoin);  // (1.001: sums in another order)
    if (left <= 0.0f) continue;
    const int64_t parts = cdiv(I, s.bm) * cdiv(J, s.bn) * most_s, slots = kCUs * s.occ, by_time = (int64_t)(left * kJoinRate / 8);
    const int64_t n = (parts < slots ? parts : slots) * s.bm * s.bn;
    const int64_t need = n < by_time ? n : by_time;
    if (need > most) most = need;
  }
  return most;
}

// of every direction, for up to M rows
inline int64_t workspace_floats(int64_t M, int64_t N, int64_t K) {
  const int64_t f = most_floats(M, N, K, odd_fwd(K)), d = most_floats(M, K, N, odd_grad(N, K));
  const int64_t w = most_floats(N, K, M, odd_grad(N, K)) + col_floats(M, N);
  const int64_t a = f > d ? f : d;
  return a > w ? a : w;
}

}  // namespace bqm
