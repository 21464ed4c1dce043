"""How the dense product is laid over the CUs, and its workspace, by sizes alone (host only)."""
import ctypes as C
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

bqm = pytest.importorskip("bit_quantized_moe_amd._lib")

# what the library's entry points ask of their workspace, from the header that they use
SHIM = """
#include "linear_plan.h"
using namespace bqm;
extern "C" {
// floats that a call takes
int64_t need(int64_t M, int64_t N, int64_t K, int dir) {
  if (dir == 0) return few_rows(M, N, K) ? 0 : plan_fwd(M, N, K).part;
  return dir == 1 ? plan_dgrad(M, N, K).part : plan_wgrad(M, N, K).part + col_floats(M, N);
}
// tile's rows and columns, whole tiles, those left over, their parts, steps per part, steps
void plan_at(int64_t M, int64_t N, int64_t K, int dir, int64_t *o) {
  const Plan p = dir == 0 ? plan_fwd(M, N, K) : dir == 1 ? plan_dgrad(M, N, K) : plan_wgrad(M, N, K);
  const int64_t v[7] = {kShapes[p.shape].bm, kShapes[p.shape].bn, p.full, p.rem, p.S, p.per, p.nk};
  for (int i = 0; i < 7; ++i) o[i] = v[i];
}
int64_t enough(int64_t M, int64_t N, int64_t K) { return workspace_floats(M, N, K); }
// the first row count up to M that needs more than has been promised, or 0; every one of them
// in steps, and those on either side of a row of tiles
int64_t short_of(int64_t M, int64_t N, int64_t K, int64_t step) {
  int64_t most = 0, last = 0;
  for (int64_t m = 1; m <= M; m += step) {
    for (int64_t q = m; q <= m + 1; ++q)
      for (int d = 0; d < 3; ++d) {
        const int64_t n = need(q, N, K, d);
        if (n > most) most = n;
      }
    const int64_t e = enough(m + 1, N, K);
    if (e < most || e < last) return m;
    last = e;
  }
  return 0;
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cc").write_text(SHIM)
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I" + os.path.join(ROOT, "bit_quantized_moe_amd", "csrc"),
                    str(d / "shim.cc"), "-o", str(d / "shim.so")], check=True)
    lib = C.CDLL(str(d / "shim.so"))
    for f, n in (("need", 3), ("enough", 3), ("short_of", 4)):
        getattr(lib, f).restype = C.c_int64
        getattr(lib, f).argtypes = [C.c_int64] * n + ([C.c_int] if f == "need" else [])
    lib.plan_at.restype, lib.plan_at.argtypes = None, [C.c_int64] * 3 + [C.c_int, C.POINTER(C.c_int64)]
    lib.at = lambda *a: (lambda o: (lib.plan_at(*a, o), tuple(o))[1])((C.c_int64 * 7)())
    return lib


SIZES = [(4096, 6144), (8192, 8192), (6144, 2048), (2048, 768), (768, 2048), (2848, 2080), (3032, 6192), (256, 1024), (64, 64),
         (8, 8), (8, 40008), (70000, 64), (264, 264), (1024, 8192)]


@pytest.mark.parametrize("N,K", SIZES)
def test_workspace_is_enough_for_fewer_rows(N, K):
    """A workspace made for the largest batch serves the smaller ones."""
    size = bqm.load().bqm_linear_workspace_size
    last = 0
    # the most rows that the calls take: under 2^30, and under 2^31 tiles of 64 x 64
    top = min((1 << 30) - 1, 64 * (((1 << 31) - 1) // -(-max(N, K) // 64)))
    for M in [*range(1, 200, 9), *range(200, 6000, 100), 16384, 20000, 100000, 1 << 20, top]:
        n = size(M, N, K)
        assert n >= last, f"{M} rows: {n} bytes, fewer: {last}"
        assert n % 256 == 0 and n <= 65 << 20
        last = n


@pytest.mark.parametrize("N,K", SIZES)
def test_every_call_fits_the_workspace_of_more_rows(plan, N, K):
    assert plan.short_of(2100, N, K, 1) == 0
    assert plan.short_of(40000, N, K, 64) == 0
    assert plan.short_of(1 << 23, N, K, 65408) == 0
    size = bqm.load().bqm_linear_workspace_size
    for M in (1, 8, 9, 100, 1000, 16384):
        n = size(M, N, K)
        assert 0 <= n - 4 * plan.enough(M, N, K) < 256
        assert max(plan.need(M, N, K, d) for d in range(3)) * 4 <= n


def test_every_call_fits_drawn_sizes(plan):
    rng = random.Random(11)
    for _ in range(400):
        N, K = (max(8, int(2 ** rng.uniform(3, 15)) // 8 * 8) for _ in range(2))
        assert plan.short_of(int(2 ** rng.uniform(6, 14)), N, K, rng.choice((1, 63, 64, 127))) == 0, (N, K)


@pytest.mark.parametrize("M,N,K", [(512, 4096, 6144), (300, 4096, 6144), (16384, 4096, 6144), (8192, 264, 264)])
def test_a_byte_too_few_is_refused(plan, M, N, K):
    """The check is of this call's need, not of the size for all row counts."""
    lib = bqm.load()
    calls = (lambda n: lib.bqm_linear_fwd(16, 16, None, 0, None, M, N, K, 16, None, 16, n, None),
             lambda n: lib.bqm_linear_dgrad(16, 16, None, 0, None, M, N, K, 16, 16, n, None),
             lambda n: lib.bqm_linear_wgrad(16, 16, 0, M, N, K, 16, 16, 16, n, None))
    need = [4 * plan.need(M, N, K, d) for d in range(3)]
    assert any(need)
    for f, n in zip(calls, need):
        if n:       # (a call that needs none would be launched)
            assert f(n - 1) == -5 and f" {n} needed" in bqm.bqm_last_error()


def drawn(seed, n):
    rng = random.Random(seed)
    for _ in range(n):
        yield int(2 ** rng.uniform(0, 14)), *(max(8, int(2 ** rng.uniform(6, 13)) // 8 * 8) for _ in range(2)), rng.randrange(3)


def test_every_step_is_some_part_s(plan):
    for M, N, K, d in drawn(3, 20000):
        bm, bn, full, rem, S, per, nk = plan.at(M, N, K, d)
        I, J, C_ = ((M, N, K), (M, K, N), (N, K, M))[d]
        assert full + rem == -(-I // bm) * -(-J // bn) and nk == -(-C_ // 64), (M, N, K, d)
        assert 1 <= S and per * S >= nk > per * (S - 1) and (S == 1 or rem and per >= 2), (M, N, K, d)


def test_idle_cus_get_one_part_each(plan):
    """Where a round's tiles leave CUs idle, their parts are no more than the CUs."""
    assert plan.at(72, 3064, 472, 1)[4] <= 16
    split = 0
    for M, N, K, d in drawn(5, 20000):
        _, _, full, rem, S, _, _ = plan.at(M, N, K, d)
        if S > 1 and full + rem <= 256:
            split += 1
            assert rem * S <= 256, (M, N, K, d)
    assert split > 1000


def test_tested_sizes_reach_every_plan(plan):
    """Of the sizes that the GPU tests run, some take each tile in each direction: as one round of
    tiles and as more, whole and with a part split along the contraction, and where the plan does so
    with both kinds of last step."""
    from tests.test_gpu_linear import LARGE, ROUNDS, SHAPES

    def kinds(sizes):
        for M, N, K in sizes:
            for d in range(3):
                bm, bn, full, rem, S, _, nk = plan.at(M, N, K, d)
                C_ = (K, N, M)[d]
                if d == 0 and M <= 8 and (K <= 4096 or 2 * N >= K):
                    continue        # not by tiles
                walks = full > 0 and full + rem * S > (512 if bm == 64 else 256)
                yield ("fwd", "dgrad", "wgrad")[d], (bm, bn) if C_ >= 64 else "short", walks, S > 1, C_ >= 64 and C_ % 64 > 0
    got = set(kinds(SHAPES + LARGE + ROUNDS))
    # what ordinary sizes take
    usual = {}
    for M, N, K, _ in drawn(9, 30000):
        for k in kinds([(M, N, K)]):
            usual[k] = usual.get(k, 0) + 1
    missing = {k: n for k, n in usual.items() if n >= 10 and k not in got and k[2]}
    assert not missing, missing
    missing = {k[:4] for k in usual if usual[k] >= 10} - {k[:4] for k in got}
    assert not missing, missing
