"""How the products are cut (csrc/linear_plan.h, compiled for the host): what the sizes of the GPU tests reach,
and that every call has a cut within the kernels' limits."""
import random
import subprocess

import pytest

from mixture_experts_layer_05_gb300 import build as build_mod
from tests.linear_cuts import CLUSTERS, GATED_FP8, ROOM, ROUNDS
from tests.test_gpu_linear import CUTS

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "linear_plan.h"
using namespace gbmoe;
// The clusters that the device holds, for 1 to 8 CTAs. Then per line T G K N gated fp8 and G sizes (G = 0: dense):
// many rows?, CTAs of a cluster, rows per block, weight rows per tile, rounds of units, units at most
int main() {
  int room[9];
  for (int c = 1; c <= 8; ++c)
    if (scanf("%d", &room[c]) != 1) return 1;
  int T, G, K, N, gated, fp8;
  while (scanf("%d %d %d %d %d %d", &T, &G, &K, &N, &gated, &fp8) == 6) {
    const LinSize a = {T, G ? G : 1, K, N, G > 0, gated != 0, fp8 != 0};
    std::vector<int> sizes(G);
    for (int& s : sizes)
      if (scanf("%d", &s) != 1) return 1;
    const LinPlan p = lin_plan(a, room[1], [&](int, int C) { return room[C]; });
    if (!p.ok) return 2;
    if (p.many) {
      printf("1 0 %d 0 0 %lld\n", p.bn, p.units);
      continue;
    }
    int blocks = G ? 0 : (T + p.bn - 1) / p.bn, n_tiles = p.n_tiles, pick = 0;
    for (int s : sizes) blocks += (s + p.bn - 1) / p.bn;
    const int step = p.units < room[p.cluster] ? (int)p.units : room[p.cluster];
    if (G)
      pick = lin_pick(p.rows, p.choices, a.fp8, a.gated, a.cols(), (K * (fp8 ? 1 : 2) + 127) / 128, p.cluster,
                      (T + G - 1) / G <= 8 ? 8 : p.bn, blocks, step, &n_tiles);
    printf("0 %d %d %d %lld %lld\n", p.cluster, p.bn, p.rows[pick], ((long long)blocks * n_tiles + step - 1) / step,
           p.units);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build_mod.CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")],
                   check=True)

    def ask(calls, room=ROOM):
        """calls: (rows or sizes, K, N, gated, fp8); (many, CTAs, rows per block, weight rows, rounds, units)."""
        lines = [" ".join(str(room[c]) for c in range(1, 9))]
        for rows, K, N, gated, fp8 in calls:
            sizes = [] if isinstance(rows, int) else list(rows)
            lines.append(" ".join(map(str, [rows if isinstance(rows, int) else sum(sizes), len(sizes), K, N,
                                            int(gated), int(fp8)] + sizes)))
        out = subprocess.run([str(d / "plan")], input="\n".join(lines) + "\n", text=True, capture_output=True,
                             check=True).stdout
        return [tuple(map(int, l.split())) for l in out.splitlines()]
    return ask


def test_cluster_cases_reach_their_cuts(plan):
    cases = CLUSTERS + ROUNDS
    got = plan([(rows, K, N, act == "silu_mul", fp8) for rows, K, N, act, fp8, _, _ in cases])
    for case, (many, ctas, bn, _, rounds, _) in zip(cases, got):
        assert (many, ctas, rounds) == (0, *case[5:]), (case, ctas, rounds)
    assert all(a[0] for a in plan([(rows, K, N, True, True) for rows, K, N in GATED_FP8]))
    # the e4m3 kernel's halves of a run of columns are among them
    assert any(bn == 16 and c[4] and c[6] > 1 for c, (_, _, bn, _, _, _) in zip(cases, got))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_dense_cases_reach_every_cluster(plan, gated, fp8):
    calls = [(T, K, N, gated, fp8) for T, K, N in CUTS if not (fp8 and K % 128 or gated and N % 256)]
    got = [a for a in plan(calls) if not a[0]]
    assert {a[4] for a in got} == {1, 2}
    assert {1, 2, 3, 4, 6, 8} <= {a[1] for a in got}
    mine = [c for c in CLUSTERS + ROUNDS if (c[3] == "silu_mul", c[4]) == (gated, fp8)]
    assert {a[1] for a in got} | {c[5] for c in mine} == set(range(1, 9))


def test_every_call_has_a_cut(plan):
    """Over the documented sizes, and on devices that hold fewer clusters."""
    rng = random.Random(3)

    def draw(lo, hi):
        return min(hi, int(lo * (hi / lo) ** rng.random()))

    for room in (ROOM, {c: 148 // c for c in range(1, 9)}, {c: max(1, 16 // c) for c in range(1, 9)}):
        calls = []
        for _ in range(3000):
            gated, fp8 = rng.random() < 0.5, rng.random() < 0.5
            T, K = draw(1, 1 << 22), 128 * draw(1, 1 << 17) if fp8 else 8 * draw(1, 1 << 21)
            step = 256 if gated and fp8 else 32 if gated else 1
            N = step * draw(1, (1 << 24) // step)
            if rng.random() < 0.5:
                if (T // 16 + 1) * ((N + 127) // 128) <= 1 << 30:
                    calls.append((T, K, N, gated, fp8))
                continue
            G = draw(1, 1024)
            sizes = [0] * G
            left = T
            while left > 0 and rng.random() < 0.99:
                n = min(left, draw(1, 1 << 16))
                sizes[rng.randrange(G)] += n
                left -= n
            T = sum(sizes)
            if T and (T // 16 + G) * ((N + 127) // 128) <= 1 << 30 and G * N < (1 << 31) - 1024:
                calls.append((sizes, K, N, gated, fp8))
        assert len(calls) > 1000
        for call, (many, ctas, bn, rows, rounds, units) in zip(calls, plan(calls, room)):
            fp8, gated = call[4], call[3]
            assert 0 < units < 1 << 62
            if many:
                assert bn == 128 if fp8 else bn % 32 == 0 and 32 <= bn <= 256, call
            else:
                assert 1 <= ctas <= 8 and bn % 16 == 0 and 16 <= bn <= (64 if fp8 else 128), call
                assert 8 <= rows <= 128 and rows % (32 if gated else 8) == 0, call
                assert not (gated and fp8) or 128 % (rows // 2) == 0, call
