"""The feed-forward block's host-side arithmetic (csrc/mok_ffn_plan.h), driven from a small C++ program.  No GPU."""
import os
import shutil
import subprocess

import pytest

from helpers import ROOT

CSRC = os.path.join(ROOT, "mixture_experts_layer_build_gb300", "csrc")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


def run(tmp_path, body, *args, stdin=""):
    """Compiles `body` as main() over the header and returns the lines that it prints."""
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include <initializer_list>\n#include "mok_ffn_plan.h"\nusing namespace mok;\n'
                   "int main(int argc, char** argv) {\n" + body + "\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-Wno-unused-parameter", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe), *map(str, args)], input=stdin, capture_output=True, text=True, timeout=300, check=True)
    return r.stdout.splitlines()


def test_the_wait_for_a_tile_covers_the_longest_one(tmp_path):
    """A weight gradient's tile runs over every token, 64 per K block, at up to 0.45 us each: twice that has to fit in the
    wait for it, up to the largest accepted number of tokens; few K blocks leave the limit at that of other waits."""
    lines = run(tmp_path, r'''
  for (int64_t t : {int64_t{64}, int64_t{8192}, int64_t{300000000}, int64_t{640000000}, kFfnMaxTokens}) {
    const int64_t kb = (t + 63) / 64;
    std::printf("%lld %llu\n", static_cast<long long>(kb), static_cast<unsigned long long>(tile_wait_ns(2000000000ull, kb)));
  }''')
    got = [tuple(map(int, line.split())) for line in lines]
    assert got[-1][0] == (2**31 - 257 + 63) // 64
    for kb, ns in got:
        assert ns >= 2_000_000_000 and ns >= 2 * 450 * kb
    assert got[1][1] < 2_001_000_000


def test_every_unit_of_a_plan_is_dealt_out_once(tmp_path):
    """Random numbers of tiles and K blocks of the two jobs: each unit in exactly one slot, no pair beyond the end that
    the plan gives, and the tile order a permutation of the tiles."""
    lines = run(tmp_path, r'''
  std::srand(7);
  auto any = [](int n) { return std::rand() % n; };
  for (int round = 0; round < 20000; ++round) {
    const int pairs = any(3) ? 76 : 1 + any(160);
    int64_t units[2], k[2];
    for (int j = 0; j < 2; ++j) units[j] = any(4) ? any(2) ? any(1000) : any(40) : 0, k[j] = 1 + any(200);
    if (!units[0] && !units[1]) continue;
    PairPlan g;
    const int64_t end = make_plan(units, k, any(2), pairs, &g);
    static char seen[2][1000];
    for (auto& s : seen) for (char& c : s) c = 0;
    if (g.pairs < 1 || g.pairs > pairs) return 1;
    for (int p = 0; p < g.pairs; ++p) {
      int64_t load = 0;
      for (int i = 0; i < plan_steps(g, p); ++i) {
        int job, u;
        if (!plan_unit(g, p, i, job, u)) continue;
        if (u < 0 || u >= units[job] || seen[job][u]++) return 2;
        load += k[job];
      }
      if (load > end) return 3;
    }
    for (int j = 0; j < 2; ++j) for (int u = 0; u < units[j]; ++u) if (!seen[j][u]) return 4;
    const int mt = 1 + any(30), nt = 1 + any(30);
    for (char& c : seen[0]) c = 0;
    for (int u = 0; u < mt * nt; ++u) {
      int m, n;
      ordered_tile(u, mt, nt, m, n);
      if (m < 0 || m >= mt || n < 0 || n >= nt || seen[0][m * nt + n]++) return 5;
    }
  }
  std::puts("ok");''')
    assert lines == ["ok"]


# T H I SMs per line -> widths of GATEUP, DOWN ("first+last" where there are two), and of the backward's two launches
WIDTHS = r'''
  int T, H, I, sms;
  while (std::scanf("%d %d %d %d", &T, &H, &I, &sms) == 4) {
    const int pairs = sms / 2;
    auto fwd = [&](int var, int64_t N, int64_t K) {
      if (!ffn_on_pairs(var, T, N, sms)) return std::printf("- ");
      const FwdSplit d = fwd_split(var == F_GATEUP, T, N, K, pairs);
      return d.bn1 ? std::printf("%d+%d ", d.bn0, d.bn1) : std::printf("%d ", d.bn0);
    };
    fwd(F_GATEUP, I, H);
    fwd(F_DOWN, H, I);
    BwdJobs one, two;
    bwd_jobs(T, H, I, ffn_on_pairs(F_DACT, T, I, sms), ffn_on_pairs(F_DX, T, H, sms), true, true, pairs, &one, &two);
    for (int w : {bwd_width(1, T, H, I, one, pairs).bn, bwd_width(2, T, H, I, two, pairs).bn})
      w ? std::printf("%d ", w) : std::printf("- ");
    std::puts("");
  }'''


def check_labels(tmp_path, sms):
    """The sizes of test_gpu_ffn.py's tests of tile widths take the widths that they name."""
    import test_gpu_ffn
    args = lambda f: next(m for m in f.pytestmark if m.name == "parametrize").args[1]  # noqa: E731
    one, two = args(test_gpu_ffn.test_every_tile_width), args(test_gpu_ffn.test_two_tile_widths)
    lines = run(tmp_path, WIDTHS, stdin="".join(f"{T} {H} {I} {sms}\n" for T, H, I, _ in one + two))
    got = [dict(zip(("gate/up", "down", "bwd1", "bwd2"), line.split())) for line in lines]
    for (*_, label), g in zip(one, got):
        assert [v.split("+")[0] for v in g.values()] == label.split(), (label, g)
    every = {k: {w for g in got for w in g[k].split("+")} - {"-"} for k in got[0]}
    assert all(v == {"256", "224", "192", "128"} - ({"224"} if k == "gate/up" else set()) for k, v in every.items()), every
    for (*_, label), g in zip(two, got[len(one):]):
        which, first, last = label.split()
        for k in ("gate/up", "down") if which == "both" else (which,):
            assert g[k] == f"{first}+{last}", (label, g)


def test_sizes_take_the_tile_widths_that_they_are_tested_for(tmp_path):
    check_labels(tmp_path, 152)


@pytest.mark.gpu
def test_sizes_take_the_tile_widths_that_they_are_tested_for_on_this_gpu(tmp_path):
    import torch
    check_labels(tmp_path, torch.cuda.get_device_properties(0).multi_processor_count)
