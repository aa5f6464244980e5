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
