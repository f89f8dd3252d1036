"""The runs that the packed kernels walk (csrc/packed_runs.h), on the CPU: the
header is compiled into a small host program that takes the place of the
kernels' loops, over offsets that are right and over offsets that are not.
"""

import itertools
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_ssd_scan_fwd_amd", "csrc")

# Input: lines "L len cu.."; output: for each piece of len tokens and each row
# that the search for its last token may give, "P s0 s1 row r0" for the first
# walk, and for each row it may begin with, "O s0 s1 row first r0 r1" runs.
PROGRAM = r"""
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>
#include "packed_runs.h"
int main() {
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    int64_t L, len, v;
    in >> L >> len;
    std::vector<int64_t> cu;
    while (in >> v) cu.push_back(v < 0 ? 0 : v > L ? L : v);
    const int64_t S = (int64_t)cu.size() - 1;
    std::printf("C\n");
    for (int64_t s0 = 0; s0 < L; s0 += len) {
      const int64_t s1 = s0 + len < L ? s0 + len : L;
      for (int64_t row = 0; row < S; ++row) {
        int64_t r0 = -1;
        if (ssd::passing_run(cu[row], cu[row + 1], s0, s1, r0))
          std::printf("P %ld %ld %ld %ld\n", (long)s0, (long)s1, (long)row, (long)r0);
      }
      for (int64_t begin = 0; begin < S; ++begin) {
        std::printf("B %ld %ld %ld\n", (long)s0, (long)s1, (long)begin);
        int64_t pos = s0;
        for (int64_t row = begin; pos < s1 && row < S; ++row) {
          int64_t r0 = -1, r1 = -1;
          if (!ssd::next_run(cu[row], cu[row + 1], pos, s1, r0, r1)) continue;
          std::printf("O %ld %ld %ld %ld %ld\n", (long)row, (long)cu[row], (long)r0, (long)r1, (long)pos);
          pos = r1;
        }
      }
    }
  }
}
"""


@pytest.fixture(scope="module")
def runs(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("packed_runs")
    (d / "runs.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(d / "runs.cpp"), "-o", str(d / "runs")],
                   check=True)

    def of(cases):
        text = "".join(" ".join(map(str, (L, n, *cu))) + "\n" for L, n, cu in cases)
        out = subprocess.run([str(d / "runs")], input=text, capture_output=True, text=True, check=True).stdout
        parts = [[ln.split() for ln in p.splitlines() if ln] for p in out.split("C\n")[1:]]
        assert len(parts) == len(cases)
        return [[(r[0], *map(int, r[1:])) for r in p] for p in parts]

    return of


def arbitrary():
    """Every array of up to 3 offsets out of a few, and some longer ones."""
    values = (-1, 0, 1, 3, 4, 5, 8, 9, 10, 99)
    cases = [(10, 4, cu) for n in (2, 3, 4) for cu in itertools.product(values, repeat=n)]
    return cases + [(100, 64, cu) for cu in ([70, 80, 100], [64, 100, 100], [99, 100], [100, 0, 100], [65, 64, 63, 100])]


def test_every_run_lies_inside_its_piece(runs):
    for (L, _, cu), lines in zip(arbitrary(), runs(arbitrary())):
        piece = None
        for ln in lines:
            if ln[0] == "P":
                _, s0, s1, row, r0 = ln
                assert 0 <= s0 <= r0 < s1 <= L, (cu, ln)
            elif ln[0] == "B":
                piece = ln[1:3]
            else:
                _, row, first, r0, r1, pos = ln
                assert piece[0] <= pos <= r0 < r1 <= piece[1] and first <= r0, (cu, ln)


def test_right_offsets_give_every_token_its_sequence(runs):
    cases = [(L, n, cu) for L, n, cu in arbitrary() if cu[0] == 0 and list(cu) == sorted(cu) and cu[-1] <= L]
    assert len(cases) > 50
    for (L, n, cu), lines in zip(cases, runs(cases)):
        at = 0
        while at < len(lines):
            kind, *v = lines[at]
            at += 1
            if kind != "B":
                continue
            s0, s1, begin = v
            taken = {}
            while at < len(lines) and lines[at][0] == "O":
                _, row, first, r0, r1, _ = lines[at]
                for t in range(r0, r1):
                    assert t not in taken
                    taken[t] = row
                at += 1
            # the kernels begin with the last row whose offset is not behind s0
            if begin == max(i for i in range(len(cu)) if cu[i] <= s0):
                want = {t: r for r in range(len(cu) - 1) for t in range(cu[r], cu[r + 1]) if s0 <= t < s1}
                assert taken == want, (cu, s0)


def test_offsets_may_begin_behind_the_first_token(runs):
    """A slice of a longer array of offsets: tokens before its first belong to
    no sequence, all others to theirs."""
    cases = [(L, n, cu) for L, n, cu in arbitrary() if cu[0] > 0 and list(cu) == sorted(cu) and cu[-1] <= L]
    assert len(cases) > 50
    for (L, n, cu), lines in zip(cases, runs(cases)):
        spans = {}
        for ln in lines:
            if ln[0] == "B":
                key = ln[1:]
                spans[key] = {}
            elif ln[0] == "O":
                spans[key].update({t: ln[1] for t in range(ln[3], ln[4])})
        for s0 in range(0, L, n):
            s1 = min(s0 + n, L)
            # the row that the search gives: the first where every offset lies behind s0
            begin = max([i for i in range(len(cu)) if cu[i] <= s0], default=0)
            if begin < len(cu) - 1:
                want = {t: r for r in range(len(cu) - 1) for t in range(cu[r], cu[r + 1]) if s0 <= t < s1}
                assert spans[(s0, s1, begin)] == want, (cu, s0)
