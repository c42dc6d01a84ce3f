"""The cut of the 8-bit decode's page stream in groups and ranges, on the host: the
kernel's own arithmetic (``Q8Groups`` of ``pa_internal.h``) in a small program."""

import os
import shutil
import subprocess

import pytest

from paged_kv_cache_202_gb300 import _build

_SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "pa_internal.h"
int main(int argc, char** argv) {
    for (int i = 1; i + 3 < argc; i += 4) {
        const int P = atoi(argv[i]), warps = atoi(argv[i + 1]), chunk = atoi(argv[i + 2]), cols = atoi(argv[i + 3]);
        const pa::Q8Groups cut(P, warps, chunk, cols);
        printf("%d %d %d %d %d\n", cut.at[0], cut.at[1], cut.at[2], cut.at[3], cut.cut() ? 1 : 0);
    }
}
"""


def _program(at, source):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = at / "groups.cpp", at / "groups"
    src.write_text(source)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", _build.CSRC, "-I", _build.INCLUDE,
                    "-I", os.path.join(cuda, "include"), "-o", exe, src], check=True)
    return exe


def _run(exe, cases):
    r = subprocess.run([exe, *[str(x) for c in cases for x in c]], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    return [[int(x) for x in line.split()] for line in r.stdout.splitlines()]


def test_groups_of_an_empty_stream_have_pages(tmp_path):
    """The kernel divides by a group's pages, also when no sequence of the call has any."""
    cases = [(P, warps, chunk, cols) for P in (0, 1, 2, 1000, 10 ** 6) for warps in (1, 1824) for chunk in (1, 2, 4)
             for cols in (1, 16)]
    for (P, warps, chunk, cols), (a0, a1, a2, a3, cut) in zip(cases, _run(_program(tmp_path, _SOURCE), cases)):
        assert a0 == 0 < a3 and a3 % chunk == 0 and 0 < a1 <= a2 <= a3 and cut == (a1 < a3)
        assert warps * a3 >= P
        assert P > 0 or (a3 == chunk and not cut)


_COVER = r"""
#include <cstdio>
#include <cstdlib>
#include "pa_internal.h"
// The kernel's ranges in stream order: the pages that they cover, -1 where one does not
// begin at the end of the last; the groups; the largest place reckoned on the way.
int main(int argc, char** argv) {
    for (int i = 1; i + 3 < argc; i += 4) {
        const int warps = atoi(argv[i + 1]), chunk = atoi(argv[i + 2]), cols = atoi(argv[i + 3]);
        const long long P = atoll(argv[i]) < 0 ? (long long)pa::kQ8MaxPages + 1 + atoll(argv[i]) : atoll(argv[i]);
        const pa::Q8Groups cut(P, warps, chunk, cols);
        const long long per = cut.at[3], groups = (P + per - 1) / per;
        long long end = 0, most = P + per - 1;
        bool ok = true;
        for (long long g = 0; g < groups; ++g)
            for (int k = 0; k < 3; ++k) {
                const long long x0 = g * per + cut.at[k], x1 = g * per + cut.at[k + 1];
                if (x1 > most) most = x1;
                ok = ok && (x0 < P ? x0 : P) == end && x1 >= x0;
                end = x1 < P ? x1 : P;
            }
        printf("%d %lld %lld\n", ok && end == P, groups, most);
    }
}
"""


def test_ranges_cover_the_largest_stream_in_32_bits(tmp_path):
    """Every page once, by no more groups than warps, and no sum on the way past 2^31 - 1.
    (-1: the largest stream that a call may have, -2 one page less, ...)"""
    cases = [(P, warps, chunk, cols) for P in (0, 1, 5, 4097, 10 ** 6, 2 ** 30 + 7, -10 ** 6, -2, -1)
             for warps in (256, 1064, 1672, 1824) for chunk in (1, 2, 4) for cols in (4, 16)]
    for (P, warps, _, _), (ok, groups, most) in zip(cases, _run(_program(tmp_path, _COVER), cases)):
        assert ok and groups <= warps and most < 2 ** 31 and (groups > 0) == (P != 0)
