"""The simple layer norm kernels' indices (csrc/norm_index.h), compiled for the host: each value
is visited once, and nothing leaves its array at sizes whose offsets pass 32 bits."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "deformable_convolution_dcn1d_b200", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <vector>
#include "norm_index.h"
using namespace dcn1d;
typedef __int128 wide;

static int bad = 0;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); bad = 1; } } while (0)

// Every value, statistic and step of small sizes, once each.
static void once(int64_t B, int64_t C, int64_t L) {
    const AnyIndex at(C, L, lanes_along(L));
    const int64_t nb = L == 1 ? (C + 31) / 32 : C * ((L + 31) / 32);
    std::vector<int> seen(B * C * L), stat(B * L), step(B * nb);
    for (int64_t tile = 0; tile < B * at.tiles; ++tile)
        for (int i = 0; i < kAnyThreads; ++i) {
            const int64_t b = at.b_of(tile), l = at.l_of(tile, i);
            if (l >= L)
                continue;
            if (i / at.TL == 0)
                ++stat.at(at.stat(b, l));
            for (int64_t c = i / at.TL; c < C; c += at.rows()) {
                ++seen.at(at.value(b, c, l));
                if (L == 1 ? c % 32 == 0 : l % 32 == 0)
                    ++step.at(at.step(b, c, l));
                CHECK(at.step(b, c, l) >= 0 && at.step(b, c, l) < B * nb);
            }
        }
    for (int n : seen) CHECK(n == 1);
    for (int n : stat) CHECK(n == 1);
    for (int n : step) CHECK(n == 1);
}

// First and last tiles, threads and channels of large sizes against 128-bit arithmetic.
static void large(int64_t B, int64_t C, int64_t L) {
    const AnyIndex at(C, L, lanes_along(L));
    const wide total = (wide)B * C * L, steps = L == 1 ? (wide)B * ((C + 31) / 32)
                                                       : (wide)B * C * ((L + 31) / 32);
    CHECK(total < ((wide)1 << 62));
    const int64_t n = B * at.tiles;
    wide top = -1;
    for (int64_t tile : {(int64_t)0, at.tiles - 1, n / 2, n - at.tiles, n - 1})
        for (int i = 0; i < kAnyThreads; ++i) {
            const int64_t b = at.b_of(tile), l = at.l_of(tile, i);
            CHECK(b >= 0 && b < B && l >= 0);
            if (l >= L)
                continue;
            CHECK(at.stat(b, l) == (wide)b * L + l && at.stat(b, l) < (wide)B * L);
            const int64_t row0 = i / at.TL;
            if (row0 >= C)
                continue;
            const int64_t last = row0 + (C - 1 - row0) / at.rows() * at.rows();
            for (int64_t c : {row0, last}) {
                const wide v = ((wide)b * C + c) * L + l;
                CHECK(c < C && at.value(b, c, l) == v && v < total);
                CHECK(at.step(b, c, l) >= 0 && at.step(b, c, l) < steps);
                if (v > top) top = v;
            }
        }
    CHECK(top == total - 1);   // the last value is reached
    const int64_t blocks = n < 1184 ? n : 1184;
    CHECK(at.part(blocks - 1) + C + C - 1 == (wide)blocks * 2 * C - 1);
}

int main() {
    for (int64_t B : {1, 3})
        for (int64_t C : {1, 31, 32, 33, 300})
            for (int64_t L : {1, 2, 3, 31, 32, 33, 65})
                once(B, C, L);
    large(1026, 512, 4096);                    // 2^31 + 2^22
    large(4097, 16, 32769);
    large(1, 2147483647, 3);
    large(2147483647, 2, 1);
    large(1, 2147483647, 1);
    large(3, 2147483647, 715827882);           // the largest B L and C
    large(2, 70000, 1000001);
    return bad;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_index_is_inside_and_taken_once(tmp_path):
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
