"""The arithmetic by which workgroups share the work of drafted trees (csrc/awq_tree_share.h), built for
the CPU with signed overflows trapped: borders are those of whole numbers, at the longest lines too, and a row
tile is in no more chunks than it has room for."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a16_group_quantized_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "awq_tree_share.h"
int main() {
    int all, shares, least, most, room, first, units, far;
    while (std::scanf("%d %d %d %d %d %d %d %d", &all, &shares, &least, &most, &room, &first, &units, &far) == 8) {
        const int each = awq::share_units(all, shares, least, most, room);
        std::printf("%d %d %d", each, awq::first_share_from(first + far, each), awq::last_share_upto(first + units - far, each));
        const int some[5] = {0, 1, shares / 2, shares - 1, shares};
        for (int k : some) std::printf(" %d", awq::share_border(k, each, all));
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is needed")
    at = tmp_path_factory.mktemp("share")
    (at / "share.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    str(at / "share.cpp"), "-o", str(at / "share")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        r = subprocess.run([str(at / "share")], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return [[int(x) for x in line.split()] for line in r.stdout.splitlines()]

    return run


def expect(case, got):
    all_, n, least, most, room, first, units, far = case
    each = max(-(-all_ // n), least, most // (room - 1) + 1 if room > 1 else 1)
    each = max(1, min(each, all_))
    assert got[0] == each, case
    assert got[1] == -(-(first + far) // each), case
    assert got[2] == (-1 if first + units - far < 0 else (first + units - far) // each), case
    assert got[3:] == [min(k * each, all_) for k in (0, 1, n // 2, n - 1, n)], case
    assert got[-1] == all_, case                                 # the shares reach the line's end
    if room > 1:
        assert max(got[2] - got[1] + 1, 0) + 1 <= room, case     # chunks of the row tile


def test_a_long_sequence_among_short_ones(shares):
    """2^28 tokens beside 1023 sequences of a tile or two, 1024 shares, room for three chunks: the last share's
    border, 1024 times half the longest, is past 2^31.  And up to 2^30 units, shares and room of all kinds."""
    cases = [((1 << 22) + 2046, 1024, 8, 1 << 22, 3, 0, 1 << 22, 6), ((1 << 22) + 1023, 1024, 8, 1 << 22, 33, 0, 1 << 22, 6)]
    for all_ in (1 << 30, (1 << 30) - 1, 1 << 29, 3 << 28):
        for n in (1, 2, 255, 256, 1024, 2048, 1 << 20):
            for room in (1, 2, 3, 33):
                for units in (all_, all_ // 2, 1):
                    far = 6 if room > 1 else units
                    for first in (0, all_ - units):
                        cases.append((all_, n, 8, units, room, first, units, far))
    got = shares(cases)
    assert len(got) == len(cases)
    for case, line in zip(cases, got):
        expect(case, line)


def test_lines_of_any_length(shares):
    rng = random.Random(1)
    cases = []
    for _ in range(5000):
        tiles = [max(1, int(2 ** rng.uniform(0, 16))) for _ in range(rng.randint(1, 40))]
        room = rng.choice([1, 2, 3, 5, 33])
        at = rng.randrange(len(tiles))
        cases.append((sum(tiles), rng.choice([1, 7, 64, 128, 512, 1024]), 8, max(tiles), room, sum(tiles[:at]), tiles[at],
                      6 if room > 1 else tiles[at]))
    got = shares(cases)
    assert len(got) == len(cases)
    for case, line in zip(cases, got):
        expect(case, line)


def test_nothing(shares):
    """No rows: shares are empty."""
    (line,) = shares([(0, 128, 8, 0, 3, 0, 0, 6)])
    assert line[0] == 1 and line[3:] == [0] * 5
