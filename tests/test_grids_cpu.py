"""Calls of more threads than a launch takes, and the launches they are cut
into (csrc/moe_grid.h, host arithmetic, compiled here)."""
import os
import subprocess

import pytest

import w4a16_int4_grouped_amd as M

CSRC = os.path.join(M.PKG_DIR, "csrc")
SLICES = """
#include <cinttypes>
#include <cstdio>
#include "moe_grid.h"
int main() {
  long long blocks, stop;
  int threads;
  while (std::scanf("%lld %d %lld", &blocks, &threads, &stop) == 3) {
    const int e = moe::in_slices(blocks, threads, [&](uint32_t first, uint32_t n) {
      std::printf("%" PRIu32 " %" PRIu32 " ", first, n);
      return (long long)first >= stop ? 7 : 0;
    });
    std::printf("%d\\n", e);
  }
}
"""


def compiled(tmp_path_factory, name, text):
    d = tmp_path_factory.mktemp(name)
    (d / "main.cpp").write_text(text)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "main.cpp"), "-o", str(d / name)],
                   check=True)

    def run(lines):
        r = subprocess.run([str(d / name)], input="\n".join(lines), capture_output=True, text=True, check=True)
        return [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
    return run


@pytest.fixture(scope="module")
def slices(tmp_path_factory):
    return compiled(tmp_path_factory, "slices", SLICES)


CALLS = [(1, 256), (128, 256), ((1 << 24) - 1, 256), (1 << 24, 256), ((1 << 24) + 5, 256), ((1 << 25) + 128, 256),
         ((1 << 31) - 1, 64), ((1 << 31) - 1, 320), ((1 << 31) - 1, 384), ((1 << 31) - 1, 512), ((1 << 31) - 1, 1024)]


def test_slices_cover_a_call_and_fit_a_launch(slices):
    for (blocks, threads), got in zip(CALLS, slices([f"{b} {t} {1 << 40}" for b, t in CALLS])):
        assert got.pop() == 0
        at = 0
        for first, n in zip(got[::2], got[1::2]):
            assert first == at and first % 128 == 0 and 0 < n and n * threads < 1 << 32
            at += n
        assert at == blocks
        assert len(got) == 2 * -(-blocks // (((1 << 32) - 1) // threads // 128 * 128))


def test_nothing_is_launched_behind_an_error_and_nothing_for_nothing(slices):
    assert slices(["0 256 0", f"{1 << 26} 256 1"]) == [[0], [0, 16777088, 16777088, 16777088, 7]]
