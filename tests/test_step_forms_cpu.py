"""Which form of combine's gradient each case of its tests takes, by the
library's own rule (csrc/moe_step_form.h, host arithmetic, compiled here): a
changed border that leaves a form untested fails here."""
import pytest

from tests.test_gpu_zc_combine_forms import CASES
from tests.test_grids_cpu import compiled

TEAMS = """
#include <cstdio>
#include "moe_step_form.h"
int main() {
  int T, H;
  while (std::scanf("%d %d", &T, &H) == 2) {
    const moe::Team t = moe::team_of(T, H);
    std::printf("%d %d\\n", t.threads, (int)t.one);
  }
}
"""


@pytest.fixture(scope="module")
def teams(tmp_path_factory):
    return compiled(tmp_path_factory, "teams", TEAMS)


def test_each_combine_case_takes_its_form(teams):
    want = [(16, 1), (16, 0), (16, 0), (16, 1), (64, 1), (64, 0), (64, 0), (64, 1), (64, 1), (256, 1), (256, 1), (256, 0),
            (256, 0), (256, 0)]
    got = [tuple(t) for t in teams([f"{c[0]} {c[3]}" for c in CASES])]
    assert got == want
    passes = {(t, one, -(-c[3] // (8 * 4 * t)) > 1) for c, (t, one) in zip(CASES, got)}
    # every form that there is: 64 threads take all rows of a token only in one pass, 16 never take two
    assert passes == {(16, 1, False), (16, 0, False), (64, 1, False), (64, 0, False), (64, 1, True), (256, 1, False),
                      (256, 1, True), (256, 0, False), (256, 0, True)}


def test_no_call_takes_a_form_that_its_kernel_has_not(teams):
    """16 threads add up rows of one pass only, and 64 or 256 only rows of one token."""
    T = [1, 127, 128, 129, 1023, 1024, 4095, 4096, 8191, 8192, 1 << 24]
    H = [8, 136, 256, 264, 504, 512, 520, 1024, 2048, 2056, 8192, 8200, 1 << 20]
    at = [(t, h) for t in T for h in H]
    seen = set()
    for (t, h), (threads, one) in zip(at, teams([f"{t} {h}" for t, h in at])):
        assert threads in (16, 64, 256) and (threads > 16 or h <= 16 * 8 * 4)
        seen.add((threads, one, h > 32 * threads))
    assert (64, 0, True) not in seen and len(seen) == 9
