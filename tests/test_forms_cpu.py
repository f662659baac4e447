"""Which form of tiles each case of the tile tests takes, by the library's own
rule (csrc/moe_ragged_form.h, host arithmetic, compiled here): a changed
constant that moves a case, or leaves a form untested, fails here."""
import os
import subprocess

import pytest

import w4a16_int4_grouped_amd as M
from tests import test_gpu_o_tiles as o
from tests import test_gpu_q_forms as q
from tests import test_gpu_s_scales as s
from tests import test_gpu_t_forms as t

FORMS = ["LARGE", "TWO", "FOUR", "SPLIT", "THIN"]
MAIN = """
#include <cstdio>
#include "moe_ragged_form.h"
int main() {
  moe::FormCall p;
  int mx, wgrad;
  while (std::scanf("%d %d %d %d %d %d %d %d", &mx, &wgrad, &p.E, &p.M, &p.I, &p.J, &p.C, &p.out_size) == 8) {
    p.mx = mx, p.wgrad = wgrad;
    std::printf("%d\\n", (int)moe::form_of(p));
  }
}
"""


@pytest.fixture(scope="module")
def forms_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("forms")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(M.PKG_DIR, "csrc"), str(d / "main.cpp"),
                    "-o", str(d / "forms")], check=True)

    def run(calls):
        """The forms of calls (way, E, N, K, rows, bytes of an output value)."""
        lines = []
        for way, E, N, K, rows, size in calls:
            I, J, C = {"dgrad": (K, 0, N), "wgrad": (K, N, 0)}.get(way, (N, 0, K))
            lines.append(f"{int(way == 'mx')} {int(way == 'wgrad')} {E} {rows} {I} {J} {C} {size}\n")
        r = subprocess.run([str(d / "forms")], input="".join(lines), capture_output=True, text=True, check=True)
        return [FORMS[int(f)] for f in r.stdout.split()]
    return run


def rows(counts):
    return sum(counts) if isinstance(counts, list) else counts


def same(form):
    return {4: form, 2: form}


def mx(E, N, K, counts):
    return "mx", E, N, K, counts


# test cases in their order, and the form each is there for (by the bytes of an output value; MXFP4 cases give FP32)
EXPECTED = [
    (o.CASES, ["TWO", "TWO", "TWO", "FOUR", "FOUR", "TWO", {4: "TWO", 2: "FOUR"}, "FOUR", "THIN", "THIN", "THIN", "THIN"]),
    (q.CASES, ["LARGE"] * 4 + ["TWO", "FOUR"] + ["SPLIT"] * 3 + ["THIN"] * 6),
    (t.CASES, ["FOUR", "FOUR"]),
    ([mx(*c) for c in ((9, 2056, 544, o.UNEVEN), (6, 4104, 2080, o.UNEVEN[:6]), (300, 1032, 1056, 30000),
                       (40, 4104, 96, 9000), (5, 136, 7200, 300), (2, 264, 4128, [33, 0]))],
     ["FOUR", "FOUR", "FOUR", "FOUR", "THIN", "THIN"]),
    ([mx(*c) for c in ((12, 4104, 4128, q.GROUPS), (16, 1032, 4128, 300), (20, 512, 7168, 1000), (3, 264, 4128, [1, 20, 0]),
                       (1, 4104, 7200, [64]), (1, 392, 2080, [200]))],
     ["LARGE", "TWO", "SPLIT", "THIN", "THIN", "THIN"]),
    ([mx(*c) for c in t.MX_CASES], ["TWO", "TWO", "LARGE", "LARGE"]),
    ([mx(8, 2056, K, s.ENDS) for K in (32, 256, 544, 1056, 2080, 4128)], ["TWO"] * 6),
    ([mx(32, 4104, K, s.ENDS * 4) for K in (32, 256, 544, 1056, 2080, 4128)], ["FOUR"] * 4 + ["LARGE"] * 2),
]


def test_each_case_takes_its_form(forms_of):
    reached = set()
    for cases, want in EXPECTED:
        assert len(cases) == len(want)
        want = [w if isinstance(w, dict) else same(w) for w in want]
        for size in (4, 2):
            got = forms_of([(way, E, N, K, rows(c), size) for way, E, N, K, c in cases])
            for (way, *shape), g, w in zip(cases, got, want):
                if way != "mx" or size == 4:
                    assert g == w[size], (way, *shape, size)
                    reached.add((way, g, size))
    missing = {(way, f, 4) for way in ("fwd", "dgrad", "wgrad", "mx") for f in FORMS} - reached
    missing |= {(way, f, 2) for way in ("fwd", "dgrad", "wgrad") for f in FORMS} - reached
    assert not missing


def parametrised(test):
    """The MXFP4 cases that a tile test is parametrised with."""
    return [m.args[1] for m in test.pytestmark if m.name == "parametrize"][0]


def test_the_listed_mxfp4_cases_are_the_tests_own():
    """EXPECTED repeats the two tests' inline lists; they must be those."""
    for test, at in ((o.test_every_tile_form_of_mxfp4_is_exact, 3), (q.test_forms_of_mxfp4, 4)):
        assert [tuple(c) for c in parametrised(test)] == [c[1:] for c in EXPECTED[at][0]]


def test_no_rows(forms_of):
    assert forms_of([(way, 4, 64, 64, 0, 4) for way in ("fwd", "wgrad", "mx")]) == ["LARGE"] * 3
