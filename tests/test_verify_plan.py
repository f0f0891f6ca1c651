"""How many CTAs vt_verify_draft gives a sequence (csrc/verify_plan.cuh, compiled
alone): never a larger cluster than the device can hold."""
import os
import subprocess

import pytest

import frequency_ranked_drafter_gb300 as vt

PROGRAM = """
#include <cstdio>
#include "verify_plan.cuh"
int main() {
  int B, V, sms, largest;
  while (std::scanf("%d %d %d %d", &B, &V, &sms, &largest) == 4)
    std::printf("%d\\n", vt::verify_ctas(B, V, sms, largest));
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    csrc = os.path.join(os.path.dirname(vt.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(d / "plan.cpp"), "-o",
                    str(d / "plan")], check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        r = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True)
        return [int(x) for x in r.stdout.split()]
    return ask


def test_no_larger_than_the_device_holds(plan):
    cases = [(B, V, sms, largest) for B in (1, 2, 9, 37, 38, 64, 152, 700, 65535)
             for V in (1, 1024, 1025, 5003, 32003, 128256, 1 << 19) for sms in (1, 8, 76, 152)
             for largest in (1, 2, 4, 8, 16)]
    for case, C in zip(cases, plan(cases)):
        assert 1 <= C <= case[3] and C & (C - 1) == 0, (case, C)


def test_a_whole_device_keeps_its_plans(plan):
    """Both sides of the rules' figures."""
    want = {(1, 128256): 16, (24, 128256): 16, (38, 128256): 16, (39, 128256): 8, (64, 128256): 8,
            (100, 128256): 8, (152, 128256): 8, (153, 128256): 4, (256, 128256): 4, (64, 32003): 8,
            (1, 1024): 1, (1, 1025): 2, (700, 2500): 1, (65535, 128256): 1}
    got = plan([(B, V, 152, 16) for B, V in want])
    assert got == list(want.values())
