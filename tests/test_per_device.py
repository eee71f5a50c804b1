"""The table that holds what a kernel's launch asks of a device (per_device.h),
compiled for the host: one answer per device, and a query that fails is not
remembered."""
import os
import shutil
import subprocess

import pytest

from fp8_fine_grained_gb300 import build as libbuild

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
int asked = 0;
int main()
{
    static fp8fg::PerDevice t;
    auto says = [](int n) { return [n] { ++asked; return n; }; };
    auto check = [](const char *what, int got, int want) {
        if (got != want)
            std::printf("%s: %d, not %d\n", what, got, want);
    };
    check("a failed query", t.get(0, says(0)), 0);
    check("a negative answer", t.get(0, says(-1)), 0);
    check("asked again after a failure", t.get(0, says(23)), 23);
    check("kept", t.get(0, says(5)), 23);
    check("asked three times", asked, 3);
    check("another device has its own", t.get(1, says(15)), 15);
    check("the first keeps its own", t.get(0, says(1)), 23);
    check("the last device", t.get(63, says(7)), 7);
    check("beyond the table", t.get(64, says(7)), 0);
    check("no device", t.get(-1, says(7)), 0);
    check("asked in all", asked, 5);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_answers_are_kept_per_device_and_failures_are_not(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", libbuild.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout == ""


def test_the_cluster_query_goes_through_it():
    """The number of clusters that run at once decides the split and with it the order of the sums."""
    with open(os.path.join(libbuild.CSRC, "gemm_gated.cu")) as f:
        text = f.read()
    at = text.index("int clusters_at_once(")
    body = text[at:text.index("\n}\n", at)]
    assert "PerDevice known" in body and "std::atomic" not in body
