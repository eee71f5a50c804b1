"""What the 4-bit products' kernel waits for before it leaves after a wait ran out:
every copy that its ring still has in flight, the stage that was given up on among
them (another warp's wait may have ended it early). The kernel's own function, taken
from its source and run on the CPU against copies that land at given times."""
import itertools
import os
import re
import subprocess

import pytest

from fp8_fine_grained_gb300 import build as libbuild

HARNESS = r"""
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
static uint64_t now, lands[4];
static int phase[4], ring_, strays, waits_for_all;
static uint64_t global_timer_ns() { return now += 10; }
static bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    const int st = (int)(bar - 4096) / 8;
    now += 10;
    if (bar < 4096 || st >= ring_ || phase[st] != (int)parity) { ++strays; return true; }
    return lands[st] <= now;
}
static void wait_all() { ++waits_for_all; }
FUNCTION
// ring stage parity ahead limit; when the copy of each of the ahead stages lands
int main(int argc, char **argv)
{
    long long v[16] = {};
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7, v + 8) == 9) {
        ring_ = (int)v[0];
        now = 0;
        strays = waits_for_all = 0;
        for (int i = 0; i < 4; ++i)
            phase[i] = -1;
        for (int i = 0; i < v[3]; ++i) {
            const int st = (int)(v[1] + i) % ring_;
            lands[st] = (uint64_t)v[5 + i];
            phase[st] = (int)v[2] ^ (v[1] + i >= ring_);
        }
        drain(4096, (int)v[1], (uint32_t)v[2], (int)v[3], ring_, (uint64_t)v[4]);
        int flying = 0;
        for (int i = 0; i < v[3]; ++i)
            flying += (uint64_t)v[5 + i] > now;
        printf("%d %d %d %llu\n", flying, strays, waits_for_all, (unsigned long long)now);
    }
    return 0;
}
"""
LIMIT, NEVER = 5000, 1 << 60


def source():
    with open(os.path.join(libbuild.CSRC, "w4.cu")) as f:
        text = f.read()
    at = text.index("__device__ __forceinline__ void drain(")
    body = text[at:text.index("\n}\n", at) + 3].replace("__device__ __forceinline__", "static")
    return re.sub(r'asm volatile\("cp\.async\.wait_all;"[^;]*;', "wait_all();", body)


@pytest.fixture(scope="module")
def drained(tmp_path_factory):
    d = tmp_path_factory.mktemp("drain")
    (d / "drain.cpp").write_text(HARNESS.replace("FUNCTION", source()))
    subprocess.run(["g++", "-O1", "-o", str(d / "drain"), str(d / "drain.cpp")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "drain")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def cases(times):
    for ring in (2, 3, 4):
        for stage, parity, ahead in itertools.product(range(ring), (0, 1), range(1, ring + 1)):
            for t in itertools.product(times, repeat=ahead):
                yield (ring, stage, parity, ahead, LIMIT, *t, *[0] * (4 - ahead))


def test_every_copy_lands_before_the_kernel_leaves(drained):
    todo = list(cases((0, 700, 3000)))
    for case, (flying, strays, waits, _) in zip(todo, drained(todo)):
        assert flying == 0 and strays == 0 and waits == 1, case


def test_a_copy_that_never_comes_costs_the_limit_once(drained):
    todo = [c for c in cases((0, 3000, NEVER)) if NEVER in c]
    for case, (flying, strays, waits, took) in zip(todo, drained(todo)):
        assert flying == case.count(NEVER) and strays == 0 and waits == 1, case
        assert LIMIT <= took <= LIMIT + 200, case
