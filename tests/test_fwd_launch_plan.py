"""How many threads the MoE forward's preparation launches (csrc/moe_fwd_plan.hpp), without a GPU: the runtime runs 2^32
threads or more modulo 2^32, without an error, so every layer that the library takes has to stay below."""
import ctypes as C
import os
import random
import subprocess

import pytest

import mxfp8_grouped_gemm_amd as mx

CSRC = os.path.join(os.path.dirname(os.path.abspath(mx.__file__)), "csrc")
MAIN = """
#include <cstdio>
#include "moe_fwd_plan.hpp"
int main() {
  long long T, H, I, E, N, B, s;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &T, &H, &I, &E, &N, &B, &s) == 7) {
    const mx::FwdPrepPlan p = mx::fwd_prep_plan(T, H, I, E, N, B, s != 0);
    std::printf("%d %d %lld %lld %lld %lld\\n", int(p.small), p.threads, (long long)p.nq, (long long)p.ns,
                (long long)p.nf, (long long)p.grid);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", d / "plan", d / "main.cpp"], check=True)

    def run(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes)
        out = subprocess.run([d / "plan"], input=text, capture_output=True, text=True, check=True).stdout
        return [dict(zip(("small", "threads", "nq", "ns", "nf", "grid"), map(int, line.split()))) for line in out.splitlines()]
    return run


def _taken(T, H, I, E, N, B):
    a = mx.MoeFwdArgs(T, H, I, E, N, B, *([0x10000] * 8), None, None, None, 0, 0, 0x10000)
    return mx.lib().moe_fwd_mxfp8_workspace_size(C.byref(a)) > 0


def test_small_layers_of_large_weights(plans):
    """Few slots over weights whose scales alone take more than 2^22 workgroups."""
    sizes = [(8, 64, 32768, 4096, 64, 128), (8, 32, 2 ** 18, 512, 1, 128), (1, 32, 2 ** 22, 32, 1, 128)]
    for s, p in zip(sizes, plans([(*s, 0) for s in sizes])):
        assert _taken(*s)
        assert p["ns"] > 2 ** 22 and p["grid"] * p["threads"] < 2 ** 32 and not p["small"], (s, p)


def test_a_small_layer_takes_one_launch(plans):
    p, = plans([(256, 128, 256, 4, 7, 128, 0)])
    assert p["small"] and p["threads"] == 1024 and p["grid"] == p["nq"] + p["ns"] + 1


def test_every_layer_that_is_taken(plans):
    r = random.Random(0)

    def log2(lo, hi):
        return int(2 ** r.uniform(lo, hi))
    sizes = []
    while len(sizes) < 4000:
        s = (log2(0, 24), 32 * log2(0, 12), 32 * log2(0, 17), log2(0, 23), log2(0, 14), r.choice([128, 256, 512, 1024]))
        if _taken(*s):
            sizes.append(s)
    small = 0
    for by_slot in (0, 1):
        for s, p in zip(sizes, plans([(*s, by_slot) for s in sizes])):
            if by_slot and (s[1] + 127) // 128 * 4 > 2 ** 30 // (s[4] * s[5]):
                continue      # X is not laid out by slot there
            assert p["grid"] * p["threads"] < 2 ** 32, (s, by_slot, p)
            small += p["small"]
    assert small > 500
