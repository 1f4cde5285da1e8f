"""Which copies of a ring may still be in flight (csrc/wc_ring.cuh), compiled
for the host and held against a model of the stages' barriers."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "wc_ring.cuh"
extern "C" int last_fills(uint32_t fills, uint32_t stages, uint32_t* out) {
    int n = 0;
    wc::ring_last_fills(fills, stages, [&](uint32_t s, uint32_t p) { out[2 * n] = s, out[2 * n + 1] = p, ++n; });
    return n;
}
"""


@pytest.fixture(scope="module")
def last_fills(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", str(d / "ring.so"), str(d / "ring.cpp"),
                    "-I" + os.path.join(ROOT, "lossless_weight_compression_b200", "csrc")], check=True)
    lib = ctypes.CDLL(str(d / "ring.so"))

    def call(fills, stages):
        out = (ctypes.c_uint32 * (2 * stages))()
        n = lib.last_fills(ctypes.c_uint32(fills), ctypes.c_uint32(stages), out)
        return [(out[2 * k], out[2 * k + 1]) for k in range(n)]
    return call


@pytest.mark.parametrize("stages", [1, 4, 7, 8])
def test_every_copy_that_may_be_in_flight_is_waited_for(last_fills, stages):
    """A stage's barrier counts completed phases, and a wait for parity p passes
    when the last completed phase has that parity. For every number of fills and
    every choice of one copy that has not landed, some wait holds; once all have
    landed, none does. A stage is filled again only after its copy has landed."""
    for fills in range(3 * stages + 2):
        waits = last_fills(fills, stages)
        assert len(waits) == min(fills, stages)
        for late in [None] + list(range(max(0, fills - stages), fills)):
            done = [0] * stages
            for k in range(fills):
                done[k % stages] += k != late
            held = [s for s, p in waits if done[s] == 0 or (done[s] - 1) % 2 != p]
            assert held == ([] if late is None else [late % stages]), (fills, late)
