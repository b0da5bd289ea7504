"""The weight ring of the 4-bit kernels on the CPU, when a wait for a stage runs out.

The struct's source is compiled as it stands with stand-ins for its barrier and copy operations: after a wait that ran out
nothing more may be requested (its barrier's phase is still open), and every copy on its way has to be waited for before the
warp ends, as it would land in shared memory that is no longer the kernel's.
"""
import pathlib
import re
import subprocess

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "verify_weight_streaming_b200" / "csrc"

HOST = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>
#define __device__
#define __forceinline__ inline
#define __noinline__
#define MR_DEVERR_GEMV_TIMEOUT 1u
struct Barrier { int open = 0, done = 0; bool in_flight = false; };  // phases requested and completed
static Barrier bar[8];
static int waits, fails_at, requests, bad;
static bool landed = true;      // whether a stage has arrived when it is waited for
static void mbar_init(uint32_t, uint32_t) {}
static void fence_mbar_init() {}
static void __syncwarp() {}
static void mbar_arrive_expect_tx(uint32_t b, uint32_t) {
    Barrier &x = bar[b / 8];
    if (x.open != x.done) ++bad;  // an arrival in a phase that is still open
    ++x.open;
    x.in_flight = true;
    ++requests;
}
static void bulk_g2s(uint32_t, const void *, uint32_t, uint32_t) {}
static bool mbar_wait_bounded(uint32_t b, uint32_t parity, uint32_t) {
    Barrier &x = bar[b / 8];
    if (++waits == fails_at) return false;      // runs out; its copy lands later
    if (x.open == x.done) return (uint32_t)((x.done - 1) & 1) == parity;
    if ((uint32_t)(x.done & 1) != parity) { ++bad; return false; }
    x.done = x.open;
    x.in_flight = false;
    return true;
}
RING
int main(int argc, char **argv) {
    const int slots = atoi(argv[1]), stages = atoi(argv[2]);
    fails_at = atoi(argv[3]);
    Ring ring(0, 0, slots, 16);
    int asked = 0;
    auto request = [&] { if (asked < stages) { ring.request(nullptr, 16, 0); ++asked; } };
    for (int s = 0; s < slots; ++s) request();
    for (int i = 0; i < stages; ++i) {
        ring.wait();
        ring.done();
        request();
    }
    int flying = 0;
    for (const Barrier &b : bar) flying += b.in_flight;
    printf("%d %d %d\n", bad, flying, requests);
}
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    text = (CSRC / "w4_core.cuh").read_text()
    body = re.search(r"^struct Ring \{.*?^\};$", text, re.S | re.M).group(0)
    at = tmp_path_factory.mktemp("ring")
    (at / "ring.cpp").write_text(HOST.replace("RING", body))
    subprocess.run(["g++", "-std=c++17", "-w", "-o", str(at / "ring"), str(at / "ring.cpp")], check=True)
    return lambda *args: tuple(map(int, subprocess.run([str(at / "ring"), *map(str, args)], capture_output=True, text=True,
                                                       check=True).stdout.split()))


@pytest.mark.parametrize("slots", [2, 3, 4])
@pytest.mark.parametrize("stages", [1, 2, 5, 12])
def test_no_wait_runs_out(ring, slots, stages):
    assert ring(slots, stages, 0) == (0, 0, stages)


@pytest.mark.parametrize("slots", [2, 3, 4])
@pytest.mark.parametrize("stages", [1, 2, 5, 12])
def test_a_wait_that_runs_out_is_the_last(ring, slots, stages):
    for at in range(1, stages + 1):
        bad, flying, requests = ring(slots, stages, at)
        assert bad == 0 and flying == 0 and requests == min(stages, slots + at - 1), at
