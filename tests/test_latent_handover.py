"""Bookkeeping of the expanded attention kernels' work hand-over (csrc/handover.h), compiled for the host: whichever
wait of a loader gives up, and whenever, the block waits for exactly the answer that may still be on its way."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_expert_gb300",
                    "csrc")

# A loader's loop: ask; wait for a free item slot; (loads); wait for the answer.  `gives_up` names the wait that fails in
# iteration `at`, `none_at` the iteration whose answer says that nothing is left (no request follows it).  `landed` counts
# the answers that have arrived, one phase of the barrier each; a wait on parity p returns when the phase of that parity
# is the last complete one.
SOURCE = r"""
#include <cstdio>
#include "handover.h"
enum Wait { SLOT, LOADS, ANSWER };
static bool complete(uint32_t landed, uint32_t parity) { return ((landed & 1u) ^ 1u) == parity; }
static int run(uint32_t at, Wait gives_up, uint32_t none_at) {
    fs::HandOver ho;
    uint32_t landed = 0, asked = 0;
    bool more = true;
    for (uint32_t k = 0;; ++k) {
        if (more) { ho.ask(); ++asked; }
        if (k == at && gives_up == SLOT) break;
        if (!more) break;
        if (k == at && gives_up == LOADS) break;
        if (complete(landed, ho.parity())) return 1;           // the answer is not there yet
        if (k == at && gives_up == ANSWER) break;
        ++landed;
        if (!complete(landed, ho.parity())) return 2;
        ho.answer();
        more = k != none_at;
    }
    if (ho.pending() != (asked != landed)) return 3;           // a wait for nothing, or none for an answer
    if (ho.pending()) {
        if (complete(landed, ho.parity())) return 4;           // the wait would return before the answer has landed
        if (!complete(landed + 1, ho.parity())) return 5;      // ... or not when it has
    }
    return 0;
}
int main() {
    for (uint32_t at = 0; at < 9; ++at)
        for (uint32_t none_at = 0; none_at < 9; ++none_at)
            for (int w = SLOT; w <= ANSWER; ++w)
                if (int e = run(at, static_cast<Wait>(w), none_at)) {
                    std::printf("iteration %u, wait %d, last answer %u: %d\n", at, w, none_at, e);
                    return 1;
                }
    return 0;
}
"""


def test_every_exit_waits_for_the_answer_on_its_way(tmp_path):
    src, exe = tmp_path / "handover.cpp", tmp_path / "handover"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
