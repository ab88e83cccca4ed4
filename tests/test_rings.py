"""What a kernel that gives up waits for before it leaves (csrc/rings.h), on the CPU: a model of a ring of asynchronous
copies with mbarrier phases, stopped at a random moment. No GPU fault or hang is made anywhere."""
import os
import subprocess

from tests.conftest import ROOT

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "rings.h"

// One ring: the producer asks for copy t into stage t % S once the consumer has freed copy t - S; a copy arrives at any later
// moment and completes phase t / S of the stage's `full` barrier; the consumer uses the copies in order and frees them.
struct Ring {
    int S, issued = 0, used = 0;
    std::vector<int> phase, flying;  // completed phases of a stage's barrier; its copy on the way, or -1
    explicit Ring(int s) : S(s), phase(s, 0), flying(s, -1) {}
    bool can_issue() const { return issued - used < S; }
    void issue() { flying[issued++ % S] = 1; }
    void arrive(int s) { if (flying[s] >= 0) { flying[s] = -1; ++phase[s]; } }
    bool done(int s, int parity) const { return (phase[s] & 1) != parity; }  // mbarrier.test_wait.parity
    bool can_use() const { return used < issued && done(used % S, (used / S) & 1); }
    int in_flight() const { int n = 0; for (int f : flying) n += f >= 0; return n; }
};

int main() {
    std::srand(1);
    long stopped_busy = 0;
    for (int run = 0; run < 200000; ++run) {
        Ring r(1 + std::rand() % 4);
        for (int steps = std::rand() % 60; steps > 0; --steps) {  // until some wait gives up
            const int what = std::rand() % 3;
            if (what == 0 && r.can_issue()) r.issue();
            if (what == 1) r.arrive(std::rand() % r.S);
            if (what == 2 && r.can_use()) ++r.used;
        }
        stopped_busy += r.in_flight() > 0;
        bool ran_out = false;
        q3::drain_ring(r.issued, r.S, [&](int s, int parity) {
            if (s < 0 || s >= r.S) std::exit(2);
            while (!r.done(s, parity)) {  // copies arrive in any order meanwhile
                if (r.in_flight() == 0) { ran_out = true; return; }
                r.arrive(std::rand() % r.S);
            }
        });
        if (ran_out) { std::printf("waits for a copy that was never asked for\n"); return 1; }
        if (r.in_flight()) { std::printf("leaves with %d copies on their way\n", r.in_flight()); return 1; }
    }
    if (stopped_busy < 100000) { std::printf("the model hardly stops with copies on their way\n"); return 1; }
    return 0;
}
"""


def test_a_stopped_ring_is_drained(tmp_path):
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    inc = os.path.join(ROOT, "qwen3_decoder_transformer_gb300", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", inc, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
