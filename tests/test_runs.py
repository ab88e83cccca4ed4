"""Where a (sequence, kv head) of the paged decode attention ends that is cut between CTAs (csrc/runs.h), on the CPU: a model of the
list of units, its cut into runs, and CTAs that work through theirs or give up at any unit. No GPU fault or hang is made anywhere."""
import os
import subprocess

from tests.conftest import ROOT

MODEL = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "runs.h"

int main() {
    std::srand(1);
    auto rnd = [](int n) { return std::rand() % n; };
    long open = 0, given_up = 0;
    for (int round = 0; round < 40000; ++round) {
        // segments of a few units or many, and as many runs as there are places, but no empty one
        std::vector<int> first(1, 0);  // of each segment, and behind the last
        const int segments = 1 + rnd(12), size = 1 + rnd(60);
        for (int s = 0; s < segments; ++s) first.push_back(first.back() + 1 + rnd(size));
        const int units = first.back(), places = 1 + rnd(40);
        const int runs = std::min(places, units), len = units / runs, more = units - len * runs;
        auto begin = [&](int r) { return r * len + std::min(r, more); };
        auto segment = [&](int unit) { return int(std::upper_bound(first.begin(), first.end(), unit) - first.begin()) - 1; };
        for (int r = 0; r < runs; ++r) {
            const int end = begin(r + 1), stops = begin(r) + rnd(end - begin(r) + 1);  // stops == end: worked through
            const bool gave_up = stops < end;
            // the cursor: the segment of the unit last used (or waited for), its units behind that
            const int at = gave_up ? stops : end - 1, seg = segment(at), left = first[seg + 1] - at - (gave_up ? 0 : 1);
            if (left == 0) continue;  // ends with the run
            const q3::RunEnd got = q3::run_of_end(end, left, len, more, gave_up, [](int n, int d) { return n / d; });
            if (gave_up) {
                ++given_up;
                if (got.run >= runs) { std::printf("a run past the last one: %d of %d\n", got.run, runs); return 1; }
                continue;
            }
            ++open;
            int want = r;
            while (begin(want + 1) < first[seg + 1]) ++want;
            if (got.run != want || got.with_run != (begin(want + 1) == first[seg + 1])) {
                std::printf("run %d (%d), not %d\n", got.run, got.with_run, want);
                return 1;
            }
        }
    }
    return open > 50000 && given_up > 50000 ? 0 : 2;
}
"""


def test_where_a_cut_segment_ends(tmp_path):
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    inc = os.path.join(ROOT, "qwen3_decoder_transformer_gb300", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", inc, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
