// A list of units cut into equal runs, apart from the kernels so that it runs on the host too.
#pragma once

#ifdef __CUDACC__
#define Q3_RUN_FN __device__ __forceinline__
#else
#define Q3_RUN_FN inline
#endif

namespace q3 {

// Where a segment ends that goes on behind a run: the run that holds its last unit (-1: not known), and whether the segment
// ends with that run. Run r holds len units, the first `more` runs one more. run_end: the unit behind the run that the
// segment leaves, left: the segment's units from there on. A run that was given up before its end knows neither: its
// `left` counts from the unit at which it stopped, and what it adds up to may lie past the last run.
// div(n, d): n / d rounded down.
struct RunEnd {
    int run;
    bool with_run;
};
template <typename Div>
Q3_RUN_FN RunEnd run_of_end(int run_end, int left, int len, int more, bool gave_up, Div div) {
    if (gave_up) return {-1, false};
    const int end = run_end + left, longer = more * (len + 1);  // units of the longer runs
    const int run = end <= longer ? div(end - 1, len + 1) : more + div(end - 1 - longer, len);
    return {run, (run + 1) * len + (run + 1 < more ? run + 1 : more) == end};
}

}  // namespace q3
