// Bookkeeping of rings of asynchronous copies, apart from the kernels so that it runs on the host too.
#pragma once

#ifdef __CUDACC__
#define Q3_RING_FN __device__ __forceinline__
#else
#define Q3_RING_FN inline
#endif

namespace q3 {

// wait(stage, parity) for every copy that may still be on its way when a ring's producer stops after `issued` copies.
// Copy t goes to stage t % stages, whose barrier it takes through phase t / stages, and is issued only after the stage's
// previous copy has arrived and been used: so no more than the last `stages` are outstanding, one a stage, and as
// nothing is issued behind them the parities cannot alias.
template <typename Wait>
Q3_RING_FN void drain_ring(int issued, int stages, Wait wait) {
    for (int t = issued > stages ? issued - stages : 0; t < issued; ++t) wait(t % stages, (t / stages) & 1);
}

}  // namespace q3
