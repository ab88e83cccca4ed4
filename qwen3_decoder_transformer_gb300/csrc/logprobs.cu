// Log probabilities of given tokens, the entropy of each row's distribution and its largest alternatives,
// in one pass over the logits.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace q3 {
namespace {

// For a row x of V logits with m = max x, s = sum_i e^(x_i - m) and t = sum_i e^(x_i - m) (x_i - m):
//   logsumexp = m + log s,  log p_i = (x_i - m) - log s,  entropy = -sum p_i log p_i = log s - t / s.
// s and t are kept with a running maximum (a larger one moves both: t' = (t + s (m - m')) f, s' = s f with
// f = e^(m - m')), per thread in fp32 over a few hundred elements, then joined over the CTA and the cluster
// in a fixed order, so the result does not depend on timing. -inf adds nothing; NaN and +inf make s NaN.
//
// Alternatives are ordered by a 64-bit key, the value's order-preserving bits above the complemented
// index: unique keys, so ties go to the lowest index, and NaN is the largest value. A threshold keeps the
// selection out of the main loop: the k-th largest of 64 group maxima over the first elements read (spread
// over the slice, so that sorted rows do not defeat it) is a lower bound of the slice's k-th largest, and
// only elements above it enter the candidate list. The list is then cut by the same rule and ranked by
// counting. A slice whose list overflows, or that holds NaN or +inf, is rescanned once per alternative.
//
// A cluster of C CTAs shares a row (C = 1 when the rows alone fill the SMs) and CTA 0 joins the parts
// through distributed shared memory: no workspace, one launch.
constexpr int LP_THREADS = 512;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_GROUPS = 64;           // groups of 8 threads whose maxima give the threshold
constexpr int LP_CAP = 2080;            // candidates of one CTA: a slice of fewer than 2048 + 14 elements fits whole
constexpr int LP_CUT = 256, LP_RANK = 128;
constexpr int LP_MAX_CLUSTER = 8;
static_assert(LP_THREADS == 8 * LP_GROUPS, "eight threads per group");

using u64 = unsigned long long;

template <typename T>
struct LpLoad;
template <>
struct LpLoad<float> {
    static constexpr int EPV = 4, U = 4;  // elements per 16-byte vector, vectors per thread and step
    static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
        x[0] = __uint_as_float(r.x);
        x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z);
        x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ uint4 fill() {
        const uint32_t f = 0xff800000u;  // -inf
        return make_uint4(f, f, f, f);
    }
};
template <>
struct LpLoad<__nv_bfloat16> {
    static constexpr int EPV = 8, U = 2;
    static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return bf16f(*p); }
    static __device__ __forceinline__ uint4 fill() {
        const uint32_t f = 0xff80ff80u;
        return make_uint4(f, f, f, f);
    }
};

__device__ __forceinline__ u64 lp_key(float v, int idx) {
    uint32_t u = __float_as_uint(v + 0.f);  // -0 and +0 are one value
    u = v != v ? 0xffffffffu : (u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u));
    return ((u64)u << 32) | (0xffffffffu - (uint32_t)idx);
}
__device__ __forceinline__ int lp_index(u64 key) { return (int)(0xffffffffu - (uint32_t)key); }
__device__ __forceinline__ float lp_value(u64 key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float((u >> 31) ? u ^ 0x80000000u : ~u);
}

// Running (m, s, t) of a set of elements; m starts at the lowest finite value, so that no difference below
// is inf - inf, and differences are cut where their weight is 0 anyway.
struct LpStat {
    float m, s, t;
};
constexpr float kLowest = -3.402823466e38f;
__device__ __forceinline__ LpStat lp_join(const LpStat& a, const LpStat& b) {
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf(a.m - m, -1e30f), db = fmaxf(b.m - m, -1e30f);
    const float fa = ex2_approx(da * kLog2e), fb = ex2_approx(db * kLog2e);
    return {m, a.s * fa + b.s * fb, (a.t + a.s * da) * fa + (b.t + b.s * db) * fb};
}

struct LpShared {
    u64 cand[LP_CAP];
    u64 cut[LP_CUT];
    u64 groups[LP_GROUPS];
    u64 top[kLogprobMaxTop];
    u64 warp_best[LP_WARPS];
    u64 tau;
    LpStat warp_stat[LP_WARPS];
    LpStat stat;
    int n_cand, n_cut;
};

// The k-th largest of the 64 group maxima of the threads' keys (0 = no element).
__device__ __forceinline__ u64 lp_threshold(u64 rep, int k, LpShared& sh) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const u64 other = __shfl_xor_sync(0xffffffffu, rep, o);
        rep = other > rep ? other : rep;
    }
    if ((threadIdx.x & 7) == 0) sh.groups[threadIdx.x >> 3] = rep;
    __syncthreads();
    if (threadIdx.x < LP_GROUPS) {
        const u64 mine = sh.groups[threadIdx.x];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < LP_GROUPS; ++j) {
            const u64 o = sh.groups[j];
            rank += (o > mine) | ((o == mine) & (j < (int)threadIdx.x));
        }
        if (rank == k - 1) sh.tau = mine;
    }
    __syncthreads();
    return sh.tau;
}

template <typename T>
__global__ void __launch_bounds__(LP_THREADS)
    token_logprobs_kernel(const T* __restrict__ logits, long long ld, int V, const int32_t* __restrict__ tokens, int k,
                          float* __restrict__ logprob, float* __restrict__ entropy, int32_t* __restrict__ top_ids,
                          float* __restrict__ top_logprobs, int C, int* err) {
    using L = LpLoad<T>;
    constexpr int EPV = L::EPV, U = L::U;
    __shared__ LpShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_i = blockIdx.x / C, rank = C > 1 ? (int)cluster_rank() : 0;
    pdl_wait();
    pdl_trigger();
    const T* row = logits + (size_t)row_i * ld;
    // the row in 16-byte vectors, with up to EPV - 1 elements before the first (CTA 0) and after the last
    // (CTA C - 1) taken one by one
    const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
    const int nv = (V - head) / EPV;
    const int v0 = (int)((long long)nv * rank / C), n = (int)((long long)nv * (rank + 1) / C) - v0;
    const uint4* vec = reinterpret_cast<const uint4*>(row + head) + v0;
    const int base = head + v0 * EPV;  // index of the slice's first vector element
    int one = -1;                      // this thread's single element, if any
    if (rank == 0 && tid < head) one = tid;
    if (rank == C - 1 && tid >= 32 && tid - 32 < V - head - nv * EPV) one = head + nv * EPV + tid - 32;
    if (tid == 0) {
        sh.n_cand = 0;
        sh.n_cut = 0;
    }
    if (tid < kLogprobMaxTop) sh.top[tid] = 0;

    const int chunks = (n + LP_THREADS - 1) / LP_THREADS;
    // chunk read at position p: the first U positions are spread from the first chunk to the last
    auto chunk_at = [&](int p) -> int {
        if (chunks <= U) return p;
        if (p < U) return (int)((long long)p * (chunks - 1) / (U - 1));
        int c = p - U;
#pragma unroll
        for (int i = 0; i < U; ++i) c += c >= (int)((long long)i * (chunks - 1) / (U - 1));
        return c;
    };
    LpStat st{kLowest, 0.f, 0.f};
    u64 tau = 0;
    float tau_v = -INFINITY;
    auto push = [&](float v, int idx) {
        const u64 key = lp_key(v, idx);
        if (key >= tau) {
            const int at = atomicAdd(&sh.n_cand, 1);
            if (at < LP_CAP) sh.cand[at] = key;
        }
    };
    auto accumulate = [&](const float* x, int cnt, float mx) {
        if (mx > st.m) {
            const float d = fmaxf(st.m - mx, -1e30f), f = ex2_approx(d * kLog2e);
            st.t = (st.t + st.s * d) * f;
            st.s *= f;
            st.m = mx;
        }
#pragma unroll
        for (int i = 0; i < EPV * U; ++i) {
            if (i >= cnt) break;
            const float d = x[i] - st.m;
            const float e = ex2_approx(d * kLog2e);
            st.s += e;
            st.t = fmaf(e, fmaxf(d, -200.f), st.t);
        }
    };
    for (int p = 0; p < chunks || p == 0; p += U) {
        uint4 raw[U];
        int at[U];  // vector of the slice, or -1
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = p + u < chunks ? chunk_at(p + u) * LP_THREADS + tid : n;
            at[u] = i < n ? i : -1;
            raw[u] = i < n ? __ldcs(vec + i) : L::fill();
        }
        float x[EPV * U];
#pragma unroll
        for (int u = 0; u < U; ++u) L::unpack(raw[u], x + u * EPV);
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < EPV * U; ++i) mx = fmaxf(mx, x[i]);
        if (k > 0) {
            if (p == 0) {  // threshold from the first elements read
                u64 rep = 0;
#pragma unroll
                for (int i = 0; i < EPV * U; ++i)
                    if (at[i / EPV] >= 0 && x[i] == mx) {
                        const u64 key = lp_key(x[i], base + at[i / EPV] * EPV + i % EPV);
                        rep = key > rep ? key : rep;
                    }
                __syncthreads();  // the list's counters are set
                tau = lp_threshold(rep, k, sh);
                tau_v = tau == 0 ? -INFINITY : lp_value(tau);
            }
            if (mx >= tau_v) {
#pragma unroll
                for (int i = 0; i < EPV * U; ++i)
                    if (x[i] >= tau_v && at[i / EPV] >= 0) push(x[i], base + at[i / EPV] * EPV + i % EPV);
            }
        }
        accumulate(x, EPV * U, mx);
    }
    if (one >= 0) {
        const float v = L::one(row + one);
        accumulate(&v, 1, v);
        if (k > 0 && v >= tau_v) push(v, one);
    }

    // join the threads' statistics
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const LpStat b{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                       __shfl_xor_sync(0xffffffffu, st.t, o)};
        st = lp_join(st, b);
    }
    if (lane == 0) sh.warp_stat[warp] = st;
    __syncthreads();
    if (warp == 0) {
        st = lane < LP_WARPS ? sh.warp_stat[lane] : LpStat{kLowest, 0.f, 0.f};
#pragma unroll
        for (int o = LP_WARPS / 2; o > 0; o >>= 1) {
            const LpStat b{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                           __shfl_xor_sync(0xffffffffu, st.t, o)};
            st = lp_join(st, b);
        }
        if (lane == 0) sh.stat = st;
    }
    __syncthreads();

    // this CTA's k largest, sorted, into sh.top (0 where the slice has fewer elements)
    if (k > 0) {
        const int nc = sh.n_cand;
        bool rescan = nc > LP_CAP || sh.stat.s != sh.stat.s;
        if (!rescan) {
            const u64* list = sh.cand;
            int nl = nc;
            if (nc > LP_RANK) {
                u64 rep = 0;
                for (int i = tid; i < nc; i += LP_THREADS) rep = sh.cand[i] > rep ? sh.cand[i] : rep;
                const u64 cut = lp_threshold(rep, k, sh);
                for (int i = tid; i < nc; i += LP_THREADS)
                    if (sh.cand[i] >= cut) {
                        const int at = atomicAdd(&sh.n_cut, 1);
                        if (at < LP_CUT) sh.cut[at] = sh.cand[i];
                    }
                __syncthreads();
                list = sh.cut;
                nl = sh.n_cut;
                rescan = nl > LP_CUT;
            }
            if (!rescan && tid < nl) {
                const u64 mine = list[tid];
                int r = 0;
                for (int j = 0; j < nl; ++j) r += list[j] > mine;
                if (r < k) sh.top[r] = mine;
            }
        }
        if (rescan) {  // one scan of the slice per alternative: the largest key below the previous one
            u64 prev = ~0ull;
            for (int r = 0; r < k; ++r) {
                u64 best = 0;
                auto take = [&](float v, int idx) {
                    const u64 key = lp_key(v, idx);
                    if (key < prev && key > best) best = key;
                };
                for (int i = tid; i < n; i += LP_THREADS) {
                    float x[EPV];
                    L::unpack(__ldg(vec + i), x);
#pragma unroll
                    for (int e = 0; e < EPV; ++e) take(x[e], base + i * EPV + e);
                }
                if (one >= 0) take(L::one(row + one), one);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const u64 other = __shfl_xor_sync(0xffffffffu, best, o);
                    best = other > best ? other : best;
                }
                __syncthreads();
                if (lane == 0) sh.warp_best[warp] = best;
                __syncthreads();
                best = sh.warp_best[0];
#pragma unroll
                for (int w = 1; w < LP_WARPS; ++w) best = sh.warp_best[w] > best ? sh.warp_best[w] : best;
                if (tid == 0) sh.top[r] = best;
                prev = best;
                if (best == 0) break;
            }
        }
        __syncthreads();
    }

    if (C > 1) {  // CTA 0 joins the cluster's parts
        cluster_sync();
        if (rank == 0) {
            if (k > 0) {
                if (tid < C * kLogprobMaxTop)
                    sh.cand[tid] = ld_cluster_u64(cluster_addr(&sh.top[tid % kLogprobMaxTop], tid / kLogprobMaxTop));
                __syncthreads();
                if (tid < C * kLogprobMaxTop) {
                    const u64 mine = sh.cand[tid];
                    int r = 0;
                    for (int j = 0; j < C * kLogprobMaxTop; ++j) r += sh.cand[j] > mine;
                    if (mine && r < k) sh.cut[r] = mine;
                }
            }
            if (tid == 0) {
                LpStat a = sh.stat;
                for (int c = 1; c < C; ++c) {
                    const uint32_t ad = cluster_addr(&sh.stat, c);
                    a = lp_join(a, LpStat{ld_cluster_f32(ad), ld_cluster_f32(ad + 4), ld_cluster_f32(ad + 8)});
                }
                sh.warp_stat[0] = a;
            }
        }
        cluster_sync();  // the other CTAs' shared memory stays until it has been read
        if (rank != 0) return;
    }
    const LpStat total = C > 1 ? sh.warp_stat[0] : sh.stat;
    const u64* top = C > 1 ? sh.cut : sh.top;
    // no distribution: NaN or +inf in the row (s is NaN), or nothing above -inf (s is 0)
    const float log_s = total.s > 0.f ? logf(total.s) : __uint_as_float(0x7fc00000u);
    if (tid == 0) {
        if (logprob) {
            const int tok = tokens[row_i];
            const bool in = tok >= 0 && tok < V;
            logprob[row_i] = in ? (L::one(row + tok) - total.m) - log_s : __uint_as_float(0x7fc00000u);
            if (!in && err) atomicOr(err, ERR_TOKEN);
        }
        if (entropy) entropy[row_i] = log_s - total.t / total.s;
    }
    if (tid < k) {
        const u64 key = top[tid];
        if (top_ids) top_ids[(size_t)row_i * k + tid] = lp_index(key);
        if (top_logprobs) top_logprobs[(size_t)row_i * k + tid] = (lp_value(key) - total.m) - log_s;
    }
}

// CTAs per row: as many as two CTAs on every SM take, while a slice keeps at least 4096 elements.
int lp_cluster(int M, int V) {
    int c = 1;
    while (c < LP_MAX_CLUSTER && (long long)M * c * 2 <= 2 * device_sm_count() && V / (2 * c) >= 4096) c *= 2;
    return c;
}

}  // namespace

cudaError_t token_logprobs_launch(const void* logits, int bf16, long long ld, int M, int V, const int32_t* tokens,
                                  int top_k, float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs,
                                  int* err, cudaStream_t st) {
    if (M <= 0) return cudaSuccess;
    const int C = lp_cluster(M, V);
    const dim3 grid((unsigned)M * C), block(LP_THREADS);
    if (bf16)
        return launch_pdl_cluster(token_logprobs_kernel<__nv_bfloat16>, grid, block, C, 0, st,
                                  static_cast<const __nv_bfloat16*>(logits), ld, V, tokens, top_k, logprob, entropy,
                                  top_ids, top_logprobs, C, err);
    return launch_pdl_cluster(token_logprobs_kernel<float>, grid, block, C, 0, st, static_cast<const float*>(logits), ld,
                              V, tokens, top_k, logprob, entropy, top_ids, top_logprobs, C, err);
}

}  // namespace q3
