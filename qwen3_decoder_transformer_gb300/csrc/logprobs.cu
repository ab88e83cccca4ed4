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
// over the slice, both ends included, so that sorted rows do not defeat it) is a lower bound of the slice's k-th
// largest, and only elements above it enter the candidate list; the bound is raised from the list twice on
// the way. The list is then cut by the same rule and ranked by counting. A slice whose list overflows, or
// that holds NaN or +inf, is rescanned once per alternative.
//
// A cluster of C CTAs shares a row (C = 1 when there are rows enough) and CTA 0 joins the parts
// through distributed shared memory: no workspace, one launch.
// What bounds it. Many rows: HBM, 2048 x 151,936 fp32 with one alternative 195 us, 6.38 TB/s (94% of the measured copy);
// bf16 has twice the elements a byte and is bound by their arithmetic, 121 us (5.1 TB/s), and with 32 alternatives by
// the selection, 176. Few rows: the chain of a CTA, 7.1 us for one row of 151,936 with 20 alternatives (3.4 without:
// launch, first loads, join), 11.6 for 64 rows with five (7.7 without): at eight warps a scheduler each instruction that
// every thread adds costs eight issue slots, and a threshold, a select and a join are some hundred instructions each.
constexpr int LP_GROUPS = 64;           // groups of threads whose maxima give the threshold
constexpr int LP_CAP = 2080;            // candidates of one CTA: a slice of fewer than 2048 + 14 elements fits whole
constexpr int LP_CUT = 256, LP_RANK = 128, kFill = 64;
constexpr int LP_MAX_CLUSTER = 16;  // beyond the portable size

using u64 = unsigned long long;

template <typename T>
struct LpLoad;
template <>
struct LpLoad<float> {
    static constexpr int EPV = 4;  // elements of a 16-byte vector
    static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
        x[0] = __uint_as_float(r.x);
        x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z);
        x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ float largest(const uint4& r) {
        return fmax3(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), __uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ uint4 fill() {
        const uint32_t f = 0xff800000u;  // -inf
        return make_uint4(f, f, f, f);
    }
};
template <>
struct LpLoad<__nv_bfloat16> {
    static constexpr int EPV = 8;
    static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ float largest(const uint4& r) {
        const uint32_t m = as_u32(__hmax2(__hmax2(as_bf2(r.x), as_bf2(r.y)), __hmax2(as_bf2(r.z), as_bf2(r.w))));
        return fmaxf(bf16_lo(m), bf16_hi(m));
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
// Join the threads of a warp: the maximum first, then everyone's sums at its scale.
__device__ __forceinline__ LpStat lp_warp_join(const LpStat& a) {
    const int bits = __float_as_int(a.m), top = __reduce_max_sync(0xffffffffu, bits ^ ((bits >> 31) & 0x7fffffff));
    const float m = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
    const float d = fmaxf(a.m - m, -1e30f), f = ex2_approx(d * kLog2e);
    float s = a.s * f, t = (a.t + a.s * d) * f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    return {m, s, t};
}

struct LpShared {
    u64 cand[LP_CAP];
    u64 gather[LP_MAX_CLUSTER * kLogprobMaxTop];  // CTA 0: the cluster's largest, and statistics
    LpStat gather_stat[LP_MAX_CLUSTER];
    u64 cut[LP_CUT];
    u64 groups[LP_GROUPS];
    u64 top[kLogprobMaxTop], joined[kLogprobMaxTop];
    u64 warp_best[16];
    u64 tau;
    LpStat warp_stat[16];
    LpStat stat;
    int n_cand, n_cut;
};

// The k-th largest of the 64 group maxima of the threads' keys (0 = no element). A group's threads share the count of
// its key's rank.
template <int THREADS>
__device__ __forceinline__ u64 lp_threshold(u64 rep, int k, LpShared& sh) {
    constexpr int P = THREADS / LP_GROUPS;  // threads of a group
#pragma unroll
    for (int o = 1; o < P; o <<= 1) {
        const u64 other = __shfl_xor_sync(0xffffffffu, rep, o);
        rep = other > rep ? other : rep;
    }
    const int grp = threadIdx.x / P, part = threadIdx.x % P;
    if (part == 0) sh.groups[grp] = rep;
    __syncthreads();
    int rank = 0;
#pragma unroll
    for (int i = 0; i < LP_GROUPS / P; ++i) {
        const int j = i * P + part;
        const u64 o = sh.groups[j];
        rank += (o > rep) | ((o == rep) & (j < grp));
    }
#pragma unroll
    for (int o = 1; o < P; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (part == 0 && rank == k - 1) sh.tau = rep;
    __syncthreads();
    return sh.tau;
}

// out[r] = the r-th largest of list[0 .. n), r < k; the list's keys are distinct, 0 stands for no element. P threads
// share the count of one key.
template <int P, int LP_THREADS>
__device__ __forceinline__ void lp_rank(const u64* list, int n, int k, u64* out) {
    for (int i0 = 0; i0 < n; i0 += LP_THREADS / P) {
        const int i = i0 + threadIdx.x / P, part = threadIdx.x % P;
        const u64 mine = i < n ? list[i] : 0;
        int r = 0;
#pragma unroll 4
        for (int j = part; j < n; j += P) r += list[j] > mine;
#pragma unroll
        for (int o = 1; o < P; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        if (part == 0 && mine && r < k) out[r] = mine;
    }
}

// The k largest of list[0 .. n) into out, sorted; false when the cut list overflows. n is the same in every thread;
// sh.n_cut is 0 on entry.
template <int LP_THREADS>
__device__ __forceinline__ bool lp_select(const u64* list, int n, int k, LpShared& sh, u64* out) {
    if (n > LP_RANK) {  // cut the list first
        u64 rep = 0;
        for (int i = threadIdx.x; i < n; i += LP_THREADS) rep = list[i] > rep ? list[i] : rep;
        const u64 cut = lp_threshold<LP_THREADS>(rep, k, sh);
        for (int i = threadIdx.x; i < n; i += LP_THREADS)
            if (list[i] >= cut && list[i]) {
                const int at = atomicAdd(&sh.n_cut, 1);
                if (at < LP_CUT) sh.cut[at] = list[i];
            }
        __syncthreads();
        list = sh.cut;
        n = sh.n_cut;
        if (n > LP_CUT) return false;
    }
    if (n <= LP_THREADS / 8)
        lp_rank<8, LP_THREADS>(list, n, k, out);
    else if (n <= LP_THREADS / 4)
        lp_rank<4, LP_THREADS>(list, n, k, out);
    else
        lp_rank<2, LP_THREADS>(list, n, k, out);
    return true;
}

template <typename T, int LP_THREADS>
__global__ void __launch_bounds__(LP_THREADS, 1024 / LP_THREADS)
    token_logprobs_kernel(const T* __restrict__ logits, long long ld, int V, const int32_t* __restrict__ tokens, int k,
                          float* __restrict__ logprob, float* __restrict__ entropy, int32_t* __restrict__ top_ids,
                          float* __restrict__ top_logprobs, int log_c, int* err) {
    using L = LpLoad<T>;
    constexpr int LP_WARPS = LP_THREADS / 32;
    constexpr int EPV = L::EPV, U = 4;  // U vectors a thread and step
    __shared__ LpShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = 1 << log_c, row_i = blockIdx.x >> log_c, rank = C > 1 ? (int)cluster_rank() : 0;
    if (C > 1) cluster_arrive();  // every CTA has started, by the time the parts are sent to CTA 0
    pdl_wait();
    pdl_trigger();
    const T* row = logits + (size_t)row_i * ld;
    // the row in 16-byte vectors, with up to EPV - 1 elements before the first (CTA 0) and after the last
    // (CTA C - 1) taken one by one
    const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
    const int nv = (V - head) / EPV;
    const int v0 = (int)((long long)nv * rank >> log_c), n = (int)((long long)nv * (rank + 1) >> log_c) - v0;
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

    // U streams: stream u < U - 1 runs forward from vector u * span, the last one backward from the slice's end, so that
    // the first step's elements are spread over the slice and include both ends
    const int steps = max(1, (n + U * LP_THREADS - 1) / (U * LP_THREADS)), span = steps * LP_THREADS;
    auto vector_at = [&](int step, int u) -> int {  // this thread's vector of stream u, or -1
        const int off = step * LP_THREADS + tid;
        if (u < U - 1) return u * span + off < n ? u * span + off : -1;
        return n - 1 - off >= (U - 1) * span ? n - 1 - off : -1;
    };
    auto index_of = [&](int step, int bit) -> int {  // index in the row of element bit % EPV of vector bit / EPV, or -1
        const int v = vector_at(step, bit / EPV);
        return v >= 0 ? base + v * EPV + bit % EPV : -1;
    };
    float m = kLowest;
    u64 tau = 0;
    float tau_v = kLowest;  // -inf stays out of the list: a row may hold little else
    // Elements equal to the threshold and behind it are below it: a thread whose vector of stream 0, its foremost, lies
    // behind vector tau_at has none to look at when its largest is the threshold's value. (A row masked with the type's
    // lowest value is all ties: 64 rows of 151,936, five left, five alternatives, 19.5 us against 36.4 with a look at each.)
    int tau_at = 0x7fffffff;
    auto set_tau = [&](u64 t) {
        tau = t;
        if (t == 0) return;
        tau_v = fmaxf(lp_value(t), kLowest);
        tau_at = lp_value(t) >= kLowest ? (lp_index(t) - base) / EPV : 0x7fffffff;
    };
    auto push = [&](float v, int idx) {
        const u64 key = lp_key(v, idx);
        if (key >= tau) {
            const int at = atomicAdd(&sh.n_cand, 1);
            if (at < LP_CAP) sh.cand[at] = key;
        }
    };
    float2 s2 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);  // two running sums a thread (paired fp32 arithmetic)
    auto raise = [&](float mx) {  // move the sums to a larger maximum
        if (mx > m) {
            const float d = fmaxf(m - mx, -1e30f), f = ex2_approx(d * kLog2e);
            const float2 d2 = make_float2(d, d), f2 = make_float2(f, f);
            t2 = mul2(fma2(s2, d2, t2), f2);
            s2 = mul2(s2, f2);
            m = mx;
        }
    };
    auto add_pair = [&](float a, float b) {
        const float2 d = add2(make_float2(a, b), make_float2(-m, -m));
        const float2 y = mul2(d, make_float2(kLog2e, kLog2e));
        const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        s2 = add2(s2, e);
        t2 = fma2(e, make_float2(fmaxf(d.x, -200.f), fmaxf(d.y, -200.f)), t2);
    };
    // the loads of one step ahead are in flight while a step is worked on
    uint4 nxt[U];
    auto load = [&](int step) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = vector_at(step, u);
            nxt[u] = v >= 0 ? __ldcs(vec + v) : L::fill();
        }
    };
    // the given token and its logit, two loads in turn, are on their way with the first vectors
    const bool scores = logprob && rank == 0 && tid == 0;
    const int tok = scores ? tokens[row_i] : -1;
    load(0);
    const float tok_logit = tok >= 0 && tok < V ? L::one(row + tok) : 0.f;
    for (int step = 0; step < steps; ++step) {
        uint4 raw[U];
        float vmax[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = nxt[u];
        if (step + 1 < steps) load(step + 1);
#pragma unroll
        for (int u = 0; u < U; ++u) vmax[u] = L::largest(raw[u]);
        const float mx = fmax3(fmaxf(vmax[0], vmax[1]), vmax[2], vmax[3]);
        // bit u * EPV + e: element e of vector u passes the test
        auto which = [&](auto test) -> uint32_t {
            uint32_t bits = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[EPV];
                L::unpack(raw[u], x);
#pragma unroll
                for (int e = 0; e < EPV; ++e)
                    if (test(x[e])) bits |= 1u << (u * EPV + e);
            }
            return bits;
        };
        if (k > 0) {
            if (step == 0) {  // threshold from the first elements read
                // the thread's largest, at the last index of the first vector that holds it: its own key is no smaller
                const int at = vmax[0] == mx ? 0 : vmax[1] == mx ? 1 : vmax[2] == mx ? 2 : 3;
                const int idx = mx == mx ? index_of(step, at * EPV + EPV - 1) : -1;
                const u64 rep = idx >= 0 ? lp_key(mx, idx) : 0;
                __syncthreads();  // the list's counters are set
                set_tau(lp_threshold<LP_THREADS>(rep, k, sh));
            } else if ((step == 3 || step == 8) && steps > 2 * step) {
                // raise it from the list so far, while the list is far from full and most of the slice is still to come (2048
                // fp32 rows of 151,936, 32 alternatives: never 1,964 us, since lists overflow; at step 3 alone 239; at 3 and 8
                // 216; at 2 and 5 219; at 4 and 16 211. 64 rows, five: 10.9, 11.1, 11.3, 12.3, 11.1)
                __syncthreads();
                const int nc = min(sh.n_cand, LP_CAP);
                u64 rep = 0;
                for (int i = tid; i < nc; i += LP_THREADS) rep = sh.cand[i] > rep ? sh.cand[i] : rep;
                const u64 t = lp_threshold<LP_THREADS>(rep, k, sh);
                if (t > tau) set_tau(t);
            }
            if (mx >= tau_v && (mx > tau_v || step * LP_THREADS + tid <= tau_at)) {  // a few elements of the row come here: read again unless it is the thread's largest
                uint32_t hit = which([&](float v) { return v >= tau_v; });
                if (__popc(hit) == 1) {
                    const int idx = index_of(step, __ffs(hit) - 1);
                    if (idx >= 0) push(mx, idx);
                } else {
                    for (; hit; hit &= hit - 1) {
                        const int idx = index_of(step, __ffs(hit) - 1);
                        if (idx >= 0) push(L::one(row + idx), idx);
                    }
                }
            }
        }
        raise(mx);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[EPV];
            L::unpack(raw[u], x);
#pragma unroll
            for (int e = 0; e < EPV; e += 2) add_pair(x[e], x[e + 1]);
        }
    }
    if (one >= 0) {
        const float v = L::one(row + one);
        raise(v);
        add_pair(v, -INFINITY);
        if (k > 0 && v >= tau_v) push(v, one);
    }

    // join the threads' statistics
    LpStat st = lp_warp_join({m, s2.x + s2.y, t2.x + t2.y});
    if (lane == 0) sh.warp_stat[warp] = st;
    __syncthreads();
    if (warp == 0) {
        st = lp_warp_join(lane < LP_WARPS ? sh.warp_stat[lane] : LpStat{kLowest, 0.f, 0.f});
        if (lane == 0) sh.stat = st;
    }
    __syncthreads();

    // this CTA's k largest, sorted, into sh.top (0 where the slice has fewer elements)
    if (k > 0) {
        const bool no_sum = sh.stat.s != sh.stat.s;
        // fewer than k elements above -inf (a mask): the lowest indices of the others fill the list
        const int first = rank == 0 ? 0 : base, end = rank == C - 1 ? V : base + n * EPV;
        int nc = sh.n_cand;
        for (int at = first; !no_sum && nc < k && at < end; at += kFill) {
            __syncthreads();  // every thread has read the count
            if (tid < kFill && at + tid < end && L::one(row + at + tid) == -INFINITY) {
                const int slot = atomicAdd(&sh.n_cand, 1);
                if (slot < LP_CAP) sh.cand[slot] = lp_key(-INFINITY, at + tid);
            }
            __syncthreads();
            nc = sh.n_cand;
        }
        bool rescan = nc > LP_CAP || no_sum;
        if (!rescan) rescan = !lp_select<LP_THREADS>(sh.cand, nc, k, sh, sh.top);
        if (rescan) {  // one scan of the slice per alternative: the largest key below the previous one
            u64 prev = 0;
            for (int r = 0; r < k; ++r) {
                u64 best = 0;
                auto take = [&](float v, int idx) {
                    const u64 key = lp_key(v, idx);  // (a NaN at index 0 has the largest key there is)
                    if ((r == 0 || key < prev) && key > best) best = key;
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

    if (C > 1) {  // every CTA sends its part to CTA 0, which joins them
        cluster_wait();
        if (tid < k) st_cluster_u64(cluster_addr(&sh.gather[rank * k + tid], 0), sh.top[tid]);
        if (tid == LP_THREADS - 1) {
            const uint32_t to = cluster_addr(&sh.gather_stat[rank], 0);
            st_cluster_f32(to, sh.stat.m);
            st_cluster_f32(to + 4, sh.stat.s);
            st_cluster_f32(to + 8, sh.stat.t);
        }
        if (tid == 0) sh.n_cut = 0;
        cluster_sync();
        if (rank != 0) return;
        if (warp == LP_WARPS - 1) {
            st = lp_warp_join(lane < C ? sh.gather_stat[lane] : LpStat{kLowest, 0.f, 0.f});
            if (lane == 0) sh.stat = st;
        }
        // (a cut list that overflows leaves the whole list, at most 512 keys, to be ranked)
        if (k > 0 && !lp_select<LP_THREADS>(sh.gather, C * k, k, sh, sh.joined))
            lp_rank<1, LP_THREADS>(sh.gather, C * k, k, sh.joined);
        __syncthreads();
    }
    const LpStat total = sh.stat;
    const u64* top = C > 1 ? sh.joined : sh.top;
    // no distribution: NaN or +inf in the row (s is NaN), or nothing above -inf (s is 0)
    const float log_s = total.s > 0.f ? logf(total.s) : __uint_as_float(0x7fc00000u);
    if (tid == 0) {
        if (logprob) {
            const bool in = tok >= 0 && tok < V;
            logprob[row_i] = in ? (tok_logit - total.m) - log_s : __uint_as_float(0x7fc00000u);
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

// CTAs per row: as many as two on every SM take, while a slice keeps at least 4096 elements; clusters of eight and
// sixteen only while they are few, since they wait for room in one part of the GPU (151,936 fp32 logits, five
// alternatives: 16 rows by 4 CTAs 8.2 us, by 8 8.6, by 16 11.4; 4 rows 7.6, 6.6 and 6.1).
int lp_cluster(int M, int V) {
    int c = 1;
    while (c < LP_MAX_CLUSTER && (long long)M * c * 2 <= (c * 2 >= 8 ? 64 : 2 * device_sm_count()) && V / (2 * c) >= 4096)
        c *= 2;
    return c;
}

}  // namespace

cudaError_t token_logprobs_launch(const void* logits, int bf16, long long ld, int M, int V, const int32_t* tokens,
                                  int top_k, float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs,
                                  int* err, cudaStream_t st) {
    if (M <= 0) return cudaSuccess;
    // Many rows: CTAs of 256 threads, four an SM, so that one row's selection runs beside the others' loads (2048
    // rows of 151,936 bf16 logits, one alternative 121 us against 133 with 512 threads, 32 alternatives 176
    // against 204; fp32 200 either way). Few rows: 512 threads, for a row's shorter chain (333 bf16 rows of 32,003, 32
    // alternatives 15.2 against 20.0, one row 7.1 against 8.6).
    // Rows of 151,936 about the border, 256 against 512 threads, one and 32 alternatives: bf16 304 rows 22.5 / 20.7 and 35.7 / 33.2,
    // 608 39.2 / 41.2 and 57.4 / 63.4, 1216 72.5 / 78.1 and 106 / 121; fp32 304 35.0 / 32.7 and 42.2 / 38.2, 900 94.3 / 90.2
    // and 110 / 104, 1216 115 / 120 and 128 / 138, 1500 148 / 147 and 160 / 169: past 1216 no case loses more than 1%.
    const int threads = M >= 8 * device_sm_count() ? 256 : 512;
    const int C = lp_cluster(M, V);
    int log_c = 0;
    while (1 << log_c < C) ++log_c;
    const dim3 grid((unsigned)M * C), block(threads);
    auto launch = [&](auto kernel, auto x) {
        return launch_pdl_cluster(kernel, grid, block, C, 0, st, x, ld, V, tokens, top_k, logprob, entropy, top_ids,
                                  top_logprobs, log_c, err);
    };
    if (bf16) {
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(logits);
        return threads == 512 ? launch(token_logprobs_kernel<__nv_bfloat16, 512>, x) : launch(token_logprobs_kernel<__nv_bfloat16, 256>, x);
    }
    const float* x = static_cast<const float*>(logits);
    return threads == 512 ? launch(token_logprobs_kernel<float, 512>, x) : launch(token_logprobs_kernel<float, 256>, x);
}

// Clusters of sixteen CTAs are beyond the portable size.
cudaError_t token_logprobs_prepare() {
    const void* fns[] = {(const void*)token_logprobs_kernel<float, 512>, (const void*)token_logprobs_kernel<float, 256>,
                         (const void*)token_logprobs_kernel<__nv_bfloat16, 512>,
                         (const void*)token_logprobs_kernel<__nv_bfloat16, 256>};
    for (const void* f : fns) {
        cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q3
