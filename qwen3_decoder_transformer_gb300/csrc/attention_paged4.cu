// Decode attention over the paged KV cache held in 4 bits (layout: paged4.cuh).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged4.cuh"
#include "rings.h"
#include "runs.h"

namespace q3 {
namespace {

// One query per (sequence b, query head) over the slots 0 .. len0[b] of its sequence, each sequence at its own length:
//   x_i = q . k_i log2(e) / sqrt(dh),  p_i = 2^(x_i - m),  O = sum_i p_i v_i / sum_i p_i.
// K and V stay in 4 bits up to the tensor cores. With k_id = min_ig + scale_ig code_id (g: the group of 64 dims),
//   q . k_i = sum_g scale_ig (sum_{d in g} q_d code_id) + min_ig (sum_{d in g} q_d)
//   sum_i p_i v_id = sum_i (p_i scale_ig) code_id + sum_i p_i min_ig
// so a code is only turned into a 16-bit operand, and scales are applied to scores and probabilities.
//   Codes of K and V become fp16 by a mask alone: a nibble in the lowest bits of an fp16 word is the subnormal code * 2^-24, the
//   next nibble code * 2^-20, exact on the tensor cores (K: its query value is divided by 16; V: output rows of its own).
//   q is scaled by a power of two for each head so that its fp16 form is exact (its largest value lies in [2^10, 2^11)). V's
//   weights p * scale are rounded to fp16, off by 2^-11 of themselves at most: a power of two for each head keeps the largest
//   weight of the run so far in [2^13, 2^15], so what falls below fp16's normal range is less than 2^-25 of that. p itself
//   takes 2^60 of it at most, as its sums have to stay in fp32's range; where scales below 2^-47 need more, the weights of
//   each step are lifted by a power of two of their own, up to 2^86, and the sums with them (without it, scales below 2^-85
//   left nothing of the codes).
//   (bf16 weights, with codes as 128 + code and the offset taken off again, left 0.5-1.2% of error on long sequences against
//   0.2%: a rounding of 2^-8 multiplies codes of one sign, and the tensor cores cut their sums off. e4m3 operands would halve
//   the conversions, but the warp-level fp8 product takes several times the fp16 one's cycles on this chip.)
//
// Work: the units of 64 keys of all (sequence, kv head) pairs in one list, cut into as many equal runs as there are warps.
// A warp works through its run alone: its first lanes keep a ring of two units full with untiled bulk copies, and warp-level
// mma (m16n8k16; the heads of a group are far below a tcgen05 tile) takes 16 keys by the heads: S^T = K q^T, then
// O^T += V^T P^T with P^T moved from accumulator to operand layout by movmatrix. The sums are rescaled only when a weight grows
// out of its range. A (sequence, kv head) within one run is written out at once. Of one that is cut, each warp leaves a
// piece (sums of weighted values, reference of the weights, sum of weights); pieces of one CTA are joined in shared memory, the others in the workspace by
// attn_paged4_join_kernel, in the order of their keys: the result does not depend on timing.
//
// What bounds it: many keys, HBM (16 sequences of up to 32,768 keys, 32 / 8 heads of 128: 86.5 us, 6.0 TB/s, of which some 8 us are
// start and end: in the loop 6.6 TB/s of a copy's 6.8), with the issue slots half full. Few keys: the chain of one
// unit. 1 sequence of 4096: 9.4 us; counting the lengths 0.6, finding the run 0.5, the query 1, one unit 2.2, the
// pieces 1.2, and the rest two launches and the records' way through the workspace.
// Split: one CTA of 12 warps an SM, as many rings as shared memory holds, joins the pieces of 12 runs before they leave the SM (16 @
// 32,768 two CTAs of six 90.3 us, one of twelve 85.7, when it was changed; 64 @ 4096, 16 / 8 heads, 45.6 and 44.9).
constexpr int P4_STEP = 64, P4_TILES = P4_STEP / 16;  // keys that a warp takes at once
constexpr int P4_WARPS = 12, P4_THREADS = 32 * P4_WARPS, P4_CTAS = 1, P4_MAX_G = 8;
constexpr int P4_STRIPS = P4_THREADS;  // strips of sequences whose units are counted at the start
template <int DH>
struct P4Layout {
    static constexpr int NG = DH / kP4Group;
    static constexpr int HALF = P4_STEP * p4_token_bytes(DH);  // bytes of K (or V) of a step
    static constexpr int SLOT = 2 * HALF;
    static constexpr int NS = 2 * 128 / DH;  // slots of a ring
    static constexpr int RING = NS * SLOT;
    static constexpr int PITCH = DH + 4;  // floats of a head's piece: sums; reference, adjustment, scale of scores, sum of weights
    static constexpr int SMEM = P4_WARPS * RING;
    static_assert(P4_MAX_G * PITCH * 4 <= RING, "a piece fits a ring");
    static_assert(P4_CTAS * (SMEM + 4608) <= 227 * 1024, "shared memory");
};

// A (sequence, kv head) that begins, but does not end, in a CTA's runs: its number (-1: none), the warp whose run holds its
// beginning, the one whose run holds its end, and whether the end's record is that run's first piece (0) or the last (1).
struct P4Desc {
    int seg, first, last, last_slot, team;  // team: warps of a CTA that worked
};

struct P4Args {
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    Paged4 cache;
    const int* len0;
    int B, Hq, Hkv, G, cap;  // cap: slots that the page table reaches
    P4Desc* desc;            // [CTAs]
    float* recs;             // [warps][2][G][PITCH]: of the piece at the beginning, and of the piece at the end of a run
    int* err;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// (not volatile: the compiler may order the products of a unit as it likes)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {  // d = a b
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Keys that sequence b's query sees.
__device__ __forceinline__ int p4_keys(const P4Args& a, int b) {
    const int n = __ldg(a.len0 + b);
    return n < 0 ? 0 : n >= a.cap ? a.cap : n + 1;
}

__device__ __forceinline__ int p4_units(int keys) { return (keys + P4_STEP - 1) / P4_STEP; }
// n / d for a quotient below 2^21
__device__ __forceinline__ int p4_div(int n, int d) {
    int q = (int)((float)n * rcp_approx((float)d));
    const int r = n - q * d;
    return r < 0 ? q - 1 : r >= d ? q + 1 : q;
}

// A place in the list of units (of 64 keys): unit u of n of (sequence b, kv head h).
struct P4Cursor {
    int b, h, u, n, keys;
};
// To the next (sequence, kv head); there is one.
__device__ __forceinline__ void p4_next(const P4Args& a, P4Cursor& c) {
    c.u = 0;
    if (++c.h < a.Hkv) return;
    c.h = 0;
    do {  // (sequences without keys have no units)
        c.keys = p4_keys(a, ++c.b);
    } while (c.keys == 0);
    c.n = p4_units(c.keys);
}

// BT: 16-key tiles of a page that a step takes (1, 2: pages of 16 and 32 tokens, fetched whole; 4: a part of a larger page).
// HC: columns of a product that the heads of a group take (the least power of two that holds them, 2 at least). With fewer than 8
// the columns hold the heads 8 / HC times, and of the scores of 8 / HC tiles each tile keeps its own columns: no lane
// works on the softmax of a column without a head, and O's column sets are added at the end. Against all heads in 8
// columns: groups of two 45.6 us against 61.8 (64 @ 4096; in 4 columns 46.9), groups of four 90 against 130 (16 @ 32,768).
// Groups of five to eight take a step's scores in two halves (all at once they left the registers).
template <int DH, int BT, int HC>
__global__ void __launch_bounds__(P4_THREADS, P4_CTAS)
    attn_paged4_kernel(const P4Args a) {
    using Ly = P4Layout<DH>;
    constexpr int NG = Ly::NG, NS = Ly::NS, PITCH = Ly::PITCH;
    constexpr int SHARE = 8 / HC;            // tiles whose scores share the columns
    constexpr int SUBS = HC == 8 ? 2 : 1, SUB = P4_TILES / SUBS;  // parts of a step, and tiles, whose scores are held at once
    constexpr int SETS = SUB / SHARE;        // sets of scores of a step: two rows by two columns a lane
    constexpr int LANES = HC / 2;            // lanes t that hold the columns of one tile
    extern __shared__ __align__(128) uint8_t p4_rings[];
    __shared__ uint64_t bars[P4_WARPS][NS];
    __shared__ int strip_end[P4_STRIPS];   // units of one kv head up to the strip's end
    __shared__ int strip_keys[P4_STRIPS];  // keys of the strip's (last) sequence
    __shared__ int warp_sum[P4_WARPS];
    __shared__ int seg_sh[P4_WARPS], whole_sh[P4_WARPS];
    __shared__ float2 lift_sh[P4_WARPS][4];  // [warp][pair of heads]: exponents of the lifts (every lane reads what it wrote)
    __shared__ int abort_sh;
    volatile int* abort_flag = &abort_sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;  // fragment coordinates
    uint64_t* full = bars[warp];
    if (threadIdx.x == 0) abort_sh = 0;
    if (lane == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();

    // ---------------- this warp's run of units [x0, x0 + mine)
    const int per = (a.B + P4_STRIPS - 1) / P4_STRIPS, places = (int)gridDim.x * P4_WARPS;
    {
        int sum = 0, keys = 0;
        const int b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
        for (int b = b0; b < b1; ++b) {
            keys = p4_keys(a, b);
            sum += p4_units(keys);
            if (keys == 0 && b % gridDim.x == blockIdx.x)  // a sequence without keys
                for (int e = 0; e < a.Hq * DH / 8; ++e)
                    reinterpret_cast<uint4*>(a.out + (size_t)b * a.Hq * DH)[e] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < P4_WARPS; ++w) sum += w < warp ? warp_sum[w] : 0;
        strip_end[threadIdx.x] = sum;
        strip_keys[threadIdx.x] = keys;
        __syncthreads();
    }
    auto all_units = [&]() { return strip_end[P4_STRIPS - 1] * a.Hkv; };  // (fewer than 2^31: checked on the host)
    // warps of a CTA that work: few units are spread over the SMs (1 sequence of 4096 keys, 8 kv heads: 9.3 us, with full
    // CTAs 10.0, when it was changed), but not further than a warp a scheduler: every CTA that shares a kv head leaves a
    // record for the join (2 kv heads, a warp a CTA 15.5 us, four 10.3)
    auto team_of = [&](int units) { return max(4, min(P4_WARPS, p4_div(min(units, places) + (int)gridDim.x - 1, (int)gridDim.x))); };
    const int units = all_units();
    const int gw = warp < team_of(units) ? blockIdx.x * team_of(units) + warp : places;
    // as many warps as there are places, but a unit a warp at least (no run between two others is empty); the first `more`
    // runs are a unit longer
    const int warps = min(places, units), len = units > places ? p4_div(units, places) : min(units, 1);
    const int more = units - len * warps;
    const int x0 = gw * len + min(gw, more), mine = gw < warps ? len + (gw < more ? 1 : 0) : 0;

    P4Cursor use{0, 0, 0, 1, 1};
    bool inside = true;  // the current (sequence, kv head) begins in this run
    if (mine > 0) {
        // the strip that holds unit x0, by its twelfth and then within it; then the sequence, whose units are [Hkv P_b, Hkv P_(b+1))
        static_assert(P4_STRIPS == 32 * P4_WARPS, "strips");
        const int coarse = __popc(__ballot_sync(0xffffffffu, strip_end[lane * P4_WARPS + P4_WARPS - 1] * a.Hkv <= x0));
        const int fine = strip_end[min(coarse * P4_WARPS + lane, P4_STRIPS - 1)];
        const int strip = coarse * P4_WARPS + __popc(__ballot_sync(0xffffffffu, lane < P4_WARPS && fine * a.Hkv <= x0));
        int p = strip > 0 ? strip_end[strip - 1] : 0;
        use.b = strip * per;
        use.keys = strip_keys[strip];
        while (true) {
            if (per > 1) use.keys = p4_keys(a, use.b);
            use.n = p4_units(use.keys);
            if (per == 1 || (p + use.n) * a.Hkv > x0) break;
            p += use.n;
            ++use.b;
        }
        const int in = x0 - p * a.Hkv;
        use.h = p4_div(in, use.n);
        use.u = in - use.h * use.n;
        inside = use.u == 0;
    }

    // ---------------- the ring: the run's unit i goes to slot i % NS, K in the first half of it, V in the second
    constexpr int TILE = 16 * DH / 2, SIDE = 16 * NG * 4;  // codes, and scales and minima, of 16 keys
    auto tile_at = [](int i) { return i / BT * BT * (TILE + SIDE) + i % BT * TILE; };  // tile i in its half
    auto side_at = [](int i) { return i / BT * BT * (TILE + SIDE) + BT * TILE + i % BT * SIDE; };
    // Lanes that copy K, then as many for V: one for each page, or (BT 4) one for the codes and one for the scales and minima.
    constexpr int COPY = BT == 4 ? 2 : P4_TILES / BT;
    const int page_log = a.cache.page_log;
    const uint32_t to = smem_u32(p4_rings + warp * Ly::RING) + (lane & COPY ? Ly::HALF : 0) +
                        (lane & (COPY - 1)) * (BT == 4 ? P4_TILES * TILE : BT * (TILE + SIDE));
    P4Cursor ask = use;
    int ask_left = mine, issued = 0;
    int tab = 0, tab_b = -1, tab_at = 0;  // this lane's entry of the page table, tab_at + lane of sequence tab_b
    const uint8_t* from = nullptr;
    int same_page = 0;  // BT 4: units of the sequence in the page behind this one
    bool bad_page = false;
    auto issue = [&](int slot) {  // the next unit, if the run has one
        if (ask_left == 0) return;
        const int k0 = ask.u * P4_STEP, tiles = (min(P4_STEP, ask.keys - k0) + 15) >> 4;
        const bool side = BT == 4 && (lane & 1);
        // (of several pages those that the sequence reaches)
        const bool copies = lane < 2 * COPY && (BT == 4 || (lane & (COPY - 1)) * BT < tiles);
        if (BT < 4 || --same_page < 0) {
            const int first = k0 >> page_log, at = first & ~31;
            if (tab_b != ask.b || tab_at != at) {
                tab_b = ask.b;
                tab_at = at;
                tab = at + lane < a.cache.max_pages ? __ldg(a.cache.table + (size_t)ask.b * a.cache.max_pages + at + lane) : 0;
            }
            int id = __shfl_sync(0xffffffffu, tab, (first & 31) + (BT < 4 ? lane & (COPY - 1) : 0));
            if ((unsigned)id >= (unsigned)a.cache.n_pages) {  // (flagged; the output is invalid)
                bad_page = bad_page || copies;
                id = 0;
            }
            from = (lane & COPY ? a.cache.v : a.cache.k) +
                   ((long long)id * a.Hkv + ask.h) * (long long)p4_page_bytes(1 << page_log, DH);
            if constexpr (BT == 4) {
                const int row = k0 & ((1 << page_log) - 1);
                from += side ? (DH / 2 << page_log) + row * (NG * 4) : row * (DH / 2);
                same_page = (min((1 << page_log) - row, ask.keys - k0) - 1) / P4_STEP;
            }
        } else {
            from += (side ? NG * 4 : DH / 2) * P4_STEP;
        }
        const int pages = BT == 4 ? 0 : (tiles + BT - 1) / BT;
        if (lane == 0) mbar_expect_tx(&full[slot], 2 * (TILE + SIDE) * (BT == 4 ? tiles : pages * BT));
        __syncwarp();
        if (copies)
            bulk_load(to + slot * Ly::SLOT, from, BT == 4 ? tiles * (side ? SIDE : TILE) : BT * (TILE + SIDE), &full[slot]);
        ++issued;
        if (--ask_left > 0 && ++ask.u == ask.n) {
            p4_next(a, ask);
            same_page = 0;
        }
    };

    // ---------------- products
    const int qh = g & (HC - 1);              // head of this lane's column of q
    const int ch = 2 * (t & (LANES - 1));     // head of this lane's first column of scores and outputs
    const int part = t / LANES;               // which of the tiles that share the columns they belong to
    uint4 qraw[NG][2];
    uint32_t qf[NG][2][2][2];  // q^T fragments [group][word][nibbles][half]; zero past G
    float2 qs[NG], qscale;     // heads ch, ch + 1: sums of the scaled queries over a group of dims; what scores are scaled by
    // Weights p = 2^((score - ref) * qscale + adj) and p * scale, which has to fit fp16: ref is a score, and adj a whole number
    // chosen so that the largest p * scale of the run so far lies in [2^13, 2^15] (p itself below 2^75: a score past `high` is
    // looked at first). In one number the two lose adj where scores are large. adj is 60 where it should be more: then the
    // weights are lifted; and 61 as long as all of them were 0.
    float2 ref, adj, high, l;
    float o[NG][4][4];  // sums of weight * code (with its lift), in units of 2^-24 (tiles 1 and 3 of a group: 2^-20)
    float2 z[NG];       // sums of weight * minimum
    auto fetch_q = [&]() {
        const __nv_bfloat16* row = a.q + ((size_t)use.b * a.Hq + (size_t)use.h * a.G + qh) * DH + 16 * t;
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                qraw[c][e] = qh < a.G ? __ldg(reinterpret_cast<const uint4*>(row + c * kP4Group) + e) : make_uint4(0, 0, 0, 0);
    };
    auto begin = [&]() {  // a (sequence, kv head): its query, sums of nothing
        float x[NG][16];
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w[4] = {qraw[c][e].x, qraw[c][e].y, qraw[c][e].z, qraw[c][e].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[c][e * 8 + 2 * i] = bf16_lo(w[i]);
                    x[c][e * 8 + 2 * i + 1] = bf16_hi(w[i]);
                }
            }
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) big = fmaxf(big, fabsf(x[c][i]));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^-e: the head's largest value comes to [2^10, 2^11)
        const int e = min(max((int)(__float_as_uint(big) >> 23) - 137, -100), 100);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        float sums[NG];
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[c][i] *= down;
                s += x[c][i];
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            sums[c] = s * 5.9604644775390625e-8f;  // 2^-24, the unit of the products of codes
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // nibbles 2k and that + 4; the ones after them
                    const int d = w * 8 + k * 2;
                    qf[c][w][k][0] = pack_f16(x[c][d], x[c][d + 4]);
                    qf[c][w][k][1] = pack_f16(x[c][d + 1] * 0.0625f, x[c][d + 5] * 0.0625f);
                }
        }
        // (a query of infinity has no finite form)
        const float up = big < INFINITY ? __uint_as_float((uint32_t)(127 + e) << 23) * 16777216.f * (kLog2e / sqrtf((float)DH))
                                        : __uint_as_float(0x7fc00000u);
        const int at = ch * 4;  // the lane that holds the head as a row
        qscale = make_float2(__shfl_sync(0xffffffffu, up, at), __shfl_sync(0xffffffffu, up, at + 4));
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            qs[c] = make_float2(__shfl_sync(0xffffffffu, sums[c], at), __shfl_sync(0xffffffffu, sums[c], at + 4));
            z[c] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][0][i] = o[c][1][i] = o[c][2][i] = o[c][3][i] = 0.f;
        }
        l = make_float2(0.f, 0.f);
        ref = adj = make_float2(0.f, 0.f);
        lift_sh[warp][t & (LANES - 1)] = make_float2(0.f, 0.f);
        high = make_float2(-INFINITY, -INFINITY);  // the first score moves it
    };
    float2 down;  // what takes the lifts off
    // the sums of this warp's piece: dims c * 64 + 8 g + (0..7) of head ch + e
    auto piece = [&](int c, int e, float (&v)[8]) {
        const float add = e ? z[c].y : z[c].x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = (i & 1 ? 1048576.f : 16777216.f) * (e ? down.y : down.x);
            v[i] = fmaf(o[c][i][e], u, add);
            v[4 + i] = fmaf(o[c][i][2 + e], u, add);
        }
    };
    auto rescale = [&](float2 f) {
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                o[c][q][0] *= f.x;
                o[c][q][1] *= f.y;
                o[c][q][2] *= f.x;
                o[c][q][3] *= f.y;
            }
    };
    auto total = [&]() {  // sums over the keys that other lanes took
        const float2 lift = lift_sh[warp][t & (LANES - 1)];
        down = make_float2(ex2_approx(-lift.x), ex2_approx(-lift.y));
#pragma unroll
        for (int s = LANES; s < 32; s <<= 1) {
            l.x += __shfl_xor_sync(0xffffffffu, l.x, s);
            l.y += __shfl_xor_sync(0xffffffffu, l.y, s);
#pragma unroll
            for (int c = 0; c < NG; ++c) {
                z[c].x += __shfl_xor_sync(0xffffffffu, z[c].x, s);
                z[c].y += __shfl_xor_sync(0xffffffffu, z[c].y, s);
            }
        }
#pragma unroll
        for (int s = LANES; s < 4; s <<= 1)
#pragma unroll
            for (int c = 0; c < NG; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[c][q][e] += __shfl_xor_sync(0xffffffffu, o[c][q][e], s);
    };
    // (lanes that hold the same columns' sums share the groups of dims to store)
    auto stores = [&](int c) { return SHARE == 1 || c == part; };
    auto leave = [&](float* rec) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = ch + e;
            if (h >= a.G) continue;
#pragma unroll
            for (int c = 0; c < NG; ++c) {
                if (!stores(c)) continue;
                float v[8];
                piece(c, e, v);
                float4* dst = reinterpret_cast<float4*>(rec + h * PITCH + c * kP4Group + 8 * g);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
            if (g == 0 && stores(0))
                *reinterpret_cast<float4*>(rec + h * PITCH + DH) =
                    e ? make_float4(ref.y, adj.y, qscale.y, l.y) : make_float4(ref.x, adj.x, qscale.x, l.x);
        }
    };
    auto write_out = [&]() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = ch + e;
            if (h >= a.G) continue;
            const float inv = 1.f / (e ? l.y : l.x);
#pragma unroll
            for (int c = 0; c < NG; ++c) {
                if (!stores(c)) continue;
                float v[8];
                piece(c, e, v);
                *reinterpret_cast<uint4*>(a.out + ((size_t)use.b * a.Hq + (size_t)use.h * a.G + h) * DH + c * kP4Group + 8 * g) =
                    make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                               pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
            }
        }
    };
    auto sides = [](const uint8_t* at, uint32_t (&sd)[2][NG]) {  // scales and minima of this lane's two keys of a tile
        if constexpr (NG == 2) {
            const uint2 s0 = *reinterpret_cast<const uint2*>(at), s1 = *reinterpret_cast<const uint2*>(at + 8 * NG * 4);
            sd[0][0] = s0.x;
            sd[0][1] = s0.y;
            sd[1][0] = s1.x;
            sd[1][1] = s1.y;
        } else {
            sd[0][0] = *reinterpret_cast<const uint32_t*>(at);
            sd[1][0] = *reinterpret_cast<const uint32_t*>(at + 8 * NG * 4);
        }
    };
    const int swap = (g & 4) | (g & 1) << 1 | (g >> 1 & 1);  // row g of a tile is key swap (and row g + 8 key swap + 8):
    const int vkey = (2 * t & 4) | (t & 1);                  // the keys of rows 2t, which one load of V takes, are 0, 1, 4, 5
    const int side_l = swap * (NG * 4), kcode_l = swap * (DH / 2) + 8 * t, vcode_l = vkey * (DH / 2) + 4 * g;
    int part_side = 0;  // where the lane's tile of a set has its scales and minima, from the set's first tile on
#pragma unroll
    for (int k = 1; k < SHARE; ++k)
        if (part == k) part_side = side_at(k) - side_at(0);
    bool ok = true, fresh = true;
    int slot = 0, phase = 0, run_left = mine;
    int keys_left = use.keys - use.u * P4_STEP;  // of the (sequence, kv head), from the unit at hand on
    if (mine > 0) fetch_q();
    __syncwarp();  // the barriers are set
#pragma unroll 1
    for (int i = 0; i < NS; ++i) issue(i);
    float* const my_smem = reinterpret_cast<float*>(p4_rings + warp * Ly::RING);
#pragma unroll 1
    while (run_left > 0) {
        if (fresh) begin();
        if (!__all_sync(0xffffffffu, mbar_wait_suspend(&full[slot], phase, abort_flag))) { ok = false; break; }
        uint8_t* ka = p4_rings + warp * Ly::RING + slot * Ly::SLOT;
        uint8_t* va = ka + Ly::HALF;
        const int valid = keys_left;  // keys of the unit; 64 or more: all
        if (valid < P4_STEP) {
            // what stands behind the last key may be anything: its scales and minima become 0 (0 * NaN must not reach O)
            for (int e = lane; e < (P4_STEP - valid) * NG; e += 32) {
                const int key = valid + e / NG, tile = key >> 4;
                *reinterpret_cast<uint32_t*>(va + tile / BT * BT * (TILE + SIDE) + BT * TILE + tile % BT * SIDE +
                                             (key & 15) * (NG * 4) + e % NG * 4) = 0u;
            }
            fence_proxy_async_smem();  // (the slot's next copy comes after these stores)
            __syncwarp();
        }
#pragma unroll 1
        for (int sub = 0; sub < SUBS; ++sub) {
            const int left = valid - sub * SUB * 16;  // keys from this part on
            if (SUBS > 1 && left <= 0) break;
            const int codes_at = sub * SUB * (BT == 4 ? TILE : TILE + SIDE), sides_at = sub * SUB * (BT == 4 ? SIDE : TILE + SIDE);
            const uint8_t *ka_codes = ka + codes_at, *va_codes = va + codes_at;
            const uint8_t *ka_sides = ka + sides_at, *va_sides = va + sides_at;
            float2 x[SETS][2];  // scores [set][row g, row g + 8] of heads ch, ch + 1
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                float acc[SHARE][NG][4];
#pragma unroll
                for (int j = 0; j < SHARE; ++j) {
                    const uint8_t* codes = ka_codes + tile_at(k * SHARE + j) + kcode_l;
#pragma unroll
                    for (int c = 0; c < NG; ++c) {
                        const uint2 w0 = *reinterpret_cast<const uint2*>(codes + c * 32);
                        const uint2 w1 = *reinterpret_cast<const uint2*>(codes + 8 * (DH / 2) + c * 32);
                        const uint32_t a0[2] = {w0.x, w0.y}, a1[2] = {w1.x, w1.y};
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const uint32_t y0 = a0[w] >> 8, y1 = a1[w] >> 8;
                            if (w == 0)
                                mma_f16_first(acc[j][c], a0[w] & 0x000f000fu, a1[w] & 0x000f000fu, a0[w] & 0x00f000f0u,
                                              a1[w] & 0x00f000f0u, qf[c][w][0][0], qf[c][w][0][1]);
                            else
                                mma_f16(acc[j][c], a0[w] & 0x000f000fu, a1[w] & 0x000f000fu, a0[w] & 0x00f000f0u,
                                        a1[w] & 0x00f000f0u, qf[c][w][0][0], qf[c][w][0][1]);
                            mma_f16(acc[j][c], y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u,
                                    qf[c][w][1][0], qf[c][w][1][1]);
                        }
                    }
                }
                uint32_t sd[2][NG];
                sides(ka_sides + side_at(k * SHARE) + part_side + side_l, sd);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int c = 0; c < NG; ++c) {
                        const float sc = bf16_lo(sd[r][c]), lo = bf16_hi(sd[r][c]);
                        float a0 = acc[0][c][2 * r], a1 = acc[0][c][2 * r + 1];
#pragma unroll
                        for (int j = 1; j < SHARE; ++j) {
                            a0 = part == j ? acc[j][c][2 * r] : a0;
                            a1 = part == j ? acc[j][c][2 * r + 1] : a1;
                        }
                        s0 = fmaf(sc, a0, c == 0 ? lo * qs[c].x : fmaf(lo, qs[c].x, s0));
                        s1 = fmaf(sc, a1, c == 0 ? lo * qs[c].y : fmaf(lo, qs[c].y, s1));
                    }
                    x[k][r] = make_float2(s0, s1);
                }
            }
            if (left < SUB * 16) {
#pragma unroll
                for (int k = 0; k < SETS; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if ((k * SHARE + part) * 16 + swap + 8 * r >= left) x[k][r] = make_float2(-INFINITY, -INFINITY);
            }
            // weights p, and p * scale by group of dims
            float2 p[SETS][2], wt[SETS][NG][2];
            uint32_t sd[SETS][2][NG];
#pragma unroll
            for (int k = 0; k < SETS; ++k) sides(va_sides + side_at(k * SHARE) + part_side + side_l, sd[k]);
            float2 mx = x[0][0];
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                mx.x = fmax3(mx.x, x[k][0].x, x[k][1].x);
                mx.y = fmax3(mx.y, x[k][0].y, x[k][1].y);
            }
            float2 f = make_float2(1.f, 1.f);  // what the sums so far are multiplied by (nothing is there before the first score)
            struct {
                bool x, y;
            } up{};
            // a score past `high` comes first: p is 1 for the largest
            const bool moved = __any_sync(0xffffffffu, mx.x > high.x || mx.y > high.y);
            if (moved) {
#pragma unroll
                for (int s = LANES; s < 32; s <<= 1) {
                    mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, s));
                    mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, s));
                }
                up = {mx.x > high.x, mx.y > high.y};
                auto raise = [](bool up, float mx, float qscale, float high, float& ref, float& adj, float& f) {
                    if (!up) return;
                    f = high == -INFINITY ? 0.f : ex2_approx(fmaf(ref - mx, qscale, -adj));
                    ref = mx;
                    adj = 0.f;
                };
                raise(up.x, mx.x, qscale.x, high.x, ref.x, adj.x, f.x);
                raise(up.y, mx.y, qscale.y, high.y, ref.y, adj.y, f.y);
            }
            float2 top = make_float2(0.f, 0.f);
            auto weigh = [&]() {
#pragma unroll
                for (int k = 0; k < SETS; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int c = 0; c < NG; ++c) {
                            const float sc = bf16_lo(sd[k][r][c]);
                            wt[k][c][r] = mul2(p[k][r], make_float2(sc, sc));
                        }
            };
#pragma unroll
            for (int k = 0; k < SETS; ++k)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 a = fma2(add2(x[k][r], make_float2(-ref.x, -ref.y)), qscale, adj);
                    p[k][r] = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                }
            weigh();
#pragma unroll
            for (int k = 0; k < SETS; ++k)
#pragma unroll
                for (int c = 0; c < NG; ++c) {
                    top.x = fmax3(top.x, fabsf(wt[k][c][0].x), fabsf(wt[k][c][1].x));
                    top.y = fmax3(top.y, fabsf(wt[k][c][0].y), fabsf(wt[k][c][1].y));
                }
            if (moved || __any_sync(0xffffffffu, top.x > (adj.x >= 60.f ? 0.f : 32768.f) || top.y > (adj.y >= 60.f ? 0.f : 32768.f))) {
                // then the weights of V: the largest one to [2^13, 2^14), p at most 2^60
#pragma unroll
                for (int s = LANES; s < 32; s <<= 1) {
                    top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, s));
                    top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, s));
                }
                auto suit = [](float top, bool up, float adj) {
                    const int e = (int)(__float_as_uint(top) >> 23);
                    return up || top > (adj == 61.f ? 0.f : 32768.f) ? fminf((float)(140 - e), (top > 0.f ? 60.f : 61.f) - adj) : 0.f;
                };
                const float2 more = make_float2(suit(top.x, up.x, adj.x), suit(top.y, up.y, adj.y));
                const float2 by = make_float2(ex2_approx(more.x), ex2_approx(more.y));
                adj = add2(adj, more);
                const float2 was = lift_sh[warp][t & (LANES - 1)];
                f = mul2(f, by);
#pragma unroll
                for (int k = 0; k < SETS; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r) p[k][r] = mul2(p[k][r], by);
                weigh();
                high = make_float2(ref.x + (75.f - adj.x) / qscale.x, ref.y + (75.f - adj.y) / qscale.y);
                l = mul2(l, f);
#pragma unroll
                for (int c = 0; c < NG; ++c) z[c] = mul2(z[c], f);
                if (fmaxf(adj.x, adj.y) >= 60.f || was.x + was.y > 0.f) {
                    // the lifts of this part of the step (weights take them after the scale: p and the lift alone may overflow)
                    auto lift_of = [](float top, float adj) {
                        return adj == 60.f ? (float)min(max(140 - (int)(__float_as_uint(top) >> 23), 0), 86) : 0.f;
                    };
                    const float2 lift = make_float2(lift_of(top.x * by.x, adj.x), lift_of(top.y * by.y, adj.y));
                    const float2 up_by = make_float2(ex2_approx(lift.x), ex2_approx(lift.y));
                    lift_sh[warp][t & (LANES - 1)] = lift;
                    f = mul2(f, make_float2(ex2_approx(lift.x - was.x), ex2_approx(lift.y - was.y)));
#pragma unroll
                    for (int k = 0; k < SETS; ++k)
#pragma unroll
                        for (int c = 0; c < NG; ++c)
#pragma unroll
                            for (int r = 0; r < 2; ++r) wt[k][c][r] = mul2(wt[k][c][r], up_by);
                }
                rescale(f);
            }
            uint32_t wb[SETS][NG][2];  // P^T fragments
#pragma unroll
            for (int k = 0; k < SETS; ++k)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    l = add2(l, p[k][r]);
#pragma unroll
                    for (int c = 0; c < NG; ++c) {
                        const float lo = bf16_hi(sd[k][r][c]);
                        z[c] = make_float2(fmaf(p[k][r].x, lo, z[c].x), fmaf(p[k][r].y, lo, z[c].y));
                        wb[k][c][r] = transpose8x8(pack_f16(wt[k][c][r].x, wt[k][c][r].y));
                    }
                }
#pragma unroll
            for (int k = 0; k < SUB; ++k) {
                const uint8_t* codes = va_codes + tile_at(k) + vcode_l;
                const bool mine_k = SHARE == 1 || g / HC == k % SHARE;  // this lane's column of O takes the tile
#pragma unroll
                for (int c = 0; c < NG; ++c) {
                    const uint32_t b0 = mine_k ? wb[k / SHARE][c][0] : 0u, b1 = mine_k ? wb[k / SHARE][c][1] : 0u;
                    // rows 2t, 2t + 1 (keys vkey and vkey + 2), and eight further: the first and the last four nibbles
                    auto word = [&](int key) { return *reinterpret_cast<const uint32_t*>(codes + c * 32 + key * (DH / 2)); };
                    const uint32_t wa = word(0), wb2 = word(2), wc = word(8), wd = word(10);
                    uint32_t v[4] = {__byte_perm(wa, wb2, 0x5410), __byte_perm(wa, wb2, 0x7632), __byte_perm(wc, wd, 0x5410),
                                     __byte_perm(wc, wd, 0x7632)};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (q == 2) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] >>= 8;
                        }
                        const uint32_t mask = q & 1 ? 0x00f000f0u : 0x000f000fu;
                        mma_f16(o[c][q], v[0] & mask, v[1] & mask, v[2] & mask, v[3] & mask, b0, b1);
                    }
                }
            }
        }
        __syncwarp();  // every lane has read the slot: the unit NS further may come
        issue(slot);
        if (++slot == NS) {
            slot = 0;
            phase ^= 1;
        }
        keys_left -= P4_STEP;
        fresh = keys_left <= 0;
        if (--run_left > 0 && !fresh) continue;
        // the (sequence, kv head) or the run ends: written out if all of it was in this run, left as a piece otherwise (that at the
        // end of the run in the ring, which is done)
        total();
        if (inside && fresh) write_out();
        else leave(run_left == 0 ? my_smem : a.recs + (size_t)gw * 2 * a.G * PITCH);
        if (run_left == 0) break;
        inside = true;
        p4_next(a, use);
        keys_left = use.keys;
        fetch_q();
    }
    if (__any_sync(0xffffffffu, bad_page) && lane == 0 && a.err) atomicOr(a.err, ERR_INDEX);
    if (!ok) {  // give up: wait, bounded, for the copies still on their way
        *abort_flag = 1;
        if (a.err && lane == 0) atomicOr(a.err, ERR_TIMEOUT);
        int never = 0;
        for (int j = mine - run_left; j < issued; ++j) mbar_wait_suspend(&full[j % NS], (j / NS) & 1, &never);
    }

    // ---------------- the pieces at the ends of this CTA's runs
    const bool ends = fresh;                          // the (sequence, kv head) ends with the run
    const bool open = mine > 0 && !(inside && ends);  // a part of it lies in another run
    const int seg = use.b * a.Hkv + use.h;
    if (lane == 0) {
        seg_sh[warp] = open ? seg : -1;
        whole_sh[warp] = (open && inside ? 1 : 0) | (open && ends ? 2 : 0);  // begins, ends in this run
    }
    __syncthreads();
    // Join the pieces at the ends of this CTA's runs: those of neighbouring warps that belong to one (sequence, kv head), and, where
    // it ends as the first piece of the next warp's run, that warp's record. Quads of dims of the group that begins at warp w0:
    const int G = a.G, quads = G * (DH / 4);
    constexpr int STEP = Ly::RING / 4;  // floats from one warp's piece to the next
    const int team = team_of(all_units());  // (again: not held through the loop)
    const int cta0 = blockIdx.x * team, here = max(0, min(team, warps - cta0));  // warps with a run
    for (int e0 = threadIdx.x; e0 < here * quads; e0 += P4_THREADS) {
        const int w0 = p4_div(e0, quads), e = e0 - w0 * quads, s = seg_sh[w0];
        if (s < 0 || (w0 > 0 && seg_sh[w0 - 1] == s)) continue;
        int w1 = w0 + 1;
        while (w1 < P4_WARPS && seg_sh[w1] == s) ++w1;
        const bool tail = !(whole_sh[w1 - 1] & 2) && w1 < here;
        const bool whole = (whole_sh[w0] & 1) && ((whole_sh[w1 - 1] & 2) || tail);
        const int h = e / (DH / 4), dd = e % (DH / 4) * 4;
        const float* rec = reinterpret_cast<const float*>(p4_rings) + h * PITCH;
        const float* far = a.recs + (size_t)(cta0 + w1) * 2 * G * PITCH + h * PITCH;
        float4 far_st = make_float4(-INFINITY, 0.f, 0.f, 0.f), far_y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tail && whole) {
            far_st = __ldcg(reinterpret_cast<const float4*>(far + DH));
            far_y = __ldcg(reinterpret_cast<const float4*>(far + dd));
        }
        // the joined piece so far: reference R (that of the largest scores), E: its weights are 2^E above those of R without adjustment
        const float scale = reinterpret_cast<const float*>(rec + w0 * STEP + DH)[2];
        float R = -INFINITY, E = -INFINITY, L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        auto join = [&](auto& st, auto& y) {  // (a reference of -inf: no piece)
            constexpr int N = sizeof(st) / sizeof(st[0]);
            float top = R;
#pragma unroll
            for (int k = 0; k < N; ++k) top = fmaxf(top, st[k].x);
            const float was = R == -INFINITY ? -INFINITY : fmaf(R - top, scale, E);
            R = top;
            E = was;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                st[k].x = st[k].x == -INFINITY ? -INFINITY : fmaf(st[k].x - R, scale, -st[k].y);
                E = fmaxf(E, st[k].x);
            }
            const float g = was == -INFINITY ? 0.f : ex2_approx(was - E);
            L *= g;
            v = make_float4(v.x * g, v.y * g, v.z * g, v.w * g);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float f = ex2_approx(st[k].x - E);
                L = fmaf(st[k].w, f, L);
                v = make_float4(fmaf(y[k].x, f, v.x), fmaf(y[k].y, f, v.y), fmaf(y[k].z, f, v.z), fmaf(y[k].w, f, v.w));
            }
        };
#pragma unroll 1
        for (int w = w0; w < w1; w += 4) {  // four pieces' loads at once
            float4 st[4], y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                st[k] = w + k < w1 ? *reinterpret_cast<const float4*>(rec + (w + k) * STEP + DH) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
                y[k] = w + k < w1 ? *reinterpret_cast<const float4*>(rec + (w + k) * STEP + dd) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            join(st, y);
        }
        if (tail && whole) {
            float4 st[1] = {far_st}, y[1] = {far_y};
            join(st, y);
        }
        if (whole) {
            const float inv = 1.f / L;
            const size_t row = (size_t)(s / a.Hkv) * a.Hq + (size_t)(s % a.Hkv) * G + h;
            *reinterpret_cast<uint2*>(a.out + row * DH + dd) =
                make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
        } else {
            float* dst = a.recs + ((size_t)(cta0 + w0) * 2 + 1) * G * PITCH + h * PITCH;
            *reinterpret_cast<float4*>(dst + dd) = v;
            if (dd == 0) *reinterpret_cast<float4*>(dst + DH) = make_float4(R, -E, scale, L);
        }
    }
    // the (sequence, kv head) that goes on behind this CTA, if it began here
    if (warp == team - 1 && lane == 0) {
        P4Desc d{-1, 0, 0, 0, team};
        const int s = seg_sh[warp];
        if (s >= 0 && !(whole_sh[warp] & 2)) {
            int w0 = warp;
            while (w0 > 0 && seg_sh[w0 - 1] == s) --w0;
            const RunEnd end = run_of_end(x0 + mine, p4_units(max(keys_left, 0)), len, more, *abort_flag != 0,
                                          [](int n, int d) { return p4_div(n, d); });
            if ((whole_sh[w0] & 1) && end.run >= 0) {
                d.seg = s;
                d.first = cta0 + w0;
                d.last = end.run;
                d.last_slot = end.with_run ? 1 : 0;
            }
        }
        a.desc[blockIdx.x] = d;
    }
}

// Join the records of the (sequence, kv head) that begins in CTA blockIdx.x's runs and ends in another's: the one at its
// beginning, one of each CTA behind it (in that CTA's first warp's place) and the one at its end. A thread takes
// a quad of dims and every ways-th record.
constexpr int P4_JOIN_THREADS = 512;
template <int DH>
__global__ void __launch_bounds__(P4_JOIN_THREADS)
    attn_paged4_join_kernel(const P4Args a) {
    constexpr int PITCH = P4Layout<DH>::PITCH;
    __shared__ float4 part[P4_JOIN_THREADS];
    __shared__ float4 stat[P4_JOIN_THREADS];
    pdl_wait();
    pdl_trigger();
    const P4Desc d = a.desc[blockIdx.x];
    if (d.seg < 0) return;
    const int G = a.G, quads = G * (DH / 4);  // at most 256
    const int ways = P4_JOIN_THREADS / quads;
    const int e = threadIdx.x % quads, way = threadIdx.x / quads;
    const int h = e / (DH / 4), dd = e % (DH / 4) * 4;
    // CTAs behind the first whose first warp leaves a record in place 1; then, for last_slot 0, the end's own
    const int c0 = d.first / d.team + 1, c1 = (d.last + d.last_slot - 1) / d.team;
    const int middle = max(0, c1 - c0 + 1), n = 1 + middle + (d.last_slot == 0 ? 1 : 0);
    auto record = [&](int i) -> const float* {
        const int w = i == 0 ? d.first : i <= middle ? (c0 + i - 1) * d.team : d.last;
        const int slot = i <= middle ? 1 : 0;
        return a.recs + ((size_t)w * 2 + slot) * G * PITCH + h * PITCH;
    };
    float4 t = make_float4(-INFINITY, 0.f, 0.f, 0.f);  // reference (-inf: no record yet), adjustment, scale of scores, sum of weights
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& s, const float4& y) {
        // 2^(what the record's weights are above the sum's)
        const float up = t.x == -INFINITY ? INFINITY : fmaf(s.x - t.x, s.z, t.y - s.y);
        float f = 1.f;
        if (up > 0.f) {
            const float g = ex2_approx(-up);
            t = make_float4(s.x, s.y, s.z, t.w * g);
            v = make_float4(v.x * g, v.y * g, v.z * g, v.w * g);
        } else {
            f = ex2_approx(up);
        }
        t.w = fmaf(s.w, f, t.w);
        v = make_float4(fmaf(y.x, f, v.x), fmaf(y.y, f, v.y), fmaf(y.z, f, v.z), fmaf(y.w, f, v.w));
    };
    if (way < ways) {
        constexpr int U = 4;  // records on their way at once
        for (int i0 = way; i0 < n; i0 += U * ways) {
            float4 s[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * ways < n) {
                    const float* rec = record(i0 + u * ways);
                    s[u] = __ldcg(reinterpret_cast<const float4*>(rec + DH));
                    y[u] = __ldcg(reinterpret_cast<const float4*>(rec + dd));
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * ways < n) add(s[u], y[u]);
        }
    }
    part[threadIdx.x] = v;
    stat[threadIdx.x] = t;
    __syncthreads();
    if (way > 0) return;
    for (int k = 1; k < min(ways, n); ++k) add(stat[k * quads + e], part[k * quads + e]);
    const float inv = 1.f / t.w;
    const size_t row = (size_t)(d.seg / a.Hkv) * a.Hq + (size_t)(d.seg % a.Hkv) * G + h;
    *reinterpret_cast<uint2*>(a.out + row * DH + dd) =
        make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
}

int p4_ctas() { return device_sm_count() * P4_CTAS; }

template <int DH, int BT, int HC>
cudaError_t paged4_launch_one(const P4Args& a, cudaStream_t st) {
    const int ctas = p4_ctas();
    cudaError_t e = launch_pdl(attn_paged4_kernel<DH, BT, HC>, dim3(ctas), dim3(P4_THREADS), P4Layout<DH>::SMEM, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_paged4_join_kernel<DH>, dim3(ctas), dim3(P4_JOIN_THREADS), 0, st, a);
}
template <int DH, int BT>
cudaError_t paged4_launch_bt(const P4Args& a, cudaStream_t st) {
    if (a.G <= 2) return paged4_launch_one<DH, BT, 2>(a, st);
    if (a.G <= 4) return paged4_launch_one<DH, BT, 4>(a, st);
    return paged4_launch_one<DH, BT, 8>(a, st);
}
template <int DH>
cudaError_t paged4_launch_dh(const P4Args& a, int page, cudaStream_t st) {
    if (page == 16) return paged4_launch_bt<DH, 1>(a, st);
    if (page == 32) return paged4_launch_bt<DH, 2>(a, st);
    return paged4_launch_bt<DH, 4>(a, st);
}

template <int DH, int BT>
cudaError_t paged4_prepare_bt() {
    const void* fns[] = {(const void*)attn_paged4_kernel<DH, BT, 2>, (const void*)attn_paged4_kernel<DH, BT, 4>,
                         (const void*)attn_paged4_kernel<DH, BT, 8>};
    for (const void* f : fns) {
        cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, P4Layout<DH>::SMEM);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
template <int DH>
cudaError_t paged4_prepare_dh() {
    cudaError_t e = paged4_prepare_bt<DH, 1>();
    if (e == cudaSuccess) e = paged4_prepare_bt<DH, 2>();
    if (e == cudaSuccess) e = paged4_prepare_bt<DH, 4>();
    return e;
}

size_t desc_bytes() { return ((size_t)p4_ctas() * sizeof(P4Desc) + 255) / 256 * 256; }

}  // namespace

size_t attn_decode_paged4_workspace(int G, int dh) {
    const int warps = p4_ctas() * P4_WARPS;
    return desc_bytes() + (size_t)warps * 2 * G * (dh + 4) * sizeof(float);
}

cudaError_t attn_decode_paged4_launch(const __nv_bfloat16* q, const void* k_pages, const void* v_pages, int n_pages, int page,
                                      const int* table, int max_pages, const int* len0, int B, int Hq, int Hkv, int dh,
                                      void* work, __nv_bfloat16* out, int* err, cudaStream_t st) {
    P4Args a{};
    a.q = q;
    a.out = out;
    int log = 0;
    while (1 << log < page) ++log;
    a.cache = Paged4{static_cast<const uint8_t*>(k_pages), static_cast<const uint8_t*>(v_pages), table, n_pages, max_pages, log};
    a.len0 = len0;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.cap = (int)std::min<long long>((long long)max_pages * page, 1 << 30);
    a.desc = static_cast<P4Desc*>(work);
    a.recs = reinterpret_cast<float*>(static_cast<uint8_t*>(work) + desc_bytes());
    a.err = err;
    return dh == 128 ? paged4_launch_dh<128>(a, page, st) : paged4_launch_dh<64>(a, page, st);
}

cudaError_t attention_paged4_prepare() {
    cudaError_t e = paged4_prepare_dh<128>();
    return e == cudaSuccess ? paged4_prepare_dh<64>() : e;
}

}  // namespace q3
