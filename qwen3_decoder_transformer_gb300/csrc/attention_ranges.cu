// Decode attention over key ranges: a sliding window with sink tokens, and a batch that shares a prefix.
//
// attn_ranges_kernel serves one query per (sequence, query head) over the visible keys of its sequence; a
// cluster of CTAs shares the keys of one (sequence, kv head). For a shared prefix, attn_prefix_launch
// (attention_tiles.cu) computes its part for the query rows of the whole batch at once and leaves one record per row
// tile and key chunk; attn_ranges_kernel works on the sequences' own keys beside it and joins the records, or
// attn_join_kernel does. A prefix of few keys for few sequences is another run of keys of attn_ranges_kernel.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace q3 {
namespace {

// ------------------------------------------------------------------------------------- own keys
// O = sum_i p_i v_i / sum_i p_i, p_i = 2^(q k_i log2(e) / sqrt(dh) - m) over the visible keys i: up to three
// runs of cache rows (sinks, window, the wrapped part of a rolling buffer; or the own slots before and
// behind a padding block, and a short prefix), taken in units of 16 keys.
//
// Every warp works through its own units alone, with a running maximum (lazily rescaled, as in the prefill
// kernels): its lane 0 keeps a ring full with the K and V boxes of the coming units (TMA, 128-byte
// swizzle; a stage's keys are asked for again right after its scores, its values after P V), so up to 128 KB an SM are on
// their way or in use, and no barrier joins the warps before the end. Three units a warp with two CTAs an SM instead of one
// unit with four stream no faster (64 sequences x 4,100 keys 152.5 us against 153.4) and start slower (one sequence 7.5
// against 6.8). The products are warp-level mma (m16n8k16,
// bf16 in, fp32 accumulate; the contraction is far below a tcgen05 tile) with the heads of the kv group as
// the 8 columns: S^T (keys x heads) = K q^T, P^T from accumulator to operand layout by a register transpose
// (movmatrix), O^T (head_dim x heads) += V^T P^T.
// Scores of rows behind a run are masked, and their value rows are zeroed in shared memory, so nothing
// stored in a hidden row can reach the result.
// What bounds it. Many sequences: HBM, 64 sequences x 4,100 keys of 8 kv heads, dh 128 (1.08 GB) 149-152 us from call to call
// (part of the keys still in L2), 155 us with a cold L2 under ncu, 6.9 TB/s (102% of the measured copy rate). Fragments loaded
// straight from global memory, without rings, took 219 us for any split: too little on its way per warp. One
// sequence: the chain of launch, length, first boxes and the join, 6.9 us for 4,100 keys by clusters of 16 CTAs
// (13 by 4).
constexpr int RG_KEYS = 16, RG_MAX_CLUSTER = 16, RG_MAX_G = 8, RG_WARPS = 4, RG_THREADS = 32 * RG_WARPS;
constexpr int RG_MAX_PARTS = 1 + kPrefixMaxChunks;
constexpr int RG_CTAS = 4;  // an SM
template <int DH>
struct RgLayout {
    static constexpr int NCH = DH / 64;               // 64-column boxes of a row
    static constexpr int BOX = RG_KEYS * 128;         // bytes of a box
    static constexpr int HALF = NCH * BOX;            // K (or V) of a unit
    static constexpr int RG_BYTES = 8192;             // ring of one warp
    static constexpr int ST = RG_BYTES / (2 * HALF);  // units in it: 1 (dh 128) or 2 (dh 64)
    static constexpr int SMEM = RG_WARPS * RG_BYTES + 1024;
    // the warps' results take the first bytes of the rings once all of them are done
    static constexpr int PITCH = DH + 4;
    static_assert(RG_WARPS * RG_MAX_G * PITCH * 4 <= RG_WARPS * RG_BYTES, "results fit the rings");
    static_assert(RG_CTAS * (SMEM + 8192) <= 227 * 1024, "shared memory");
};

struct RangeArgs {
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    const int* len0;
    int len_stride;
    int Hq, Hkv, G, cap;
    // window and sinks; ring > 0: rows [0, sink_rows) keep the first slots, the others wrap over ring rows
    int window, sinks, sink_rows, ring;
    const int* meta;    // own slots of a shared prefix: SeqMap::meta, or null
    int P;              // rows of the prefix that each sequence reads for itself, as a third run (0: none, or by records)
    const float* recs;  // records of the prefix to join (attn_prefix_launch)
    int nrec, row_tiles, tile_seqs;  // sequences of a row tile
    float* own;  // [B][Hkv][G][DH + 4]: where the own keys' (output sums, maximum, sum) go, to be joined by a launch of its own; or null
    int C, log_c;    // CTAs per (sequence, kv head), a power of two
    unsigned inv_g;  // 2^16 / G + 1: e / G = e * inv_g >> 16 for e < 2^8
    int* err;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_keys(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// 16-byte piece `piece` (8 columns) of row `row` in boxes of 16 rows x 128 bytes written with the 128-byte swizzle
__device__ __forceinline__ uint32_t rg_addr(uint32_t base, int row, int piece) {
    return base + (uint32_t)((piece >> 3) * RG_KEYS * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

// Four output dims dd.. of head h of the group, times scale.
template <int DH>
__device__ __forceinline__ void store_quad(const RangeArgs& a, int b, int j, int h, int dd, const float4& v, float scale) {
    const size_t row = (size_t)b * a.Hq + (size_t)j * a.G + h;
    *reinterpret_cast<uint2*>(a.out + row * DH + dd) =
        make_uint2(pack_bf16(v.x * scale, v.y * scale), pack_bf16(v.z * scale, v.w * scale));
}

// The prefix records of one (sequence, kv head): this sequence's rows in its row tile.
template <int DH>
struct Records {
    const float* rec;
    size_t step;  // between two key chunks
    int row;
    __device__ __forceinline__ Records(const RangeArgs& a, int b, int j) {
        const int tile = (int)((unsigned)b / (unsigned)a.tile_seqs);
        row = (b - tile * a.tile_seqs) * a.G;
        rec = a.recs + ((size_t)j * a.row_tiles + tile) * prefix_rec_floats(DH);
        step = (size_t)a.Hkv * a.row_tiles * prefix_rec_floats(DH);
    }
    __device__ __forceinline__ float4 quad(int r, int h, int dd) const {
        return __ldcg(reinterpret_cast<const float4*>(rec + r * step + ((size_t)(dd / 4) * kPrefixRows + row + h) * 4));
    }
    __device__ __forceinline__ float2 stat(int r, int h) const {  // maximum, sum
        return __ldcg(reinterpret_cast<const float2*>(rec + r * step + (size_t)DH * kPrefixRows + (row + h) * 2));
    }
};

__device__ __forceinline__ void add_scaled(float4& v, const float4& x, float f) {
    v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
}

// Head and first dim of quad e of the group's output (four dims of one head, the heads fastest).
__device__ __forceinline__ void quad_of(const RangeArgs& a, int e, int& h, int& dd) {
    const int d = (int)((unsigned)e * a.inv_g >> 16);
    h = e - d * a.G;
    dd = d * 4;
}

constexpr int RG_MAX_QUADS = RG_MAX_G * 32;
union JoinShared {
    struct {  // the own keys' part, then the prefix records
        float pm[RG_MAX_G][RG_MAX_PARTS], pl[RG_MAX_G][RG_MAX_PARTS], inv[RG_MAX_G];
    } records;
    struct {  // this CTA's share of the output, [its quads][CTAs of the cluster]
        float4 sums[RG_MAX_QUADS];
        float2 stat[RG_MAX_QUADS];
    } cluster;
};

// Join the own keys' result (own_stat(h) = (maximum, sum), output sums own_quad(h, dd)) and the prefix records by
// log-sum-exp: O = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
template <int DH, typename Stat, typename Quad>
__device__ __forceinline__ void join_records(const RangeArgs& a, int b, int j, JoinShared& js, Stat own_stat, Quad own_quad) {
    auto& pm = js.records.pm;
    auto& pl = js.records.pl;
    auto& inv = js.records.inv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int quads = a.G * (DH / 4), parts = 1 + a.nrec;
    const Records<DH> rec(a, b, j);
    // the output sums of the first records are on their way while the weights are worked out
    constexpr int PRE = 8;
    float4 pre[PRE];
    const int e0 = threadIdx.x;
    int h0, d0;
    quad_of(a, e0, h0, d0);
#pragma unroll
    for (int r = 0; r < PRE; ++r)
        if (r < a.nrec && e0 < quads) pre[r] = rec.quad(r, h0, d0);
    for (int e = threadIdx.x; e < parts * RG_MAX_G; e += RG_THREADS) {
        const int p = e / RG_MAX_G, h = e % RG_MAX_G;
        if (h < a.G) {
            const float2 ml = p == 0 ? own_stat(h) : rec.stat(p - 1, h);
            pm[h][p] = ml.x;
            pl[h][p] = ml.y;
        }
    }
    __syncthreads();
    for (int h = warp; h < a.G; h += RG_WARPS) {  // the parts' weights, into pm
        float M = -INFINITY, L = 0.f;
        for (int p = lane; p < parts; p += 32) M = fmaxf(M, pm[h][p]);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
        for (int p = lane; p < parts; p += 32) {
            const float f = pm[h][p] == -INFINITY ? 0.f : ex2_approx(pm[h][p] - M);
            L = fmaf(pl[h][p], f, L);
            pm[h][p] = f;
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
        if (lane == 0) inv[h] = L == 0.f ? 0.f : 1.f / L;
    }
    __syncthreads();
    for (int e = e0; e < quads; e += RG_THREADS) {
        int h, dd;
        quad_of(a, e, h, dd);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        add_scaled(v, own_quad(h, dd), pm[h][0]);
        int r = 0;
        if (e == e0) {
#pragma unroll
            for (; r < PRE; ++r)
                if (r < a.nrec) add_scaled(v, pre[r], pm[h][1 + r]);
        }
#pragma unroll 4
        for (; r < a.nrec; ++r) add_scaled(v, rec.quad(r, h, dd), pm[h][1 + r]);
        store_quad<DH>(a, b, j, h, dd, v, inv[h]);
    }
}

// The same over the a.C CTAs of a cluster, which have sent every CTA their parts of its share of the output (quad e is CTA
// e mod C's): C neighbouring threads take one quad, each one CTA's part and every C-th record, and add up by shuffles.
// (4,100 keys of one sequence by clusters of 16: one thread a quad reading the other CTAs' parts in turn 9.7 us, C threads
// reading them at once 8.4; sent, with one copy a unit and no divisions, 6.9.)
template <int DH>
__device__ __forceinline__ void join_cluster(const RangeArgs& a, int b, int j, int rank, const JoinShared& js) {
    const int C = a.C, quads = a.G * (DH / 4), p = threadIdx.x & (C - 1);  // C, up to 16, divides quads
    const Records<DH> rec(a, b, j);  // (not read without records)
    for (int t0 = 0; t0 < quads; t0 += RG_THREADS) {
        const bool on = t0 + threadIdx.x < quads;
        const int t = on ? t0 + threadIdx.x : p;
        int h, dd;
        quad_of(a, (t & ~(C - 1)) + rank, h, dd);
        const float m = js.cluster.stat[t].x, l = js.cluster.stat[t].y;
        const float4 x = js.cluster.sums[t];
        constexpr int PRE = 4;
        float2 rml[PRE];
        float4 rx[PRE];
#pragma unroll
        for (int k = 0; k < PRE; ++k)
            if (p + k * C < a.nrec) {
                rml[k] = rec.stat(p + k * C, h);
                rx[k] = rec.quad(p + k * C, h, dd);
            }
        float M = m;
#pragma unroll
        for (int k = 0; k < PRE; ++k)
            if (p + k * C < a.nrec) M = fmaxf(M, rml[k].x);
#pragma unroll 4
        for (int r = p + PRE * C; r < a.nrec; r += C) M = fmaxf(M, rec.stat(r, h).x);
        for (int o = C / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float pm, float pl, const float4& px) {
            const float f = pm == -INFINITY ? 0.f : ex2_approx(pm - M);
            L = fmaf(pl, f, L);
            add_scaled(v, px, f);
        };
        add(m, l, x);
#pragma unroll
        for (int k = 0; k < PRE; ++k)
            if (p + k * C < a.nrec) add(rml[k].x, rml[k].y, rx[k]);
#pragma unroll 4
        for (int r = p + PRE * C; r < a.nrec; r += C) {
            const float2 ml = rec.stat(r, h);
            add(ml.x, ml.y, rec.quad(r, h, dd));
        }
        for (int o = C / 2; o > 0; o >>= 1) {
            L += __shfl_xor_sync(0xffffffffu, L, o);
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
            v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
            v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
        }
        if (p == 0 && on) store_quad<DH>(a, b, j, h, dd, v, L == 0.f ? 0.f : 1.f / L);
    }
}

template <int DH, bool SINKS>
__global__ void __launch_bounds__(RG_THREADS, RG_CTAS)
    attn_ranges_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmPK, const __grid_constant__ CUtensorMap tmPV, const RangeArgs a) {
    using Ly = RgLayout<DH>;
    constexpr int NW = RG_WARPS, THREADS = RG_THREADS, ST = Ly::ST, RG_BYTES = Ly::RG_BYTES;
    extern __shared__ uint8_t rg_raw[];
    const uint32_t raw_addr = smem_u32(rg_raw);
    uint8_t* rings = rg_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    auto so = reinterpret_cast<float(*)[RG_MAX_G][Ly::PITCH]>(rings);  // the warps' output sums, once the rings are done
    __shared__ uint64_t bars[RG_WARPS][2 * ST];                 // [K of each stage, V of each stage]
    __shared__ float sm[NW][RG_MAX_G], sl[NW][RG_MAX_G];
    __shared__ float cm[RG_MAX_G], cl[RG_MAX_G];                   // this CTA's maximum and sum
    __shared__ JoinShared js;
    __shared__ int abort_sh;
    volatile int* abort_flag = &abort_sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, tq = lane & 3;  // fragment coordinates
    const int rank = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
    uint64_t* k_full = bars[warp];
    uint64_t* v_full = bars[warp] + ST;
    if (a.C > 1) cluster_arrive();  // every CTA has started, by the time parts are sent
    if (threadIdx.x == 0) abort_sh = 0;
    if (lane == 0) {
        for (int i = 0; i < 2 * ST; ++i) mbar_init(&bars[warp][i], 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    __syncthreads();
    // Without partial results to join this is an ordinary dependent launch. With them, the prefix kernel
    // before it has itself waited for everything earlier before it let this kernel start, and only the
    // join below has to wait for the prefix kernel.
    if (a.nrec == 0) {
        pdl_wait();
        pdl_trigger();
    }
    // q^T fragments: column gq = query head gq of the group (zero past G)
    uint32_t qf[DH / 16][2];
    {
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(a.q + ((size_t)b * a.Hq + (size_t)j * a.G + gq) * DH);
#pragma unroll
        for (int ks = 0; ks < DH / 16; ++ks) {
            qf[ks][0] = gq < a.G ? __ldcg(qrow + ks * 8 + tq) : 0u;
            qf[ks][1] = gq < a.G ? __ldcg(qrow + ks * 8 + 4 + tq) : 0u;
        }
    }
    int n = __ldcg(a.len0 + (size_t)b * a.len_stride);
    n = n < 0 ? 0 : min(n, 1 << 30) + 1;
    if (!SINKS || a.ring == 0) n = min(n, a.cap);
    // the runs of visible rows
    int row[3] = {0, 0, 0}, cnt[3] = {0, 0, 0};
    if constexpr (SINKS) {
        const int lo = max(0, n - a.window);
        cnt[0] = min(a.sinks, lo);
        if (a.ring == 0) {
            row[1] = lo;
            cnt[1] = n - lo;
        } else if (lo < a.sink_rows) {  // the ring's first turn
            row[1] = lo;
            cnt[1] = min(n, a.sink_rows) - lo;
            row[2] = a.sink_rows;
            cnt[2] = max(0, n - a.sink_rows);
        } else {
            const int at = (lo - a.sink_rows) % a.ring;
            row[1] = a.sink_rows + at;
            cnt[1] = min(n - lo, a.ring - at);
            row[2] = a.sink_rows;
            cnt[2] = n - lo - cnt[1];
        }
    } else {
        int ps = 0, pe = 0, psh = 0;
        if (a.meta) {
            ps = __ldcg(a.meta);
            psh = __ldcg(a.meta + 1);
            pe = ps + __ldcg(a.meta + kSeqMetaHead + b);
        }
        row[0] = min(max(psh, 0), n);
        const int end = min(max(ps, row[0]), n);
        cnt[0] = end - row[0];
        row[1] = min(max(pe, end), n);
        cnt[1] = n - row[1];
        cnt[2] = a.P;
    }
    const int n0 = (cnt[0] + RG_KEYS - 1) / RG_KEYS, n1 = n0 + (cnt[1] + RG_KEYS - 1) / RG_KEYS;
    const int units = n1 + (cnt[2] + RG_KEYS - 1) / RG_KEYS;
    // first cache row of unit u, and how many rows of it are visible
    auto unit = [&](int u, int& valid) -> int {
        const int first = u < n0 ? 0 : u < n1 ? n0 : n1;
        const int r = u < n0 ? row[0] : u < n1 ? row[1] : row[2], c = u < n0 ? cnt[0] : u < n1 ? cnt[1] : cnt[2];
        valid = min(RG_KEYS, c - (u - first) * RG_KEYS);
        return r + (u - first) * RG_KEYS;
    };
    const int u0 = (int)((unsigned)units * (unsigned)rank >> a.log_c), u1 = (int)((unsigned)units * (rank + 1u) >> a.log_c);
    const int mine = u1 - u0 > warp ? (u1 - u0 - warp + NW - 1) / NW : 0;  // units u0 + warp + NW i

    uint8_t* ring_p = rings + warp * RG_BYTES;
    const uint32_t ring_a = smem_u32(ring_p);
    auto load = [&](int i, const CUtensorMap* map, const CUtensorMap* pmap, uint64_t* full, int off) {
        int valid;
        const int u = u0 + warp + NW * i, y = unit(u, valid), st = i % ST;
        const bool prefix = !SINKS && u >= n1;
        const int z = prefix ? j : b * a.Hkv + j;
        uint8_t* dst = ring_p + st * 2 * Ly::HALF + off;
        mbar_expect_tx(&full[st], Ly::HALF);
        tma_load_4d(dst, prefix ? pmap : map, &full[st], 0, y, 0, z);
    };
    auto load_k = [&](int i) { load(i, &tmK, &tmPK, k_full, 0); };  // lane 0: K or V of unit i
    auto load_v = [&](int i) { load(i, &tmV, &tmPV, v_full, Ly::HALF); };
    if (lane == 0)
        for (int i = 0; i < min(ST, mine); ++i) {
            load_k(i);
            load_v(i);
        }

    const float sl2 = kLog2e / sqrtf((float)DH);
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2 tq and 2 tq + 1
    float o[DH / 16][4];                                       // tile t: rows are dims 16 t + gq and 16 t + gq + 8
#pragma unroll
    for (int t = 0; t < DH / 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    bool ok = true, k_ahead = false;  // k_ahead: the keys of unit i + ST are on their way
    int i = 0;
    for (; i < mine; ++i) {
        const int st = i % ST, ph = (i / ST) & 1;
        int valid;
        unit(u0 + warp + NW * i, valid);
        const uint32_t ka = ring_a + st * 2 * Ly::HALF, va = ka + Ly::HALF;
        if (!__all_sync(0xffffffffu, mbar_wait_suspend(&k_full[st], ph, abort_flag))) { ok = false; break; }
        float d[4] = {0.f, 0.f, 0.f, 0.f}, d2[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of products
        const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int ks = 0; ks < DH / 16; ++ks) {
            uint32_t f[4];
            ldsm4(rg_addr(ka, krow, 2 * ks + (lane >> 4)), f);
            mma_keys(ks & 1 ? d2 : d, f, qf[ks][0], qf[ks][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] += d2[e];
        __syncwarp();  // every lane has read the unit's keys: the next ones may come
        k_ahead = i + ST < mine;
        if (lane == 0 && k_ahead) load_k(i + ST);
        const bool in0 = gq < valid, in1 = gq + 8 < valid;
        const float v0 = in0 ? d[0] * sl2 : -INFINITY, v1 = in0 ? d[1] * sl2 : -INFINITY;
        const float v2 = in1 ? d[2] * sl2 : -INFINITY, v3 = in1 ? d[3] * sl2 : -INFINITY;
        float x0 = fmaxf(v0, v2), x1 = fmaxf(v1, v3);
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, s));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, s));
        }
        // O and the sums move to a larger maximum only when it grew by more than 8 (P <= 2^8)
        const bool g0 = x0 > m0 + 8.f, g1 = x1 > m1 + 8.f;
        if (__any_sync(0xffffffffu, g0 | g1)) {
            const float f0 = g0 ? ex2_approx(m0 - x0) : 1.f, f1 = g1 ? ex2_approx(m1 - x1) : 1.f;
            m0 = g0 ? x0 : m0;
            m1 = g1 ? x1 : m1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int t = 0; t < DH / 16; ++t) {
                o[t][0] *= f0;
                o[t][1] *= f1;
                o[t][2] *= f0;
                o[t][3] *= f1;
            }
        }
        const float s0 = m0 == -INFINITY ? 0.f : m0, s1 = m1 == -INFINITY ? 0.f : m1;
        const float p0 = ex2_approx(v0 - s0), p1 = ex2_approx(v1 - s1);
        const float p2 = ex2_approx(v2 - s0), p3 = ex2_approx(v3 - s1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        // P to bf16 for the product, as in the other attention kernels; the sums keep fp32
        const uint32_t b_lo = transpose8x8(pack_bf16(p0, p1)), b_hi = transpose8x8(pack_bf16(p2, p3));
        if (!__all_sync(0xffffffffu, mbar_wait_suspend(&v_full[st], ph, abort_flag))) { ok = false; break; }
        if (valid < RG_KEYS) {  // value rows behind the run may hold anything: 0 * NaN must not reach O
            for (int e = lane; e < (RG_KEYS - valid) * (DH / 8); e += 32) {
                const int r = valid + e / (DH / 8), piece = e % (DH / 8);
                *reinterpret_cast<uint4*>(ring_p + (rg_addr(va, r, piece) - ring_a)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();  // the ring's next copy comes after these stores
            __syncwarp();
        }
        const int vrow = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
        for (int t = 0; t < DH / 16; ++t) {
            uint32_t f[4];
            ldsm4_trans(rg_addr(va, vrow, 2 * t + ((lane >> 3) & 1)), f);
            mma_keys(o[t], f, b_lo, b_hi);
        }
        __syncwarp();
        if (lane == 0 && k_ahead) load_v(i + ST);
        k_ahead = false;
    }
    if (!ok) {  // give up: wait, bounded, for the copies still on their way
        *abort_flag = 1;
        if (a.err && lane == 0) atomicOr(a.err, ERR_TIMEOUT);
        int never = 0;
        for (int r = i; r < min(i + ST, mine); ++r) mbar_wait_suspend(&v_full[r % ST], (r / ST) & 1, &never);
        for (int r = i; r < min(i + ST + 1, mine); ++r)
            if (r < i + ST || k_ahead) mbar_wait_suspend(&k_full[r % ST], (r / ST) & 1, &never);
    }
#pragma unroll
    for (int s = 4; s < 32; s <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, s);
        l1 += __shfl_xor_sync(0xffffffffu, l1, s);
    }
    __syncthreads();  // the rings are done: their first bytes take the warps' results
    // the warps' partial results
#pragma unroll
    for (int t = 0; t < DH / 16; ++t) {
        const int dim = t * 16 + gq;
        so[warp][2 * tq][dim] = o[t][0];
        so[warp][2 * tq + 1][dim] = o[t][1];
        so[warp][2 * tq][dim + 8] = o[t][2];
        so[warp][2 * tq + 1][dim + 8] = o[t][3];
    }
    if (gq == 0) {
        sm[warp][2 * tq] = m0;
        sm[warp][2 * tq + 1] = m1;
        sl[warp][2 * tq] = l0;
        sl[warp][2 * tq + 1] = l1;
    }
    __syncthreads();
    // four dims of one head per thread and step, the group's heads fastest
    const int quads = a.G * (DH / 4);
    const bool alone = a.C == 1 && a.nrec == 0;
    float* own = a.own ? a.own + ((size_t)b * a.Hkv + j) * a.G * (DH + 4) : nullptr;
    if (a.C > 1) cluster_wait();
    for (int e = threadIdx.x; e < quads; e += THREADS) {  // join the warps
        int h, dd;
        quad_of(a, e, h, dd);
        float M = sm[0][h], L = 0.f;
#pragma unroll
        for (int w = 1; w < NW; ++w) M = fmaxf(M, sm[w][h]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = sm[w][h] == -INFINITY ? 0.f : ex2_approx(sm[w][h] - M);
            const float4 x = *reinterpret_cast<const float4*>(&so[w][h][dd]);
            L = fmaf(sl[w][h], f, L);
            v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
        }
        if (own) {
            *reinterpret_cast<float4*>(own + h * (DH + 4) + dd) = v;
            if (dd == 0) *reinterpret_cast<float2*>(own + h * (DH + 4) + DH) = make_float2(M, L);
        } else if (alone) {
            store_quad<DH>(a, b, j, h, dd, v, L == 0.f ? 0.f : 1.f / L);  // no visible key: zeros
        } else if (a.C > 1) {
            const int owner = e & (a.C - 1), slot = e - owner + rank;
            st_cluster_f32x4(cluster_addr(&js.cluster.sums[slot], owner), v);
            st_cluster_f32x2(cluster_addr(&js.cluster.stat[slot], owner), make_float2(M, L));
        } else {
            *reinterpret_cast<float4*>(&so[0][h][dd]) = v;
            if (dd == 0) {
                cm[h] = M;
                cl[h] = L;
            }
        }
    }
    if (own) {
        // The join is a launch of its own, which waits for this one only: this one must not end before the
        // prefix kernel has.
        if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) pdl_wait();
        return;
    }
    if (alone) return;
    // join the cluster's CTAs and the prefix records
    if (a.nrec > 0) {
        pdl_wait();  // the prefix kernel's records
        pdl_trigger();
    }
    if (a.C > 1) {
        cluster_sync();
        join_cluster<DH>(a, b, j, rank, js);
    } else {
        __syncthreads();
        join_records<DH>(
            a, b, j, js, [&](int h) { return make_float2(cm[h], cl[h]); },
            [&](int h, int dd) { return *reinterpret_cast<const float4*>(&so[0][h][dd]); });
    }
}

// The own keys' results (attn_ranges_kernel with a.own) and the prefix records of one (sequence, kv head).
template <int DH>
__global__ void __launch_bounds__(RG_THREADS) attn_join_kernel(const RangeArgs a) {
    __shared__ JoinShared js;
    const int j = blockIdx.x, b = blockIdx.y;
    const float* own = a.own + ((size_t)b * a.Hkv + j) * a.G * (DH + 4);
    pdl_trigger();
    pdl_wait();
    join_records<DH>(
        a, b, j, js, [&](int h) { return __ldcg(reinterpret_cast<const float2*>(own + h * (DH + 4) + DH)); },
        [&](int h, int dd) { return __ldcg(reinterpret_cast<const float4*>(own + h * (DH + 4) + dd)); });
}

// Whether an own CTA for every (sequence, kv head) can run on the SMs that the prefix kernel leaves.
bool fits_beside_prefix(int B, int Hkv, int free_sms) {
    return (long long)B * Hkv <= (long long)free_sms * RG_CTAS;
}

// CTAs per (sequence, kv head). Clusters of up to four CTAs while all CTAs fit the GPU (four an SM), of eight while they
// are two an SM at most and of sixteen while they are one, since larger clusters wait for room in one part of the GPU; each
// warp keeps a 16-key unit, two once there is a CTA for every SM and in clusters of sixteen, eight past two CTAs an SM.
// Measured (us, caches from HBM, 8 kv heads, dh 128): 1 sequence of 4096 keys by 8 CTAs 10.7, by 16 8.3; 4 by 8 15.0, by 16 17.5;
// 8 of 1024 keys by 4 9.7, by 8 10.1; 16 of 4096 by 2 44.1, by 4 42.4; 32 of 4096 by 1 82.2, by 2 79.9; 1 of 1024 by 8 4.7, by 16
// 4.9; 32 of 256 by 1 8.9, by 2 10.0. Beside a prefix kernel: two CTAs an SM at most, since they cannot all start
// before its CTAs end.
int ranges_cluster(int B, int Hkv, int max_keys, bool beside) {
    const long long sms = device_sm_count();
    int c = 1;
    while (c < RG_MAX_CLUSTER) {
        const int d = 2 * c;
        const long long ctas = (long long)B * Hkv * d;
        if (ctas > (beside || d == 8 ? 2 * sms : d < 8 ? 4 * sms : sms)) break;
        const int units = beside ? 1 : ctas > 2 * sms ? 8 : d == 16 || ctas > sms ? 2 : 1;
        if (max_keys < d * RG_WARPS * RG_KEYS * units) break;
        c = d;
    }
    return c;
}

struct Prefix {
    const __nv_bfloat16 *k, *v;
    int cap;
};

template <int DH, bool SINKS>
cudaError_t ranges_launch_dh(RangeArgs a, const __nv_bfloat16* k, const __nv_bfloat16* v, const Prefix& p, int B,
                             int max_keys, int free_sms, cudaStream_t st) {
    CUtensorMap maps[4];  // K and V of the caches and of the prefix
    const uint64_t heads = (uint64_t)B * a.Hkv;
    if (!encode_tmap_bf16_units(&maps[0], k, DH, a.cap, a.cap, heads, RG_KEYS) ||
        !encode_tmap_bf16_units(&maps[1], v, DH, a.cap, a.cap, heads, RG_KEYS))
        return cudaErrorInvalidValue;
    if (a.P == 0) {
        maps[2] = maps[0];
        maps[3] = maps[1];
    } else if (!encode_tmap_bf16_units(&maps[2], p.k, DH, a.P, p.cap, a.Hkv, RG_KEYS) ||
               !encode_tmap_bf16_units(&maps[3], p.v, DH, a.P, p.cap, a.Hkv, RG_KEYS)) {
        return cudaErrorInvalidValue;
    }
    a.C = ranges_cluster(B, a.Hkv, max_keys, a.nrec > 0);
    while (1 << a.log_c < a.C) ++a.log_c;
    a.inv_g = 65536u / a.G + 1;
    a.tile_seqs = kPrefixRows / a.G;
    // Own CTAs that cannot all run beside the prefix kernel would keep the others out while they wait for its
    // records: their results then go through memory to a launch that joins them.
    if (a.nrec == 0 || a.C > 1 || fits_beside_prefix(B, a.Hkv, free_sms)) a.own = nullptr;
    const cudaError_t e = launch_pdl_cluster(attn_ranges_kernel<DH, SINKS>, dim3(a.C, a.Hkv, B), dim3(RG_THREADS), a.C,
                                             RgLayout<DH>::SMEM, st, maps[0], maps[1], maps[2], maps[3], a);
    if (e != cudaSuccess || !a.own) return e;
    return launch_pdl(attn_join_kernel<DH>, dim3(a.Hkv, B), dim3(RG_THREADS), 0, st, a);
}

template <bool SINKS>
cudaError_t ranges_launch(const RangeArgs& a, const __nv_bfloat16* k, const __nv_bfloat16* v, const Prefix& p, int B, int dh,
                          int max_keys, int free_sms, cudaStream_t st) {
    if (dh == 128) return ranges_launch_dh<128, SINKS>(a, k, v, p, B, max_keys, free_sms, st);
    if (dh == 64) return ranges_launch_dh<64, SINKS>(a, k, v, p, B, max_keys, free_sms, st);
    return cudaErrorInvalidValue;
}

// Clusters of sixteen CTAs are beyond the portable size.
template <int DH, bool SINKS>
cudaError_t ranges_prepare() {
    const void* f = (const void*)attn_ranges_kernel<DH, SINKS>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, RgLayout<DH>::SMEM);
}

// Key chunks of the prefix. The prefix kernel runs one CTA an SM, the own keys' CTAs run on the SMs it leaves, so
// fewer chunks than SMs can pay: the estimate (us, on the measured rates) is the prefix kernel's time or, if it is
// longer, the time to read everything, plus what is left of the own keys when the prefix kernel ends.
// An item of the prefix kernel takes 0.9 us a key tile (its softmax warps), more when all of them together would read
// more than 5 TB/s (the row tiles of a chunk share its keys), and 4.5 us for its start and end; an SM's own CTAs read
// 55 GB/s; a join launch takes 2.5 us, records past the eighth 0.5 us each (they are not read ahead); half of the own
// cache is taken to be filled. Measured (us, dh 128, 8 kv heads): 64 sequences, 32768 keys, 32 heads, 512 own keys on average,
// 6 chunks 47, 9 chunks 53; 4096 keys, 16 heads, 256 own keys, 3 chunks 14.5, 19 chunks 23.6; 16 sequences, 8192 keys, 32 heads,
// 8 chunks 12.9, 13 chunks 15.7; 8 sequences, 32768 keys, 9 chunks 30.3, 16 chunks 31.5, 5 chunks 44.
constexpr int kPrefixMaxRounds = 2;
int prefix_max_chunks(int B, int Hq, int Hkv, int P) {
    const long long tiles = (P + 127ll) / 128, items = (long long)prefix_row_tiles(B, Hq / Hkv) * Hkv;
    return (int)std::max<long long>(
        1, std::min<long long>(std::min<long long>(tiles, kPrefixMaxChunks), kPrefixMaxRounds * device_sm_count() / items));
}
int prefix_chunks(int B, int Hq, int Hkv, int dh, int P, int own_cap) {
    const int row_tiles = prefix_row_tiles(B, Hq / Hkv), sms = device_sm_count();
    const long long tiles = (P + 127ll) / 128, items = (long long)row_tiles * Hkv;
    constexpr double hbm = 6.8e6, prefix_hbm = 5.0e6, sm_rate = 0.055e6;  // bytes per us
    const double own = (double)B * Hkv * (own_cap / 2.0) * dh * 4, tile = 128.0 * dh * 4;
    const int max_chunks = prefix_max_chunks(B, Hq, Hkv, P);
    int best = 1;
    double best_t = 0;
    for (int c = 1; c <= max_chunks; ++c) {
        const long long n = items * c, rounds = (n + sms - 1) / sms;
        const double running = (double)std::min<long long>(n, sms);
        const double per_tile = std::max(0.9, running / row_tiles * tile / prefix_hbm);
        const double t_prefix = rounds * (((tiles + c - 1) / c) * per_tile + 4.5);
        const double rate = n < sms ? std::min(hbm, (sms - n) * sm_rate) : 0;
        const bool join = !fits_beside_prefix(B, Hkv, (int)std::max<long long>(0, sms - n));
        const double t = std::max(t_prefix + std::max(0.0, own - rate * t_prefix) / hbm, (own + Hkv * tiles * tile) / hbm) +
                         0.05 * c + 0.5 * std::max(0, c - 8) + (join ? 2.5 : 0);
        if (c == 1 || t < best_t) {
            best_t = t;
            best = c;
        }
    }
    return best;
}

// Whether every sequence reads the prefix (if there is one) for itself, in one launch: little to read again (from L2, about 10 TB/s) costs
// less than the prefix kernel and its records. Measured (us, here against with records; 16 query heads, 8 kv heads, dh 128,
// own caches of 64 slots): 1 sequence, 600 keys 4.3 / 7.3, 4096 6.7 / 9.9; 2 at 4096 8.5 / 10.0; 16 at 600 7.0 / 7.4; 8 at 2048
// 8.8 / 8.3. Where the own keys already fill the GPU the second reading is not hidden: 64 sequences, 128 keys, 512 own
// slots 10.8 / 10.5, 64 own slots 5.8 / 7.3. And the host has one launch to make: 9.4 us a call against 12.
bool prefix_read_by_each(int B, int Hkv, int P, int own_cap) {
    const long long pairs = (long long)B * Hkv;
    return P == 0 || (pairs * P <= 1 << 16 && pairs * (P + own_cap / 2ll) <= 1 << 17);
}

}  // namespace

// The prefix records, then the own keys' results.
size_t attn_decode_shared_workspace(int B, int Hq, int Hkv, int dh, int prefix_len) {
    if (prefix_len <= 0) return 0;
    const size_t recs = prefix_rec_floats(dh) * prefix_row_tiles(B, Hq / Hkv) * Hkv * prefix_max_chunks(B, Hq, Hkv, prefix_len);
    return (recs + (size_t)B * Hq * (dh + 4)) * sizeof(float);
}

cudaError_t attn_decode_shared_launch(const __nv_bfloat16* q, const __nv_bfloat16* kp, const __nv_bfloat16* vp,
                                      int prefix_cap, int P, const __nv_bfloat16* kc, const __nv_bfloat16* vc, int B,
                                      int Hq, int Hkv, int dh, int cap, const int* len0, int len_stride, const int* meta,
                                      float* work, __nv_bfloat16* out, int* err, cudaStream_t st) {
    if (B <= 0) return cudaSuccess;
    RangeArgs a{};
    a.q = q;
    a.out = out;
    a.len0 = len0;
    a.len_stride = len_stride;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.cap = cap;
    a.meta = meta;
    int free_sms = 0;
    const int own_cap = meta ? std::max(0, cap - P) : cap;  // with a layout the first slots are the prefix
    if (prefix_read_by_each(B, Hkv, P, own_cap)) {
        a.P = P;
    } else {
        a.nrec = prefix_chunks(B, Hq, Hkv, dh, P, own_cap);
        a.row_tiles = prefix_row_tiles(B, a.G);
        a.recs = work;
        a.own = work + prefix_rec_floats(dh) * a.row_tiles * Hkv * a.nrec;
        free_sms = (int)std::max<long long>(0, device_sm_count() - (long long)a.row_tiles * Hkv * a.nrec);
        const cudaError_t e = attn_prefix_launch(q, kp, vp, B, Hq, Hkv, dh, prefix_cap, P, a.nrec, work, err, st);
        if (e != cudaSuccess) return e;
    }
    a.err = err;
    return ranges_launch<false>(a, kc, vc, Prefix{kp, vp, prefix_cap}, B, dh, (int)std::min(cap + (long long)a.P, 1ll << 30),
                                free_sms, st);
}

cudaError_t attn_decode_sinks_launch(const __nv_bfloat16* q, const __nv_bfloat16* kc, const __nv_bfloat16* vc, int B, int Hq,
                                     int Hkv, int dh, int cap, const int* len0, int len_stride, SinkMap sm,
                                     __nv_bfloat16* out, int* err, cudaStream_t st) {
    if (B <= 0) return cudaSuccess;
    RangeArgs a{};
    a.q = q;
    a.out = out;
    a.len0 = len0;
    a.len_stride = len_stride;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.cap = cap;
    a.window = sm.window;
    a.sinks = sm.sinks;
    a.sink_rows = sm.sink_rows;
    a.ring = sm.ring;
    a.err = err;
    return ranges_launch<true>(a, kc, vc, Prefix{}, B, dh, (int)std::min<long long>((long long)sm.window + sm.sinks, cap), 0,
                               st);
}

cudaError_t attention_ranges_prepare() {
    cudaError_t (*const prepare[])() = {
        ranges_prepare<128, false>, ranges_prepare<128, true>, ranges_prepare<64, false>, ranges_prepare<64, true>};
    for (auto f : prepare) {
        cudaError_t e = f();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q3
