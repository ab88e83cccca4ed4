// Decode attention over key ranges: a sliding window with sink tokens, and a batch that shares a prefix.
//
// attn_ranges_kernel serves one query per (sequence, query head) over the visible keys of its sequence; a
// cluster of CTAs shares the keys of one (sequence, kv head). The prefix form of the persistent prefill kernel
// computes the part of a shared prefix for the query rows of the whole batch at once and leaves one partial
// result per query row and key chunk, which attn_ranges_kernel joins to the sequence's own keys.
#include <algorithm>

#include <cstdlib>

#include "common.cuh"
#include "internal.h"

namespace q3 {
namespace {

// ------------------------------------------------------------------------------------- own keys
// O = sum_i p_i v_i / sum_i p_i, p_i = 2^(q k_i log2(e) / sqrt(dh) - m) over the visible keys i: up to three
// runs of cache rows (sinks, window, the wrapped part of a rolling buffer; or the own slots before and
// behind a padding block), taken in units of 16 keys.
//
// Every warp works through its own units alone, with a running maximum (lazily rescaled, as in the prefill
// kernels): its lane 0 keeps a ring of RG_BYTES full with the K and V boxes of the coming units (TMA, 128-byte
// swizzle), so 24 KB a warp and 192 KB an SM are on their way or in use, four times what HBM latency x
// bandwidth needs, and no barrier joins the warps before the end. The products are warp-level mma (m16n8k16,
// bf16 in, fp32 accumulate; the contraction is far below a tcgen05 tile) with the heads of the kv group as
// the 8 columns: S^T (keys x heads) = K q^T, P^T from accumulator to operand layout by a register transpose
// (movmatrix), O^T (head_dim x heads) += V^T P^T.
// Scores of rows behind a run are masked, and their value rows are zeroed in shared memory, so nothing
// stored in a hidden row can reach the result.
constexpr int RG_KEYS = 16, RG_MAX_CLUSTER = 16, RG_MAX_G = 8, RG_WARPS = 4, RG_THREADS = 32 * RG_WARPS;
constexpr int RG_BYTES = 24576;  // ring of one warp
template <int DH>
struct RgLayout {
    static constexpr int NCH = DH / 64;               // 64-column boxes of a row
    static constexpr int BOX = RG_KEYS * 128;         // bytes of a box
    static constexpr int HALF = NCH * BOX;            // K (or V) of a unit
    static constexpr int ST = RG_BYTES / (2 * HALF);  // units in the ring: 3 (dh 128) or 6 (dh 64)
    static constexpr int SMEM = RG_WARPS * RG_BYTES + 1024;
};
// two CTAs an SM; the warps' results take the first 16 KB of the rings once all of them are done
static_assert(2 * (RG_WARPS * RG_BYTES + 1024 + 8192) <= 227 * 1024, "shared memory");

struct RangeArgs {
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    const int* len0;
    int len_stride;
    int Hq, Hkv, G, cap;
    // window and sinks; ring > 0: rows [0, sink_rows) keep the first slots, the others wrap over ring rows
    int window, sinks, sink_rows, ring;
    const int* meta;    // own slots of a shared prefix: SeqMap::meta, or null
    const float* recs;  // [B * Hq][nrec][DH + 4] partial results to join (output sums, maximum, sum)
    int nrec;
    int C;  // CTAs per (sequence, kv head)
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
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// 16-byte piece `piece` (8 columns) of row `row` in boxes of 16 rows x 128 bytes written with the 128-byte swizzle
__device__ __forceinline__ uint32_t rg_addr(uint32_t base, int row, int piece) {
    return base + (uint32_t)((piece >> 3) * RG_KEYS * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

template <int DH, bool SINKS>
__global__ void __launch_bounds__(RG_THREADS, 2)
    attn_ranges_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const RangeArgs a) {
    using Ly = RgLayout<DH>;
    constexpr int NW = RG_WARPS, THREADS = RG_THREADS, ST = Ly::ST;
    constexpr int MAX_PARTS = RG_MAX_CLUSTER + kPrefixMaxChunks;
    extern __shared__ uint8_t rg_raw[];
    const uint32_t raw_addr = smem_u32(rg_raw);
    uint8_t* rings = rg_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    auto so = reinterpret_cast<float(*)[RG_MAX_G][DH]>(rings);  // the warps' output sums, once the rings are done
    __shared__ uint64_t bars[RG_WARPS][2 * ST];                 // [K of each stage, V of each stage]
    __shared__ float sm[NW][RG_MAX_G], sl[NW][RG_MAX_G];
    __shared__ float cm[RG_MAX_G], cl[RG_MAX_G];                   // this CTA's maximum and sum
    __shared__ float pm[RG_MAX_G][MAX_PARTS], pl[RG_MAX_G][MAX_PARTS];  // of every part: CTAs, then prefix records
    __shared__ float inv[RG_MAX_G];
    __shared__ int abort_sh;
    volatile int* abort_flag = &abort_sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, tq = lane & 3;  // fragment coordinates
    const int rank = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
    uint64_t* k_full = bars[warp];
    uint64_t* v_full = bars[warp] + ST;
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
    const int u0 = (int)((long long)units * rank / a.C), u1 = (int)((long long)units * (rank + 1) / a.C);
    const int mine = u1 - u0 > warp ? (u1 - u0 - warp + NW - 1) / NW : 0;  // units u0 + warp + NW i

    uint8_t* ring_p = rings + warp * RG_BYTES;
    const uint32_t ring_a = smem_u32(ring_p);
    const int z = b * a.Hkv + j;
    auto load = [&](int i) {  // lane 0
        int valid;
        const int y = unit(u0 + warp + NW * i, valid), st = i % ST;
        uint8_t* dst = ring_p + st * 2 * Ly::HALF;
        mbar_expect_tx(&k_full[st], Ly::HALF);
#pragma unroll
        for (int c = 0; c < Ly::NCH; ++c) tma_load_3d(dst + c * Ly::BOX, &tmK, &k_full[st], c * 64, y, z);
        mbar_expect_tx(&v_full[st], Ly::HALF);
#pragma unroll
        for (int c = 0; c < Ly::NCH; ++c)
            tma_load_3d(dst + Ly::HALF + c * Ly::BOX, &tmV, &v_full[st], c * 64, y, z);
    };
    if (lane == 0)
        for (int i = 0; i < min(ST, mine); ++i) load(i);

    const float sl2 = kLog2e / sqrtf((float)DH);
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2 tq and 2 tq + 1
    float o[DH / 16][4];                                       // tile t: rows are dims 16 t + gq and 16 t + gq + 8
#pragma unroll
    for (int t = 0; t < DH / 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    bool ok = true;
    int i = 0;
    for (; i < mine; ++i) {
        const int st = i % ST, ph = (i / ST) & 1;
        int valid;
        unit(u0 + warp + NW * i, valid);
        const uint32_t ka = ring_a + st * 2 * Ly::HALF, va = ka + Ly::HALF;
        if (!__all_sync(0xffffffffu, mbar_wait_suspend(&k_full[st], ph, abort_flag))) { ok = false; break; }
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int ks = 0; ks < DH / 16; ++ks) {
            uint32_t f[4];
            ldsm4(rg_addr(ka, krow, 2 * ks + (lane >> 4)), f);
            mma_keys(d, f, qf[ks][0], qf[ks][1]);
        }
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
        __syncwarp();  // every lane has read the stage
        if (lane == 0 && i + ST < mine) load(i + ST);
    }
    if (!ok) {  // give up: wait, bounded, for the copies still on their way
        *abort_flag = 1;
        if (a.err && lane == 0) atomicOr(a.err, ERR_TIMEOUT);
        int never = 0;
        for (int r = i; r < min(i + ST, mine); ++r) {
            mbar_wait_suspend(&k_full[r % ST], (r / ST) & 1, &never);
            mbar_wait_suspend(&v_full[r % ST], (r / ST) & 1, &never);
        }
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
    // four dims of one head per thread and step
    const int quads = a.G * (DH / 4);
    const bool alone = a.C == 1 && a.nrec == 0;
    auto store = [&](int h, int dd, float4 v, float scale) {
        const size_t row = (size_t)b * a.Hq + (size_t)j * a.G + h;
        *reinterpret_cast<uint2*>(a.out + row * DH + dd) =
            make_uint2(pack_bf16(v.x * scale, v.y * scale), pack_bf16(v.z * scale, v.w * scale));
    };
    for (int e = threadIdx.x; e < quads; e += THREADS) {  // join the warps
        const int h = e / (DH / 4), dd = e % (DH / 4) * 4;
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
        if (alone) {
            store(h, dd, v, L == 0.f ? 0.f : 1.f / L);  // no visible key: zeros
        } else {
            *reinterpret_cast<float4*>(&so[0][h][dd]) = v;
            if (dd == 0) {
                cm[h] = M;
                cl[h] = L;
            }
        }
    }
    if (alone) return;
    // join the cluster's CTAs and the prefix records; each CTA finishes a share of the output
    if (a.C > 1) {
        cluster_sync();
    } else {
        __syncthreads();
    }
    if (a.nrec > 0) {
        pdl_wait();  // the prefix kernel's partial results
        pdl_trigger();
    }
    const int parts = a.C + a.nrec;
    const float* rec0 = a.recs + ((size_t)b * a.Hq + (size_t)j * a.G) * a.nrec * (DH + 4);
    for (int e = threadIdx.x; e < parts * RG_MAX_G; e += THREADS) {
        const int p = e / RG_MAX_G, h = e % RG_MAX_G;
        if (h < a.G) {
            if (p < a.C) {
                pm[h][p] = ld_cluster_f32(cluster_addr(&cm[h], p));
                pl[h][p] = ld_cluster_f32(cluster_addr(&cl[h], p));
            } else {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(
                    rec0 + ((size_t)h * a.nrec + p - a.C) * (DH + 4) + DH));
                pm[h][p] = ml.x;
                pl[h][p] = ml.y;
            }
        }
    }
    __syncthreads();
    for (int h = warp; h < a.G; h += NW) {  // the parts' weights, into pm
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
    for (int e = threadIdx.x + THREADS * rank; e < quads; e += THREADS * a.C) {
        const int h = e / (DH / 4), dd = e % (DH / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4& x, float f) {
            v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
        };
        if (a.C == 1) {
            add(*reinterpret_cast<const float4*>(&so[0][h][dd]), pm[h][0]);
        } else {
#pragma unroll 4
            for (int p = 0; p < a.C; ++p) add(ld_cluster_f32x4(cluster_addr(&so[0][h][dd], p)), pm[h][p]);
        }
        const float* rec = rec0 + (size_t)h * a.nrec * (DH + 4) + dd;
#pragma unroll 8
        for (int r = 0; r < a.nrec; ++r)
            add(__ldcg(reinterpret_cast<const float4*>(rec + (size_t)r * (DH + 4))), pm[h][a.C + r]);
        store(h, dd, v, inv[h]);
    }
    if (a.C > 1) cluster_sync();  // every CTA's partial stays in shared memory until the others have read it
}

// CTAs per (sequence, kv head): as many as two CTAs on every SM take, while each warp keeps a 16-key unit.
int ranges_cluster(int B, int Hkv, int max_keys) {
    int c = 1;
    while (c < RG_MAX_CLUSTER && (long long)B * Hkv * c * 2 <= 2 * device_sm_count() &&
           max_keys >= 2 * c * RG_WARPS * RG_KEYS)
        c *= 2;
    if (getenv("Q3_C")) c = atoi(getenv("Q3_C"));
    return c;
}

template <int DH, bool SINKS>
cudaError_t ranges_launch_dh(RangeArgs a, const __nv_bfloat16* k, const __nv_bfloat16* v, int B, int max_keys,
                             cudaStream_t st) {
    CUtensorMap tk, tv;
    const uint64_t heads = (uint64_t)B * a.Hkv;
    if (!encode_tmap_bf16_rows(&tk, k, DH, a.cap, a.cap, heads, RG_KEYS) ||
        !encode_tmap_bf16_rows(&tv, v, DH, a.cap, a.cap, heads, RG_KEYS))
        return cudaErrorInvalidValue;
    a.C = ranges_cluster(B, a.Hkv, max_keys);
    return launch_pdl_cluster(attn_ranges_kernel<DH, SINKS>, dim3(a.C, a.Hkv, B), dim3(RG_THREADS), a.C,
                              RgLayout<DH>::SMEM, st, tk, tv, a);
}

template <bool SINKS>
cudaError_t ranges_launch(const RangeArgs& a, const __nv_bfloat16* k, const __nv_bfloat16* v, int B, int dh, int max_keys,
                          cudaStream_t st) {
    if (dh == 128) return ranges_launch_dh<128, SINKS>(a, k, v, B, max_keys, st);
    if (dh == 64) return ranges_launch_dh<64, SINKS>(a, k, v, B, max_keys, st);
    return cudaErrorInvalidValue;
}

// Clusters of sixteen CTAs are beyond the portable size.
template <int DH, bool SINKS>
cudaError_t ranges_prepare() {
    cudaError_t e = cudaFuncSetAttribute(attn_ranges_kernel<DH, SINKS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(attn_ranges_kernel<DH, SINKS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                RgLayout<DH>::SMEM);
}

}  // namespace

size_t attn_decode_shared_workspace(int B, int Hq, int Hkv, int dh, int prefix_len) {
    if (prefix_len <= 0) return 0;
    return (size_t)B * Hq * attn_prefix_chunks(B, Hq, Hkv, prefix_len) * (dh + 4) * sizeof(float);
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
    if (P > 0) {
        a.recs = work;
        a.nrec = attn_prefix_chunks(B, Hq, Hkv, P);
        const cudaError_t e = attn_prefix_launch(q, kp, vp, B, Hq, Hkv, dh, prefix_cap, P, work, err, st);
        if (e != cudaSuccess) return e;
    }
    a.err = err;
    return ranges_launch<false>(a, kc, vc, B, dh, cap, st);
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
    return ranges_launch<true>(a, kc, vc, B, dh, (int)std::min<long long>((long long)sm.window + sm.sinks, cap), st);
}

cudaError_t attention_ranges_prepare() {
    cudaError_t (*const prepare[])() = {ranges_prepare<128, false>, ranges_prepare<128, true>, ranges_prepare<64, false>,
                                        ranges_prepare<64, true>};
    for (auto f : prepare) {
        cudaError_t e = f();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q3
