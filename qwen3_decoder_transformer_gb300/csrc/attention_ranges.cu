// Decode attention over key ranges: a sliding window with sink tokens, and a batch that shares a prefix.
//
// attn_ranges_kernel serves one query per (sequence, query head) over the visible keys of its sequence; a
// cluster of CTAs shares the keys of one (sequence, kv head). attn_prefix_kernel computes the part of a
// shared prefix for the query rows of the whole batch at once and leaves one partial result per query row
// and key chunk, which attn_ranges_kernel joins to the sequence's own keys.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace q3 {
namespace {

// ------------------------------------------------------------------------------------- own keys
// O = sum_i p_i v_i / sum_i p_i, p_i = 2^(q k_i log2(e) / sqrt(dh) - m) over the visible keys i, which are
// numbered 0 .. total-1 across two slot ranges [a0, a0 + na) and [b0, b0 + nb): sinks and window, or the own
// slots before and behind a padding block. Only visible rows are ever read (the numbers past the end repeat
// the last key with weight 0), so nothing stored in a hidden row can reach the result.
//
// A warp takes 16 keys at a time straight from global memory into the fragments of warp-level mma
// (m16n8k16, bf16 in, fp32 accumulate), heads of the kv group as the 8 columns:
//   S^T (keys x heads) = K q^T: the lane of key row g loads 16-byte pieces 4c + t of its row; the inner
//   index of a product may be permuted freely, and q is loaded with the same permutation;
//   P^T moves from accumulator to operand layout by a register transpose (movmatrix);
//   O^T (head_dim x heads) += V^T P^T: the lane pairs the 16-bit halves of its four key rows.
// No shared memory, barrier or tensor map stands between HBM and the products, and warps run
// independently with a running maximum each (lazily rescaled, as in the prefill kernels). 16 warps an SM hold
// two 4 KB loads each in flight, about twice what HBM latency x bandwidth needs.
constexpr int RG_WARPS = 8, RG_THREADS = 32 * RG_WARPS, RG_KEYS = 16, RG_MAX_CLUSTER = 8, RG_MAX_G = 8;

struct RangeArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* out;
    const int* len0;
    int len_stride;
    int Hq, Hkv, G, cap;
    // window and sinks; ring > 0: rows [0, sink_rows) keep the first slots, the others wrap over ring rows
    int window, sinks, sink_rows, ring;
    const int* meta;    // own slots of a shared prefix: SeqMap::meta, or null
    const float* recs;  // [B * Hq][nrec][DH + 4] partial results to join (output floats, maximum, sum)
    int nrec;
    int C;  // CTAs per (sequence, kv head)
};

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
__device__ __forceinline__ void mma_keys(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int DH, bool SINKS>
__global__ void __launch_bounds__(RG_THREADS, 2) attn_ranges_kernel(const RangeArgs a) {
    constexpr int KC = DH / 32;  // 16-byte pieces of a key row per lane
    constexpr int VC = DH / 64;  // 16-byte pieces of a value row per lane
    __shared__ float so[RG_WARPS][RG_MAX_G][DH];
    __shared__ float sm[RG_WARPS][RG_MAX_G], sl[RG_WARPS][RG_MAX_G], sf[RG_WARPS][RG_MAX_G];
    __shared__ float cm[RG_MAX_G], cl[RG_MAX_G];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, tq = lane & 3;  // fragment coordinates
    const int rank = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
    // Without partial results to join this is an ordinary dependent launch. With them, the prefix kernel
    // before it has itself waited for everything earlier before it let this kernel start, and only the
    // join below has to wait for the prefix kernel.
    if (a.nrec == 0) {
        pdl_wait();
        pdl_trigger();
    }
    int n = __ldcg(a.len0 + (size_t)b * a.len_stride);
    n = n < 0 ? 0 : min(n, 1 << 30) + 1;
    if (!SINKS || a.ring == 0) n = min(n, a.cap);
    int a0 = 0, na, b0, nb;
    if constexpr (SINKS) {
        b0 = max(0, n - a.window);
        nb = n - b0;
        na = min(a.sinks, b0);
    } else {
        int ps = 0, pe = 0, psh = 0;
        if (a.meta) {
            ps = __ldcg(a.meta);
            psh = __ldcg(a.meta + 1);
            pe = ps + __ldcg(a.meta + kSeqMetaHead + b);
        }
        a0 = min(max(psh, 0), n);
        const int a1 = min(max(ps, a0), n);
        na = a1 - a0;
        b0 = min(max(pe, a1), n);
        nb = n - b0;
    }
    const int total = na + nb;
    // rolling buffer: whole turns before the first slot of the second range
    int turns = 0;
    if (SINKS && a.ring > 0) turns = (max(b0, a.sink_rows) - a.sink_rows) / a.ring * a.ring;
    auto row_of = [&](int i) -> int {  // cache row of visible key i
        if (i < na) return a0 + i;
        int s = b0 + (i - na);
        if (SINKS && a.ring > 0 && s >= a.sink_rows) {
            s -= turns;
            if (s >= a.sink_rows + a.ring) s -= a.ring;
        }
        return s;
    };
    const int units = (total + RG_KEYS - 1) / RG_KEYS;
    const int u0 = (int)((long long)units * rank / a.C), u1 = (int)((long long)units * (rank + 1) / a.C);

    const __nv_bfloat16* kb = a.k + ((size_t)b * a.Hkv + j) * a.cap * DH;
    const __nv_bfloat16* vb = a.v + ((size_t)b * a.Hkv + j) * a.cap * DH;
    // q^T fragments: column gq = query head gq of the group (zero past G)
    uint4 qf[KC];
    {
        const __nv_bfloat16* qrow = a.q + ((size_t)b * a.Hq + (size_t)j * a.G + gq) * DH;
#pragma unroll
        for (int c = 0; c < KC; ++c)
            qf[c] = gq < a.G ? __ldcg(reinterpret_cast<const uint4*>(qrow) + c * 4 + tq) : make_uint4(0, 0, 0, 0);
    }
    uint4 kr[2][KC], vr[4][VC];
    // lane i < 16 works out the row of the unit's key i, the others take it from there
    auto unit_row = [&](int u) { return row_of(min(u * RG_KEYS + (lane & 15), total - 1)); };
    auto load_k = [&](int my_row) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = __shfl_sync(0xffffffffu, my_row, gq + 8 * r);
            const uint4* p = reinterpret_cast<const uint4*>(kb + (size_t)row * DH) + tq;
#pragma unroll
            for (int c = 0; c < KC; ++c) kr[r][c] = ld_stream16(p + c * 4);
        }
    };
    auto load_v = [&](int my_row) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = __shfl_sync(0xffffffffu, my_row, 2 * tq + (r & 1) + 8 * (r >> 1));
            const uint4* p = reinterpret_cast<const uint4*>(vb + (size_t)row * DH) + gq;
#pragma unroll
            for (int c = 0; c < VC; ++c) vr[r][c] = ld_stream16(p + c * 8);
        }
    };
    const float sl2 = kLog2e / sqrtf((float)DH);
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2 tq and 2 tq + 1
    float o[DH / 16][4];  // tile (c, w): rows gq and gq + 8 are dims c*64 + 8 gq + 2 w and the next one
#pragma unroll
    for (int t = 0; t < DH / 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    int u = u0 + warp;
    if (u < u1) {
        int my_row = unit_row(u);
        load_k(my_row);
        load_v(my_row);
        for (; u < u1; u += RG_WARPS) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                mma_keys(d, kr[0][c].x, kr[1][c].x, kr[0][c].y, kr[1][c].y, qf[c].x, qf[c].y);
                mma_keys(d, kr[0][c].z, kr[1][c].z, kr[0][c].w, kr[1][c].w, qf[c].z, qf[c].w);
            }
            const bool more = u + RG_WARPS < u1;
            if (more) {
                my_row = unit_row(u + RG_WARPS);
                load_k(my_row);
            }
            const int i0 = u * RG_KEYS + gq;
            const bool in0 = i0 < total, in1 = i0 + 8 < total;
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
            const float n0 = m0 == -INFINITY ? 0.f : m0, n1 = m1 == -INFINITY ? 0.f : m1;
            const float p0 = ex2_approx(v0 - n0), p1 = ex2_approx(v1 - n1);
            const float p2 = ex2_approx(v2 - n0), p3 = ex2_approx(v3 - n1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            // P to bf16 for the product, as in the other attention kernels; the sums keep fp32
            const uint32_t b_lo = transpose8x8(pack_bf16(p0, p1)), b_hi = transpose8x8(pack_bf16(p2, p3));
#pragma unroll
            for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t e0 = word(vr[0][c], w), e1 = word(vr[1][c], w), e2 = word(vr[2][c], w), e3 = word(vr[3][c], w);
                    mma_keys(o[c * 4 + w], __byte_perm(e0, e1, 0x5410), __byte_perm(e0, e1, 0x7632),
                             __byte_perm(e2, e3, 0x5410), __byte_perm(e2, e3, 0x7632), b_lo, b_hi);
                }
            if (more) load_v(my_row);
        }
    }
#pragma unroll
    for (int s = 4; s < 32; s <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, s);
        l1 += __shfl_xor_sync(0xffffffffu, l1, s);
    }
    // join the warps
#pragma unroll
    for (int t = 0; t < DH / 16; ++t) {
        const int dim = (t >> 2) * 64 + gq * 8 + (t & 3) * 2;
        *reinterpret_cast<float2*>(&so[warp][2 * tq][dim]) = make_float2(o[t][0], o[t][2]);
        *reinterpret_cast<float2*>(&so[warp][2 * tq + 1][dim]) = make_float2(o[t][1], o[t][3]);
    }
    if (gq == 0) {
        sm[warp][2 * tq] = m0;
        sm[warp][2 * tq + 1] = m1;
        sl[warp][2 * tq] = l0;
        sl[warp][2 * tq + 1] = l1;
    }
    __syncthreads();
    if (threadIdx.x < RG_MAX_G) {
        const int h = threadIdx.x;
        float M = sm[0][h], Lh = 0.f;
#pragma unroll
        for (int w = 1; w < RG_WARPS; ++w) M = fmaxf(M, sm[w][h]);
#pragma unroll
        for (int w = 0; w < RG_WARPS; ++w) {
            const float f = sm[w][h] == -INFINITY ? 0.f : ex2_approx(sm[w][h] - M);
            sf[w][h] = f;
            Lh = fmaf(sl[w][h], f, Lh);
        }
        cm[h] = M;
        cl[h] = Lh;
    }
    __syncthreads();
    const int elems = a.G * DH;
    if (a.C > 1) {
        for (int e = threadIdx.x; e < elems; e += RG_THREADS) {
            const int h = e / DH, dd = e % DH;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < RG_WARPS; ++w) v = fmaf(so[w][h][dd], sf[w][h], v);
            so[0][h][dd] = v;
        }
        cluster_sync();
    }
    if (a.nrec > 0) {
        pdl_wait();  // the prefix kernel's partial results
        pdl_trigger();
    }
    // join the cluster's CTAs and the prefix records; each CTA finishes a share of the output
    for (int e = threadIdx.x + RG_THREADS * rank; e < elems; e += RG_THREADS * a.C) {
        const int h = e / DH, dd = e % DH;
        const size_t row = (size_t)b * a.Hq + (size_t)j * a.G + h;
        const float* rec = a.recs + row * a.nrec * (DH + 4);
        float M = a.C > 1 ? -INFINITY : cm[h];
        if (a.C > 1)
            for (int c = 0; c < a.C; ++c) M = fmaxf(M, ld_cluster_f32(cluster_addr(&cm[h], c)));
        for (int r = 0; r < a.nrec; ++r) M = fmaxf(M, __ldcg(rec + (size_t)r * (DH + 4) + DH));
        float num = 0.f, den = 0.f;
        if (a.C > 1) {
            for (int c = 0; c < a.C; ++c) {
                const float mc = ld_cluster_f32(cluster_addr(&cm[h], c));
                const float f = mc == -INFINITY ? 0.f : ex2_approx(mc - M);
                den = fmaf(ld_cluster_f32(cluster_addr(&cl[h], c)), f, den);
                num = fmaf(ld_cluster_f32(cluster_addr(&so[0][h][dd], c)), f, num);
            }
        } else {
            const float f = cm[h] == -INFINITY ? 0.f : ex2_approx(cm[h] - M);
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < RG_WARPS; ++w) v = fmaf(so[w][h][dd], sf[w][h], v);
            den = cl[h] * f;
            num = v * f;
        }
        for (int r = 0; r < a.nrec; ++r) {
            const float* rc = rec + (size_t)r * (DH + 4);
            const float mc = __ldcg(rc + DH);
            const float f = mc == -INFINITY ? 0.f : ex2_approx(mc - M);
            den = fmaf(__ldcg(rc + DH + 1), f, den);
            num = fmaf(__ldcg(rc + dd), f, num);
        }
        a.out[row * DH + dd] = __float2bfloat16_rn(den == 0.f ? 0.f : num / den);  // no visible key: zeros
    }
    if (a.C > 1) cluster_sync();  // every CTA's partial stays in shared memory until the others have read it
}

// CTAs per (sequence, kv head): enough to give two CTAs to every SM, while each warp keeps a 16-key unit.
int ranges_cluster(int B, int Hkv, int max_keys) {
    int c = 1;
    while (c < RG_MAX_CLUSTER && (long long)B * Hkv * c * 2 <= 2 * device_sm_count() &&
           max_keys >= 2 * c * RG_WARPS * RG_KEYS)
        c *= 2;
    return c;
}

template <bool SINKS>
cudaError_t ranges_launch(const RangeArgs& a0, int B, int dh, int max_keys, cudaStream_t st) {
    RangeArgs a = a0;
    a.C = ranges_cluster(B, a.Hkv, max_keys);
    const dim3 grid(a.C, a.Hkv, B), block(RG_THREADS);
    if (dh == 128) return launch_pdl_cluster(attn_ranges_kernel<128, SINKS>, grid, block, a.C, 0, st, a);
    if (dh == 64) return launch_pdl_cluster(attn_ranges_kernel<64, SINKS>, grid, block, a.C, 0, st, a);
    return cudaErrorInvalidValue;
}

// ------------------------------------------------------------------------------------ shared prefix
// Flash attention of all the batch's query rows of one kv head against a chunk of the prefix keys, on the
// tensor cores (tcgen05, accumulators in tensor memory, operands by TMA). A tile of 128 rows holds the G
// query heads of floor(128 / G) sequences; a CTA serves NT tiles from one read of each key and value tile.
// K and V of the prefix are read once from HBM for up to 256 query rows, where the read (64 KB a 128-key tile,
// 1.5 us at an SM's share of HBM) still covers the products (0.55 us a row tile at the measured tensor rate).
// Roles as in the prefill kernel with a split key range: warp 0 TMA, warp 1 MMA, then four softmax warps
// per row tile, thread <-> query row. With one row tile the scores run a tile ahead in a second region;
// with two, one tile's scores are computed while the other's softmax runs.
constexpr int PX_BM = 128, PX_BN = 128;
template <int DH, int NT>
struct PxLayout {
    static constexpr int NCH = DH / 64;
    static constexpr int ST = NT == 1 ? 3 : 2;  // stages of the key ring and of the value ring
    static constexpr int Q_BYTES = PX_BM * DH * 2;
    static constexpr int KV_BYTES = PX_BN * DH * 2;
    static constexpr int K_OFF = NT * Q_BYTES;
    static constexpr int V_OFF = K_OFF + ST * KV_BYTES;
    static constexpr int BAR_OFF = V_OFF + ST * KV_BYTES;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
    static constexpr int THREADS = 64 + 128 * NT;
};
static_assert(PxLayout<128, 1>::SMEM <= 227 * 1024 && PxLayout<128, 2>::SMEM <= 227 * 1024, "shared memory");

template <int DH, int NT>
__global__ void __launch_bounds__(PxLayout<DH, NT>::THREADS, 1)
    attn_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, int B, int Hq, int G, int P, int row_blocks, int chunks,
                       float* __restrict__ recs, int* err) {
    using Ly = PxLayout<DH, NT>;
    constexpr int NCH = Ly::NCH, ST = Ly::ST;
    constexpr uint32_t IDESC_S = idesc_bf16(PX_BM, PX_BN);
    constexpr uint32_t IDESC_O = idesc_bf16(PX_BM, DH, true);
    constexpr uint32_t TM_O = 2 * PX_BN;  // O of row tile x at TM_O + 128 x
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::BAR_OFF);
    uint64_t* q_full = bars;
    uint64_t* k_full = bars + 1;   // [ST]
    uint64_t* v_full = bars + 4;   // [ST]
    uint64_t* k_empty = bars + 7;  // [ST]
    uint64_t* v_empty = bars + 10; // [ST]
    uint64_t* s_full = bars + 13;  // [2] per score region
    uint64_t* p_full = bars + 15;  // [2] per score region
    uint64_t* o_done = bars + 17;  // [NT]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 19);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 20);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rb = blockIdx.x % row_blocks, chunk = blockIdx.x / row_blocks % chunks;
    const int j = blockIdx.x / (row_blocks * chunks);
    const int spt = PX_BM / G;  // sequences per row tile
    const int tiles = (P + PX_BN - 1) / PX_BN;
    const int t0 = (int)((long long)tiles * chunk / chunks), nt = (int)((long long)tiles * (chunk + 1) / chunks) - t0;
    // the last row block may hold fewer row tiles
    const int live = min(NT, (B - rb * NT * spt + spt - 1) / spt);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
        }
        for (int x = 0; x < NT; ++x) mbar_init(&o_done[x], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    pdl_wait();
    pdl_trigger();
    // score region of row tile x at the CTA's key tile i, and how many earlier key tiles used it
    auto region = [](int x, int i) { return NT == 2 ? x : (i & 1); };
    auto uses = [](int i) { return NT == 2 ? i : (i >> 1); };

    if (warp == 0) {
        if (lane == 0) {
            mbar_expect_tx(q_full, live * NCH * spt * G * 128);
            for (int x = 0; x < live; ++x)
                for (int c = 0; c < NCH; ++c)
                    tma_load_4d(smem + x * Ly::Q_BYTES + c * PX_BM * 128, &tmQ, q_full, c * 64, 0, j, (rb * NT + x) * spt);
            for (int i = 0; i < nt; ++i) {
                const int s = i % ST, y = (t0 + i) * PX_BN;
                const uint32_t free_ph = ((i / ST) & 1) ^ 1;
                if (!mbar_wait_suspend(&k_empty[s], free_ph, abort_flag)) { ok = false; break; }
                mbar_expect_tx(&k_full[s], Ly::KV_BYTES);
                for (int c = 0; c < NCH; ++c)
                    tma_load_3d(smem + Ly::K_OFF + s * Ly::KV_BYTES + c * PX_BN * 128, &tmK, &k_full[s], c * 64, y, j);
                if (!mbar_wait_suspend(&v_empty[s], free_ph, abort_flag)) { ok = false; break; }
                mbar_expect_tx(&v_full[s], Ly::KV_BYTES);
                for (int c = 0; c < NCH; ++c)
                    tma_load_3d(smem + Ly::V_OFF + s * Ly::KV_BYTES + c * PX_BN * 128, &tmV, &v_full[s], c * 64, y, j);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            auto issue_s = [&](int x, int i) -> bool {
                const int s = i % ST, r = region(x, i);
                if (!mbar_wait_suspend(&k_full[s], (i / ST) & 1, abort_flag)) return false;
                tc_fence_after();
                const uint32_t sq = smem_u32(smem + x * Ly::Q_BYTES);
                const uint32_t sk = smem_u32(smem + Ly::K_OFF + s * Ly::KV_BYTES);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * PX_BM * 128 + (kk & 3) * 32;
                    umma_bf16_ss(tmem + r * PX_BN, sdesc_kmajor_sw128(sq + off), sdesc_kmajor_sw128(sk + off), IDESC_S,
                                 kk > 0);
                }
                umma_commit(&s_full[r]);
                if (x == live - 1) umma_commit(&k_empty[s]);
                return true;
            };
            ok = mbar_wait_suspend(q_full, 0, abort_flag);
            for (int x = 0; ok && x < live; ++x) ok = issue_s(x, 0);
            if (NT == 1 && ok && nt > 1) ok = issue_s(0, 1);
            for (int i = 0; ok && i < nt; ++i) {
                const int s = i % ST;
                if (!mbar_wait_suspend(&v_full[s], (i / ST) & 1, abort_flag)) { ok = false; break; }
                const uint32_t sv = smem_u32(smem + Ly::V_OFF + s * Ly::KV_BYTES);
                for (int x = 0; ok && x < live; ++x) {
                    const int r = region(x, i);
                    if (!mbar_wait_suspend(&p_full[r], uses(i) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < PX_BN / 16; ++kk) {
                        const uint64_t bd = sdesc_mnmajor_sw128(sv + kk * 16 * 128, PX_BN * 128);
                        umma_bf16_ts(tmem + TM_O + x * 128, tmem + r * PX_BN + kk * 8, bd, IDESC_O, (i | kk) != 0);
                    }
                    umma_commit(&o_done[x]);
                    if (x == live - 1) umma_commit(&v_empty[s]);
                    const int nxt = NT == 2 ? i + 1 : i + 2;  // the next key tile whose scores go to this region
                    if (nxt < nt) ok = issue_s(x, nxt);
                }
            }
        }
    } else if ((warp - 2) / 4 < live) {
        const int x = (warp - 2) >> 2;
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tm_o = tmem + lane_off + TM_O + x * 128;
        const float sl2 = kLog2e / sqrtf((float)DH);
        float m_used = -INFINITY, l = 0.f;
        int pv_seen = 0;
        auto confirm_pv = [&](int upto) -> bool {
            while (pv_seen < upto) {
                if (!mbar_wait_suspend(&o_done[x], pv_seen & 1, abort_flag)) return false;
                ++pv_seen;
            }
            return true;
        };
        for (int i = 0; i < nt; ++i) {
            const int r = region(x, i);
            const uint32_t tm_s = tmem + lane_off + r * PX_BN;
            if (!__all_sync(0xffffffffu, mbar_wait_suspend(&s_full[r], uses(i) & 1, abort_flag))) { ok = false; break; }
            tc_fence_after();
            uint32_t sr[PX_BN];
#pragma unroll
            for (int c = 0; c < PX_BN / 32; ++c)
                tmem_ld_32x32b_x32(tm_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
            tmem_ld_wait();
            const int left = P - (t0 + i) * PX_BN;  // keys of this tile
            if (left < PX_BN) {
#pragma unroll
                for (int e = 0; e < PX_BN; ++e) sr[e] = e < left ? sr[e] : __float_as_uint(-INFINITY);
            }
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < PX_BN; e += 2) mx = fmax3(mx, __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
            mx *= sl2;
            // lazy rescale, decided per row but executed by the whole warp (tcgen05.ld/st are warp-wide)
            const bool grow = mx > m_used + 8.0f;
            const float alpha = grow ? ex2_approx(m_used - mx) : 1.0f;
            if (i > 0 && __any_sync(0xffffffffu, grow)) {
                const bool w = confirm_pv(i);
                if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < DH / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tm_o + c * 32, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_st_32x32b_x32(tm_o + c * 32, o);
                }
                tmem_st_wait();
            }
            if (grow) {
                l *= alpha;
                m_used = mx;
            }
            const float nm = m_used == -INFINITY ? 0.f : -m_used;
            const float2 sl2x2 = make_float2(sl2, sl2), nmx2 = make_float2(nm, nm);
            float2 rs2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 z = fma2(make_float2(__uint_as_float(sr[half * 64 + 2 * e]),
                                                      __uint_as_float(sr[half * 64 + 2 * e + 1])),
                                          sl2x2, nmx2);
                    const float2 pp = make_float2(ex2_approx(z.x), ex2_approx(z.y));
                    rs2 = add2(rs2, pp);
                    pk[e] = pack_bf16(pp.x, pp.y);
                }
                tmem_st_32x32b_x32(tm_s + half * 32, pk);
            }
            tmem_st_wait();
            l += rs2.x + rs2.y;
            // see the previous P V complete before releasing this P: o_done then stays within one phase
            if (i > 0) {
                const bool w = confirm_pv(i);
                if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
            }
            tc_fence_before();
            mbar_arrive(&p_full[r]);
        }
        if (ok) ok = confirm_pv(nt);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            tc_fence_after();
            const int s = (rb * NT + x) * spt + row / G;  // sequence of this row
            const bool mine = row < spt * G && s < B;
            float* rec = recs + (((size_t)s * Hq + (size_t)j * G + row % G) * chunks + chunk) * (DH + 4);
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(tm_o + c * 32, o);
                tmem_ld_wait();
                if (mine) {
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        reinterpret_cast<uint4*>(rec + c * 32)[v] =
                            make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                }
            }
            if (mine) *reinterpret_cast<float4*>(rec + DH) = make_float4(m_used, l, 0.f, 0.f);
        }
    }
    if (!ok) {
        *abort_flag = 1;
        if (err) atomicOr(err, ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

struct PrefixPlan {
    int nt, row_blocks, chunks;
};
// Two row tiles a CTA once one does not hold the batch; then as many key chunks as fill the SMs in one wave.
PrefixPlan prefix_plan(int B, int Hkv, int G, int P) {
    const int spt = PX_BM / G, row_tiles = (B + spt - 1) / spt, tiles = (P + PX_BN - 1) / PX_BN;
    PrefixPlan p;
    p.nt = row_tiles > 1 ? 2 : 1;
    p.row_blocks = (row_tiles + p.nt - 1) / p.nt;
    const long long ctas = (long long)Hkv * p.row_blocks;
    p.chunks = (int)std::max<long long>(1, std::min<long long>(tiles, device_sm_count() / ctas));
    return p;
}

template <int DH, int NT>
cudaError_t prefix_launch(const PrefixPlan& p, const __nv_bfloat16* q, const __nv_bfloat16* kp, const __nv_bfloat16* vp, int B,
                          int Hq, int Hkv, int prefix_cap, int P, float* recs, int* err, cudaStream_t st) {
    using Ly = PxLayout<DH, NT>;
    const int G = Hq / Hkv, spt = PX_BM / G;
    CUtensorMap tq, tk, tv;
    if (!encode_tmap_bf16_groups(&tq, q, DH, G, Hkv, B, spt) || !encode_tmap_bf16_rows(&tk, kp, DH, P, prefix_cap, Hkv) ||
        !encode_tmap_bf16_rows(&tv, vp, DH, P, prefix_cap, Hkv))
        return cudaErrorInvalidValue;
    return launch_pdl(attn_prefix_kernel<DH, NT>, dim3((unsigned)p.row_blocks * p.chunks * Hkv), dim3(Ly::THREADS),
                      Ly::SMEM, st, tq, tk, tv, B, Hq, G, P, p.row_blocks, p.chunks, recs, err);
}

}  // namespace

size_t attn_decode_shared_workspace(int B, int Hq, int Hkv, int dh, int prefix_len) {
    if (prefix_len <= 0) return 0;
    return (size_t)B * Hq * prefix_plan(B, Hkv, Hq / Hkv, prefix_len).chunks * (dh + 4) * sizeof(float);
}

cudaError_t attn_decode_shared_launch(const __nv_bfloat16* q, const __nv_bfloat16* kp, const __nv_bfloat16* vp,
                                      int prefix_cap, int P, const __nv_bfloat16* kc, const __nv_bfloat16* vc, int B,
                                      int Hq, int Hkv, int dh, int cap, const int* len0, int len_stride, const int* meta,
                                      float* work, __nv_bfloat16* out, int* err, cudaStream_t st) {
    if (B <= 0) return cudaSuccess;
    RangeArgs a{};
    a.q = q;
    a.k = kc;
    a.v = vc;
    a.out = out;
    a.len0 = len0;
    a.len_stride = len_stride;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.cap = cap;
    a.meta = meta;
    if (P > 0) {
        const PrefixPlan p = prefix_plan(B, Hkv, a.G, P);
        a.recs = work;
        a.nrec = p.chunks;
        cudaError_t e;
        if (dh == 128)
            e = p.nt == 2 ? prefix_launch<128, 2>(p, q, kp, vp, B, Hq, Hkv, prefix_cap, P, work, err, st)
                          : prefix_launch<128, 1>(p, q, kp, vp, B, Hq, Hkv, prefix_cap, P, work, err, st);
        else
            e = p.nt == 2 ? prefix_launch<64, 2>(p, q, kp, vp, B, Hq, Hkv, prefix_cap, P, work, err, st)
                          : prefix_launch<64, 1>(p, q, kp, vp, B, Hq, Hkv, prefix_cap, P, work, err, st);
        if (e != cudaSuccess) return e;
    }
    return ranges_launch<false>(a, B, dh, cap, st);
}

cudaError_t attn_decode_sinks_launch(const __nv_bfloat16* q, const __nv_bfloat16* kc, const __nv_bfloat16* vc, int B, int Hq,
                                     int Hkv, int dh, int cap, const int* len0, int len_stride, SinkMap sm,
                                     __nv_bfloat16* out, cudaStream_t st) {
    if (B <= 0) return cudaSuccess;
    RangeArgs a{};
    a.q = q;
    a.k = kc;
    a.v = vc;
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
    return ranges_launch<true>(a, B, dh, (int)std::min<long long>((long long)sm.window + sm.sinks, cap), st);
}

cudaError_t attention_ranges_prepare() {
    const void* fns[] = {(const void*)attn_prefix_kernel<128, 1>, (const void*)attn_prefix_kernel<128, 2>,
                         (const void*)attn_prefix_kernel<64, 1>, (const void*)attn_prefix_kernel<64, 2>};
    const int smem[] = {PxLayout<128, 1>::SMEM, PxLayout<128, 2>::SMEM, PxLayout<64, 1>::SMEM, PxLayout<64, 2>::SMEM};
    for (int i = 0; i < 4; ++i) {
        cudaError_t e = cudaFuncSetAttribute(fns[i], cudaFuncAttributeMaxDynamicSharedMemorySize, smem[i]);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q3
