// Appending to and reading from the paged KV cache held in 4 bits (layout: paged4.cuh).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged4.cuh"

namespace q3 {
namespace {

// A packed batch: the tokens [cu[s], cu[s + 1]) belong to sequence s, whose slots they take from start[s] on.
struct Packed {
    const int *cu, *start;
    int S;
};

// The sequence of token t, or -1: every lane of a warp looks at another entry of cu, so 32 sequences take one step and
// 1024 two. (Of sequences that begin at the same token the last one owns it: the others are empty.)
__device__ __forceinline__ int find_sequence(const Packed& p, int t, int lane) {
    int lo = 0, n = p.S + 1;  // the last entry of cu[lo .. lo + n) that is <= t is looked for
    while (true) {
        const int step = (n + 31) / 32, i = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, i < n && __ldg(p.cu + lo + i) <= t);
        if (lo == 0 && !(below & 1)) return -1;
        const int at = 31 - __clz((int)below);
        if (step == 1) {
            lo += at;
            break;
        }
        n = min(step, n - at * step);
        lo += at * step;
    }
    return lo < p.S ? lo : -1;
}

// Where token t goes: its slot (also its position), and the byte offset of its page, or -1 where it has none.
struct Place {
    int slot;
    long long page;  // page id * Hkv, or -1
    int row;         // within the page
};
__device__ __forceinline__ bool place_token(const Packed& p, const Paged4& c, int Hkv, int t, int lane, Place& pl) {
    const int s = find_sequence(p, t, lane);
    if (s < 0) return false;
    const long long slot = (long long)__ldg(p.start + s) + (t - __ldg(p.cu + s));
    pl.slot = slot < 0 || slot > 0x7fffffff ? -1 : (int)slot;
    pl.page = -1;
    const int at = pl.slot >> c.page_log;
    if (pl.slot >= 0 && at < c.max_pages) {
        const int id = __ldg(c.table + (size_t)s * c.max_pages + at);
        if ((unsigned)id < (unsigned)c.n_pages) pl.page = (long long)id * Hkv;
    }
    pl.row = pl.slot & ((1 << c.page_log) - 1);
    return true;
}

__device__ __forceinline__ void unpack8(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Quantise a group's values, of which this thread holds n: minimum rounded down to bf16 and scale = (max - minimum) / 15
// rounded up, so that the codes 0..15 cover the group and a value is off by half a scale at most. The scale's pair is
// returned; a group that holds NaN or infinity (or spans more than fp32 does) gets NaN for both.
template <int N, int LANES>
__device__ __forceinline__ uint32_t quantize(const float* x, uint32_t (&codes)[N / 8]) {
    float mn = x[0], mx = x[0], bad = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
        bad += x[i] * 0.f;  // 0, or NaN
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        bad += __shfl_xor_sync(0xffffffffu, bad, o);
    }
    const __nv_bfloat16 lo = __float2bfloat16_rd(mn);
    const float low = __bfloat162float(lo);
    const __nv_bfloat16 sc = __float2bfloat16_ru(__fdiv_rn(__fsub_rn(mx, low), 15.f));
    const float scale = __bfloat162float(sc);
    if (bad != 0.f || !(scale < INFINITY)) {
#pragma unroll
        for (int w = 0; w < N / 8; ++w) codes[w] = 0;
        return 0x7fff7fffu;
    }
    const float div = scale > 0.f ? scale : 1.f;
#pragma unroll
    for (int w = 0; w < N / 8; ++w) {
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // a true quotient: ties (bf16 values between two codes) go to the even code as the definition says
            const int q = __float2int_rn(__fdiv_rn(__fsub_rn(x[w * 8 + i], low), div));
            c |= (uint32_t)min(max(q, 0), 15) << (4 * i);
        }
        codes[w] = c;
    }
    return (uint32_t)__bfloat16_as_ushort(sc) | (uint32_t)__bfloat16_as_ushort(lo) << 16;
}

struct AppendArgs {
    const __nv_bfloat16* qkv;
    long long ld;
    Packed batch;
    Paged4 cache;
    int N, Hq, Hkv;
    const __nv_bfloat16 *q_gamma, *k_gamma;  // null: no head norm
    float eps;
    const __nv_bfloat16* cos_sin;  // [n_pos][dh]
    int n_pos;
    __nv_bfloat16 *q_out, *k_out;  // [N][Hq][dh], [N][Hkv][dh] or null
    uint8_t *k_pages, *v_pages;
    int* err;
};

// One token a CTA. A head takes DH / 16 lanes; each holds 8 dims of the first half and the 8 dims that they are rotated with.
//   q, k: y = x * rsqrt(mean x^2 + eps) * gamma; rotated (a, b) -> (a cos - b sin, b cos + a sin), fp32, rounded once
template <int DH>
__global__ void __launch_bounds__(512)
    append_paged4_kernel(const AppendArgs a) {
    constexpr int LPH = DH / 16;
    const int lane = threadIdx.x & 31, t = blockIdx.x;
    const int heads = a.Hq + 2 * a.Hkv, l = threadIdx.x % LPH;
    pdl_wait();
    pdl_trigger();
    Place pl;
    if (!place_token(a.batch, a.cache, a.Hkv, t, lane, pl)) return;  // behind the last sequence: left as it was
    if (pl.slot < 0 || pl.slot >= a.n_pos) {  // no position to rotate by
        if (threadIdx.x == 0 && a.err) atomicOr(a.err, ERR_INDEX);
        return;
    }
    if (pl.page < 0 && threadIdx.x == 0 && a.err) atomicOr(a.err, ERR_INDEX);
    const __nv_bfloat16* cs = a.cos_sin + (size_t)pl.slot * DH + l * 8;
    float c[8], s[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(cs)), c);
    unpack8(__ldg(reinterpret_cast<const uint4*>(cs + DH / 2)), s);
    const int page = 1 << a.cache.page_log;
    // (whole warps stay in the loop: the lanes of the last heads work on head 0 and store nothing)
    for (int h0 = threadIdx.x / LPH - lane / LPH; h0 < heads; h0 += blockDim.x / LPH) {
        const int h = h0 + lane / LPH;
        const bool on = h < heads;
        const int hh = on ? h : 0;
        const __nv_bfloat16* x = a.qkv + (size_t)t * a.ld + (size_t)hh * DH + l * 8;
        float y[16];
        unpack8(__ldg(reinterpret_cast<const uint4*>(x)), y);
        unpack8(__ldg(reinterpret_cast<const uint4*>(x + DH / 2)), y + 8);
        const bool is_q = hh < a.Hq, is_v = hh >= a.Hq + a.Hkv;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!is_v) {
            const __nv_bfloat16* gamma = is_q ? a.q_gamma : a.k_gamma;
            if (gamma) {
                const float r = rsqrtf(ss / DH + a.eps);
                float g[16];
                unpack8(__ldg(reinterpret_cast<const uint4*>(gamma + l * 8)), g);
                unpack8(__ldg(reinterpret_cast<const uint4*>(gamma + DH / 2 + l * 8)), g + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = y[i] * r * g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = y[i], q = y[8 + i];
                y[i] = p * c[i] - q * s[i];
                y[8 + i] = q * c[i] + p * s[i];
            }
            __nv_bfloat16* dst = nullptr;
            if (is_q)
                dst = a.q_out + ((size_t)t * a.Hq + hh) * DH;
            else if (a.k_out)
                dst = a.k_out + ((size_t)t * a.Hkv + (hh - a.Hq)) * DH;
            if (on && dst) {
                *reinterpret_cast<uint4*>(dst + l * 8) = pack8(y);
                *reinterpret_cast<uint4*>(dst + DH / 2 + l * 8) = pack8(y + 8);
            }
        }
        if (__all_sync(0xffffffffu, is_q)) continue;
        uint32_t w[2], side[2];
        if constexpr (DH == 128) {
            uint32_t w0[1], w1[1];
            side[0] = quantize<8, LPH>(y, w0);
            side[1] = quantize<8, LPH>(y + 8, w1);
            w[0] = w0[0];
            w[1] = w1[0];
        } else {
            side[0] = quantize<16, LPH>(y, w);
            side[1] = 0;
        }
        if (on && !is_q && pl.page >= 0) {
            uint8_t* base = (is_v ? a.v_pages : a.k_pages) +
                            (size_t)(pl.page + (hh - a.Hq - (is_v ? a.Hkv : 0))) * p4_page_bytes(page, DH);
            uint32_t* codes = reinterpret_cast<uint32_t*>(base + (size_t)pl.row * (DH / 2));
            codes[l] = w[0];
            codes[DH / 16 + l] = w[1];
            uint32_t* sd = reinterpret_cast<uint32_t*>(base + (size_t)page * (DH / 2)) + pl.row * (DH / kP4Group);
            if (l < DH / kP4Group) sd[l] = l == 0 ? side[0] : side[1];
        }
    }
}

struct ReadArgs {
    Packed batch;
    Paged4 cache;
    int N, Hkv;
    __nv_bfloat16 *k_out, *v_out;  // [N][Hkv][dh]
    int* err;
};

// One warp a token: LPH lanes take the 16 dims each of one row (K or V of a head). Every value is rounded once.
template <int DH>
__global__ void __launch_bounds__(256)
    read_paged4_kernel(const ReadArgs a) {
    constexpr int LPH = DH / 16;
    const int lane = threadIdx.x & 31, t = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    pdl_wait();
    pdl_trigger();
    Place pl;
    if (t >= a.N || !place_token(a.batch, a.cache, a.Hkv, t, lane, pl)) return;
    if (pl.page < 0) {  // nothing to read: left as it was
        if (lane == 0 && a.err) atomicOr(a.err, ERR_INDEX);
        return;
    }
    const int page = 1 << a.cache.page_log, l = lane % LPH;
    for (int h = lane / LPH; h < 2 * a.Hkv; h += 32 / LPH) {
        const bool is_v = h >= a.Hkv;
        const int hh = is_v ? h - a.Hkv : h;
        const uint8_t* base = (is_v ? a.cache.v : a.cache.k) + (size_t)(pl.page + hh) * p4_page_bytes(page, DH);
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(base + (size_t)pl.row * (DH / 2)) + l);
        const uint32_t sd = __ldg(reinterpret_cast<const uint32_t*>(base + (size_t)page * (DH / 2)) +
                                  pl.row * (DH / kP4Group) + l * 16 / kP4Group);
        const float scale = bf16_lo(sd), low = bf16_hi(sd);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = fmaf((float)(((i < 8 ? w.x : w.y) >> (4 * (i & 7))) & 15u), scale, low);
        __nv_bfloat16* dst = (is_v ? a.v_out : a.k_out) + ((size_t)t * a.Hkv + hh) * DH + l * 16;
        reinterpret_cast<uint4*>(dst)[0] = pack8(x);
        reinterpret_cast<uint4*>(dst)[1] = pack8(x + 8);
    }
}

int log2_of(int v) {
    int l = 0;
    while (1 << l < v) ++l;
    return l;
}

}  // namespace

cudaError_t append_paged4_launch(const __nv_bfloat16* qkv, long long ld, int N, const int* cu, const int* start, int S, int Hq,
                                 int Hkv, int dh, const __nv_bfloat16* q_gamma, const __nv_bfloat16* k_gamma, float eps,
                                 const __nv_bfloat16* cos_sin, int n_pos, __nv_bfloat16* q_out, __nv_bfloat16* k_out,
                                 void* k_pages, void* v_pages, int n_pages, int page, const int* table, int max_pages,
                                 int* err, cudaStream_t st) {
    AppendArgs a{qkv, ld, {cu, start, S}, {nullptr, nullptr, table, n_pages, max_pages, log2_of(page)}, N, Hq, Hkv, q_gamma,
                 k_gamma, eps, cos_sin, n_pos, q_out, k_out, static_cast<uint8_t*>(k_pages), static_cast<uint8_t*>(v_pages),
                 err};
    const int threads = std::min(512, ((Hq + 2 * Hkv) * (dh / 16) + 31) / 32 * 32);
    return dh == 128 ? launch_pdl(append_paged4_kernel<128>, dim3(N), dim3(threads), 0, st, a)
                     : launch_pdl(append_paged4_kernel<64>, dim3(N), dim3(threads), 0, st, a);
}

cudaError_t read_paged4_launch(const void* k_pages, const void* v_pages, int n_pages, int page, const int* table, int max_pages,
                               const int* cu, const int* start, int S, int N, int Hkv, int dh, __nv_bfloat16* k_out,
                               __nv_bfloat16* v_out, int* err, cudaStream_t st) {
    ReadArgs a{{cu, start, S},
               {static_cast<const uint8_t*>(k_pages), static_cast<const uint8_t*>(v_pages), table, n_pages, max_pages,
                log2_of(page)},
               N, Hkv, k_out, v_out, err};
    const unsigned grid = ((unsigned)N + 7) / 8;
    return dh == 128 ? launch_pdl(read_paged4_kernel<128>, dim3(grid), dim3(256), 0, st, a)
                     : launch_pdl(read_paged4_kernel<64>, dim3(grid), dim3(256), 0, st, a);
}

}  // namespace q3
