// Appending to and reading from the paged KV cache held in 4 bits (layout: paged4.cuh).
#include <algorithm>
#include <cmath>

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
__device__ __forceinline__ void place_at(const Packed& p, const Paged4& c, int Hkv, int s, int t, Place& pl) {
    const long long slot = (long long)__ldg(p.start + s) + (t - __ldg(p.cu + s));
    pl.slot = slot < 0 || slot > 0x7fffffff ? -1 : (int)slot;
    pl.page = -1;
    const int at = pl.slot >> c.page_log;
    if (pl.slot >= 0 && at < c.max_pages) {
        const int id = __ldg(c.table + (size_t)s * c.max_pages + at);
        if ((unsigned)id < (unsigned)c.n_pages) pl.page = (long long)id * Hkv;
    }
    pl.row = pl.slot & ((1 << c.page_log) - 1);
}
__device__ __forceinline__ bool place_token(const Packed& p, const Paged4& c, int Hkv, int t, int lane, Place& pl) {
    const int s = find_sequence(p, t, lane);
    if (s < 0) return false;
    place_at(p, c, Hkv, s, t, pl);
    return true;
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ float min_nan(float a, float b) {  // (a NaN stays)
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The pair (scale, minimum) of a group with these extremes: minimum rounded down to bf16 and scale = (max - minimum) / 15 rounded
// up, so that the codes 0..15 cover the group and a value is off by half a scale at most. A group that holds NaN or
// infinity, or spans more than fp32 does, gets NaN.
__device__ __forceinline__ uint32_t side_of(float mn, float mx) {
    const __nv_bfloat16 lo = __float2bfloat16_rd(mn);
    const __nv_bfloat16 sc = __float2bfloat16_ru(__fdiv_rn(__fsub_rn(mx, __bfloat162float(lo)), 15.f));
    if (!(__bfloat162float(sc) < INFINITY)) return 0x7fff7fffu;
    return (uint32_t)__bfloat16_as_ushort(sc) | (uint32_t)__bfloat16_as_ushort(lo) << 16;
}

// The codes of eight values, the first one in the lowest nibble: the whole number nearest to (x - minimum) / scale, the even one
// of a tie (of bf16 values there are many), with the difference d = x - minimum in fp32. Without a division a value: d times a float just
// below 1 / scale, rounded to a whole number by one fused multiply-add, is that code or the one before it; the middle between
// the two, (code + 1/2) scale, is exact, so the sign of what d has over it tells which. (Quotients bracketed by two
// products, those that end at different codes taken for ties, saved 2 us of these 164, and took quotients within 2^-20 of
// a tie for one.)
__device__ __forceinline__ uint32_t codes_of(const float2 (&x)[4], uint32_t side) {
    const float scale = bf16_lo(side), low = bf16_hi(side);
    // scale 0 (all values alike), NaN, and scales whose reciprocal is no normal float: one by one
    if (!(scale >= 2e-38f && scale < 4e37f)) {
        uint32_t c = 0;
        if (scale > 0.f)
            for (int i = 0; i < 8; ++i) {
                const float d = __fsub_rn(i & 1 ? x[i / 2].y : x[i / 2].x, low);
                int y = max(__float2int_rn(__fdiv_rn(d, scale)) - 1, 0);  // a rounded quotient's code may be off by one
                for (int k = 0; k < 2; ++k) {
                    const float over = __fsub_rn(d, ((float)y + 0.5f) * scale);
                    y += over > 0.f || (over == 0.f && (y & 1));
                }
                c |= (uint32_t)min(y, 15) << (4 * i);
            }
        return c;
    }
    const uint32_t inv = __float_as_uint(rcp_approx(scale));  // off by one unit in the last place at most
    const float below = __uint_as_float(inv - 2);
    constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, in the lowest bits
    const float2 whole = make_float2(kWhole, kWhole), b2 = make_float2(below, below), s2 = make_float2(-scale, -scale),
                 h2 = make_float2(-0.5f * scale, -0.5f * scale);
    uint32_t c = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float2 d = add2(x[i], make_float2(-low, -low)), q = fma2(d, b2, whole);
        const float2 over = add2(d, fma2(add2(q, make_float2(-kWhole, -kWhole)), s2, h2));
        // y if the next code is meant (over > 0, or 0 and y odd: its bits, less 1 where y is even, have no sign; 0 is never negative
        // here), else y - 1. (The shift in PTX: from C++ nvcc 13.0 made code that added nibbles in the wrong places. With
        // comparisons of floats 32,768 tokens and their read take 168 us, so 164.)
        auto next = [](uint32_t y, float over) {
            uint32_t stays;
            asm("shr.u32 %0, %1, 31;" : "=r"(stays) : "r"(__float_as_uint(over) + (y & 1u) - 1u));
            return y - stays;
        };
        c = c * 16u + next(__float_as_uint(q.y), over.y);
        c = c * 16u + next(__float_as_uint(q.x), over.x);
    }
    return c - 0x11111111u * (0x4b400000u - 1u);  // every code carries the bits of kWhole, and is one short
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// A warp takes every `parts`-th piece of the heads of `per` consecutive tokens; a piece is 32 / LPH heads of LPH = DH / 16 lanes,
// each with 8 dims of the first half and the 8 dims that they are rotated with. With r = (mean x^2 + eps)^-1/2,
//   (a, b) -> (r (g_a cos a - g_b sin b), r (g_b cos b + g_a sin a)) in fp32, rounded once;
// the products of gains and angles are made once a token and kind of head. The next pieces' values, and the next token's
// angles, are on their way meanwhile; a sequence is looked up once, then followed from token to token.
// What bounds it: many tokens, HBM and issue (32,768 tokens of 32 / 8 heads of 128, 776 MB: 136 us, 5.7 TB/s of a copy's 6.8, 0.60
// instructions a cycle and scheduler; one warp a head with loads waited for in turn took 410); few, the chain of
// look-up, page, gains, norm, codes: 3 us with its launch. Pieces ahead and CTAs of four warps an SM: for these tokens and the read of their slots 162 us when
// it was chosen (164 now); five CTAs 172, six 172; two pieces ahead 168, eight 177.
constexpr int AP_AHEAD = 4, AP_CTAS = 4, AP_START = 2, AP_ALL = 4;
template <int DH>
__global__ void __launch_bounds__(128, AP_CTAS)
    append_paged4_kernel(const AppendArgs a, int per, int parts) {
    constexpr int LPH = DH / 16, HPW = 32 / LPH;
    const int lane = threadIdx.x & 31, l = lane % LPH;
    const int w = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    const int chunk = (int)((unsigned)w / (unsigned)parts), part = w - chunk * parts;
    const int t0 = chunk * per, t1 = min(a.N, t0 + per);
    const int heads = a.Hq + 2 * a.Hkv, pieces = (heads + HPW - 1) / HPW;
    const int page_log = a.cache.page_log, head_bytes = (int)p4_page_bytes(1 << page_log, DH);
    __shared__ float gains[2][DH];  // of queries and keys
    __shared__ float4 turn[4][2][8][LPH];  // [warp][queries, keys]: the products of gains and angles of the token, 32 floats a lane l
    pdl_wait();
    pdl_trigger();
    for (int i = threadIdx.x; i < 2 * DH; i += blockDim.x) {
        const __nv_bfloat16* gamma = i < DH ? a.q_gamma : a.k_gamma;
        gains[0][i] = gamma ? bf16f(gamma[i % DH]) : 1.f;
    }
    __syncthreads();
    if (t0 >= t1) return;
    const int hl = lane / LPH;  // this lane's head of a piece
    // The pieces ahead, copied to shared memory asynchronously; every lane reads back what it copied itself. (Held in registers
    // they were waited for as soon as they moved up a place.)
    __shared__ uint4 ahead[4][AP_AHEAD][2][32];
    uint4(*const mine)[2][32] = ahead[threadIdx.x >> 5];
    const __nv_bfloat16* load_row = a.qkv + (size_t)t0 * a.ld + l * 8;
    int load_left = t1 - t0, load_piece = part, load_slot = 0, slot = 0;
    auto load = [&]() {  // the next piece of this warp, if there is one (a group of copies either way)
        if (load_left > 0) {
            const __nv_bfloat16* x = load_row + min(load_piece * HPW + hl, heads - 1) * DH;
            copy_async16(smem_u32(&mine[load_slot][0][lane]), x);
            copy_async16(smem_u32(&mine[load_slot][1][lane]), x + DH / 2);
            if ((load_piece += parts) >= pieces) {
                load_piece = part;
                load_row += a.ld;
                --load_left;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        load_slot = (load_slot + 1) % AP_AHEAD;
    };
#pragma unroll
    for (int i = 0; i + 1 < AP_AHEAD; ++i) load();
    int seq = -1, seq_end = t0;  // the sequence at hand and the row behind it
    Place pl{-1, -1, 0};
    uint4 ang[2];  // the token's cos and sin
    auto place = [&](int t) {  // where row t goes
        if (t < seq_end && seq >= 0) {
            ++pl.slot;  // (a slot below n_pos - 1, or the row before had none)
            pl.row = pl.slot & ((1 << page_log) - 1);
            if (pl.slot <= 0 || pl.row != 0) return;
            pl.page = -1;
            const int at = pl.slot >> page_log;
            if (at < a.cache.max_pages) {
                const int id = __ldg(a.cache.table + (size_t)seq * a.cache.max_pages + at);
                if ((unsigned)id < (unsigned)a.cache.n_pages) pl.page = (long long)id * a.Hkv;
            }
            return;
        }
        seq = -1;
        seq_end = t;
        const int s = find_sequence(a.batch, t, lane);
        if (s < 0) return;
        place_at(a.batch, a.cache, a.Hkv, s, t, pl);
        seq = s;
        // (from a slot that is no position on, every row is looked up by itself)
        seq_end = pl.slot >= 0 && pl.slot < (1 << 30) ? __ldg(a.batch.cu + s + 1) : t;
    };
    auto angles = [&]() {
        if (seq >= 0 && pl.slot >= 0 && pl.slot < a.n_pos) {
            const __nv_bfloat16* cs = a.cos_sin + (size_t)pl.slot * DH + l * 8;
            ang[0] = __ldg(reinterpret_cast<const uint4*>(cs));
            ang[1] = __ldg(reinterpret_cast<const uint4*>(cs + DH / 2));
        }
    };
    auto floats = [](const uint4& v, float2 (&x)[4]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
    };
    auto bytes = [](const float2 (&x)[4]) {
        return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                          pack_bf16(x[3].x, x[3].y));
    };
    place(t0);
    angles();
    for (int t = t0; t < t1; ++t) {
        const Place at = pl;
        const bool in = seq >= 0, rotates = in && at.slot >= 0 && at.slot < a.n_pos;
        // behind the last sequence: left as it was; no position to rotate by, or no page: flagged
        if (part == 0 && lane == 0 && a.err && in && (!rotates || at.page < 0)) atomicOr(a.err, ERR_INDEX);
        const uint4 now[2] = {ang[0], ang[1]};
        if (t + 1 < t1) {
            place(t + 1);
            angles();
        }
        __nv_bfloat16* const q_row = a.q_out + (size_t)t * a.Hq * DH + l * 8;
        __nv_bfloat16* const k_row = a.k_out ? a.k_out + (size_t)t * a.Hkv * DH + l * 8 : nullptr;
        uint8_t* const k_page = a.k_pages + at.page * head_bytes;
        uint8_t* const v_page = a.v_pages + at.page * head_bytes;
        float4(*const my_turn)[8][LPH] = turn[threadIdx.x >> 5];
        if (rotates) {
            __syncwarp();  // the row before is done with them
            if (hl < 2) {  // the first head's lanes make the queries' products, the second's the keys'
                float2 c[4], s[4];
                floats(now[0], c);
                floats(now[1], s);
                const float2* g = reinterpret_cast<const float2*>(gains[hl] + l * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // g_a cos, -g_b sin; g_b cos, g_a sin
                    const float2 ga = g[i], gb = g[DH / 4 + i];
                    my_turn[hl][2 * i][l] = make_float4(ga.x * c[i].x, ga.y * c[i].y, -gb.x * s[i].x, -gb.y * s[i].y);
                    my_turn[hl][2 * i + 1][l] = make_float4(gb.x * c[i].x, gb.y * c[i].y, ga.x * s[i].x, ga.y * s[i].y);
                }
            }
            __syncwarp();
        }
        for (int piece = part; piece < pieces; piece += parts) {
            const int h = piece * HPW + hl, hh = min(h, heads - 1);
            const bool on = h < heads;
            float2 x[4], y[4];
            load();  // (into the slot that the piece before has left)
            asm volatile("cp.async.wait_group %0;" ::"n"(AP_AHEAD - 1) : "memory");
            floats(mine[slot][0][lane], x);
            floats(mine[slot][1][lane], y);
            slot = (slot + 1) % AP_AHEAD;
            if (!rotates) continue;
            const int is = hh < a.Hq ? 0 : hh < a.Hq + a.Hkv ? 1 : 2;
            if (piece * HPW < a.Hq + a.Hkv) {  // (the same for the whole warp, as is what follows but for the heads' kinds)
                float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = fma2(y[i], y[i], fma2(x[i], x[i], ss));
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = 1; o < LPH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float r = (is == 0 ? a.q_gamma : a.k_gamma) ? rsqrtf(sum * (1.f / DH) + a.eps) : 1.f;
                if (is < 2) {
                    const float2 r2 = make_float2(r, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 u = my_turn[is][2 * i][l], v = my_turn[is][2 * i + 1][l];
                        const float2 p = x[i], q = y[i];
                        x[i] = mul2(fma2(make_float2(u.x, u.y), p, mul2(make_float2(u.z, u.w), q)), r2);
                        y[i] = mul2(fma2(make_float2(v.x, v.y), q, mul2(make_float2(v.z, v.w), p)), r2);
                    }
                    __nv_bfloat16* dst = is == 0 ? q_row + hh * DH : k_row ? k_row + (hh - a.Hq) * DH : nullptr;
                    if (on && dst) {
                        *reinterpret_cast<uint4*>(dst) = bytes(x);
                        *reinterpret_cast<uint4*>(dst + DH / 2) = bytes(y);
                    }
                }
            }
            if ((piece + 1) * HPW <= a.Hq) continue;
            // the extremes of the first and the second 64 dims (dh 64: of all)
            auto low = [](const float2 (&v)[4]) {
                return min_nan(min_nan(min_nan(v[0].x, v[0].y), min_nan(v[1].x, v[1].y)),
                               min_nan(min_nan(v[2].x, v[2].y), min_nan(v[3].x, v[3].y)));
            };
            auto high = [](const float2 (&v)[4]) {
                return max_nan(max_nan(max_nan(v[0].x, v[0].y), max_nan(v[1].x, v[1].y)),
                               max_nan(max_nan(v[2].x, v[2].y), max_nan(v[3].x, v[3].y)));
            };
            float mn = low(x), mx = high(x), mn1 = low(y), mx1 = high(y);
            uint32_t side0, side1;
            if constexpr (DH == 128) {  // lanes 0-3 of a head go on with the first group, lanes 4-7 with the second
                const bool second = l >= 4;
                const float mn2 = __shfl_xor_sync(0xffffffffu, second ? mn : mn1, 4);
                const float mx2 = __shfl_xor_sync(0xffffffffu, second ? mx : mx1, 4);
                mn = min_nan(second ? mn1 : mn, mn2);
                mx = max_nan(second ? mx1 : mx, mx2);
            } else {
                mn = min_nan(mn, mn1);
                mx = max_nan(mx, mx1);
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            const uint32_t side = side_of(mn, mx);
            if constexpr (DH == 128) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, side, 4);
                side0 = l >= 4 ? other : side;
                side1 = l >= 4 ? side : other;
            } else {
                side0 = side1 = side;
            }
            const uint32_t c0 = codes_of(x, side0), c1 = codes_of(y, side1);
            if (on && is > 0 && at.page >= 0) {
                uint8_t* base = is == 2 ? v_page + (hh - a.Hq - a.Hkv) * head_bytes : k_page + (hh - a.Hq) * head_bytes;
                uint32_t* codes = reinterpret_cast<uint32_t*>(base + at.row * (DH / 2));
                codes[l] = c0;
                codes[DH / 16 + l] = c1;
                uint32_t* sd = reinterpret_cast<uint32_t*>(base + (DH / 2 << page_log)) + at.row * (DH / kP4Group);
                if (l == 0) sd[0] = side0;
                if (DH == 128 && l == 4) sd[1] = side1;
            }
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

// One warp a token: DH / 8 lanes take a row (K or V of a head), eight dims each, so that a store of the warp fills 512 contiguous
// bytes; RD_ROWS rows' loads are on their way at once. Every value is rounded once. What bounds it: HBM writes, most of its
// bytes (100,000 tokens of 8 heads of 128, 525 MB: 83 us, 6.3 TB/s; two rows at once 87, eight 89; a lane 16 dims in two
// stores 104). Where two rows at once are all of a token's, more would only repeat them: RD_ROWS is 2 (65,536 tokens of 2
// heads of 128 or 4 of 64: 20 us, with four 23.5).
template <int DH, int RD_ROWS>
__global__ void __launch_bounds__(256)
    read_paged4_kernel(const ReadArgs a) {
    constexpr int LPR = DH / 8, RPW = 32 / LPR;  // lanes a row, rows a warp at once
    const int lane = threadIdx.x & 31, t = (int)(blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5));
    pdl_wait();
    pdl_trigger();
    Place pl;
    if (t >= a.N || !place_token(a.batch, a.cache, a.Hkv, t, lane, pl)) return;
    if (pl.page < 0) {  // nothing to read: left as it was
        if (lane == 0 && a.err) atomicOr(a.err, ERR_INDEX);
        return;
    }
    const int page_log = a.cache.page_log, head_bytes = (int)p4_page_bytes(1 << page_log, DH), l = lane % LPR;
    const int code_at = pl.row * (DH / 2) + l * 4, side_at = (DH / 2 << page_log) + pl.row * (DH / kP4Group * 4) + l * 8 / kP4Group * 4;
    for (int h0 = 0; h0 < a.Hkv; h0 += RPW * RD_ROWS / 2) {
        uint32_t code[RD_ROWS], side[RD_ROWS];
#pragma unroll
        for (int i = 0; i < RD_ROWS; ++i) {  // K and V of a head in turn
            const int h = min(h0 + i / 2 * RPW + lane / LPR, a.Hkv - 1);
            const uint8_t* base = (i & 1 ? a.cache.v : a.cache.k) + pl.page * head_bytes + (size_t)h * head_bytes;
            code[i] = __ldg(reinterpret_cast<const uint32_t*>(base + code_at));
            side[i] = __ldg(reinterpret_cast<const uint32_t*>(base + side_at));
        }
#pragma unroll
        for (int i = 0; i < RD_ROWS; ++i) {
            const int h = h0 + i / 2 * RPW + lane / LPR;
            const float scale = bf16_lo(side[i]), low = bf16_hi(side[i]);
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = fmaf((float)((code[i] >> (4 * k)) & 15u), scale, low);
            if (h < a.Hkv)
                *reinterpret_cast<uint4*>((i & 1 ? a.v_out : a.k_out) + ((size_t)t * a.Hkv + h) * DH + l * 8) = pack8(x);
        }
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
    // `parts` warps share the pieces of a token, and each takes `per` tokens. The split with the shortest way of a warp, in pieces: a
    // token costs AP_START more, and a GPU full of warps that start together AP_ALL more. With the reads of the same slots, 32 / 8
    // heads of 128: 1 token 5.9 us (a warp a token 10.5), 200 tokens 7.2 (as many warps as there are pieces 10.0), 3,000 23.7 (a
    // warp a token 28.5), 32,768 164.
    const double room = 4. * AP_CTAS * device_sm_count();
    const int pieces = (Hq + 2 * Hkv + 512 / dh - 1) / (512 / dh);
    int parts = 1, per = 0;
    double least = 0;
    for (int p = 1; p <= std::min(pieces, 64); ++p) {
        const int n = (int)std::ceil(N * (double)p / room);
        const double way = n * (double)((pieces + p - 1) / p + AP_START) + AP_ALL * (N * (double)p / (n * room));
        if (per == 0 || way < least) {
            parts = p;
            per = n;
            least = way;
        }
    }
    const long long warps = ((long long)N + per - 1) / per * parts;
    const dim3 grid((unsigned)((warps + 3) / 4));
    return dh == 128 ? launch_pdl(append_paged4_kernel<128>, grid, dim3(128), 0, st, a, per, parts)
                     : launch_pdl(append_paged4_kernel<64>, grid, dim3(128), 0, st, a, per, parts);
}

cudaError_t read_paged4_launch(const void* k_pages, const void* v_pages, int n_pages, int page, const int* table, int max_pages,
                               const int* cu, const int* start, int S, int N, int Hkv, int dh, __nv_bfloat16* k_out,
                               __nv_bfloat16* v_out, int* err, cudaStream_t st) {
    ReadArgs a{{cu, start, S},
               {static_cast<const uint8_t*>(k_pages), static_cast<const uint8_t*>(v_pages), table, n_pages, max_pages,
                log2_of(page)},
               N, Hkv, k_out, v_out, err};
    const unsigned grid = ((unsigned)N + 7) / 8;
    if (dh == 128)  // (a step is 2 RD_ROWS rows, or at head_dim 64 4 RD_ROWS)
        return Hkv <= 2 ? launch_pdl(read_paged4_kernel<128, 2>, dim3(grid), dim3(256), 0, st, a)
                        : launch_pdl(read_paged4_kernel<128, 4>, dim3(grid), dim3(256), 0, st, a);
    return Hkv <= 4 ? launch_pdl(read_paged4_kernel<64, 2>, dim3(grid), dim3(256), 0, st, a)
                    : launch_pdl(read_paged4_kernel<64, 4>, dim3(grid), dim3(256), 0, st, a);
}

}  // namespace q3
