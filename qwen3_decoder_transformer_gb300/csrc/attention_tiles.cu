// Attention of 128-row query tiles over chosen key tiles on the tensor cores (tcgen05, TMA): prefill with a sliding
// window and sink tokens, and a decode batch's query rows against a prefix that all its sequences share.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "rings.h"

namespace q3 {
namespace {

// Flash attention with an online softmax over the 128-key tiles of a work item. Persistent: grid = min(items, SMs),
// CTA c takes items c, 2G-1-c, 2G+c, ... Tiles are counted across items (g), so ring stages, score regions and
// barrier phases simply continue, and the next item's Q, keys and scores are on their way while the softmax warps
// finish the current one.
//
// TL_SINKS: item = (query tile, sequence, head). The token in slot i sees slots j <= i with i - j < window or
// j < sinks. The item walks the key tiles of the sinks and those of its window; sequence b starts at slot
// len0[b * len_stride]. A rolling buffer keeps sink_rows rows in front of its ring.
// TL_PREFIX: item = (row tile, kv head, key chunk) of a shared prefix. A row tile holds the G query heads of
// floor(128 / G) sequences; the item leaves a record (output sums, maximum, sum of each row) instead of an output.
// The row tiles of one (kv head, chunk) are neighbours in the item order and share the chunk's keys in L2.
//
// Warps: 0 Q and keys (TMA), 1 score MMAs, 2 values (TMA), 3 P V MMAs, 4-7 softmax (thread <-> query row). Tensor
// memory: three score regions of 128 columns and the output accumulator, so the scores run two tiles ahead of P V;
// P (bf16) takes the first 64 columns of its score region. O is rescaled only when a row's maximum grew by more
// than 2^8.
// What bounds it: a softmax thread's chain over a tile (scores from tensor memory, maximum, exponentials, P back),
// about 1,600 cycles against 1,024 of MMA work (tensor pipe 63% active under ncu). 8192 tokens, 32 heads, dh 128, window
// 4096 and 4 sinks: 284 us, 300 with inputs that are not in L2 (dh 64, 8 query and 8 kv heads, 16384 tokens, 128 sinks: 163).
// The comparisons that follow were made when it took 307 (where the roles' code lies in the kernel moves its time by some per
// cent either way): timing copies of the kernel without the copies of K and V 298, with half of the MMAs 284,
// without the exponentials 258. Other forms of the softmax, on the same case: two threads a row that exchange their
// maxima 310-322; the same with the next tile's scores loaded ahead 409; the two 64-key halves as streams of their own
// with two accumulators and two score regions 322; a tile's exponentials at the scale of the tiles before it, its
// maximum beside them, 341; two warpgroups on alternate tiles (the causal prefill's ALT form) 305, but slower
// from 1024 keys down.
// 16384 tokens, window 4096, 128 sinks: 640-680 us, 1.5 PFLOP/s of visible pairs (76-80% of the measured tensor rate; the power
// limit lowers the clock after some 0.2 s of it). Looking for the next tile's scores in the middle of a tile: no gain.
// Few new tokens: an item's tiles run in turn on one CTA, so 1 to 256 tokens over a window of 4096 take 29-30 us.
constexpr int TL_SINKS = 0, TL_PREFIX = 1;
constexpr int TL_BM = 128, TL_BN = 128, TL_THREADS = 256, TL_NR = 3, TL_KST = 3, TL_VST = 3;

template <int DH>
struct TlLayout {
    static constexpr int NCH = DH / 64;
    static constexpr int Q_BYTES = TL_BM * DH * 2;
    static constexpr int KV_BYTES = TL_BN * DH * 2;
    static constexpr int K_OFF = Q_BYTES;
    static constexpr int V_OFF = K_OFF + TL_KST * KV_BYTES;
    static constexpr int BAR_OFF = V_OFF + TL_VST * KV_BYTES;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
};
static_assert(TlLayout<128>::SMEM <= 227 * 1024, "shared memory");

struct TileArgs {
    int T, Hq, Hkv, B;  // T: new tokens of a sequence, or keys of the prefix
    int* err;
    // TL_SINKS
    const int* len0;
    int len_stride, len_max, window, sinks, sink_rows, ring;
    __nv_bfloat16* out;
    // TL_PREFIX
    int row_tiles, chunks;
    float* recs;
};

template <int DH, int MODE>
__global__ void __launch_bounds__(TL_THREADS, 1)
    attn_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const TileArgs a) {
    using Ly = TlLayout<DH>;
    constexpr int NCH = Ly::NCH, NR = TL_NR, KST = TL_KST, VST = TL_VST;
    constexpr bool PREFIX = MODE == TL_PREFIX;
    constexpr uint32_t IDESC_S = idesc_bf16(TL_BM, TL_BN);
    constexpr uint32_t IDESC_O = idesc_bf16(TL_BM, DH, true);
    constexpr uint32_t TM_O = NR * TL_BN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::BAR_OFF);
    uint64_t* q_full = bars;
    uint64_t* q_empty = bars + 1;
    uint64_t* k_full = bars + 2;    // [KST]
    uint64_t* k_empty = bars + 5;   // [KST]
    uint64_t* v_full = bars + 8;    // [VST]
    uint64_t* v_empty = bars + 11;  // [VST]
    uint64_t* s_full = bars + 14;   // [NR] scores of the region are complete
    uint64_t* p_full = bars + 17;   // [NR] P of the region is written (one arrival a warp, as for o_free)
    uint64_t* r_free = bars + 20;   // [NR] P V of the region's tile is done
    uint64_t* o_free = bars + 23;   // the item's output has been read out
    uint64_t* v_clean = bars + 24;  // [VST] hidden value rows of the stage's tile are zeroed (one phase per such tile)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 27);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 28);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < KST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < VST; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&v_clean[i], 1);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&r_free[i], 1);
        }
        mbar_init(o_free, 4);
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
    pdl_wait();  // Q and the cache come from earlier kernels
    pdl_trigger();

    const int T = a.T, Hq = a.Hq, Hkv = a.Hkv, group = Hq / Hkv, tile_seqs = TL_BM / group;
    const int n_qt = (T + TL_BM - 1) / TL_BM, per_qt = a.B * Hq;
    const int n_items = PREFIX ? a.row_tiles * Hkv * a.chunks : n_qt * per_qt;
    const int G = (int)gridDim.x, cta = (int)blockIdx.x;
    // The CTA's round-th item (n_tiles = 0 when it has none left). Its i-th key tile is slot tile i below ja
    // and i + skip from there; TL_PREFIX: the tiles from skip on.
    struct Item {
        int b, h, q0, q_end, len0, ja, skip, n_tiles, chunk;
    };
    auto item_of = [&](int round) -> Item {
        Item it{};
        const int k = round * G + ((round & 1) ? G - 1 - cta : cta);
        if (k >= n_items) return it;
        if constexpr (PREFIX) {
            const unsigned strip = (unsigned)k / (unsigned)a.row_tiles;  // (kv head, chunk)
            it.b = k - (int)strip * a.row_tiles;                         // row tile
            it.chunk = (int)(strip / (unsigned)Hkv);
            it.h = (int)strip - it.chunk * Hkv;
            const unsigned tiles = ((unsigned)T + TL_BN - 1) / TL_BN;  // at most 2^23, by at most 64 chunks
            it.skip = (int)(tiles * it.chunk / (unsigned)a.chunks);
            it.n_tiles = (int)(tiles * (it.chunk + 1) / (unsigned)a.chunks) - it.skip;
        } else {
            const int from_end = (int)((unsigned)k / (unsigned)per_qt), rem = k - from_end * per_qt;
            it.q0 = (n_qt - 1 - from_end) * TL_BM;  // the longest key ranges first
            it.b = (int)((unsigned)rem / (unsigned)Hq);
            it.h = rem - it.b * Hq;
            it.q_end = min(T, it.q0 + TL_BM);
            it.len0 = min(max(0, a.len0[(size_t)it.b * a.len_stride]), a.len_max);
            const int jw = max(0, it.len0 + it.q0 - a.window + 1) / TL_BN;  // first tile of the window
            it.ja = min((a.sinks + TL_BN - 1) / TL_BN, jw);                 // tiles of the sinks before it
            it.skip = jw - it.ja;
            it.n_tiles = (it.len0 + it.q_end + TL_BN - 1) / TL_BN - it.skip;
        }
        return it;
    };
    auto tile_of = [](const Item& it, int i) { return i < it.ja ? i : i + it.skip; };
    auto tile_row = [&](int j) -> int {  // cache row of slot tile j
        const int s = j * TL_BN;
        return !PREFIX && a.ring > 0 && s >= a.sink_rows ? a.sink_rows + (s - a.sink_rows) % a.ring : s;
    };
    // tiles of an item that can hold value rows which none of its query rows sees
    auto edge = [](const Item& it, int i) {
        return !PREFIX && (i + 1 == it.ja || i == it.ja || i + 1 == it.n_tiles);
    };
    // Value rows of tile j that some row of the item may see: [v0, v1), without [h0, h1).
    struct Seen {
        int v0, v1, h0, h1;
    };
    auto seen_rows = [&](const Item& it, int j) -> Seen {
        const int k0 = j * TL_BN, sk = a.sinks - k0, lo = it.len0 + it.q0 - a.window + 1 - k0;  // first row's window
        Seen s{0, min(TL_BN, it.len0 + it.q_end - k0), 0, 0};
        if (lo >= TL_BN) {
            s.v1 = min(s.v1, sk);
        } else if (sk <= 0) {
            s.v0 = max(0, lo);
        } else if (sk < lo) {
            s.h0 = sk;
            s.h1 = lo;
        }
        return s;
    };

    // A role ends when what it has asked for is done, also after a wait of the CTA gave up: no copy or product of this CTA may
    // land in shared or tensor memory that the next one has taken over. These last waits are bounded, all of a role's by
    // one limit, and look at no abort flag. (In an ordinary run they end before the softmax warps' last tile does.)
    int never = 0;
    bool arrives = true;
    auto last_wait = [&](uint64_t* bar, int parity) { arrives = arrives && mbar_wait_suspend(bar, parity, &never); };

    if (warp == 0) {
        // ---------------- Q and key tiles
        if (lane == 0) {
            int g = 0, q_copies = 0;
            for (int round = 0; ok; ++round) {
                const Item it = item_of(round);
                if (it.n_tiles <= 0) break;
                const int jkv = PREFIX ? it.h : it.h / group;
                if (!mbar_wait_suspend(q_empty, (round & 1) ^ 1, abort_flag)) { ok = false; break; }
                if constexpr (PREFIX) {  // the rows behind the last whole group keep whatever they held
                    mbar_expect_tx(q_full, NCH * tile_seqs * group * 128);
                    for (int cc = 0; cc < NCH; ++cc)
                        tma_load_4d(smem + cc * TL_BM * 128, &tmQ, q_full, cc * 64, 0, it.h, it.b * tile_seqs);
                } else {
                    mbar_expect_tx(q_full, Ly::Q_BYTES);
                    tma_load_4d(smem, &tmQ, q_full, 0, it.q0, 0, it.b * Hq + it.h);
                }
                ++q_copies;
                for (int i = 0; i < it.n_tiles; ++i, ++g) {
                    const int s = g % KST, y = tile_row(tile_of(it, i)), z = PREFIX ? jkv : it.b * Hkv + jkv;
                    if (!mbar_wait_suspend(&k_empty[s], ((g / KST) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    mbar_expect_tx(&k_full[s], Ly::KV_BYTES);
                    tma_load_4d(smem + Ly::K_OFF + s * Ly::KV_BYTES, &tmK, &k_full[s], 0, y, 0, z);
                }
            }
            drain_ring(g, KST, [&](int s, int parity) { last_wait(&k_full[s], parity); });
            drain_ring(q_copies, 1, [&](int, int parity) { last_wait(q_full, parity); });
        }
    } else if (warp == 1) {
        // ---------------- S of tile g into region g % NR, once P V of tile g - NR has finished with it
        if (lane == 0) {
            int g = 0;
            for (int round = 0; ok; ++round) {
                const Item it = item_of(round);
                const int nt = it.n_tiles;
                if (nt <= 0) break;
                if (!mbar_wait_suspend(q_full, round & 1, abort_flag)) { ok = false; break; }
                for (int i = 0; i < nt; ++i, ++g) {
                    const int s = g % KST, r = g % NR;
                    if (!mbar_wait_suspend(&k_full[s], (g / KST) & 1, abort_flag)) { ok = false; break; }
                    // the region's next completion would be P V of tile g itself: the parity cannot alias
                    if (g >= NR && !mbar_wait_suspend(&r_free[r], ((g - NR) / NR) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sq = smem_u32(smem), sk = smem_u32(smem + Ly::K_OFF + s * Ly::KV_BYTES);
#pragma unroll
                    for (int kk = 0; kk < DH / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * TL_BM * 128 + (kk & 3) * 32;
                        umma_bf16_ss(tmem + r * TL_BN, sdesc_kmajor_sw128(sq + off), sdesc_kmajor_sw128(sk + off), IDESC_S,
                                     kk > 0);
                    }
                    umma_commit(&s_full[r]);
                    umma_commit(&k_empty[s]);
                    if (i == nt - 1) umma_commit(q_empty);  // the item's last score releases Q
                }
            }
            if (g > 0) last_wait(&s_full[(g - 1) % NR], ((g - 1) / NR) & 1);  // (completes behind every earlier tile's)
        }
    } else if (warp == 2) {
        // ---------------- value tiles; and zeros in the rows that no row of the item sees, which may hold anything
        // (0 * NaN must not reach O), within the 16-row steps that P V takes. A tile is cleaned after the next
        // tile's load has been issued (which needs P V of the tile before it at most, so nothing waits in a ring).
        int g = 0;
        int pend_s = 0, pend_ph = 0;
        bool pend = false;
        Seen pv{};
        auto clean = [&]() -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait_suspend(&v_full[pend_s], pend_ph, abort_flag))) return false;
            uint8_t* sv = smem + Ly::V_OFF + pend_s * Ly::KV_BYTES;
            auto zero = [&](int z0, int z1) {
                for (int e = lane; e < (z1 - z0) * 8 * NCH; e += 32) {
                    const int row = z0 + e / (8 * NCH), piece = e % (8 * NCH);
                    reinterpret_cast<uint4*>(sv + (piece >> 3) * TL_BN * 128 + row * 128)[piece & 7] = make_uint4(0, 0, 0, 0);
                }
            };
            zero(pv.v0 / 16 * 16, pv.v0);
            zero(pv.h0, pv.h1);
            zero(pv.v1, (pv.v1 + 15) / 16 * 16);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_clean[pend_s]);
            pend = false;
            return true;
        };
        for (int round = 0; ok; ++round) {
            const Item it = item_of(round);
            if (it.n_tiles <= 0) break;
            const int z = PREFIX ? it.h : it.b * Hkv + it.h / group;
            for (int i = 0; i < it.n_tiles; ++i, ++g) {
                const int s = g % VST, j = tile_of(it, i);
                if (!__all_sync(0xffffffffu, mbar_wait_suspend(&v_empty[s], ((g / VST) & 1) ^ 1, abort_flag))) { ok = false; break; }
                if (lane == 0) {
                    const int y = tile_row(j);
                    mbar_expect_tx(&v_full[s], Ly::KV_BYTES);
                    tma_load_4d(smem + Ly::V_OFF + s * Ly::KV_BYTES, &tmV, &v_full[s], 0, y, 0, z);
                }
                __syncwarp();
                if (pend && !clean()) { ok = false; ++g; break; }  // (g: tiles asked for)
                if (edge(it, i)) {
                    pend = true;
                    pend_s = s;
                    pend_ph = (g / VST) & 1;
                    pv = seen_rows(it, j);
                }
            }
        }
        if (ok && pend) ok = clean();
        if (lane == 0) drain_ring(g, VST, [&](int s, int parity) { last_wait(&v_full[s], parity); });
        __syncwarp();
    } else if (warp == 3) {
        // ---------------- O += P V of tile g: P from region g % NR (A operand in tensor memory), V from stage g % VST
        if (lane == 0) {
            int g = 0;
            uint32_t cleaned = 0;  // bit s: parity of the cleaned tiles seen in stage s
            for (int round = 0; ok; ++round) {
                const Item it = item_of(round);
                const int nt = it.n_tiles;
                if (nt <= 0) break;
                for (int i = 0; i < nt; ++i, ++g) {
                    const int s = g % VST, r = g % NR;
                    int step0 = 0, step1 = TL_BN / 16;  // 16-row steps that some row of the item sees
                    if (edge(it, i)) {
                        const Seen sn = seen_rows(it, tile_of(it, i));
                        step0 = sn.v0 / 16;
                        step1 = (sn.v1 + 15) / 16;
                        if (!mbar_wait_suspend(&v_clean[s], (cleaned >> s) & 1, abort_flag)) { ok = false; break; }
                        cleaned ^= 1u << s;
                    } else if (!mbar_wait_suspend(&v_full[s], (g / VST) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (i == 0 && !mbar_wait_suspend(o_free, (round & 1) ^ 1, abort_flag)) { ok = false; break; }
                    if (!mbar_wait_suspend(&p_full[r], (g / NR) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sv = smem_u32(smem + Ly::V_OFF + s * Ly::KV_BYTES);
                    if (step1 - step0 < TL_BN / 16) {
                        for (int kk = step0; kk < step1; ++kk)
                            umma_bf16_ts(tmem + TM_O, tmem + r * TL_BN + kk * 8,
                                         sdesc_mnmajor_sw128(sv + kk * 16 * 128, TL_BN * 128), IDESC_O, i != 0 || kk != step0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < TL_BN / 16; ++kk)
                            umma_bf16_ts(tmem + TM_O, tmem + r * TL_BN + kk * 8,
                                         sdesc_mnmajor_sw128(sv + kk * 16 * 128, TL_BN * 128), IDESC_O, (i | kk) != 0);
                    }
                    umma_commit(&v_empty[s]);
                    umma_commit(&r_free[r]);
                }
            }
            if (g > 0) last_wait(&r_free[(g - 1) % NR], ((g - 1) / NR) & 1);
        }
    } else {
        // ---------------- softmax: thread <-> query row (TMEM lane)
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tm_o = tmem + lane_off + TM_O;
        const float sl2 = kLog2e / sqrtf((float)DH);
        // P V of global tile k (and so every earlier one) is done. The region's next completion would be P V of
        // tile k + NR, which needs a P this thread has not released yet: the parity cannot alias.
        auto pv_done = [&](int k) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_suspend(&r_free[k % NR], (k / NR) & 1, abort_flag));
        };
        // An item's results leave after the first tile of the next item, whose scores are ready by then, so that the
        // wait for the last P V and the stores run beside the next item's first products.
        struct Pending {
            Item it;
            float m, l;
            int last;  // the item's last global tile, or -1
        };
        Pending pend{Item{}, 0.f, 0.f, -1};
        auto finish = [&](const Pending& p) -> bool {
            if (!pv_done(p.last)) return false;
            tc_fence_after();
            if constexpr (PREFIX) {
                // a warp stores 512 contiguous bytes at a time; every row of the tile has its place in the record
                float* rec = a.recs + ((size_t)(p.it.chunk * Hkv + p.it.h) * a.row_tiles + p.it.b) * prefix_rec_floats(DH);
#pragma unroll 1
                for (int c = 0; c < DH / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tm_o + c * 32, o);
                    tmem_ld_wait();
                    float* dst = rec + ((size_t)c * 8 * TL_BM + row) * 4;
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        *reinterpret_cast<uint4*>(dst + (size_t)v * TL_BM * 4) =
                            make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                }
                *reinterpret_cast<float2*>(rec + (size_t)DH * TL_BM + row * 2) = make_float2(p.m, p.l);
            } else {
                const float inv = 1.f / p.l;
                const int t0 = p.it.q0 + quarter * 32 + (lane & ~3);
                __nv_bfloat16* dst = a.out + (((size_t)p.it.b * T + t0) * Hq + p.it.h) * DH + (lane & 3) * 8;
#pragma unroll 1
                for (int c = 0; c < DH / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tm_o + c * 32, o);
                    tmem_ld_wait();
                    // 16-byte pieces change places within groups of four lanes, so that a group stores 64
                    // contiguous bytes of one row at a time (lane k piece j -> lane j piece k)
                    uint4 w[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        w[v] = make_uint4(
                            pack_bf16(__uint_as_float(o[8 * v]) * inv, __uint_as_float(o[8 * v + 1]) * inv),
                            pack_bf16(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv),
                            pack_bf16(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv),
                            pack_bf16(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv));
                    auto swap = [&](uint4& lo, uint4& hi, int bit) {  // the low lane's hi with the high lane's lo
                        const bool up = lane & bit;
                        uint4 x = up ? lo : hi;
                        x.x = __shfl_xor_sync(0xffffffffu, x.x, bit);
                        x.y = __shfl_xor_sync(0xffffffffu, x.y, bit);
                        x.z = __shfl_xor_sync(0xffffffffu, x.z, bit);
                        x.w = __shfl_xor_sync(0xffffffffu, x.w, bit);
                        if (up) lo = x;
                        else hi = x;
                    };
                    swap(w[0], w[1], 1);
                    swap(w[2], w[3], 1);
                    swap(w[0], w[2], 2);
                    swap(w[1], w[3], 2);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (t0 + v < T) *reinterpret_cast<uint4*>(dst + (size_t)v * Hq * DH + c * 32) = w[v];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            return true;
        };
        int g = 0;
        for (int round = 0; ok; ++round) {
            const Item it = item_of(round);
            const int nt = it.n_tiles;
            if (nt <= 0) break;
            const int pos = it.len0 + it.q0 + row;
            float m = -INFINITY, l = 0.f;  // the row's scale (log2 units) and sum
            for (int i = 0; i < nt; ++i) {
                const int gi = g + i, r = gi % NR, k0 = tile_of(it, i) * TL_BN;
                const uint32_t tm_s = tmem + lane_off + r * TL_BN;
                if (!__all_sync(0xffffffffu, mbar_wait_suspend(&s_full[r], (gi / NR) & 1, abort_flag))) { ok = false; break; }
                tc_fence_after();
                uint32_t sr[TL_BN];
#pragma unroll
                for (int c = 0; c < TL_BN / 32; ++c)
                    tmem_ld_32x32b_x32(tm_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
                tmem_ld_wait();
                // Hidden keys, only in the tiles at the ends of the sinks, of the window and of the item: the visible
                // columns of the row as a bit mask, one test and one select per score (range tests per score made
                // such a tile take two to four times an ordinary one's time).
                if (PREFIX ? k0 + TL_BN > T
                           : ((i <= it.ja + 1 && i + 1 >= it.ja) || i + 2 >= nt) &&
                                 (k0 + TL_BN - 1 > it.len0 + it.q0 ||
                                  (k0 < it.len0 + it.q_end - a.window && k0 + TL_BN > a.sinks))) {
                    const int lim = PREFIX ? T - k0 - 1 : pos - k0;  // last visible column
                    const int lo = PREFIX ? 0 : lim - a.window + 1;  // first column of the window
                    const int sk = PREFIX ? 0 : a.sinks - k0;        // columns below it are sinks
#pragma unroll
                    for (int c = 0; c < TL_BN / 32; ++c) {
                        const uint32_t vis = low_bits(lim + 1 - 32 * c) & (~low_bits(lo - 32 * c) | low_bits(sk - 32 * c));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            sr[c * 32 + e] = vis & (1u << e) ? sr[c * 32 + e] : __float_as_uint(-INFINITY);
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // independent chains: 3% of a long window's time
#pragma unroll
                for (int e = 0; e < TL_BN; e += 2)
                    mx4[e / 2 % 4] = fmax3(mx4[e / 2 % 4], __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
                // lazy rescale, decided per row but executed by the whole warp (tcgen05.ld/st are warp-wide)
                const bool grow = mx > m + 8.0f;
                const float alpha = grow ? ex2_approx(m - mx) : 1.0f;
                if (i > 0 && __any_sync(0xffffffffu, grow)) {
                    if (!pv_done(gi - 1)) { ok = false; break; }  // O must hold every earlier tile's P V before it is scaled
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
                    m = mx;
                }
                // P = 2^(s * sl2 - m) as packed bf16, the type that the tensor cores take beside V's (off by 2^-8 of itself at
                // most; the sum keeps fp32). A row with no visible key yet keeps m = -inf and gets P = 0.
                const float nm = m == -INFINITY ? 0.f : -m;
                const float2 sl2x2 = make_float2(sl2, sl2), nmx2 = make_float2(nm, nm);
                float2 rs2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 x = fma2(make_float2(__uint_as_float(sr[half * 64 + 2 * e]),
                                                          __uint_as_float(sr[half * 64 + 2 * e + 1])),
                                              sl2x2, nmx2);
                        const float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                        rs2 = add2(rs2, pp);
                        pk[e] = pack_bf16(pp.x, pp.y);
                    }
                    tmem_st_32x32b_x32(tm_s + half * 32, pk);
                }
                tmem_st_wait();
                l += rs2.x + rs2.y;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[r]);
                if (i == 0 && pend.last >= 0) {
                    ok = finish(pend);
                    if (!ok) break;
                }
            }
            if (!ok) break;
            pend = Pending{it, m, l, g + nt - 1};
            g += nt;
        }
        if (ok && pend.last >= 0) ok = finish(pend);
    }
    if (!ok) {
        *abort_flag = 1;
        if (a.err) atomicOr(a.err, ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DH, int MODE>
cudaError_t tiles_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, long long items,
                         const TileArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)std::min<long long>(items, device_sm_count());
    return launch_pdl(attn_tiles_kernel<DH, MODE>, dim3(grid), dim3(TL_THREADS), TlLayout<DH>::SMEM, st, tq, tk, tv, a);
}

template <int DH>
cudaError_t prefill_sinks_launch_dh(const __nv_bfloat16* q, const __nv_bfloat16* kc, const __nv_bfloat16* vc, int B, int T,
                                    int Hq, int Hkv, int cap, const int* len0, int len_stride, SinkMap sm,
                                    __nv_bfloat16* out, int* err, cudaStream_t st) {
    CUtensorMap tq, tk, tv;
    if (!encode_tmap_bf16_units(&tq, q, DH, T, T, (uint64_t)B * Hq, TL_BM) ||
        !encode_tmap_bf16_units(&tk, kc, DH, cap, cap, (uint64_t)B * Hkv, TL_BN) ||
        !encode_tmap_bf16_units(&tv, vc, DH, cap, cap, (uint64_t)B * Hkv, TL_BN))
        return cudaErrorInvalidValue;
    TileArgs a{};
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.B = B;
    a.err = err;
    a.len0 = len0;
    a.len_stride = len_stride;
    // largest start: the call's tokens end inside a full cache; a rolling buffer only bounds the slot arithmetic
    a.len_max = sm.ring > 0 ? 1 << 30 : std::max(0, cap - T);
    a.window = sm.window;
    a.sinks = sm.sinks;
    a.sink_rows = sm.sink_rows;
    a.ring = sm.ring;
    a.out = out;
    return tiles_launch<DH, TL_SINKS>(tq, tk, tv, (long long)((T + TL_BM - 1) / TL_BM) * Hq * B, a, st);
}

template <int DH>
cudaError_t prefix_launch_dh(const __nv_bfloat16* q, const __nv_bfloat16* kp, const __nv_bfloat16* vp, int B, int Hq, int Hkv,
                             int prefix_cap, int P, int chunks, float* recs, int* err, cudaStream_t st) {
    const int G = Hq / Hkv;
    CUtensorMap tq, tk, tv;
    if (!encode_tmap_bf16_groups(&tq, q, DH, G, Hkv, B, TL_BM / G) ||
        !encode_tmap_bf16_units(&tk, kp, DH, P, prefix_cap, Hkv, TL_BN) ||
        !encode_tmap_bf16_units(&tv, vp, DH, P, prefix_cap, Hkv, TL_BN))
        return cudaErrorInvalidValue;
    TileArgs a{};
    a.T = P;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.B = B;
    a.err = err;
    a.row_tiles = prefix_row_tiles(B, G);
    a.chunks = chunks;
    a.recs = recs;
    return tiles_launch<DH, TL_PREFIX>(tq, tk, tv, (long long)a.row_tiles * Hkv * chunks, a, st);
}

}  // namespace

cudaError_t attn_prefill_sinks_launch(const __nv_bfloat16* q, const __nv_bfloat16* kc, const __nv_bfloat16* vc, int B,
                                      int T, int Hq, int Hkv, int dh, int cap, const int* len0, int len_stride,
                                      SinkMap sm, __nv_bfloat16* out, int* err, cudaStream_t st) {
    if (B <= 0 || T <= 0) return cudaSuccess;
    if (dh == 128)
        return prefill_sinks_launch_dh<128>(q, kc, vc, B, T, Hq, Hkv, cap, len0, len_stride, sm, out, err, st);
    if (dh == 64) return prefill_sinks_launch_dh<64>(q, kc, vc, B, T, Hq, Hkv, cap, len0, len_stride, sm, out, err, st);
    return cudaErrorInvalidValue;
}

cudaError_t attn_prefix_launch(const __nv_bfloat16* q, const __nv_bfloat16* kp, const __nv_bfloat16* vp, int B, int Hq,
                               int Hkv, int dh, int prefix_cap, int P, int chunks, float* recs, int* err, cudaStream_t st) {
    if (dh == 128) return prefix_launch_dh<128>(q, kp, vp, B, Hq, Hkv, prefix_cap, P, chunks, recs, err, st);
    if (dh == 64) return prefix_launch_dh<64>(q, kp, vp, B, Hq, Hkv, prefix_cap, P, chunks, recs, err, st);
    return cudaErrorInvalidValue;
}

cudaError_t attention_tiles_prepare() {
    const void* fns[] = {(const void*)attn_tiles_kernel<128, TL_SINKS>, (const void*)attn_tiles_kernel<128, TL_PREFIX>,
                         (const void*)attn_tiles_kernel<64, TL_SINKS>, (const void*)attn_tiles_kernel<64, TL_PREFIX>};
    const int smem[] = {TlLayout<128>::SMEM, TlLayout<128>::SMEM, TlLayout<64>::SMEM, TlLayout<64>::SMEM};
    for (int i = 0; i < 4; ++i) {
        cudaError_t e = cudaFuncSetAttribute(fns[i], cudaFuncAttributeMaxDynamicSharedMemorySize, smem[i]);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q3
