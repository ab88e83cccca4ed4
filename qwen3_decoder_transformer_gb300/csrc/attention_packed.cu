// Causal attention over packed sequences of different lengths on the tensor cores (tcgen05, TMA): the work list of a batch, and
// the kernel that walks it.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "rings.h"

namespace q3 {
namespace {

constexpr int PK_BM = 128, PK_BN = 128;

// ------------------------------------------------------------------------------------- packed sequences
// The work lists of a packed batch, one for each size of a query tile: list L has an entry for every 128 >> L query rows of a
// sequence (first query row, rows, the sequence's first key row, key position of the first query row), the longest key ranges first
// (a counting sort by key tiles, those past kPlanBins - 1 together). The attention kernel takes the list of its tiles' tokens,
// 128 / PG (the finest one for larger groups): with one list of 128 rows and up to PG places an entry, places that a
// sequence's last rows do not fill left CTAs without work (16 turns of 300 tokens over up to 4096 keys: 230 us against 203;
// 64 prompts of about 512 tokens 278 and 252).
// One CTA, a warp a sequence (all of them a long one). The order of equal tiles depends on timing; it decides which SM
// computes a tile, not its result. 16 sequences of 300 queries over 4,096 keys each: 7 us, 64 prompts
// of 512 tokens 9, 3,000 of five 44, once for all layers.
constexpr int kPlanThreads = 1024, kPlanBins = 1024, kPlanLevels = 4, kPlanLong = 4096;
struct PlanHeader {
    int count[kPlanLevels];        // entries of a list
    long long first[kPlanLevels];  // where it begins
};
constexpr int kPlanHeader = 256;
static_assert(sizeof(PlanHeader) <= kPlanHeader, "header");
size_t plan_level(int Nq, int S, int level) {  // entries that list `level` can have
    const int rows = PK_BM >> level;
    return (size_t)(Nq + rows - 1) / rows + (size_t)S;
}
__global__ void __launch_bounds__(kPlanThreads)
    attn_packed_plan_kernel(const int* __restrict__ cu_q, const int* __restrict__ cu_k, int S, int Nq, int Nk,
                            const __grid_constant__ PlanHeader at, PlanHeader* header, int4* items, int* err) {
    __shared__ int bins[kPlanLevels][kPlanBins], bin_sum[kPlanLevels][32], warp_sum[kPlanThreads / 32];
    __shared__ int4 seqs[kPlanThreads];  // first query row, queries (0: left out), first key row, keys in front of the queries
    __shared__ unsigned longs[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a warp's lanes share the lists of a sequence: 16 the finest one, 8, 4 and 4 the others
    const int level = lane < 16 ? 3 : lane < 24 ? 2 : lane < 28 ? 1 : 0, lanes = level == 3 ? 16 : level == 2 ? 8 : 4;
    const int at_lane = lane & (lanes - 1), rows_log = 7 - level;
    pdl_wait();
    pdl_trigger();
    for (int i = threadIdx.x; i < kPlanLevels * kPlanBins; i += kPlanThreads) bins[0][i] = 0;
    auto each = [&](auto take) {  // take(item, bin) for every tile of this lane's level
        auto tiles_of = [&](const int4& v, int group, int groups) {
            for (int t = group * lanes + at_lane; t << rows_log < v.y; t += groups * lanes) {
                const int row = t << rows_log, rows = min(1 << rows_log, v.y - row), pos = v.w + row;
                const int tiles = (max(pos + rows, 0) + PK_BN - 1) / PK_BN;
                take(make_int4(v.x + row, rows, v.z, pos), kPlanBins - 1 - min(tiles, kPlanBins - 1));
            }
        };
        int end = 0;  // of the query rows of the sequences so far
        for (int base = 0; base < S; base += kPlanThreads) {
            const int s = base + threadIdx.x;
            int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
            if (s < S) {
                q0 = __ldg(cu_q + s);
                q1 = __ldg(cu_q + s + 1);
                k0 = __ldg(cu_k + s);
                k1 = __ldg(cu_k + s + 1);
            }
            // the largest bound before this one: a sequence that begins before it would write rows of another
            int top = q0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, top, o);
                if (lane >= o) top = max(top, v);
            }
            __syncthreads();  // the previous round's sequences are done
            if (lane == 31) warp_sum[warp] = top;
            __syncthreads();
            top = max(top, __reduce_max_sync(0xffffffffu, lane < warp ? max(warp_sum[lane], end) : end));
            end = max(end, __reduce_max_sync(0xffffffffu, warp_sum[lane]));
            const bool ok = q0 >= top && q1 >= q0 && q1 <= Nq && k0 >= 0 && k1 >= k0 && k1 <= Nk;
            if (s < S && !ok && err) atomicOr(err, ERR_INDEX);
            seqs[threadIdx.x] = make_int4(q0, ok ? q1 - q0 : 0, k0, ok ? k1 - k0 - (q1 - q0) : 0);
            const unsigned is_long = __ballot_sync(0xffffffffu, ok && q1 - q0 > kPlanLong);
            if (lane == 0) longs[warp] = is_long;
            __syncthreads();
            for (int i = warp; i < min(kPlanThreads, S - base); i += kPlanThreads / 32) {
                const int4 v = seqs[i];
                if (v.y <= kPlanLong) tiles_of(v, 0, 1);
            }
            for (int w = 0; w < kPlanThreads / 32; ++w)
                for (unsigned left = longs[w]; left != 0; left &= left - 1)
                    tiles_of(seqs[w * 32 + __ffs((int)left) - 1], warp, kPlanThreads / 32);
        }
    };
    __syncthreads();
    each([&](const int4&, int bin) { atomicAdd(&bins[level][bin], 1); });
    static_assert(kPlanBins == kPlanThreads, "a thread a bin");
    __syncthreads();
    int mine[kPlanLevels], sum[kPlanLevels];
#pragma unroll
    for (int l = 0; l < kPlanLevels; ++l) {
        sum[l] = mine[l] = bins[l][threadIdx.x];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum[l], o);
            if (lane >= o) sum[l] += v;
        }
        if (lane == 31) bin_sum[l][warp] = sum[l];
    }
    __syncthreads();
#pragma unroll
    for (int l = 0; l < kPlanLevels; ++l) {
        sum[l] += __reduce_add_sync(0xffffffffu, lane < warp ? bin_sum[l][lane] : 0);
        bins[l][threadIdx.x] = sum[l] - mine[l];
        if (threadIdx.x == kPlanThreads - 1) {  // (no more than there is room for: the sequences do not overlap)
            header->count[l] = min(sum[l], at.count[l]);
            header->first[l] = at.first[l];
        }
    }
    __syncthreads();
    int4* const list = items + at.first[level];
    const int room = at.count[level];
    each([&](const int4& item, int bin) {
        const int n = atomicAdd(&bins[level][bin], 1);
        if (n < room) list[n] = item;
    });
}

// ------------------------------------------------------------------------------------- the kernel
// Flash attention with an online softmax over 128-key tiles. An item is a tile of 128 query rows, PG = the largest power of two
// in the group's query heads by 128 / PG tokens (so short runs of queries fill a tile), with one kv head.
// Persistent: CTA c of G takes items c, 2G-1-c, 2G+c, ... of the list, which has the longest key ranges first. Tiles are counted
// across items, so rings, score regions and barrier phases simply continue.
//
// Warps: 0 Q and K (TMA), 1 score MMAs, 2 V (TMA), 3 P V MMAs, 4-7 softmax (thread <-> query row), 8-11 output. Tensor memory: one
// score region of 128 columns, free again as soon as the softmax has its 128 scores in registers (hence the register
// split), two regions of 64 for P in bf16, and two output accumulators, items taking turns: while warps 8-11 read
// one item's output out, the next item's products and softmax go on. With one accumulator that the softmax warps read
// out themselves (and three score regions) short prompts stood still at every item's end: 64 prompts of 512 tokens, 32
// heads, 315 us against 260. Two query tiles at once, each with softmax warps and an accumulator of its own, reached
// 0.57 of the tensor peak on 8,192 tokens: their scores and P share a region, so the products of one wait for its softmax.
// O is rescaled only when a row's maximum grew by more than 2^8. Rows of another sequence that a tile reaches into are masked
// (keys), zeroed (values) and not stored (queries).
// What bounds it: the way of a tile through tensor memory, 128 scores a thread, and back, about 1,500 cycles of 128 query rows by
// 128 keys, against 1,024 of products. One prompt of 8,192 tokens, 32 / 8 heads of 128: 352 us, 0.82 of the tensor peak
// (1,562 TFLOP/s of visible pairs); 17,000 tokens in three prompts 550 us; in a loop, with the clock that the power limit
// leaves, 380 and 575. Short prompts: masked tiles, 2,500 cycles each, are 40% of the key tiles of prompts of 512 tokens at
// groups of four (64 of them: 253 us). Leaving out the parts of a masked tile that no row sees made 242 us of that, in the
// form for short key ranges, but 377-381 of the 352 of one long prompt, in the other: tried in both forms at once, it is
// in neither.
constexpr int PK_THREADS = 384;
constexpr uint32_t PK_REG_PRODUCER = 56, PK_REG_SOFTMAX = 208, PK_REG_OUTPUT = 104;
static_assert(PK_REG_PRODUCER + PK_REG_SOFTMAX + PK_REG_OUTPUT <= 3 * 168, "register split exceeds the launch");
// Shared memory holds seven tiles at head_dim 128 and little else. Long key ranges take a third stage of keys; short ones
// (LONG false), with many items a CTA, room for more of them looked up at its start (64 prompts of 512 tokens 260 us
// against 266, three of 5,000 and more 548 against 535; head_dim 64 has room for both).
template <int DH, bool LONG>
struct PkLayout {
    static constexpr int NCH = DH / 64;
    static constexpr int TILE_BYTES = 128 * DH * 2;
    static constexpr int QST = 2, KST = LONG ? 3 : 2, VST = 2;
    static constexpr int TABLE = LONG && DH == 128 ? 48 : 512;  // items of a CTA that are looked up at its start
    static constexpr int K_OFF = QST * TILE_BYTES, V_OFF = K_OFF + KST * TILE_BYTES;
    static constexpr int INV_OFF = V_OFF + VST * TILE_BYTES;  // [item parity][row]: 1 / sum
    static constexpr int TABLE_OFF = INV_OFF + 2 * PK_BM * 4;
    static constexpr int BAR_OFF = TABLE_OFF + TABLE * 16;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
};
static_assert(PkLayout<128, true>::SMEM <= 227 * 1024 && PkLayout<128, false>::SMEM <= 227 * 1024, "shared memory");

struct PackedArgs {
    const int4* items;
    const PlanHeader* plan;
    int capacity, max_keys;
    int Nq, Hq, Hkv, pg_log;
    __nv_bfloat16* out;
    int* err;
};

template <int DH, bool LONG>
__global__ void __launch_bounds__(PK_THREADS, 1)
    attn_packed_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PackedArgs a) {
    using Ly = PkLayout<DH, LONG>;
    constexpr int NCH = Ly::NCH, QST = Ly::QST, KST = Ly::KST, VST = Ly::VST, TB = Ly::TILE_BYTES;
    constexpr uint32_t IDESC_S = idesc_bf16(PK_BM, PK_BN);
    constexpr uint32_t IDESC_O = idesc_bf16(PK_BM, DH, true);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::BAR_OFF);
    uint64_t* q_full = bars;              // [QST]
    uint64_t* q_empty = q_full + QST;     // [QST]
    uint64_t* k_full = q_empty + QST;     // [KST]
    uint64_t* k_empty = k_full + KST;     // [KST]
    uint64_t* v_full = k_empty + KST;     // [VST]
    uint64_t* v_empty = v_full + VST;     // [VST]
    uint64_t* s_full = v_empty + VST;     // the tile's scores are complete
    uint64_t* s_empty = s_full + 1;       // they have been read (one arrival a warp, as for p_full, l_full and o_free)
    uint64_t* p_full = s_empty + 1;       // [tile parity] P is written
    uint64_t* pv_done = p_full + 2;       // [tile parity] P V is done
    uint64_t* o_full = pv_done + 2;       // [item parity] the item's last P V is done
    uint64_t* l_full = o_full + 2;        // [item parity] the rows' sums are in shared memory
    uint64_t* o_free = l_full + 2;        // [item parity] accumulator and sums have been read out
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_free + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(o_free + 3);
    static_assert((2 * (QST + KST + VST) + 6 + 6 + 2) * 8 <= 256, "barriers");
    volatile float* inv_sh = reinterpret_cast<volatile float*>(smem + Ly::INV_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (uint64_t* b = bars; b < o_free + 2; ++b) {
            const bool by_warps = (b >= s_empty && b < pv_done) || b >= l_full;
            mbar_init(b, by_warps ? 4 : 1);
        }
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
    // scores; P of tile g at tmem_p + (g & 1) * 64; O of item n at tmem_o + (n & 1) * 128
    const uint32_t tmem = *tmem_slot, tmem_p = tmem + PK_BN, tmem_o = tmem_p + PK_BN;
    bool ok = true;
    pdl_wait();  // the plan, Q, K and V come from earlier kernels
    pdl_trigger();

    // This CTA's items, n_tiles = 0: none left. The first Ly::TABLE are looked up at the start by all threads (looked up by each role
    // when its turn came, an item cost some 1,000 cycles of it).
    const int Hq = a.Hq, pg_log = a.pg_log, groups = Hq >> pg_log, tpt_log = 7 - pg_log;  // tokens of a tile
    const int level = min(pg_log, kPlanLevels - 1), places = groups << (pg_log - level);  // tiles of an entry
    const int first_entry = (int)min(max(a.plan->first[level], 0ll), (long long)a.capacity);
    const int n_items = min(max(a.plan->count[level], 0), a.capacity - first_entry) * places;
    const int G = (int)gridDim.x, me = (int)blockIdx.x;
    int4* table = reinterpret_cast<int4*>(smem + Ly::TABLE_OFF);
    auto look_up = [&](int round) -> int4 {  // first query row, query rows + 256 * group of heads, first key row, key position
        const int k = round * G + ((round & 1) ? G - 1 - me : me);
        const int entry = (int)((unsigned)k / (unsigned)places), rem = k - entry * places;
        const int sub = (int)((unsigned)rem / (unsigned)groups), first = sub << tpt_log;
        const int4 v = __ldg(a.items + first_entry + entry);
        // 0: the entry has fewer tokens, or is none of a plan for these queries
        const int rows = (unsigned)v.x < (unsigned)a.Nq ? max(0, min(v.y - first, 1 << tpt_log)) : 0;
        return make_int4(v.x + first, rows + 256 * (rem - sub * groups), v.z, v.w + first);
    };
    auto is_item = [&](int round) { return round * G + ((round & 1) ? G - 1 - me : me) < n_items; };
    for (int round = threadIdx.x; round < Ly::TABLE && round <= n_items / G && is_item(round); round += PK_THREADS)
        table[round] = look_up(round);
    __syncthreads();
    struct Item {
        int q0, q_end, k0, pos0, hg, n_valid, n_tiles;  // hg: group of PG heads
    };
    int next_round = 0;
    auto next_item = [&]() -> Item {
        Item it{};
        while (true) {
            const int round = next_round;
            if (!is_item(round)) return it;
            ++next_round;
            const int4 v = round < Ly::TABLE ? table[round] : look_up(round);
            const int rows = v.y & 255;
            if (rows == 0) continue;
            it.hg = v.y >> 8;
            it.q0 = v.x;
            it.q_end = min(v.x + rows, a.Nq);
            it.k0 = v.z;
            it.pos0 = v.w;
            it.n_valid = min(max(v.w + rows, 0), a.max_keys);
            it.n_tiles = max(1, (it.n_valid + PK_BN - 1) / PK_BN);  // without a key: one tile, all of it masked
            return it;
        }
    };

    // A role ends when what it has asked for is done, also after a wait of the CTA gave up: no copy or product of this CTA may
    // land in shared or tensor memory that the next one has taken over. These last waits are bounded and look at no flag.
    int never = 0;
    bool arrives = true;
    auto last_wait = [&](uint64_t* bar, int parity) { arrives = arrives && mbar_wait_suspend(bar, parity, &never); };

    if (warp < 4) {
        setmaxnreg_dec<PK_REG_PRODUCER>();
        if (warp == 0) {
            // ---------------- Q and key tiles
            if (lane == 0) {
                int g = 0, n = 0;
                for (; ok; ++n) {
                    const Item it = next_item();
                    if (it.n_tiles == 0) break;
                    const int jkv = it.hg / (groups / a.Hkv), qs = n % QST;
                    if (!mbar_wait_suspend(&q_empty[qs], ((n / QST) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    mbar_expect_tx(&q_full[qs], TB);
                    tma_load_5d(smem + qs * TB, &tmQ, &q_full[qs], 0, 0, it.q0, 0, it.hg);
                    for (int i = 0; i < it.n_tiles; ++i, ++g) {
                        const int s = g % KST;
                        if (!mbar_wait_suspend(&k_empty[s], ((g / KST) & 1) ^ 1, abort_flag)) { ok = false; break; }
                        mbar_expect_tx(&k_full[s], TB);
                        tma_load_3d(smem + Ly::K_OFF + s * TB, &tmK, &k_full[s], 0, it.k0 + i * PK_BN, jkv * NCH);
                    }
                    if (!ok) {
                        ++n;  // (its Q was asked for)
                        break;
                    }
                }
                drain_ring(g, KST, [&](int s, int parity) { last_wait(&k_full[s], parity); });
                drain_ring(n, QST, [&](int s, int parity) { last_wait(&q_full[s], parity); });
            }
        } else if (warp == 1) {
            // ---------------- S of tile g, once the scores of the tile before have been read
            if (lane == 0) {
                int g = 0;
                for (int n = 0; ok; ++n) {
                    const Item it = next_item();
                    const int nt = it.n_tiles, qs = n % QST;
                    if (nt == 0) break;
                    if (!mbar_wait_suspend(&q_full[qs], (n / QST) & 1, abort_flag)) { ok = false; break; }
                    for (int i = 0; i < nt; ++i, ++g) {
                        const int s = g % KST;
                        if (!mbar_wait_suspend(&k_full[s], (g / KST) & 1, abort_flag)) { ok = false; break; }
                        if (!mbar_wait_suspend(s_empty, (g & 1) ^ 1, abort_flag)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t sq = smem_u32(smem + qs * TB), sk = smem_u32(smem + Ly::K_OFF + s * TB);
#pragma unroll
                        for (int kk = 0; kk < DH / 16; ++kk) {
                            const uint32_t off = (kk >> 2) * PK_BM * 128 + (kk & 3) * 32;
                            umma_bf16_ss(tmem, sdesc_kmajor_sw128(sq + off), sdesc_kmajor_sw128(sk + off), IDESC_S, kk > 0);
                        }
                        umma_commit(s_full);
                        umma_commit(&k_empty[s]);
                        if (i == nt - 1) umma_commit(&q_empty[qs]);  // the item's last scores release Q
                    }
                }
                if (g > 0) last_wait(s_full, (g - 1) & 1);  // (completes behind every earlier tile's)
            }
        } else if (warp == 2) {
            // ---------------- value tiles
            if (lane == 0) {
                int g = 0;
                while (ok) {
                    const Item it = next_item();
                    if (it.n_tiles == 0) break;
                    const int jkv = it.hg / (groups / a.Hkv);
                    for (int i = 0; i < it.n_tiles; ++i, ++g) {
                        const int s = g % VST;
                        if (!mbar_wait_suspend(&v_empty[s], ((g / VST) & 1) ^ 1, abort_flag)) { ok = false; break; }
                        mbar_expect_tx(&v_full[s], TB);
                        tma_load_3d(smem + Ly::V_OFF + s * TB, &tmV, &v_full[s], 0, it.k0 + i * PK_BN, jkv * NCH);
                    }
                }
                drain_ring(g, VST, [&](int s, int parity) { last_wait(&v_full[s], parity); });
            }
        } else {
            // ---------------- O += P V of tile g: P as A operand in tensor memory, V from stage g % VST
            int g = 0, done = 0;
            for (int n = 0; ok; ++n) {
                const Item it = next_item();
                const int nt = it.n_tiles;
                if (nt == 0) break;
                const uint32_t to = tmem_o + (n & 1) * 128;
                for (int i = 0; ok && i < nt; ++i, ++g) {
                    const int s = g % VST;
                    const uint32_t tp = tmem_p + (g & 1) * 64;
                    if (!__all_sync(0xffffffffu, mbar_wait_suspend(&v_full[s], (g / VST) & 1, abort_flag))) { ok = false; break; }
                    uint8_t* sv_p = smem + Ly::V_OFF + s * TB;
                    const int r0 = it.n_valid - i * PK_BN;  // value rows from here on are not seen by the item, and may hold anything
                    const int steps = min(PK_BN / 16, (max(r0, 1) + 15) / 16);  // 16-row steps that hold a seen one
                    if (r0 < PK_BN) {  // (0 * NaN must not reach O)
                        for (int e = lane; e < (steps * 16 - r0) * 8 * NCH; e += 32) {
                            const int row = r0 + e / (8 * NCH), p = e % (8 * NCH);
                            reinterpret_cast<uint4*>(sv_p + (p >> 3) * PK_BN * 128 + row * 128)[p & 7] = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        bool w = i > 0 || mbar_wait_suspend(&o_free[n & 1], ((n >> 1) & 1) ^ 1, abort_flag);  // item n - 2's O is read out
                        w = w && mbar_wait_suspend(&p_full[g & 1], (g >> 1) & 1, abort_flag);
                        if (w) {
                            tc_fence_after();
                            const uint32_t sv = smem_u32(sv_p);
                            if (steps < PK_BN / 16) {
                                for (int kk = 0; kk < steps; ++kk)
                                    umma_bf16_ts(to, tp + kk * 8, sdesc_mnmajor_sw128(sv + kk * 16 * 128, PK_BN * 128),
                                                 IDESC_O, (i | kk) != 0);
                            } else {
#pragma unroll
                                for (int kk = 0; kk < PK_BN / 16; ++kk)
                                    umma_bf16_ts(to, tp + kk * 8, sdesc_mnmajor_sw128(sv + kk * 16 * 128, PK_BN * 128),
                                                 IDESC_O, (i | kk) != 0);
                            }
                            umma_commit(&pv_done[g & 1]);
                            umma_commit(&v_empty[s]);
                            if (i == nt - 1) umma_commit(&o_full[n & 1]);
                            ++done;
                        }
                        ok = w;
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                }
            }
            if (lane == 0 && done > 0) last_wait(&pv_done[(done - 1) & 1], ((done - 1) >> 1) & 1);
            __syncwarp();
        }
    } else if (warp < 8) {
        setmaxnreg_inc<PK_REG_SOFTMAX>();
        // ---------------- softmax: thread <-> query row (TMEM lane)
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const float sl2 = kLog2e / sqrtf((float)DH);
        int g = 0;
        for (int n = 0; ok; ++n) {
            const Item it = next_item();
            const int nt = it.n_tiles;
            if (nt == 0) break;
            const int pos = it.pos0 + (row >> pg_log);
            const uint32_t to = tmem_o + (n & 1) * 128 + lane_off;
            float m = -INFINITY, l = 0.f;  // the row's scale (log2 units) and sum
            for (int i = 0; i < nt; ++i, ++g) {
                const uint32_t ts = tmem + lane_off, tp = tmem_p + (g & 1) * 64 + lane_off;
                if (!__all_sync(0xffffffffu, mbar_wait_suspend(s_full, g & 1, abort_flag))) { ok = false; break; }
                tc_fence_after();
                uint32_t sr[PK_BN];
#pragma unroll
                for (int c = 0; c < PK_BN / 32; ++c)
                    tmem_ld_32x32b_x32(ts + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty);  // the next tile's scores may come
                if (i * PK_BN + PK_BN - 1 > it.pos0) {  // some row does not see all of the tile
                    const int lim = pos - i * PK_BN;    // last visible column
#pragma unroll
                    for (int c = 0; c < PK_BN / 32; ++c) {  // (a warp's rows are 32 tokens at most: one or two parts are mixed)
                        const uint32_t vis = low_bits(lim + 1 - 32 * c);
                        if (__all_sync(0xffffffffu, vis == 0xffffffffu)) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            sr[c * 32 + e] = vis & (1u << e) ? sr[c * 32 + e] : __float_as_uint(-INFINITY);
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // independent chains
#pragma unroll
                for (int e = 0; e < PK_BN; e += 2)
                    mx4[e / 2 % 4] = fmax3(mx4[e / 2 % 4], __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
                // lazy rescale, decided per row but executed by the whole warp (tcgen05.ld/st are warp-wide)
                const bool grow = mx > m + 8.0f;
                const float alpha = grow ? ex2_approx(m - mx) : 1.0f;
                if (i > 0 && __any_sync(0xffffffffu, grow)) {
                    // O must hold every earlier tile's P V. (The next P V of this parity needs a P that is not released yet: the
                    // phase cannot alias.)
                    const int k = g - 1;
                    if (!__all_sync(0xffffffffu, mbar_wait_suspend(&pv_done[k & 1], (k >> 1) & 1, abort_flag))) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DH / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(to + c * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st_32x32b_x32(to + c * 32, o);
                    }
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
                // P V of the tile before last has used the place
                if (!__all_sync(0xffffffffu, mbar_wait_suspend(&pv_done[g & 1], ((g >> 1) & 1) ^ 1, abort_flag))) { ok = false; break; }
                tc_fence_after();
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
                    tmem_st_32x32b_x32(tp + half * 32, pk);
                }
                tmem_st_wait();
                l += rs2.x + rs2.y;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[g & 1]);
            }
            if (!ok) break;
            // the sums go to the output warps, once those of item n - 2 have been read
            if (!__all_sync(0xffffffffu, mbar_wait_suspend(&o_free[n & 1], ((n >> 1) & 1) ^ 1, abort_flag))) { ok = false; break; }
            inv_sh[(n & 1) * PK_BM + row] = l == 0.f ? 0.f : 1.f / l;  // (a row without a key: zeros)
            __syncwarp();
            if (lane == 0) mbar_arrive(&l_full[n & 1]);
        }
    } else {
        setmaxnreg_dec<PK_REG_OUTPUT>();
        // ---------------- output: thread <-> query row
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        for (int n = 0; ok; ++n) {
            const Item it = next_item();
            if (it.n_tiles == 0) break;
            const int ph = (n >> 1) & 1;
            const uint32_t to = tmem_o + (n & 1) * 128 + lane_off;
            if (!__all_sync(0xffffffffu, mbar_wait_suspend(&l_full[n & 1], ph, abort_flag) &&
                                             mbar_wait_suspend(&o_full[n & 1], ph, abort_flag))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float inv = inv_sh[(n & 1) * PK_BM + row];
            const int row0 = quarter * 32 + (lane & ~3);  // of the four rows that four neighbouring lanes hold and store together
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + c * 32, o);
                tmem_ld_wait();
                // 16-byte pieces change places within groups of four lanes, so that a group stores 64 contiguous bytes of
                // one row at a time (lane k piece j -> lane j piece k)
                uint4 w[4];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    w[v] = make_uint4(pack_bf16(__uint_as_float(o[8 * v]) * inv, __uint_as_float(o[8 * v + 1]) * inv),
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
                for (int v = 0; v < 4; ++v) {
                    const int r = row0 + v, t = it.q0 + (r >> pg_log), h = (it.hg << pg_log) + (r & ((1 << pg_log) - 1));
                    if (t < it.q_end)
                        *reinterpret_cast<uint4*>(a.out + ((size_t)t * Hq + h) * DH + c * 32 + (lane & 3) * 8) = w[v];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[n & 1]);
        }
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

// Keys up to which a batch's longest sequence counts as short.
constexpr int kPackedShort = 1024;

template <int DH, bool LONG>
cudaError_t packed_launch_form(const PackedCall& c, cudaStream_t st) {
    // heads of a tile: the largest power of two in the group, up to a tile's rows
    int pg_log = 0;
    while (pg_log < 7 && (c.Hq / c.Hkv) % (2 << pg_log) == 0) ++pg_log;
    CUtensorMap tq, tk, tv;
    // without a key row there is nothing to read: any memory serves as the masked tile
    const bool none = c.Nk == 0;
    const void *k = none ? c.q : c.k, *v = none ? c.q : c.v;
    const uint64_t rows = none ? 1 : c.Nk, ldk = none ? c.ldq : c.ldk, ldv = none ? c.ldq : c.ldv;
    const uint64_t blocks = (uint64_t)c.Hkv * (DH / 64);
    if (!encode_tmap_bf16_head_groups(&tq, c.q, DH, 1u << pg_log, c.Hq >> pg_log, c.Nq, (uint64_t)c.ldq * 2, PK_BM >> pg_log) ||
        !encode_tmap_bf16_rows(&tk, k, blocks, rows, ldk * 2, PK_BN, DH / 64) ||
        !encode_tmap_bf16_rows(&tv, v, blocks, rows, ldv * 2, PK_BN, DH / 64))
        return cudaErrorInvalidValue;
    const PackedArgs a{reinterpret_cast<const int4*>(static_cast<const char*>(c.plan) + kPlanHeader),
                       static_cast<const PlanHeader*>(c.plan), c.capacity, c.Nk, c.Nq, c.Hq, c.Hkv, pg_log, c.out, c.err};
    const unsigned grid = (unsigned)std::min<long long>((long long)c.capacity * c.Hq, device_sm_count());
    return launch_pdl(attn_packed_kernel<DH, LONG>, dim3(grid), dim3(PK_THREADS), PkLayout<DH, LONG>::SMEM, st, tq, tk, tv, a);
}
template <int DH>
cudaError_t packed_launch_dh(const PackedCall& c, cudaStream_t st) {
    if constexpr (DH == 128)
        if (c.longest <= kPackedShort) return packed_launch_form<DH, false>(c, st);
    return packed_launch_form<DH, true>(c, st);
}

// setmaxnreg.inc waits until the registers it asks for are free: the compiled kernel has to be given at least those that its
// split hands out.
template <int DH, bool LONG>
cudaError_t packed_prepare_form() {
    cudaFuncAttributes fa{};
    cudaError_t e = cudaFuncGetAttributes(&fa, attn_packed_kernel<DH, LONG>);
    if (e != cudaSuccess) return e;
    if (PK_THREADS * fa.numRegs < 128 * (int)(PK_REG_PRODUCER + PK_REG_SOFTMAX + PK_REG_OUTPUT)) return cudaErrorLaunchOutOfResources;
    return cudaFuncSetAttribute(attn_packed_kernel<DH, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, PkLayout<DH, LONG>::SMEM);
}

}  // namespace

size_t attn_packed_plan_bytes(int Nq, int S) {
    size_t n = 0;
    for (int level = 0; level < kPlanLevels; ++level) n += plan_level(Nq, S, level);
    return kPlanHeader + n * sizeof(int4);
}
int attn_packed_capacity(size_t bytes) {
    return bytes < kPlanHeader ? 0 : (int)std::min<size_t>((bytes - kPlanHeader) / sizeof(int4), 0x7fffffff);
}
cudaError_t attn_packed_plan_launch(const int* cu_q, const int* cu_k, int S, int Nq, int Nk, void* plan, int* err,
                                    cudaStream_t st) {
    PlanHeader at{};
    long long first = 0;
    for (int level = 0; level < kPlanLevels; ++level) {
        at.count[level] = (int)plan_level(Nq, S, level);
        at.first[level] = first;
        first += at.count[level];
    }
    return launch_pdl(attn_packed_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, cu_q, cu_k, S, Nq, Nk, at,
                      static_cast<PlanHeader*>(plan), reinterpret_cast<int4*>(static_cast<char*>(plan) + kPlanHeader), err);
}
cudaError_t attn_packed_launch(const PackedCall& c, int dh, cudaStream_t st) {
    if (dh == 128) return packed_launch_dh<128>(c, st);
    if (dh == 64) return packed_launch_dh<64>(c, st);
    return cudaErrorInvalidValue;
}
cudaError_t attention_packed_prepare() {
    cudaError_t e = packed_prepare_form<128, true>();
    if (e == cudaSuccess) e = packed_prepare_form<128, false>();
    return e == cudaSuccess ? packed_prepare_form<64, true>() : e;
}

}  // namespace q3
