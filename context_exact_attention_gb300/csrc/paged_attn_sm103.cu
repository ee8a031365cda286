// paged_attn_sm103.cu -- paged_attn_fwd for calls with many query rows per key/value head
// (chunks of prompts, mixed batches), bf16 on the tensor cores (tcgen05 + TMEM + TMA).
//
// One persistent CTA per SM takes its part of the call's tiles (paged_plan.cuh).  A tile is
// two 128-row query sub-tiles of one key/value head: 128 / G tokens with the G query heads
// that read the head, token-major, so that every key block loaded into shared memory serves
// all of them.  The roles are those of the dense forward (attn_bf16_sm103.cu):
//   warp 0      producer: walks the CTA's segments, publishes each to the other warps
//               through a two-slot ring in shared memory, and loads the query sub-tiles
//               and the 128-key blocks of K by TMA, in boxes of keys that share a page
//               (one lane each, the page-table entries fetched a block ahead);
//   warp 2      loads the blocks of V in the same way;
//   warp 1      issues S_t = Q_t K^T and O_t += P_t V;
//   warps 4-7, 8-11  softmax of sub-tile 0, 1: one thread per row.
// The sub-tiles ping-pong, and the next segment's loads and first products overlap the
// output of the last.  A tile with no more than one sub-tile of rows would leave the tensor
// core idle during its softmax; it ping-pongs with itself instead: the two warpgroups take
// its even and odd key blocks, each with its own running softmax and its own O, and the
// first one adds the second's result to its own at the end (both hold a row in the same
// lane, so it reads the other's O from TMEM directly).
//
// A box of a page that the table does not name properly, or of a page behind the last key,
// is loaded at an index outside the tensor, which TMA fills with zeros without reading
// memory.  Slots behind the last key in its page hold whatever they hold: their scores are
// masked, and their rows of V are zeroed in shared memory before the product (0 times NaN
// is NaN), which only the last block of a sequence needs.
//
// TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D).
//
// Measured (1.9 GHz cycles): a block of two sub-tiles takes 2500 cycles at head dim 128, of
// which the four products are 2048, and 2700 at 64, where each sub-tile's softmax (1750) and
// its turn at the issuing warp bound it; a block of a single sub-tile 2300 at 128 (the K and V
// loads: 64 KB at an SM's share of HBM) and 1500 at 64.  A chunk of 2048 tokens ending at
// 32768, 32 heads over 8, takes 625 to 635 us (1.68 to 1.70 PFLOP/s; 690 to 720 us back to
// back at the power cap); 32 sequences of 5 proposed tokens over up to 8192 keys 54 us
// (5.1 TB/s).  Outside the blocks a CTA spends 6000 cycles before the first, 2500 to 4800 on
// an output, 3000 to 8000 on a partial, and a joining CTA 6000 (40 rows) to 24000 (256 rows).
// The weights go into P V as one bf16 each (2^-9 to 2^-8 relative): a second part, which the
// kernel for few rows adds, would double the product that bounds this one.  Relative to the
// result's size the error is 2.1e-3 to 2.3e-3 where fp32 weights have 1.6e-3 to 1.7e-3, the
// output's own rounding.
#include <cuda.h>

#include <type_traits>

#include "paged_plan.cuh"

namespace ra {
namespace {

constexpr int kSub = 128;         // rows of a sub-tile = TMEM lanes
constexpr int kKeys = 128;        // keys per block
constexpr int kThreads = 384;
constexpr int kReaders = 2 + 8;   // warps that read a published segment
constexpr float kRescaleThreshold = 8.0f;
// A scaled maximum is rounded by up to 2^-24 of it, and that is what the fused multiply-add
// leaves of its exponent, which for huge scores would overflow.  From 2^29 on (rounded by 32)
// two scores that differ at all differ by 2^-23 2^29, and a weight is 1 or nothing whatever the
// scale is: they are taken times a power of two, which rounds nothing.
constexpr float kFar = 536870912.f;
constexpr float kFarScale = 0.25f;

template <int D>
struct Layout {
    static constexpr int kBoxes = D / 64;
    static constexpr int kTile = 128 * D * 2;
    static constexpr int kStages = D == 64 ? 4 : 2;   // of the K and the V ring: 64 KB each
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kStage = kV + kStages * kTile;   // 8 warps x 32 rows x D/2 bf16
    // (a slice holds 32 rows of 32 floats or of D/2 bf16)
    static constexpr int kBar = kStage + 8 * 32 * 128;
    static constexpr int kSmem = kBar + 2048 + 1024;  // barriers, segments; alignment slack
    __device__ static constexpr uint32_t col_s(int t) { return 128u * t; }
    __device__ static constexpr uint32_t col_o(int t) { return 256u + static_cast<uint32_t>(D) * t; }
};

enum : int {
    kBarQ = 0,           // +sub-tile: queries loaded
    kBarQEmpty = 2,      // +sub-tile: the segment's last Q K^T of the sub-tile finished
    kBarKFull = 4,       // +stage (up to 4)
    kBarKEmpty = 8,      // +stage
    kBarVFull = 12,      // +stage
    kBarVEmpty = 16,     // +stage
    kBarSFull = 20,      // +sub-tile
    kBarPFull = 22,      // +2 sub-tile + half
    kBarOFull = 26,      // +sub-tile
    kBarSegFull = 28,    // +slot
    kBarSegEmpty = 30,   // +slot
    kBarPart = 32,       // the eight softmax warps have written their partials
    kBarFlag = 33,       // whether this CTA joins them is known
    kBarOdd = 34,        // single sub-tile: the odd blocks' statistics are in shared memory
    kBarAdded = 35,      // ... and their O has been read
    kBarDone = 36,
    kBarCount = 37
};
// shared-memory words after the barriers
constexpr int kTmemSlot = kBarCount * 8, kAbort = kTmemSlot + 4, kLast = kTmemSlot + 8;
constexpr int kSegInts = 14;
constexpr int kSegSlots = kTmemSlot + 16;                   // 2 slots of kSegInts ints
constexpr int kOddStat = (kSegSlots + 2 * kSegInts * 4 + 7) / 8 * 8;   // 128 x (maximum, denominator)
static_assert(kOddStat + kSub * 8 <= 2048, "barrier area");

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}

// What the other warps need of a segment.
struct Seg {
    int g, hk, rows, n_sub, first, n, kv, k0, n_blocks, c_first, c_last, row0;
    int once;               // the sequence's keys are read by this tile alone
};
__device__ __forceinline__ void publish(volatile int* e, int more, const Seg& s)
{
    e[0] = more;
    e[1] = s.hk;
    e[2] = s.rows;
    e[3] = s.n_sub;
    e[4] = s.first;
    e[5] = s.n;
    e[6] = s.kv;
    e[7] = s.k0;
    e[8] = s.n_blocks;
    e[9] = s.c_first;
    e[10] = s.c_last;
    e[11] = s.row0;
    e[12] = s.g;
    e[13] = s.once;
}
__device__ __forceinline__ bool consume(volatile int* e, Seg& s)
{
    s.hk = e[1];
    s.rows = e[2];
    s.n_sub = e[3];
    s.first = e[4];
    s.n = e[5];
    s.kv = e[6];
    s.k0 = e[7];
    s.n_blocks = e[8];
    s.c_first = e[9];
    s.c_last = e[10];
    s.row0 = e[11];
    s.g = e[12];
    s.once = e[13];
    return e[0] != 0;
}

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }

// kTree: rows see the new tokens that their masks name.
template <int D, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmap_q,
                    const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v,
                    const __grid_constant__ PagedParams p)
{
    using Lay = Layout<D>;
    using Walk = PagedWalk<std::conditional_t<kTree, WeighedTiles, StepTiles>, kKeys>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    uint8_t* area = smem + Lay::kBar;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(area + kTmemSlot);
    int* abort_flag = reinterpret_cast<int*>(area + kAbort);
    volatile int* last_flag = reinterpret_cast<volatile int*>(area + kLast);
    volatile int* seg_slot = reinterpret_cast<volatile int*>(area + kSegSlots);
    auto bar = [&](int i) -> uint32_t { return sbase + Lay::kBar + 8u * i; };
    const PagedArgs& a = p.a;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int sub_tokens = p.tile_tokens / 2;
    const int sub_rows = sub_tokens * p.G;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Lay::kStages; ++i) {
            mbar_init(bar(kBarKFull + i), 1);
            mbar_init(bar(kBarKEmpty + i), 1);
            mbar_init(bar(kBarVFull + i), 1);
            mbar_init(bar(kBarVEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarQ + i), 1);
            mbar_init(bar(kBarQEmpty + i), 1);
            mbar_init(bar(kBarSFull + i), 1);
            mbar_init(bar(kBarPFull + 2 * i), kSub);
            mbar_init(bar(kBarPFull + 2 * i + 1), kSub);
            mbar_init(bar(kBarOFull + i), 1);
            mbar_init(bar(kBarSegFull + i), 1);
            mbar_init(bar(kBarSegEmpty + i), kReaders);
        }
        mbar_init(bar(kBarPart), 8);
        mbar_init(bar(kBarFlag), 1);
        mbar_init(bar(kBarOdd), 4);
        mbar_init(bar(kBarAdded), 4);
        mbar_init(bar(kBarDone), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    wait_for_earlier_work();
    const uint32_t tmem = *tmem_slot;
    WaitCtx wc{abort_flag, a.status, a.timeout_ns};

    // The i-th segment of this CTA, as the consumer warps get it (false: no more).
    auto get_seg = [&](int i, Seg& s) -> bool {
        const int slot = i & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarSegFull + slot), (i >> 1) & 1, wc)))
            return false;
        const bool more = consume(seg_slot + kSegInts * slot, s);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarSegEmpty + slot));
        return more;
    };

    constexpr int kStages = Lay::kStages;
    auto stage_of = [](uint32_t n) -> int { return n % kStages; };
    auto phase_of = [](uint32_t n) -> uint32_t { return (n / kStages) & 1; };

    // Loads the blocks of a segment into the K or the V ring and counts them in N, the blocks
    // loaded so far (whole warp; false: a wait ran out).  Lane: box lane / kBoxes of the block,
    // columns 64 (lane mod kBoxes).
    auto load_blocks = [&](const Seg& s, const CUtensorMap* map, int ring, int full, int empty,
                           uint32_t& N, bool leader) -> bool {
        const uint64_t policy = s.once ? l2_policy_evict_first() : l2_policy_evict_last();
        const int box_rows = p.box_rows;
        const int my_box = lane / Lay::kBoxes, my_col = lane % Lay::kBoxes;
        const bool loads = my_box < kKeys / box_rows;         // at most 16 boxes a block
        const uint32_t to = my_col * 16384 + my_box * box_rows * 128;
        // the page and slot of this lane's box of the block at key kb: an index outside the
        // cache (zeros) behind the last key and for an entry that names no page
        auto page_of = [&](int kb, int& in_page) -> int {
            const int key = kb + my_box * box_rows;
            const int col = p.page_shift >= 0 ? key >> p.page_shift : key / a.page_size;
            int page = -1;
            if (loads && key < s.kv)
                page = checked_ldg(a.page_table, s.g * a.table_stride + col, a.table_elems, a.status);
            in_page = key - col * a.page_size;
            return static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages) ? page
                                                                                  : a.num_pages;
        };
        int in_page = 0, in_next = 0;
        int page = page_of(s.k0, in_page);
        for (int n = 0; n < s.n_blocks; ++n, ++N) {
            const int kb = s.k0 + n * kKeys;
            const int page_next = n + 1 < s.n_blocks ? page_of(kb + kKeys, in_next) : 0;
            const int st = stage_of(N);
            if (!__all_sync(0xffffffffu, mbar_wait(bar(empty + st), phase_of(N) ^ 1, wc)))
                return false;
            if (leader) mbar_arrive_expect_tx(bar(full + st), Lay::kTile);
            __syncwarp();
            if (loads)
                tma_load_4d(sbase + ring + st * Lay::kTile + to, map, bar(full + st), my_col * 64,
                            s.hk, in_page, page, policy);
            page = page_next;
            in_page = in_next;
        }
        return true;
    };
    // Lets this warp's own copies into a ring land (N blocks loaded).
    auto drain = [&](int full, uint32_t N) {
        for (uint32_t n = N > kStages ? N - kStages : 0; n < N; ++n)
            mbar_wait_drain(bar(full + stage_of(n)), phase_of(n), wc);
        __syncwarp();
    };

    if (warp == 0) {
        // ---------------------------------------------- segments, queries and keys
        const bool leader = elect_one();
        if (leader) {
            tma_prefetch_desc(&tmap_q);
            tma_prefetch_desc(&tmap_k);
        }
        const uint64_t once = l2_policy_evict_first();
        uint32_t N = 0;
        uint32_t q_loads[2] = {0, 0};                         // query loads per sub-tile so far
        bool ok = true;
        Segment t;
        Walk walk;
        walk.begin(p);
        for (int i = 0; ok; ++i) {
            const bool more = walk.next(p, t);
            Seg s{};
            if (more) {
                s.g = t.g;
                s.hk = t.hk;
                s.rows = t.rows;
                s.n_sub = t.rows > sub_rows ? 2 : 1;
                s.first = t.s.first;
                s.n = t.s.n;
                s.kv = t.s.kv;
                s.k0 = t.k0;
                s.n_blocks = t.k1 > t.k0 ? (t.k1 - t.k0 + kKeys - 1) / kKeys : 0;
                s.c_first = t.c_first;
                s.c_last = t.c_last;
                s.row0 = t.row0;
                s.once = t.s.n <= p.tile_tokens;
            }
            const int slot = i & 1;
            if (i >= 2 &&
                !(ok = __all_sync(0xffffffffu,
                                  mbar_wait(bar(kBarSegEmpty + slot), ((i - 2) >> 1) & 1, wc))))
                break;
            if (leader) {
                publish(seg_slot + kSegInts * slot, more, s);
                mbar_arrive(bar(kBarSegFull + slot));
            }
            __syncwarp();
            if (!more) break;
            if (s.n_blocks == 0) continue;
            const int tok0 = s.first + p.token_of(s.row0);
#pragma unroll
            for (int tq = 0; tq < 2; ++tq) {
                if (tq >= s.n_sub) break;
                if (q_loads[tq] > 0 &&
                    !(ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarQEmpty + tq),
                                                             (q_loads[tq] - 1) & 1, wc))))
                    break;
                if (leader) {
                    mbar_arrive_expect_tx(bar(kBarQ + tq), sub_rows * D * 2);
                    for (int bx = 0; bx < Lay::kBoxes; ++bx)
                        tma_load_3d(sbase + Lay::kQ + tq * Lay::kTile + bx * 16384, &tmap_q,
                                    bar(kBarQ + tq), bx * 64, s.hk * p.G, tok0 + tq * sub_tokens, once);
                }
                ++q_loads[tq];
                __syncwarp();
            }
            if (!ok) break;
            ok = load_blocks(s, &tmap_k, Lay::kK, kBarKFull, kBarKEmpty, N, leader);
        }
        for (int tq = 0; tq < 2; ++tq)
            if (q_loads[tq] > 0) mbar_wait_drain(bar(kBarQ + tq), (q_loads[tq] - 1) & 1, wc);
        drain(kBarKFull, N);
    } else if (warp == 2) {
        // ---------------------------------------------------------------- values
        // (a warp of their own: a stage of V is held until its weights are ready, and the
        // next keys must not wait for that)
        const bool leader = elect_one();
        if (leader) tma_prefetch_desc(&tmap_v);
        uint32_t N = 0;
        bool ok = true;
        Seg s;
        for (int i = 0; ok; ++i) {
            if (!get_seg(i, s)) break;
            ok = load_blocks(s, &tmap_v, Lay::kV, kBarVFull, kBarVEmpty, N, leader);
        }
        drain(kBarVFull, N);
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        constexpr uint32_t kIdescQK = idesc_bf16_f32(kSub, kKeys, false);
        constexpr uint32_t kIdescPV = idesc_bf16_f32(kSub, D, true);
        constexpr uint64_t kTileU = Lay::kTile >> 4;
        const uint64_t dq = sdesc_sw128(sbase + Lay::kQ, 16, 1024);
        const uint64_t dk = sdesc_sw128(sbase + Lay::kK, 16, 1024);
        const uint64_t dv = sdesc_sw128(sbase + Lay::kV, 16384, 1024);
        // S_x = Q_tq K^T, O_x += P_x V
        auto issue_qk = [&](int tq, int x, int st) {
            const uint32_t d_t = tmem + Lay::col_s(x);
            const uint64_t a0 = dq + tq * kTileU, b0 = dk + st * kTileU;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                mma_ss(d_t, a0 + off, b0 + off, kIdescQK, k > 0 ? 1u : 0u);
            }
        };
        auto issue_pv = [&](int tq, int st, int half, bool acc) {
            const uint32_t d_t = tmem + Lay::col_o(tq);
            const uint32_t pa = tmem + Lay::col_s(tq) + 32 * half;
            const uint64_t b0 = dv + st * kTileU + ((half * 64 * 128) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_ts(d_t, pa + k * 8, b0 + ((k * 2048) >> 4), kIdescPV, (acc || k > 0) ? 1u : 0u);
        };
        auto wait_all = [&](int idx, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar(idx), parity, wc));
        };
        // rows of V behind the last key of the sequence become zeros (block n of the segment)
        auto clean_tail = [&](const Seg& s, int n, int st, uint32_t ph) -> bool {
            const int held = s.kv - (s.k0 + n * kKeys);       // keys of the block that exist
            if (held >= kKeys) return true;
            if (!wait_all(kBarVFull + st, ph)) return false;
            const int from = max(held, 0);
            uint8_t* v = smem + Lay::kV + st * Lay::kTile;
            for (int i = lane; i < (kKeys - from) * 8 * Lay::kBoxes; i += 32) {
                const int r = i / (8 * Lay::kBoxes), c = i % (8 * Lay::kBoxes);
                *reinterpret_cast<uint4*>(v + (c >> 3) * 16384 + (from + r) * 128 + (c & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            return true;
        };
        uint32_t N = 0;
        uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};     // query loads; blocks of each sub-tile
        bool ok = true;
        Seg s;
        for (int i = 0; ok; ++i) {
            if (!get_seg(i, s)) break;
            if (s.n_blocks == 0) continue;
            const int st0 = stage_of(N);
            ok = wait_all(kBarQ, qn[0] & 1) && wait_all(kBarKFull + st0, phase_of(N));
            if (!ok) break;
            ++qn[0];
            if (s.n_sub == 1) {
                // even blocks through S0, O0, odd ones through S1, O1, the same queries
                tc_fence_after();
                if (leader) {
                    issue_qk(0, 0, st0);
                    tc_commit(bar(kBarSFull + 0));
                    tc_commit(bar(kBarKEmpty + st0));
                    if (s.n_blocks == 1) tc_commit(bar(kBarQEmpty + 0));
                }
                __syncwarp();
                if (s.n_blocks > 1) {
                    const int st1 = stage_of(N + 1);
                    if (!(ok = wait_all(kBarKFull + st1, phase_of(N + 1)))) break;
                    tc_fence_after();
                    if (leader) {
                        issue_qk(0, 1, st1);
                        tc_commit(bar(kBarSFull + 1));
                        tc_commit(bar(kBarKEmpty + st1));
                        if (s.n_blocks == 2) tc_commit(bar(kBarQEmpty + 0));
                    }
                    __syncwarp();
                }
                for (int n = 0; n < s.n_blocks; ++n) {
                    const int x = n & 1;
                    const int st = stage_of(N + n), st2 = stage_of(N + n + 2);
                    const uint32_t ph = phase_of(N + n);
                    const bool more = n + 2 < s.n_blocks;         // of this block's parity
                    if (!(ok = clean_tail(s, n, st, ph))) break;
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait2(bar(kBarVFull + st), ph,
                                                                  bar(kBarPFull + 2 * x), pn[x] & 1,
                                                                  wc))))
                        break;
                    tc_fence_after();
                    if (leader) issue_pv(x, st, 0, n > 1);
                    __syncwarp();
                    ok = more ? mbar_wait2(bar(kBarPFull + 2 * x + 1), pn[x] & 1,
                                           bar(kBarKFull + st2), phase_of(N + n + 2), wc)
                              : mbar_wait(bar(kBarPFull + 2 * x + 1), pn[x] & 1, wc);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    if (leader) {
                        issue_pv(x, st, 1, true);
                        tc_commit(bar(kBarVEmpty + st));
                        if (!more) tc_commit(bar(kBarOFull + x));
                        if (more) {
                            issue_qk(0, x, st2);
                            tc_commit(bar(kBarSFull + x));
                            tc_commit(bar(kBarKEmpty + st2));
                            if (n + 3 == s.n_blocks) tc_commit(bar(kBarQEmpty + 0));
                        }
                    }
                    __syncwarp();
                    ++pn[x];
                }
                N += s.n_blocks;
                continue;
            }
            tc_fence_after();
            if (leader) {
                issue_qk(0, 0, st0);
                tc_commit(bar(kBarSFull + 0));
                if (s.n_blocks == 1) tc_commit(bar(kBarQEmpty + 0));
            }
            __syncwarp();
            if (!(ok = wait_all(kBarQ + 1, qn[1] & 1))) break;
            tc_fence_after();
            if (leader) {
                issue_qk(1, 1, st0);
                tc_commit(bar(kBarSFull + 1));
                if (s.n_blocks == 1) tc_commit(bar(kBarQEmpty + 1));
                tc_commit(bar(kBarKEmpty + st0));
            }
            __syncwarp();
            ++qn[1];
            for (int n = 0; n < s.n_blocks; ++n) {
                const int st = stage_of(N + n), st1 = stage_of(N + n + 1);
                const uint32_t ph = phase_of(N + n), ph1 = phase_of(N + n + 1);
                const bool more = n + 1 < s.n_blocks;
                const bool last_qk = n + 2 == s.n_blocks;
                if (!(ok = clean_tail(s, n, st, ph))) break;
                if (!(ok = __all_sync(0xffffffffu, mbar_wait2(bar(kBarVFull + st), ph,
                                                              bar(kBarPFull + 0), pn[0] & 1, wc))))
                    break;
                tc_fence_after();
                if (leader) issue_pv(0, st, 0, n > 0);
                __syncwarp();
                ok = more ? mbar_wait2(bar(kBarPFull + 1), pn[0] & 1, bar(kBarKFull + st1), ph1, wc)
                          : mbar_wait(bar(kBarPFull + 1), pn[0] & 1, wc);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                if (leader) {
                    issue_pv(0, st, 1, true);
                    if (!more) tc_commit(bar(kBarOFull + 0));
                    if (more) {
                        issue_qk(0, 0, st1);
                        tc_commit(bar(kBarSFull + 0));
                        if (last_qk) tc_commit(bar(kBarQEmpty + 0));
                    }
                }
                __syncwarp();
                ++pn[0];
                if (!(ok = wait_all(kBarPFull + 2, pn[1] & 1))) break;
                tc_fence_after();
                if (leader) issue_pv(1, st, 0, n > 0);
                __syncwarp();
                if (!(ok = wait_all(kBarPFull + 3, pn[1] & 1))) break;
                tc_fence_after();
                if (leader) {
                    issue_pv(1, st, 1, true);
                    tc_commit(bar(kBarVEmpty + st));
                    if (!more) tc_commit(bar(kBarOFull + 1));
                    if (more) {
                        issue_qk(1, 1, st1);
                        tc_commit(bar(kBarSFull + 1));
                        if (last_qk) tc_commit(bar(kBarQEmpty + 1));
                        tc_commit(bar(kBarKEmpty + st1));
                    }
                }
                __syncwarp();
                ++pn[1];
            }
            N += s.n_blocks;
        }
        // every MMA this CTA issued has finished before TMEM is released
        if (leader) tc_commit(bar(kBarDone));
        __syncwarp();
        mbar_wait_drain(bar(kBarDone), 0, wc);
        __syncwarp();
    } else if (warp >= 4) {
        // -------------------------------------------------------------- softmax
        const int tq = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;                   // within the sub-tile
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + Lay::col_s(tq);
        const uint32_t tO = tmem + lane_off + Lay::col_o(tq);
        const float sl2 = p.scale_log2;
        uint32_t sn = 0;                                       // S tiles seen by this sub-tile
        uint32_t on = 0;                                       // finished outputs of it
        uint32_t splits = 0;                                   // split segments of the CTA
        uint32_t adds = 0;                                     // segments whose halves were added
        uint32_t odd_n = 0;                                    // outputs of O1 so far
        float2* odd_stat = reinterpret_cast<float2*>(area + kOddStat);
        bool ok = true;
        Seg s;
        for (int i = 0; ok; ++i) {
            if (!get_seg(i, s)) break;
            // single sub-tile: both warpgroups hold its rows and take alternate key blocks
            const bool single = s.n_sub == 1;
            const int in_tile = (single ? 0 : tq * sub_rows) + row;   // packed row within the tile
            const int stride = single ? 2 * kKeys : kKeys;
            const int first_key = s.k0 + (single ? tq * kKeys : 0);
            const bool valid = row < sub_rows && in_tile < s.rows;
            const int tok = p.token_of(s.row0 + in_tile);            // within the sequence
            // keys that this row sees: [0, seen)
            // (of a tree: those from before the step.  Rows that the tile does not have may see
            // anything there: they are not written, and masking them in every block is what took
            // 40 tokens of 32 heads over 8 from 109 us to 120)
            const int seen = kTree ? (valid ? s.kv - s.n : 0x7fffffff)
                             : !valid ? 0 : a.causal ? s.kv - s.n + tok + 1 : s.kv;
            const int n_blocks = single ? (s.n_blocks + 1 - tq) / 2 : s.n_blocks;

            float m = -INFINITY, l = 0.f;
            float top = -INFINITY;                             // the score that m is the scaled one of
            for (int n = 0; n < n_blocks; ++n) {
                ok = mbar_wait(bar(kBarSFull + tq), sn & 1, wc);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++sn;
                tc_fence_after();

                uint32_t sraw[128];
                tmem_ld128(tS, sraw);
                float sv[128];
#pragma unroll
                for (int c = 0; c < 128; ++c) sv[c] = u2f(sraw[c]);
                const int kb = first_key + n * stride;
                const int lim = seen - kb;                     // columns [0, lim) are seen
                if (kTree && lim < kKeys) {
                    // of the new tokens, from column lim on, what the row's mask names
                    unsigned bits[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int left = s.kv - (kb + 32 * w);       // keys that there are
                        bits[w] = 0;
                        if (left > 0)
                            bits[w] = seen_from(p, s.first + tok, 32 * w - lim) &
                                      (left < 32 ? (1u << left) - 1 : 0xffffffffu);
                    }
#pragma unroll
                    for (int c = 0; c < 128; ++c) sv[c] = bits[c >> 5] >> (c & 31) & 1 ? sv[c] : -INFINITY;
                } else if (lim < kKeys) {
#pragma unroll
                    for (int c = 0; c < 128; ++c) sv[c] = c >= lim ? -INFINITY : sv[c];
                }
                float mx0 = fmaxf(sv[0], sv[1]), mx1 = fmaxf(sv[2], sv[3]);
                float mx2 = fmaxf(sv[4], sv[5]), mx3 = fmaxf(sv[6], sv[7]);
#pragma unroll
                for (int c = 8; c < 128; c += 8) {
                    mx0 = fmax3(mx0, sv[c], sv[c + 1]);
                    mx1 = fmax3(mx1, sv[c + 2], sv[c + 3]);
                    mx2 = fmax3(mx2, sv[c + 4], sv[c + 5]);
                    mx3 = fmax3(mx3, sv[c + 6], sv[c + 7]);
                }
                const float top_blk = fmax3(mx0, mx1, fmaxf(mx2, mx3));
                const float m_new = fmaxf(m, top_blk * sl2);
                const bool raise = m_new > m + kRescaleThreshold;
                const float m_ref = raise ? m_new : m;
                top = raise ? top_blk : top;
                const float alpha = raise ? ex2(m - m_ref) : 1.f;
                const bool far = !(fabsf(m_ref) < kFar);       // (minus infinity, too)
                const float far_neg = top == -INFINITY ? 0.f : -top * kFarScale;
                const float scale = far ? kFarScale : sl2, neg_m = far ? far_neg : -m_ref;
                // weights 2^(s - m_ref), rounded to bf16 (the product's operand type) over S
                // in two halves; the denominator is summed in fp32 before the rounding
                const uint64_t scale2 = f2pack(scale, scale), negm2 = f2pack(neg_m, neg_m);
                uint64_t sum_a = 0, sum_b = 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i2 = 0; i2 < 32; ++i2) {
                        const int c = 64 * half + 2 * i2;
                        float x0, x1;
                        f2unpack(ffma2(f2pack(sv[c], sv[c + 1]), scale2, negm2), x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        if (i2 & 1) sum_b = fadd2(sum_b, f2pack(p0, p1));
                        else sum_a = fadd2(sum_a, f2pack(p0, p1));
                        pk[i2] = pack_bf16x2(p0, p1);
                    }
                    tmem_st32(tS + 32 * half, pk);
                    // O was last written by P V of the previous block, finished before this
                    // block's S; it is rescaled before this block's P V accumulates into it
                    if (half == 0 && n > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * c, o);
#pragma unroll
                            for (int i2 = 0; i2 < 32; ++i2) o[i2] = f2u(u2f(o[i2]) * alpha);
                            tmem_st32(tO + 32 * c, o);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(bar(kBarPFull + 2 * tq + half));
                }
                float sa0, sa1;
                f2unpack(fadd2(sum_a, sum_b), sa0, sa1);
                l = l * alpha + (sa0 + sa1);
                m = m_ref;
            }
            if (!ok) break;
            const bool empty = n_blocks == 0;
            if (!empty) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarOFull + tq), on & 1, wc));
                if (!ok) break;
                ++on;
                tc_fence_after();
            }

            if (single && s.n_blocks > 1) {
                // the odd blocks' result is added to the even blocks'
                if (tq == 1) {
                    odd_stat[row] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarOdd));
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarAdded), adds & 1, wc));
                    if (!ok) break;
                } else {
                    // (once the other warpgroup is here, all its earlier outputs are done, so
                    // the parity of its last one is not mistaken for an older one's)
                    ok = mbar_wait(bar(kBarOdd), adds & 1, wc) &&
                         mbar_wait(bar(kBarOFull + 1), odd_n & 1, wc);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const float2 odd = odd_stat[row];
                    const float M = fmaxf(m, odd.x);
                    const float f0 = part_weight(m, l, M), f1 = part_weight(odd.x, odd.y, M);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o0[32], o1[32];
                        tmem_ld32(tO + 32 * c, o0);
                        tmem_ld32(tO + D + 32 * c, o1);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o0[j] = f2u(fmaf(f0, u2f(o0[j]), f1 * u2f(o1[j])));
                        tmem_st32(tO + 32 * c, o0);
                    }
                    l = (l == 0.f ? 0.f : f0 * l) + (odd.y == 0.f ? 0.f : f1 * odd.y);
                    m = M;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarAdded));
                }
                ++adds;
            }
            if (single ? s.n_blocks > 1 : s.n_blocks > 0) ++odd_n;

            const bool mine = !single || tq == 0;              // holds the rows' result
            const TileRows tile{s.first, s.row0, s.rows, s.hk, s.c_first, s.c_last};
            uint8_t* stage = smem + Lay::kStage + (warp - 4) * 32 * 128;
            if (s.c_first != s.c_last) {
                // this CTA's partial, row by row as the joining warps read it; the sums go
                // through the warp's staging slice, 32 columns at a time, so that a store
                // covers whole 128-byte runs of four rows
                const long long all_rows = 2ll * p.grid * 2 * kSub;
                const long long at0 = part_slot(tile, blockIdx.x) * 2 * kSub + tq * kSub;
                if (valid && mine && in_bounds(at0 + row, 1, all_rows, a.status))
                    __stcg(reinterpret_cast<float2*>(p.part_stat) + at0 + row, make_float2(m, l));
                if (mine && __any_sync(0xffffffffu, valid)) {
                    const unsigned rows_in = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32] = {};                   // zeros if it saw no key
                        if (!empty) tmem_ld32(tO + 32 * c, o);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int rr = 4 * k + (lane >> 3), cc = lane & 7;
                            const float4 val = *reinterpret_cast<const float4*>(
                                stage + rr * 128 + ((cc ^ (rr & 7)) << 4));
                            const long long at = (at0 + quarter * 32 + rr) * D + 32 * c + 4 * cc;
                            if (((rows_in >> rr) & 1) && in_bounds(at, 4, all_rows * D, a.status))
                                __stcg(reinterpret_cast<float4*>(p.part_o + at), val);
                        }
                        __syncwarp();
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarPart));
                if (warp == 4) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarPart), splits & 1, wc));
                    if (!ok) break;
                    if (lane == 0) {
                        *last_flag = arrive_last(p, tile);
                        mbar_arrive(bar(kBarFlag));
                    }
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarFlag), splits & 1, wc));
                if (!ok) break;
                ++splits;
                if (*last_flag)
                    join_rows<__nv_bfloat16, D / 4, 1, 8, 2>(
                        p, tile, warp - 4, 8, 2 * kSub,
                        [&](int r) { return r < sub_rows ? r : kSub + r - sub_rows; });
            } else if (mine) {
                // Rows leave through the staging slice too, half of the columns at a time: a
                // thread writes its row's 16-byte chunk c at slot c ^ (row mod kChunks).
                constexpr int kHalf = D / 2;
                constexpr int kChunks = kHalf / 8;             // 16-byte chunks per staged row
                constexpr int kRowsPerStore = 32 / kChunks;
                const float inv = inverse_of(l);
                const long long my_row = valid ? out_row(p, tile, in_tile) : -1;
#pragma unroll 1
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int c = 0; c < kHalf / 32; ++c) {
                        uint32_t o[32] = {};
                        if (!empty) tmem_ld32(tO + hh * kHalf + 32 * c, o);
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            pk[j] = pack_bf16x2(u2f(o[2 * j]) * inv, u2f(o[2 * j + 1]) * inv);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int sl = (4 * c + j) ^ (lane & (kChunks - 1));
                            *reinterpret_cast<uint4*>(stage + lane * (2 * kHalf) + sl * 16) =
                                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
                        }
                    }
                    __syncwarp();
                    const int part = lane / kChunks, cc = lane % kChunks;
#pragma unroll
                    for (int k = 0; k < 32 / kRowsPerStore; ++k) {
                        const int rr = k * kRowsPerStore + part;
                        const long long orow = __shfl_sync(0xffffffffu, my_row, rr);
                        const uint4 val = *reinterpret_cast<const uint4*>(
                            stage + rr * (2 * kHalf) + ((cc ^ (rr & (kChunks - 1))) * 16));
                        const long long at = orow * D + hh * kHalf + cc * 8;
                        if (orow >= 0 && in_bounds(at, 8, a.out_elems, a.status))
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at) = val;
                    }
                    __syncwarp();
                }
                if (valid && a.lse != nullptr && in_bounds(my_row, 1, a.lse_elems, a.status))
                    a.lse[my_row] = lse_of(m, l);
            }
        }
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool kTree>
cudaError_t launch_d(PagedParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv)
{
    static std::atomic<int> known[kMaxDevices];
    int grid = 0;
    const cudaError_t e = resident_ctas(known, paged_tc_kernel<D, kTree>, kThreads, Layout<D>::kSmem, &grid);
    if (e != cudaSuccess) return e;
    p.grid = grid < kPagedTcCtas ? grid : kPagedTcCtas;
    // a block of a single sub-tile takes half the time of a double one at head dim 64 (1500
    // cycles to 2700) and nearly the same at 128 (2300 to 2600: K and V loads bound it)
    p.key_shift = 1;
    p.key_shift_single = D == 64 ? 0 : 1;
    p.tile_cost = 256 << p.key_shift;
    p.snap = 3 * kKeys;
    p.min_chunk = 3 * kKeys << p.key_shift;
    // 10 cycles a unit: 6000 cycles a partial of two sub-tiles, 2000 of a single one.  Measured
    // with the rule that this feeds and without: 297 tokens over 11606 keys of 2 heads 52 us
    // against 59 (69 with parts of 2 blocks at least instead of 3), 8 tokens over 4000 keys of 8
    // heads 20 against 22.
    const bool two = static_cast<long long>(p.a.T) * p.G > static_cast<long long>(kSub) * p.a.n_seqs;
    p.join_cost = two ? 600 : 200;
    // Tiles of two sub-tiles of up to eight blocks are faster whole: half the time of one that
    // is longer pays for the partials and their joining (26 prompts of 30 to 60 tokens over 300
    // to 600 keys, 4 key heads, 17 us and 31 cut; 5 prompts of 757, 19 and 28; at a third more
    // a mixed batch loses 3 %).
    p.whole = two ? 2800 : 0;
    if (kTree) {
        // Trees bring tiles of one and of two sub-tiles in one call.  With their outputs, partials
        // and joins a block of one takes 1.37 us and of two 1.78 at head dim 128, but the CTAs of
        // the former also start on their blocks together and wait for HBM longer.  Measured, 32
        // trees of up to 64 tokens over up to 8192 keys, price of one against two: 1 (the other
        // calls') 108 us, the CTAs ending between 74 and 112; 0.81 102; 0.75 101; 0.69 97; 0.63 98.
        // Other batches at 128 dims, price 1, 0.69 and 0.5: 16 trees of up to 16384 keys 106, 91 and
        // 91 us; 64 of up to 40 tokens and 4096 keys, 16 heads over 4, 70, 62 and 66; 48 of up to 30
        // over 3000, 65 each.  At 64 dims a half is right: the first batch 86, 71 and 71 us, the
        // second 79, 65 and 64, the third 58, 51 and 46, the last 49 each.
        constexpr int kTwo = 16, kOne = D == 64 ? 8 : 11;
        p.key_cost = kTwo;
        p.key_cost_single = kOne;
        p.tile_cost *= kTwo / 2;        // (units of half a key so far)
        p.min_chunk *= kTwo / 2;
        p.join_cost *= kTwo / 2;
        p.whole *= kTwo / 2;
    }
    const PagedWorkspace w = paged_workspace_of(p.grid, 2 * kSub, D);
    uint8_t* ws = static_cast<uint8_t*>(p.a.workspace);
    p.counters = reinterpret_cast<unsigned int*>(ws);
    p.part_stat = reinterpret_cast<float*>(ws + w.stat);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    return launch_early(paged_tc_kernel<D, kTree>, p.grid, kThreads, Layout<D>::kSmem, p.a.stream, tq, tk, tv, p);
}

}  // namespace

bool paged_tc_applies(const PagedArgs& a)
{
    // A page must hold whole 8-row swizzle atoms (2048 tokens that end at key 32768, 32 heads
    // over 8: pages of 8 slots 717 us, pages of 4, which go 16 rows at a time, 7070), a sub-tile
    // at least one token, and the strides must fit a tensor map (2^40 bytes).
    const long long most = 1ll << 39;
    if (a.q_stride >= most || a.page_stride >= most || a.token_stride >= most || a.head_stride >= most)
        return false;
    if (a.elem != 2 || a.page_size % 8 != 0 || a.H / a.H_kv > kSub) return false;
    // More than one 16-row tile per sequence and key head on average (the lengths are not known
    // here, so a chunk beside very many single tokens goes 16 rows at a time: 99 tokens over
    // 2000 keys and a chunk of 1000 over 30000, 8 heads, G 1, take 840 us, apart 149 and 122).
    // Measured, few-rows kernel against this one, head dim 128, 8 key heads: 32
    // sequences of up to 8000 keys, 16 rows 108 us against 100, 20 rows 182 against 102, 64
    // rows 360 against 101; 64 sequences of up to 500 keys, 16 rows 25 against 39, 20 rows 39
    // against 39, 64 rows 74 against 39; one of 32768, 16 rows 42 against 40, 64 rows 62
    // against 41; head dim 64, 32 sequences: 16 rows 64 against 72, 20 rows 96 against 72.
    return static_cast<long long>(a.T) * (a.H / a.H_kv) > 16ll * a.n_seqs;
}

cudaError_t launch_paged_tc(const PagedArgs& a)
{
    PagedParams p;
    fill_params(&p, a);
    const int sub_tokens = kSub / p.G;
    p.tile_tokens = 2 * sub_tokens;
    // a block is loaded in boxes of as many keys as divide both it and a page: a box never
    // crosses a page (24 slots: boxes of 8)
    p.box_rows = a.page_size & -a.page_size;
    if (p.box_rows > kKeys) p.box_rows = kKeys;
    using ull = unsigned long long;
    const ull D = static_cast<ull>(a.D);
    CUtensorMap tq, tk, tv;
    const ull qd[3] = {D, static_cast<ull>(a.H), static_cast<ull>(a.T)};
    const ull qs[2] = {2 * D, 2ull * a.q_stride};
    const unsigned qb[3] = {64, static_cast<unsigned>(p.G), static_cast<unsigned>(sub_tokens)};
    const ull kd[4] = {D, static_cast<ull>(a.H_kv), static_cast<ull>(a.page_size),
                       static_cast<ull>(a.num_pages)};
    // (a dimension of one entry never uses its stride, which need not be a valid one)
    const ull ks[3] = {a.H_kv > 1 ? 2ull * a.head_stride : 2 * D,
                       a.page_size > 1 ? 2ull * a.token_stride : 2 * D,
                       a.num_pages > 1 ? 2ull * a.page_stride : 2 * D};
    const unsigned kb[4] = {64, 1, static_cast<unsigned>(p.box_rows), 1};
    if (!encode_bf16_map(&tq, a.q, 3, qd, qs, qb) || !encode_bf16_map(&tk, a.k_pages, 4, kd, ks, kb) ||
        !encode_bf16_map(&tv, a.v_pages, 4, kd, ks, kb))
        return cudaErrorInvalidValue;
    if (a.D == 64) return a.masks ? launch_d<64, true>(p, tq, tk, tv) : launch_d<64, false>(p, tq, tk, tv);
    if (a.D == 128) return a.masks ? launch_d<128, true>(p, tq, tk, tv) : launch_d<128, false>(p, tq, tk, tv);
    return cudaErrorInvalidValue;
}

}  // namespace ra
