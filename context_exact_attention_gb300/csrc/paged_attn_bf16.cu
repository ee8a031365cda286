// paged_attn_bf16.cu -- paged_attn_fwd for calls with few query rows per key/value head
// (single tokens, a few proposed ones), bf16: a stream over the cache.
//
// With R query rows per key/value head a key costs 4 D bytes and 4 D R operations, so up to
// R of about 288 (the measured matrix rate over the measured bandwidth) the call is bound by
// reading the cache.  This kernel serves the low end, where a 128-row tensor-memory tile
// would be nearly empty: a tile is 16 packed rows (tokens x heads of the group), the rows
// of an m16n8k16 warp product, held by a block of four warps.
//
// Each warp takes 16 of every 64 keys and runs by itself: it copies its 16 keys and values
// into its own shared-memory ring with 16-byte asynchronous copies (zero-filled for keys
// that the tile does not see, so that what lies in their slots never matters), multiplies
// S = Q K^T from the ring, keeps its own running maximum and denominator and adds P V to its
// own 16 x D sum.  No barrier is met inside a segment; the four results are joined at its end
// through shared memory.  The copies run ahead of the products, into the next segment too, so
// a sequence's end does not empty the pipeline, and the page-table entry of a step is fetched
// one step before its copies are issued.  Two blocks of 96 KB of ring each fit an SM: 128 KB
// in flight, where a latency of 1.5 us at 44 GB/s per SM asks for 66.
//
// The maximum used in the exponentials is raised only when it grows by more than 2^8 (as
// in the dense kernels: any common reference leaves the quotient unchanged), so the sums
// are rarely rescaled.
//
// Measured: 64 sequences of 1000 to 16384 keys, 32 heads over 8, head dim 128 (2.26 GB) in
// 344 to 357 us, 6.3 to 6.6 TB/s (95 to 98 % of the measured copy rate; the tensor pipe is 28 %
// busy); one token over 131072 keys of 8 heads (0.54 GB) in 89 to 90 us, of which the plan, the
// first reads and the joining of 19 partials per head take about 6; one token over 1000 keys in
// 9 us, a chain of code that runs once (plan 2, first reads 1.5, sums and partial 2, joining
// 1.5, launch 2).  It was 16 us while the walk and the copies were compiled into several places:
// a call this short is bound by fetching instructions.
#include <algorithm>

#include "paged_mma.cuh"
#include "paged_plan.cuh"

namespace ra {
namespace {

constexpr int kRows = 16;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kKeysW = 16;                     // keys per warp and step
constexpr int kUnit = kKeysW * kWarps;         // keys per block and step
constexpr float kRescaleThreshold = 8.0f;

template <int D>
struct Smem {
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kTile = kKeysW * D * 2;              // a warp's keys (or values)
    static constexpr int kStage = 2 * kTile * kWarps;
    static constexpr int kLdo = D + 8;                        // padded: rows in different banks
    static constexpr int kBuf = kStages * kStage;
    static constexpr int kStatW = kBuf + kRows * kLdo * 4;
    static constexpr int kStat = kStatW + kWarps * kRows * 8;
    static constexpr int kFlag = kStat + kRows * 8;
    static constexpr int kBytes = kFlag + 16;
};

// kTree: rows see the new tokens that their masks name.
template <int D, bool kTree>
__global__ void __launch_bounds__(kThreads, 2) paged_bf16_kernel(const __grid_constant__ PagedParams p)
{
    using S = Smem<D>;
    using Walk = PagedWalk<FlatTiles<kRows>, kUnit>;
    constexpr int kStages = S::kStages;
    constexpr int kChunks = D / 8;                            // 16-byte chunks per key
    constexpr int kRowsPerCopy = 32 / kChunks;                // keys one warp-wide copy covers
    constexpr int kSteps = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    float* buf = reinterpret_cast<float*>(smem + S::kBuf);
    float2* stat_w = reinterpret_cast<float2*>(smem + S::kStatW);
    float2* stat = reinterpret_cast<float2*>(smem + S::kStat);
    int* flag = reinterpret_cast<int*>(smem + S::kFlag);
    const PagedArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(a.k_pages);
    const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(a.v_pages);
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.q);
    const uint32_t ring = smem_addr(smem) + warp * 2 * S::kTile;

    wait_for_earlier_work();
    Walk walk;
    walk.begin(p);
    Segment t{}, nt{};                          // the segment being multiplied, the next one
    bool have = false, have_next = walk.next(p, nt);
    // The copies: step `lk` of segment nt (in_next) or t, up to kStages steps ahead of the
    // products.  They cross into the next segment but not beyond it.
    bool in_next = true;
    int lk = have_next ? nt.k0 : 0;
    uint32_t issued = 0, used = 0;              // steps
    long long off = -1;                         // lane < 16: where the step's key lies
    auto look_up = [&]() {
        const int key = lk + kKeysW * warp + lane;
        const int k1 = in_next ? (have_next ? nt.k1 : 0) : t.k1;
        off = -1;
        if (lane < kKeysW && key < k1)
            off = key_offset(p, in_next ? nt.g : t.g, in_next ? nt.hk : t.hk, key);
    };
    auto loadable = [&]() { return lk < (in_next ? (have_next ? nt.k1 : 0) : t.k1); };
    auto issue = [&]() {
        const uint32_t dst = ring + (issued % kStages) * S::kStage;
#pragma unroll
        for (int j = 0; j < kKeysW / kRowsPerCopy; ++j) {
            const int row = j * kRowsPerCopy + lane / kChunks, c = lane % kChunks;
            const long long o = __shfl_sync(0xffffffffu, off, row);
            const bool real = o >= 0 && in_bounds(o + 8 * c, 8, a.page_elems, a.status);
            const long long at = real ? o + 8 * c : 0;
            const uint32_t to = dst + row * (2 * D) + ((c ^ (row & 7)) << 4);
            cp_async16(to, K + at, real);
            cp_async16(to + S::kTile, V + at, real);
        }
        cp_async_commit();
        ++issued;
        lk += kUnit;
        if (!in_next && lk >= t.k1) {
            in_next = true;
            lk = have_next ? nt.k0 : 0;
        }
        look_up();
    };
    // The query fragments of a segment: thread's rows lane / 4 and lane / 4 + 8, columns
    // 16 step + 2 (lane mod 4) and 8 further.
    auto load_q = [&](const Segment& t, uint32_t (&q)[kSteps][4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = (lane >> 2) + 8 * h;
            long long at = -1;
            if (r < t.rows) {
                const int pr = t.row0 + r, tok = p.token_of(pr);
                at = (t.s.first + tok) * a.q_stride +
                     static_cast<long long>(t.hk * p.G + (pr - tok * p.G)) * D + 2 * (lane & 3);
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x = 0;
                    const long long i = at + 16 * k + 8 * c;
                    if (at >= 0 && in_bounds(i, 2, a.q_elems, a.status))
                        x = __ldg(reinterpret_cast<const unsigned int*>(Q + i));
                    q[k][2 * c + h] = x;
                }
        }
    };

    look_up();
    // Each turn moves on to the next segment, fetches its queries, finishes the segment
    // before while they come, and walks its keys.
#pragma unroll 1
    for (;;) {
        uint32_t q[kSteps][4];
        if (have_next) load_q(nt, q);
        if (have) finish_segment<__nv_bfloat16, kRows, kThreads>(p, t, buf, S::kLdo, stat, flag);
        have = have_next;
        if (!have) break;
        t = nt;
        have_next = walk.next(p, nt);
        in_next = lk >= t.k1;
        if (in_next) lk = have_next ? nt.k0 : 0;
        look_up();
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        // keys that this thread's two rows see, and that every row of the tile sees
        // (of a tree: the keys from before the step)
        auto seen_by = [&](int r) {
            if (kTree) return t.s.kv - t.s.n;
            const int tok = p.token_of(t.row0 + r);
            return a.causal ? t.s.kv - t.s.n + tok + 1 : t.s.kv;
        };
        const int see0 = seen_by(lane >> 2), see1 = seen_by((lane >> 2) + 8);
        const int see_all = min(seen_by(0), t.k1);
        for (int k = t.k0; k < t.k1; k += kUnit) {
            // (every lane has read the step before, whose place in the ring is taken next)
            __syncwarp();
#pragma unroll 1
            while (issued - used < kStages && loadable()) issue();
            if (issued - used == kStages) cp_async_wait<kStages - 1>();
            else cp_async_wait<0>();
            __syncwarp();
            const uint32_t kt = ring + (used % kStages) * S::kStage, vt = kt + S::kTile;
            ++used;

            float s[2][4] = {};
            {
                const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
                const uint32_t row = kt + key * (2 * D);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t b[4];
                    ldmatrix4(row + (((2 * i + half) ^ (key & 7)) << 4), b);
                    mma16816(s[0], q[i], b[0], b[1]);
                    mma16816(s[1], q[i], b[2], b[3]);
                }
            }
            const int k0w = k + kKeysW * warp;
            if (kTree && k0w + kKeysW > see_all) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (lane >> 2) + 8 * h;
                    unsigned seen = 0;
                    if (r < t.rows)
                        seen = seen_from(p, t.s.first + p.token_of(t.row0 + r), k0w - (t.s.kv - t.s.n));
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int in = 8 * i + 2 * (lane & 3) + j;
                            if (!(seen >> in & 1) || k0w + in >= t.k1) s[i][2 * h + j] = -INFINITY;
                        }
                }
            } else if (k0w + kKeysW > see_all) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = k0w + 8 * i + 2 * (lane & 3) + j;
                        if (key >= see0 || key >= t.k1) s[i][j] = -INFINITY;
                        if (key >= see1 || key >= t.k1) s[i][2 + j] = -INFINITY;
                    }
            }
            float mx0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
            float mx1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2)) * p.scale_log2;
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2)) * p.scale_log2;
            const bool up0 = mx0 > m0 + kRescaleThreshold, up1 = mx1 > m1 + kRescaleThreshold;
            if (__any_sync(0xffffffffu, up0 || up1)) {
                const float a0 = up0 ? ex2(m0 - mx0) : 1.f, a1 = up1 ? ex2(m1 - mx1) : 1.f;
                m0 = up0 ? mx0 : m0;
                m1 = up1 ? mx1 : m1;
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= a0;
                    o[i][1] *= a0;
                    o[i][2] *= a1;
                    o[i][3] *= a1;
                }
            }
            const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
            // (the product rounded, as the maximum's was, so that the maximum's own exponent is 0: a
            // fused multiply-add leaves it the rounding, which for huge scores overflows)
            auto weight = [&](float x, float n) { return ex2(__fadd_rn(__fmul_rn(x, p.scale_log2), n)); };
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s[i][0] = weight(s[i][0], n0);
                s[i][1] = weight(s[i][1], n0);
                s[i][2] = weight(s[i][2], n1);
                s[i][3] = weight(s[i][3], n1);
                l0 += s[i][0] + s[i][1];
                l1 += s[i][2] + s[i][3];
            }
            // The matrix product takes its weights in bf16.  Each goes in as two of them, which
            // keeps it to 2^-16: the products are not what bounds this kernel (17 % of the tensor
            // pipe with one part, 28 % with two), and without the second the weights' rounding
            // would cost as much precision as the output's own.  Both parts of a weight above 0 are above 0 (the
            // first is the weight less its last bit, cut off, the second the rest, rounded to
            // nearest), so that an infinite value gives that infinity: with a part of 0 or of
            // the other sign the two products would add up to NaN.
            uint32_t pf[4], pr[4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x0 = s[i][2 * h], x1 = s[i][2 * h + 1];
                    const uint32_t b0 = below(x0), b1 = below(x1);
                    pf[2 * i + h] = __byte_perm(b0, b1, 0x7632);
                    pr[2 * i + h] = pack_bf16x2(x0 - __uint_as_float(b0 & 0xffff0000u),
                                                x1 - __uint_as_float(b1 & 0xffff0000u));
                }
            {
                const int key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
                const uint32_t row = vt + key * (2 * D);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t b[4];
                    ldmatrix4_trans(row + (((2 * i + half) ^ (key & 7)) << 4), b);
                    mma16816(o[2 * i], pf, b[0], b[1]);
                    mma16816(o[2 * i + 1], pf, b[2], b[3]);
                    mma16816(o[2 * i], pr, b[0], b[1]);
                    mma16816(o[2 * i + 1], pr, b[2], b[3]);
                }
            }
        }
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        const int r0 = lane >> 2, r1 = r0 + 8;
        if ((lane & 3) == 0) {
            stat_w[warp * kRows + r0] = make_float2(m0, l0);
            stat_w[warp * kRows + r1] = make_float2(m1, l1);
        }
        __syncthreads();
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h ? r1 : r0;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat_w[w * kRows + r].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 x = stat_w[w * kRows + r];
                if (!(x.y == 0.f)) L += part_weight(x.x, x.y, M) * x.y;
            }
            f[h] = part_weight(h ? m1 : m0, h ? l1 : l0, M);
            if (warp == 0 && (lane & 3) == 0) stat[r] = make_float2(M, L);
        }
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((h ? r1 : r0) >= t.rows) continue;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        float2* dst = reinterpret_cast<float2*>(
                            buf + (h ? r1 : r0) * S::kLdo + 8 * i + 2 * (lane & 3));
                        float2 x = w == 0 ? make_float2(0.f, 0.f) : *dst;
                        x.x = fmaf(f[h], o[i][2 * h], x.x);
                        x.y = fmaf(f[h], o[i][2 * h + 1], x.y);
                        *dst = x;
                    }
                }
            }
            __syncthreads();
        }
    }
    cp_async_wait<0>();
}

template <int D, bool kTree>
cudaError_t launch_d(PagedParams& p)
{
    const PagedArgs& a = p.a;
    static std::atomic<int> known[kMaxDevices];
    int grid = 0;
    const cudaError_t e =
        resident_ctas(known, paged_bf16_kernel<D, kTree>, kThreads, Smem<D>::kBytes, &grid);
    if (e != cudaSuccess) return e;
    // With so few tiles that each would fall into 24 parts or more, one block an SM: it copies
    // nearly as fast as two and halves the joining (one token over 131072 keys of 8 heads 89 us
    // against 93, 36000 of 4 heads of 64 dims 19.5 against 21.4; 32 tiles in 10 parts each, 38
    // us, would take 40).
    const long long tiles =
        static_cast<long long>(a.H_kv) *
        std::max<long long>(a.n_seqs, (static_cast<long long>(a.T) * p.G + kRows - 1) / kRows);
    if (tiles * 24 <= grid) grid /= 2;
    p.grid = grid < kPagedMaxCtas ? grid : kPagedMaxCtas;
    p.tile_cost = 64;
    p.key_shift = 0;
    p.snap = 2 * kUnit;
    // 12 keys' time (0.1 us).  Measured with 6, 12, 24 and 40: one token over 120000 keys of one
    // head 39, 35, 36, 40 us, 8000 keys of 8 heads 18.8, 18.2, 17.6, 19.0, 2000 of 8 heads 10.1,
    // 10.1, 13.7, 14.0.
    p.join_cost = 12;
    p.whole = 0;                    // (480: 100 to 450 keys 0.7 to 0.9 times as fast)
    p.min_chunk = 2 * kUnit;
    const PagedWorkspace w = paged_workspace_of(p.grid, kRows, D);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.counters = reinterpret_cast<unsigned int*>(ws);
    p.part_stat = reinterpret_cast<float*>(ws + w.stat);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    return launch_early(paged_bf16_kernel<D, kTree>, p.grid, kThreads, Smem<D>::kBytes, a.stream, p);
}

}  // namespace

cudaError_t launch_paged_bf16(const PagedArgs& a)
{
    PagedParams p;
    fill_params(&p, a);
    if (a.D == 64) return a.masks ? launch_d<64, true>(p) : launch_d<64, false>(p);
    if (a.D == 128) return a.masks ? launch_d<128, true>(p) : launch_d<128, false>(p);
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged(const PagedArgs& a)
{
    cudaError_t e = cudaSuccess;
    if (a.masks != nullptr && (a.elem == 2 ? paged_tree_bf16(a, &e) : paged_tree_f32(a, &e))) return e;
    if (a.elem != 2) return paged_rows_applies(a) ? launch_paged_rows(a) : launch_paged_simt(a);
    return paged_tc_applies(a) ? launch_paged_tc(a) : launch_paged_bf16(a);
}

unsigned long long paged_workspace_bytes(int D, int elem)
{
    if (elem != 2)
        return std::max(paged_workspace_of(kPagedMaxCtas, 4, D).total,
                        paged_workspace_of(kPagedRowsCtas, 64, D).total);
    const unsigned long long few = paged_workspace_of(kPagedMaxCtas, kRows, D).total;
    const unsigned long long many = paged_workspace_of(kPagedTcCtas, 256, D).total;
    return few > many ? few : many;
}

}  // namespace ra
