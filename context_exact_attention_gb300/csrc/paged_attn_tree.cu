// paged_attn_tree.cu -- paged_attn_tree_fwd for calls with few tiles (a tree or two of drafted
// tokens), bf16: a cluster of CTAs for every tile.
//
// Such a call is a chain of latencies: lengths, table, keys, a few products, the joining of the
// parts.  A tile -- 16, 32 or 64 packed rows (tokens x heads of the group) of one key/value head
// -- is one cluster's, whose CTAs take equal parts of its keys; no plan over the whole call is
// needed, and the parts are joined through the cluster's shared memory, each CTA taking an equal
// share of the rows, where the kernels that split tiles at any place write partials to memory
// for one CTA to join.
//
// A CTA is four warps.  Keys and values come 64 at a time through a ring that all warps fill
// with 16-byte asynchronous copies (zeros for keys that there are not).  Warps share the rows
// first, 16 each (an m16n8k16 product's), and where the tile has fewer rows the keys of a step:
// then each keeps its own running softmax, joined at the end.  Weights enter the value product
// as in the kernels for more tiles: as two bf16 parts where a sequence and key head has up to 16
// rows on average, rounded to one beyond.
//
// What bounds it: the latencies, and from some steps a CTA on the products: mma.sync runs at an
// eighth of the tcgen05 rate here, so that a step of 64 rows takes 2000 cycles, where HBM brings
// its 32 KB in 1400; calls of many tiles or long contexts go to paged_attn_sm103.cu.  A tree of
// 26 tokens over 2000 keys, 32 heads over 8, takes 13 us (22 there), one of 4 tokens 8.5.
#include <algorithm>

#include "paged_cluster.cuh"
#include "paged_mma.cuh"

namespace ra {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 64;                      // keys of a step
constexpr int kKeysW = kKeys / kWarps;         // ... that a warp copies
constexpr float kRescaleThreshold = 8.0f;

template <int D>
struct Smem {
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kTile = kKeys * D * 2;               // a step's keys (or values)
    static constexpr int kLdo = D + 8;                        // padded: rows in different banks
    // the warps' sums, 16 rows each, over the ring when it is done with
    static constexpr int kRing = kStages * 2 * kTile;
    static_assert(kWarps * 16 * kLdo * 4 <= kRing, "sums over the ring");
    static constexpr int kStatW = kRing;                      // [warp][row] (maximum, denominator)
    static constexpr int kStat = kStatW + kWarps * 16 * 8;    // [row] of the tile, over the warps
    static constexpr int kBytes = kStat + kWarps * 16 * 8;
};

// kRowWarps: warps that share the tile's rows; the others share the keys of a step with them.
template <int D, int kRowWarps>
__global__ void __launch_bounds__(kThreads, 2) paged_tree_kernel(const __grid_constant__ PagedParams p)
{
    using S = Smem<D>;
    constexpr int kStages = S::kStages;
    constexpr int kRows = 16 * kRowWarps;
    constexpr int kKeyWarps = kWarps / kRowWarps;
    constexpr bool kTwoParts = kRowWarps == 1;
    constexpr int kMine = kKeys / kKeyWarps;                  // keys of a step that a warp multiplies
    constexpr int kChunks = D / 8;                            // 16-byte chunks per key
    constexpr int kRowsPerCopy = 32 / kChunks;                // keys one warp-wide copy covers
    constexpr int kSteps = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    float* buf = reinterpret_cast<float*>(smem);
    float2* stat_w = reinterpret_cast<float2*>(smem + S::kStatW);
    float2* stat = reinterpret_cast<float2*>(smem + S::kStat);
    const PagedArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row_warp = warp % kRowWarps, key_warp = warp / kRowWarps;
    const int ctas = p.grid, rank = static_cast<int>(cluster_ctarank());
    const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(a.k_pages);
    const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(a.v_pages);
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.q);
    const uint32_t ring = smem_addr(smem);

    wait_for_earlier_work();
    TileRows t{};
    SeqSpan span{};
    const int g = cluster_tile<kRows>(p, t, span);
    if (g < 0) {                                // (meeting the barriers of join_cluster all the same, so
        cluster_sync_all();                     // that CTAs wait for none that has left, whatever the
        cluster_sync_all();                     // lengths held while each of them read them)
        return;
    }
    const int steps = (span.kv + kKeys - 1) / kKeys;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * rank / ctas);
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (rank + 1) / ctas);

    // The copies run up to kStages - 1 steps ahead.  A warp's 16 keys: their places are looked up
    // a step before they are copied.
    long long off = -1;                         // lane < 16: where the key lies
    int issued = s0;
    auto look_up = [&]() {
        const int key = issued * kKeys + kKeysW * warp + lane;
        off = -1;
        if (lane < kKeysW && issued < s1 && key < span.kv) off = key_offset(p, g, t.hk, key);
    };
    auto issue = [&]() {
        if (issued < s1) {
            const uint32_t dst = ring + (issued - s0) % kStages * (2 * S::kTile);
#pragma unroll
            for (int j = 0; j < kKeysW / kRowsPerCopy; ++j) {
                const int in_warp = j * kRowsPerCopy + lane / kChunks, c = lane % kChunks;
                const long long o = __shfl_sync(0xffffffffu, off, in_warp);
                const bool real = o >= 0 && in_bounds(o + 8 * c, 8, a.page_elems, a.status);
                const long long at = real ? o + 8 * c : 0;
                const int row = kKeysW * warp + in_warp;
                const uint32_t to = dst + row * (2 * D) + ((c ^ (row & 7)) << 4);
                cp_async16(to, K + at, real);
                cp_async16(to + S::kTile, V + at, real);
            }
            ++issued;
            look_up();
        }
        cp_async_commit();                      // (an empty group where there is no step)
    };
    look_up();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    // The query fragments: thread's rows lane / 4 and lane / 4 + 8 of its warp's 16, columns
    // 16 step + 2 (lane mod 4) and 8 further.
    uint32_t q[kSteps][4];
    int token[2];                               // its rows' tokens in the call, or -1
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 16 * row_warp + (lane >> 2) + 8 * h;
        long long at = -1;
        token[h] = -1;
        if (r < t.rows) {
            const int pr = t.row0 + r, tok = p.token_of(pr);
            token[h] = t.first + tok;
            at = token[h] * a.q_stride + static_cast<long long>(t.hk * p.G + (pr - tok * p.G)) * D + 2 * (lane & 3);
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
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int before = span.kv - span.n;        // keys from before the step, which all rows see
#pragma unroll 1
    for (int n = s0; n < s1; ++n) {
        cp_async_wait<kStages - 2>();
        __syncthreads();                        // the step is here, and the one before has been read
        issue();
        const uint32_t kt = ring + (n - s0) % kStages * (2 * S::kTile) + key_warp * kMine * (2 * D);
        const uint32_t vt = kt + S::kTile;
        float s[kMine / 8][4] = {};
        {
            const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < kMine / 16; ++j) {
                const uint32_t row = kt + (16 * j + key) * (2 * D);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t b[4];
                    ldmatrix4(row + (((2 * i + half) ^ (key & 7)) << 4), b);
                    mma16816(s[2 * j], q[i], b[0], b[1]);
                    mma16816(s[2 * j + 1], q[i], b[2], b[3]);
                }
            }
        }
        const int k0 = n * kKeys + key_warp * kMine;          // this warp's first key
        if (k0 + kMine > min(before, span.kv)) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int w = 0; w < (kMine + 31) / 32; ++w) {
                    unsigned seen = 0;
                    const int left = span.kv - (k0 + 32 * w);        // keys that there are
                    if (token[h] >= 0 && left > 0)
                        seen = seen_from(p, token[h], k0 + 32 * w - before) &
                               (left < 32 ? (1u << left) - 1 : 0xffffffffu);
#pragma unroll
                    for (int i = 4 * w; i < 4 * w + 4 && i < kMine / 8; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int in = 8 * (i - 4 * w) + 2 * (lane & 3) + j;
                            if (!(seen >> in & 1)) s[i][2 * h + j] = -INFINITY;
                        }
                }
        }
        float alpha[2];
        bool raised = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < kMine / 8; ++i) mx = fmax3(mx, s[i][2 * h], s[i][2 * h + 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.scale_log2;
            const bool up = mx > m[h] + kRescaleThreshold;
            alpha[h] = up ? ex2(m[h] - mx) : 1.f;
            m[h] = up ? mx : m[h];
            l[h] *= alpha[h];
            raised |= up;
        }
        if (__any_sync(0xffffffffu, raised)) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= alpha[j >> 1];
        }
        // (the product rounded, as the maximum's was, so that the maximum's own exponent is 0)
#pragma unroll
        for (int i = 0; i < kMine / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float ref = m[j >> 1] == -INFINITY ? 0.f : -m[j >> 1];
                s[i][j] = ex2(__fadd_rn(__fmul_rn(s[i][j], p.scale_log2), ref));
                l[j >> 1] += s[i][j];
            }
        {
            const int key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
#pragma unroll
            for (int k = 0; k < kMine / 16; ++k) {
                uint32_t pf[4], pr[4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x0 = s[2 * k + i][2 * h], x1 = s[2 * k + i][2 * h + 1];
                        if (!kTwoParts) {
                            pf[2 * i + h] = pack_bf16x2(x0, x1);
                            continue;
                        }
                        const uint32_t b0 = below(x0), b1 = below(x1);
                        pf[2 * i + h] = __byte_perm(b0, b1, 0x7632);
                        pr[2 * i + h] = pack_bf16x2(x0 - __uint_as_float(b0 & 0xffff0000u),
                                                    x1 - __uint_as_float(b1 & 0xffff0000u));
                    }
                const uint32_t row = vt + (16 * k + key) * (2 * D);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t b[4];
                    ldmatrix4_trans(row + (((2 * i + half) ^ (key & 7)) << 4), b);
                    mma16816(o[2 * i], pf, b[0], b[1]);
                    mma16816(o[2 * i + 1], pf, b[2], b[3]);
                    if (kTwoParts) {
                        mma16816(o[2 * i], pr, b[0], b[1]);
                        mma16816(o[2 * i + 1], pr, b[2], b[3]);
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();                            // the ring is done with
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int r = (lane >> 2) + 8 * h;
        if ((lane & 3) == 0) {
            stat_w[warp * 16 + r] = make_float2(m[h], l[h]);
            if (kKeyWarps == 1) stat[warp * 16 + r] = make_float2(m[h], l[h]);
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(buf + (warp * 16 + r) * S::kLdo + 8 * i + 2 * (lane & 3)) =
                make_float2(o[i][2 * h], o[i][2 * h + 1]);
    }
    if (kKeyWarps > 1) {
        // the warps that share the rows' keys, in order; the sum lies with the first of them
        __syncthreads();
        for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4);
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kKeyWarps; ++w) M = fmaxf(M, stat_w[w * kRows + r].x);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kKeyWarps; ++w) {
                const float2 st = stat_w[w * kRows + r];
                const float f = part_weight(st.x, st.y, M);
                if (!(st.y == 0.f)) L += f * st.y;
                const float4 y = *reinterpret_cast<const float4*>(buf + (w * kRows + r) * S::kLdo + 4 * c);
                x.x = fmaf(f, y.x, x.x);
                x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z);
                x.w = fmaf(f, y.w, x.w);
            }
            *reinterpret_cast<float4*>(buf + r * S::kLdo + 4 * c) = x;     // (which only this thread has read)
            if (c == 0) stat[r] = make_float2(M, L);
        }
    }
    join_cluster<__nv_bfloat16, 1, D / 4>(p, t, buf, S::kLdo, stat, warp, kWarps);
}

// Rows of a tile by what a sequence and key head have on average, in units of 16.
int row_warps(const PagedArgs& a)
{
    const long long rows = static_cast<long long>(a.T) * (a.H / a.H_kv);
    return rows <= 16ll * a.n_seqs ? 1 : rows <= 32ll * a.n_seqs ? 2 : 4;
}

// The cluster size of a call, or 0 where the kernels for more tiles are better: the largest with
// which all tiles are held at once, if no CTA then gets more than 16 steps, or 8 of 64 rows beside
// others (two CTAs of an SM share its matrix units).  Only the table tells beforehand how many
// keys there may be.  Measured against those kernels, 32 heads over 8 of 128 dims: one sequence of
// 2000 keys, 4 tokens 8.5 us and 14.5, 26 tokens 13.4 and 22, 64 tokens 15.4 and 33; of 8000 keys,
// 4 tokens 14 and 20, 26 tokens 33 and 33; of 32000, 4 tokens 41 and 39; four sequences, 8 tokens
// over 1000 keys 10 and 17, over 4000 20 and 25, 26 tokens over 500 14 and 18, over 4000 keys of
// two 27 and 26; sixteen, 5 tokens over 700 (12 heads over 4) 10.5 and 16.6, 4 over 1000 18.6 and
// 20.6.  (13 tokens over 200, one CTA a tile of 64 rows, 13.7 and 12.0: not this way.)
template <int D, int kRowWarps>
int ctas_of(const PagedArgs& a)
{
    static std::atomic<int> known[5][kMaxDevices];
    const long long tiles = most_tiles(a, 16 * kRowWarps);
    const long long keys = static_cast<long long>(a.max_pages) * a.page_size;
    for (int i = 0; i < (kRowWarps < 4 ? 5 : 4); ++i) {
        const int ctas = kMostCtas >> i;
        if (keys > static_cast<long long>(ctas) * kKeys * (i < 2 || kRowWarps < 4 ? 16 : 8)) return 0;
        int held = 0;
        if (clusters_held(known[i], paged_tree_kernel<D, kRowWarps>, kThreads, Smem<D>::kBytes, ctas, &held) == cudaSuccess &&
            tiles <= held)
            return ctas;
    }
    return 0;
}

// Launches the call if it goes this way.
template <int D, int kRowWarps>
bool go(const PagedArgs& a, cudaError_t* e)
{
    const int ctas = ctas_of<D, kRowWarps>(a);
    if (ctas == 0) return false;
    PagedParams p;
    fill_params(&p, a);
    *e = launch_clusters(paged_tree_kernel<D, kRowWarps>, p, most_tiles(a, 16 * kRowWarps), ctas, kThreads,
                         Smem<D>::kBytes);
    return true;
}
template <int D>
bool go_rows(const PagedArgs& a, cudaError_t* e)
{
    switch (row_warps(a)) {
    case 1: return go<D, 1>(a, e);
    case 2: return go<D, 2>(a, e);
    default: return go<D, 4>(a, e);
    }
}

}  // namespace

bool paged_tree_bf16(const PagedArgs& a, cudaError_t* e)
{
    if (a.D == 64) return go_rows<64>(a, e);
    return a.D == 128 && go_rows<128>(a, e);
}

}  // namespace ra
