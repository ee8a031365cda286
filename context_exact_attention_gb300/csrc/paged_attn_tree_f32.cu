// paged_attn_tree_f32.cu -- paged_attn_tree_fwd for calls with few tiles, fp32: a cluster of CTAs
// for every tile (paged_attn_tree.cu), whose products are tiled in registers
// (paged_attn_simt_rows.cu).
//
// A tile is 16 or 32 packed rows.  Of its 128 threads, (ty, tx) holds the scores of kR rows,
// ty + 8 i, with the keys tx + 16 j of a step, and the output of the same rows in columns
// 4 (tx + 16 u).  Keys lie with their 16-byte chunks permuted by the key's low bits, weights with
// bit 4 of the key flipped in odd rows.  Keys and values come 32 at a time through a ring, a step
// ahead.
//
// What bounds it: instructions, of one or two warps a scheduler, with few of each other's latencies
// to hide: a step of 32 keys of 16 rows of 128 dims takes 2.5 us.  Measured against the kernels
// for more tiles (four rows at a time, or 64 in paged_attn_simt_rows.cu): 8 sequences of 13
// tokens, 8 heads over 2 of 128 dims, 500 keys, 23 us and 25; 26 tokens, 32 heads over 8, 2000
// keys, 47 and 64; 100 tokens, 8 heads over 2, 1000 keys, 30 and 60; of 64 dims, 16 of 4 tokens,
// 500 keys, 9 and 16; 2 of 40 tokens, 16 heads over 4, 1000 keys, 22 and 44.
#include <algorithm>
#include <type_traits>

#include "paged_cluster.cuh"

namespace ra {
namespace {

constexpr int kThreads = 128;
constexpr int kTy = kThreads / 16;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 32;                       // keys of a step
constexpr int kKeysW = kKeys / kWarps;         // ... that a warp copies
constexpr int kPer = kKeys / 16;               // ... of a thread's scores

// Shared memory: queries, a ring of keys and values (then the tile's sums), weights, statistics.
constexpr int kStages = 2;                     // (a third costs the second CTA of an SM: 12 to 90 % slower)
template <int kCols, int kR>
constexpr int kSmem = ((kTy * kR + kStages * 2 * kKeys) * 64 * kCols + kTy * kR * kKeys) * 4 + kTy * kR * 8;

// kCols: column groups of 64 (D <= 64 kCols; the columns behind D are zeros).
template <int kCols, int kR>
__global__ void __launch_bounds__(kThreads, kCols <= 2 ? 2 : 1)
    paged_tree_f32_kernel(const __grid_constant__ PagedParams p)
{
    constexpr int kD = 64 * kCols, kChunks = 16 * kCols, kRows = kTy * kR;
    extern __shared__ __align__(16) float smem[];
    float* qs = smem;
    float* ring = qs + kRows * kD;
    float* ps = ring + kStages * 2 * kKeys * kD;
    float2* stat = reinterpret_cast<float2*>(ps + kRows * kKeys);
    const PagedArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int D4 = a.D / 4;
    const int ctas = p.grid, rank = static_cast<int>(cluster_ctarank());
    const float* Q = static_cast<const float*>(a.q);
    const float* K = static_cast<const float*>(a.k_pages);
    const float* V = static_cast<const float*>(a.v_pages);

    // `count` rows of a warp, whose offsets its first lanes hold (-1: zeros).
    auto copy = [&](float* dst, const float* src, long long off, long long extent, int count, bool permuted) {
        const uint32_t to = smem_addr(dst) + count * warp * kD * 4;
#pragma unroll 4
        for (int i = 0; i < count * kChunks / 32; ++i) {
            const int e = lane + 32 * i, r = e / kChunks, c = e % kChunks;
            const long long o = __shfl_sync(0xffffffffu, off, r);
            const bool real = o >= 0 && c < D4 && in_bounds(o + 4 * c, 4, extent, a.status);
            cp_async16(to + (r * kD + 4 * (permuted ? c ^ (r & 7) : c)) * 4, src + (real ? o + 4 * c : 0), real);
        }
    };

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
    // The copies run up to kStages - 1 steps ahead; a warp's keys are looked up a step before.
    long long off = -1;
    int issued = s0;
    auto look_up = [&]() {
        const int key = kKeys * issued + kKeysW * warp + lane;
        off = issued < s1 && lane < kKeysW && key < span.kv ? key_offset(p, g, t.hk, key) : -1;
    };
    auto issue = [&]() {
        if (issued < s1) {
            float* k = ring + (issued - s0) % kStages * (2 * kKeys * kD);
            copy(k, K, off, a.page_elems, kKeysW, true);
            copy(k + kKeys * kD, V, off, a.page_elems, kKeysW, false);
            ++issued;
            look_up();
        }
        cp_async_commit();                      // (an empty group where there is no step)
    };
    look_up();
    {
        constexpr int kMine = kRows / kWarps;   // rows of the tile that a warp copies
        const int r = kMine * warp + lane, pr = t.row0 + r, tok = p.token_of(pr);
        copy(qs, Q,
             lane < kMine && r < t.rows ? (t.first + tok) * a.q_stride +
                                              static_cast<long long>(t.hk * p.G + (pr - tok * p.G)) * a.D
                                        : -1,
             a.q_elems, kMine, false);
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    const int before = min(span.kv - span.n, span.kv);      // keys from before the step
    uint64_t o[kR][kCols][2];
    float m[kR], l[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int u = 0; u < kCols; ++u) o[i][u][0] = o[i][u][1] = 0;
    }
#pragma unroll 1
    for (int n = s0; n < s1; ++n) {
        cp_async_wait<kStages - 2>();
        __syncthreads();                        // the step is here, and the one before has been read
        issue();
        const float* ks = ring + (n - s0) % kStages * (2 * kKeys * kD);
        const float* vs = ks + kKeys * kD;
        uint64_t acc[kR][kPer] = {};
#pragma unroll 8
        for (int c = 0; c < D4; ++c) {
            ulonglong2 q[kR], k[kPer];
#pragma unroll
            for (int i = 0; i < kR; ++i)
                q[i] = *reinterpret_cast<const ulonglong2*>(qs + (ty + kTy * i) * kD + 4 * c);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                k[j] = *reinterpret_cast<const ulonglong2*>(ks + (tx + 16 * j) * kD + 4 * (c ^ (tx & 7)));
#pragma unroll
            for (int i = 0; i < kR; ++i)
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    acc[i][j] = ffma2(q[i].x, k[j].x, acc[i][j]);
                    acc[i][j] = ffma2(q[i].y, k[j].y, acc[i][j]);
                }
        }
        const int kb = kKeys * n;
        const bool tail = kb + kKeys > before;
        bool raised = false;
        float alpha[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const int r = ty + kTy * i;
            float s[kPer], mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int key = kb + tx + 16 * j;
                float lo, hi;
                f2unpack(acc[i][j], lo, hi);
                bool sees = true;
                if (tail && key >= before)
                    sees = key < span.kv && r < t.rows &&
                           (seen_from(p, t.first + p.token_of(t.row0 + r), key - (span.kv - span.n)) & 1);
                s[j] = sees ? (lo + hi) * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[j]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float m_new = fmaxf(m[i], mx);
            alpha[i] = m_new > m[i] ? ex2(m[i] - m_new) : 1.f;
            raised |= alpha[i] != 1.f;
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const float w = ex2(s[j] - ref);
                sum += w;
                ps[r * kKeys + ((tx + 16 * j) ^ (16 * (ty & 1)))] = w;
            }
            l[i] = l[i] * alpha[i] + sum;
            m[i] = m_new;
        }
        if (__any_sync(0xffffffffu, raised)) {
#pragma unroll
            for (int i = 0; i < kR; ++i)
#pragma unroll
                for (int u = 0; u < kCols; ++u) {
                    o[i][u][0] = fmul2(o[i][u][0], f2pack(alpha[i], alpha[i]));
                    o[i][u][1] = fmul2(o[i][u][1], f2pack(alpha[i], alpha[i]));
                }
        }
        __syncthreads();                        // the weights are here
        auto add_values = [&](auto every) {
#pragma unroll 2
            for (int k4 = 0; k4 < kKeys / 4; ++k4) {
                float w[kR][4];
#pragma unroll
                for (int i = 0; i < kR; ++i)
                    *reinterpret_cast<float4*>(w[i]) = *reinterpret_cast<const float4*>(
                        ps + (ty + kTy * i) * kKeys + ((4 * k4) ^ (16 * (ty & 1))));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    ulonglong2 v[kCols];
#pragma unroll
                    for (int u = 0; u < kCols; ++u)
                        v[u] = *reinterpret_cast<const ulonglong2*>(vs + (4 * k4 + kk) * kD + 4 * (tx + 16 * u));
#pragma unroll
                    for (int i = 0; i < kR; ++i) {
                        if (!every.value && w[i][kk] == 0.f) continue;
                        const uint64_t ww = f2pack(w[i][kk], w[i][kk]);
#pragma unroll
                        for (int u = 0; u < kCols; ++u) {
                            o[i][u][0] = ffma2(ww, v[u].x, o[i][u][0]);
                            o[i][u][1] = ffma2(ww, v[u].y, o[i][u][1]);
                        }
                    }
                }
            }
        };
        // a value that a row does not see stays out even if it is not finite
        if (!tail) add_values(std::true_type());
        else add_values(std::false_type());
    }
    cp_async_wait<0>();
    __syncthreads();                            // the ring is done with
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        const int r = ty + kTy * i;
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
        if (tx == 0) stat[r] = make_float2(m[i], l[i]);
#pragma unroll
        for (int u = 0; u < kCols; ++u) {
            float4 x;
            f2unpack(o[i][u][0], x.x, x.y);
            f2unpack(o[i][u][1], x.z, x.w);
            *reinterpret_cast<float4*>(ring + r * kD + 4 * (tx + 16 * u)) = x;
        }
    }
    join_cluster<float, kCols == 1 ? 1 : kCols / 2 + kCols % 2, kCols == 1 ? 16 : 32>(p, t, ring, kD, stat, warp,
                                                                                     kWarps);
}

// Rows of a tile: 32 where a sequence and key head has more than 16 on average and the call then
// still has enough tiles.
int tile_rows(const PagedArgs& a)
{
    const long long rows = static_cast<long long>(a.T) * (a.H / a.H_kv);
    return rows > 16ll * a.n_seqs && most_tiles(a, 16) >= 48 ? 32 : 16;
}

// The cluster size of a call, or 0 where the other kernels are better: where its tiles are so few
// that the GPU would be empty (8 heads over 2 of 128 dims: 4 tokens, 2000 keys, 15.5 us and 13.5;
// 13 tokens, 4000 keys, 34 and 25; 4 sequences of up to 13 tokens and 1500 keys, 22 and 18.6), or a
// CTA would get too many steps.  Only the table tells beforehand how many keys there may be.
template <int kCols, int kR>
int ctas_of(const PagedArgs& a)
{
    constexpr int kLeastTiles = kCols == 1 ? 16 : 48, kMostSteps = 32;
    static std::atomic<int> known[5][kMaxDevices];
    const long long tiles = most_tiles(a, kTy * kR);
    const long long keys = static_cast<long long>(a.max_pages) * a.page_size;
    if (most_tiles(a, 16) < kLeastTiles) return 0;
    for (int i = 0; i < 5; ++i) {
        const int ctas = kMostCtas >> i;
        if (keys > static_cast<long long>(ctas) * kKeys * kMostSteps) return 0;
        int held = 0;
        if (clusters_held(known[i], paged_tree_f32_kernel<kCols, kR>, kThreads, kSmem<kCols, kR>, ctas, &held) ==
                cudaSuccess &&
            tiles <= held)
            return ctas;
    }
    return 0;
}

// Launches the call if it goes this way.
template <int kCols, int kR>
bool go(const PagedArgs& a, cudaError_t* e)
{
    const int ctas = ctas_of<kCols, kR>(a);
    if (ctas == 0) return false;
    PagedParams p;
    fill_params(&p, a);
    *e = launch_clusters(paged_tree_f32_kernel<kCols, kR>, p, most_tiles(a, kTy * kR), ctas, kThreads, kSmem<kCols, kR>);
    return true;
}
template <int kCols>
bool go_cols(const PagedArgs& a, cudaError_t* e)
{
    return tile_rows(a) == 16 ? go<kCols, 16 / kTy>(a, e) : go<kCols, 32 / kTy>(a, e);
}

}  // namespace

bool paged_tree_f32(const PagedArgs& a, cudaError_t* e)
{
    return a.D <= 64    ? go_cols<1>(a, e)
           : a.D <= 128 ? go_cols<2>(a, e)
           : a.D <= 192 ? go_cols<3>(a, e)
                        : go_cols<4>(a, e);
}

}  // namespace ra
