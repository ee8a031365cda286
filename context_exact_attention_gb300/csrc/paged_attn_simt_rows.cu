// paged_attn_simt_rows.cu -- paged_attn_fwd for fp32 calls with many query rows per key/value
// head (prompts, chunks of them): both products tiled in registers.
//
// A tile is 64 packed rows (whole tokens with the G query heads that read the head) in shared
// memory; the block walks its keys 64 at a time.  Thread (ty, tx) holds the scores of 8 rows
// (4 above 128 dims, whose sums fill the registers), ty apart by the number of ty, with the
// keys tx + 16 j, and the output of the same rows in columns 4 (tx + 16 u): 8 x 4 dot products
// from twelve 16-byte reads per four columns of S = Q K^T, and 8 rows of columns from one read
// per key and column group of P V, the arithmetic in pairs.  A row's 16 threads are half of a
// warp, so its maximum takes four shuffles.  Keys lie with their 16-byte chunks permuted by the
// key's low bits, and weights with bit 4 of the key flipped in odd rows, so that the reads of a
// warp spread over the banks.  The next keys are copied (asynchronously) during the second
// product, the next values during the first; two blocks on an SM up to 128 dims fill each
// other's gaps.
//
// What bounds it: fp32 arithmetic (64 keys of 64 rows take 2 64 64 D FMA, 8192 cycles of an SM
// at 128 dims), the reads from shared memory that feed it, and eight warps an SM that wait for
// both in turn.
// Measured: a prompt of 1000 tokens, 8 heads of 128, 106 us (216 four rows at a time), 19 TFLOP/s
// of pairs that are seen: the SMs have work 63 % of the time (128 tiles of unequal length for 304
// CTAs), in which the FMA pipe is busy 52 %, the shared memory 42 % and the issue slots 44 %.  8
// heads over 2 of 64, 56 us (187).  4 rows a thread instead of 8: 113 and 62.
#include <type_traits>

#include "paged_plan.cuh"

namespace ra {
namespace {

constexpr int kRows = 64;
constexpr int kKeys = 64;
// rows of a thread, and threads: 8 rows as long as their sums fit the registers
template <int kCols>
constexpr int kPer = kCols <= 2 ? 8 : 4;
template <int kCols>
constexpr int kThreads = 16 * kRows / kPer<kCols>;

// Shared memory: queries (then the tile's sums), keys, values, weights.
template <int kCols>
constexpr int kSmem = (3 * kRows * 64 * kCols + kRows * kKeys) * 4;

// kCols: column groups of 64 (D <= 64 kCols; the columns behind D are zeros).
// kTree: rows see the new tokens that their masks name.
template <int kCols, bool kTree>
__global__ void __launch_bounds__(kThreads<kCols>, kCols <= 2 ? 2 : 1)
    paged_rows_kernel(const __grid_constant__ PagedParams p)
{
    using Walk = PagedWalk<StepTiles, kKeys>;
    constexpr int kD = 64 * kCols, kChunks = 16 * kCols;
    constexpr int kR = kPer<kCols>, kStep = kRows / kR;       // a thread's rows are kStep apart
    constexpr int kCopied = kRows / (kThreads<kCols> / 32);   // rows of a tile that a warp copies
    extern __shared__ __align__(16) float smem[];
    float* qs = smem;
    float* ks = qs + kRows * kD;
    float* vs = ks + kKeys * kD;
    float* ps = vs + kKeys * kD;
    __shared__ float2 stat[kRows];
    __shared__ int flag;
    const PagedArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int D4 = a.D / 4;
    const float* Q = static_cast<const float*>(a.q);
    const float* K = static_cast<const float*>(a.k_pages);
    const float* V = static_cast<const float*>(a.v_pages);

    // This warp's rows of a 64-row tile, whose offsets its first lanes hold (-1: zeros).
    auto copy = [&](float* dst, const float* src, long long off, long long extent, bool permuted) {
        const uint32_t to = smem_addr(dst) + kCopied * warp * kD * 4;
#pragma unroll
        for (int i = 0; i < kCopied * kChunks / 32; ++i) {
            const int e = lane + 32 * i, r = e / kChunks, c = e % kChunks;
            const long long o = __shfl_sync(0xffffffffu, off, r);
            const bool real = o >= 0 && c < D4 && in_bounds(o + 4 * c, 4, extent, a.status);
            cp_async16(to + (r * kD + 4 * (permuted ? c ^ (r & 7) : c)) * 4, src + (real ? o + 4 * c : 0), real);
        }
    };

    wait_for_earlier_work();
    Walk walk;
    walk.begin(p);
    Segment t;
#pragma unroll 1
    while (walk.next(p, t)) {
        const int steps = t.k1 > t.k0 ? (t.k1 - t.k0 + kKeys - 1) / kKeys : 0;
        auto look_up = [&](int n) -> long long {
            const int key = t.k0 + kKeys * n + kCopied * warp + lane;
            return n < steps && lane < kCopied && key < t.k1 ? key_offset(p, t.g, t.hk, key) : -1;
        };
        long long off = look_up(0);
        if (steps > 0) {
            const int r = kCopied * warp + lane, pr = t.row0 + r, tok = p.token_of(pr);
            copy(qs, Q,
                 lane < kCopied && r < t.rows ? (t.s.first + tok) * a.q_stride +
                                              static_cast<long long>(t.hk * p.G + (pr - tok * p.G)) * a.D
                                        : -1,
                 a.q_elems, false);
            copy(ks, K, off, a.page_elems, true);
            cp_async_commit();
            copy(vs, V, off, a.page_elems, false);
            cp_async_commit();
        }
        // keys that this thread's rows see of those before t.k1
        int end[kR], least = t.k1;
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const int r = ty + kStep * i, tok = p.token_of(t.row0 + r);
            // (of a tree: those from before the step)
            const int seen = kTree ? t.s.kv - t.s.n : a.causal ? t.s.kv - t.s.n + tok + 1 : t.s.kv;
            end[i] = r >= t.rows ? 0 : min(seen, t.k1);
            if (r < t.rows) least = min(least, end[i]);
        }
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
        for (int n = 0; n < steps; ++n) {
            off = look_up(n + 1);
            cp_async_wait<1>();                                // this step's keys (and the queries)
            __syncthreads();
            uint64_t acc[kR][4] = {};
#pragma unroll 2
            for (int c = 0; c < D4; ++c) {
                ulonglong2 q[kR], k[4];
#pragma unroll
                for (int i = 0; i < kR; ++i)
                    q[i] = *reinterpret_cast<const ulonglong2*>(qs + (ty + kStep * i) * kD + 4 * c);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    k[j] = *reinterpret_cast<const ulonglong2*>(ks + (tx + 16 * j) * kD +
                                                                4 * (c ^ (tx & 7)));
#pragma unroll
                for (int i = 0; i < kR; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[i][j] = ffma2(q[i].x, k[j].x, acc[i][j]);
                        acc[i][j] = ffma2(q[i].y, k[j].y, acc[i][j]);
                    }
            }
            __syncthreads();                                   // the keys have been read
            copy(ks, K, off, a.page_elems, true);
            cp_async_commit();
            const int kb = t.k0 + kKeys * n;
            bool raised = false;
            float alpha[kR];
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                float s[4], mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    f2unpack(acc[i][j], lo, hi);
                    const int key = kb + tx + 16 * j, r = ty + kStep * i;
                    bool sees = key < end[i];
                    if (kTree && key >= end[i] && key < t.k1 && r < t.rows)
                        sees = seen_from(p, t.s.first + p.token_of(t.row0 + r), key - (t.s.kv - t.s.n)) & 1;
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
                const int row = ty + kStep * i;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = ex2(s[j] - ref);
                    sum += w;
                    ps[row * kKeys + ((tx + 16 * j) ^ (16 * (ty & 1)))] = w;
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
            cp_async_wait<1>();                                // this step's values
            __syncthreads();
            auto add_values = [&](auto every) {
#pragma unroll 1
                for (int k4 = 0; k4 < kKeys / 4; ++k4) {
                    float w[kR][4];
#pragma unroll
                    for (int i = 0; i < kR; ++i)
                        *reinterpret_cast<float4*>(w[i]) = *reinterpret_cast<const float4*>(
                            ps + (ty + kStep * i) * kKeys + ((4 * k4) ^ (16 * (ty & 1))));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        ulonglong2 v[kCols];
#pragma unroll
                        for (int u = 0; u < kCols; ++u)
                            v[u] = *reinterpret_cast<const ulonglong2*>(vs + (4 * k4 + kk) * kD +
                                                                        4 * (tx + 16 * u));
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
            if (__all_sync(0xffffffffu, kb + kKeys <= least)) add_values(std::true_type());
            else add_values(std::false_type());
            __syncthreads();                                   // the values have been read
            copy(vs, V, off, a.page_elems, false);
            cp_async_commit();
        }
        cp_async_wait<0>();
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const int row = ty + kStep * i;
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
            if (tx == 0) stat[row] = make_float2(m[i], l[i]);
#pragma unroll
            for (int u = 0; u < kCols; ++u) {
                float4 x;
                f2unpack(o[i][u][0], x.x, x.y);
                f2unpack(o[i][u][1], x.z, x.w);
                *reinterpret_cast<float4*>(qs + row * kD + 4 * (tx + 16 * u)) = x;
            }
        }
        __syncthreads();
        finish_segment<float, kRows, kThreads<kCols>, (kD > 128 ? 2 : 1)>(p, t, qs, kD, stat, &flag);
    }
}

template <int kCols, bool kTree>
cudaError_t launch_cols(PagedParams& p)
{
    constexpr auto kernel = paged_rows_kernel<kCols, kTree>;
    static std::atomic<int> known[kMaxDevices];
    int grid = 0;
    const cudaError_t e = resident_ctas(known, kernel, kThreads<kCols>, kSmem<kCols>, &grid);
    if (e != cudaSuccess) return e;
    p.grid = grid < kPagedRowsCtas ? grid : kPagedRowsCtas;
    const PagedWorkspace w = paged_workspace_of(p.grid, kRows, p.a.D);
    uint8_t* ws = static_cast<uint8_t*>(p.a.workspace);
    p.counters = reinterpret_cast<unsigned int*>(ws);
    p.part_stat = reinterpret_cast<float*>(ws + w.stat);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    return launch_early(kernel, p.grid, kThreads<kCols>, kSmem<kCols>, p.a.stream, p);
}

}  // namespace

bool paged_rows_applies(const PagedArgs& a)
{
    // Many rows, counted per sequence and key head on average (the lengths are not known here),
    // and many tiles or very many rows.  Measured, four rows at a time against this kernel, 2
    // key heads of 128 dims: 16 sequences of 1000 keys, 32 rows 47 us against 59, 64 rows 80
    // against 63, 400 rows 420 against 249; one of 8000 keys, 160 rows 92 against 99, 400 rows
    // 209 against 132; 32 of 64 keys, 64 rows 22 against 20, 96 rows 28 against 33, 400 rows 108
    // against 73; 8 heads, one sequence of 4763 keys, 195 rows 242 against 170; 64 dims, 4000
    // rows over 1000 keys 187 against 56; 256 dims, 1200 rows over 3000 keys 557 against 248.
    // Where the table holds a few steps of keys only, a tile cannot be split and many are needed
    // to fill the GPU (three prompts of 180 tokens, 6 heads over 3, 36 tiles: 27 us against 41).
    const int G = a.H / a.H_kv;
    const long long rows = static_cast<long long>(a.T) * G;
    const bool few_keys = static_cast<long long>(a.max_pages) * a.page_size <= 4 * kKeys;
    return a.elem == 4 && G <= kRows && rows >= 64ll * a.n_seqs &&
           (rows * a.H_kv >= (few_keys ? 128ll : 24ll) * kRows || (!few_keys && rows >= 384ll * a.n_seqs));
}

cudaError_t launch_paged_rows(const PagedArgs& a)
{
    PagedParams p;
    fill_params(&p, a);
    p.tile_tokens = kRows / p.G;
    p.key_shift = p.key_shift_single = 0;
    p.tile_cost = 128;
    p.snap = 2 * kKeys;
    p.min_chunk = 2 * kKeys;
    p.whole = 0;
    p.join_cost = 8;                // (4, 16, 64: 83, 103, 144 us for 64 rows over 8000 keys of 2 heads)
    if (a.D <= 64) return a.masks ? launch_cols<1, true>(p) : launch_cols<1, false>(p);
    if (a.D <= 128) return a.masks ? launch_cols<2, true>(p) : launch_cols<2, false>(p);
    if (a.D <= 192) return a.masks ? launch_cols<3, true>(p) : launch_cols<3, false>(p);
    return a.masks ? launch_cols<4, true>(p) : launch_cols<4, false>(p);
}

}  // namespace ra
