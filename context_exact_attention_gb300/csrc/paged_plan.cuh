// paged_plan.cuh -- how the kernels of paged_attn_fwd share out their work, and how the
// pieces of a row's softmax that different CTAs computed are joined.
//
// A tile is the query rows of one key/value head that one CTA holds at a time: the new
// tokens of a sequence times the H / H_kv query heads that read the head, packed
// token-major ("packed row" r is token r / G, head r % G of the group).  The tiles of a
// call are laid end to end, sequence by sequence, head by head, on one axis whose unit is
// a visited key, each tile kTileCost + its keys long, and CTA c takes the part
// [c chunk, (c + 1) chunk) of that axis: whatever the lengths are, every CTA reads the
// same number of keys, and one token over a long cache fills the whole GPU.  Everything is
// computed from the lengths on the device in each CTA (a scan over the sequences), so a
// captured call follows the lengths that it finds when it is replayed.
//
// A tile that lies in one CTA's part is written by that CTA.  Of a tile cut by a part's
// end each CTA writes its unnormalised sum, maximum and denominator to its own place in
// the workspace and counts itself in; the last one to arrive reads all of them and joins
// them in CTA order, so the result does not depend on who is last.  Nobody waits.
#pragma once

#include <cuda_bf16.h>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {

constexpr float kPagedLn2 = 0.6931471805599453f;
constexpr int kTileCost = 64;       // a tile's fixed cost (its queries and output), in keys

// Kernel-side copy of PagedArgs, with the split.
struct PagedParams {
    PagedArgs a;
    int G;                  // query heads per key/value head
    int grid;
    int min_chunk;          // smallest part worth a CTA, in keys
    int tile_tokens;        // new tokens of a tile (StepTiles)
    int page_shift;         // log2 of the page size, or -1
    float scale_log2;       // log2(e) / sqrt(D): scores in base-2 units
    unsigned int* counters; // [kPagedMaxCtas], zero between calls
    float* part_stat;       // [2 grid][rows][2]: maximum, denominator
    float* part_o;          // [2 grid][rows][D]
};

// The workspace, in bytes: work counters, then the statistics and sums of two partial tiles
// for every CTA.  (rows packed rows of a tile; the sums lie as each kernel likes.)
struct PagedWorkspace {
    unsigned long long stat, o, total;
};
inline PagedWorkspace paged_workspace_of(int ctas, int rows, int D)
{
    PagedWorkspace w;
    w.stat = 4ull * kPagedMaxCtas;
    w.o = w.stat + 2ull * ctas * rows * 8;
    w.total = w.o + 2ull * ctas * rows * D * 4;
    return w;
}

inline int page_shift_of(int page_size)
{
    int k = 0;
    while ((1 << k) < page_size) ++k;
    return (1 << k) == page_size ? k : -1;
}

// The new tokens and keys of sequence g, clamped to what the call's tensors hold.
struct SeqSpan {
    int first, n;           // first token row, new tokens
    int kv;                 // keys
};
__device__ __forceinline__ SeqSpan seq_span_of(const PagedArgs& a, int g)
{
    SeqSpan s;
    const int lo = checked_ldg(a.cu_new, g, a.n_seqs + 1, a.status);
    const int hi = checked_ldg(a.cu_new, g + 1, a.n_seqs + 1, a.status);
    const int kv = checked_ldg(a.kv_lens, g, a.n_seqs, a.status);
    s.first = min(max(lo, 0), a.T);
    s.n = min(max(hi, s.first), a.T) - s.first;
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
    s.kv = static_cast<int>(min(static_cast<long long>(max(kv, 0)), cap));
    return s;
}

// a / b of non-negative values, in 32 bits where they fit (several times shorter).
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    if (static_cast<unsigned long long>(a | b) >> 32) return a / b;
    return static_cast<unsigned>(a) / static_cast<unsigned>(b);
}

// Tiles of one (sequence, head).  kRows packed rows a tile; every tile of a sequence
// counts all the keys (sequences with few new tokens see nearly all in every tile).
template <int kRows>
struct FlatTiles {
    int n_tiles;
    long long cost;         // of one tile
    __device__ __forceinline__ static int rows(const PagedParams&) { return kRows; }
    __device__ __forceinline__ void init(const PagedParams& p, const SeqSpan& s)
    {
        n_tiles = (s.n * p.G + kRows - 1) / kRows;        // n G <= T H < 2^31 - 16
        cost = kTileCost + s.kv;
    }
    __device__ __forceinline__ long long prefix(int j) const { return j * cost; }
    __device__ __forceinline__ int at(long long x) const { return static_cast<int>(quotient(x, cost)); }
};

// The same where a sequence may have many tiles: under the causal rule tile j of `per` tokens
// sees (up to) the keys before the new tokens and the first (j + 1) per of those, so a
// sequence's costs form an arithmetic series, summed in closed form and searched by halving.
struct StepTiles {
    int n_tiles, per, n, kv, causal;
    long long before;       // keys before the new tokens
    __device__ __forceinline__ static int rows(const PagedParams& p) { return p.tile_tokens * p.G; }
    __device__ __forceinline__ void init(const PagedParams& p, const SeqSpan& s)
    {
        per = p.tile_tokens;
        n = s.n;
        kv = s.kv;
        causal = p.a.causal;
        before = max(s.kv - s.n, 0);
        n_tiles = (s.n + per - 1) / per;
    }
    __device__ __forceinline__ long long prefix(int j) const
    {
        if (!causal) return j * (static_cast<long long>(kTileCost) + kv);
        // full tiles before j, and the last one, which ends with the last token
        long long c = j * (kTileCost + before);
        const long long full = j < n_tiles ? j : n_tiles - 1;
        c += per * (full * (full + 1) / 2);
        return j < n_tiles ? c : c + n;
    }
    __device__ __forceinline__ int at(long long x) const
    {
        if (!causal) return static_cast<int>(quotient(x, static_cast<long long>(kTileCost) + kv));
        int lo = 0, hi = n_tiles;               // prefix(lo) <= x < prefix(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix(mid) <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

// One CTA's share of one tile.
struct Segment {
    int g, hk;              // sequence, key/value head
    int row0;               // first packed row of the tile within the sequence (T * H < 2^31)
    int rows;               // packed rows of the tile
    SeqSpan s;
    int keys;               // keys that some row of the tile sees: [0, keys)
    int k0, k1;             // this CTA's part of them
    int c_first, c_last;    // the CTAs that share the tile
};

// Walk over the segments of this CTA.  kUnit: keys per step of the kernel, to which cuts
// inside a tile are rounded.
template <typename Tiles, int kUnit>
struct PagedWalk {
    long long x, end, chunk;
    long long seq0, seq_cost, head_cost;
    int g;
    SeqSpan s;
    Tiles tiles;

    __device__ __forceinline__ void load_seq(const PagedParams& p)
    {
        s = seq_span_of(p.a, g);
        tiles.init(p, s);
        head_cost = tiles.prefix(tiles.n_tiles);
        seq_cost = head_cost * p.a.H_kv;
    }
    // keys before the cut at offset x of a tile that has `keys` keys and cost `cost`
    __device__ __forceinline__ static int cut(long long x, long long cost, int keys)
    {
        if (x <= 0) return 0;
        if (x >= cost) return keys;
        const long long k = x - kTileCost;
        if (k <= 0) return 0;
        return static_cast<int>(min(static_cast<long long>(keys), k / kUnit * kUnit));
    }
    __device__ __forceinline__ bool next(const PagedParams& p, Segment& t)
    {
        if (x >= end) return false;
        while (x >= seq0 + seq_cost) {
            seq0 += seq_cost;
            if (++g >= p.a.n_seqs) return false;
            load_seq(p);
        }
        const long long rel = x - seq0;
        t.hk = static_cast<int>(quotient(rel, head_cost));
        const long long head0 = t.hk * head_cost;
        const int j = tiles.at(rel - head0);
        const long long a = seq0 + head0 + tiles.prefix(j), b = seq0 + head0 + tiles.prefix(j + 1);
        t.g = g;
        t.s = s;
        const int rows = Tiles::rows(p);
        t.row0 = j * rows;
        t.rows = min(rows, s.n * p.G - t.row0);
        // the last token of the tile sees the most keys
        const int last = (t.row0 + t.rows - 1) / p.G;
        t.keys = p.a.causal ? min(max(s.kv - s.n + last + 1, 0), s.kv) : s.kv;
        const long long stop = min(end, b);
        t.k0 = cut(x - a, b - a, t.keys);
        t.k1 = cut(stop - a, b - a, t.keys);
        t.c_first = static_cast<int>(quotient(a, chunk));
        t.c_last = static_cast<int>(quotient(b - 1, chunk));
        x = stop;
        return true;
    }
    // The same in every thread of the block; scratch: 34 long longs of shared memory.
    template <int kThreads>
    __device__ void begin(const PagedParams& p, long long* scratch)
    {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        constexpr int kWarps = kThreads / 32;
        // pass 0 sums the costs; pass 1 finds the sequence at the start of this CTA's part
        // (one round of loads when the sequences fit the block)
        long long total = 0, mine = 0;
        auto cost_of = [&](int i) -> long long {
            if (i >= p.a.n_seqs) return 0;
            Tiles t;
            t.init(p, seq_span_of(p.a, i));
            return t.prefix(t.n_tiles) * p.a.H_kv;
        };
        auto block_scan = [&](long long v, long long& sum) -> long long {   // exclusive
            long long inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            __syncthreads();
            if (lane == 31) scratch[warp] = inc;
            __syncthreads();
            long long before = 0;
            sum = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const long long z = scratch[w];
                if (w < warp) before += z;
                sum += z;
            }
            return before + inc - v;
        };
        long long excl = 0;
        for (int base = 0; base < p.a.n_seqs; base += kThreads) {
            mine = cost_of(base + tid);
            long long sum;
            excl = block_scan(mine, sum);
            total += sum;
        }
        chunk = max((total + p.grid - 1) / p.grid, static_cast<long long>(p.min_chunk));
        x = blockIdx.x * chunk;
        end = min(total, x + chunk);
        g = 0;
        seq0 = 0;
        if (x >= total) {
            x = end;                // nothing for this CTA
            return;
        }
        if (tid == 0) scratch[32] = 0;
        __syncthreads();
        long long before = 0;
        for (int base = 0; base < p.a.n_seqs; base += kThreads) {
            long long sum = total;
            if (p.a.n_seqs > kThreads) {
                mine = cost_of(base + tid);
                excl = block_scan(mine, sum);
            }
            if (x >= before + excl && x < before + excl + mine) {
                scratch[32] = base + tid;
                scratch[33] = before + excl;
            }
            before += sum;
            if (x < before) break;
        }
        __syncthreads();
        g = static_cast<int>(scratch[32]);
        seq0 = scratch[33];
        __syncthreads();
        load_seq(p);
    }
};

template <typename T>
__device__ __forceinline__ void store4(T* dst, float4 v)
{
    if constexpr (sizeof(T) == 2) {
        // the result's one rounding to bf16, nearest even
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
        *reinterpret_cast<float4*>(dst) = v;
    }
}

// Weight of a partial with maximum m and denominator l against the common maximum M.  A
// partial that saw no key has l = 0 and weight 0; one whose scores are all NaN has
// m = -inf and l = NaN, and passes its NaN on.
__device__ __forceinline__ float part_weight(float m, float l, float M)
{
    if (m == -INFINITY) return l == 0.f ? 0.f : 1.f;
    return ex2(m - M);
}

// Output row of packed row r of a segment.
__device__ __forceinline__ long long out_row(const PagedParams& p, const Segment& t, int r)
{
    const int pr = t.row0 + r, tok = pr / p.G;
    return static_cast<long long>(t.s.first + tok) * p.a.H + t.hk * p.G + (pr - tok * p.G);
}

template <typename T>
__device__ __forceinline__ void write_row4(const PagedParams& p, const Segment& t, int r, int c4,
                                           float4 o, float M, float L)
{
    const float inv = L == 0.f ? 0.f : 1.f / L;       // a row that saw no key: 0 and -inf
    const long long row = out_row(p, t, r);
    const long long idx = row * p.a.D + 4 * c4;
    if (in_bounds(idx, 4, p.a.out_elems, p.a.status))
        store4(static_cast<T*>(p.a.out) + idx, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (c4 == 0 && p.a.lse != nullptr && in_bounds(row, 1, p.a.lse_elems, p.a.status))
        p.a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPagedLn2;
}

// End of a segment, by the whole block: buf[rows][ldo] holds the CTA's unnormalised sums
// and stat[rows] = (maximum in base-2 units, denominator).  Writes the tile's output, or
// the CTA's partial and, in the last CTA of the tile, the joined output.
template <typename T, int kRows, int kThreads, int kVec4 = 1>
__device__ void finish_segment(const PagedParams& p, const Segment& t, const float* buf, int ldo,
                               const float2* stat, int* flag)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v4 = p.a.D / 4;
    if (t.c_first == t.c_last) {
        for (int i = tid; i < t.rows * v4; i += kThreads) {
            const int r = i / v4, c = i - r * v4;
            write_row4<T>(p, t, r, c, *reinterpret_cast<const float4*>(buf + r * ldo + 4 * c),
                          stat[r].x, stat[r].y);
        }
        __syncthreads();
        return;
    }
    // slot 1: the tile begins in this CTA's part and runs on; slot 0: it began before
    const int c = blockIdx.x;
    auto slot_of = [&](int cta) { return 2 * cta + (cta == t.c_first ? 1 : 0); };
    const long long n_slots = 2ll * p.grid;
    {
        const long long slot = slot_of(c);
        for (int r = tid; r < t.rows; r += kThreads)
            if (in_bounds(slot * kRows + r, 1, n_slots * kRows, p.a.status))
                __stcg(reinterpret_cast<float2*>(p.part_stat) + slot * kRows + r, stat[r]);
        if (t.k1 > t.k0) {
            for (int i = tid; i < t.rows * v4; i += kThreads) {
                const int r = i / v4, cc = i - r * v4;
                const long long at = (slot * kRows + r) * p.a.D + 4 * cc;
                if (in_bounds(at, 4, n_slots * kRows * p.a.D, p.a.status))
                    __stcg(reinterpret_cast<float4*>(p.part_o + at),
                           *reinterpret_cast<const float4*>(buf + r * ldo + 4 * cc));
            }
        }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const unsigned n = static_cast<unsigned>(t.c_last - t.c_first + 1);
        int last = 0;
        if (in_bounds(t.c_first, 1, kPagedMaxCtas, p.a.status)) {
            last = atomicAdd(p.counters + t.c_first, 1u) == n - 1;
            if (last) p.counters[t.c_first] = 0;       // as the next call expects it
        }
        *flag = last;
    }
    __syncthreads();
    if (*flag) {
        __threadfence();
        const int nc = t.c_last - t.c_first + 1;
        // kVec4 float4 per lane: D <= 128 kVec4
        for (int r = warp; r < t.rows; r += kThreads / 32) {
            auto stat_at = [&](int i) -> float2 {
                const long long at = static_cast<long long>(slot_of(t.c_first + i)) * kRows + r;
                if (i >= nc || !in_bounds(at, 1, n_slots * kRows, p.a.status))
                    return make_float2(-INFINITY, 0.f);
                return __ldcg(reinterpret_cast<const float2*>(p.part_stat) + at);
            };
            const float2 mine = stat_at(lane);             // of the first 32 contributors
            float M = mine.x;
            for (int i0 = 32; i0 < nc; i0 += 32) M = fmaxf(M, stat_at(i0 + lane).x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            float L = 0.f;
            float4 acc[kVec4];
#pragma unroll
            for (int u = 0; u < kVec4; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int i0 = 0; i0 < nc; i0 += 32) {
                const float2 st = i0 == 0 ? mine : stat_at(i0 + lane);
                const float w = part_weight(st.x, st.y, M);
                L += st.y == 0.f ? 0.f : w * st.y;
                const unsigned have = __ballot_sync(0xffffffffu, !(st.y == 0.f));
                const int cnt = min(32, nc - i0);
                // eight contributors' sums in flight; an empty one wrote none
#pragma unroll 1
                for (int i = 0; i < cnt; i += 8) {
                    float4 o[8][kVec4];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const long long at =
                            (static_cast<long long>(slot_of(t.c_first + i0 + i + e)) * kRows + r) * p.a.D;
#pragma unroll
                        for (int u = 0; u < kVec4; ++u) {
                            const int cc = lane + 32 * u;
                            o[e][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (i + e < cnt && ((have >> (i + e)) & 1) && cc < v4 &&
                                in_bounds(at + 4 * cc, 4, n_slots * kRows * p.a.D, p.a.status))
                                o[e][u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at + 4 * cc));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float wi = __shfl_sync(0xffffffffu, w, (i + e) & 31);
#pragma unroll
                        for (int u = 0; u < kVec4; ++u) {
                            acc[u].x = fmaf(wi, o[e][u].x, acc[u].x);
                            acc[u].y = fmaf(wi, o[e][u].y, acc[u].y);
                            acc[u].z = fmaf(wi, o[e][u].z, acc[u].z);
                            acc[u].w = fmaf(wi, o[e][u].w, acc[u].w);
                        }
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
            for (int u = 0; u < kVec4; ++u)
                if (lane + 32 * u < v4) write_row4<T>(p, t, r, lane + 32 * u, acc[u], M, L);
        }
    }
    __syncthreads();
}

// Element offset of key `key` of head hk of a sequence in the pages, or -1 (a page index
// outside the cache: the key and its value read as zeros).
__device__ __forceinline__ long long key_offset(const PagedParams& p, int g, int hk, int key)
{
    const PagedArgs& a = p.a;
    const int col = p.page_shift >= 0 ? key >> p.page_shift : key / a.page_size;
    const int page = checked_ldg(a.page_table, g * a.table_stride + col, a.table_elems, a.status);
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) return -1;
    return page * a.page_stride + (key - col * a.page_size) * a.token_stride + hk * a.head_stride;
}

}  // namespace ra
