// paged_plan.cuh -- how the kernels of paged_attn_fwd share out their work, and how the
// pieces of a row's softmax that different CTAs computed are joined.
//
// A tile is the query rows of one key/value head that one CTA holds at a time: the new
// tokens of a sequence times the H / H_kv query heads that read the head, packed
// token-major ("packed row" r is token r / G, head r % G of the group).  The tiles of a
// call are laid end to end, sequence by sequence, head by head, on one axis of cost, each
// tile as long as its fixed cost and its keys times a weight, and CTA c takes the part
// [c chunk, (c + 1) chunk) of that axis: whatever the lengths are, the CTAs' parts are equal up
// to one tile of at most PagedParams::whole, which is never cut, and one token over a long cache
// fills the whole GPU.  Everything is computed from the lengths on the device, by each warp that
// needs it (a scan over the sequences), so a captured call follows the lengths that it finds when
// it is replayed.
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
constexpr long long kMostKeys = 0x7fffffffll - 1023;

// Kernel-side copy of PagedArgs, with the split.
struct PagedParams {
    PagedArgs a;
    int G;                  // query heads per key/value head
    int grid;
    int min_chunk;          // smallest part worth a CTA, in cost
    int join_cost;          // of joining one more partial of a tile
    int snap;               // shortest piece of a cut tile, in keys
    int whole;              // tiles of up to this cost are never cut
    int tile_cost;          // a tile's fixed cost (its queries and output)
    int key_shift;          // log2 of a key's cost
    int key_shift_single;   // StepTiles: the same in a tile with one sub-tile of rows
    int key_cost, key_cost_single;      // WeighedTiles: a key's cost itself
    int tile_tokens;        // new tokens of a tile (StepTiles)
    int page_shift;         // log2 of the page size, or -1
    int box_rows;           // keys of one tensor-map box (tensor-core kernel)
    unsigned g_magic;       // division by G: see token_of
    int g_shift;
    // r / G of a packed row (r < 2^31), by multiplication
    __device__ __forceinline__ int token_of(int r) const
    {
        return static_cast<int>((__umulhi(static_cast<unsigned>(r), g_magic) + r) >> g_shift);
    }
    float scale_log2;       // log2(e) / sqrt(D): scores in base-2 units
    unsigned int* counters; // [kPagedMaxCtas], zero between calls
    float* part_stat;       // [2 grid][rows of a tile][2]: maximum, denominator
    float* part_o;          // [2 grid][rows of a tile][D]
};

// The workspace, in bytes: work counters, then the statistics and sums of two partial tiles
// for every CTA.
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

// The parts of the parameters that every kernel fills alike.
inline void fill_params(PagedParams* p, const PagedArgs& a)
{
    p->a = a;
    p->G = a.H / a.H_kv;
    int k = 0;
    while ((1ll << k) < a.page_size) ++k;
    p->page_shift = (1ll << k) == a.page_size ? k : -1;
    // ceil(2^(32 + s) / G) - 2^32 with 2^s >= G: r / G = (r + hi(r magic)) >> s exactly for
    // r < 2^31 (the sum does not overflow, and the error r e / (G 2^(32 + s)), e < G <= 2^s,
    // stays below 1 / G)
    int s = 0;
    while ((1ll << s) < p->G) ++s;
    p->g_shift = s;
    p->g_magic = static_cast<unsigned>((((1ull << s) - p->G) << 32) / p->G + 1);
    p->scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(a.D));
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
    // (kMostKeys: key indices plus a step of the kernels stay below 2^31)
    const long long cap = min(static_cast<long long>(a.max_pages) * a.page_size, kMostKeys);
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
// counts all the keys: sequences with few new tokens see nearly all in every tile.  (Of a causal
// prompt that goes this way the first tiles see few of the keys that they are priced at, and
// the split is that uneven.)
template <int kRows>
struct FlatTiles {
    static constexpr bool kLongest = true;
    __device__ __forceinline__ static long long keys_of(long long cost, int shift) { return cost >> shift; }
    int n_tiles;
    long long cost;         // of one tile
    __device__ __forceinline__ static int rows(const PagedParams&) { return kRows; }
    __device__ __forceinline__ void init(const PagedParams& p, const SeqSpan& s)
    {
        n_tiles = (s.n * p.G + kRows - 1) / kRows;        // n G <= T H < 2^31 - 16
        cost = p.tile_cost + (static_cast<long long>(s.kv) << p.key_shift);
    }
    __device__ __forceinline__ long long prefix(int j) const { return j * cost; }
    __device__ __forceinline__ int at(long long x) const { return static_cast<int>(quotient(x, cost)); }
    __device__ __forceinline__ int shift(const PagedParams& p, int) const { return p.key_shift; }
};

// The same where a sequence may have many tiles: under the causal rule tile j of `per` tokens
// sees (up to) the keys before the new tokens and the first (j + 1) per of those, so a
// sequence's costs form an arithmetic series, summed in closed form and searched by halving.
// Its last tile may have one sub-tile of rows only, whose keys cost less.
//
// kWeighed: keys cost what key_cost and key_cost_single say, not powers of two.
template <bool kWeighed>
struct StepTilesOf {
    static constexpr bool kLongest = false;
    // the cost of keys of weight w, and the keys that a cost pays for
    __device__ __forceinline__ static long long cost_of(long long keys, int w)
    {
        return kWeighed ? keys * w : keys << w;
    }
    __device__ __forceinline__ static long long keys_of(long long cost, int w)
    {
        return kWeighed ? quotient(cost, w) : cost >> w;
    }
    int n_tiles, per, fixed, wide, last_shift;
    long long seen, last_keys;      // keys of tile j < n_tiles - 1: seen + j step; of the last
    int step;
    __device__ __forceinline__ static int rows(const PagedParams& p) { return p.tile_tokens * p.G; }
    __device__ __forceinline__ void init(const PagedParams& p, const SeqSpan& s)
    {
        per = p.tile_tokens;
        n_tiles = (s.n + per - 1) / per;
        fixed = p.tile_cost;
        wide = kWeighed ? p.key_cost : p.key_shift;
        const long long before = max(s.kv - s.n, 0);
        step = p.a.causal ? per : 0;
        seen = p.a.causal ? before + per : s.kv;
        last_keys = p.a.causal ? before + s.n : s.kv;
        last_shift = 2 * (s.n - (n_tiles - 1) * per) > per ? wide
                     : kWeighed                            ? p.key_cost_single
                                                           : p.key_shift_single;
    }
    __device__ __forceinline__ long long prefix(int j) const
    {
        if (n_tiles == 0) return 0;
        const long long full = j < n_tiles ? j : n_tiles - 1;
        const long long keys = full * seen + step * (full * (full - 1) / 2);
        const long long c = static_cast<long long>(j) * fixed + cost_of(keys, wide);
        return j < n_tiles ? c : c + cost_of(last_keys, last_shift);
    }
    __device__ __forceinline__ int at(long long x) const
    {
        int lo = 0, hi = n_tiles;               // prefix(lo) <= x < prefix(hi)
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix(mid) <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    __device__ __forceinline__ int shift(const PagedParams&, int j) const
    {
        return j + 1 < n_tiles ? wide : last_shift;
    }
};

using StepTiles = StepTilesOf<false>;
using WeighedTiles = StepTilesOf<true>;

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

    __device__ __forceinline__ void take_seq(const PagedParams& p)
    {
        tiles.init(p, s);
        head_cost = tiles.prefix(tiles.n_tiles);
        seq_cost = head_cost * p.a.H_kv;
    }
    // Keys before the cut at offset x of a tile that has `keys` keys of weight `shift`: whole
    // steps of the kernel, and no piece at either end shorter than `snap` keys (a piece costs a
    // partial result and its share of the joining).
    __device__ __forceinline__ static int cut(long long x, int keys, int fixed, int shift, int snap)
    {
        const long long k = x - fixed;
        if (k <= 0) return 0;
        const long long n = Tiles::keys_of(k, shift) & -static_cast<long long>(kUnit);
        static_assert((kUnit & (kUnit - 1)) == 0, "cuts at a power of two");
        if (n < snap) return 0;
        return n > keys - snap ? keys : static_cast<int>(n);
    }
    __device__ __forceinline__ bool next(const PagedParams& p, Segment& t)
    {
#pragma unroll 1
        while (x < end) {
            while (x >= seq0 + seq_cost) {
                seq0 += seq_cost;
                if (++g >= p.a.n_seqs) return false;
                s = seq_span_of(p.a, g);
                take_seq(p);
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
            const int last = p.token_of(t.row0 + t.rows - 1);
            t.keys = p.a.causal ? min(max(s.kv - s.n + last + 1, 0), s.kv) : s.kv;
            const int shift = tiles.shift(p, j);
            const int c = blockIdx.x;
            if (!Tiles::kLongest && b - a <= p.whole) {
                // never cut: the tile of the CTA whose part holds its middle
                t.c_first = t.c_last = static_cast<int>(quotient(a + ((b - a) >> 1), chunk));
                t.k0 = 0;
                t.k1 = t.keys;
                x = min(end, b);
                if (c == t.c_first) return true;
                continue;
            }
            const int snap = Tiles::kLongest && b - a <= p.whole
                                 ? t.keys / 2 + 1               // not cut
                                 : static_cast<int>(min(static_cast<long long>(p.snap),
                                                        Tiles::keys_of(chunk, shift) >> 2));
            // The CTAs that touch the tile, without the first and the last of them where their
            // piece has no keys; the first keeps a tile without keys.  Others can have none
            // too (a part inside the fixed cost, and with FlatTiles the parts behind the last
            // key that a causal tile sees): they contribute a partial of weight 0.
            t.c_first = a >= c * chunk ? c : static_cast<int>(quotient(a, chunk));
            t.c_last = b <= (c + 1) * chunk ? c : static_cast<int>(quotient(b - 1, chunk));
            auto before = [&](int cta) -> int {             // keys before that CTA's part
                return cta <= t.c_first ? 0
                       : cta > t.c_last ? t.keys
                                        : cut(cta * chunk - a, t.keys, p.tile_cost, shift, snap);
            };
            t.k0 = before(c);
            t.k1 = before(c + 1);
            const int first = t.c_first, top = t.c_last;
            const bool first_empty = first < top && before(first + 1) == 0 && t.keys > 0;
            const bool last_empty = first < top && (before(top) == t.keys || t.keys == 0);
            if (first_empty) ++t.c_first;
            if (last_empty && t.c_last > t.c_first) --t.c_last;
            x = min(end, b);
            if (t.keys == 0) t.c_last = t.c_first;
            if (c >= t.c_first && c <= t.c_last) return true;
        }
        return false;
    }
    // The start of this CTA's part, found by each warp for itself: a lane sums the costs of
    // its share of the sequences, a scan over the lanes tells whose share holds the start,
    // and that lane looks for the sequence.
    __device__ void begin(const PagedParams& p)
    {
        const int lane = threadIdx.x & 31;
        SeqSpan mine{0, 0, 0};      // the last sequence this lane looked at
        int longest = 0;            // keys of a sequence with new tokens
        float n_tiles = 0.f;
        auto cost_of = [&](int i) -> long long {
            mine = seq_span_of(p.a, i);
            Tiles t;
            t.init(p, mine);
            if (Tiles::kLongest) longest = mine.n > 0 ? max(longest, mine.kv) : longest;
            else n_tiles += static_cast<float>(t.n_tiles) * p.a.H_kv;
            return t.prefix(t.n_tiles) * p.a.H_kv;
        };
        const int per = (p.a.n_seqs + 31) / 32;
        const int first = min(lane * per, p.a.n_seqs), stop = min(first + per, p.a.n_seqs);
        long long sum = 0;
#pragma unroll 2
        for (int i = first; i < stop; ++i) sum += cost_of(i);
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const long long total = __shfl_sync(0xffffffffu, inc, 31);
        // A tile of cost t in parts of x takes x for the parts, which run side by side, and
        // join_cost t / x for joining them, one after the other: least at x = sqrt(join_cost t).
        // A part need not be longer than a tile, though (26 sequences of 3 tokens and keys
        // 9.2 us, 13 with parts of a fixed least length, which hold a tile and a half).
        long long least;
        if constexpr (Tiles::kLongest) {
            // the longest tile's t, since the call ends with it (one token of 8 heads that share
            // a key head, 40000 keys: 26 us, and 63 in as many parts as there are CTAs)
            longest = __reduce_max_sync(0xffffffffu, longest);
            const float tile = static_cast<float>(longest) * static_cast<float>(p.join_cost << p.key_shift);
            least = p.tile_cost + (static_cast<long long>(longest) << p.key_shift);
            if (least > p.whole)
                least = min(least, static_cast<long long>(max(p.min_chunk, static_cast<int>(sqrtf(tile)))));
        } else {
            // the mean tile's (of tiles that stay whole three quarters, so that two a little
            // shorter than the mean do not fall to one CTA while another has none)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) n_tiles += __shfl_xor_sync(0xffffffffu, n_tiles, o);
            const float tile = static_cast<float>(total) / fmaxf(n_tiles, 1.f);
            const float part = fmaxf(sqrtf(tile * static_cast<float>(p.join_cost)),
                                     static_cast<float>(p.min_chunk));
            least = static_cast<long long>(
                tile <= static_cast<float>(p.whole) ? 0.75f * tile : fminf(part, tile + 1.f));
        }
        chunk = max(quotient(total + p.grid - 1, p.grid), least);
        x = blockIdx.x * chunk;
        end = min(total, x + chunk);
        g = 0;
        seq0 = 0;
        if (x >= total) {
            x = end;                // nothing for this CTA
            return;
        }
        long long at = inc - sum;
        int i = first;
        const bool holds = at <= x && x < inc;
        if (holds && per > 1) {
#pragma unroll 1
            for (;; ++i) {
                const long long c = cost_of(i);
                if (x < at + c || i == stop - 1) break;
                at += c;
            }
        }
        const int owner = __ffs(__ballot_sync(0xffffffffu, holds)) - 1;
        g = __shfl_sync(0xffffffffu, i, owner);
        seq0 = __shfl_sync(0xffffffffu, at, owner);
        s.first = __shfl_sync(0xffffffffu, mine.first, owner);
        s.n = __shfl_sync(0xffffffffu, mine.n, owner);
        s.kv = __shfl_sync(0xffffffffu, mine.kv, owner);
        take_seq(p);
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
    const float none = l == 0.f ? 0.f : 1.f;
    return m == -INFINITY ? none : ex2(m - M);
}

// The rows of one tile, as far as its output needs them.
struct TileRows {
    int first, row0, rows, hk;      // the sequence's first token row; packed rows; head
    int c_first, c_last;            // the CTAs that share the tile
};

// Output row of packed row r of a tile.
__device__ __forceinline__ long long out_row(const PagedParams& p, const TileRows& t, int r)
{
    const int pr = t.row0 + r, tok = p.token_of(pr);
    return static_cast<long long>(t.first + tok) * p.a.H + t.hk * p.G + (pr - tok * p.G);
}

// 1 / L and the log-sum-exp of a row with maximum M (base 2) and denominator L; 0 and -inf
// for a row that saw no key.  (The approximate reciprocal and logarithm are good to an ulp and
// to 2^-22; their exact forms' branches cost the joining loop below more than its reads.)
__device__ __forceinline__ float inverse_of(float L) { return L == 0.f ? 0.f : __fdividef(1.f, L); }
__device__ __forceinline__ float lse_of(float M, float L)
{
    return L == 0.f ? -INFINITY : (M + __log2f(L)) * kPagedLn2;
}

template <typename T>
__device__ __forceinline__ void write_row4(const PagedParams& p, const TileRows& t, int r, int c4,
                                           float4 o, float M, float L)
{
    const float inv = inverse_of(L), lse = lse_of(M, L);
    const long long row = out_row(p, t, r);
    const long long idx = row * p.a.D + 4 * c4;
    if (in_bounds(idx, 4, p.a.out_elems, p.a.status))
        store4(static_cast<T*>(p.a.out) + idx, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (c4 == 0 && p.a.lse != nullptr && in_bounds(row, 1, p.a.lse_elems, p.a.status))
        p.a.lse[row] = lse;
}

// Where CTA `cta` keeps its partial of tile t: slot 1 if the tile begins in its part and
// runs on, slot 0 if it began before.
__device__ __forceinline__ long long part_slot(const TileRows& t, int cta)
{
    return 2ll * cta + (cta == t.c_first ? 1 : 0);
}

// Counts this CTA in as a contributor of tile t (one thread, the CTA's partial being written
// and ordered before by a barrier); true in the last one.
__device__ __forceinline__ bool arrive_last(const PagedParams& p, const TileRows& t)
{
    if (!in_bounds(t.c_first, 1, kPagedMaxCtas, p.a.status)) return false;
    // releases what the barrier before ordered, the whole CTA's partial, and acquires the others'
    unsigned before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                 : "=r"(before)
                 : "l"(p.counters + t.c_first)
                 : "memory");
    const bool last = before == static_cast<unsigned>(t.c_last - t.c_first);
    if (last) p.counters[t.c_first] = 0;               // as the next call expects it
    return last;
}

// The tile's output from all contributors' partials, joined one after the other in CTA order
// (the running maximum and sum of the softmax once more), by warp `warp` of n_warps.  kLanes
// lanes share a row (four columns each, and kVec4 times that); kRowsAt times 32 / kLanes rows
// and kDeep contributors are read at once: a read takes a microsecond while the rest of the
// GPU streams.  slot_rows: rows a partial slot has; place(r): the row of a slot that holds
// packed row r.
template <typename T, int kLanes, int kVec4, int kRowsAt, int kDeep, typename Place>
__device__ void join_rows(const PagedParams& p, const TileRows& t, int warp, int n_warps,
                          int slot_rows, Place place)
{
    constexpr int kAbreast = 32 / kLanes;
    const int lane = threadIdx.x & 31, col = lane % kLanes;
    const int step = n_warps * kAbreast;
    const int D = p.a.D;
    const int nc = t.c_last - t.c_first + 1;
    const unsigned all_rows = 2u * p.grid * slot_rows;
    // columns of this lane: four at 4 (col + kLanes u), or none
    int at_col[kVec4];
#pragma unroll
    for (int u = 0; u < kVec4; ++u) {
        const int c = 4 * (col + kLanes * u);
        at_col[u] = c < D ? c : -1;
    }
#pragma unroll 1
    for (int r0 = warp * kAbreast + lane / kLanes; r0 - lane / kLanes < t.rows; r0 += step * kRowsAt) {
        float M[kRowsAt], L[kRowsAt];
        float4 acc[kRowsAt][kVec4];
        unsigned at0[kRowsAt];                         // row of contributor 0 if it had slot 0
#pragma unroll
        for (int b = 0; b < kRowsAt; ++b) {
            M[b] = -INFINITY;
            L[b] = 0.f;
            // (rows behind the last one repeat it and are not written)
            at0[b] = 2u * t.c_first * slot_rows + place(min(r0 + b * step, t.rows - 1));
#pragma unroll
            for (int u = 0; u < kVec4; ++u) acc[b][u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int k = 0; k < nc; k += kDeep) {
            float2 st[kDeep][kRowsAt];
            float4 o[kDeep][kRowsAt][kVec4];
            // all reads first, under no condition but the contributors' number
#pragma unroll
            for (int e = 0; e < kDeep; ++e) {
                // contributor 0 has slot 1 of its CTA, the others slot 0 of theirs
                const bool real = k + e < nc;
                const unsigned slot = (k + e == 0 ? 1u : 2u * (k + e)) * slot_rows;
#pragma unroll
                for (int b = 0; b < kRowsAt; ++b) {
                    const unsigned at = at0[b] + slot;
                    const bool in = real && in_bounds(at, 1, all_rows, p.a.status);
                    st[e][b] = make_float2(-INFINITY, 0.f);
                    if (in) st[e][b] = __ldcg(reinterpret_cast<const float2*>(p.part_stat) + at);
                    const float* src = p.part_o + static_cast<unsigned long long>(at) * D;
#pragma unroll
                    for (int u = 0; u < kVec4; ++u) {
                        o[e][b][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (in)
                            o[e][b][u] = __ldcg(reinterpret_cast<const float4*>(src + max(at_col[u], 0)));
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kRowsAt; ++b) {
                float Mn = M[b];
#pragma unroll
                for (int e = 0; e < kDeep; ++e) Mn = fmaxf(Mn, st[e][b].x);
                const float old = part_weight(M[b], L[b], Mn);
                M[b] = Mn;
                L[b] *= old;
#pragma unroll
                for (int u = 0; u < kVec4; ++u) {
                    acc[b][u].x *= old;
                    acc[b][u].y *= old;
                    acc[b][u].z *= old;
                    acc[b][u].w *= old;
                }
#pragma unroll
                for (int e = 0; e < kDeep; ++e) {
                    const float2 x = st[e][b];
                    const float w = part_weight(x.x, x.y, Mn);
                    L[b] = fmaf(w, x.y, L[b]);
#pragma unroll
                    for (int u = 0; u < kVec4; ++u) {
                        acc[b][u].x = fmaf(w, o[e][b][u].x, acc[b][u].x);
                        acc[b][u].y = fmaf(w, o[e][b][u].y, acc[b][u].y);
                        acc[b][u].z = fmaf(w, o[e][b][u].z, acc[b][u].z);
                        acc[b][u].w = fmaf(w, o[e][b][u].w, acc[b][u].w);
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < kRowsAt; ++b) {
            const int r = r0 + b * step;
            if (r >= t.rows) continue;
#pragma unroll
            for (int u = 0; u < kVec4; ++u)
                if (at_col[u] >= 0) write_row4<T>(p, t, r, col + kLanes * u, acc[b][u], M[b], L[b]);
        }
    }
}

// End of a segment, by the whole block: buf[rows][ldo] holds the CTA's unnormalised sums
// and stat[rows] = (maximum in base-2 units, denominator).  Writes the tile's output, or
// the CTA's partial and, in the last CTA of the tile, the joined output.
template <typename T, int kRows, int kThreads, int kVec4 = 1>
__device__ void finish_segment(const PagedParams& p, const Segment& seg, const float* buf, int ldo,
                               const float2* stat, int* flag)
{
    const TileRows t{seg.s.first, seg.row0, seg.rows, seg.hk, seg.c_first, seg.c_last};
    const int tid = threadIdx.x;
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
    const long long all_rows = 2ll * p.grid * kRows;
    const long long at0 = part_slot(t, blockIdx.x) * kRows;
    for (int r = tid; r < t.rows; r += kThreads)
        if (in_bounds(at0 + r, 1, all_rows, p.a.status))
            __stcg(reinterpret_cast<float2*>(p.part_stat) + at0 + r, stat[r]);
    for (int i = tid; i < t.rows * v4; i += kThreads) {        // (zeros if it saw no key)
        const int r = i / v4, cc = i - r * v4;
        const long long at = (at0 + r) * p.a.D + 4 * cc;
        if (in_bounds(at, 4, all_rows * p.a.D, p.a.status))
            __stcg(reinterpret_cast<float4*>(p.part_o + at),
                   *reinterpret_cast<const float4*>(buf + r * ldo + 4 * cc));
    }
    __syncthreads();
    if (tid == 0) *flag = arrive_last(p, t);
    __syncthreads();
    if (*flag)
        join_rows<T, 32, kVec4, kRows >= 64 ? 8 / kVec4 : 1, kRows >= 64 ? 2 : 8>(
            p, t, tid >> 5, kThreads / 32, kRows, [](int r) { return r; });
    __syncthreads();
}

// Trees of drafted tokens (a.masks): which of the new tokens node .. node + 31 of its sequence a
// row sees, a bit each; what lies before node 0 are keys from before the step, which all rows see.
// row: its index in the call.
__device__ __forceinline__ unsigned seen_from(const PagedParams& p, int row, int node)
{
    const PagedArgs& a = p.a;
    auto word = [&](int w) -> unsigned {
        if (w >= a.mask_words) return 0u;
        return static_cast<unsigned>(checked_ldg(a.masks, row * a.mask_stride + w, a.mask_elems, a.status));
    };
    if (node <= -32) return 0xffffffffu;
    if (node < 0) return word(0) << -node | ((1u << -node) - 1);
    return __funnelshift_r(word(node >> 5), word((node >> 5) + 1), node & 31);
}

// Asynchronous 16-byte copies into shared memory.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real)
{
    const int n = real ? 16 : 0;                              // 0: the 16 bytes become zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
