// rope.cu -- rotary positions (rope_fwd, rope_bwd) and the paged key/value append that
// rotates on the way (paged_kv_append), as one HBM stream.
//
// A rotated head vector of `rot` leading dims forms rot/2 pairs -- (x[i], x[i + rot/2]) in
// the half style, (x[2i], x[2i + 1]) in the interleaved one -- and pair i of a token at
// position p turns by the angle t = p f_i:
//   y_a = A (x_a cos t - x_b sin t),   y_b = A (x_b cos t + x_a sin t),
// A being the amplitude of the scaling.  The backward is the transpose: the same with
// sin t negated.  The dims behind `rot` pass through.
//
// Angles.  p f_i loses its low bits in fp32 once p is in the thousands (at p = 10^6 an
// angle is known to 0.06 rad), and fp64 arithmetic is slow here, so the frequencies come
// as 64-bit fixed-point fractions of a turn: phase_i = f_i / (2 pi) 2^64.  p phase_i
// modulo 2^64 is then the angle modulo a turn, exactly, in one integer product for any
// position (negative ones too); its upper 32 bits, taken as a signed number, are the
// angle in (-pi, pi] and go through sincospif.
//
// What bounds it: every element is read and written once, so the copy bandwidth.  A block
// takes a few tokens.  Its threads first send for the rows they will rotate first, then work
// out the tokens' positions and their tokens * rot/2 sines and cosines, once for all heads,
// in shared memory, and then stream the tokens' heads, two rows in flight each.  A thread
// keeps one item of a head vector -- a 16-byte vector of each half of the pairs, or a vector of
// the dims behind `rot` (half style), or two vectors of whole pairs (interleaved) -- and walks
// over the tokens, so that only its pointers move.  In the half style a rot/2 that is no
// multiple of the vector takes pieces of half of one, or rope_shift_kernel below.
// Measured: 32768 tokens of 64 heads of 128 dims in bf16 in 161 to 164 us, 6.5 to 6.7 TB/s
// (the measured copy rate is 6.69); before the items kept their columns and the sines lay
// where neighbouring lanes read them side by side it was 214 us, bound by instructions.

#include <cuda_bf16.h>

#include "rope_pos.cuh"

namespace ra {
namespace {

constexpr int kMaxBlock = 512;
constexpr int kMaxPairs = 2048;     // sines and cosines of one block: tokens * rot / 2
constexpr int kMaxTokens = 32;
constexpr int kAhead = 2;           // rows in flight per thread

// (ya, yb) of two pairs at once: xa c - xb s, xb c + xa s.
__device__ __forceinline__ void turn2(uint64_t xa, uint64_t xb, uint64_t c, uint64_t s, uint64_t& ya,
                                      uint64_t& yb)
{
    constexpr uint64_t kSigns = 0x8000000080000000ull;
    ya = ffma2(xa, c, fmul2(xb, s ^ kSigns));
    yb = ffma2(xb, c, fmul2(xa, s));
}

// A piece of N elements, moved in one access.
template <typename T, int N>
struct alignas(N * sizeof(T)) Piece {
    T e[N];
};

// Rotates an item: pieces x0, x1 of N pairs' first and second elements (half style), or x0 with
// N / 2 whole pairs, the first `pairs` of which turn (interleaved).  cs, sn: the item's cosines
// and sines in groups of kGroup, `step` floats apart.
template <typename T, bool kHalfStyle, int N, int kGroup>
__device__ __forceinline__ void rotate_item(Piece<T, N>& x0, Piece<T, N>& x1, const float* cs,
                                            const float* sn, int step, int pairs)
{
    using Floats = Piece<float, kGroup>;
    constexpr int kPairs = kHalfStyle ? N : N / 2;
#pragma unroll
    for (int g = 0; g < kPairs / kGroup; ++g) {
        const Floats c = *reinterpret_cast<const Floats*>(cs + g * step);
        const Floats s = *reinterpret_cast<const Floats*>(sn + g * step);
        if constexpr (kHalfStyle && sizeof(T) == 2 && kGroup >= 2) {
            uint32_t* a = reinterpret_cast<uint32_t*>(&x0.e[g * kGroup]);
            uint32_t* b = reinterpret_cast<uint32_t*>(&x1.e[g * kGroup]);
#pragma unroll
            for (int i = 0; i < kGroup / 2; ++i) {
                uint64_t ya, yb;
                turn2(unpack2(a[i]), unpack2(b[i]), f2pack(c.e[2 * i], c.e[2 * i + 1]),
                      f2pack(s.e[2 * i], s.e[2 * i + 1]), ya, yb);
                a[i] = pack2(ya);
                b[i] = pack2(yb);
            }
        } else if constexpr (!kHalfStyle && sizeof(T) == 2) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&x0.e[2 * g * kGroup]);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const float xa = __uint_as_float(w[i] << 16), xb = __uint_as_float(w[i] & 0xffff0000u);
                const uint32_t y = pack_bf16x2(fmaf(xa, c.e[i], -(xb * s.e[i])),
                                               fmaf(xb, c.e[i], xa * s.e[i]));
                w[i] = g * kGroup + i < pairs ? y : w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const int j = g * kGroup + i;
                T& ea = kHalfStyle ? x0.e[j] : x0.e[(2 * j) % N];
                T& eb = kHalfStyle ? x1.e[j] : x0.e[(2 * j + 1) % N];
                const float xa = to_f(ea), xb = to_f(eb);
                const T ya = from_f<T>(fmaf(xa, c.e[i], -(xb * s.e[i])));
                const T yb = from_f<T>(fmaf(xb, c.e[i], xa * s.e[i]));
                if (kHalfStyle || j < pairs) {
                    ea = ya;
                    eb = yb;
                }
            }
        }
    }
}

// How a head vector is shared out.  Half style: the rotating items are a piece of each half,
// the others a piece behind `rot`.  Interleaved: item i of `all` is vectors i and i + all of
// the `rotating` = D / N vectors of the head, of which each turns what lies before `rot`.
// Measured with two vectors an item and with one: 8191 tokens of 16 heads of 96 in fp32 19.8 us
// and 22.3, 1458 of 32 heads of 80 in bf16 5.2 and 6.5; single tokens 3.1 and 3.0.
struct RopeItems {
    int rotating, all;
};
template <bool kHalfStyle, int N>
__host__ __device__ __forceinline__ RopeItems items_of(const RopeArgs& a)
{
    if (kHalfStyle) return {a.rot / 2 / N, a.rot / 2 / N + (a.D - a.rot) / N};
    return {a.D / N, (a.D / N + 1) / 2};
}

// N: elements of a piece (a 16-byte vector, or in the half style half of one where half of `rot`
// is no multiple of that).  kPaged: the heads are q's (to q_out), k's (rotated, to the pages)
// and v's (to the pages).
template <typename T, bool kHalfStyle, int N, bool kPaged>
__global__ void __launch_bounds__(kMaxBlock) rope_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int kPairs = kHalfStyle ? N : N / 2;
    // sines and cosines lie in groups of kGroup (what one read of an item takes), group g of
    // an item behind group g of all items before it, so that neighbouring lanes read
    // neighbouring groups
    constexpr int kGroup = kPairs < 4 ? kPairs : 4;
    using Vec = Piece<T, N>;

    __shared__ alignas(16) float cos_s[kMaxPairs];
    __shared__ alignas(16) float sin_s[kMaxPairs];
    __shared__ TokenPos tok_s[kMaxTokens];

    const int half = a.rot / 2;
    const RopeItems it = items_of<kHalfStyle, N>(a);
    const int rot_items = it.rotating, n_items = it.all;
    const int cs_row = rot_items * kPairs;         // sines and cosines of a token
    const int heads = a.H + (kPaged ? 2 : 1) * a.H_kv;
    const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
    const int n_tok = static_cast<int>(min(static_cast<long long>(a.tokens), a.rows - t0));

    // A thread keeps its item and takes heads h, h + step_h, ..., of each every step_t-th
    // token: in the inner walk over tokens only the pointers move.
    const int item = threadIdx.x % n_items;
    const int row = threadIdx.x / n_items;
    const int step_t = a.step_t, step_h = a.step_h;
    const int first_tok = row / step_h;
    const bool works = first_tok < step_t;
    const bool rotates = item < rot_items;
    // the item's second piece
    const int apart = kHalfStyle ? half : n_items * N;
    const bool two = kHalfStyle ? rotates : item + n_items < rot_items;
    const int c0 = kHalfStyle && !rotates ? a.rot + (item - rot_items) * N : item * N;

    int h = row - first_tok * step_h, tok = first_tok;
    const T* src = nullptr;
    T* dst = nullptr;                              // (kPaged: of q heads; of the others, the pages)
    long long src_step = 0, dst_step = 0, si = 0, di = 0;
    int kind = 0;                                  // 0 q, 1 k, 2 v
    auto enter = [&]() {                           // head h from its first token on
        kind = h < a.H ? 0 : h < a.H + a.H_kv ? 1 : 2;
        const int hh = h - (kind == 0 ? 0 : kind == 1 ? a.H : a.H + a.H_kv);
        const void* s = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        void* d = kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out;
        src_step = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
        dst_step = kind == 0 ? a.q_out_stride : a.k_out_stride;
        si = (t0 + tok) * src_step + static_cast<long long>(hh) * a.D;
        if (kPaged && kind > 0) {
            di = hh * a.head_stride;
            dst_step = 0;
        } else {
            di = (t0 + tok) * dst_step + static_cast<long long>(hh) * a.D;
            dst_step *= step_t;
        }
        src_step *= step_t;
        src = static_cast<const T*>(s) + si + c0;
        dst = static_cast<T*>(d) + di + c0;
    };
    struct Row {
        Vec x0, x1;             // x1: half style, rotated items
        T* dst;
        long long di;
        int tok, kind;          // tok: n_tok if there is none
    };
    auto fetch = [&](Row& r) {
        r.tok = tok;
        if (tok >= n_tok) return;
        r.kind = kind;
        r.dst = dst;
        r.di = di;
        if (in_bounds(si, a.D, kind == 0 ? a.q_elems : kind == 1 ? a.k_elems : a.v_elems, a.status)) {
            r.x0 = *reinterpret_cast<const Vec*>(src);
            if (two) r.x1 = *reinterpret_cast<const Vec*>(src + apart);
        }
        src += src_step;
        dst += dst_step;
        si += src_step;
        di += dst_step;
        tok += step_t;
        if (tok >= n_tok) {
            h += step_h;
            if (h < heads) {
                tok = first_tok;
                enter();
            }
        }
    };
    auto finish = [&](Row& r) {
        if (r.tok >= n_tok) return;
        const TokenPos p = tok_s[r.tok];
        T* out = r.dst;
        long long at = r.di;
        if (kPaged && r.kind > 0) {
            if (p.slot < 0) return;
            out += p.slot;
            at += p.slot;
        } else if (!p.live) {
            return;
        }
        if (!in_bounds(at, a.D, r.kind == 0 ? a.q_out_elems : a.k_out_elems, a.status)) return;
        // (the paged append's values stay as they are)
        if (rotates && (!kPaged || r.kind < 2)) {
            const int cs = r.tok * cs_row + item * kGroup;
            rotate_item<T, kHalfStyle, N, kGroup>(r.x0, r.x1, cos_s + cs, sin_s + cs,
                                                  rot_items * kGroup, half - item * kPairs);
            if (!kHalfStyle && two) {
                const int cs1 = cs + n_items * kGroup;
                rotate_item<T, kHalfStyle, N, kGroup>(r.x1, r.x0, cos_s + cs1, sin_s + cs1,
                                                      rot_items * kGroup,
                                                      half - (item + n_items) * kPairs);
            }
        }
        *reinterpret_cast<Vec*>(out) = r.x0;
        if (two) *reinterpret_cast<Vec*>(out + apart) = r.x1;
    };

    wait_for_earlier_work();
    if (!works || h >= heads) tok = n_tok;
    if (tok < n_tok) enter();
    // the first rows are on their way while the positions and angles are worked out
    Row r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(r[u]);

    for (int i = threadIdx.x >> 5; i < n_tok; i += blockDim.x >> 5) {
        const TokenPos p = token_pos<kPaged>(a, t0 + i);
        if ((threadIdx.x & 31) == 0) tok_s[i] = p;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * half; i += blockDim.x) {
        const int tk = i / half, pair = i - tk * half;
        unsigned long long ph = 0;
        if (in_bounds(pair, 1, half, a.status)) ph = __ldg(a.phases + pair);
        float s, c;
        angle_of(ph, tok_s[tk].pos, s, c);
        const int of = pair / kPairs, in = pair % kPairs;
        const int at = tk * cs_row + ((in / kGroup) * rot_items + of) * kGroup + in % kGroup;
        cos_s[at] = c * a.amplitude;
        sin_s[at] = s * a.amplitude * a.sign;
    }
    __syncthreads();

    // a row is written and the one kAhead further fetched in its place
    while (r[0].tok < n_tok) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            finish(r[u]);
            fetch(r[u]);
        }
    }
}

// ---- half style, rot / 2 no multiple of 8 bytes ----
//
// The partners of a vector's elements then straddle two vectors of the row.  A lane takes one
// vector of the row, reads the two that hold its partners behind it (its first-half elements)
// or before it (its second-half ones) -- the same lines, from L1 -- and shifts them into place
// by whole words and half words, `half` modulo the vector's length being the same for all.
// A row's lanes are in one warp, which has read everything before it stores, so rotating in
// place is safe.  Per element: y = x C + partner S, with C and S laid out by element in
// shared memory (S = -sin in the first half, +sin in the second).  What bounds it: the
// instructions, five reads and the shifts per vector.
constexpr int kShiftFloats = 2048;      // cosines of one block: tokens * D

// The kFull elements from element s on of the two vectors a, b.
template <typename T>
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int s)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    constexpr int kWord = 4 / sizeof(T);            // elements of a word
    if (s & (2 * kWord)) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (s & kWord) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (kWord == 2 && (s & 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, bool kPaged>
__global__ void __launch_bounds__(256) rope_shift_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int kFull = 16 / sizeof(T);
    __shared__ alignas(16) float c_s[kShiftFloats];
    __shared__ alignas(16) float s_s[kShiftFloats];
    __shared__ TokenPos tok_s[kMaxTokens];
    const int half = a.rot / 2, D = a.D;
    const int items = D / kFull;                    // at most 32
    const int heads = a.H + (kPaged ? 2 : 1) * a.H_kv;
    const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
    const int n_tok = static_cast<int>(min(static_cast<long long>(a.tokens), a.rows - t0));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;

    wait_for_earlier_work();
    for (int i = warp; i < n_tok; i += n_warps) {
        const TokenPos p = token_pos<kPaged>(a, t0 + i);
        if (lane == 0) tok_s[i] = p;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * half; i += blockDim.x) {
        const int tk = i / half, pair = i - tk * half;
        unsigned long long ph = 0;
        if (in_bounds(pair, 1, half, a.status)) ph = __ldg(a.phases + pair);
        float s, c;
        angle_of(ph, tok_s[tk].pos, s, c);
        c *= a.amplitude;
        s *= a.amplitude * a.sign;
        c_s[tk * D + pair] = c_s[tk * D + half + pair] = c;
        s_s[tk * D + pair] = -s;
        s_s[tk * D + half + pair] = s;
    }
    __syncthreads();

    const int abreast = 32 / items;                 // rows of a warp at a time
    const int sub = lane / items, v = lane - sub * items;
    const bool works = sub < abreast;
    const int rows = n_tok * heads;
    // partners behind the vector start at element e0 + half, those before it at e0 - half
    const int e0 = v * kFull, shift = half % kFull;
    const int behind = v + half / kFull, ahead = v - half / kFull - 1;
    const bool first = e0 < half, second = e0 + kFull > half && e0 < a.rot;
    for (int base = warp * abreast; base < rows; base += n_warps * abreast) {
        const int r = base + sub;
        const bool go = works && r < rows;
        const int tk = go ? r / heads : 0, h = go ? r - tk * heads : 0;
        const int kind = h < a.H ? 0 : h < a.H + a.H_kv ? 1 : 2;
        const int hh = h - (kind == 0 ? 0 : kind == 1 ? a.H : a.H + a.H_kv);
        const long long t = t0 + tk;
        const TokenPos p = tok_s[tk];
        const long long si = t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                             static_cast<long long>(hh) * D;
        const bool to_page = kPaged && kind > 0;
        const long long di = to_page ? p.slot + hh * a.head_stride
                                     : t * (kind == 0 ? a.q_out_stride : a.k_out_stride) +
                                           static_cast<long long>(hh) * D;
        const bool write = go && (to_page ? p.slot >= 0 : p.live) &&
                           in_bounds(si, D, kind == 0 ? a.q_elems : kind == 1 ? a.k_elems : a.v_elems,
                                     a.status) &&
                           in_bounds(di, D, kind == 0 ? a.q_out_elems : a.k_out_elems, a.status);
        uint4 x = make_uint4(0, 0, 0, 0), after = x, before = x;
        if (write) {
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + si);
            x = src[v];
            if (kind < 2 && first)
                after = shifted<T>(src[min(behind, items - 1)], src[min(behind + 1, items - 1)], shift);
            if (kind < 2 && second)
                before = shifted<T>(src[max(ahead, 0)], src[max(ahead + 1, 0)], kFull - shift);
        }
        __syncwarp();
        if (!write) continue;
        if (kind < 2) {
            T* e = reinterpret_cast<T*>(&x);
            const T* pa = reinterpret_cast<const T*>(&after);
            const T* pb = reinterpret_cast<const T*>(&before);
            const float* c = c_s + tk * D + e0;
            const float* s = s_s + tk * D + e0;
#pragma unroll
            for (int g = 0; g < kFull / 4; ++g) {
                const float4 c4 = *reinterpret_cast<const float4*>(c + 4 * g);
                const float4 s4 = *reinterpret_cast<const float4*>(s + 4 * g);
                const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 4 * g + i;
                    const float partner = to_f(e0 + j < half ? pa[j] : pb[j]);
                    const T y = from_f<T>(fmaf(to_f(e[j]), cc[i], partner * ss[i]));
                    if (e0 + j < a.rot) e[j] = y;
                }
            }
        }
        T* out = static_cast<T*>(kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out) + di;
        reinterpret_cast<uint4*>(out)[v] = x;
    }
}

// Tokens of a block, up to `most`: the number whose blocks are done first, taking that the
// blocks go in waves of `slots`, that a block takes as long as kFixed rows of a thread (start,
// first reads, positions) besides its rows and angles, and that the last wave, where it is not
// full, takes as long as a full one.  Measured, against eight blocks per SM whatever the heads
// are: 8191 tokens of 16 heads of 96 in fp32 22 us and 23.6 (one vector an item), 8913 of 20
// heads of 64 (12 pairs, bf16) 17 and 22, 8406 of 2 heads of 80 4.7 and 6.4; large calls the same.
int best_tokens(const RopeArgs& a, int most, int threads, int heads, int half, int slots)
{
    constexpr int kFixed = 3;
    int best = 1;
    long long least = 0;
    for (int t = 1; t <= most; ++t) {
        const long long blocks = (a.rows + t - 1) / t;
        const int rows = (t + a.step_t - 1) / a.step_t * ((heads + a.step_h - 1) / a.step_h);
        const int angles = (t * half + threads - 1) / threads, tokens = (32 * t + threads - 1) / threads;
        // halves of a row
        const long long cost = (blocks + slots - 1) / slots * (2 * (kFixed + rows) + angles + tokens);
        if (t == 1 || cost < least) {
            least = cost;
            best = t;
        }
        if (blocks <= slots) break;                 // one wave: longer blocks take longer
    }
    return best;
}

template <typename T>
cudaError_t launch_shift(RopeArgs& a, int sms)
{
    const int items = a.D / (16 / static_cast<int>(sizeof(T)));
    const int heads = a.H + (a.paged ? 2 : 1) * a.H_kv;
    // a token's heads by whole warps, up to eight
    int warps = (heads + 32 / items - 1) / (32 / items);
    if (warps > 8) warps = 8;
    int most = kShiftFloats / a.D;
    if (most > kMaxTokens) most = kMaxTokens;
    a.step_h = warps * (32 / items);                // rows of a pass
    a.step_t = 1;
    int slots = 0;
    static std::atomic<int> known[2][kMaxDevices];
    const cudaError_t e =
        a.paged ? slots_of(known[1], rope_shift_kernel<T, true>, 32 * warps, sms, &slots)
                : slots_of(known[0], rope_shift_kernel<T, false>, 32 * warps, sms, &slots);
    if (e != cudaSuccess) return e;
    a.tokens = best_tokens(a, most, 32 * warps, heads, a.rot / 2, slots);
    const long long blocks = (a.rows + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(blocks);
    return launch_early(a.paged ? rope_shift_kernel<T, true> : rope_shift_kernel<T, false>, grid,
                        32 * warps, 0, a.stream, a);
}

template <typename T, bool kHalfStyle, int N>
cudaError_t launch(RopeArgs& a, int sms)
{
    constexpr int kPairs = kHalfStyle ? N : N / 2;
    const int half = a.rot / 2, heads = a.H + (a.paged ? 2 : 1) * a.H_kv;
    const RopeItems it = items_of<kHalfStyle, N>(a);
    const int cs_row = it.rotating * kPairs, items = it.all;      // at most 256 items
    // Threads: a token's heads in equal parts of at most 256 threads, so that no part runs
    // with idle rows, or several tokens of few heads at once.  Measured: 48 heads of 8 items
    // (15,000 tokens appended) take 61 us in two parts of 24 rows; 68 in one of 48 (fewer
    // blocks per SM), 73 to 79 in parts of 32 and 16.
    if (heads * items <= 128) {
        a.step_h = heads;
        a.step_t = 256 / (heads * items);
        if (a.step_t > kMaxTokens) a.step_t = kMaxTokens;
    } else {
        const int parts = (heads * items + 255) / 256;
        a.step_h = (heads + parts - 1) / parts;
        a.step_t = 1;
    }
    const int threads = (a.step_h * a.step_t * items + 31) / 32 * 32;
    // Tokens of a block: up to as many as give every thread about one sine and cosine, or one
    // pass over the tokens side by side.
    int most = half > 0 ? 256 / half : kMaxTokens;
    if (most < a.step_t) most = a.step_t;
    if (cs_row > 0 && most > kMaxPairs / cs_row) most = kMaxPairs / cs_row;
    if (most > kMaxTokens) most = kMaxTokens;
    int slots = 0;
    static std::atomic<int> known[2][kMaxDevices];
    const cudaError_t e =
        a.paged ? slots_of(known[1], rope_kernel<T, kHalfStyle, N, true>, threads, sms, &slots)
                : slots_of(known[0], rope_kernel<T, kHalfStyle, N, false>, threads, sms, &slots);
    if (e != cudaSuccess) return e;
    a.tokens = best_tokens(a, most, threads, heads, half, slots);
    const long long blocks = (a.rows + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(blocks);
    return launch_early(a.paged ? rope_kernel<T, kHalfStyle, N, true> : rope_kernel<T, kHalfStyle, N, false>,
                        grid, threads, 0, a.stream, a);
}

template <typename T>
cudaError_t launch_t(RopeArgs& a, int sms)
{
    constexpr int kFull = 16 / sizeof(T);
    if (!a.half_style) return launch<T, false, kFull>(a, sms);
    // half style: pieces of 16 or 8 bytes if each half is whole ones.  Else vectors with shifted
    // partners (8913 tokens of 16 heads of 128 dims, bf16, 63 pairs: 28 us, piece by piece of 2
    // bytes 43; 20 heads of 80, 10 pairs: 25, by 4 bytes 38; fp32, 10 heads of 128, 63 pairs: 28,
    // by 4 bytes 35 -- while with 12 pairs of 64 dims in bf16 pieces of 8 bytes take 17 and this
    // 23, with 50 of 100 in fp32 17 and 29) if a row fits a warp, as all in bf16 do; the wide
    // rows of fp32 take single elements.
    const int half = a.rot / 2;
    if (half % kFull == 0) return launch<T, true, kFull>(a, sms);
    if (half % (kFull / 2) == 0) return launch<T, true, kFull / 2>(a, sms);
    if constexpr (sizeof(T) == 4) {
        if (a.D > 32 * kFull) return launch<T, true, 1>(a, sms);
    }
    return launch_shift<T>(a, sms);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args)
{
    RopeArgs a = args;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    return a.elem == 2 ? launch_t<__nv_bfloat16>(a, sms) : launch_t<float>(a, sms);
}

}  // namespace ra
