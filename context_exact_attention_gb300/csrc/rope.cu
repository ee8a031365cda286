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
// What bounds it: every element is read and written once (bytes), the arithmetic is a few
// instructions per element.  One block takes `tokens` tokens: it first finds their
// positions and computes their tokens * rot/2 sines and cosines into shared memory (once
// for all heads), while the first rows' loads are already in flight; then its threads
// stream the tokens' heads.  A thread keeps one item of a head vector -- a 16-byte vector
// of each half of the pairs (half style), a vector of whole pairs (interleaved), or a
// vector of the dims behind `rot` -- and steps over the (token, head) rows, so the column
// arithmetic is done once.  Head vectors whose pairs do not fill 16-byte vectors go one
// pair at a time through the same code (kVec false).
#include <cuda_bf16.h>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxPairs = 256;      // sines and cosines of one block: tokens * rot / 2
constexpr int kMaxTokens = 16;
constexpr int kUnroll = 2;          // rows in flight per thread

struct TokenPos {
    long long pos;      // position in its sequence
    long long slot;     // paged: element offset of the token's page slot, or -1 (not stored)
    int live;           // 0: the row belongs to no sequence and is left as it is
};

// The largest j in [0, n) with v[j] <= x (0 if there is none) for a non-decreasing v, by
// one warp: every step loads 32 evenly spaced entries at once, so 1024 entries take two
// dependent loads where a binary search takes ten.
__device__ __forceinline__ int warp_upper(const int* v, int n, long long x, long long extent,
                                          unsigned int* status)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;                       // the answer lies in [lo, lo + len)
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int j = lo + lane * step;
        const bool le = lane * step < len && checked_ldg(v, j, extent, status) <= x;
        const int cnt = __popc(__ballot_sync(0xffffffffu, le));
        const int k = cnt > 0 ? cnt - 1 : 0;
        lo += k * step;
        len = min(step, len - k * step);
    }
    return lo;
}

// Position (and page slot) of token row `t`, computed by one warp.
template <bool kPaged>
__device__ __forceinline__ TokenPos token_pos(const RopeArgs& a, long long t)
{
    TokenPos r{0, -1, 0};
    if (t >= a.rows) return r;
    if constexpr (kPaged) {
        const int g = warp_upper(a.cu_seqlens, a.n_seqs, t, a.n_seqs + 1, a.status);
        const int first = checked_ldg(a.cu_seqlens, g, a.n_seqs + 1, a.status);
        const int end = checked_ldg(a.cu_seqlens, g + 1, a.n_seqs + 1, a.status);
        if (t < first || t >= end) return r;
        r.live = 1;
        r.pos = static_cast<long long>(checked_ldg(a.kv_lens, g, a.n_seqs, a.status)) -
                (static_cast<long long>(end) - t);
        const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
        if (r.pos >= 0 && r.pos < cap) {
            const int col = static_cast<int>(r.pos / a.page_size);
            const int in_page = static_cast<int>(r.pos - static_cast<long long>(col) * a.page_size);
            const int page = checked_ldg(a.page_table, g * a.table_stride + col, a.table_elems,
                                         a.status);
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
                r.slot = page * a.page_stride + in_page * a.token_stride;
        }
        return r;
    } else {
        r.live = 1;
        const int l = static_cast<int>(t % a.L);
        if (a.positions != nullptr) {
            r.pos = checked_ldg(a.positions, t, a.rows, a.status);
        } else if (a.layout == RA_LAYOUT_ZIGZAG) {
            // shard s holds chunks s and 2P-1-s of 2P chunks of c positions
            const int c = a.L / (2 * a.P);
            const int piece = l / c, s = piece >> 1;
            r.pos = static_cast<long long>((piece & 1) ? 2 * a.P - 1 - s : s) * c + (l - piece * c);
        } else if (a.layout == RA_LAYOUT_PACKED) {
            const int g = warp_upper(a.cu_seqlens, a.n_seqs, t, a.n_seqs + 1, a.status);
            const int first = checked_ldg(a.cu_seqlens, g, a.n_seqs + 1, a.status);
            if (t < first || t >= checked_ldg(a.cu_seqlens, g + 1, a.n_seqs + 1, a.status))
                r.live = 0;
            r.pos = t - first;
        } else {
            r.pos = l;
        }
        r.pos += a.position_offset;
        return r;
    }
}

template <typename T>
__device__ __forceinline__ float to_f(T x)
{
    if constexpr (sizeof(T) == 2) return __bfloat162float(x);
    else return x;
}
// The one rounding of the operation: the rotated value, computed in fp32, to the tensor's
// type (nearest even).
template <typename T>
__device__ __forceinline__ T from_f(float x)
{
    if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(x);
    else return x;
}

// kHalf pieces of kN elements each, moved as one 16-byte (or one-element) access per piece.
template <typename T, int kN>
struct alignas(kN * sizeof(T)) Piece {
    T e[kN];
};

// kVec: items are 16-byte vectors; otherwise single pairs (and single elements behind
// `rot`).  kPaged: rows are q heads (to q_out), k heads (rotated, to the pages) and v
// heads (to the pages).
template <typename T, bool kHalfStyle, bool kVec, bool kPaged>
__global__ void __launch_bounds__(kBlock) rope_kernel(const RopeArgs a)
{
    // elements of a piece, pieces of a rotated item, and pairs it holds
    constexpr int kFull = 16 / sizeof(T);
    constexpr int kN = kVec ? kFull : (kHalfStyle ? 1 : 2);
    constexpr int kPieces = kHalfStyle ? 2 : 1;
    constexpr int kPairs = kHalfStyle ? kN : kN / 2;
    // an item behind `rot` is one piece; without vectors it is one element
    constexpr int kPassN = kVec ? kFull : 1;
    using Rot = Piece<T, kN>;
    using Pass = Piece<T, kPassN>;

    __shared__ alignas(16) float cos_s[kMaxPairs];
    __shared__ alignas(16) float sin_s[kMaxPairs];
    __shared__ TokenPos tok_s[kMaxTokens];

    const int half = a.rot / 2;
    const int rot_items = half / kPairs;
    const int n_items = rot_items + (a.D - a.rot) / kPassN;
    const int rows_per_pass = kBlock / n_items;
    const int heads = a.H + (kPaged ? 2 : 1) * a.H_kv;
    const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
    const int n_tok = static_cast<int>(min(static_cast<long long>(a.tokens), a.rows - t0));

    for (int i = threadIdx.x >> 5; i < n_tok; i += kBlock / 32) {
        const TokenPos p = token_pos<kPaged>(a, t0 + i);
        if ((threadIdx.x & 31) == 0) tok_s[i] = p;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * half; i += kBlock) {
        const int tok = i / half, pair = i - tok * half;
        unsigned long long ph = 0;
        if (in_bounds(pair, 1, half, a.status)) ph = __ldg(a.phases + pair);
        const unsigned long long turn = ph * static_cast<unsigned long long>(tok_s[tok].pos);
        // upper 32 bits as a signed number: [-2^31, 2^31) is [-1, 1) half turns
        const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;
        float s, c;
        sincospif(x, &s, &c);
        cos_s[i] = c * a.amplitude;
        sin_s[i] = s * a.amplitude * a.sign;
    }
    __syncthreads();

    const int item = threadIdx.x % n_items;
    const int row0 = threadIdx.x / n_items;
    if (row0 >= rows_per_pass) return;
    const bool rotates = item < rot_items;
    // element offsets of the item's pieces within a head vector
    const int c0 = rotates ? item * kN : a.rot + (item - rot_items) * kPassN;
    const int c1 = c0 + half;                      // second piece (half style)
    const int total = n_tok * heads;

    for (int base = row0; base < total; base += kUnroll * rows_per_pass) {
        Rot x0[kUnroll], x1[kUnroll];
        Pass y0[kUnroll];
        const T* src[kUnroll];
        T* dst[kUnroll];
        int tok[kUnroll];
        bool go[kUnroll], turn[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int row = base + u * rows_per_pass;
            go[u] = row < total;
            turn[u] = false;
            src[u] = nullptr;
            dst[u] = nullptr;
            tok[u] = 0;
            if (!go[u]) continue;
            tok[u] = row / heads;
            int h = row - tok[u] * heads;
            const long long t = t0 + tok[u];
            const TokenPos p = tok_s[tok[u]];
            long long si, di, s_ext, d_ext;        // element offsets and extents (checks)
            turn[u] = rotates;
            if (h < a.H) {
                si = t * a.q_stride + static_cast<long long>(h) * a.D;
                di = t * a.q_out_stride + static_cast<long long>(h) * a.D;
                src[u] = static_cast<const T*>(a.q) + si;
                dst[u] = static_cast<T*>(a.q_out) + di;
                s_ext = a.q_elems;
                d_ext = a.q_out_elems;
                go[u] = p.live;
            } else if (h - a.H < a.H_kv) {
                h -= a.H;
                si = t * a.k_stride + static_cast<long long>(h) * a.D;
                di = kPaged ? p.slot + h * a.head_stride
                            : t * a.k_out_stride + static_cast<long long>(h) * a.D;
                src[u] = static_cast<const T*>(a.k) + si;
                dst[u] = static_cast<T*>(a.k_out) + di;
                s_ext = a.k_elems;
                d_ext = a.k_out_elems;
                go[u] = kPaged ? p.slot >= 0 : p.live;
            } else {
                h -= a.H + a.H_kv;
                si = t * a.v_stride + static_cast<long long>(h) * a.D;
                di = p.slot + h * a.head_stride;
                src[u] = static_cast<const T*>(a.v) + si;
                dst[u] = static_cast<T*>(a.v_out) + di;
                s_ext = a.v_elems;
                d_ext = a.k_out_elems;
                go[u] = p.slot >= 0;
                turn[u] = false;
            }
            go[u] = go[u] && in_bounds(si, a.D, s_ext, a.status) &&
                    in_bounds(di, a.D, d_ext, a.status);
            if (!go[u]) continue;
            if (rotates) {
                x0[u] = *reinterpret_cast<const Rot*>(src[u] + c0);
                if constexpr (kPieces == 2) x1[u] = *reinterpret_cast<const Rot*>(src[u] + c1);
            } else {
                y0[u] = *reinterpret_cast<const Pass*>(src[u] + c0);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!go[u]) continue;
            if (!rotates) {
                *reinterpret_cast<Pass*>(dst[u] + c0) = y0[u];
                continue;
            }
            if (turn[u]) {
                const float* cs = cos_s + tok[u] * half + item * kPairs;
                const float* sn = sin_s + tok[u] * half + item * kPairs;
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    T& ea = kHalfStyle ? x0[u].e[i] : x0[u].e[(2 * i) % kN];
                    T& eb = kHalfStyle ? x1[u].e[i] : x0[u].e[(2 * i + 1) % kN];
                    const float xa = to_f(ea), xb = to_f(eb), c = cs[i], s = sn[i];
                    ea = from_f<T>(fmaf(xa, c, -(xb * s)));
                    eb = from_f<T>(fmaf(xb, c, xa * s));
                }
            }
            *reinterpret_cast<Rot*>(dst[u] + c0) = x0[u];
            if constexpr (kPieces == 2) *reinterpret_cast<Rot*>(dst[u] + c1) = x1[u];
        }
    }
}

template <typename T, bool kHalfStyle, bool kVec>
cudaError_t launch(const RopeArgs& a, unsigned blocks)
{
    if (a.paged) rope_kernel<T, kHalfStyle, kVec, true><<<blocks, kBlock, 0, a.stream>>>(a);
    else rope_kernel<T, kHalfStyle, kVec, false><<<blocks, kBlock, 0, a.stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, unsigned blocks)
{
    constexpr int kFull = 16 / sizeof(T);
    // whole 16-byte vectors of pairs: each half (half style) or the rotated part
    // (interleaved) a multiple of the vector
    if (a.half_style)
        return a.rot % (2 * kFull) == 0 ? launch<T, true, true>(a, blocks)
                                        : launch<T, true, false>(a, blocks);
    return a.rot % kFull == 0 ? launch<T, false, true>(a, blocks)
                              : launch<T, false, false>(a, blocks);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args)
{
    RopeArgs a = args;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // tokens per block: as many as keep every thread one sine and cosine, but no fewer than
    // eight blocks per SM while there are rows for them
    const int half = a.rot / 2;
    int most = half > 0 ? kBlock / half : kMaxTokens;
    if (most < 1) most = 1;
    if (most > kMaxTokens) most = kMaxTokens;
    long long per = a.rows / (8ll * sms);
    if (per < 1) per = 1;
    a.tokens = static_cast<int>(per < most ? per : most);
    const long long blocks = (a.rows + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return a.elem == 2 ? launch_t<__nv_bfloat16>(a, static_cast<unsigned>(blocks))
                       : launch_t<float>(a, static_cast<unsigned>(blocks));
}

}  // namespace ra
