// qk_norm.cu -- norms of query and key heads with the rotation in the same pass: forward
// (qk_norm_rope_fwd, and paged_kv_append with weights) and backward (qk_norm_rope_bwd).
//
// A head vector x of D dims becomes
//   y = R(p) (w o x r),   r = 1 / sqrt(mean(x^2) + eps),
// w the weights (plus an offset), o the product by elements, R(p) the rotation by the token's
// position (rope.cu).  With z = R^T dy, g = w o z and u = x r its gradients are
//   dx = r (g - u mean(g o u)),   dw = sum over rows of z o u.
// Everything is computed in fp32 from the inputs and rounded once at the end; the backward
// takes r from x again, which costs no bytes, instead of reading it.
//
// What bounds it: every element is read and written once (backward: two reads, one write), so
// the copy bandwidth.  A power of two of lanes shares a head vector, two 16-byte vectors each,
// chosen so that a pair's elements are in one lane; sums over the vector are shuffles among
// them.  A warp takes as many head vectors at once as its lanes hold (a round), a token's heads
// one round after the other, and an equal share of all rounds; it works out its tokens' sines
// and cosines for itself, once for all their heads, while the next rounds are on their way, and
// meets no barrier.  In the half style with a rot/2 that is no multiple of the vector the lanes
// exchange their elements through shared memory.
//
// The weights' gradients: a lane keeps its columns' sums over all its rows in registers; the
// lanes of a block are added through shared memory, and the blocks' sums through the workspace, in
// two steps of a fixed order, so that repeated calls give the same bits.
#include <algorithm>

#include "rope_pos.cuh"

namespace ra {
namespace {

// Threads of a block, blocks that an SM should hold (of 128 threads with 64 registers each and 94,
// and of 256 with 128) and rounds in flight.  Measured: 32768 tokens of 40 heads of 128 in bf16
// 100 us (three rounds in flight, six blocks: 102); 8192 tokens of 32 and 8 heads appended 38 us
// (two rounds, six blocks: 40; blocks of 256: 42); gradients of 16381 tokens of 40 heads 89 us
// (two rounds: 90; one, three blocks: 105; blocks of 128: 91 to 93).
constexpr int kFwdThreads = 128, kBwdThreads = 256;
constexpr int kFwdBlocks = 8, kPagedBlocks = 5, kBwdBlocks = 2;
constexpr int kFwdAhead = 2, kPagedAhead = 3, kBwdAhead = 3;

enum Mode { kHalf, kInterleaved, kExchange };

// 16 bytes of a row, and as pairs of fp32.
template <typename T>
struct alignas(16) Vec {
    T e[16 / sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void widen(const Vec<T>& v, uint64_t* f)
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v.e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = unpack2(w[i]);
    } else {
        f[0] = f2pack(v.e[0], v.e[1]);
        f[1] = f2pack(v.e[2], v.e[3]);
    }
}
// The one rounding (nearest even).
template <typename T>
__device__ __forceinline__ Vec<T> narrow(const uint64_t* f)
{
    Vec<T> v;
    if constexpr (sizeof(T) == 2) {
        uint32_t* w = reinterpret_cast<uint32_t*>(v.e);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack2(f[i]);
    } else {
        f2unpack(f[0], v.e[0], v.e[1]);
        f2unpack(f[1], v.e[2], v.e[3]);
    }
    return v;
}

// How a head vector's vectors are shared out: item i has those at c0 and c1 (-1: none).
template <Mode kMode, int N>
__host__ __device__ __forceinline__ int items_of(int D, int rot)
{
    if (kMode == kHalf) return rot / 2 / N + ((D - rot) / N + 1) / 2;
    return (D / N + 1) / 2;
}
template <Mode kMode, int N>
__device__ __forceinline__ void columns_of(int D, int rot, int item, int items, int& c0, int& c1)
{
    c0 = c1 = -1;
    if (item >= items) return;
    if (kMode == kHalf) {
        const int turning = rot / 2 / N;
        if (item < turning) {
            c0 = item * N;
            c1 = rot / 2 + c0;
            return;
        }
        const int apart = items - turning;          // (D - rot) / N vectors, two an item
        c0 = rot + (item - turning) * N;
        c1 = c0 + apart * N < D ? c0 + apart * N : -1;
    } else {
        c0 = item * N;
        c1 = c0 + items * N < D ? c0 + items * N : -1;
    }
}

// (all of it is read or written in pieces of 8 and 16 bytes)
template <typename T, Mode kMode, int kWarps, bool kBack>
struct Smem {
    alignas(16) float cos_s[kWarps][128];
    alignas(16) float sin_s[kWarps][128];
    alignas(16) float weight[2][256];
    alignas(16) float exchange[kMode == kExchange ? kWarps : 1][kMode == kExchange ? 32 * 2 * (16 / sizeof(T)) : 4];
    alignas(16) float sums[kBack ? kWarps : 1][kBack ? 256 : 4];
    int last;
};

// The rotation of a lane's elements (N / 2 pairs of neighbours of vector c0, then of c1), or with
// kSign -1 its transpose.  `row`: the lanes' exchange area for this head vector (kExchange).  All
// lanes of the warp take part.
template <Mode kMode, int N, int kSign>
__device__ __forceinline__ void turn(uint64_t* f, const float* cs, const float* sn, int rot, int item, int c0,
                                     int c1, float* row)
{
    const int half = rot / 2;
    if constexpr (kMode == kHalf) {
        const int turning = half / N;
        if (item >= turning) return;
        const uint64_t minus = f2pack(-1.f, -1.f);
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(cs + 4 * (q * turning + item));
            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(sn + 4 * (q * turning + item));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint64_t& a = f[2 * q + i];
                uint64_t& b = f[N / 2 + 2 * q + i];
                const uint64_t cc = i ? c.y : c.x, ss = i ? s.y : s.x;
                const uint64_t as = fmul2(a, ss), bs = fmul2(b, ss);
                a = ffma2(a, cc, kSign > 0 ? fmul2(bs, minus) : bs);
                b = ffma2(b, cc, kSign > 0 ? as : fmul2(as, minus));
            }
        }
    } else if constexpr (kMode == kInterleaved) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int p0 = (v ? c1 : c0) / 2;
            if ((v ? c1 : c0) < 0) continue;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (p0 + i >= half) continue;
                const float c = cs[p0 + i], s = kSign * sn[p0 + i];
                float a, b;
                f2unpack(f[N / 2 * v + i], a, b);
                f[N / 2 * v + i] = f2pack(fmaf(a, c, -(b * s)), fmaf(b, c, a * s));
            }
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int at = v ? c1 : c0;
            if (at < 0) continue;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                *reinterpret_cast<uint64_t*>(row + at + 2 * i) = f[N / 2 * v + i];
        }
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int at = v ? c1 : c0;
            if (at < 0) continue;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float x[2];
                f2unpack(f[(N * v + i) / 2], x[0], x[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int e = at + i + j;
                    if (e >= rot) continue;
                    const bool first = e < half;
                    const int pair = first ? e : e - half;
                    const float other = row[first ? e + half : e - half];
                    const float s = kSign * (first ? -sn[pair] : sn[pair]);
                    x[j] = fmaf(x[j], cs[pair], other * s);
                }
                f[(N * v + i) / 2] = f2pack(x[0], x[1]);
            }
        }
    }
}

// Sines and cosines (times the amplitude) of a position, by one warp into its own area.
template <Mode kMode, int N>
__device__ __forceinline__ void angles(const RopeArgs& a, float* cs, float* sn, long long pos)
{
    const int half = a.rot / 2, turning = half / N;
    __syncwarp();
    for (int pair = threadIdx.x & 31; pair < half; pair += 32) {
        unsigned long long ph = 0;
        if (in_bounds(pair, 1, half, a.status)) ph = __ldg(a.phases + pair);
        float s, c;
        angle_of(ph, pos, s, c);
        // (half style: in groups of four, group q of an item behind group q of all items, so
        // that neighbouring lanes read neighbouring groups)
        int at = pair;
        if (kMode == kHalf) {
            const int item = pair / N, in = pair % N;
            at = ((in / 4) * turning + item) * 4 + in % 4;
        }
        cs[at] = c * a.amplitude;
        sn[at] = s * a.amplitude;
    }
    __syncwarp();
}

// The weights of this lane's columns, from shared memory: in groups of four, group q of a lane
// behind group q of all lanes.
template <int N>
__device__ __forceinline__ void weights_of(const float* w, int item, int lanes, uint64_t* out)
{
#pragma unroll
    for (int q = 0; q < N / 2; ++q) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(w + 4 * (q * lanes + item));
        out[2 * q] = x.x;
        out[2 * q + 1] = x.y;
    }
}

__device__ __forceinline__ float both(uint64_t v)
{
    float lo, hi;
    f2unpack(v, lo, hi);
    return lo + hi;
}
// Sum over the lanes of a head vector.  kLanes 0: a number known at run time only.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float x, int lanes)
{
#pragma unroll
    for (int o = kLanes ? kLanes / 2 : 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = kLanes || o < lanes ? x + y : x;
    }
    return x;
}

// This thread's share of the weights on their way, and then in shared memory for weights_of.
template <Mode kMode, int N, int kThreads>
struct Weights {
    static constexpr int kEach = 512 / kThreads;        // 4 N lanes <= 512 of them
    float x[kEach];
    __device__ __forceinline__ void fetch(const NormArgs& n, int D, int lanes, int items)
    {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads;
            x[k] = 1.f;
            if (i >= 4 * N * lanes) continue;
            const int which = i / (2 * N * lanes), at = i - which * 2 * N * lanes;
            const int q = at / (4 * lanes), item = at / 4 - q * lanes;
            int c0, c1;
            columns_of<kMode, N>(D, n.rope.rot, item, items, c0, c1);
            const int from = 4 * q < N ? c0 : c1, c = from + (4 * q) % N + at % 4;
            const void* w = which ? n.k_weight : n.q_weight;
            if (w != nullptr && from >= 0 && in_bounds(c, 1, D, n.rope.status))
                x[k] = (n.weight_elem == 2 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c])
                                           : static_cast<const float*>(w)[c]) +
                       n.weight_offset;
        }
    }
    __device__ __forceinline__ void store(float (&weight)[2][256], int lanes)
    {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i >= 4 * N * lanes) continue;
            const int which = i / (2 * N * lanes);
            weight[which][i - which * 2 * N * lanes] = x[k];
        }
        __syncthreads();
    }
};

// A warp's share of the forward's rounds: one part of a token's, of `parts` equal to a round.
struct Share {
    long long t;            // token
    int j;                  // the first round's number within the token
    int rounds;
};
__device__ __forceinline__ Share share_of(const NormArgs& n)
{
    const long long w = static_cast<long long>(blockIdx.x) * (kFwdThreads / 32) + (threadIdx.x >> 5);
    Share s;
    s.t = w;
    s.j = 0;
    s.rounds = n.per_token;
    if (n.parts > 1) {                          // (up to 64, of fewer than 2^25 rounds)
        const unsigned parts = n.parts, per_token = n.per_token;
        s.t = w >> 32 ? w / n.parts : static_cast<unsigned>(w) / parts;
        const unsigned part = static_cast<unsigned>(w - s.t * n.parts);
        s.j = part * per_token / parts;
        s.rounds = (part + 1) * per_token / parts - s.j;
    }
    if (s.t >= n.rope.rows) s.rounds = 0;
    return s;
}

// Where a group of lanes is in its warp's share: the head vector that it holds of each round.
// The tensors' heads follow one another (q's, k's, and in the paged append v's): only where one
// ends is the address worked out anew.
template <typename E>
struct Cursor {
    E* p;                   // the head vector
    long long at;           // ... as an element offset in its tensor
    long long step;         // to the next round's, of the same tensor
    long long t;
    int h;
    int kind;               // 0 q, 1 k, 2 v, 3: no head left for this group
    int bound;              // the kind's last head, one further
};
struct Side {               // a tensor of q's, k's and v's rows
    const void* base[3];
    long long token[3];     // strides
    long long head[3];
};

template <typename E>
__device__ __forceinline__ void locate(Cursor<E>& c, const NormArgs& n, const Side& s, int abreast)
{
    const RopeArgs& a = n.rope;
    const int e1 = a.H, e2 = a.H + a.H_kv, e3 = e2 + (a.paged ? a.H_kv : 0);
    c.kind = c.h < e1 ? 0 : c.h < e2 ? 1 : c.h < e3 ? 2 : 3;
    c.bound = c.kind == 0 ? e1 : c.kind == 1 ? e2 : c.kind == 2 ? e3 : 0x7fffffff;
    const int hh = c.h - (c.kind == 0 ? 0 : c.kind == 1 ? e1 : e2);
    const bool q = c.kind == 0, k = c.kind == 1;
    const long long head = q ? s.head[0] : k ? s.head[1] : s.head[2];
    c.at = c.t * (q ? s.token[0] : k ? s.token[1] : s.token[2]) + hh * head;
    c.step = abreast * head;
    c.p = const_cast<E*>(static_cast<const E*>(q ? s.base[0] : k ? s.base[1] : s.base[2])) + c.at;
}
template <typename E>
__device__ __forceinline__ void advance(Cursor<E>& c, const NormArgs& n, const Side& s, int abreast)
{
    c.h += abreast;
    c.p += c.step;
    c.at += c.step;
    if (c.h >= c.bound) locate(c, n, s, abreast);
}
template <typename E>
__device__ __forceinline__ Cursor<E> cursor_at(const Share& w, const NormArgs& n, const Side& s, int sub,
                                               int abreast)
{
    Cursor<E> c;
    c.t = w.t;
    c.h = w.j * abreast + sub;
    locate(c, n, s, abreast);
    return c;
}

// A head vector's lanes where its length is known at compile time (0: it is not) and every lane
// holds two vectors of it.
template <typename T, int kD>
constexpr int kLanesOf = kD / (2 * (16 / static_cast<int>(sizeof(T))));

// kD: the head dim, or 0 for any.
template <typename T, Mode kMode, int kD, bool kPaged>
__global__ void __launch_bounds__(kFwdThreads, kPaged ? kPagedBlocks : kFwdBlocks) norm_fwd_kernel(const __grid_constant__ NormArgs n)
{
    constexpr int N = 16 / sizeof(T);
    constexpr int kAhead = kPaged ? kPagedAhead : kFwdAhead;
    __shared__ Smem<T, kMode, kFwdThreads / 32, false> s;
    const RopeArgs& a = n.rope;
    constexpr int kLanes = kLanesOf<T, kD>;
    const int lanes = kD ? kLanes : n.lanes, abreast = 32 / lanes, D = kD ? kD : a.D;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = lane & (lanes - 1), sub = lane / lanes;
    int c0, c1;
    columns_of<kMode, N>(D, a.rot, item, kD ? kLanes : n.items, c0, c1);
    float* row = s.exchange[kMode == kExchange ? warp : 0] + (kMode == kExchange ? sub * lanes * 2 * N : 0);
    const float over_D = 1.f / D;
    const Side in{{a.q, a.k, a.v}, {a.q_stride, a.k_stride, a.v_stride}, {D, D, D}};
    // (in the pages a token's place is added by its slot)
    const Side out = kPaged ? Side{{a.q_out, a.k_out, a.v_out}, {a.q_out_stride, 0, 0},
                                   {D, a.head_stride, a.head_stride}}
                            : Side{{a.q_out, a.k_out, nullptr}, {a.q_out_stride, a.k_out_stride, 0},
                                   {D, D, D}};
    const Share share = share_of(n);

    struct Row {
        Vec<T> x0, x1;
    };
    int left = share.rounds;                // to be fetched
    Cursor<const T> from = cursor_at<const T>(share, n, in, sub, abreast);
    auto fetch = [&](Row& r) {
        r.x0 = Vec<T>{};
        r.x1 = Vec<T>{};
        if (left <= 0) return;
        --left;
        const long long extent = from.kind == 0 ? a.q_elems : from.kind == 1 ? a.k_elems : a.v_elems;
        if (from.kind < 3 && in_bounds(from.at, D, extent, a.status)) {
            if (kD || c0 >= 0) r.x0 = *reinterpret_cast<const Vec<T>*>(from.p + c0);
            if (kD || c1 >= 0) r.x1 = *reinterpret_cast<const Vec<T>*>(from.p + c1);
        }
        advance(from, n, in, abreast);
    };
    wait_for_earlier_work();
    // the first rounds are on their way while the weights, positions and angles are worked out
    Row r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(r[u]);
    Weights<kMode, N, kFwdThreads> weights;
    weights.fetch(n, D, lanes, kD ? kLanes : n.items);
    Cursor<T> to = cursor_at<T>(share, n, out, sub, abreast);
    const TokenPos pos = token_pos<kPaged>(a, to.t);
    weights.store(s.weight, lanes);
    angles<kMode, N>(a, s.cos_s[warp], s.sin_s[warp], pos.pos);
    auto finish = [&](Row& r) {
        uint64_t f[N];
        widen(r.x0, f);
        widen(r.x1, f + N / 2);
        uint64_t ss = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) ss = ffma2(f[i], f[i], ss);
        const float rs = rsqrtf(fmaf(lanes_sum<kLanes>(both(ss), lanes), over_D, n.eps));
        uint64_t w[N];
        weights_of<N>(s.weight[to.kind == 0 ? 0 : 1], item, lanes, w);
        const uint64_t rr = f2pack(rs, rs);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = fmul2(fmul2(f[i], rr), w[i]);
        turn<kMode, N, 1>(f, s.cos_s[warp], s.sin_s[warp], a.rot, item, c0, c1, row);
        // (the paged append's values stay as they are)
        if (!kPaged || to.kind < 2) {
            r.x0 = narrow<T>(f);
            r.x1 = narrow<T>(f + N / 2);
        }
        const bool to_page = kPaged && to.kind > 0;
        const long long skip = to_page ? pos.slot : 0;
        if (to.kind < 3 && (to_page ? pos.slot >= 0 : pos.live) &&
            in_bounds(to.at + skip, D, to.kind == 0 ? a.q_out_elems : a.k_out_elems, a.status)) {
            T* dst = to.p + skip;
            if (kD || c0 >= 0) *reinterpret_cast<Vec<T>*>(dst + c0) = r.x0;
            if (kD || c1 >= 0) *reinterpret_cast<Vec<T>*>(dst + c1) = r.x1;
        }
        advance(to, n, out, abreast);
    };
    for (int i = 0; i < share.rounds; i += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i + u >= share.rounds) break;
            finish(r[u]);
            fetch(r[u]);
        }
    }
}

template <typename T, Mode kMode, int kD>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks) norm_bwd_kernel(const __grid_constant__ NormArgs n)
{
    constexpr int N = 16 / sizeof(T);
    constexpr int kAhead = kBwdAhead;
    constexpr int kWarps = kBwdThreads / 32;
    __shared__ Smem<T, kMode, kWarps, true> s;
    const RopeArgs& a = n.rope;
    constexpr int kLanes = kLanesOf<T, kD>;
    const int lanes = kD ? kLanes : n.lanes, abreast = 32 / lanes, D = kD ? kD : a.D;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = lane & (lanes - 1), sub = lane / lanes;
    int c0, c1;
    columns_of<kMode, N>(D, a.rot, item, kD ? kLanes : n.items, c0, c1);
    float* row = s.exchange[kMode == kExchange ? warp : 0] + (kMode == kExchange ? sub * lanes * 2 * N : 0);
    const float over_D = 1.f / D;
    const unsigned warps = gridDim.x * kWarps, w0 = blockIdx.x * kWarps + warp;

    struct Row {
        Vec<T> x0, x1, y0, y1;
    };
    wait_for_earlier_work();
    // Queries, then keys: a warp's rounds of them are an equal share of all, one after the other.
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const int heads = kind ? a.H_kv : a.H;
        if (heads == 0) continue;
        const int per = (heads + abreast - 1) / abreast;        // rounds of a token
        const long long total = a.rows * per, each = total / warps, more = total - each * warps;
        const long long first = w0 * each + min(static_cast<long long>(w0), more);
        const int rounds = static_cast<int>(each) + (w0 < more ? 1 : 0);
        const long long t0 = first / per;
        const int j0 = static_cast<int>(first - t0 * per);
        const long long x_step = kind ? a.k_stride : a.q_stride;
        const long long y_step = kind ? n.dk_out_stride : n.dq_out_stride;
        const long long d_step = kind ? a.k_out_stride : a.q_out_stride;
        const long long extent_x = kind ? a.k_elems : a.q_elems, extent_y = kind ? n.dk_out_elems : n.dq_out_elems;
        const long long extent_d = kind ? a.k_out_elems : a.q_out_elems;
        const long long next = abreast * D;                      // from round to round of a token
        long long xi = t0 * x_step + (j0 * abreast + sub) * static_cast<long long>(D);
        long long yi = t0 * y_step + (j0 * abreast + sub) * static_cast<long long>(D);
        long long di = t0 * d_step + (j0 * abreast + sub) * static_cast<long long>(D);
        const T* X = static_cast<const T*>(kind ? a.k : a.q);
        const T* Y = static_cast<const T*>(kind ? n.dk_out : n.dq_out);
        T* DX = static_cast<T*>(kind ? a.k_out : a.q_out);
        int left = rounds, jf = j0;                              // to be fetched
        auto fetch = [&](Row& r) {
            r.x0 = r.x1 = r.y0 = r.y1 = Vec<T>{};
            if (left <= 0) return;
            --left;
            if (jf * abreast + sub < heads && in_bounds(xi, D, extent_x, a.status) &&
                in_bounds(yi, D, extent_y, a.status)) {
                if (kD || c0 >= 0) {
                    r.x0 = *reinterpret_cast<const Vec<T>*>(X + xi + c0);
                    r.y0 = *reinterpret_cast<const Vec<T>*>(Y + yi + c0);
                }
                if (kD || c1 >= 0) {
                    r.x1 = *reinterpret_cast<const Vec<T>*>(X + xi + c1);
                    r.y1 = *reinterpret_cast<const Vec<T>*>(Y + yi + c1);
                }
            }
            xi += next;
            yi += next;
            if (++jf == per) {
                jf = 0;
                xi += x_step - per * next;
                yi += y_step - per * next;
            }
        };
        Row r[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) fetch(r[u]);
        if (kind == 0 || a.H == 0) {
            Weights<kMode, N, kBwdThreads> weights;
            weights.fetch(n, D, lanes, kD ? kLanes : n.items);
            weights.store(s.weight, lanes);
        }

        // this lane's columns of the weights' gradient
        uint64_t dw[N];
#pragma unroll
        for (int i = 0; i < N; ++i) dw[i] = 0;
        long long t = t0;
        int j = j0;
        bool live = false, new_token = true;
        auto finish = [&](Row& r) {
            if (new_token) {
                const TokenPos pos = token_pos<false>(a, t);
                live = pos.live;
                angles<kMode, N>(a, s.cos_s[warp], s.sin_s[warp], pos.pos);
            }
            uint64_t x[N], z[N], w[N];
            widen(r.x0, x);
            widen(r.x1, x + N / 2);
            widen(r.y0, z);
            widen(r.y1, z + N / 2);
            turn<kMode, N, -1>(z, s.cos_s[warp], s.sin_s[warp], a.rot, item, c0, c1, row);
            weights_of<N>(s.weight[kind], item, lanes, w);
            uint64_t ss = 0, dot = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                w[i] = fmul2(w[i], z[i]);                           // g
                ss = ffma2(x[i], x[i], ss);
                dot = ffma2(w[i], x[i], dot);
            }
            const float sum = lanes_sum<kLanes>(both(ss), lanes), product = lanes_sum<kLanes>(both(dot), lanes);
            const float rs = rsqrtf(fmaf(sum, over_D, n.eps));
            const float c = -(product * rs * over_D);               // - mean(g o u)
            const uint64_t rr = f2pack(rs, rs), cc = f2pack(c, c);
            if (live && j * abreast + sub < heads) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    x[i] = fmul2(x[i], rr);                         // u
                    dw[i] = ffma2(z[i], x[i], dw[i]);
                    z[i] = fmul2(rr, ffma2(x[i], cc, w[i]));
                }
                if (in_bounds(di, D, extent_d, a.status)) {
                    if (kD || c0 >= 0) *reinterpret_cast<Vec<T>*>(DX + di + c0) = narrow<T>(z);
                    if (kD || c1 >= 0) *reinterpret_cast<Vec<T>*>(DX + di + c1) = narrow<T>(z + N / 2);
                }
            }
            di += next;
            new_token = ++j == per;
            if (new_token) {
                j = 0;
                ++t;
                di += d_step - per * next;
            }
        };
        for (int i = 0; i < rounds; i += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (i + u >= rounds) break;
                finish(r[u]);
                fetch(r[u]);
            }
        }
        // This block's sums: over a warp's groups, then over the warps in order.
#pragma unroll
        for (int i = 0; i < N; ++i)
            for (int o = lanes; o < 32; o <<= 1) dw[i] = fadd2(dw[i], __shfl_xor_sync(0xffffffffu, dw[i], o));
        if (lane < lanes) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (kD || c0 >= 0) *reinterpret_cast<uint64_t*>(&s.sums[warp][c0 + 2 * i]) = dw[i];
                if (kD || c1 >= 0) *reinterpret_cast<uint64_t*>(&s.sums[warp][c1 + 2 * i]) = dw[N / 2 + i];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += kBwdThreads) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) x += s.sums[i][c];
            const long long at = (static_cast<long long>(blockIdx.x) * 2 + kind) * 256 + c;
            if (in_bounds(at, 1, 512ll * kNormCtas, a.status)) __stcg(n.partials + at, x);
        }
        __syncthreads();
    }
    // Then over kNormGroup blocks, by the last of them, in order, and over these groups, by the
    // last of all, in order.
    auto arrive_last = [&](unsigned int* counter, unsigned of) -> bool {
        if (threadIdx.x == 0) {
            unsigned before;
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                         : "=r"(before)
                         : "l"(counter)
                         : "memory");
            s.last = before == of - 1;
            if (s.last) *counter = 0;
        }
        __syncthreads();
        return s.last;
    };
    // column c of kind's sums, over the slots first, first + apart, ..., count of them
    auto sum_of = [&](int kind, int c, int first, int apart, int count) -> float {
        float x = 0.f;
#pragma unroll 1
        for (int b = 0; b < count; b += kNormGroup) {
            float v[kNormGroup];
#pragma unroll
            for (int u = 0; u < kNormGroup; ++u) {
                const long long at = (static_cast<long long>(first + min(b + u, count - 1) * apart) * 2 + kind) * 256 + c;
                v[u] = in_bounds(at, 1, 512ll * kNormCtas, a.status) ? __ldcg(n.partials + at) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kNormGroup; ++u) x += b + u < count ? v[u] : 0.f;
        }
        return x;
    };
    const int blocks = gridDim.x, groups = (blocks + kNormGroup - 1) / kNormGroup;
    const int group = blockIdx.x / kNormGroup, first = group * kNormGroup;
    if (!arrive_last(n.ticket + 1 + group, min(kNormGroup, blocks - first))) return;
    for (int i = threadIdx.x; i < 2 * D; i += kBwdThreads) {
        const int kind = i >= D, c = i - kind * D;
        const float x = sum_of(kind, c, first, 1, min(kNormGroup, blocks - first));
        const long long at = (static_cast<long long>(first) * 2 + kind) * 256 + c;
        if (in_bounds(at, 1, 512ll * kNormCtas, a.status)) __stcg(n.partials + at, x);
    }
    __syncthreads();
    if (!arrive_last(n.ticket, groups)) return;
    for (int i = threadIdx.x; i < 2 * D; i += kBwdThreads) {
        const int kind = i >= D, c = i - kind * D;
        float* dst = kind ? n.dk_weight : n.dq_weight;
        if (dst == nullptr || !in_bounds(c, 1, D, a.status)) continue;
        dst[c] = sum_of(kind, c, 0, kNormGroup, groups);
    }
}

template <typename T, Mode kMode, int kD>
cudaError_t launch(NormArgs& n, bool backward)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    RopeArgs& a = n.rope;
    n.items = items_of<kMode, N>(a.D, a.rot);
    n.lanes = 1;
    while (n.lanes < n.items) n.lanes *= 2;
    const int heads = a.H + (a.paged ? 2 : 1) * a.H_kv, abreast = 32 / n.lanes;
    n.per_token = (heads + abreast - 1) / abreast;
    // as many blocks as the GPU holds at once, or as there are rounds for
    static std::atomic<int> known[3][kMaxDevices];
    const auto kernel = backward ? norm_bwd_kernel<T, kMode, kD>
                        : a.paged ? norm_fwd_kernel<T, kMode, kD, true>
                                  : norm_fwd_kernel<T, kMode, kD, false>;
    int slots = 0;
    const int threads = backward ? kBwdThreads : kFwdThreads, warps = threads / 32;
    const cudaError_t e = resident_ctas(known[backward ? 2 : a.paged ? 1 : 0], kernel, threads, 0, &slots);
    if (e != cudaSuccess) return e;
    if (backward) slots = std::min(slots, kNormCtas);
    if (backward) {
        const long long rounds = a.rows * ((std::max(a.H, a.H_kv) + abreast - 1) / abreast);
        const unsigned grid = static_cast<unsigned>(std::min<long long>((rounds + warps - 1) / warps, slots));
        return launch_early(kernel, grid, threads, 0, a.stream, n);
    }
    // The parts of a token's rounds, a warp each, with which the call is done first, taking that
    // the warps go in waves of as many as the GPU holds and that one takes as long as kFixed
    // rounds (first reads, position, angles) besides its own.
    constexpr int kFixed = 4;
    const long long held = static_cast<long long>(slots) * warps;
    long long least = 0;
    for (int p = 1; p <= std::min(n.per_token, 64); ++p) {
        const long long waves = (a.rows * p + held - 1) / held;
        const long long cost = waves * (kFixed + (n.per_token + p - 1) / p);
        if (p == 1 || cost < least) {
            least = cost;
            n.parts = p;
        }
        if (waves > 64) break;                      // (more parts only cost more)
    }
    const long long blocks = (a.rows * n.parts + warps - 1) / warps;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(blocks);
    return launch_early(kernel, grid, threads, 0, a.stream, n);
}

template <typename T>
cudaError_t launch_t(NormArgs& n, bool backward)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const RopeArgs& a = n.rope;
    // (the usual head dims with their length known at compile time: see kLanesOf)
    if (!a.half_style)
        return a.D == 128 ? launch<T, kInterleaved, 128>(n, backward) : launch<T, kInterleaved, 0>(n, backward);
    if (a.rot / 2 % N != 0) return launch<T, kExchange, 0>(n, backward);
    if (a.D == 64) return launch<T, kHalf, 64>(n, backward);
    if (a.D == 128) return launch<T, kHalf, 128>(n, backward);
    if (a.D == 256) return launch<T, kHalf, 256>(n, backward);
    return launch<T, kHalf, 0>(n, backward);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& args, bool backward)
{
    NormArgs n = args;
    return n.rope.elem == 2 ? launch_t<__nv_bfloat16>(n, backward) : launch_t<float>(n, backward);
}

}  // namespace ra
