// qk_norm.cuh -- what the forward and the backward of normalised heads share: how a head vector is
// shared out over lanes, its weights, angles and rotation (see qk_norm.cu).
#pragma once

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
    alignas(16) float cos_s[kWarps][kMode == kExchange ? 256 : 128];
    alignas(16) float sin_s[kWarps][kMode == kExchange ? 256 : 128];
    alignas(16) float weight[2][256];
    alignas(16) float exchange[kMode == kExchange ? kWarps : 1][kMode == kExchange ? 32 * 2 * (16 / sizeof(T)) : 4];
    alignas(16) float sums[kBack ? kWarps : 1][kBack ? 256 : 4];
    int last;
};

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

// The rotation of a lane's elements (N / 2 pairs of neighbours of vector c0, then of c1), or with
// kSign -1 its transpose.  `row`: the lanes' exchange area for this head vector (kExchange).  All
// lanes of the warp take part.
template <Mode kMode, int N, int kSign>
__device__ __forceinline__ void turn(uint64_t* f, const float* cs, const float* sn, int rot, int item, int c0,
                                     int c1, int lanes, int items, float* row)
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
        // `row` holds the head vectors of the warp's groups side by side, element e at
        // (e mod N) apart + e / N, so that neighbouring lanes meet different banks both ways;
        // cosines and signed sines lie by element, as the weights do (weights_of).
        const int apart = (32 / lanes) * 2 * items;
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (item >= items) break;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float x, y;
                f2unpack(f[(N * v + i) / 2], x, y);
                row[i * apart + item + v * items] = x;
                row[(i + 1) * apart + item + v * items] = y;
            }
        }
        __syncwarp();
        uint64_t c[N], s[N];
        weights_of<N>(cs, item, lanes, c);
        weights_of<N>(sn, item, lanes, s);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int at = v ? c1 : c0;
            if (at < 0 || at >= rot) continue;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float other[2], x[2], y[2];
                f2unpack(f[(N * v + i) / 2], x[0], x[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int e = at + i + j, partner = e < half ? e + half : e >= rot ? e : e - half;
                    other[j] = row[partner % N * apart + partner / N];
                }
                const uint64_t o2 = f2pack(kSign * other[0], kSign * other[1]), x2 = f[(N * v + i) / 2];
                f2unpack(ffma2(x2, c[(N * v + i) / 2], fmul2(o2, s[(N * v + i) / 2])), y[0], y[1]);
                f[(N * v + i) / 2] = f2pack(at + i < rot ? y[0] : x[0], at + i + 1 < rot ? y[1] : x[1]);
            }
        }
    }
}

// Sines and cosines (times the amplitude) of a position, by one warp into its own area.
template <Mode kMode, int N>
__device__ __forceinline__ void angles(const RopeArgs& a, float* cs, float* sn, long long pos, int lanes,
                                       int items)
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
        if (kMode == kExchange) {
            // both elements', where weights_of looks for them
            for (int second = 0; second < 2; ++second) {
                const int e = pair + second * half, v = e / N, in = e % N;
                const int q = (v < items ? 0 : N / 4) + in / 4;
                const int to = 4 * (q * lanes + (v < items ? v : v - items)) + in % 4;
                cs[to] = c * a.amplitude;
                sn[to] = (second ? s : -s) * a.amplitude;
            }
            continue;
        }
        if (kMode == kHalf) {
            const int item = pair / N, in = pair % N;
            at = ((in / 4) * turning + item) * 4 + in % 4;
        }
        cs[at] = c * a.amplitude;
        sn[at] = s * a.amplitude;
    }
    __syncwarp();
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

// Where a head vector's length is known at compile time (kD; 0: it is not), an even number of
// vectors: its items, which all hold two, and its lanes.
template <typename T, int kD>
constexpr int kItemsOf = kD / (2 * (16 / static_cast<int>(sizeof(T))));
__host__ __device__ constexpr int lanes_for(int items)
{
    int n = 1;
    while (n < items) n *= 2;
    return n;
}

// The launch function below for a call's type, pair style and head dim (the usual ones known at
// compile time: 32768 tokens of 40 heads of 128 dims 100 us, 111 without; gradients 89 and 108;
// odd halves, 16384 tokens of 16 heads of 128 dims, 50 and 74; of 80 dims 40 and 51).
template <typename T, Mode kMode, int kD>
cudaError_t launch(NormArgs& n);

template <typename T, Mode kMode>
cudaError_t launch_d(NormArgs& n)
{
    switch (n.rope.D) {
    case 64: return launch<T, kMode, 64>(n);
    case 80: return launch<T, kMode, 80>(n);
    case 96: return launch<T, kMode, 96>(n);
    case 128: return launch<T, kMode, 128>(n);
    case 256: return launch<T, kMode, 256>(n);
    default: return launch<T, kMode, 0>(n);
    }
}
template <typename T>
cudaError_t launch_t(NormArgs& n)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    if (!n.rope.half_style) return launch_d<T, kInterleaved>(n);
    return n.rope.rot / 2 % N == 0 ? launch_d<T, kHalf>(n) : launch_d<T, kExchange>(n);
}

}  // namespace
}  // namespace ra
