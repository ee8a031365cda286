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
// them.  A block takes a few tokens, works out their sines and cosines once for all heads, and
// streams the heads with two rows in flight per lane.  In the half style with a rot/2 that is
// no multiple of the vector the lanes exchange their elements through shared memory.
//
// The weights' gradients: a lane keeps its columns' sums over all its rows in registers; the
// lanes of a block are added through shared memory, a block's sums go to the workspace, and
// the last block to arrive adds them up in block order, so that repeated calls give the same bits.
#include <algorithm>

#include "rope_pos.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 2048;     // sines and cosines of one block: tokens * rot / 2
constexpr int kMaxTokens = 32;
constexpr int kAhead = 2;           // rows in flight per group of lanes

enum Mode { kHalf, kInterleaved, kExchange };

// 16 bytes of a row, and as fp32.
template <typename T>
struct alignas(16) Vec {
    T e[16 / sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void widen(const Vec<T>& v, float* f)
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v.e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = v.e[i];
    }
}
// The one rounding (nearest even).
template <typename T>
__device__ __forceinline__ Vec<T> narrow(const float* f)
{
    Vec<T> v;
    if constexpr (sizeof(T) == 2) {
        uint32_t* w = reinterpret_cast<uint32_t*>(v.e);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v.e[i] = f[i];
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

template <typename T, Mode kMode, bool kBack>
struct alignas(16) Smem {
    float cos_s[kMaxPairs];
    float sin_s[kMaxPairs];
    float weight[2][256];
    float exchange[kMode == kExchange ? kWarps : 1][kMode == kExchange ? 32 * 2 * (16 / sizeof(T)) : 1];
    float sums[kBack ? kWarps : 1][kBack ? 256 : 1];
    TokenPos tok[kMaxTokens];
    int last;
};

// The rotation of a lane's elements f (N of vector c0, N of c1), sines times `sign`.  `row`: the
// lanes' exchange area for this head vector (kExchange).  All lanes of the warp take part.
template <Mode kMode, int N>
__device__ __forceinline__ void turn(float* f, const float* cs, const float* sn, int rot, int item, int c0,
                                     int c1, float sign, float* row)
{
    const int half = rot / 2;
    if constexpr (kMode == kHalf) {
        const int turning = half / N;
        if (item >= turning) return;
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            const float4 c4 = *reinterpret_cast<const float4*>(cs + 4 * (q * turning + item));
            const float4 s4 = *reinterpret_cast<const float4*>(sn + 4 * (q * turning + item));
            const float c[4] = {c4.x, c4.y, c4.z, c4.w};
            const float s[4] = {s4.x * sign, s4.y * sign, s4.z * sign, s4.w * sign};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = f[4 * q + i], b = f[N + 4 * q + i];
                f[4 * q + i] = fmaf(a, c[i], -(b * s[i]));
                f[N + 4 * q + i] = fmaf(b, c[i], a * s[i]);
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
                const float c = cs[p0 + i], s = sn[p0 + i] * sign;
                const float a = f[N * v + 2 * i], b = f[N * v + 2 * i + 1];
                f[N * v + 2 * i] = fmaf(a, c, -(b * s));
                f[N * v + 2 * i + 1] = fmaf(b, c, a * s);
            }
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int at = v ? c1 : c0;
            if (at < 0) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) row[at + i] = f[N * v + i];
        }
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int at = v ? c1 : c0;
            if (at < 0) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = at + i;
                if (e >= rot) continue;
                const bool first = e < half;
                const int pair = first ? e : e - half;
                const float other = row[first ? e + half : e - half];
                const float s = first ? -sn[pair] : sn[pair];
                f[N * v + i] = fmaf(f[N * v + i], cs[pair], other * (s * sign));
            }
        }
    }
}

// Sines and cosines (times the amplitude) of n_tok tokens from t0 on, and where they stand.
template <typename T, Mode kMode, bool kPaged, typename S>
__device__ __forceinline__ void angles(const RopeArgs& a, S& s, long long t0, int n_tok)
{
    constexpr int N = 16 / sizeof(T);
    const int half = a.rot / 2, turning = half / N;
    for (int i = threadIdx.x >> 5; i < n_tok; i += kWarps) {
        const TokenPos p = token_pos<kPaged>(a, t0 + i);
        if ((threadIdx.x & 31) == 0) s.tok[i] = p;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * half; i += kThreads) {
        const int tk = i / half, pair = i - tk * half;
        unsigned long long ph = 0;
        if (in_bounds(pair, 1, half, a.status)) ph = __ldg(a.phases + pair);
        float sn, cs;
        angle_of(ph, s.tok[tk].pos, sn, cs);
        // (half style: in groups of four, group q of an item behind group q of all items, so
        // that neighbouring lanes read neighbouring groups)
        int at = tk * half + pair;
        if (kMode == kHalf) {
            const int item = pair / N, in = pair % N;
            at = tk * half + ((in / 4) * turning + item) * 4 + in % 4;
        }
        s.cos_s[at] = cs * a.amplitude;
        s.sin_s[at] = sn * a.amplitude;
    }
    __syncthreads();
}

// The weights of this lane's columns, from shared memory (as they lie in the head vector).
template <int N>
__device__ __forceinline__ void weights_of(const float* w, int c0, int c1, float* out)
{
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int c = v ? c1 : c0;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(w + max(c, 0) + i);
            out[N * v + i] = x.x;
            out[N * v + i + 1] = x.y;
            out[N * v + i + 2] = x.z;
            out[N * v + i + 3] = x.w;
        }
    }
}

// Sum over the lanes of a head vector.
__device__ __forceinline__ float lanes_sum(float x, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename S>
__device__ __forceinline__ void load_weights(const NormArgs& n, S& s)
{
    for (int i = threadIdx.x; i < 2 * n.rope.D; i += kThreads) {
        const int which = i / n.rope.D, c = i - which * n.rope.D;
        const void* w = which ? n.k_weight : n.q_weight;
        float x = 1.f;
        if (w != nullptr && in_bounds(c, 1, n.rope.D, n.rope.status))
            x = (n.weight_elem == 2 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c])
                                    : static_cast<const float*>(w)[c]) +
                n.weight_offset;
        s.weight[which][c] = x;
    }
}

// Walk over the rows (token, head) of a block: a group of lanes takes every groups-th.
struct Rows {
    int tok, h, heads, step_t, step_h;
    __device__ __forceinline__ void begin(int group, int groups, int n_heads)
    {
        heads = n_heads;
        tok = group / heads;
        h = group - tok * heads;
        step_t = groups / heads;
        step_h = groups - step_t * heads;
    }
    __device__ __forceinline__ void advance()
    {
        tok += step_t;
        h += step_h;
        if (h >= heads) {
            h -= heads;
            ++tok;
        }
    }
};

template <typename T, Mode kMode, bool kPaged>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const __grid_constant__ NormArgs n)
{
    constexpr int N = 16 / sizeof(T);
    __shared__ Smem<T, kMode, false> s;
    const RopeArgs& a = n.rope;
    const int heads = a.H + (kPaged ? 2 : 1) * a.H_kv;
    const int lanes = n.lanes, groups = kThreads / lanes;
    const int lane = threadIdx.x & 31, item = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
    int c0, c1;
    columns_of<kMode, N>(a.D, a.rot, item, n.items, c0, c1);
    float* row = s.exchange[kMode == kExchange ? threadIdx.x >> 5 : 0] +
                 (kMode == kExchange ? (lane / lanes) * lanes * 2 * N : 0);
    const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
    const int n_tok = static_cast<int>(min(static_cast<long long>(a.tokens), a.rows - t0));
    const float over_D = 1.f / a.D;

    struct Row {
        Vec<T> x0, x1;
        int tok, h;
    };
    Rows walk;
    walk.begin(group, groups, heads);
    auto fetch = [&](Row& r) {
        r.tok = walk.tok;
        r.h = walk.h;
        walk.advance();
        r.x0 = Vec<T>{};
        r.x1 = Vec<T>{};
        if (r.tok >= n_tok) return;
        const int kind = r.h < a.H ? 0 : r.h < a.H + a.H_kv ? 1 : 2;
        const int hh = r.h - (kind == 0 ? 0 : kind == 1 ? a.H : a.H + a.H_kv);
        const long long si = (t0 + r.tok) * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                             static_cast<long long>(hh) * a.D;
        const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + si;
        if (!in_bounds(si, a.D, kind == 0 ? a.q_elems : kind == 1 ? a.k_elems : a.v_elems, a.status)) return;
        if (c0 >= 0) r.x0 = *reinterpret_cast<const Vec<T>*>(src + c0);
        if (c1 >= 0) r.x1 = *reinterpret_cast<const Vec<T>*>(src + c1);
    };
    auto finish = [&](Row& r) {
        const bool real = r.tok < n_tok;
        const int kind = r.h < a.H ? 0 : r.h < a.H + a.H_kv ? 1 : 2;
        const int hh = r.h - (kind == 0 ? 0 : kind == 1 ? a.H : a.H + a.H_kv);
        const int tk = real ? r.tok : 0;
        float f[2 * N];
        widen(r.x0, f);
        widen(r.x1, f + N);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) ss = fmaf(f[i], f[i], ss);
        const float rs = rsqrtf(lanes_sum(ss, lanes) * over_D + n.eps);
        float w[2 * N];
        weights_of<N>(s.weight[kind == 0 ? 0 : 1], c0, c1, w);
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) f[i] = f[i] * rs * w[i];
        const int cs = tk * (a.rot / 2);
        turn<kMode, N>(f, s.cos_s + cs, s.sin_s + cs, a.rot, item, c0, c1, 1.f, row);
        if (!real) return;
        // (the paged append's values stay as they are)
        if (!kPaged || kind < 2) {
            r.x0 = narrow<T>(f);
            r.x1 = narrow<T>(f + N);
        }
        const TokenPos p = s.tok[tk];
        const bool to_page = kPaged && kind > 0;
        if (to_page ? p.slot < 0 : !p.live) return;
        const long long di = to_page ? p.slot + hh * a.head_stride
                                     : (t0 + tk) * (kind == 0 ? a.q_out_stride : a.k_out_stride) +
                                           static_cast<long long>(hh) * a.D;
        if (!in_bounds(di, a.D, kind == 0 ? a.q_out_elems : a.k_out_elems, a.status)) return;
        T* dst = static_cast<T*>(kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out) + di;
        if (c0 >= 0) *reinterpret_cast<Vec<T>*>(dst + c0) = r.x0;
        if (c1 >= 0) *reinterpret_cast<Vec<T>*>(dst + c1) = r.x1;
    };

    wait_for_earlier_work();
    // the first rows are on their way while the positions and angles are worked out
    Row r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(r[u]);
    load_weights(n, s);
    angles<T, kMode, kPaged>(a, s, t0, n_tok);
    while (__any_sync(0xffffffffu, r[0].tok < n_tok)) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            finish(r[u]);
            fetch(r[u]);
        }
    }
}

template <typename T, Mode kMode>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const __grid_constant__ NormArgs n)
{
    constexpr int N = 16 / sizeof(T);
    __shared__ Smem<T, kMode, true> s;
    const RopeArgs& a = n.rope;
    const int lanes = n.lanes, groups = kThreads / lanes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
    int c0, c1;
    columns_of<kMode, N>(a.D, a.rot, item, n.items, c0, c1);
    float* row = s.exchange[kMode == kExchange ? warp : 0] +
                 (kMode == kExchange ? (lane / lanes) * lanes * 2 * N : 0);
    const float over_D = 1.f / a.D;

    struct Row {
        Vec<T> x0, x1, y0, y1;
        int tok, h;
    };
    wait_for_earlier_work();
    load_weights(n, s);
    __syncthreads();
    // queries, then keys: a lane's columns of dw stay in registers
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const int heads = kind ? a.H_kv : a.H;
        if (heads == 0) continue;
        const T* X = static_cast<const T*>(kind ? a.k : a.q);
        const T* Y = static_cast<const T*>(kind ? n.dk_out : n.dq_out);
        T* DX = static_cast<T*>(kind ? a.k_out : a.q_out);
        const long long x_step = kind ? a.k_stride : a.q_stride;
        const long long y_step = kind ? n.dk_out_stride : n.dq_out_stride;
        const long long d_step = kind ? a.k_out_stride : a.q_out_stride;
        float w[2 * N], dw[2 * N];
        weights_of<N>(s.weight[kind], c0, c1, w);
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) dw[i] = 0.f;
        for (long long t0 = static_cast<long long>(blockIdx.x) * a.tokens; t0 < a.rows;
             t0 += static_cast<long long>(gridDim.x) * a.tokens) {
            const int n_tok = static_cast<int>(min(static_cast<long long>(a.tokens), a.rows - t0));
            Rows walk;
            walk.begin(group, groups, heads);
            auto fetch = [&](Row& r) {
                r.tok = walk.tok;
                r.h = walk.h;
                walk.advance();
                r.x0 = r.x1 = r.y0 = r.y1 = Vec<T>{};
                if (r.tok >= n_tok) return;
                const long long at = static_cast<long long>(r.h) * a.D;
                const long long xi = (t0 + r.tok) * x_step + at, yi = (t0 + r.tok) * y_step + at;
                if (!in_bounds(xi, a.D, kind ? a.k_elems : a.q_elems, a.status) ||
                    !in_bounds(yi, a.D, kind ? n.dk_out_elems : n.dq_out_elems, a.status))
                    return;
                if (c0 >= 0) {
                    r.x0 = *reinterpret_cast<const Vec<T>*>(X + xi + c0);
                    r.y0 = *reinterpret_cast<const Vec<T>*>(Y + yi + c0);
                }
                if (c1 >= 0) {
                    r.x1 = *reinterpret_cast<const Vec<T>*>(X + xi + c1);
                    r.y1 = *reinterpret_cast<const Vec<T>*>(Y + yi + c1);
                }
            };
            auto finish = [&](Row& r) {
                const bool real = r.tok < n_tok && s.tok[min(r.tok, n_tok - 1)].live;
                float x[2 * N], z[2 * N];
                widen(r.x0, x);
                widen(r.x1, x + N);
                widen(r.y0, z);
                widen(r.y1, z + N);
                const int cs = min(r.tok, n_tok - 1) * (a.rot / 2);
                turn<kMode, N>(z, s.cos_s + cs, s.sin_s + cs, a.rot, item, c0, c1, -1.f, row);
                // (the amplitude is in the sines and cosines; the dims behind rot have none)
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) {
                    ss = fmaf(x[i], x[i], ss);
                    dot = fmaf(w[i] * z[i], x[i], dot);
                }
                ss = lanes_sum(ss, lanes);
                dot = lanes_sum(dot, lanes);
                const float rs = rsqrtf(ss * over_D + n.eps);
                const float c = dot * rs * over_D;               // mean(g o u)
                if (!real) return;
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) {
                    const float u = x[i] * rs;
                    dw[i] = fmaf(z[i], u, dw[i]);
                    z[i] = rs * fmaf(-u, c, w[i] * z[i]);
                }
                const long long di = (t0 + r.tok) * d_step + static_cast<long long>(r.h) * a.D;
                if (!in_bounds(di, a.D, kind ? a.k_out_elems : a.q_out_elems, a.status)) return;
                if (c0 >= 0) *reinterpret_cast<Vec<T>*>(DX + di + c0) = narrow<T>(z);
                if (c1 >= 0) *reinterpret_cast<Vec<T>*>(DX + di + c1) = narrow<T>(z + N);
            };
            Row r[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) fetch(r[u]);
            __syncthreads();                // the tokens before are done with
            angles<T, kMode, false>(a, s, t0, n_tok);
            while (__any_sync(0xffffffffu, r[0].tok < n_tok)) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    finish(r[u]);
                    fetch(r[u]);
                }
            }
        }
        // this block's sums: over a warp's groups, then over the warps in order
#pragma unroll
        for (int i = 0; i < 2 * N; ++i)
            for (int o = lanes; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
        if (lane < lanes) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (c0 >= 0) s.sums[warp][c0 + i] = dw[i];
                if (c1 >= 0) s.sums[warp][c1 + i] = dw[N + i];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) x += s.sums[i][c];
            const long long at = (static_cast<long long>(blockIdx.x) * 2 + kind) * 256 + c;
            if (in_bounds(at, 1, 512ll * kNormCtas, a.status)) __stcg(n.partials + at, x);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        unsigned before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                     : "=r"(before)
                     : "l"(n.ticket)
                     : "memory");
        s.last = before == gridDim.x - 1;
        if (s.last) *n.ticket = 0;
    }
    __syncthreads();
    if (!s.last) return;
    // eight warps take every eighth block's sums of a column, in order, then these in order
    for (int kind = 0; kind < 2; ++kind) {
        float* dst = kind ? n.dk_weight : n.dq_weight;
        if (dst == nullptr) continue;
        for (int c = lane; c < a.D; c += 32) {
            float x = 0.f;
#pragma unroll 8
            for (int b = warp; b < gridDim.x; b += kWarps) {
                const long long at = (static_cast<long long>(b) * 2 + kind) * 256 + c;
                if (in_bounds(at, 1, 512ll * kNormCtas, a.status)) x += __ldcg(n.partials + at);
            }
            s.sums[warp][c] = x;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) x += s.sums[i][c];
            if (in_bounds(c, 1, a.D, a.status)) dst[c] = x;
        }
        __syncthreads();
    }
}

// Tokens of a block, such that the blocks fill the GPU a few times over and every group of
// lanes has several rows.
int tokens_of(const RopeArgs& a, int heads, int groups, int slots)
{
    int most = kMaxTokens;
    if (a.rot > 0) most = std::min(most, kMaxPairs / (a.rot / 2));
    const long long waves = (a.rows + slots - 1) / slots;        // tokens a block, in one wave
    const long long rows = (8ll * groups + heads - 1) / heads;   // tokens that give 8 rows a group
    return static_cast<int>(std::max(1ll, std::min<long long>(most, std::min(waves, rows))));
}

template <typename T, Mode kMode>
cudaError_t launch(NormArgs& n, bool backward)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    RopeArgs& a = n.rope;
    n.items = items_of<kMode, N>(a.D, a.rot);
    n.lanes = 1;
    while (n.lanes < n.items) n.lanes *= 2;
    const int groups = kThreads / n.lanes;
    static std::atomic<int> known[3][kMaxDevices];
    int slots = 0;
    if (backward) {
        cudaError_t e = resident_ctas(known[2], norm_bwd_kernel<T, kMode>, kThreads, 0, &slots);
        if (e != cudaSuccess) return e;
        slots = std::min(slots, kNormCtas);
        a.tokens = tokens_of(a, std::max(a.H, a.H_kv), groups, slots);
        const long long chunks = (a.rows + a.tokens - 1) / a.tokens;
        const unsigned grid = static_cast<unsigned>(std::min<long long>(chunks, slots));
        return launch_early(norm_bwd_kernel<T, kMode>, grid, kThreads, 0, a.stream, n);
    }
    const cudaError_t e =
        a.paged ? resident_ctas(known[1], norm_fwd_kernel<T, kMode, true>, kThreads, 0, &slots)
                : resident_ctas(known[0], norm_fwd_kernel<T, kMode, false>, kThreads, 0, &slots);
    if (e != cudaSuccess) return e;
    a.tokens = tokens_of(a, a.H + (a.paged ? 2 : 1) * a.H_kv, groups, slots);
    const long long blocks = (a.rows + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_early(a.paged ? norm_fwd_kernel<T, kMode, true> : norm_fwd_kernel<T, kMode, false>,
                        static_cast<unsigned>(blocks), kThreads, 0, a.stream, n);
}

template <typename T>
cudaError_t launch_t(NormArgs& n, bool backward)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const RopeArgs& a = n.rope;
    if (!a.half_style) return launch<T, kInterleaved>(n, backward);
    return a.rot / 2 % N == 0 ? launch<T, kHalf>(n, backward) : launch<T, kExchange>(n, backward);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& args, bool backward)
{
    NormArgs n = args;
    return n.rope.elem == 2 ? launch_t<__nv_bfloat16>(n, backward) : launch_t<float>(n, backward);
}

}  // namespace ra
