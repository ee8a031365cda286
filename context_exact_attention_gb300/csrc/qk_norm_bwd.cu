// qk_norm_bwd.cu -- gradients of normalised and rotated heads (qk_norm_rope_bwd): the mathematics and
// the layout stand in qk_norm.cu.
//
// The weights' gradients: a lane keeps its columns' sums over all its rows in registers; the
// lanes of a block are added through shared memory, and the blocks' sums through the workspace, in
// two steps of a fixed order, so that repeated calls give the same bits.
//
// What bounds it: HBM and instructions, 330 of a warp for a round's 12 KB at head dim 128, of which
// the positions and angles, worked out for queries and for keys, are 60 (16381 packed tokens of 32
// and 8 heads of 128 in bf16: 90 us, 5.6 TB/s; 52 % of the issue slots; in fp32 167 us, 6.0 TB/s).
#include "qk_norm.cuh"

namespace ra {
namespace {

template <typename T, Mode kMode, int kD>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks) norm_bwd_kernel(const __grid_constant__ NormArgs n)
{
    constexpr int N = 16 / sizeof(T);
    constexpr int kAhead = kBwdAhead;
    constexpr int kWarps = kBwdThreads / 32;
    __shared__ Smem<T, kMode, kWarps, true> s;
    const RopeArgs& a = n.rope;
    constexpr int kItems = kItemsOf<T, kD>, kLanes = kD ? lanes_for(kItems) : 0;
    constexpr bool kFull = kD && kLanes == kItems;     // every lane holds two vectors
    const int lanes = kD ? kLanes : n.lanes, abreast = 32 / lanes, D = kD ? kD : a.D;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = lane & (lanes - 1), sub = lane / lanes;
    const int items = kD ? kItems : n.items;
    int c0, c1;
    columns_of<kMode, N>(D, a.rot, item, items, c0, c1);
    float* row = s.exchange[kMode == kExchange ? warp : 0] + (kMode == kExchange ? sub * 2 * items : 0);
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
                if (kFull || c0 >= 0) {
                    r.x0 = *reinterpret_cast<const Vec<T>*>(X + xi + c0);
                    r.y0 = *reinterpret_cast<const Vec<T>*>(Y + yi + c0);
                }
                if (kFull || c1 >= 0) {
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
            weights.fetch(n, D, lanes, items);
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
                angles<kMode, N>(a, s.cos_s[warp], s.sin_s[warp], pos.pos, lanes, items);
            }
            uint64_t x[N], z[N], w[N];
            widen(r.x0, x);
            widen(r.x1, x + N / 2);
            widen(r.y0, z);
            widen(r.y1, z + N / 2);
            turn<kMode, N, -1>(z, s.cos_s[warp], s.sin_s[warp], a.rot, item, c0, c1, lanes, items, row);
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
            // - mean(g o u); u = 0 in a head whose squares' sum is infinite, though the sum of
            // products may be, too
            const float c = rs == 0.f ? 0.f : -(product * rs * over_D);
            const uint64_t rr = f2pack(rs, rs), cc = f2pack(c, c);
            if (live && j * abreast + sub < heads) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    x[i] = fmul2(x[i], rr);                         // u
                    dw[i] = ffma2(z[i], x[i], dw[i]);
                    z[i] = fmul2(rr, ffma2(x[i], cc, w[i]));
                }
                if (in_bounds(di, D, extent_d, a.status)) {
                    if (kFull || c0 >= 0) *reinterpret_cast<Vec<T>*>(DX + di + c0) = narrow<T>(z);
                    if (kFull || c1 >= 0) *reinterpret_cast<Vec<T>*>(DX + di + c1) = narrow<T>(z + N / 2);
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
                if (kFull || c0 >= 0) *reinterpret_cast<uint64_t*>(&s.sums[warp][c0 + 2 * i]) = dw[i];
                if (kFull || c1 >= 0) *reinterpret_cast<uint64_t*>(&s.sums[warp][c1 + 2 * i]) = dw[N / 2 + i];
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
cudaError_t launch(NormArgs& n)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    RopeArgs& a = n.rope;
    n.items = items_of<kMode, N>(a.D, a.rot);
    n.lanes = lanes_for(n.items);
    const int abreast = 32 / n.lanes;
    static std::atomic<int> known[kMaxDevices];
    int slots = 0;                                  // blocks that the GPU holds at once
    const cudaError_t e = resident_ctas(known, norm_bwd_kernel<T, kMode, kD>, kBwdThreads, 0, &slots);
    if (e != cudaSuccess) return e;
    const long long rounds = a.rows * ((std::max(a.H, a.H_kv) + abreast - 1) / abreast);
    constexpr int warps = kBwdThreads / 32;
    const unsigned grid =
        static_cast<unsigned>(std::min<long long>((rounds + warps - 1) / warps, std::min(slots, kNormCtas)));
    return launch_early(norm_bwd_kernel<T, kMode, kD>, grid, kBwdThreads, 0, a.stream, n);
}

}  // namespace

cudaError_t launch_norm_bwd(const NormArgs& args)
{
    NormArgs n = args;
    return n.rope.elem == 2 ? launch_t<__nv_bfloat16>(n) : launch_t<float>(n);
}

}  // namespace ra
