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
// them.  A warp takes as many head vectors at once as its lanes hold (a round) and a token's
// rounds one after the other, or in small calls a part of them; it works out the token's
// position, sines and cosines for itself, once for all its rounds, while the first of these are
// on their way, and meets no barrier but the weights'.  In the half style with a rot/2 that is no
// multiple of the vector the lanes exchange their elements through shared memory.
//
// Measured: 32768 tokens of 32 and 8 heads of 128 in bf16 100 us, 6.7 TB/s, the copy rate; 8192
// tokens of the same heads appended to pages 37 us, 5.4 TB/s (launch 2, and the positions: rows
// starts and lengths, then the page, before a token's first store); one decoding step of 64
// tokens 2.9 us.  16384 tokens of 12 and 4 heads of 128, 96, 80, 64 dims 5.4, 4.0, 3.4, 4.7 TB/s
// (their angles serve few heads, and 6 or 5 of 8 lanes work at 96 and 80), of 112 and 192, known at
// run time only, 3.6 and 3.8; with halves that are no whole vectors 1.7 to 2.9, at run time 1.3 to
// 1.9.  In fp32 the 32768 tokens 199 us, 6.7 TB/s, the appended ones 64, 6.3 TB/s.
#include "qk_norm.cuh"

namespace ra {
namespace {

// kD: the head dim, or 0 for any.
template <typename T, Mode kMode, int kD, bool kPaged>
__global__ void __launch_bounds__(kFwdThreads, kPaged ? kPagedBlocks : kFwdBlocks) norm_fwd_kernel(const __grid_constant__ NormArgs n)
{
    constexpr int N = 16 / sizeof(T);
    constexpr int kAhead = kPaged ? kPagedAhead : kFwdAhead;
    __shared__ Smem<T, kMode, kFwdThreads / 32, false> s;
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
            if (kFull || c0 >= 0) r.x0 = *reinterpret_cast<const Vec<T>*>(from.p + c0);
            if (kFull || c1 >= 0) r.x1 = *reinterpret_cast<const Vec<T>*>(from.p + c1);
        }
        advance(from, n, in, abreast);
    };
    wait_for_earlier_work();
    // the first rounds are on their way while the weights, positions and angles are worked out
    Row r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(r[u]);
    Weights<kMode, N, kFwdThreads> weights;
    weights.fetch(n, D, lanes, items);
    Cursor<T> to = cursor_at<T>(share, n, out, sub, abreast);
    const TokenPos pos = token_pos<kPaged>(a, to.t);
    weights.store(s.weight, lanes);
    angles<kMode, N>(a, s.cos_s[warp], s.sin_s[warp], pos.pos, lanes, items);
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
        turn<kMode, N, 1>(f, s.cos_s[warp], s.sin_s[warp], a.rot, item, c0, c1, lanes, items, row);
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
            if (kFull || c0 >= 0) *reinterpret_cast<Vec<T>*>(dst + c0) = r.x0;
            if (kFull || c1 >= 0) *reinterpret_cast<Vec<T>*>(dst + c1) = r.x1;
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
cudaError_t launch(NormArgs& n)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    RopeArgs& a = n.rope;
    n.items = items_of<kMode, N>(a.D, a.rot);
    n.lanes = lanes_for(n.items);
    const int abreast = 32 / n.lanes;
    const int heads = a.H + (a.paged ? 2 : 1) * a.H_kv;
    n.per_token = (heads + abreast - 1) / abreast;
    static std::atomic<int> known[2][kMaxDevices];
    const auto kernel = a.paged ? norm_fwd_kernel<T, kMode, kD, true> : norm_fwd_kernel<T, kMode, kD, false>;
    constexpr int warps = kFwdThreads / 32;
    int slots = 0;                                  // blocks that the GPU holds at once
    const cudaError_t e = resident_ctas(known[a.paged ? 1 : 0], kernel, kFwdThreads, 0, &slots);
    if (e != cudaSuccess) return e;
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
    return launch_early(kernel, grid, kFwdThreads, 0, a.stream, n);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& args)
{
    NormArgs n = args;
    return n.rope.elem == 2 ? launch_t<__nv_bfloat16>(n) : launch_t<float>(n);
}

}  // namespace ra
