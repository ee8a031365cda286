// paged_attn_simt.cu -- paged_attn_fwd without tensor cores: fp32 caches, few query rows per
// key/value head.
//
// One block holds four query rows of one key/value head in registers (a lane keeps four
// consecutive columns of each) and its four warps walk the CTA's part of the keys in turns
// of eight.  A lane copies its own columns of a turn's keys and values into its warp's
// shared-memory ring asynchronously, turns ahead (no lane reads another's copies, so nothing
// is synchronised), and uses every element for four rows.  The 32 dot products of a turn (8
// keys x 4 rows) are partial sums over columns in every lane; a butterfly that halves the
// values at each step leaves the total of (key, row) in lane 4 key + row with 31 shuffles,
// where reducing them one by one would take 160.  That lane then owns the score: mask,
// maximum over the keys (three shuffles), exponential, and the eight weights of a row are
// read back by shuffle for the value sum.
//
// What bounds it: bytes, for up to four rows a head and long contexts.  A turn moves 8 keys (8
// KB at D 128), which HBM delivers to an SM in about 350 cycles, for about 600 warp
// instructions of one dependent chain, some 3000 cycles; so it takes many warps, and three
// blocks of two stages do better than two of three (same bytes in flight): 40 tokens over 405
// keys of 8 heads of 64, G 5, 41 us against 48, 195 tokens over 4763 keys of 8 heads 240
// against 273, the case below 26.5 against 26.3.  More rows per head are taken four at a
// time and re-read the keys, which then come from L2 (many more: paged_attn_simt_rows.cu).
// Measured: 16 single tokens over 100 to 4000 keys of 2 heads of 128 (91 MB) in 26 us, 3.5 TB/s:
// each warp has only five turns, and the call's fixed parts (plan, first reads, joining,
// launch: about 10 us) show.  Loading straight into registers, a turn at a time, took 33 to 37.
#include "paged_plan.cuh"

namespace ra {
namespace {

constexpr int kRows = 4;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTurn = 8;                       // keys per warp and turn
constexpr int kUnit = kTurn * kWarps;

constexpr int kStages = 2;                     // of a warp's ring: turns in flight

// A warp's ring: per stage the keys of a turn, then its values, float4 by lane.
template <int kVec4>
constexpr int kRing = kStages * 2 * kTurn * kVec4 * 32 * 16;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

// kTree: rows see the new tokens that their masks name.
template <int kVec4, bool kTree>
__global__ void __launch_bounds__(kThreads, kVec4 == 1 ? 3 : 1) paged_simt_kernel(const __grid_constant__ PagedParams p)
{
    using Walk = PagedWalk<FlatTiles<kRows>, kUnit>;
    __shared__ float2 stat_w[kWarps][kRows];
    __shared__ float2 stat[kRows];
    __shared__ int flag;
    __shared__ alignas(16) float4 part[kWarps][kRows][kVec4 * 32];   // the warps' sums; then the tile's
    const PagedArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.D;
    const float* Q = static_cast<const float*>(a.q);
    const float* K = static_cast<const float*>(a.k_pages);
    const float* V = static_cast<const float*>(a.v_pages);

    extern __shared__ __align__(16) uint8_t dyn[];
    uint8_t* ring = dyn + warp * kRing<kVec4> + lane * 16;
    const uint32_t ring_s = smem_addr(ring);
    constexpr int kHalf = kTurn * kVec4 * 512;     // bytes of a stage's keys

    wait_for_earlier_work();
    Walk walk;
    walk.begin(p);
    Segment t{}, nt{};                          // the segment being worked on, the next one
    bool have = false, have_next = walk.next(p, nt);
    // The copies: the warp's turn of the step at key `lk` of segment nt (in_next) or t, up to
    // kStages steps ahead.  They cross into the next segment but not beyond it.
    bool in_next = true;
    int lk = have_next ? nt.k0 : 0;
    uint32_t issued = 0, used = 0;
    long long off = -1;                         // lane < 8: where the turn's key lies
    auto look_up = [&]() {
        const int key = lk + kTurn * warp + lane;
        const int k1 = in_next ? (have_next ? nt.k1 : 0) : t.k1;
        off = -1;
        if (lane < kTurn && key < k1)
            off = key_offset(p, in_next ? nt.g : t.g, in_next ? nt.hk : t.hk, key);
    };
    auto loadable = [&]() { return lk < (in_next ? (have_next ? nt.k1 : 0) : t.k1); };
    auto issue = [&]() {
        const uint32_t dst = ring_s + (issued % kStages) * (2 * kHalf);
#pragma unroll
        for (int j = 0; j < kTurn; ++j) {
            const long long oj = __shfl_sync(0xffffffffu, off, j);
#pragma unroll
            for (int u = 0; u < kVec4; ++u) {
                const int c = 4 * (lane + 32 * u);
                const bool real = oj >= 0 && c < D && in_bounds(oj + c, 4, a.page_elems, a.status);
                const long long at = real ? oj + c : 0;
                cp_async16(dst + (j * kVec4 + u) * 512, K + at, real);
                cp_async16(dst + kHalf + (j * kVec4 + u) * 512, V + at, real);
            }
        }
        cp_async_commit();
        ++issued;
        lk += kUnit;
        if (!in_next && lk >= t.k1) {
            in_next = true;
            lk = have_next ? nt.k0 : 0;
        }
        look_up();
    };
    look_up();
    // the queries of segment nt, fetched a segment ahead
    float4 q_next[kRows][kVec4];
    auto fetch_q = [&]() {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int u = 0; u < kVec4; ++u) {
                const int c = 4 * (lane + 32 * u);
                q_next[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (have_next && r < nt.rows && c < D) {
                    const int pr = nt.row0 + r, tok = p.token_of(pr);
                    const long long at = (nt.s.first + tok) * a.q_stride +
                                         static_cast<long long>(nt.hk * p.G + (pr - tok * p.G)) * D + c;
                    if (in_bounds(at, 4, a.q_elems, a.status)) q_next[r][u] = load4(Q + at);
                }
            }
        }
    };
    fetch_q();
#pragma unroll 1
    for (;;) {
        if (have)
            finish_segment<float, kRows, kThreads, kVec4>(p, t, &part[0][0][0].x, kVec4 * 128, stat, &flag);
        have = have_next;
        if (!have) break;
        t = nt;
        have_next = walk.next(p, nt);
        in_next = lk >= t.k1;
        if (in_next) lk = have_next ? nt.k0 : 0;
        look_up();
        // pairs of columns: (0, 1) and (2, 3) of the four
        uint64_t q[kRows][kVec4][2], o[kRows][kVec4][2];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int u = 0; u < kVec4; ++u) {
                q[r][u][0] = f2pack(q_next[r][u].x, q_next[r][u].y);
                q[r][u][1] = f2pack(q_next[r][u].z, q_next[r][u].w);
                o[r][u][0] = o[r][u][1] = 0;
            }
        }
        fetch_q();
        // bits 4 j + r of the rows that the tile has
        const unsigned rows_in = 0x11111111u * ((1u << t.rows) - 1);
        // this lane's score is of row lane & 3: the keys it sees are [0, seen)
        const int my_row = lane & 3, my_key = lane >> 2;
        int seen = 0;                      // (of a tree: those from before the step)
        int my_token = -1;
        if (my_row < t.rows) {
            const int tok = p.token_of(t.row0 + my_row);
            my_token = t.s.first + tok;
            seen = kTree ? t.s.kv - t.s.n : a.causal ? t.s.kv - t.s.n + tok + 1 : t.s.kv;
        }
        float m = -INFINITY, l = 0.f;      // of row my_row; l over this lane's keys only
        for (int k = t.k0 + kTurn * warp; k - kTurn * warp < t.k1; k += kUnit) {
#pragma unroll 1
            while (issued - used < kStages && loadable()) issue();
            if (issued - used == kStages) cp_async_wait<kStages - 1>();
            else cp_async_wait<0>();
            const uint8_t* stage = ring + (used % kStages) * (2 * kHalf);
            ++used;
            auto key_at = [&](int j, int u) {
                return *reinterpret_cast<const ulonglong2*>(stage + (j * kVec4 + u) * 512);
            };
            auto value_at = [&](int j, int u) {
                return *reinterpret_cast<const ulonglong2*>(stage + kHalf + (j * kVec4 + u) * 512);
            };
            float s[32];
#pragma unroll
            for (int j = 0; j < kTurn; ++j) {
                ulonglong2 kk[kVec4];
#pragma unroll
                for (int u = 0; u < kVec4; ++u) kk[u] = key_at(j, u);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    uint64_t x = fmul2(q[r][0][0], kk[0].x);
                    x = ffma2(q[r][0][1], kk[0].y, x);
#pragma unroll
                    for (int u = 1; u < kVec4; ++u) {
                        x = ffma2(q[r][u][0], kk[u].x, x);
                        x = ffma2(q[r][u][1], kk[u].y, x);
                    }
                    float lo, hi;
                    f2unpack(x, lo, hi);
                    s[4 * j + r] = lo + hi;
                }
            }
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) {
                const bool up = lane & w;
#pragma unroll
                for (int i = 0; i < w; ++i) {
                    const float send = up ? s[i] : s[i + w];
                    const float keep = up ? s[i + w] : s[i];
                    s[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
            }
            const int key = k + my_key;
            bool sees = key < seen && key < t.k1;
            if (kTree && key >= seen && key < t.k1 && my_token >= 0)
                sees = seen_from(p, my_token, key - seen) & 1;
            const unsigned vis = __ballot_sync(0xffffffffu, sees);
            const float x = sees ? s[0] * p.scale_log2 : -INFINITY;
            float mx = x;
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float m_new = fmaxf(m, mx);
            const float alpha = m_new > m ? ex2(m - m_new) : 1.f;
            const float pe = ex2(x - (m_new == -INFINITY ? 0.f : m_new));
            l = l * alpha + pe;
            m = m_new;
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float ar = __shfl_sync(0xffffffffu, alpha, r);
#pragma unroll
                    for (int u = 0; u < kVec4; ++u) {
                        o[r][u][0] = fmul2(o[r][u][0], f2pack(ar, ar));
                        o[r][u][1] = fmul2(o[r][u][1], f2pack(ar, ar));
                    }
                }
            }
            // the values of key j, to the rows in `rows` (a bit each)
            auto add_value = [&](int j, unsigned rows) {
                ulonglong2 vv[kVec4];
#pragma unroll
                for (int u = 0; u < kVec4; ++u) vv[u] = value_at(j, u);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float w = __shfl_sync(0xffffffffu, pe, 4 * j + r);
                    if (!((rows >> r) & 1)) continue;
#pragma unroll
                    for (int u = 0; u < kVec4; ++u) {
                        o[r][u][0] = ffma2(f2pack(w, w), vv[u].x, o[r][u][0]);
                        o[r][u][1] = ffma2(f2pack(w, w), vv[u].y, o[r][u][1]);
                    }
                }
            };
            if ((~vis & rows_in) == 0) {
#pragma unroll
                for (int j = 0; j < kTurn; ++j) add_value(j, 15);
            } else {
                // a value that a row does not see stays out even if it is not finite
#pragma unroll 1
                for (int j = 0; j < kTurn; ++j) add_value(j, vis >> (4 * j));
            }
        }
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
        // the four warps' results, joined in warp order
        if (lane < kRows) stat_w[warp][lane] = make_float2(m, l);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int u = 0; u < kVec4; ++u) {
                float4 x;
                f2unpack(o[r][u][0], x.x, x.y);
                f2unpack(o[r][u][1], x.z, x.w);
                part[warp][r][lane + 32 * u] = x;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = threadIdx.x; i < kRows * kVec4 * 32; i += kThreads) {
            const int r = i / (kVec4 * 32), c = i % (kVec4 * 32);
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat_w[w][r].x);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 st = stat_w[w][r];
                const float f = part_weight(st.x, st.y, M);
                if (!(st.y == 0.f)) L += f * st.y;
                const float4 y = part[w][r][c];
                x.x = fmaf(f, y.x, x.x);
                x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z);
                x.w = fmaf(f, y.w, x.w);
            }
            part[0][r][c] = x;                     // (which only this thread has read)
            if (c == 0) stat[r] = make_float2(M, L);
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

}  // namespace

cudaError_t launch_paged_simt(const PagedArgs& a)
{
    PagedParams p;
    fill_params(&p, a);
    static std::atomic<int> known[4][kMaxDevices];
    const int which = (a.D <= 128 ? 0 : 2) + (a.masks ? 1 : 0);
    constexpr auto kOne = paged_simt_kernel<1, false>, kOneTree = paged_simt_kernel<1, true>;
    constexpr auto kTwo = paged_simt_kernel<2, false>, kTwoTree = paged_simt_kernel<2, true>;
    const auto kernel = a.D <= 128 ? (a.masks ? kOneTree : kOne) : (a.masks ? kTwoTree : kTwo);
    const int ring = kWarps * (a.D <= 128 ? kRing<1> : kRing<2>);
    int grid = 0;
    const cudaError_t e = resident_ctas(known[which], kernel, kThreads, ring, &grid);
    if (e != cudaSuccess) return e;
    p.grid = grid < kPagedMaxCtas ? grid : kPagedMaxCtas;
    p.tile_cost = 64;
    p.key_shift = 0;
    p.snap = 2 * kUnit;
    // 6 keys' time.  Measured without the rule and with 6 and 12: one token over 20000 keys of 2
    // heads and sequences 33.7, 29.5, 34.5 us, 30000 keys of one head, G 4, 30.6, 26.7, 31.1, 3000
    // of one head 11.7, 12.9, 13.9.
    p.join_cost = 6;
    p.whole = 140;                  // (4 single tokens over 50 to 100 keys: 9.0 us, 11.5 cut; 300: 0.6 to 1.0)
    p.min_chunk = 4 * kUnit;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const PagedWorkspace w = paged_workspace_of(p.grid, kRows, a.D);
    p.counters = reinterpret_cast<unsigned int*>(ws);
    p.part_stat = reinterpret_cast<float*>(ws + w.stat);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    return launch_early(kernel, p.grid, kThreads, ring, a.stream, p);
}

}  // namespace ra
