// paged_cluster.cuh -- calls of paged_attn_tree_fwd with few tiles: a cluster of CTAs for every
// tile, whose parts of the keys are joined through the cluster's shared memory.
#pragma once

#include "paged_plan.cuh"

namespace ra {

constexpr int kMostCtas = 16;                  // of a cluster

__device__ __forceinline__ float4 load_remote4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 load_remote2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// This cluster's tile (of p.grid CTAs), found by each warp for itself: the tiles lie one after the
// other, sequence by sequence, head by head.  Returns its sequence, or -1 if there is none left.
template <int kRows>
__device__ __forceinline__ int cluster_tile(const PagedParams& p, TileRows& t, SeqSpan& span)
{
    const PagedArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    int rest = static_cast<int>(blockIdx.x) / p.grid;
#pragma unroll 1
    for (int base = 0; base < a.n_seqs; base += 32) {
        SeqSpan mine{};
        int tiles = 0;
        if (base + lane < a.n_seqs) {
            mine = seq_span_of(a, base + lane);
            tiles = (mine.n * p.G + kRows - 1) / kRows * a.H_kv;
        }
        int inc = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned holds = __ballot_sync(0xffffffffu, inc > rest);
        if (holds == 0) {
            rest -= __shfl_sync(0xffffffffu, inc, 31);
            continue;
        }
        const int k = __ffs(holds) - 1;
        rest -= __shfl_sync(0xffffffffu, inc - tiles, k);
        span.first = __shfl_sync(0xffffffffu, mine.first, k);
        span.n = __shfl_sync(0xffffffffu, mine.n, k);
        span.kv = __shfl_sync(0xffffffffu, mine.kv, k);
        const int per_head = __shfl_sync(0xffffffffu, tiles, k) / a.H_kv;
        t.first = span.first;
        t.hk = rest / per_head;
        t.row0 = (rest - t.hk * per_head) * kRows;
        t.rows = min(kRows, span.n * p.G - t.row0);
        return base + k;
    }
    return -1;
}

// End of a tile, by all of its cluster: buf[rows][ldo] holds a CTA's unnormalised sums and stat[rows]
// = (maximum in base-2 units, denominator), in the same place of every CTA's shared memory.  The
// CTAs' parts are joined in their order; rows rank, rank + ctas, ... are this CTA's, kRowLanes lanes
// (kVec4 times four columns each) a row.  No CTA returns while others read its parts.
template <typename T, int kVec4, int kRowLanes>
__device__ __forceinline__ void join_cluster(const PagedParams& p, const TileRows& t, const float* buf,
                                             int ldo, const float2* stat, int warp, int n_warps)
{
    static_assert(kRowLanes >= kMostCtas, "a lane for every part's statistics");
    constexpr int kAbreast = 32 / kRowLanes;
    const int lane = threadIdx.x & 31, sub = lane / kRowLanes, c = lane % kRowLanes;
    const int ctas = p.grid, rank = static_cast<int>(cluster_ctarank());
    const uint32_t buf_s = smem_addr(buf), stat_s = smem_addr(stat);
    cluster_sync_all();
#pragma unroll 1
    for (int r0 = rank + ctas * warp * kAbreast; r0 < t.rows; r0 += ctas * n_warps * kAbreast) {
        const int r = r0 + ctas * sub;
        const bool mine = r < t.rows;
        // (all reads of a batch first: a read of another CTA's shared memory takes some 200 ns)
        constexpr int kBatch = 8;
        float2 st = make_float2(-INFINITY, 0.f);
        if (mine && c < ctas) st = load_remote2(mapa_shared(stat_s + 8 * r, c));
        float4 y[kBatch][kVec4];
        auto read = [&](int k0) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (!mine || k0 + k >= ctas) continue;
#pragma unroll
                for (int u = 0; u < kVec4; ++u)
                    y[k][u] = load_remote4(mapa_shared(buf_s + (r * ldo + 4 * (c + kRowLanes * u)) * 4, k0 + k));
            }
        };
        read(0);
        float M = st.x;
#pragma unroll
        for (int w = kRowLanes / 2; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
        const float f = st.y == 0.f ? 0.f : part_weight(st.x, st.y, M), fl = st.y == 0.f ? 0.f : f * st.y;
        float L = 0.f;
        float4 x[kVec4];
#pragma unroll
        for (int u = 0; u < kVec4; ++u) x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = 0; k0 < ctas; k0 += kBatch) {
            if (k0 > 0) read(k0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float w = __shfl_sync(0xffffffffu, f, sub * kRowLanes + ((k0 + k) & (kMostCtas - 1)));
                L += __shfl_sync(0xffffffffu, fl, sub * kRowLanes + ((k0 + k) & (kMostCtas - 1)));
                if (!mine || k0 + k >= ctas) continue;
#pragma unroll
                for (int u = 0; u < kVec4; ++u) {
                    x[u].x = fmaf(w, y[k][u].x, x[u].x);
                    x[u].y = fmaf(w, y[k][u].y, x[u].y);
                    x[u].z = fmaf(w, y[k][u].z, x[u].z);
                    x[u].w = fmaf(w, y[k][u].w, x[u].w);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kVec4; ++u)
            if (mine && 4 * (c + kRowLanes * u) < p.a.D) write_row4<T>(p, t, r, c + kRowLanes * u, x[u], M, L);
    }
    cluster_sync_all();
}

// At most so many tiles of `of` rows does a call have, whatever its lengths are.
inline long long most_tiles(const PagedArgs& a, int of)
{
    const long long rows = static_cast<long long>(a.T) * (a.H / a.H_kv);
    return a.H_kv * ((rows + a.n_seqs * (of - 1ll)) / of);
}

// Clusters of `ctas` CTAs that the current device holds at once, asked once per device (known: 0,
// not asked yet).
template <typename Kernel>
cudaError_t clusters_held(std::atomic<int>* known, Kernel kernel, int threads, int bytes, int ctas,
                          int* clusters)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    *clusters = known[dev].load(std::memory_order_acquire) - 1;
    if (*clusters >= 0) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(ctas);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = bytes;
    config.attrs = &at;
    config.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(clusters, kernel, &config);
    if (e != cudaSuccess) {
        cudaGetLastError();                     // (a size that the GPU does not take)
        *clusters = 0;
    }
    known[dev].store(*clusters + 1, std::memory_order_release);
    return cudaSuccess;
}

// Launches a kernel on clusters of `ctas` CTAs, one for each of `tiles` tiles, as launch_early does.
template <typename Kernel>
cudaError_t launch_clusters(Kernel kernel, PagedParams& p, long long tiles, int ctas, int threads, int bytes)
{
    p.grid = ctas;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(static_cast<unsigned>(tiles) * ctas);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = bytes;
    config.stream = p.a.stream;
    config.attrs = at;
    config.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&config, kernel, p);
    if (e != cudaSuccess) cudaGetLastError();       // reported here, not to the next caller who asks
    return e;
}

}  // namespace ra
