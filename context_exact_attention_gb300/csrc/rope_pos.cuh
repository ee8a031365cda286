// rope_pos.cuh -- what the kernels that rotate heads share: where a token row stands, the sine
// and cosine of its angles, conversions.
#pragma once

#include <cuda_bf16.h>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {

struct TokenPos {
    long long pos;      // position that it turns by
    long long slot;     // paged: element offset of the token's page slot, or -1 (not stored)
    int live;           // 0: the row belongs to no sequence and is left as it is
};

// One step of warp_upper: the answer lies in [lo, lo + len), before and afterwards.
__device__ __forceinline__ void warp_narrow(const int* v, int& lo, int& len, long long x, long long extent,
                                            unsigned int* status)
{
    const int lane = threadIdx.x & 31;
    const int step = (len + 31) / 32;
    const int j = lo + lane * step;
    const bool le = lane * step < len && checked_ldg(v, j, extent, status) <= x;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    const int k = cnt > 0 ? cnt - 1 : 0;
    lo += k * step;
    len = min(step, len - k * step);
}

// The largest j in [0, n) with v[j] <= x (0 if there is none) for a non-decreasing v, by
// one warp: every step loads 32 evenly spaced entries at once, so 1024 entries take two
// dependent loads where a binary search takes ten.
__device__ __forceinline__ int warp_upper(const int* v, int n, long long x, long long extent,
                                          unsigned int* status)
{
    int lo = 0, len = n;
    while (len > 1) warp_narrow(v, lo, len, x, extent, status);
    return lo;
}

// Position (and page slot) of token row `t`, computed by one warp.
template <bool kPaged>
__device__ __forceinline__ TokenPos token_pos(const RopeArgs& a, long long t)
{
    TokenPos r{0, -1, 0};
    if (t >= a.rows) return r;
    if constexpr (kPaged) {
        // The last 32 sequences that the search leaves are looked at with their ends and
        // lengths, so that a step of up to 32 sequences waits for one read before the table's.
        const int lane = threadIdx.x & 31;
        int lo = 0, len = a.n_seqs;
        while (len > 32) warp_narrow(a.cu_seqlens, lo, len, t, a.n_seqs + 1, a.status);
        int first = 0x7fffffff, end = 0, keys = 0;
        if (lane < len) {
            first = checked_ldg(a.cu_seqlens, lo + lane, a.n_seqs + 1, a.status);
            end = checked_ldg(a.cu_seqlens, lo + lane + 1, a.n_seqs + 1, a.status);
            keys = checked_ldg(a.kv_lens, lo + lane, a.n_seqs, a.status);
        }
        const int before = __popc(__ballot_sync(0xffffffffu, lane < len && first <= t));
        const int k = before > 0 ? before - 1 : 0, g = lo + k;
        first = __shfl_sync(0xffffffffu, first, k);
        end = __shfl_sync(0xffffffffu, end, k);
        keys = __shfl_sync(0xffffffffu, keys, k);
        if (t < first || t >= end) return r;
        r.live = 1;
        r.pos = static_cast<long long>(keys) - (static_cast<long long>(end) - t);
        const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
        if (r.pos >= 0 && r.pos < cap) {                // (below 2^31, as the lengths are)
            const int col = static_cast<int>(static_cast<unsigned>(r.pos) / static_cast<unsigned>(a.page_size));
            const int in_page = static_cast<int>(r.pos) - col * a.page_size;
            const int page = checked_ldg(a.page_table, g * a.table_stride + col, a.table_elems,
                                         a.status);
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
                r.slot = page * a.page_stride + in_page * a.token_stride;
        }
        // (a drafted token turns by its depth in the tree, not by where it is stored)
        if (a.positions != nullptr) r.pos = checked_ldg(a.positions, t, a.rows, a.status);
        return r;
    } else {
        r.live = 1;
        const int l = t >> 31 ? static_cast<int>(t % a.L)
                              : static_cast<int>(static_cast<unsigned>(t) % static_cast<unsigned>(a.L));
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

// Sine and cosine of position times phase.
__device__ __forceinline__ void angle_of(unsigned long long phase, long long pos, float& s, float& c)
{
    const unsigned long long turn = phase * static_cast<unsigned long long>(pos);
    // upper 32 bits as a signed number: [-2^31, 2^31) is [-1, 1) half turns
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &s, &c);
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

__device__ __forceinline__ uint64_t unpack2(uint32_t w)       // two bf16 to two fp32
{
    return f2pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v)
{
    float lo, hi;
    f2unpack(v, lo, hi);
    return pack_bf16x2(lo, hi);
}

// Blocks of `threads` threads that the GPU holds at once.
template <typename Kernel>
cudaError_t slots_of(std::atomic<int>* known, Kernel kernel, int threads, int sms, int* slots)
{
    int ctas = 0;                                   // of 128 threads
    const cudaError_t e = resident_ctas(known, kernel, 128, 0, &ctas);
    if (e != cudaSuccess) return e;
    const int per_sm = ctas / sms * 128 / threads;
    *slots = sms * (per_sm > 0 ? per_sm : 1);
    return cudaSuccess;
}

}  // namespace ra
