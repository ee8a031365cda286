// pages.cu -- the bookkeeping of the paged key/value cache on the device: a step's pages, rows,
// positions, slots and tree masks from the requests' lengths (paged_reserve), pages given back
// (paged_release), and accepted drafted tokens moved to their places (paged_kv_keep).
//
// Reserving.  With need_g = max(0, ceil((len_g + new_g) / page) - held_g), page number
// P_g + c of the step (P the exclusive sum of need) is the P_g + c th entry from the top of the
// stack of free pages, and row t of the step belongs to the sequence g whose
// [cu_g, cu_{g+1}), cu the exclusive sum of new, holds t.  Both sums are over the sequences and
// every row needs them, so each block works them out for itself in shared memory -- a few
// thousand integers, from L2 -- which saves a second launch; rows and new pages are then shared
// out evenly over the blocks, whatever the lengths are, and find their sequence by halving.
// Nothing that a block reads is written before all blocks have read it: the pool's counters and
// the lengths (which may be updated in place) are written by the block that counts itself in
// last, and new table entries are columns that no one reads.
//
// What bounds it: the launch and a chain of dependent reads (lengths, table or stack, stores), as
// the data are a few bytes a row: 64 sequences of a token each 3.2 us, their release 1.8.  With many
// sequences the sums, which every block works out (one token each of 1024 sequences 6.1 us, of
// 8192 58; releases 3.3 and 27), and with parents the deepest path, whose reads wait for one another
// (1024 trees of up to 61 tokens 9.4 us; a prompt of 975 tokens as one chain of parents 177, 0.18 a
// token, where long prompts without parents walk nothing).
#include <algorithm>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDeep = 8;                    // reads (of keep_kernel: moves) in flight of a thread

// Exclusive sum of two values over the block's threads; totals in *all_a, *all_b.
__device__ __forceinline__ void block_sums(long long& a, long long& b, long long* all_a, long long* all_b)
{
    __shared__ long long warp_a[kWarps], warp_b[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ya = __shfl_up_sync(0xffffffffu, ia, o), yb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += ya;
            ib += yb;
        }
    }
    if (lane == 31) {
        warp_a[warp] = ia;
        warp_b[warp] = ib;
    }
    __syncthreads();
    long long before_a = 0, before_b = 0, ta = 0, tb = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
            before_a = ta;
            before_b = tb;
        }
        ta += warp_a[w];
        tb += warp_b[w];
    }
    a = before_a + ia - a;
    b = before_b + ib - b;
    *all_a = ta;
    *all_b = tb;
}

// The last g in [0, n) with first[g] <= x, for a non-decreasing first with first[0] <= x.
__device__ __forceinline__ int seq_of(const int* first, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Counts this block in; true in all threads of the last one, which finds the counter zero again.
__device__ __forceinline__ bool last_block(int* ticket)
{
    if (gridDim.x == 1) return true;
    __shared__ int last;
    __syncthreads();                        // the block's reads are done
    if (threadIdx.x == 0) {
        unsigned before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
        last = before == gridDim.x - 1;
        if (last) *ticket = 0;
    }
    __syncthreads();
    return last;
}

// (plain loads, not the read-only path: the launch's last block writes these)
__device__ __forceinline__ int held_of(const PoolArgs& a, int g)
{
    return in_bounds(g, 1, a.n_seqs, a.status) ? min(max(a.held[g], 0), a.max_pages) : 0;
}
__device__ __forceinline__ int free_count(const PoolArgs& a) { return min(max(a.state[0], 0), a.num_pages); }
__device__ __forceinline__ int length_of(const PoolArgs& a, const int* v, int g)
{
    return in_bounds(g, 1, a.n_seqs, a.status) ? max(v[g], 0) : 0;
}

__global__ void __launch_bounds__(kThreads) reserve_kernel(const __grid_constant__ ReserveArgs r)
{
    const PoolArgs& a = r.pool;
    extern __shared__ int sums[];
    const int n = a.n_seqs;
    int* cu = sums;                         // first row of every sequence
    int* fresh = sums + n;                  // pages that the sequences before it take
    int* len = fresh + n;
    int* held = len + n;
    __shared__ int too_long, unmasked;
    if (threadIdx.x == 0) too_long = unmasked = 0;
    wait_for_earlier_work();
    const int available = free_count(a);
    __syncthreads();

    // a thread's sequences, in order
    const int per = (n + kThreads - 1) / kThreads;
    const int g0 = min(static_cast<int>(threadIdx.x) * per, n), g1 = min(g0 + per, n);
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
    auto need_of = [&](int g, int add) -> long long {
        // (below 2^33: a sum of three numbers below 2^31)
        const unsigned long long keys = static_cast<unsigned long long>(len[g]) + add + a.page_size - 1;
        const long long pages = keys >> 32 ? static_cast<long long>(keys / a.page_size)
                                           : static_cast<unsigned>(keys) / static_cast<unsigned>(a.page_size);
        return max(pages - held[g], 0ll);
    };
    long long rows = 0, pages = 0;
    for (int first = g0; first < g1; first += kDeep) {
        int add[kDeep], before[kDeep], has[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {               // (all reads first)
            const int g = min(first + k, g1 - 1);
            add[k] = length_of(a, r.new_lens, g);
            before[k] = length_of(a, r.lens, g);
            has[k] = held_of(a, g);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int g = first + k;
            if (g >= g1) break;
            len[g] = before[k];
            held[g] = has[k];
            cu[g] = add[k];
            rows += add[k];
            pages += need_of(g, add[k]);
            if (static_cast<long long>(before[k]) + add[k] > min(cap, 0x7fffffffll)) too_long = 1;
        }
    }
    long long all_rows, all_pages;
    long long at_row = rows, at_page = pages;
    block_sums(at_row, at_page, &all_rows, &all_pages);
    // a step that does not fit becomes one without rows
    const int status = all_rows > r.T ? 2 : too_long ? 3 : all_pages > available ? 1 : 0;
    if (status != 0) all_rows = all_pages = at_row = at_page = 0;
    for (int g = g0; g < g1; ++g) {
        const int add = status == 0 ? cu[g] : 0;
        const long long need = status == 0 ? need_of(g, add) : 0;
        cu[g] = static_cast<int>(at_row);
        fresh[g] = static_cast<int>(at_page);
        at_row += add;
        at_page += need;
    }
    const bool last = last_block(a.state + 1);
    if (gridDim.x == 1) __syncthreads();

    // (64-bit counters: rows and pages may be so many that a step beyond the last passes 2^31)
    const int step = gridDim.x * kThreads, first = blockIdx.x * kThreads + threadIdx.x;
    // the page of entry p of those that this step takes
    auto page_from = [&](int p) {
        const int i = available - 1 - p;
        return in_bounds(i, 1, a.num_pages, a.status) ? a.free_pages[i] : -1;
    };
    for (int g = first; g <= n; g += step)
        if (in_bounds(g, 1, n + 1, a.status)) r.cu_new[g] = g < n ? cu[g] : static_cast<int>(all_rows);
    for (long long i = first; i < all_pages; i += step) {
        const int p = static_cast<int>(i);
        const int g = seq_of(fresh, n, p);
        const long long at = g * a.table_stride + held[g] + (p - fresh[g]);
        if (in_bounds(at, 1, a.table_elems, a.status)) a.page_table[at] = page_from(p);
    }
    // (no rows to fill in where a program wants the starts, lengths and pages only)
    const bool fills = r.positions != nullptr || r.slots != nullptr || r.masks != nullptr;
    for (long long row = first; fills && row < r.T; row += step) {
        const int t = static_cast<int>(row);
        int pos = 0, i = 0, c = 0;
        long long slot = -1;
        const bool real = t < all_rows;
        if (real) {
            const int g = seq_of(cu, n, t);
            c = cu[g];
            i = t - c;
            pos = len[g] + i;
            const int col = static_cast<int>(static_cast<unsigned>(pos) / static_cast<unsigned>(a.page_size));
            int page;
            if (col < held[g]) {
                const long long at = g * a.table_stride + col;
                page = in_bounds(at, 1, a.table_elems, a.status) ? a.page_table[at] : -1;
            } else {
                page = page_from(fresh[g] + col - held[g]);
            }
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
                slot = static_cast<long long>(page) * a.page_size + (pos - col * a.page_size);
            pos -= i;
        }
        if (r.slots != nullptr && in_bounds(t, 1, r.T, a.status)) r.slots[t] = slot;
        auto put = [&](int w, unsigned b) {
            const long long at = static_cast<long long>(t) * r.mask_words + w;
            if (in_bounds(at, 1, static_cast<long long>(r.T) * r.mask_words, a.status))
                r.masks[at] = static_cast<int>(b);
        };
        if (r.parents == nullptr) {
            // a chain: every token follows all before it
            if (r.positions != nullptr && in_bounds(t, 1, r.T, a.status)) r.positions[t] = real ? pos + i : 0;
            for (int w = 0; w < r.mask_words; ++w) {
                const int bits = real ? i + 1 - 32 * w : 0;
                put(w, bits <= 0 ? 0u : bits >= 32 ? 0xffffffffu : (1u << bits) - 1);
            }
            continue;
        }
        // Up the chain of parents: the depth, and a bit for every ancestor.  Parents come
        // before their children (others count as none), so the words are done from the top.
        unsigned bits = 0;
        int word = r.mask_words - 1, depth = -1;
        for (int node = real ? i : -1; node >= 0;) {
            ++depth;
            const int w = node >> 5;
            if (w < r.mask_words) {
                while (word > w) {
                    put(word--, bits);
                    bits = 0;
                }
                bits |= 1u << (node & 31);
            }
            const int up = in_bounds(c + node, 1, r.T, a.status) ? __ldg(r.parents + c + node) : -1;
            node = up < node ? up : -1;
        }
        for (; word >= 0; --word) {
            put(word, bits);
            bits = 0;
        }
        if (r.positions != nullptr && in_bounds(t, 1, r.T, a.status)) r.positions[t] = real ? pos + depth : 0;
    }
    if (!last) return;
    // what others read before, and the tokens that masks have no bit for
    const long long bits = r.mask_words > 0 ? 32ll * r.mask_words : 0x7fffffffll;
    for (int g = threadIdx.x; g < n; g += kThreads) {
        const int end = g + 1 < n ? cu[g + 1] : static_cast<int>(all_rows);
        const int taken = g + 1 < n ? fresh[g + 1] : static_cast<int>(all_pages);
        if (!in_bounds(g, 1, n, a.status)) continue;
        r.kv_lens[g] = len[g] + (end - cu[g]);
        if (end - cu[g] > bits) atomicAdd(&unmasked, static_cast<int>(end - cu[g] - bits));
        a.held[g] = held[g] + (taken - fresh[g]);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.state[0] = available - static_cast<int>(all_pages);
        a.state[2] = status;
        if (r.unmasked != nullptr) *r.unmasked = unmasked;
    }
}

// Gives back the pages behind every sequence's length: page number p of them (sequence by
// sequence, column by column) ends p places below the top, so that a reserve finds the pages
// that it took in the same order.
__global__ void __launch_bounds__(kThreads) release_kernel(const __grid_constant__ ReserveArgs r)
{
    const PoolArgs& a = r.pool;
    extern __shared__ int sums[];
    const int n = a.n_seqs;
    int* gone = sums;                       // pages that the sequences before it give back
    int* left = sums + n;
    wait_for_earlier_work();
    const int available = free_count(a);
    const int per = (n + kThreads - 1) / kThreads;
    const int g0 = min(static_cast<int>(threadIdx.x) * per, n), g1 = min(g0 + per, n);
    long long pages = 0, none = 0, all_none, all;
    for (int first = g0; first < g1; first += kDeep) {
        int has[kDeep], keys[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {               // (all reads first)
            const int g = min(first + k, g1 - 1);
            has[k] = held_of(a, g);
            keys[k] = length_of(a, r.lens, g);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int g = first + k;
            if (g >= g1) break;
            const int want = static_cast<int>((keys[k] + static_cast<unsigned>(a.page_size) - 1) /
                                              static_cast<unsigned>(a.page_size));
            left[g] = min(want, has[k]);
            gone[g] = has[k] - left[g];
            pages += gone[g];
        }
    }
    long long at = pages;
    block_sums(at, none, &all, &all_none);
    // (more than the pool has room for: a table or count that the program has damaged; those
    // that do not fit are lost)
    for (int g = g0; g < g1; ++g) {
        const int k = gone[g];
        gone[g] = static_cast<int>(min(at, 0x7fffffffll));
        at += k;
    }
    const bool last = last_block(a.state + 1);
    if (gridDim.x == 1) __syncthreads();
    const long long top = available + all - 1;
    const int step = gridDim.x * kThreads;
    const int total = static_cast<int>(min(all, 0x7fffffffll));
    for (long long i = blockIdx.x * kThreads + threadIdx.x; i < total; i += step) {
        const int p = static_cast<int>(i);
        const int g = seq_of(gone, n, p);
        const long long from = g * a.table_stride + left[g] + (p - gone[g]);
        if (!in_bounds(from, 1, a.table_elems, a.status)) continue;
        if (top - p < a.num_pages) a.free_pages[top - p] = a.page_table[from];
        a.page_table[from] = -1;
    }
    if (!last) return;
    for (int g = threadIdx.x; g < n; g += kThreads)
        if (in_bounds(g, 1, n, a.status)) a.held[g] = left[g];
    if (threadIdx.x == 0) a.state[0] = static_cast<int>(min(top + 1, static_cast<long long>(a.num_pages)));
}

// ---- keeping accepted tokens ----
//
// Entry i of a sequence's path moves from the step's slot kept_i to slot i.  kept ascends, so
// kept_i >= i: no later entry is read from a slot that an earlier one was written to, and a
// thread that walks the path with its own 16 bytes of a token may read as far ahead as it likes.
// A block takes a piece of one sequence: 256 threads' 16-byte columns of (layer, keys or values,
// head); its first warp looks the path's slots up once for all of them.
constexpr int kPath = 32;                   // entries looked up at a time

__global__ void __launch_bounds__(kThreads) keep_kernel(const __grid_constant__ KeepArgs a)
{
    __shared__ long long from_s[kPath], to_s[kPath];
    __shared__ int count_s, more_s;
    const int g = blockIdx.x / a.pieces, piece = blockIdx.x - g * a.pieces;
    const int lane = threadIdx.x & 31;
    const int vecs = a.D * a.elem / 16;     // columns of a head vector
    long long x = static_cast<long long>(piece) * kThreads + threadIdx.x;
    const bool works = x < a.columns;
    const int col = static_cast<int>(x % vecs);
    x /= vecs;
    const int head = static_cast<int>(x % a.H_kv);
    x /= a.H_kv;
    const bool values = x & 1;
    const long long base = (x >> 1) * a.layer_stride + head * a.head_stride;
    const int per = 16 / a.elem;            // elements of a column
    char* pages = static_cast<char*>(values ? a.v_pages : a.k_pages);
    wait_for_earlier_work();
    const int lo = checked_ldg(a.cu_new, g, a.n_seqs + 1, a.status);
    const int hi = checked_ldg(a.cu_new, g + 1, a.n_seqs + 1, a.status);
    const int kv = checked_ldg(a.kv_lens, g, a.n_seqs, a.status);
    const int n = max(hi - lo, 0);
    const long long first = static_cast<long long>(kv) - n;
    int kept_before = -1, total = 0;        // warp 0's: the last valid entry, how many
    for (long long i0 = 0; i0 < a.width; i0 += kPath) {
        if (threadIdx.x < 32) {
            const long long i = i0 + lane;
            int node = -1;
            if (i < a.width) node = checked_ldg(a.kept, g * a.kept_stride + i, a.kept_elems, a.status);
            // RA_KEEP_ALL in front: every new token stays where it is
            const bool all = i0 == 0 && __shfl_sync(0xffffffffu, node, 0) == RA_KEEP_ALL;
            int before = __shfl_up_sync(0xffffffffu, node, 1);
            if (lane == 0) before = kept_before;
            const unsigned bad = __ballot_sync(0xffffffffu, !(node > before && node < n));
            const int good = all ? 0 : bad ? __ffs(bad) - 1 : 32;
            kept_before = __shfl_sync(0xffffffffu, node, 31);
            total = all ? n : total + good;
            auto offset = [&](long long pos) -> long long {
                const long long c = pos / a.page_size;
                if (pos < 0 || c >= a.max_pages) return -1;
                const int page = checked_ldg(a.page_table, g * a.table_stride + c, a.table_elems, a.status);
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) return -1;
                return page * a.page_stride + (pos - c * a.page_size) * a.token_stride;
            };
            long long from = -1, to = -1;
            if (lane < good && node != i) {
                from = offset(first + node);
                to = offset(first + i);
            }
            from_s[lane] = to < 0 ? -1 : from;
            to_s[lane] = to;
            if (lane == 0) {
                count_s = good;
                more_s = good == 32;
            }
        }
        __syncthreads();
        const int count = count_s;
        const bool more = more_s;
        for (int k = 0; works && k < count; k += kDeep) {
            uint4 v[kDeep];
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const long long from = k + u < count ? from_s[k + u] : -1;
                const long long at = base + from + col * per;
                if (from >= 0 && in_bounds(at, per, a.page_elems, a.status))
                    v[u] = *reinterpret_cast<const uint4*>(pages + at * a.elem);
            }
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                if (k + u >= count || from_s[k + u] < 0) continue;
                const long long at = base + to_s[k + u] + col * per;
                if (in_bounds(at, per, a.page_elems, a.status))
                    *reinterpret_cast<uint4*>(pages + at * a.elem) = v[u];
            }
        }
        if (!more) break;
        __syncthreads();
    }
    if (piece == 0 && threadIdx.x == 0 && in_bounds(g, 1, a.n_seqs, a.status))
        a.lens[g] = static_cast<int>(max(first + total, 0ll));
}

cudaError_t sms_of(int* sms)
{
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

cudaError_t launch_reserve(const ReserveArgs& r)
{
    int sms = 0, dev = 0;
    cudaError_t e = sms_of(&sms);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int bytes = 16 * r.pool.n_seqs;
    static std::atomic<int> done[kMaxDevices];
    e = smem_limit_once(done, dev, reserve_kernel, 16 * kPoolSeqs);
    if (e != cudaSuccess) return e;
    const int blocks = std::max(1, std::min((r.T + kThreads - 1) / kThreads, 2 * sms));
    return launch_early(reserve_kernel, blocks, kThreads, bytes, r.stream, r);
}

cudaError_t launch_release(const ReserveArgs& r)
{
    int sms = 0, dev = 0;
    cudaError_t e = sms_of(&sms);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<int> done[kMaxDevices];
    e = smem_limit_once(done, dev, release_kernel, 8 * kPoolSeqs);
    if (e != cudaSuccess) return e;
    // Most calls give back a page or two a sequence, so one block will do up to 255 sequences,
    // and one in 128 beyond, lest a server's worth of ended prompts is left to one.
    const int blocks = std::max(1, std::min(r.pool.n_seqs / 128, sms));
    return launch_early(release_kernel, blocks, kThreads, 8 * r.pool.n_seqs, r.stream, r);
}

cudaError_t launch_keep(const KeepArgs& args)
{
    KeepArgs a = args;
    a.columns = 2ll * a.layers * a.H_kv * (a.D * a.elem / 16);
    const long long pieces = (a.columns + kThreads - 1) / kThreads;
    if (pieces * a.n_seqs > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    a.pieces = static_cast<int>(pieces);
    return launch_early(keep_kernel, static_cast<unsigned>(pieces * a.n_seqs), kThreads, 0, a.stream, a);
}

}  // namespace ra
