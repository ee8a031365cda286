// ra_internal.h -- host-side interface between the C ABI layer (api.cu) and
// the kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "ring_attn.h"

namespace ra {

constexpr int kMaxDevices = 64;

// Raises a kernel's dynamic shared-memory limit the first time a device launches it.
// `done` is one flag per device (static storage: starts at zero).  Safe to call from
// several host threads at once: the flag is atomic, and the attribute call is
// idempotent, so two threads that both see the flag clear both make it harmlessly.
template <typename Kernel>
cudaError_t smem_limit_once(std::atomic<int>* done, int dev, Kernel kernel, int bytes)
{
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done[dev].store(1, std::memory_order_release);
    return e;
}

// CTAs of a kernel that the current device holds at once (SMs times resident CTAs), asked
// once per device: `known` is one value per device (static storage: 0, not asked yet).  Also
// raises the kernel's dynamic shared-memory limit to `bytes`.
template <typename Kernel>
cudaError_t resident_ctas(std::atomic<int>* known, Kernel kernel, int threads, int bytes, int* ctas)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    *ctas = known[dev].load(std::memory_order_acquire);
    if (*ctas > 0) return cudaSuccess;
    int sms = 0, per_sm = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, bytes);
    if (e != cudaSuccess) return e;
    *ctas = sms * (per_sm > 0 ? per_sm : 1);
    known[dev].store(*ctas, std::memory_order_release);
    return cudaSuccess;
}

// Launches a kernel that begins with wait_for_earlier_work() as a programmatic dependent: its
// blocks are set up while the work before it in the stream drains.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned grid, int threads, int bytes,
                         cudaStream_t stream, const Args&... args)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(grid);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = bytes;
    config.stream = stream;
    config.attrs = &early;
    config.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&config, kernel, args...);
    if (e != cudaSuccess) cudaGetLastError();       // reported here, not to the next caller who asks
    return e;
}

// Everything one attention launch needs; validated by the ABI layer.
struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* lse;      // may be null
    int* trace;      // may be null
    int B, L, H, D, P, causal;
    int Hkv;                       // key/value heads (H for plain attention)
    int zigzag;                    // zigzag shard layout (causal)
    const int* cu_seqlens;         // packed sequences (device), or null
    int n_seqs;
    const int* schedule;           // packed sequences: unit orders (VarlenSchedLayout), or null
    // Ulysses head groups read from / written to the sequence-sharded buffers
    // [u_P][u_B][L/u_P][u_H][D] (0 = not used): B = u_P * u_B head-group batches of
    // H = u_H / u_P heads, ring P = 1; the tensor maps are then 5-D.
    int u_P, u_B, u_H;
    unsigned int* status;          // device status word
    unsigned long long timeout_ns; // limit of one bounded wait
    cudaStream_t stream;
};

// Packed-sequence schedule (ring_attn_varlen_schedule), in int32 entries: the forward's
// query-tile pairs, the backward's key tiles and query tiles, each a permutation of the
// units of one (batch, head) given by their natural index (shard * per-shard units +
// tile or pair), heaviest first; then scratch for the work counts of all three; then
// kCounters work counters of the persistent kernels (a claim counter and a finished-CTA
// counter per kernel: forward, backward key tiles, backward query tiles), zeroed by the
// schedule kernel and reset to zero by the last CTA of each launch that uses them.
constexpr int kCounters = 8;
struct VarlenSchedLayout {
    long long n_t, n_pair;           // 128-row tiles and tile pairs per shard
    long long fwd, bwd_k, bwd_q;     // offsets of the three orders
    long long scratch;               // offset of the scratch
    long long counters;              // offset of the work counters
    long long total;                 // total entries
};
inline VarlenSchedLayout varlen_sched_layout(int L, int P)
{
    VarlenSchedLayout s;
    const long long Ls = static_cast<long long>(L) / P;
    s.n_t = (Ls + 127) / 128;
    s.n_pair = (s.n_t + 1) / 2;
    s.fwd = 0;
    s.bwd_k = s.fwd + P * s.n_pair;
    s.bwd_q = s.bwd_k + P * s.n_t;
    s.scratch = s.bwd_q + P * s.n_t;
    s.counters = s.scratch + s.scratch;
    s.total = s.counters + kCounters;
    return s;
}
cudaError_t launch_varlen_schedule(const int* cu_seqlens, int n_seqs, int L, int P, int causal,
                                   int* schedule, unsigned int* status, cudaStream_t stream);

// bf16 tcgen05 kernel; tensor maps describe q, k, v as 4-D [B][L][H][D] with
// 64-element, 128-byte-swizzled boxes of 128 rows -- except that k has boxes of 64 rows
// when attn_bf16_pair_applies(a) (the pair-of-SMs kernel loads half a key block per CTA).
bool attn_bf16_pair_applies(const AttnArgs& a);
cudaError_t launch_attn_bf16(const AttnArgs& a, const CUtensorMap& tmap_q,
                             const CUtensorMap& tmap_k, const CUtensorMap& tmap_v);

// fp32 SIMT kernel.
cudaError_t launch_attn_f32(const AttnArgs& a);

// Backward (bf16): Dvec into the workspace, then the dK/dV and dQ kernels.
struct BwdArgs {
    const void* out;     // forward output O
    const void* dout;    // upstream gradient dO
    const float* lse;    // forward lse [B, L, H]
    float* dvec;         // workspace [B, L, H]
    void* dq;
    void* dk;
    void* dv;
    int B, L, H, D, P, causal;
    int Hkv;             // key/value heads (H % Hkv == 0); dk, dv are [B, L, Hkv, D]
    int zigzag;          // zigzag shard layout (causal; Hkv == H)
    const int* cu_seqlens;   // packed sequences (device; B == 1, Hkv == H), or null
    int n_seqs;
    const int* schedule;     // packed sequences: unit orders (VarlenSchedLayout), or null
    unsigned int* status;
    unsigned long long timeout_ns;
    cudaStream_t stream;
};
// tmap_k64, tmap_v64: k and v with 64-row boxes, required when bwd_dq_pair_applies(a) (the
// pair-of-SMs dQ kernel stages half a key block per CTA), else null.
cudaError_t launch_attn_bwd_bf16(const BwdArgs& a, const CUtensorMap& tmap_q,
                                 const CUtensorMap& tmap_k, const CUtensorMap& tmap_v,
                                 const CUtensorMap& tmap_do, const CUtensorMap* tmap_k64,
                                 const CUtensorMap* tmap_v64);
bool bwd_dq_pair_applies(const BwdArgs& a);

cudaError_t launch_merge(const void* o_a, const float* lse_a, const void* o_b, const float* lse_b,
                         void* o_out, float* lse_out, long long rows, int D, int elem_bytes,
                         unsigned int* status, cudaStream_t stream);

// dir = 0: seq2head, dir = 1: head2seq.
// Copy-engine path of the same transposes: seq_map is the 5-D view {D, H/P, P, L/P, P*B}
// of the sequence-sharded buffer with box {D, H/P, 1, R, 1} (encoded by the caller),
// head_side the head-sharded buffer.  Valid when ulysses_permute_tma_fits.
bool ulysses_permute_tma_fits(int H, int D, int P, int elem_bytes);
int ulysses_permute_tma_rows(int L, int H, int D, int P, int elem_bytes);
cudaError_t launch_ulysses_permute_tma(const CUtensorMap& seq_map, void* head_side, int B, int L,
                                       int H, int D, int P, int elem_bytes, int dir, int R,
                                       unsigned int* status, unsigned long long timeout_ns,
                                       cudaStream_t stream);

cudaError_t launch_ulysses_permute(const void* in, void* out, int B, int L, int H, int D, int P,
                                   int elem_bytes, int dir, unsigned int* status, cudaStream_t stream);

cudaError_t launch_wait_probe(unsigned int* status, unsigned long long timeout_ns,
                              cudaStream_t stream);

// Rotary positions (rope_fwd, rope_bwd) and the paged append: rows of heads, rotated.
struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;                 // paged append only
    void* q_out;
    void* k_out;                   // paged append: the k pages
    void* v_out;                   // paged append: the v pages
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // elements per token
    long long q_elems, k_elems, v_elems, q_out_elems, k_out_elems;        // extents, for checks
    long long rows;                // tokens
    int L, P, H, H_kv, D, elem;    // H, H_kv: heads of q, of k (and v); elem: bytes
    int rot, half_style;
    float amplitude, sign;
    const unsigned long long* phases;
    ra_layout layout;
    const int* positions;          // or null: by layout
    int position_offset;
    const int* cu_seqlens;         // packed layout; paged append: the new tokens' starts
    int n_seqs;
    int paged;
    const int* kv_lens;
    const int* page_table;
    long long table_stride, table_elems, page_stride, token_stride, head_stride;
    int num_pages, page_size, max_pages;
    int tokens, step_t, step_h;    // tokens per block, and taken at once; heads at once (set
                                   // by the launch)
    unsigned int* status;
    cudaStream_t stream;
};
cudaError_t launch_rope(const RopeArgs& a);

// The same with a norm of every head before the rotation (qk_norm_rope_fwd, _bwd, and the
// paged append with weights).
struct NormArgs {
    RopeArgs rope;                 // backward: q, k the inputs, q_out, k_out their gradients
    const void* q_weight;          // [D] each, or null: ones
    const void* k_weight;
    int weight_elem;               // bytes
    float eps, weight_offset;
    // backward: gradients of the outputs, and of the weights (or null)
    const void* dq_out;
    const void* dk_out;
    long long dq_out_stride, dk_out_stride, dq_out_elems, dk_out_elems;
    float* dq_weight;
    float* dk_weight;
    float* partials;               // [kNormCtas][2][256]
    unsigned int* ticket;          // [1 + groups of blocks], zero between calls
    int lanes;                     // of a head vector, a power of two (set by the launch)
    int items;                     // of them, those that hold some of it (set by the launch)
    int per_token, parts;          // rounds of a warp for a token's heads, and the parts that they
                                   // are shared out in (set by the launch)
};
constexpr int kNormCtas = 640;     // of the backward
constexpr int kNormGroup = 16;     // of its blocks, whose sums are added at once
static_assert(4 * (1 + (kNormCtas + kNormGroup - 1) / kNormGroup) <= 256, "counters before the partial sums");
cudaError_t launch_norm(const NormArgs& a);
cudaError_t launch_norm_bwd(const NormArgs& a);

// The pool of pages (paged_reserve, paged_release).
struct PoolArgs {
    int* free_pages;               // [num_pages], a stack
    int* held;                     // [n_seqs]
    int* state;                    // free pages, block counter, status of the last reserve
    int* page_table;
    long long table_stride, table_elems;
    int num_pages, n_seqs, max_pages, page_size;
    unsigned int* status;
};
constexpr int kPoolSeqs = 8192;    // sequences (their sums lie in shared memory)
struct ReserveArgs {
    PoolArgs pool;
    const int* new_lens;
    const int* lens;
    int* cu_new;
    int* kv_lens;
    int* positions;                // these four may be null
    long long* slots;
    const int* parents;
    int* masks;
    int* unmasked;                 // or null: new tokens that masks have no bit for
    int T, mask_words;
    cudaStream_t stream;
};
cudaError_t launch_reserve(const ReserveArgs& r);
cudaError_t launch_release(const ReserveArgs& r);

// Accepted tokens to the front of a step's slots (paged_kv_keep).
struct KeepArgs {
    void* k_pages;
    void* v_pages;
    long long page_stride, token_stride, head_stride, layer_stride, table_stride;
    long long page_elems, table_elems, kept_elems, kept_stride;
    int layers, n_seqs, H_kv, D, elem, num_pages, page_size, max_pages, width;
    const int* kept;
    const int* page_table;
    const int* cu_new;
    const int* kv_lens;
    int* lens;
    long long columns;             // 16-byte columns of a token over all layers (by the launch)
    int pieces;                    // blocks of a sequence (by the launch)
    unsigned int* status;
    cudaStream_t stream;
};
cudaError_t launch_keep(const KeepArgs& a);

// Attention over a paged cache (paged_attn_fwd).
struct PagedArgs {
    const void* q;
    const void* k_pages;
    const void* v_pages;
    void* out;
    float* lse;                    // may be null
    void* workspace;
    long long q_stride;            // elements per token
    long long q_elems, page_elems, out_elems, lse_elems, table_elems;     // extents, for checks
    long long page_stride, token_stride, head_stride, table_stride;
    const int* masks;              // a drafted tree: bits of the new tokens that a row sees, or null
    long long mask_stride, mask_elems;
    int mask_words;
    int T, n_seqs, H, H_kv, D, elem, causal;
    int num_pages, page_size, max_pages;
    const int* cu_new;
    const int* kv_lens;
    const int* page_table;
    unsigned int* status;
    unsigned long long timeout_ns;
    cudaStream_t stream;
};
// CTAs a call may launch (the workspace holds two partial results for each).
constexpr int kPagedMaxCtas = 1024;
constexpr int kPagedRowsCtas = 320;   // of the fp32 kernel for many rows
constexpr int kPagedTcCtas = 160;     // of the tensor-core kernel (one per SM)
unsigned long long paged_workspace_bytes(int D, int elem);
cudaError_t launch_paged(const PagedArgs& a);        // chooses among:
cudaError_t launch_paged_simt(const PagedArgs& a);   // fp32, few rows per key/value head
bool paged_rows_applies(const PagedArgs& a);
cudaError_t launch_paged_rows(const PagedArgs& a);   // fp32, many rows
cudaError_t launch_paged_bf16(const PagedArgs& a);   // bf16, few rows per key/value head
// Trees of drafted tokens in calls of few tiles, a cluster for each: launch the call, with *e what
// became of it, or leave it to the others (false).
bool paged_tree_bf16(const PagedArgs& a, cudaError_t* e);
bool paged_tree_f32(const PagedArgs& a, cudaError_t* e);
// bf16, many rows: CTAs, and tensor maps of q ({D, H, T}, boxes of 64 x G x tokens) and of
// the pages ({D, H_kv, page_size, num_pages}, boxes of 64 x 1 x keys of one page x 1).
bool paged_tc_applies(const PagedArgs& a);
cudaError_t launch_paged_tc(const PagedArgs& a);

// bf16 tensor of `rank` dims (innermost first, strides in bytes of dims 1 and up) with boxes
// of 64 innermost elements, 128-byte swizzle, zeros outside.  False if the driver refuses it.
bool encode_bf16_map(CUtensorMap* map, const void* base, int rank, const unsigned long long* dims,
                     const unsigned long long* strides, const unsigned int* box);

// Device address of the current device's status word (api.cu).
ra_status current_status_word(unsigned int** out);

// One thread whose index check fails (debug build): exercises RA_STATUS_BOUNDS.
cudaError_t launch_bounds_probe(unsigned int* status, cudaStream_t stream);

}  // namespace ra
