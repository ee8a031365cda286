// api_paged.cu -- the extern "C" entry points for rotary positions and the paged key/value
// cache: host-side argument checks (nothing is launched on a bad argument) and dispatch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ra_internal.h"

namespace {

using ull = unsigned long long;
constexpr ull kMaxElems = 1ull << 40;
constexpr unsigned long long kWaitLimitNs = 4000000000ull;   // 4 s for any single wait

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of `row` bytes, `stride` bytes apart.
struct Rows {
    const void* base;
    ull rows, row, stride;
    ull span() const { return rows == 0 || row == 0 ? 0 : (rows - 1) * stride + row; }
};

bool overlap(const void* a, ull na, const void* b, ull nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// Whether two tensors of rows share memory.  Interleaved views of one buffer (the same
// stride, rows side by side) do not; interleaved with other strides counts as shared.
bool overlap(const Rows& a, const Rows& b)
{
    if (!overlap(a.base, a.span(), b.base, b.span())) return false;
    if (a.stride != b.stride || a.stride == 0) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
    const ull d = (x <= y ? y - x : a.stride - (x - y) % a.stride) % a.stride;   // b after a
    return d < a.row || a.stride - d < b.row;
}

ra_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RA_OK : RA_ERR_CUDA; }

// Token stride in elements (0: contiguous), checked: rows of n elements that do not overlap
// themselves and start on 16-byte boundaries.
ra_status row_stride(long long* stride, long long n, int elem)
{
    if (*stride == 0) *stride = n;
    if (*stride < n || *stride >= static_cast<long long>(kMaxElems)) return RA_ERR_INVALID_ARG;
    return (*stride * elem) % 16 == 0 ? RA_OK : RA_ERR_MISALIGNED;
}

ra_status check_rope(const ra_rope* rope, int D)
{
    if (!rope || !rope->phases) return RA_ERR_INVALID_ARG;
    if (rope->rot_dim < 2 || rope->rot_dim > D || rope->rot_dim % 2 != 0) return RA_ERR_INVALID_ARG;
    if (rope->style != RA_ROPE_HALF && rope->style != RA_ROPE_INTERLEAVED) return RA_ERR_INVALID_ARG;
    if (!std::isfinite(rope->amplitude)) return RA_ERR_INVALID_ARG;
    return aligned(rope->phases, 8) ? RA_OK : RA_ERR_MISALIGNED;
}

// The checks of a call that rotates q into q_out and k into k_out, and its arguments for the
// kernels.  rope may be NULL where a norm goes before it (norm: whether one does).
ra_status rope_args(const ra_rope_desc* d, const ra_rope* rope, bool norm, const void* q, const void* k,
                    void* q_out, void* k_out, float sign, ra_stream_t stream, ra::RopeArgs* args)
{
    if (!d) return RA_ERR_INVALID_ARG;
    if (d->B < 1 || d->L < 1 || d->D < 1 || d->P < 1 || d->H < 0 || d->H_kv < 0 ||
        d->H + static_cast<long long>(d->H_kv) < 1)
        return RA_ERR_INVALID_ARG;
    if (d->dtype != RA_BF16 && d->dtype != RA_F32) return RA_ERR_UNSUPPORTED;
    const int elem = d->dtype == RA_BF16 ? 2 : 4;
    if ((d->D * elem) % 16 != 0 || d->D > 256) return RA_ERR_UNSUPPORTED;
    ra_status st = norm && !rope ? RA_OK : check_rope(rope, d->D);
    if (st != RA_OK) return st;
    if ((d->H > 0) != (q != nullptr) || (d->H > 0) != (q_out != nullptr) ||
        (d->H_kv > 0) != (k != nullptr) || (d->H_kv > 0) != (k_out != nullptr))
        return RA_ERR_INVALID_ARG;
    switch (d->layout) {
    case RA_LAYOUT_CONTIGUOUS:
        if (d->cu_seqlens) return RA_ERR_INVALID_ARG;
        if (d->L % d->P != 0) return RA_ERR_NOT_DIVISIBLE;
        break;
    case RA_LAYOUT_ZIGZAG:
        if (d->cu_seqlens) return RA_ERR_INVALID_ARG;
        if (d->P > d->L || d->L % (2ll * d->P) != 0) return RA_ERR_NOT_DIVISIBLE;
        break;
    case RA_LAYOUT_PACKED:
        if (!d->cu_seqlens || d->n_seqs < 1 || d->B != 1) return RA_ERR_INVALID_ARG;
        if (!aligned(d->cu_seqlens, 4)) return RA_ERR_MISALIGNED;
        if (d->L % d->P != 0) return RA_ERR_NOT_DIVISIBLE;
        break;
    default:
        return RA_ERR_INVALID_ARG;
    }
    // positions given and positions of a layout exclude one another
    if (d->positions && d->layout != RA_LAYOUT_CONTIGUOUS) return RA_ERR_INVALID_ARG;
    if (d->positions && !aligned(d->positions, 4)) return RA_ERR_MISALIGNED;

    ra::RopeArgs& a = *args;
    a = {};
    a.rows = static_cast<long long>(d->B) * d->L;
    const long long nq = static_cast<long long>(d->H) * d->D, nk = static_cast<long long>(d->H_kv) * d->D;
    if (nq + nk > 0x7fffffffll || static_cast<ull>(a.rows) * (nq + nk) >= kMaxElems)
        return RA_ERR_INVALID_ARG;
    a.q_stride = d->q_stride;
    a.k_stride = d->k_stride;
    a.q_out_stride = d->q_out_stride;
    a.k_out_stride = d->k_out_stride;
    if (nq > 0 && ((st = row_stride(&a.q_stride, nq, elem)) != RA_OK ||
                   (st = row_stride(&a.q_out_stride, nq, elem)) != RA_OK))
        return st;
    if (nk > 0 && ((st = row_stride(&a.k_stride, nk, elem)) != RA_OK ||
                   (st = row_stride(&a.k_out_stride, nk, elem)) != RA_OK))
        return st;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
        return RA_ERR_MISALIGNED;
    const ull n = static_cast<ull>(a.rows);
    const Rows rq{q, n, static_cast<ull>(nq) * elem, static_cast<ull>(a.q_stride) * elem};
    const Rows rk{k, n, static_cast<ull>(nk) * elem, static_cast<ull>(a.k_stride) * elem};
    const Rows rqo{q_out, n, static_cast<ull>(nq) * elem, static_cast<ull>(a.q_out_stride) * elem};
    const Rows rko{k_out, n, static_cast<ull>(nk) * elem, static_cast<ull>(a.k_out_stride) * elem};
    const void* phases = rope ? rope->phases : nullptr;
    const ull phase_bytes = rope ? 4ull * rope->rot_dim : 0;
    // in place (the same rows) is allowed, any other overlap is not
    const bool q_in_place = q == q_out && a.q_stride == a.q_out_stride;
    const bool k_in_place = k == k_out && a.k_stride == a.k_out_stride;
    if (nq > 0 && ((!q_in_place && overlap(rqo, rq)) || (nk > 0 && overlap(rqo, rk)) ||
                   overlap(q_out, rqo.span(), phases, phase_bytes)))
        return RA_ERR_INVALID_ARG;
    if (nk > 0 && ((!k_in_place && overlap(rko, rk)) || (nq > 0 && overlap(rko, rq)) ||
                   overlap(k_out, rko.span(), phases, phase_bytes)))
        return RA_ERR_INVALID_ARG;
    if (nq > 0 && nk > 0 && overlap(rqo, rko)) return RA_ERR_INVALID_ARG;
    if (d->positions && (overlap(q_out, rqo.span(), d->positions, 4 * n) ||
                         overlap(k_out, rko.span(), d->positions, 4 * n)))
        return RA_ERR_INVALID_ARG;
    if (d->cu_seqlens && (overlap(q_out, rqo.span(), d->cu_seqlens, 4ull * d->n_seqs + 4) ||
                          overlap(k_out, rko.span(), d->cu_seqlens, 4ull * d->n_seqs + 4)))
        return RA_ERR_INVALID_ARG;
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_elems = nq > 0 ? (a.rows - 1) * a.q_stride + nq : 0;
    a.k_elems = nk > 0 ? (a.rows - 1) * a.k_stride + nk : 0;
    a.q_out_elems = nq > 0 ? (a.rows - 1) * a.q_out_stride + nq : 0;
    a.k_out_elems = nk > 0 ? (a.rows - 1) * a.k_out_stride + nk : 0;
    a.L = d->L;
    a.P = d->P;
    a.H = d->H;
    a.H_kv = d->H_kv;
    a.D = d->D;
    a.elem = elem;
    a.rot = rope ? rope->rot_dim : 0;
    a.half_style = !rope || rope->style == RA_ROPE_HALF;
    a.amplitude = rope ? rope->amplitude : 1.f;
    a.sign = sign;
    a.phases = rope ? rope->phases : nullptr;
    a.layout = d->layout;
    a.positions = d->positions;
    a.position_offset = d->position_offset;
    a.cu_seqlens = d->cu_seqlens;
    a.n_seqs = d->n_seqs;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return RA_OK;
}

ra_status rope_impl(const ra_rope_desc* d, const ra_rope* rope, const void* q, const void* k,
                    void* q_out, void* k_out, float sign, ra_stream_t stream)
{
    ra::RopeArgs a;
    ra_status st = rope_args(d, rope, false, q, k, q_out, k_out, sign, stream, &a);
    if (st == RA_OK) st = ra::current_status_word(&a.status);
    return st != RA_OK ? st : from_cuda(ra::launch_rope(a));
}

// The norm's part of the arguments of a call with heads of D dims; the outputs outs[i] of
// bytes[i] must not share memory with the weights.
ra_status norm_args(const ra_head_norm* norm, int D, void* const* outs, const ull* bytes, int n_outs,
                    ra::NormArgs* n)
{
    if (!norm) return RA_ERR_INVALID_ARG;
    if (norm->weight_dtype != RA_BF16 && norm->weight_dtype != RA_F32) return RA_ERR_UNSUPPORTED;
    if (!(norm->eps >= 0) || !std::isfinite(norm->eps) || !std::isfinite(norm->weight_offset))
        return RA_ERR_INVALID_ARG;
    n->weight_elem = norm->weight_dtype == RA_BF16 ? 2 : 4;
    n->q_weight = norm->q_weight;
    n->k_weight = norm->k_weight;
    n->eps = norm->eps;
    n->weight_offset = norm->weight_offset;
    for (const void* w : {norm->q_weight, norm->k_weight}) {
        if (!aligned(w, n->weight_elem)) return RA_ERR_MISALIGNED;
        for (int i = 0; w && i < n_outs; ++i)
            if (overlap(outs[i], bytes[i], w, static_cast<ull>(D) * n->weight_elem))
                return RA_ERR_INVALID_ARG;
    }
    return RA_OK;
}


// The cache's extent in elements; RA_OK only if distinct (layer, page, slot, head) quadruples are
// distinct memory and every head vector starts on a 16-byte boundary.
struct Dim {
    ull size, stride;
};
ra_status page_extent(const ra_paged_desc* d, int layers, long long layer_stride, int elem, ull* elems,
                      Dim (&dims)[4])
{
    dims[0] = {static_cast<ull>(d->num_pages), static_cast<ull>(d->page_stride)};
    dims[1] = {static_cast<ull>(d->page_size), static_cast<ull>(d->token_stride)};
    dims[2] = {static_cast<ull>(d->H_kv), static_cast<ull>(d->head_stride)};
    dims[3] = {static_cast<ull>(layers), static_cast<ull>(layer_stride)};
    if (layer_stride < 0 || d->page_stride < 0 || d->token_stride < 0 || d->head_stride < 0) return RA_ERR_INVALID_ARG;
    for (const Dim& x : dims) {
        if (x.stride >= kMaxElems) return RA_ERR_INVALID_ARG;
        if (x.size > 1 && (x.stride * elem) % 16 != 0) return RA_ERR_MISALIGNED;
    }
    std::sort(dims, dims + 4, [](const Dim& a, const Dim& b) {
        return a.stride != b.stride ? a.stride < b.stride : a.size < b.size;
    });
    ull span = static_cast<ull>(d->D);
    for (const Dim& x : dims) {
        if (x.size == 1) continue;
        if (x.stride < span) return RA_ERR_INVALID_ARG;
        span += (x.size - 1) * x.stride;
        if (span >= kMaxElems) return RA_ERR_INVALID_ARG;
    }
    *elems = span;
    return RA_OK;
}

// Whether two caches of one geometry share memory.  Interleaved views of one buffer (keys
// and values of a page, of a token or of a head side by side) do not.
bool pages_overlap(const void* k, const void* v, const Dim (&dims)[4], ull D, ull span, int elem)
{
    if (!overlap(k, span * elem, v, span * elem)) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(k), y = reinterpret_cast<uintptr_t>(v);
    const ull bytes = x < y ? y - x : x - y;
    if (bytes % elem != 0) return true;
    ull delta = bytes / elem;
    // spans of the dims inside each level, outermost first
    ull inner[4], s = D;
    for (int i = 0; i < 4; ++i) {
        inner[i] = s;
        if (dims[i].size > 1) s += (dims[i].size - 1) * dims[i].stride;
    }
    for (int i = 3; i >= 0; --i) {
        if (dims[i].size == 1) continue;
        delta %= dims[i].stride;
        if (delta >= inner[i] && dims[i].stride - delta >= inner[i]) return false;
        for (int j = i - 1; j >= 0; --j)
            if (dims[j].size > 1) {
                if (dims[i].stride % dims[j].stride != 0) return true;
                break;
            }
    }
    return true;
}

ra_status check_paged(const ra_paged_desc* d, int* elem, ull* page_elems, Dim (&dims)[4], int layers = 1,
                      long long layer_stride = 0)
{
    if (!d) return RA_ERR_INVALID_ARG;
    if (d->T < 0 || d->n_seqs < 1 || d->H_kv < 1 || d->D < 1 || d->num_pages < 1 ||
        d->page_size < 1 || d->max_pages < 1)
        return RA_ERR_INVALID_ARG;
    if (d->dtype != RA_BF16 && d->dtype != RA_F32) return RA_ERR_UNSUPPORTED;
    if (!d->page_table || !d->cu_new || !d->kv_lens) return RA_ERR_INVALID_ARG;
    if (!aligned(d->page_table, 4) || !aligned(d->cu_new, 4) || !aligned(d->kv_lens, 4))
        return RA_ERR_MISALIGNED;
    if (d->table_stride < d->max_pages) return RA_ERR_INVALID_ARG;
    *elem = d->dtype == RA_BF16 ? 2 : 4;
    return page_extent(d, layers, layer_stride, *elem, page_elems, dims);
}

struct Span {
    const void* base;
    ull bytes;
};

// The checks of a pool and a page table with it, and their part of the kernels' arguments.
ra_status pool_args(const ra_page_pool* pool, const int* lens, int* page_table, int max_pages,
                    long long table_stride, int page_size, ra::ReserveArgs* r)
{
    if (!pool || !pool->free_pages || !pool->held || !pool->state || !lens || !page_table)
        return RA_ERR_INVALID_ARG;
    if (pool->num_pages < 1 || pool->n_seqs < 1 || max_pages < 1 || page_size < 1) return RA_ERR_INVALID_ARG;
    if (pool->n_seqs > ra::kPoolSeqs || pool->num_pages > 0x7fffffff - 1024) return RA_ERR_UNSUPPORTED;
    if (table_stride < max_pages || table_stride >= static_cast<long long>(kMaxElems)) return RA_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(pool->free_pages), static_cast<const void*>(pool->held),
                          static_cast<const void*>(pool->state), static_cast<const void*>(lens),
                          static_cast<const void*>(page_table)})
        if (!aligned(p, 4)) return RA_ERR_MISALIGNED;
    ra::PoolArgs& a = r->pool;
    a.free_pages = pool->free_pages;
    a.held = pool->held;
    a.state = pool->state;
    a.page_table = page_table;
    a.table_stride = table_stride;
    a.table_elems = (pool->n_seqs - 1ll) * table_stride + max_pages;
    a.num_pages = pool->num_pages;
    a.n_seqs = pool->n_seqs;
    a.max_pages = max_pages;
    a.page_size = page_size;
    return RA_OK;
}

// paged_attn_fwd, and paged_attn_tree_fwd with the new tokens' masks.
ra_status attn_impl(const ra_paged_desc* d, const int* masks, int mask_words, long long mask_stride,
                    const void* q, long long q_stride, const void* k_pages, const void* v_pages,
                    void* out, float* lse, void* workspace, unsigned long long workspace_bytes,
                    ra_stream_t stream)
{
    int elem = 0;
    ull page_elems = 0;
    Dim dims[4];
    ra_status st = check_paged(d, &elem, &page_elems, dims);
    if (st != RA_OK) return st;
    const ull need = paged_attn_workspace_bytes(d->D, d->dtype);
    if (need == 0) return RA_ERR_UNSUPPORTED;
    if (!q || !k_pages || !v_pages || !out || !workspace) return RA_ERR_INVALID_ARG;
    if (d->H < 1) return RA_ERR_INVALID_ARG;
    if (d->H % d->H_kv != 0) return RA_ERR_NOT_DIVISIBLE;
    const long long nq = static_cast<long long>(d->H) * d->D;
    if (nq > 0x7fffffffll || static_cast<ull>(d->T) * nq >= kMaxElems ||
        static_cast<ull>(d->T) * d->H > 0x7fffff00ull)
        return RA_ERR_INVALID_ARG;
    if ((st = row_stride(&q_stride, nq, elem)) != RA_OK) return st;
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(workspace, 256))
        return RA_ERR_MISALIGNED;
    if (workspace_bytes < need) return RA_ERR_INVALID_ARG;
    const ull n = static_cast<ull>(d->T), pb = page_elems * elem;
    const ull ob = n * nq * elem, lb = lse ? n * d->H * 4 : 0;
    const ull table_elems = (d->n_seqs - 1ull) * d->table_stride + d->max_pages;
    const Rows rq{q, n, static_cast<ull>(nq) * elem, static_cast<ull>(q_stride) * elem};
    const long long mask_elems = masks && n > 0 ? (static_cast<long long>(n) - 1) * mask_stride + mask_words : 0;
    if (mask_elems >= static_cast<long long>(kMaxElems)) return RA_ERR_INVALID_ARG;
    const void* ins[7] = {q, k_pages, v_pages, d->page_table, d->cu_new, d->kv_lens, masks};
    const ull in_bytes[7] = {rq.span(), pb, pb, 4 * table_elems, 4ull * d->n_seqs + 4, 4ull * d->n_seqs,
                             4ull * mask_elems};
    for (int i = 0; i < 7; ++i)
        if (overlap(out, ob, ins[i], in_bytes[i]) || overlap(lse, lb, ins[i], in_bytes[i]) ||
            overlap(workspace, need, ins[i], in_bytes[i]))
            return RA_ERR_INVALID_ARG;
    if (overlap(out, ob, lse, lb) || overlap(out, ob, workspace, need) ||
        overlap(lse, lb, workspace, need))
        return RA_ERR_INVALID_ARG;
    if (d->T == 0) return RA_OK;
    ra::PagedArgs a{};
    a.q = q;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.q_stride = q_stride;
    a.q_elems = (static_cast<long long>(d->T) - 1) * q_stride + nq;
    a.page_elems = static_cast<long long>(page_elems);
    a.out_elems = static_cast<long long>(n) * nq;
    a.lse_elems = static_cast<long long>(n) * d->H;
    a.table_elems = static_cast<long long>(table_elems);
    a.page_stride = d->page_stride;
    a.token_stride = d->token_stride;
    a.head_stride = d->head_stride;
    a.table_stride = d->table_stride;
    a.T = d->T;
    a.n_seqs = d->n_seqs;
    a.H = d->H;
    a.H_kv = d->H_kv;
    a.D = d->D;
    a.elem = elem;
    // a tree's rows may see any of the new tokens: their tiles run to the last key
    a.causal = d->causal && !masks ? 1 : 0;
    a.masks = masks;
    a.mask_words = mask_words;
    a.mask_stride = mask_stride;
    a.mask_elems = mask_elems;
    a.num_pages = d->num_pages;
    a.page_size = d->page_size;
    a.max_pages = d->max_pages;
    a.cu_new = d->cu_new;
    a.kv_lens = d->kv_lens;
    a.page_table = d->page_table;
    a.timeout_ns = kWaitLimitNs;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    st = ra::current_status_word(&a.status);
    if (st != RA_OK) return st;
    return from_cuda(ra::launch_paged(a));
}

}  // namespace

extern "C" {

ra_status ra_rope_phases(const ra_rope_config* c, unsigned long long* phases, float* amplitude)
{
    if (!c || !phases || !amplitude) return RA_ERR_INVALID_ARG;
    if (c->rot_dim < 2 || c->rot_dim % 2 != 0 || !(c->base > 0) || !std::isfinite(c->base))
        return RA_ERR_INVALID_ARG;
    if (c->scaling != RA_ROPE_NONE && (!(c->factor > 0) || !std::isfinite(c->factor)))
        return RA_ERR_INVALID_ARG;
    const double pi2 = 6.283185307179586476925286766559;
    double base = c->base, lo = 0, hi = 0;
    *amplitude = 1.f;
    switch (c->scaling) {
    case RA_ROPE_NONE:
    case RA_ROPE_LINEAR:
        break;
    case RA_ROPE_NTK:
        if (c->rot_dim > 2) base *= std::pow(c->factor, c->rot_dim / (c->rot_dim - 2.0));
        break;
    case RA_ROPE_YARN: {
        if (!(c->original_length > 0) || !(c->beta_slow > 0) || !(c->beta_fast > c->beta_slow) ||
            !std::isfinite(c->original_length) || !std::isfinite(c->beta_fast) || c->base == 1.0)
            return RA_ERR_INVALID_ARG;
        // the pair that makes beta turns over the original length
        auto pair_of = [&](double beta) {
            return c->rot_dim * std::log(c->original_length / (beta * pi2)) / (2 * std::log(base));
        };
        lo = std::max(std::floor(pair_of(c->beta_fast)), 0.0);
        hi = std::min(std::ceil(pair_of(c->beta_slow)), c->rot_dim - 1.0);
        if (c->factor > 1) *amplitude = static_cast<float>(0.1 * std::log(c->factor) + 1.0);
        break;
    }
    default:
        return RA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < c->rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / c->rot_dim);
        if (c->scaling == RA_ROPE_LINEAR) f /= c->factor;
        if (c->scaling == RA_ROPE_YARN) {
            const double slow = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            f = f * (1 - slow) + f / c->factor * slow;
        }
        const ra_status st = ra_rope_phases_of(&f, 1, phases + i);
        if (st != RA_OK) return st;
    }
    return RA_OK;
}

ra_status ra_rope_phases_of(const double* inv_freq, int n, unsigned long long* phases)
{
    if (!inv_freq || !phases || n < 1) return RA_ERR_INVALID_ARG;
    const double pi2 = 6.283185307179586476925286766559;
    for (int i = 0; i < n; ++i) {
        if (!std::isfinite(inv_freq[i])) return RA_ERR_INVALID_ARG;
        // fraction of a turn in [0, 1), then 2^64 of it (below 2^64: a double under 1 is at
        // most 1 - 2^-53)
        double turns = inv_freq[i] / pi2;
        turns -= std::floor(turns);
        if (turns >= 1.0) turns = 0.0;          // a tiny negative angle rounds up to a turn
        phases[i] = static_cast<unsigned long long>(std::ldexp(turns, 64));
    }
    return RA_OK;
}

ra_status rope_fwd(const ra_rope_desc* desc, const ra_rope* rope, const void* q, const void* k,
                   void* q_out, void* k_out, ra_stream_t stream)
{
    return rope_impl(desc, rope, q, k, q_out, k_out, 1.f, stream);
}

ra_status rope_bwd(const ra_rope_desc* desc, const ra_rope* rope, const void* dq_out,
                   const void* dk_out, void* dq, void* dk, ra_stream_t stream)
{
    return rope_impl(desc, rope, dq_out, dk_out, dq, dk, -1.f, stream);
}

ra_status paged_kv_append(const ra_paged_desc* d, const ra_rope* rope, const void* q,
                          long long q_stride, const void* k, long long k_stride, const void* v,
                          long long v_stride, void* q_out, long long q_out_stride, void* k_pages,
                          void* v_pages, ra_stream_t stream)
{
    return paged_kv_append_ex(d, rope, nullptr, nullptr, q, q_stride, k, k_stride, v, v_stride, q_out,
                              q_out_stride, k_pages, v_pages, stream);
}

ra_status paged_kv_append_ex(const ra_paged_desc* d, const ra_rope* rope, const ra_head_norm* norm,
                             const int* positions, const void* q, long long q_stride, const void* k,
                             long long k_stride, const void* v, long long v_stride, void* q_out,
                             long long q_out_stride, void* k_pages, void* v_pages, ra_stream_t stream)
{
    int elem = 0;
    ull page_elems = 0;
    Dim dims[4];
    ra_status st = check_paged(d, &elem, &page_elems, dims);
    if (st != RA_OK) return st;
    if ((d->D * elem) % 16 != 0 || d->D > 256) return RA_ERR_UNSUPPORTED;
    if (rope && (st = check_rope(rope, d->D)) != RA_OK) return st;
    if (!k || !v || !k_pages || !v_pages || (q != nullptr) != (q_out != nullptr))
        return RA_ERR_INVALID_ARG;
    if (q && d->H < 1) return RA_ERR_INVALID_ARG;
    const int H = q ? d->H : 0;
    const long long nq = static_cast<long long>(H) * d->D, nk = static_cast<long long>(d->H_kv) * d->D;
    if (nq + 2 * nk > 0x7fffffffll || static_cast<ull>(d->T) * (nq + 2 * nk) >= kMaxElems)
        return RA_ERR_INVALID_ARG;
    if (q && ((st = row_stride(&q_stride, nq, elem)) != RA_OK ||
              (st = row_stride(&q_out_stride, nq, elem)) != RA_OK))
        return st;
    if ((st = row_stride(&k_stride, nk, elem)) != RA_OK ||
        (st = row_stride(&v_stride, nk, elem)) != RA_OK)
        return st;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
        !aligned(k_pages, 16) || !aligned(v_pages, 16))
        return RA_ERR_MISALIGNED;
    const ull n = static_cast<ull>(d->T), pb = page_elems * elem;
    const ull table_elems = (d->n_seqs - 1ull) * d->table_stride + d->max_pages;
    const Rows rq{q, q ? n : 0, static_cast<ull>(nq) * elem, static_cast<ull>(q_stride) * elem};
    const Rows rqo{q_out, q ? n : 0, static_cast<ull>(nq) * elem, static_cast<ull>(q_out_stride) * elem};
    const Rows rk{k, n, static_cast<ull>(nk) * elem, static_cast<ull>(k_stride) * elem};
    const Rows rv{v, n, static_cast<ull>(nk) * elem, static_cast<ull>(v_stride) * elem};
    const bool in_place = q == q_out && q_stride == q_out_stride;
    if ((!in_place && overlap(rqo, rq)) || overlap(rqo, rk) || overlap(rqo, rv))
        return RA_ERR_INVALID_ARG;
    for (void* pages : {k_pages, v_pages})
        for (const Rows& r : {rq, rqo, rk, rv})
            if (overlap(pages, pb, r.base, r.span())) return RA_ERR_INVALID_ARG;
    if (pages_overlap(k_pages, v_pages, dims, d->D, page_elems, elem)) return RA_ERR_INVALID_ARG;
    if (!aligned(positions, 4)) return RA_ERR_MISALIGNED;
    const void* ins[5] = {d->page_table, d->cu_new, d->kv_lens, rope ? rope->phases : nullptr, positions};
    const ull in_bytes[5] = {4 * table_elems, 4ull * d->n_seqs + 4, 4ull * d->n_seqs,
                             rope ? 4ull * rope->rot_dim : 0, 4 * n};
    for (int i = 0; i < 5; ++i)
        if (overlap(k_pages, pb, ins[i], in_bytes[i]) || overlap(v_pages, pb, ins[i], in_bytes[i]) ||
            overlap(q_out, rqo.span(), ins[i], in_bytes[i]))
            return RA_ERR_INVALID_ARG;
    ra::NormArgs args{};
    void* const outs[3] = {q_out, k_pages, v_pages};
    const ull out_bytes[3] = {rqo.span(), pb, pb};
    if (norm && (st = norm_args(norm, d->D, outs, out_bytes, 3, &args)) != RA_OK) return st;
    if (d->T == 0) return RA_OK;
    ra::RopeArgs& a = args.rope;
    a.paged = 1;
    a.rows = d->T;
    a.L = d->T;
    a.P = 1;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_pages;
    a.v_out = v_pages;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.q_elems = q ? (a.rows - 1) * q_stride + nq : 0;
    a.q_out_elems = q ? (a.rows - 1) * q_out_stride + nq : 0;
    a.k_elems = (a.rows - 1) * k_stride + nk;
    a.v_elems = (a.rows - 1) * v_stride + nk;
    a.k_out_elems = static_cast<long long>(page_elems);
    a.H = H;
    a.H_kv = d->H_kv;
    a.D = d->D;
    a.elem = elem;
    a.rot = rope ? rope->rot_dim : 0;
    a.half_style = !rope || rope->style == RA_ROPE_HALF;
    a.amplitude = rope ? rope->amplitude : 1.f;
    a.sign = 1.f;
    a.phases = rope ? rope->phases : nullptr;
    a.layout = RA_LAYOUT_PACKED;
    a.positions = positions;
    a.cu_seqlens = d->cu_new;
    a.n_seqs = d->n_seqs;
    a.kv_lens = d->kv_lens;
    a.page_table = d->page_table;
    a.table_stride = d->table_stride;
    a.table_elems = static_cast<long long>(table_elems);
    a.page_stride = d->page_stride;
    a.token_stride = d->token_stride;
    a.head_stride = d->head_stride;
    a.num_pages = d->num_pages;
    a.page_size = d->page_size;
    a.max_pages = d->max_pages;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    st = ra::current_status_word(&a.status);
    if (st != RA_OK) return st;
    return from_cuda(norm ? ra::launch_norm(args) : ra::launch_rope(a));
}

unsigned long long paged_attn_workspace_bytes(int D, ra_dtype dtype)
{
    if (dtype == RA_BF16 && D != 64 && D != 128) return 0;
    if (dtype == RA_F32 && (D < 4 || D % 4 != 0 || D > 256)) return 0;
    if (dtype != RA_BF16 && dtype != RA_F32) return 0;
    return ra::paged_workspace_bytes(D, dtype == RA_BF16 ? 2 : 4);
}

ra_status paged_attn_fwd(const ra_paged_desc* d, const void* q, long long q_stride,
                         const void* k_pages, const void* v_pages, void* out, float* lse,
                         void* workspace, unsigned long long workspace_bytes, ra_stream_t stream)
{
    return attn_impl(d, nullptr, 0, 0, q, q_stride, k_pages, v_pages, out, lse, workspace,
                     workspace_bytes, stream);
}

ra_status paged_attn_tree_fwd(const ra_paged_desc* d, const int* masks, int mask_words,
                              long long mask_stride, const void* q, long long q_stride,
                              const void* k_pages, const void* v_pages, void* out, float* lse,
                              void* workspace, unsigned long long workspace_bytes, ra_stream_t stream)
{
    if (!masks || mask_words < 1) return RA_ERR_INVALID_ARG;
    if (!aligned(masks, 4)) return RA_ERR_MISALIGNED;
    if (mask_stride == 0) mask_stride = mask_words;
    if (mask_stride < mask_words || mask_stride >= static_cast<long long>(kMaxElems)) return RA_ERR_INVALID_ARG;
    return attn_impl(d, masks, mask_words, mask_stride, q, q_stride, k_pages, v_pages, out, lse, workspace,
                     workspace_bytes, stream);
}

unsigned long long qk_norm_workspace_bytes(void) { return 256 + 2048ull * ra::kNormCtas; }

ra_status qk_norm_rope_fwd(const ra_rope_desc* desc, const ra_rope* rope, const ra_head_norm* norm,
                           const void* q, const void* k, void* q_out, void* k_out, ra_stream_t stream)
{
    ra::NormArgs n{};
    ra_status st = rope_args(desc, rope, true, q, k, q_out, k_out, 1.f, stream, &n.rope);
    if (st != RA_OK) return st;
    void* const outs[2] = {q_out, k_out};
    const ull bytes[2] = {static_cast<ull>(n.rope.q_out_elems) * n.rope.elem,
                          static_cast<ull>(n.rope.k_out_elems) * n.rope.elem};
    st = norm_args(norm, n.rope.D, outs, bytes, 2, &n);
    if (st == RA_OK) st = ra::current_status_word(&n.rope.status);
    return st != RA_OK ? st : from_cuda(ra::launch_norm(n));
}

ra_status qk_norm_rope_bwd(const ra_rope_desc* desc, const ra_rope* rope, const ra_head_norm* norm,
                           const void* q, const void* k, const void* dq_out, long long dq_out_stride,
                           const void* dk_out, long long dk_out_stride, void* dq, void* dk,
                           float* dq_weight, float* dk_weight, void* workspace,
                           unsigned long long workspace_bytes, ra_stream_t stream)
{
    ra::NormArgs n{};
    ra_status st = rope_args(desc, rope, true, q, k, dq, dk, 1.f, stream, &n.rope);
    if (st != RA_OK) return st;
    ra::RopeArgs& a = n.rope;
    const long long nq = static_cast<long long>(a.H) * a.D, nk = static_cast<long long>(a.H_kv) * a.D;
    if ((nq > 0) != (dq_out != nullptr) || (nk > 0) != (dk_out != nullptr) || (!nq && dq_weight) ||
        (!nk && dk_weight) || !workspace || workspace_bytes < qk_norm_workspace_bytes())
        return RA_ERR_INVALID_ARG;
    if (nq > 0 && (st = row_stride(&dq_out_stride, nq, a.elem)) != RA_OK) return st;
    if (nk > 0 && (st = row_stride(&dk_out_stride, nk, a.elem)) != RA_OK) return st;
    if (!aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) ||
        !aligned(workspace, 256))
        return RA_ERR_MISALIGNED;
    const ull r = static_cast<ull>(a.rows), e = static_cast<ull>(a.elem);
    const Rows rx[2] = {{q, nq ? r : 0, nq * e, a.q_stride * e}, {k, nk ? r : 0, nk * e, a.k_stride * e}};
    const Rows ry[2] = {{dq_out, nq ? r : 0, nq * e, dq_out_stride * e},
                        {dk_out, nk ? r : 0, nk * e, dk_out_stride * e}};
    const Rows rd[2] = {{dq, nq ? r : 0, nq * e, a.q_out_stride * e}, {dk, nk ? r : 0, nk * e, a.k_out_stride * e}};
    // over its own upstream gradient a gradient may be written, over nothing else of them
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (!(i == j && rd[i].base == ry[j].base && rd[i].stride == ry[j].stride) && overlap(rd[i], ry[j]))
                return RA_ERR_INVALID_ARG;
    void* const outs[5] = {dq_weight, dk_weight, workspace, dq, dk};
    const ull bytes[5] = {dq_weight ? 4ull * a.D : 0, dk_weight ? 4ull * a.D : 0, qk_norm_workspace_bytes(),
                          rd[0].span(), rd[1].span()};
    for (int i = 0; i < 3; ++i) {
        for (const Rows* x : {rx, rx + 1, ry, ry + 1})
            if (overlap(outs[i], bytes[i], x->base, x->span())) return RA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 5; ++j)
            if (overlap(outs[i], bytes[i], outs[j], bytes[j])) return RA_ERR_INVALID_ARG;
        if (overlap(outs[i], bytes[i], a.phases, 4ull * a.rot) || overlap(outs[i], bytes[i], a.positions, 4 * r) ||
            overlap(outs[i], bytes[i], a.cu_seqlens, a.cu_seqlens ? 4ull * a.n_seqs + 4 : 0))
            return RA_ERR_INVALID_ARG;
    }
    if ((st = norm_args(norm, a.D, outs, bytes, 5, &n)) != RA_OK) return st;
    n.dq_out = dq_out;
    n.dk_out = dk_out;
    n.dq_out_stride = dq_out_stride;
    n.dk_out_stride = dk_out_stride;
    n.dq_out_elems = nq ? (a.rows - 1) * dq_out_stride + nq : 0;
    n.dk_out_elems = nk ? (a.rows - 1) * dk_out_stride + nk : 0;
    n.dq_weight = dq_weight;
    n.dk_weight = dk_weight;
    n.ticket = static_cast<unsigned int*>(workspace);
    n.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
    st = ra::current_status_word(&a.status);
    return st != RA_OK ? st : from_cuda(ra::launch_norm_bwd(n));
}

ra_status paged_reserve(const ra_page_pool* pool, const int* new_lens, const int* lens, int* page_table,
                        int max_pages, long long table_stride, int page_size, int T, int* cu_new,
                        int* kv_lens, int* positions, long long* slots, const int* parents, int* masks,
                        int mask_words, ra_stream_t stream)
{
    return paged_reserve_ex(pool, new_lens, lens, page_table, max_pages, table_stride, page_size, T, cu_new,
                            kv_lens, positions, slots, parents, masks, mask_words, nullptr, stream);
}

ra_status paged_reserve_ex(const ra_page_pool* pool, const int* new_lens, const int* lens, int* page_table,
                           int max_pages, long long table_stride, int page_size, int T, int* cu_new,
                           int* kv_lens, int* positions, long long* slots, const int* parents, int* masks,
                           int mask_words, int* unmasked, ra_stream_t stream)
{
    ra::ReserveArgs r{};
    ra_status st = pool_args(pool, lens, page_table, max_pages, table_stride, page_size, &r);
    if (st != RA_OK) return st;
    const ull n = static_cast<ull>(pool->n_seqs), t = static_cast<ull>(std::max(T, 0));
    if (!new_lens || !cu_new || !kv_lens || T < 0 || mask_words < 0 || (mask_words > 0) != (masks != nullptr) ||
        t * static_cast<ull>(mask_words) >= kMaxElems)
        return RA_ERR_INVALID_ARG;
    if (T > 0x7fffffff - 1024) return RA_ERR_UNSUPPORTED;
    for (const void* p : {static_cast<const void*>(new_lens), static_cast<const void*>(cu_new),
                          static_cast<const void*>(kv_lens), static_cast<const void*>(positions),
                          static_cast<const void*>(parents), static_cast<const void*>(masks),
                          static_cast<const void*>(unmasked)})
        if (!aligned(p, 4)) return RA_ERR_MISALIGNED;
    if (!aligned(slots, 8)) return RA_ERR_MISALIGNED;
    // what is written, and what is only read; kv_lens may be lens
    const Span outs[10] = {{cu_new, 4 * n + 4}, {kv_lens, 4 * n}, {positions, positions ? 4 * t : 0},
                          {slots, slots ? 8 * t : 0}, {masks, masks ? 4 * t * mask_words : 0},
                          {page_table, 4ull * r.pool.table_elems}, {pool->held, 4 * n}, {pool->state, 12},
                          {pool->free_pages, 4ull * pool->num_pages}, {unmasked, unmasked ? 4ull : 0}};
    const Span ins[3] = {{new_lens, 4 * n}, {parents, parents ? 4 * t : 0}, {lens, 4 * n}};
    for (int i = 0; i < 10; ++i) {
        for (int j = i + 1; j < 10; ++j)
            if (overlap(outs[i].base, outs[i].bytes, outs[j].base, outs[j].bytes)) return RA_ERR_INVALID_ARG;
        for (int j = 0; j < 3; ++j)
            if (!(i == 1 && j == 2 && kv_lens == lens) &&
                overlap(outs[i].base, outs[i].bytes, ins[j].base, ins[j].bytes))
                return RA_ERR_INVALID_ARG;
    }
    r.new_lens = new_lens;
    r.lens = lens;
    r.cu_new = cu_new;
    r.kv_lens = kv_lens;
    r.positions = positions;
    r.slots = slots;
    r.parents = parents;
    r.masks = masks;
    r.unmasked = unmasked;
    r.T = T;
    r.mask_words = mask_words;
    r.stream = reinterpret_cast<cudaStream_t>(stream);
    st = ra::current_status_word(&r.pool.status);
    return st != RA_OK ? st : from_cuda(ra::launch_reserve(r));
}

ra_status paged_release(const ra_page_pool* pool, const int* lens, int* page_table, int max_pages,
                        long long table_stride, int page_size, ra_stream_t stream)
{
    ra::ReserveArgs r{};
    ra_status st = pool_args(pool, lens, page_table, max_pages, table_stride, page_size, &r);
    if (st != RA_OK) return st;
    const ull n = static_cast<ull>(pool->n_seqs);
    const Span all[5] = {{page_table, 4ull * r.pool.table_elems}, {pool->held, 4 * n}, {pool->state, 12},
                         {pool->free_pages, 4ull * pool->num_pages}, {lens, 4 * n}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (overlap(all[i].base, all[i].bytes, all[j].base, all[j].bytes)) return RA_ERR_INVALID_ARG;
    r.lens = lens;
    r.stream = reinterpret_cast<cudaStream_t>(stream);
    st = ra::current_status_word(&r.pool.status);
    return st != RA_OK ? st : from_cuda(ra::launch_release(r));
}

ra_status paged_kv_keep(const ra_paged_desc* d, const int* kept, int width, long long kept_stride, int layers,
                        long long layer_stride, void* k_pages, void* v_pages, int* lens, ra_stream_t stream)
{
    int elem = 0;
    ull page_elems = 0;
    Dim dims[4];
    if (layers < 1) return RA_ERR_INVALID_ARG;
    const ra_status st = check_paged(d, &elem, &page_elems, dims, layers, layers > 1 ? layer_stride : 0);
    if (st != RA_OK) return st;
    if ((d->D * elem) % 16 != 0) return RA_ERR_UNSUPPORTED;
    if (!kept || !k_pages || !v_pages || !lens || width < 1) return RA_ERR_INVALID_ARG;
    if (kept_stride == 0) kept_stride = width;
    if (kept_stride < width || kept_stride >= static_cast<long long>(kMaxElems)) return RA_ERR_INVALID_ARG;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(kept, 4) || !aligned(lens, 4))
        return RA_ERR_MISALIGNED;
    const ull n = static_cast<ull>(d->n_seqs), pb = page_elems * elem;
    const ull table_elems = (n - 1) * d->table_stride + d->max_pages;
    const ull kept_elems = (n - 1) * kept_stride + width;
    if (pages_overlap(k_pages, v_pages, dims, d->D, page_elems, elem)) return RA_ERR_INVALID_ARG;
    const Span ins[4] = {{kept, 4 * kept_elems}, {d->page_table, 4 * table_elems}, {d->cu_new, 4 * n + 4},
                         {d->kv_lens, 4 * n}};
    for (const Span& x : ins)
        if (overlap(k_pages, pb, x.base, x.bytes) || overlap(v_pages, pb, x.base, x.bytes) ||
            overlap(lens, 4 * n, x.base, x.bytes))
            return RA_ERR_INVALID_ARG;
    if (overlap(lens, 4 * n, k_pages, pb) || overlap(lens, 4 * n, v_pages, pb)) return RA_ERR_INVALID_ARG;
    ra::KeepArgs a{};
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.page_stride = d->page_stride;
    a.token_stride = d->token_stride;
    a.head_stride = d->head_stride;
    a.layer_stride = layers > 1 ? layer_stride : 0;
    a.table_stride = d->table_stride;
    a.page_elems = static_cast<long long>(page_elems);
    a.table_elems = static_cast<long long>(table_elems);
    a.kept_elems = static_cast<long long>(kept_elems);
    a.kept_stride = kept_stride;
    a.layers = layers;
    a.n_seqs = d->n_seqs;
    a.H_kv = d->H_kv;
    a.D = d->D;
    a.elem = elem;
    a.num_pages = d->num_pages;
    a.page_size = d->page_size;
    a.max_pages = d->max_pages;
    a.width = width;
    a.kept = kept;
    a.page_table = d->page_table;
    a.cu_new = d->cu_new;
    a.kv_lens = d->kv_lens;
    a.lens = lens;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    const ra_status word = ra::current_status_word(&a.status);
    return word != RA_OK ? word : from_cuda(ra::launch_keep(a));
}

}  // extern "C"
