// ops_pages.cu -- host side of the page ledger, of copying pages, of the
// verification of drafted trees and of moving the accepted nodes' rows.
// Argument checks and launches; nothing here synchronises.
#include <algorithm>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "../../include/b2pa.h"
#include "host.cuh"
#include "pages.cuh"
#include "verify.cuh"

using namespace b2pa;

namespace {

// The largest power of two up to 16 that divides all of them.
int piece_of(uintptr_t all) { return all & 15u ? (int)(all & (~all + 1)) : 16; }

// The tensors of a cache as planes of bytes; kv_scales may be null.
int parse_planes(const b2pa_tensor* k_pool, const b2pa_tensor* v_pool, const b2pa_tensor* k_scales,
                 const b2pa_tensor* v_scales, int32_t layout, Problem* pr, Plane* plane, int* planes)
{
    std::memset(pr, 0, sizeof *pr);
    int st = parse_pools(k_pool, v_pool, layout, pr);
    if (st)
        return st;
    if ((k_scales == nullptr) != (v_scales == nullptr))
        return fail(B2PA_ERR_INVALID_ARG, "k_scales and v_scales: both or none");
    if (k_scales && ((st = check_scales(k_scales, "k_scales", k_pool)) || (st = check_scales(v_scales, "v_scales", v_pool))))
        return st;
    const b2pa_tensor* t[kMaxPlanes] = {k_pool, v_pool, k_scales, v_scales};
    const int dim[3] = {0, layout == B2PA_HND ? 1 : 2, layout == B2PA_HND ? 2 : 1};  // page, kv head, slot
    const int ext[3] = {pr->N, pr->Hkv, pr->P};
    *planes = k_scales ? 4 : 2;
    for (int i = 0; i < *planes; ++i) {
        const int es = i >= 2 ? 4 : pr->fp8 ? 1 : 2;
        Plane& x = plane[i];
        x.base = static_cast<uint8_t*>(t[i]->data);
        x.row = i >= 2 ? 4 : pr->D * es;
        uintptr_t all = reinterpret_cast<uintptr_t>(x.base) | (uintptr_t)x.row;
        int by[3] = {0, 1, 2};  // dims by stride, the smallest first
        for (int k = 0; k < 3; ++k) {
            x.st[k] = t[i]->stride[dim[k]] * es;
            if (ext[k] > 1)
                all |= (uintptr_t)x.st[k];
        }
        std::sort(by, by + 3, [&](int a, int b) { return x.st[a] < x.st[b]; });
        long long end = x.row;  // bytes that the dims so far span
        for (int k : by) {
            if (ext[k] > 1 && x.st[k] < end)
                return fail(B2PA_ERR_INVALID_ARG, "pool and scale strides must be positive, and no rows may overlap");
            end += ext[k] > 1 ? x.st[k] * (ext[k] - 1) : 0;
        }
        x.vec = piece_of(all);
    }
    return B2PA_OK;
}

// int32 [n], contiguous (null where n is 0)
int check_ints(const b2pa_tensor* t, const char* what, int64_t n)
{
    if (!t || t->ndim != 1 || t->dtype != B2PA_INT32 || t->shape[0] != n || (n > 0 && !is_vec(t, B2PA_INT32, n)))
        return fail(B2PA_ERR_INVALID_ARG, "%s must be contiguous int32 [%lld]", what, (long long)n);
    return B2PA_OK;
}

int* ints(const b2pa_tensor* t) { return static_cast<int*>(t->data); }

// A tensor of 4-byte elements as rows of bytes.
struct RowBytes {
    long long at, bytes, step, n;
    explicit RowBytes(const b2pa_tensor* t)
        : at((long long)reinterpret_cast<uintptr_t>(t->data)),
          bytes(4 * t->shape[t->ndim - 1]),
          step(t->ndim == 2 ? 4 * t->stride[0] : 0),
          n(t->ndim == 2 ? t->shape[0] : 1)
    {
        if (step < 0) {  // from the other end
            at += (n - 1) * step;
            step = -step;
        }
        if (step <= bytes && n > 1) {  // in one piece
            bytes += (n - 1) * step;
            n = 1;
        }
    }
    // whether the bytes [from, from + count) reach into a row
    bool reached(long long from, long long count) const
    {
        if (n <= 0 || bytes <= 0 || count <= 0 || from + count <= at)
            return false;
        const long long last = n > 1 ? std::min(n - 1, (from + count - 1 - at) / step) : 0;  // that starts before their end
        return from < at + last * step + bytes;
    }
};

// Whether two tensors of 4-byte elements, unit stride in their rows, share any.  (What
// lies between the rows of one is no part of it.)
bool meet(const b2pa_tensor* a, const b2pa_tensor* b)
{
    RowBytes x(a), y(b);
    if (x.n > y.n)
        std::swap(x, y);
    // (of two with room between their rows, row by row of the one that has fewer)
    for (long long i = 0; i < x.n; ++i)
        if (y.reached(x.at + i * x.step, x.bytes))
            return true;
    return false;
}

// Whether `out` shares any element with one of the others (null: none).
bool meets_any(const b2pa_tensor* out, std::initializer_list<const b2pa_tensor*> others)
{
    for (const b2pa_tensor* t : others)
        if (t && meet(out, t))
            return true;
    return false;
}

int copy_impl(const b2pa_tensor* k_pool, const b2pa_tensor* v_pool, const b2pa_tensor* k_scales,
              const b2pa_tensor* v_scales, const b2pa_tensor* src, const b2pa_tensor* dst, int32_t layout,
              cudaStream_t stream)
{
    Problem pr;
    CopyPagesParams p;
    std::memset(&p, 0, sizeof p);
    int st = parse_planes(k_pool, v_pool, k_scales, v_scales, layout, &pr, p.plane, &p.planes);
    if (st)
        return st;
    if (!src || src->ndim != 1 || src->shape[0] < 0 || src->shape[0] > 0x7FFFFFFF)
        return fail(B2PA_ERR_INVALID_ARG, "src must be contiguous int32 [n]");
    const int64_t n = src->shape[0];
    if ((st = check_ints(src, "src", n)) || (st = check_ints(dst, "dst", n)))
        return st;
    if (n == 0)
        return B2PA_OK;
    for (int i = 0; i < p.planes; ++i) {
        Plane& x = p.plane[i];
        // dims within a page: the one of the smaller stride inside
        long long in = x.st[2], out = x.st[1];
        int in_n = pr.P, out_n = pr.Hkv;
        if (in_n == 1 || (out_n > 1 && out < in)) {
            std::swap(in, out);
            std::swap(in_n, out_n);
        }
        long long row = x.row;
        if (in_n == 1 || in == row) {  // one piece
            row *= in_n;
            in_n = 1;
            if (out_n == 1 || out == row) {
                row *= out_n;
                out_n = 1;
            }
        }
        p.row[i] = row;
        p.inner[i] = in_n;
        p.outer[i] = out_n;
        p.inner_st[i] = in;
        p.outer_st[i] = out;
        uintptr_t all = reinterpret_cast<uintptr_t>(x.base) | (uintptr_t)row;
        all |= (pr.N > 1 ? (uintptr_t)x.st[0] : 0) | (in_n > 1 ? (uintptr_t)in : 0) | (out_n > 1 ? (uintptr_t)out : 0);
        x.vec = piece_of(all);
        if (row / x.vec * in_n * out_n > 0x7FFFFFFFLL)
            return fail(B2PA_ERR_UNSUPPORTED, "pages of 2^31 pieces or more");
    }
    int dev;
    DevInfo di;
    if ((st = device_info(&dev, &di)) || (st = status_word(dev, stream, &p.err)))
        return st;
    p.n = (int)n;
    p.num_pages = pr.N;
    p.src = ints(src);
    p.dst = ints(dst);
    const cudaError_t e = launch_copy_pages(p, stream);
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, "page copy launch");
}

int compact_impl(const b2pa_tensor* k_pool, const b2pa_tensor* v_pool, const b2pa_tensor* k_scales,
                 const b2pa_tensor* v_scales, const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens,
                 const b2pa_tensor* cum_q, const b2pa_tensor* accepted, const b2pa_tensor* counts,
                 b2pa_tensor* new_lens, int32_t layout, cudaStream_t stream)
{
    Problem pr;
    CompactParams p;
    std::memset(&p, 0, sizeof p);
    int st = parse_planes(k_pool, v_pool, k_scales, v_scales, layout, &pr, p.plane, &p.planes);
    if (st)
        return st;
    if (!seq_lens || seq_lens->ndim != 1 || seq_lens->shape[0] < 0 || seq_lens->shape[0] > 0x7FFFFFF)
        return fail(B2PA_ERR_INVALID_ARG, "seq_lens must be contiguous int32 [B]");
    const int64_t B = seq_lens->shape[0];
    if ((st = check_ints(seq_lens, "seq_lens", B)) || (st = check_ints(cum_q, "cum_q", B + 1)) ||
        (st = check_ints(counts, "counts", B)) || (st = check_ints(new_lens, "new_lens", B)))
        return st;
    if (!block_tables || block_tables->ndim != 2 || block_tables->dtype != B2PA_INT32 || block_tables->shape[0] != B ||
        block_tables->shape[1] < 0 || block_tables->shape[1] > 0x7FFFFFFF ||
        (block_tables->shape[1] > 1 && block_tables->stride[1] != 1) ||
        (B > 0 && block_tables->shape[1] > 0 && !block_tables->data))
        return fail(B2PA_ERR_INVALID_ARG, "block_tables must be int32 [B, max_pages] with unit column stride");
    if (!accepted || accepted->ndim != 2 || accepted->dtype != B2PA_INT32 || accepted->shape[0] != B ||
        accepted->shape[1] < 0 || accepted->shape[1] > 0x7FFFFFFF ||
        (accepted->shape[1] > 1 && accepted->stride[1] != 1) || (B > 0 && accepted->shape[1] > 0 && !accepted->data))
        return fail(B2PA_ERR_INVALID_ARG, "accepted must be int32 [B, width] with unit column stride");
    if (B == 0)
        return B2PA_OK;
    if (meets_any(new_lens, {seq_lens, counts, cum_q, accepted, block_tables}))
        return fail(B2PA_ERR_INVALID_ARG, "new_lens must not be an input: several blocks read those");
    long long pieces = 0;
    for (int i = 0; i < p.planes; ++i)
        pieces += (long long)p.plane[i].row / p.plane[i].vec * pr.Hkv;
    if (pieces > 0x7FFFFFFF)
        return fail(B2PA_ERR_UNSUPPORTED, "rows of 2^31 pieces or more");
    int dev;
    DevInfo di;
    if ((st = device_info(&dev, &di)) || (st = status_word(dev, stream, &p.err)))
        return st;
    p.pieces = (int)pieces;
    p.Hkv = pr.Hkv;
    p.page_size = pr.P;
    p.num_pages = pr.N;
    p.max_pages = (int)block_tables->shape[1];
    p.block_tables = ints(block_tables);
    p.bt_stride = block_tables->stride[0];
    p.seq_lens = ints(seq_lens);
    p.cum_q = ints(cum_q);
    p.counts = ints(counts);
    p.accepted = ints(accepted);
    p.acc_stride = accepted->stride[0];
    p.width = (int)accepted->shape[1];
    p.new_lens = ints(new_lens);
    p.B = (int)B;
    const cudaError_t e = launch_compact(p, stream);
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, "compaction launch");
}

// fp32 rows [T, V], contiguous in V
int check_probs(const b2pa_tensor* t, const char* what, int64_t T, int64_t V)
{
    if (!t || t->ndim != 2 || t->dtype != B2PA_FP32 || t->shape[0] != T || t->shape[1] != V ||
        (V > 1 && t->stride[1] != 1) || (T > 1 && t->stride[0] < 0) || (T > 0 && !t->data))
        return fail(B2PA_ERR_INVALID_ARG, "%s must be fp32 [%lld, %lld], contiguous in its rows", what, (long long)T,
                    (long long)V);
    if (T > 0 && (reinterpret_cast<uintptr_t>(t->data) & 3u))
        return fail(B2PA_ERR_INVALID_ARG, "%s must be 4-byte aligned", what);
    return B2PA_OK;
}

int verify_impl(const b2pa_tensor* target, const b2pa_tensor* draft, const b2pa_tensor* tokens,
                const b2pa_tensor* parents, const b2pa_tensor* uniforms, const b2pa_tensor* last,
                const b2pa_tensor* cum_q, int32_t max_q_len, b2pa_tensor* accepted, b2pa_tensor* counts,
                b2pa_tensor* next, cudaStream_t stream)
{
    if (!target || target->ndim != 2 || target->shape[0] < 0 || target->shape[0] > 0x7FFFFFFF || target->shape[1] < 1 ||
        target->shape[1] >= 1 << 30)
        return fail(B2PA_ERR_INVALID_ARG, "target_probs must be fp32 [T, V], 1 <= V < 2^30");
    const int64_t T = target->shape[0], V = target->shape[1];
    int st;
    if ((st = check_probs(target, "target_probs", T, V)) || (draft && (st = check_probs(draft, "draft_probs", T, V))) ||
        (st = check_ints(tokens, "tokens", T)) || (st = check_ints(parents, "parents", T)))
        return st;
    if (!uniforms || uniforms->dtype != B2PA_FP32 || uniforms->ndim != 1 || uniforms->shape[0] != T ||
        (T > 0 && !is_vec(uniforms, B2PA_FP32, T)))
        return fail(B2PA_ERR_INVALID_ARG, "uniforms must be contiguous fp32 [T]");
    if (!counts || counts->ndim != 1 || counts->shape[0] < 0 || counts->shape[0] > 0x7FFFFFF)
        return fail(B2PA_ERR_INVALID_ARG, "counts must be contiguous int32 [B]");
    const int64_t B = counts->shape[0];
    if ((st = check_ints(counts, "counts", B)) || (st = check_ints(next, "next_tokens", B)) ||
        (st = check_ints(cum_q, "cum_q", B + 1)))
        return st;
    if (!last || last->dtype != B2PA_FP32 || last->ndim != 1 || last->shape[0] != B || (B > 0 && !is_vec(last, B2PA_FP32, B)))
        return fail(B2PA_ERR_INVALID_ARG, "last_uniforms must be contiguous fp32 [B]");
    if (max_q_len < 0)
        return fail(B2PA_ERR_INVALID_ARG, "max_q_len must be >= 0");
    if (max_q_len > kVerifyMaxNodes)
        return fail(B2PA_ERR_UNSUPPORTED, "max_q_len must be at most %d", kVerifyMaxNodes);
    if (!accepted || accepted->ndim != 2 || accepted->dtype != B2PA_INT32 || accepted->shape[0] != B ||
        accepted->shape[1] < max_q_len || accepted->shape[1] > 0x7FFFFFFF ||
        (accepted->shape[1] > 1 && accepted->stride[1] != 1) || (B > 1 && accepted->stride[0] < accepted->shape[1]) ||
        (B > 0 && accepted->shape[1] > 0 && !accepted->data))
        return fail(B2PA_ERR_INVALID_ARG,
                    "accepted must be int32 [B, width] with unit column stride, its rows apart and width >= max_q_len");
    if (B == 0)
        return B2PA_OK;
    // (a request's CTAs each read its nodes and have to find the same)
    const b2pa_tensor* outs[3] = {accepted, counts, next};
    for (int i = 0; i < 3; ++i) {
        if (meets_any(outs[i], {target, draft, tokens, parents, uniforms, last, cum_q}))
            return fail(B2PA_ERR_INVALID_ARG, "outputs must not overlap inputs");
        if (meet(outs[i], outs[(i + 1) % 3]))
            return fail(B2PA_ERR_INVALID_ARG, "accepted, counts and next_tokens must be three tensors");
    }
    int dev;
    DevInfo di;
    VerifyParams p;
    std::memset(&p, 0, sizeof p);
    if ((st = device_info(&dev, &di)) || (st = status_word(dev, stream, &p.err)))
        return st;
    p.target = static_cast<const float*>(target->data);
    p.target_st = target->stride[0];
    bool aligned = aligned16(p.target) && (T <= 1 || p.target_st % 4 == 0);
    if (draft) {
        p.draft = static_cast<const float*>(draft->data);
        p.draft_st = draft->stride[0];
        aligned = aligned && aligned16(p.draft) && (T <= 1 || p.draft_st % 4 == 0);
    }
    p.aligned = aligned;
    p.tokens = ints(tokens);
    p.parents = ints(parents);
    p.uniforms = static_cast<const float*>(uniforms->data);
    p.last = static_cast<const float*>(last->data);
    p.cum_q = ints(cum_q);
    p.accepted = ints(accepted);
    p.acc_st = accepted->stride[0];
    p.counts = ints(counts);
    p.next = ints(next);
    p.B = (int)B;
    p.T = (int)T;
    p.V = (int)V;
    p.max_q = max_q_len;
    p.width = (int)accepted->shape[1];
    const cudaError_t e = launch_verify(p, di.sms, stream);
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, "verification launch");
}

// What the ledger's calls share; `rows` are [n].
int parse_ledger(const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* page_refs,
                 const b2pa_tensor* rows, const char* what, int32_t page_size, LedgerParams* p)
{
    std::memset(p, 0, sizeof *p);
    if (!seq_lens || seq_lens->ndim != 1 || seq_lens->shape[0] < 0 || seq_lens->shape[0] > 0x7FFFFFFF)
        return fail(B2PA_ERR_INVALID_ARG, "seq_lens must be contiguous int32 [R]");
    if (!page_refs || page_refs->ndim != 1 || page_refs->shape[0] < 0 || page_refs->shape[0] >= 1 << 30)
        return fail(B2PA_ERR_INVALID_ARG, "page_refs must be contiguous int32 [num_pages], fewer than 2^30");
    if (!rows || rows->ndim != 1 || rows->shape[0] < 0)
        return fail(B2PA_ERR_INVALID_ARG, "%s must be contiguous int32 [n]", what);
    const int64_t R = seq_lens->shape[0], N = page_refs->shape[0], n = rows->shape[0];
    int st;
    if ((st = check_ints(seq_lens, "seq_lens", R)) || (st = check_ints(page_refs, "page_refs", N)) ||
        (st = check_ints(rows, what, n)))
        return st;
    if (!block_tables || block_tables->ndim != 2 || block_tables->dtype != B2PA_INT32 || block_tables->shape[0] != R ||
        block_tables->shape[1] < 0 || block_tables->shape[1] >= 1 << 30 ||
        (block_tables->shape[1] > 1 && block_tables->stride[1] != 1) ||
        (R > 1 && block_tables->stride[0] < block_tables->shape[1]) ||
        (R > 0 && block_tables->shape[1] > 0 && !block_tables->data))
        return fail(B2PA_ERR_INVALID_ARG,
                    "block_tables must be int32 [R, max_pages] with unit column stride, its rows apart");
    if (page_size < 1)
        return fail(B2PA_ERR_INVALID_ARG, "page_size must be >= 1");
    if (n > kLedgerMax)
        return fail(B2PA_ERR_UNSUPPORTED, "more than %d requests in one call", kLedgerMax);
    p->tables = ints(block_tables);
    p->stride = block_tables->stride[0];
    p->seq = ints(seq_lens);
    p->refs = ints(page_refs);
    p->rows = ints(rows);
    p->n = (int)n;
    p->R = (int)R;
    p->max_pages = (int)block_tables->shape[1];
    p->N = (int)N;
    p->page_size = page_size;
    return B2PA_OK;
}

// The ledger's three are written in place, and read and written by several CTAs:
// nothing else of a call may lie over them.
int check_apart(const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* page_refs,
                std::initializer_list<const b2pa_tensor*> others)
{
    bool over = meets_any(block_tables, {seq_lens, page_refs}) || meet(seq_lens, page_refs);
    for (const b2pa_tensor* t : others)
        over = over || meets_any(t, {block_tables, seq_lens, page_refs});
    return over ? fail(B2PA_ERR_INVALID_ARG,
                       "block_tables, seq_lens and page_refs must not overlap one another or other arguments")
                : B2PA_OK;
}

int run_ledger(LedgerParams& p, cudaStream_t stream, int which)
{
    int dev, st;
    DevInfo di;
    if ((st = device_info(&dev, &di)) || (st = status_word(dev, stream, &p.err)))
        return st;
    const cudaError_t e = which == 0 ? launch_free_pages(p, stream) : launch_take_pages(p, which == 1, stream);
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, "page ledger launch");
}

}  // namespace

// ====================================================================== C ABI

extern "C" {

int b2pa_copy_pages(const b2pa_tensor* k_pool, const b2pa_tensor* v_pool, const b2pa_tensor* k_scales,
                    const b2pa_tensor* v_scales, const b2pa_tensor* src, const b2pa_tensor* dst, int32_t layout,
                    b2pa_stream_t stream)
{
    return guarded([&] {
        return copy_impl(k_pool, v_pool, k_scales, v_scales, src, dst, layout, reinterpret_cast<cudaStream_t>(stream));
    });
}

int b2pa_compact_kv(const b2pa_tensor* k_pool, const b2pa_tensor* v_pool, const b2pa_tensor* k_scales,
                    const b2pa_tensor* v_scales, const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens,
                    const b2pa_tensor* cum_q, const b2pa_tensor* accepted, const b2pa_tensor* counts,
                    b2pa_tensor* new_lens, int32_t layout, b2pa_stream_t stream)
{
    return guarded([&] {
        return compact_impl(k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, cum_q, accepted, counts,
                            new_lens, layout, reinterpret_cast<cudaStream_t>(stream));
    });
}

int b2pa_verify_trees(const b2pa_tensor* target_probs, const b2pa_tensor* draft_probs, const b2pa_tensor* tokens,
                      const b2pa_tensor* parents, const b2pa_tensor* uniforms, const b2pa_tensor* last_uniforms,
                      const b2pa_tensor* cum_q, int32_t max_q_len, b2pa_tensor* accepted, b2pa_tensor* counts,
                      b2pa_tensor* next_tokens, b2pa_stream_t stream)
{
    return guarded([&] {
        return verify_impl(target_probs, draft_probs, tokens, parents, uniforms, last_uniforms, cum_q, max_q_len,
                           accepted, counts, next_tokens, reinterpret_cast<cudaStream_t>(stream));
    });
}

int b2pa_free_pages(const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* page_refs,
                    const b2pa_tensor* rows, int32_t page_size, b2pa_stream_t stream)
{
    return guarded([&] {
        LedgerParams p;
        int st = parse_ledger(block_tables, seq_lens, page_refs, rows, "rows", page_size, &p);
        if (st || p.n == 0 || (st = check_apart(block_tables, seq_lens, page_refs, {rows})))
            return st;
        return run_ledger(p, reinterpret_cast<cudaStream_t>(stream), 0);
    });
}

int b2pa_fork_pages(const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* page_refs,
                    const b2pa_tensor* parents, const b2pa_tensor* children, int32_t page_size, b2pa_tensor* src,
                    b2pa_tensor* dst, b2pa_stream_t stream)
{
    return guarded([&] {
        LedgerParams p;
        int st = parse_ledger(block_tables, seq_lens, page_refs, children, "children", page_size, &p);
        if (st || (st = check_ints(parents, "parents", p.n)) || (st = check_ints(src, "src", p.n)) ||
            (st = check_ints(dst, "dst", p.n)) || p.n == 0 ||
            (st = check_apart(block_tables, seq_lens, page_refs, {children, parents, src, dst})))
            return st;
        if (meet(src, dst))
            return fail(B2PA_ERR_INVALID_ARG, "src and dst must not overlap");
        p.parents = ints(parents);
        p.src = ints(src);
        p.dst = ints(dst);
        return run_ledger(p, reinterpret_cast<cudaStream_t>(stream), 1);
    });
}

int b2pa_grow_pages(const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* page_refs,
                    const b2pa_tensor* rows, const b2pa_tensor* new_lens, int32_t page_size, b2pa_stream_t stream)
{
    return guarded([&] {
        LedgerParams p;
        int st = parse_ledger(block_tables, seq_lens, page_refs, rows, "rows", page_size, &p);
        if (st || (st = check_ints(new_lens, "new_lens", p.n)) || p.n == 0 ||
            (st = check_apart(block_tables, seq_lens, page_refs, {rows, new_lens})))
            return st;
        p.to = ints(new_lens);
        return run_ledger(p, reinterpret_cast<cudaStream_t>(stream), 2);
    });
}

}  // extern "C"
