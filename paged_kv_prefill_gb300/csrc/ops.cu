// ops.cu -- host side of the entry points around the attention call: the
// query/key norm with the rotation, the write and read of a cache with one
// scale per row, and the attention of token trees and of requests that share
// prefixes.  Argument checks and launches; nothing here synchronises.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/b2pa.h"
#include "host.cuh"
#include "kv_scaled.cuh"
#include "rope.cuh"
#include "tree.cuh"

using namespace b2pa;

int b2pa::check_scales(const b2pa_tensor* s, const char* what, const b2pa_tensor* pool)
{
    if (!s || !s->data || s->dtype != B2PA_FP32 || s->ndim != 3)
        return fail(B2PA_ERR_INVALID_ARG, "%s must be fp32 with the pool's shape without head_dim", what);
    for (int i = 0; i < 3; ++i)
        if (s->shape[i] != pool->shape[i])
            return fail(B2PA_ERR_INVALID_ARG, "%s must be fp32 with the pool's shape without head_dim", what);
    if (reinterpret_cast<uintptr_t>(s->data) & 3u)
        return fail(B2PA_ERR_INVALID_ARG, "%s must be 4-byte aligned", what);
    return B2PA_OK;
}

namespace {

// t is [T, heads, D] bf16, contiguous in head_dim, in 16-byte steps.
int check_rows(const b2pa_tensor* t, const char* what, int64_t T, int64_t heads, int64_t D)
{
    if (!t || t->ndim != 3 || t->dtype != B2PA_BF16)
        return fail(B2PA_ERR_INVALID_ARG, "%s must be a bf16 tensor [T, heads, D]", what);
    if (t->shape[0] != T || t->shape[1] != heads || t->shape[2] != D)
        return fail(B2PA_ERR_INVALID_ARG, "%s must have shape [%lld, %lld, %lld]", what, (long long)T,
                    (long long)heads, (long long)D);
    if (T == 0)
        return B2PA_OK;  // empty tensors may carry null data pointers
    if (!t->data)
        return fail(B2PA_ERR_INVALID_ARG, "%s: null data", what);
    if (t->stride[2] != 1 || !aligned16(t->data) || (T > 1 && t->stride[0] % 8) || (heads > 1 && t->stride[1] % 8))
        return fail(B2PA_ERR_INVALID_ARG,
                    "%s: head_dim contiguous, token and head strides multiples of 8, 16-byte aligned", what);
    return B2PA_OK;
}

// The rows of an output must not overlap (a broadcast view).
int check_rows_apart(const b2pa_tensor* t, const char* what)
{
    const int64_t D = t->shape[2];
    int64_t n[2] = {t->shape[0], t->shape[1]}, st[2] = {t->stride[0], t->stride[1]};
    for (int i = 0; i < 2; ++i)
        if (n[i] <= 1)
            st[i] = INT64_MAX;
    const int lo = st[0] <= st[1] ? 0 : 1, hi = 1 - lo;
    if (st[lo] < D || (st[hi] != INT64_MAX && st[hi] < st[lo] * (n[lo] - 1) + D))
        return fail(B2PA_ERR_INVALID_ARG, "%s: its rows overlap", what);
    return B2PA_OK;
}

// Outputs of [T, heads, D] rows must be two, and one at an input's address that
// input itself (rows are read ahead of others' writes).
int check_places(const b2pa_tensor* const out[2], const char* const names[2], const b2pa_tensor* const in[2])
{
    if (out[0]->data == out[1]->data)
        return fail(B2PA_ERR_INVALID_ARG, "%s in the place of %s", names[1], names[0]);
    for (int i = 0; in && i < 2; ++i)
        for (int j = 0; j < 2; ++j) {
            if (out[i]->data != in[j]->data)
                continue;
            bool same = i == j;
            for (int d = 0; d < 2; ++d)
                same = same && (out[i]->shape[d] <= 1 || out[i]->stride[d] == in[j]->stride[d]);
            if (!same)
                return fail(B2PA_ERR_INVALID_ARG, "%s in the place of other rows of an input", names[i]);
        }
    return B2PA_OK;
}

int check_weight(const b2pa_tensor* w, const char* what, int64_t D)
{
    if (!w)
        return B2PA_OK;
    if (!(is_vec(w, B2PA_BF16, D) || is_vec(w, B2PA_FP32, D)) || !aligned16(w->data))
        return fail(B2PA_ERR_INVALID_ARG, "%s must be contiguous bf16 or fp32 [D], 16-byte aligned (or NULL)", what);
    return B2PA_OK;
}

int rope_impl(const b2pa_tensor* q, const b2pa_tensor* k, const b2pa_tensor* cos_sin, const b2pa_tensor* positions,
              const b2pa_tensor* q_weight, const b2pa_tensor* k_weight, float eps, const int32_t* axis_of,
              int32_t interleaved, b2pa_tensor* q_out, b2pa_tensor* k_out, cudaStream_t stream)
{
    if (!q || !k || q->ndim != 3 || k->ndim != 3)
        return fail(B2PA_ERR_INVALID_ARG, "q and k must be bf16 tensors [T, heads, D]");
    const int64_t T = q->shape[0], D = q->shape[2];
    if (T < 0 || T > 0x7FFFFFFF || q->shape[1] < 1 || q->shape[1] > 0x7FFFFF || k->shape[1] < 1 ||
        k->shape[1] > 0x7FFFFF || D < 1)
        return fail(B2PA_ERR_INVALID_ARG, "q / k extents");
    if (D % 8 || D > kRopeMaxD)
        return fail(B2PA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most %d", kRopeMaxD);
    int st;
    if ((st = check_rows(q, "q", T, q->shape[1], D)) || (st = check_rows(k, "k", T, k->shape[1], D)) ||
        (st = check_rows(q_out, "q_out", T, q->shape[1], D)) || (st = check_rows(k_out, "k_out", T, k->shape[1], D)) ||
        (st = check_weight(q_weight, "q_weight", D)) || (st = check_weight(k_weight, "k_weight", D)))
        return st;
    if (T > 0 && ((st = check_rows_apart(q_out, "q_out")) || (st = check_rows_apart(k_out, "k_out"))))
        return st;
    if (!std::isfinite(eps) || eps < 0.f)
        return fail(B2PA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!cos_sin || !cos_sin->data || cos_sin->ndim != 2 || cos_sin->dtype != B2PA_FP32 || cos_sin->shape[0] < 1 ||
        cos_sin->shape[0] > 0x7FFFFFFF || cos_sin->stride[1] != 1 || (cos_sin->shape[0] > 1 && cos_sin->stride[0] < 1))
        return fail(B2PA_ERR_INVALID_ARG, "cos_sin must be fp32 [max_position, R], contiguous in R");
    const int64_t R = cos_sin->shape[1];
    if (R < 2 || R % 2 || R > D)
        return fail(B2PA_ERR_INVALID_ARG, "cos_sin must have an even number R <= D of columns, not %lld", (long long)R);
    int64_t axes = 1;
    if (!positions || positions->dtype != B2PA_INT32 || (positions->ndim != 1 && positions->ndim != 2))
        return fail(B2PA_ERR_INVALID_ARG, "positions must be int32 [T] or [axes, T]");
    if (positions->ndim == 2)
        axes = positions->shape[0];
    const int64_t pt = positions->shape[positions->ndim - 1], pst = positions->stride[positions->ndim - 1];
    if (axes < 1 || axes > kRopeMaxAxes || pt != T || (T > 1 && pst != 1) || (T > 0 && !positions->data))
        return fail(B2PA_ERR_INVALID_ARG, "positions must be int32 [T] or [axes, T] with 1 to %d axes, contiguous in T",
                    kRopeMaxAxes);
    if (axes > 1 && !axis_of)
        return fail(B2PA_ERR_INVALID_ARG, "axis_of must say which axis each frequency belongs to");
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    const int half = (int)(R / 2);
    for (int i = 0; axis_of && i < half; ++i) {
        if (axis_of[i] < 0 || axis_of[i] >= axes)
            return fail(B2PA_ERR_INVALID_ARG, "axis_of[%d] = %d is outside [0, %lld)", i, axis_of[i], (long long)axes);
        p.axis_of[i] = (uint8_t)axis_of[i];
    }
    if (T == 0)
        return B2PA_OK;
    const b2pa_tensor *in[2] = {q, k}, *out[2] = {q_out, k_out}, *w[2] = {q_weight, k_weight};
    const char* const names[2] = {"q_out", "k_out"};
    if ((st = check_places(out, names, in)))
        return st;
    for (int g = 0; g < (half + 3) / 4; ++g) {
        p.axis_of4[g] = 4 * g + 4 <= half ? p.axis_of[4 * g] : 255;
        for (int i = 4 * g; i < 4 * g + 4 && i < half; ++i)
            if (p.axis_of[i] != p.axis_of[4 * g])
                p.axis_of4[g] = 255;
    }
    int dev;
    DevInfo di;
    if ((st = device_info(&dev, &di)) || (st = status_word(dev, stream, &p.err)))
        return st;
    for (int i = 0; i < 2; ++i) {
        RopeTensor& x = p.x[i];
        x.in = static_cast<const uint16_t*>(in[i]->data);
        x.out = static_cast<uint16_t*>(out[i]->data);
        x.in_tok = in[i]->stride[0];
        x.in_head = in[i]->stride[1];
        x.out_tok = out[i]->stride[0];
        x.out_head = out[i]->stride[1];
        x.weight = w[i] ? w[i]->data : nullptr;
        x.weight_f32 = w[i] && w[i]->dtype == B2PA_FP32;
        x.heads = (int)in[i]->shape[1];
    }
    p.cos_sin = static_cast<const float*>(cos_sin->data);
    p.cs_stride = cos_sin->stride[0];
    p.positions = static_cast<const int*>(positions->data);
    p.pos_stride = positions->ndim == 2 ? positions->stride[0] : 0;
    p.T = (int)T;
    p.D = (int)D;
    p.R = (int)R;
    p.axes = (int)axes;
    p.max_pos = (int)cos_sin->shape[0];
    p.vec_table = half % 4 == 0 && p.cs_stride % 4 == 0 && aligned16(p.cos_sin);
    p.eps = eps;
    p.inv_d = 1.f / (float)D;
    const cudaError_t e = launch_qk_norm_rope(p, interleaved != 0, di.sms, stream);
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, "norm and rotation launch");
}

// What the write and the read share; rows: k_new/v_new or k_out/v_out.
int scaled_kv_impl(bool write, const b2pa_tensor* const rows[2], const char* const names[2], const b2pa_tensor* k_pool,
                   const b2pa_tensor* v_pool, const b2pa_tensor* k_scales, const b2pa_tensor* v_scales,
                   const b2pa_tensor* cache_loc, int32_t layout, cudaStream_t stream)
{
    Problem pr;
    std::memset(&pr, 0, sizeof pr);
    int st = parse_pools(k_pool, v_pool, layout, &pr);
    if (st)
        return st;
    if (!pr.fp8)
        return fail(B2PA_ERR_INVALID_ARG, "the pools must be fp8_e4m3");
    if ((st = check_scales(k_scales, "k_scales", k_pool)) || (st = check_scales(v_scales, "v_scales", v_pool)))
        return st;
    if (!cache_loc || cache_loc->ndim != 1 || cache_loc->dtype != B2PA_INT32)
        return fail(B2PA_ERR_INVALID_ARG, "cache_loc must be int32 [T]");
    const int64_t T = cache_loc->shape[0];
    if (T < 0 || T > 0x7FFFFFFF)
        return fail(B2PA_ERR_INVALID_ARG, "cache_loc extents");
    if (pr.D % 8 || pr.D > 256)
        return fail(B2PA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most 256");
    for (int i = 0; i < 2; ++i)
        if ((st = check_rows(rows[i], names[i], T, pr.Hkv, pr.D)) || (!write && T > 0 && (st = check_rows_apart(rows[i], names[i]))))
            return st;
    if ((long long)pr.N * pr.P > 0x7FFFFFFFLL)
        return fail(B2PA_ERR_UNSUPPORTED, "num_pages * page_size must be < 2^31 (int32 slots)");
    const b2pa_tensor* sc[2] = {k_scales, v_scales};
    const int dim[3] = {0, layout == B2PA_HND ? 1 : 2, layout == B2PA_HND ? 2 : 1};  // page, kv head, slot
    const int ext[3] = {pr.N, pr.Hkv, pr.P};
    for (int i = 0; i < 3; ++i) {
        if (ext[i] > 1 && (pr.k_st[i] % 8 || pr.v_st[i] % 8))
            return fail(B2PA_ERR_INVALID_ARG, "pool page / head / slot strides must be multiples of 8 elements");
        if (write && ext[i] > 1 &&
            (pr.k_st[i] < 1 || pr.v_st[i] < 1 || sc[0]->stride[dim[i]] < 1 || sc[1]->stride[dim[i]] < 1))
            return fail(B2PA_ERR_INVALID_ARG, "pool and scale strides must be positive");
    }
    if ((reinterpret_cast<uintptr_t>(pr.k) | reinterpret_cast<uintptr_t>(pr.v)) & 7u)
        return fail(B2PA_ERR_INVALID_ARG, "pools must be 8-byte aligned");
    if (T == 0)
        return B2PA_OK;
    if (!is_vec(cache_loc, B2PA_INT32, T))
        return fail(B2PA_ERR_INVALID_ARG, "cache_loc must be contiguous int32 [T]");
    if (!write && (st = check_places(rows, names, nullptr)))
        return st;
    int dev;
    DevInfo di;
    ScaledKvParams p;
    std::memset(&p, 0, sizeof p);
    if ((st = device_info(&dev, &di)) || (st = status_word(dev, stream, &p.err)))
        return st;
    const void* pool[2] = {pr.k, pr.v};
    const long long* pool_st[2] = {pr.k_st, pr.v_st};
    for (int i = 0; i < 2; ++i) {
        if (write)
            p.x[i] = static_cast<const uint16_t*>(rows[i]->data);
        else
            p.y[i] = static_cast<uint16_t*>(rows[i]->data);
        p.tok[i] = rows[i]->stride[0];
        p.head[i] = rows[i]->stride[1];
        p.pool[i] = static_cast<uint8_t*>(const_cast<void*>(pool[i]));
        p.scale[i] = static_cast<float*>(sc[i]->data);
        for (int j = 0; j < 3; ++j) {
            p.pool_st[i][j] = pool_st[i][j];
            p.scale_st[i][j] = sc[i]->stride[dim[j]];
        }
    }
    p.cache_loc = static_cast<const int*>(cache_loc->data);
    p.T = (int)T;
    p.Hkv = pr.Hkv;
    p.D = pr.D;
    p.page_size = pr.P;
    p.num_pages = pr.N;
    const cudaError_t e = write ? launch_append_scaled(p, stream) : launch_read_scaled(p, stream);
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, write ? "scaled append launch" : "scaled read launch");
}

// How a tree attention call runs: on the tensor cores or not, and what its
// workspace holds.
struct TreePlan {
    bool tc;
    int tiles;     // query tiles per item
    bool whole;    // no unit is cut
    size_t off_ml, off_o, bytes;
};

int plan_tree(const Problem& pr, int max_q_len, int max_kv_len, int window, const DevInfo& di, TreePlan* out)
{
    const char* why = tc_reject(pr, di);
    const int path = kernel_path();
    if (path == B2PA_PATH_TCGEN05 && why)
        return fail(B2PA_ERR_UNSUPPORTED, "tensor-core path: %s", why);
    TreePlan t{};
    t.tc = path != B2PA_PATH_GENERIC && !why;
    if (t.tc) {
        const int G = pr.H / pr.Hkv;
        // one query tile where one is enough: both softmax groups work on it (8 nodes x
        // 4 heads over 2048 keys 14.3 us, 15.1 with the second group idle; 32 requests
        // of up to 16 nodes 104 and 109, of up to 8 over an e4m3 cache 161 and 244)
        t.tiles = max_q_len <= tree_rows(G).tile_toks ? 1 : 2;
        // kv tiles of a unit at most: its keys start at 0, or anywhere with a window
        const long long all = ((long long)max_kv_len + kKvTile - 1) / kKvTile;
        const long long seen = ((long long)window + max_q_len + kKvTile - 2) / kKvTile + 1;
        const long long kv_tiles = window >= 0 ? std::min(all, seen) : all;
        // Units stay whole, and nothing is merged, where they are small, or about as
        // many as SMs: 8 nodes x 4 heads, 8 kv heads, cut and whole, 8 requests of 768
        // keys 16.9 and 14.7 us, 24 of 1024 30.8 and 28.4; but 40 of 768 39.0 and 39.7, one of
        // 1024 13.3 and 15.7.
        const int item = t.tiles * tree_rows(G).tile_toks;
        const long long units = (long long)pr.B * pr.Hkv * ((max_q_len + item - 1) / item);
        t.whole = kv_tiles <= kTreeWholeTiles || (kv_tiles <= 8 && 3 * units >= di.sms && 2 * units <= 3 * di.sms);
        const size_t rows = (size_t)di.sms * 2 * t.tiles * kQRows;  // two segments of every CTA
        t.off_ml = ((size_t)di.sms * 2 * 2 * sizeof(int4) + 255) / 256 * 256;
        t.off_o = t.off_ml + rows * sizeof(float2);
        t.bytes = t.whole ? 0 : t.off_o + rows * pr.D * sizeof(float);
    }
    *out = t;
    return B2PA_OK;
}

// What the calls of a few rows per request hand to their kernels alike.
int fill_tree(const Problem& pr, int max_q_len, int max_kv_len, float bmm1_scale, float bmm2_scale, const DevInfo& di,
              int dev, cudaStream_t stream, TreeParams* out)
{
    TreeParams& p = *out;
    std::memset(&p, 0, sizeof p);
    if (const int st = status_word(dev, stream, &p.err))
        return st;
    p.rows = tree_rows(pr.H / pr.Hkv);
    p.q = static_cast<const uint16_t*>(pr.q);
    p.k = pr.k;
    p.v = pr.v;
    p.out = static_cast<uint16_t*>(pr.out);
    p.q_st_tok = pr.q_st_tok;
    p.q_st_head = pr.q_st_head;
    p.out_st_tok = pr.out_st_tok;
    p.out_st_head = pr.out_st_head;
    for (int i = 0; i < 3; ++i) {
        p.k_st[i] = pr.k_st[i];
        p.v_st[i] = pr.v_st[i];
    }
    p.cum_q = pr.cum_q;
    p.seq_lens = pr.seq;
    p.block_tables = pr.bt;
    p.bt_stride = pr.bt_stride;
    p.sinks = pr.sinks;
    p.B = pr.B;
    p.T = pr.T;
    p.H = pr.H;
    p.Hkv = pr.Hkv;
    p.D = pr.D;
    p.page_size = pr.P;
    p.max_pages = pr.max_pages;
    p.num_pages = pr.N;
    p.max_q_len = max_q_len;
    p.max_kv_len = max_kv_len;
    p.window = -1;
    p.grid = di.sms;
    p.scale_log2 = (float)((double)bmm1_scale * 1.4426950408889634);
    p.bmm2 = bmm2_scale;
    p.wait_limit_ns = wait_limit_ns();
    p.inject_stall = inject_stall();
    return B2PA_OK;
}

// The tensor maps of the tensor-core path.
int encode_tree_maps(const Problem& pr, TreeParams* p)
{
    int st;
    if ((st = encode_q_map(&p->tm_q, pr, p->rows.box_toks)) || (st = encode_pool_map(&p->tm_k, pr, pr.k, pr.k_st)) ||
        (st = encode_pool_map(&p->tm_v, pr, pr.v, pr.v_st)))
        return st;
    return B2PA_OK;
}

int tree_impl(const b2pa_tensor* q, const b2pa_tensor* k_pool, const b2pa_tensor* v_pool,
              const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* cum_q,
              const b2pa_tensor* tree_mask, const b2pa_tensor* positions, int32_t max_q_len, int32_t max_kv_len,
              float bmm1_scale, float bmm2_scale, int32_t window_left, const b2pa_tensor* sinks, int32_t layout,
              b2pa_tensor* out, void* workspace, uint64_t workspace_bytes, uint64_t* bytes_needed, cudaStream_t stream)
{
    if (!bytes_needed)
        return fail(B2PA_ERR_INVALID_ARG, "bytes_needed: null");
    // empty tensors may carry null data pointers
    b2pa_tensor no_q, no_out;
    if (q && out && k_pool && q->ndim == 3 && q->shape[0] == 0) {
        no_q = *q;
        no_out = *out;
        no_q.data = no_out.data = k_pool->data;
        q = &no_q;
        out = &no_out;
    }
    Problem pr;
    int st = parse_problem(q, k_pool, v_pool, block_tables, seq_lens, cum_q, nullptr, sinks, layout, out, &pr);
    if (st)
        return st;
    if (max_q_len < 0 || max_kv_len < 0)
        return fail(B2PA_ERR_INVALID_ARG, "max_q_len / max_kv_len must be >= 0");
    if (max_kv_len > 0x7FFFFFFF - 2 * kKvTile)  // (a tile behind the last key is an int still)
        return fail(B2PA_ERR_UNSUPPORTED, "max_kv_len must be at most 2^31 - 257");
    if (!std::isfinite(bmm1_scale) || !(bmm1_scale > 0.f) || !std::isfinite(bmm2_scale))
        return fail(B2PA_ERR_INVALID_ARG, "bmm1_scale must be finite and > 0, bmm2_scale finite");
    const int64_t words = ((int64_t)max_q_len + 31) / 32;
    if (!tree_mask || tree_mask->ndim != 2 || tree_mask->dtype != B2PA_INT32 || tree_mask->shape[0] != pr.T ||
        tree_mask->shape[1] < words || tree_mask->shape[1] > 0x7FFFFFF ||
        (tree_mask->shape[1] > 1 && tree_mask->stride[1] != 1) || (pr.T > 0 && words > 0 && !tree_mask->data))
        return fail(B2PA_ERR_INVALID_ARG,
                    "tree_mask must be int32 [T, words] with unit column stride and words >= ceil(max_q_len / 32)");
    const int window = window_left < 0 ? -1 : window_left;
    if (window >= 0 && pr.T > 0 && !is_vec(positions, B2PA_INT32, pr.T))
        return fail(B2PA_ERR_INVALID_ARG, "a window needs positions, contiguous int32 [T]");
    if (pr.T > 0 && (st = check_rows_apart(out, "out")))
        return st;
    if (pr.T > 0 && pr.out == pr.q)
        return fail(B2PA_ERR_INVALID_ARG, "out must not be q: rows are read by several blocks");
    *bytes_needed = 0;
    if (pr.B == 0 || pr.T == 0)
        return B2PA_OK;
    int dev;
    DevInfo di;
    TreePlan plan;
    if ((st = device_info(&dev, &di)) || (st = plan_tree(pr, max_q_len, max_kv_len, window, di, &plan)))
        return st;
    *bytes_needed = plan.bytes;
    if (workspace_bytes < plan.bytes)
        return fail(B2PA_ERR_WORKSPACE, "workspace: %llu bytes are needed", (unsigned long long)plan.bytes);
    if (plan.bytes && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(B2PA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    TreeParams p;
    if ((st = fill_tree(pr, max_q_len, max_kv_len, bmm1_scale, bmm2_scale, di, dev, stream, &p)))
        return st;
    p.mask = static_cast<const unsigned*>(tree_mask->data);
    p.mask_stride = tree_mask->stride[0];
    p.mask_words = (int)tree_mask->shape[1];
    p.positions = window >= 0 ? static_cast<const int*>(positions->data) : nullptr;
    p.window = window;
    cudaError_t e;
    if (plan.tc) {
        p.whole = plan.whole;
        if (!plan.whole) {
            uint8_t* ws = static_cast<uint8_t*>(workspace);
            p.part_seg = reinterpret_cast<int4*>(ws);
            p.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
            p.part_o = reinterpret_cast<float4*>(ws + plan.off_o);
        }
        if ((st = encode_tree_maps(pr, &p)))
            return st;
        e = launch_attention_tree(p, pr.fp8, plan.tiles, stream);
    } else {
        e = launch_tree_generic(p, pr.fp8, stream);
    }
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, "tree attention launch");
}

// Scratch of a prefix attention call on the tensor cores.
struct PrefixPlan {
    bool tc;
    int tiles;  // query tiles per item of a prefix
    bool few;   // the requests' own keys as single tokens with few heads
    size_t off_o[2], off_rec[2], off_cut_o, off_cut_rec, off_ends, bytes;
};

int plan_prefix(const Problem& pr, int max_q_len, int max_group_q_len, const DevInfo& di, PrefixPlan* out)
{
    const char* why = tc_reject(pr, di);
    const int path = kernel_path();
    if (path == B2PA_PATH_TCGEN05 && why)
        return fail(B2PA_ERR_UNSUPPORTED, "tensor-core path: %s", why);
    PrefixPlan t{};
    t.tc = path != B2PA_PATH_GENERIC && !why;
    if (t.tc) {
        t.few = max_q_len <= 1 && pr.H / pr.Hkv <= 16;  // (two sets of eight rows; see launch_prefix)
        t.tiles = std::max(max_q_len, max_group_q_len) <= tree_rows(pr.H / pr.Hkv).tile_toks ? 1 : 2;
        size_t at = 0;
        auto take = [&](size_t bytes) {
            const size_t here = at;
            at += (bytes + 255) / 256 * 256;
            return here;
        };
        const size_t rows = (size_t)pr.T * pr.H, cut = (size_t)di.sms * 2 * kQRows;
        for (int i = 0; i < 2; ++i) {
            t.off_o[i] = take(rows * pr.D * sizeof(float));
            t.off_rec[i] = take(rows * sizeof(float4));
        }
        t.off_cut_o = take(cut * pr.D * sizeof(float));
        t.off_cut_rec = take(cut * sizeof(float4));
        t.off_ends = take((size_t)di.sms * sizeof(int));
        t.bytes = at;
    }
    *out = t;
    return B2PA_OK;
}

int prefix_impl(const b2pa_tensor* q, const b2pa_tensor* k_pool, const b2pa_tensor* v_pool,
                const b2pa_tensor* prefix_tables, const b2pa_tensor* prefix_lens, const b2pa_tensor* cum_groups,
                const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* cum_q,
                int32_t max_q_len, int32_t max_group_q_len, int32_t max_prefix_len, int32_t max_kv_len,
                float bmm1_scale, float bmm2_scale, const b2pa_tensor* sinks, int32_t layout, b2pa_tensor* out,
                void* workspace, uint64_t workspace_bytes, uint64_t* bytes_needed, cudaStream_t stream)
{
    if (!bytes_needed)
        return fail(B2PA_ERR_INVALID_ARG, "bytes_needed: null");
    // empty tensors may carry null data pointers
    b2pa_tensor no_q, no_out;
    if (q && out && k_pool && q->ndim == 3 && q->shape[0] == 0) {
        no_q = *q;
        no_out = *out;
        no_q.data = no_out.data = k_pool->data;
        q = &no_q;
        out = &no_out;
    }
    Problem pr;
    int st = parse_problem(q, k_pool, v_pool, block_tables, seq_lens, cum_q, nullptr, sinks, layout, out, &pr);
    if (st)
        return st;
    if (max_q_len < 0 || max_group_q_len < 0 || max_prefix_len < 0 || max_kv_len < 0)
        return fail(B2PA_ERR_INVALID_ARG, "max_q_len / max_group_q_len / max_prefix_len / max_kv_len must be >= 0");
    if (max_kv_len > 0x7FFFFFFF - 2 * kKvTile || max_prefix_len > 0x7FFFFFFF - 2 * kKvTile)
        return fail(B2PA_ERR_UNSUPPORTED, "max_prefix_len and max_kv_len must be at most 2^31 - 257");
    if (!std::isfinite(bmm1_scale) || !(bmm1_scale > 0.f) || !std::isfinite(bmm2_scale))
        return fail(B2PA_ERR_INVALID_ARG, "bmm1_scale must be finite and > 0, bmm2_scale finite");
    if (!prefix_lens || prefix_lens->ndim != 1 || prefix_lens->shape[0] < 0 || prefix_lens->shape[0] > 0x7FFFFFF ||
        (prefix_lens->shape[0] > 0 && !is_vec(prefix_lens, B2PA_INT32, prefix_lens->shape[0])))
        return fail(B2PA_ERR_INVALID_ARG, "prefix_lens must be contiguous int32 [groups]");
    const int64_t groups = prefix_lens->shape[0];
    if (!is_vec(cum_groups, B2PA_INT32, groups + 1))
        return fail(B2PA_ERR_INVALID_ARG, "cum_groups must be contiguous int32 [groups + 1]");
    if (!prefix_tables || prefix_tables->ndim != 2 || prefix_tables->dtype != B2PA_INT32 ||
        prefix_tables->shape[0] != groups || prefix_tables->shape[1] < 0 || prefix_tables->shape[1] > 0x7FFFFFFF ||
        (prefix_tables->shape[1] > 1 && prefix_tables->stride[1] != 1) ||
        (groups > 0 && prefix_tables->shape[1] > 0 && !prefix_tables->data))
        return fail(B2PA_ERR_INVALID_ARG, "prefix_tables must be int32 [groups, max_pages] with unit column stride");
    if (pr.T > 0 && (st = check_rows_apart(out, "out")))
        return st;
    if (pr.T > 0 && pr.out == pr.q)
        return fail(B2PA_ERR_INVALID_ARG, "out must not be q: rows are read by several blocks");
    *bytes_needed = 0;
    if (pr.B == 0 || pr.T == 0)
        return B2PA_OK;
    int dev;
    DevInfo di;
    PrefixPlan plan;
    if ((st = device_info(&dev, &di)) ||
        (st = plan_prefix(pr, max_q_len, std::min(max_group_q_len, pr.T), di, &plan)))
        return st;
    *bytes_needed = plan.bytes;
    if (workspace_bytes < plan.bytes)
        return fail(B2PA_ERR_WORKSPACE, "workspace: %llu bytes are needed", (unsigned long long)plan.bytes);
    if (plan.bytes && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(B2PA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    TreeParams p;
    if ((st = fill_tree(pr, max_q_len, max_kv_len, bmm1_scale, bmm2_scale, di, dev, stream, &p)))
        return st;
    PrefixParams& x = p.prefix;
    x.tables = static_cast<const int*>(prefix_tables->data);
    x.stride = prefix_tables->stride[0];
    x.lens = static_cast<const int*>(prefix_lens->data);
    x.cum_groups = static_cast<const int*>(cum_groups->data);
    x.groups = (int)groups;
    x.max_pages = (int)prefix_tables->shape[1];
    x.max_len = max_prefix_len;
    // (steps of a unit, units of a kv head: both at most, whatever cum_groups and cum_q hold)
    const long long steps = std::max(max_prefix_len, max_kv_len) / kKvTile + 1 + kTreeUnitCost;
    const long long units = groups * (pr.T / p.rows.tile_toks + 1LL) + pr.B;
    x.split = (double)steps * (double)units * (double)pr.Hkv < 2e9;
    cudaError_t e;
    if (plan.tc) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        for (int i = 0; i < 2; ++i) {
            x.part_o[i] = reinterpret_cast<float4*>(ws + plan.off_o[i]);
            x.part_rec[i] = reinterpret_cast<float4*>(ws + plan.off_rec[i]);
        }
        x.cut_o = reinterpret_cast<float4*>(ws + plan.off_cut_o);
        x.cut_rec = reinterpret_cast<float4*>(ws + plan.off_cut_rec);
        x.cut_ends = reinterpret_cast<int*>(ws + plan.off_ends);
        if ((st = encode_tree_maps(pr, &p)))
            return st;
        e = launch_attention_prefix(p, pr.fp8, plan.tiles, plan.few, stream);
    } else {
        e = launch_prefix_generic(p, pr.fp8, stream);
    }
    return e == cudaSuccess ? B2PA_OK : cuda_fail(e, "prefix attention launch");
}

}  // namespace

// ====================================================================== C ABI

extern "C" {

int b2pa_qk_norm_rope(const b2pa_tensor* q, const b2pa_tensor* k, const b2pa_tensor* cos_sin,
                      const b2pa_tensor* positions, const b2pa_tensor* q_weight, const b2pa_tensor* k_weight, float eps,
                      const int32_t* axis_of, int32_t interleaved, b2pa_tensor* q_out, b2pa_tensor* k_out,
                      b2pa_stream_t stream)
{
    return guarded([&] {
        return rope_impl(q, k, cos_sin, positions, q_weight, k_weight, eps, axis_of, interleaved, q_out, k_out,
                         reinterpret_cast<cudaStream_t>(stream));
    });
}

int b2pa_append_kv_scaled(const b2pa_tensor* k_new, const b2pa_tensor* v_new, const b2pa_tensor* k_pool,
                          const b2pa_tensor* v_pool, const b2pa_tensor* k_scales, const b2pa_tensor* v_scales,
                          const b2pa_tensor* cache_loc, int32_t layout, b2pa_stream_t stream)
{
    return guarded([&] {
        const b2pa_tensor* rows[2] = {k_new, v_new};
        const char* names[2] = {"k_new", "v_new"};
        return scaled_kv_impl(true, rows, names, k_pool, v_pool, k_scales, v_scales, cache_loc, layout,
                              reinterpret_cast<cudaStream_t>(stream));
    });
}

int b2pa_read_kv_scaled(const b2pa_tensor* k_pool, const b2pa_tensor* v_pool, const b2pa_tensor* k_scales,
                        const b2pa_tensor* v_scales, const b2pa_tensor* cache_loc, int32_t layout, b2pa_tensor* k_out,
                        b2pa_tensor* v_out, b2pa_stream_t stream)
{
    return guarded([&] {
        const b2pa_tensor* rows[2] = {k_out, v_out};
        const char* names[2] = {"k_out", "v_out"};
        return scaled_kv_impl(false, rows, names, k_pool, v_pool, k_scales, v_scales, cache_loc, layout,
                              reinterpret_cast<cudaStream_t>(stream));
    });
}

int b2pa_tree_attention(const b2pa_tensor* q, const b2pa_tensor* k_pool, const b2pa_tensor* v_pool,
                        const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* cum_q,
                        const b2pa_tensor* tree_mask, const b2pa_tensor* positions, int32_t max_q_len,
                        int32_t max_kv_len, float bmm1_scale, float bmm2_scale, int32_t window_left,
                        const b2pa_tensor* sinks, int32_t layout, b2pa_tensor* out, void* workspace,
                        uint64_t workspace_bytes, uint64_t* bytes_needed, b2pa_stream_t stream)
{
    return guarded([&] {
        return tree_impl(q, k_pool, v_pool, block_tables, seq_lens, cum_q, tree_mask, positions, max_q_len, max_kv_len,
                         bmm1_scale, bmm2_scale, window_left, sinks, layout, out, workspace, workspace_bytes,
                         bytes_needed, reinterpret_cast<cudaStream_t>(stream));
    });
}

int b2pa_prefix_attention(const b2pa_tensor* q, const b2pa_tensor* k_pool, const b2pa_tensor* v_pool,
                          const b2pa_tensor* prefix_tables, const b2pa_tensor* prefix_lens,
                          const b2pa_tensor* cum_groups, const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens,
                          const b2pa_tensor* cum_q, int32_t max_q_len, int32_t max_group_q_len, int32_t max_prefix_len,
                          int32_t max_kv_len, float bmm1_scale, float bmm2_scale, const b2pa_tensor* sinks,
                          int32_t layout, b2pa_tensor* out, void* workspace, uint64_t workspace_bytes,
                          uint64_t* bytes_needed, b2pa_stream_t stream)
{
    return guarded([&] {
        return prefix_impl(q, k_pool, v_pool, prefix_tables, prefix_lens, cum_groups, block_tables, seq_lens, cum_q,
                           max_q_len, max_group_q_len, max_prefix_len, max_kv_len, bmm1_scale, bmm2_scale, sinks, layout,
                           out, workspace, workspace_bytes, bytes_needed, reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
