// attn_tree.cu -- attention of drafted token trees over a paged cache on the
// 5th-generation tensor cores (tcgen05), and the merge of its partial rows.
//
// For node i of a request (its q row, head h, keys as tree.cuh says):
//   out = bmm2 * sum_j e^{s_ij - m} V_j / (sum_j e^{s_ij - m} + [sinks] e^{sink_h - m}),
// s_ij = bmm1 <q_i, K_j> over the keys node i sees, 0 where it sees none.
//
// What bounds it.  A tree has few rows (nodes x G per kv head) against a long
// context, so K and V are read once for all of them: up to about 280 rows per
// kv head the time is that of the K/V stream from HBM, beyond that of the
// tensor cores and the exponentials.
//
// Work.  A unit is (request, kv head, up to kTiles query tiles of 128 rows);
// all units' kv tiles of 128 keys, laid end to end, are cut into equal runs,
// one per CTA, one CTA per SM (TreeCut).  Every CTA finds its run from the
// lengths alone: no list, no counters, nothing that two launches or two graphs
// could share, and equal shares whatever the lengths.  A CTA thus has at most
// two segments that are parts of a unit, the first and the last of its run;
// those leave unnormalised rows with (m, l) in the workspace, which
// tree_merge_kernel puts together in a fixed order.
//
//   warp 0   producer: walks the run, posts each segment's description to the
//            other roles, and loads K/V pages (one TMA box per page and
//            128-byte column block) into a ring of K and V entries.
//   warp 1   MMA issuer; owns TMEM.
//   warp 2   loads Q (a TMA box per softmax warp's tokens and column block);
//            e4m3 caches: splits it into two e4m3 terms.
//   warp 3   makes V safe where rows see different keys (see below).
//   warps 4-7, 8-11   softmax A and B: one thread per MMA row.
//
// kTiles 2 (more than one tile of rows in some request): A and B each have
// their own query tile, and K/V are read once for both.  kTiles 1: there is
// one query tile; A takes the even kv tiles of a segment and B the odd ones,
// each with its own S and O in TMEM, so that the tensor core, the two softmax
// groups and the loads overlap although there is a single tile of rows; they
// merge at the end, each writing half of the columns.
//
// e4m3 caches.  K and V go to the tensor core as they are (kind::f8f6f4), so
// that no thread touches them; what is 16 or 32 bits wide is split instead.
// A Q row is scaled by a power of two and split into two e4m3 terms whose sum
// is exact for every element within 2^-9 of the row's largest, and off by at
// most 2^-17 of the largest below; S = Qh K^T + Ql K^T.  A probability, kept in
// (0, 2^8] with its row's largest at 2^7 or more, is split into its leading
// four bits and the rest rounded to four: off by at most half a step of bf16
// (2^-8), down to 2^-17 of the row's largest.  Two 8-bit MMAs take the time of
// one 16-bit MMA.
//
// V and keys that some rows of a tile do not see: their P is 0, but 0 times
// an infinity or NaN is NaN.  Keys before the item's first and past the last
// are zeroed in shared memory; keys that some rows see (tree nodes, a window's
// edge) are looked over, and one that is not finite is zeroed and added to the
// rows that see it in the epilogue, from global memory, in fp32.
//
// TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+D), O1
// [256+D,256+2D).  P overwrites the first 64 columns of S.
//
// Every wait is bounded, as in attn_tc.cu.
#include <mutex>

#include "attn_common.cuh"
#include "tree.cuh"

namespace b2pa {

namespace {

constexpr int kTreeThreads = 384;
constexpr int kTreeSlots = 4;     // posted segments in flight
constexpr int kTreeConsumers = 11;  // warps that read a posted segment
constexpr int kBadSlots = 8;

template <int D, bool FP8, int kTiles>
struct TreeCfg {
    static constexpr int kBlockBytes = kQRows * 128;        // 128 rows of one 128-byte column block
    static constexpr int kHalves = FP8 ? 1 : D / 64;        // column blocks of a K/V row
    static constexpr int kQHalves = D / 64;                 // column blocks of a Q row (bf16; e4m3: its two terms)
    static constexpr int kKvBytes = kHalves * kBlockBytes;
    static constexpr int kQBytes = kQHalves * kBlockBytes;
    static constexpr int kQBufs = D == 128 && !FP8 ? 1 : 2;
    static constexpr int kRing = 224 * 1024 - kQBufs * kTiles * kQBytes;
    static constexpr int kEntries = kRing / kKvBytes;       // K and V tiles, alternating
    static constexpr int kOffRing = kQBufs * kTiles * kQBytes;
    static constexpr int kOffBar = kOffRing + kEntries * kKvBytes;
    static constexpr int kNumBars = 3 * kEntries + 3 * kQBufs + 3 * 2 + 2 + 1 + 2 * kTreeSlots + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem address, abort flag
    static constexpr int kOffItems = kOffMisc + 16;
    static constexpr int kOffBad = kOffItems + kTreeSlots * 12 * 4;
    static constexpr int kOffExp = kOffBad + kBadSlots * 4;  // e4m3: exponent of each Q row (int8)
    static constexpr int kOffMl = (kOffExp + (FP8 ? kQBufs * kTiles * kQRows : 0) + 15) / 16 * 16;
    static constexpr int kSmemBytes = kOffMl + (kTiles == 1 ? 2 * kQRows * 8 : 0);
    static constexpr int kTmemCols = 512;
    static constexpr int kOCol = 2 * kKvTile;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(!FP8 || D == 128, "e4m3 caches: D = 128");
    static_assert(kEntries >= 5 && kEntries <= 32, "ring");
    static_assert(kSmemBytes <= 232448, "shared memory");
};

struct TreeCtx : Ctx {
    uint64_t *kv_full, *kv_empty, *v_ready;  // [kEntries]
    uint64_t *q_full, *q_empty, *q_conv;     // [kQBufs]
    uint64_t *s_full, *p_full, *o_full;      // [2]
    uint64_t *met, *left;                    // kTiles 1: both groups posted (m, l); both have read O
    uint64_t *drain, *it_full, *it_empty, *never;
};

// A segment: kv tiles j0 .. j0 + tiles - 1 of a unit.
struct Seg {
    int on, kvh, q0, n, kv_len, tok0, toks, j0, tiles, whole, slot;
    __device__ __forceinline__ int ctx() const { return kv_len - n; }
    // first key any row sees; first key from which on every row sees the context
    __device__ __forceinline__ int lo(int window) const { return window < 0 ? 0 : max(0, ctx() - window); }
    __device__ __forceinline__ int lo_all(int window) const { return window < 0 ? 0 : max(0, kv_len - 1 - window); }
    // a tile with keys that not every row sees
    __device__ __forceinline__ bool mixed(int j, int window) const
    {
        return j * kKvTile + kKvTile > ctx() || j * kKvTile < lo_all(window);
    }
};

__device__ __forceinline__ void post_seg(volatile int* rec, const Seg& s)
{
    rec[0] = s.on;
    rec[1] = s.kvh;
    rec[2] = s.q0;
    rec[3] = s.n;
    rec[4] = s.kv_len;
    rec[5] = s.tok0;
    rec[6] = s.toks;
    rec[7] = s.j0;
    rec[8] = s.tiles;
    rec[9] = s.whole;
    rec[10] = s.slot;
}

// The n-th segment of this CTA (on = 0: no more); false if the CTA gave up.
__device__ __forceinline__ bool take_seg(const TreeCtx& c, uint32_t n, Seg* s)
{
    const uint32_t slot = n % kTreeSlots;
    if (!wait_bar(&c.it_full[slot], (n / kTreeSlots) & 1, c))
        return false;
    const volatile int* rec = c.item_slot + slot * 12;
    s->on = rec[0];
    s->kvh = rec[1];
    s->q0 = rec[2];
    s->n = rec[3];
    s->kv_len = rec[4];
    s->tok0 = rec[5];
    s->toks = rec[6];
    s->j0 = rec[7];
    s->tiles = rec[8];
    s->whole = rec[9];
    s->slot = rec[10];
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&c.it_empty[slot]);
    return true;
}

// Tokens of query tile t of a segment.
__device__ __forceinline__ int tile_tokens(const TreeRows& r, const Seg& s, int t)
{
    return min(r.tile_toks, s.toks - t * r.tile_toks);
}

// ---------------------------------------------------------------------------
// warp 0
// ---------------------------------------------------------------------------
template <int D, bool FP8, int kTiles>
__device__ void tree_producer(const TreeParams& p, const TreeCtx& c, long long pos, long long end, int b, long long base)
{
    using C = TreeCfg<D, FP8, kTiles>;
    const int lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(c.base + C::kOffRing);
    const int P = p.page_size, log2_p = 31 - __clz(P);  // the tensor-core path takes powers of two only
    const int box_rows = P >= kKvTile ? kKvTile : P;
    const int item_toks = kTiles * p.rows.tile_toks;
    uint32_t q = 0;  // ring entries filled
    bool ok = true;
    TreeReq r = pos < end ? tree_request(p, b, item_toks) : TreeReq{};
    const long long begin = pos;
    int4* note = p.part_seg + (long long)blockIdx.x * 4;  // of slots 0 and 1
    if (lane < 2)
        TreePart{}.write(note + 2 * lane);
    __syncwarp();
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kTreeSlots;
        if (!wait_bar(&c.it_empty[slot], ((n / kTreeSlots) & 1) ^ 1, c))
            break;
        Seg s{};
        if (pos < end) {
            while (pos - base >= r.work(p.Hkv) && b + 1 < p.B) {
                base += r.work(p.Hkv);
                r = tree_request(p, ++b, item_toks);
            }
            const long long at = pos - base, unit = at / r.tiles;
            const int off = (int)(at - unit * r.tiles);
            const int it = (int)(unit % r.items);
            s.on = 1;
            s.kvh = (int)(unit / r.items);
            s.q0 = r.q0;
            s.n = r.n;
            s.kv_len = r.kv_len;
            s.tok0 = it * item_toks;
            s.toks = min(item_toks, r.n - s.tok0);
            s.j0 = r.n_lo + off;
            s.tiles = (int)min((long long)(r.tiles - off), end - pos);
            s.whole = s.tiles == r.tiles;
            s.slot = pos == begin ? 0 : 1;
            pos += s.tiles;
            if (!s.whole && lane == 0)
                TreePart{r.tiles, off, s.tiles, s.q0 + s.tok0, s.toks, s.kvh}.write(note + 2 * s.slot);
        }
        if (lane == 0) {
            post_seg(c.item_slot + slot * 12, s);
            mbar_arrive(&c.it_full[slot]);
        }
        __syncwarp();
        if (!s.on)
            break;
        const int* row = p.block_tables + (long long)b * p.bt_stride;
        const int n_pages = (int)(((long long)s.kv_len + P - 1) >> log2_p);
        const int first_page = r.lo >> log2_p;  // pages before it are not read: no row sees their keys
        for (int i = 0; ok && i < s.tiles; ++i) {
            TileLoad tl = tile_load(row, s.j0 + i, lane, log2_p, n_pages);
            const int col = (int)(((long long)(s.j0 + i) * kKvTile) >> log2_p) + lane;
            tl.valid = tl.valid && col >= first_page;
            if (tl.valid && (tl.page < 0 || tl.page >= p.num_pages))
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, tl.valid)) * (uint32_t)box_rows * 128u * C::kHalves;
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                const uint32_t e = q % C::kEntries;
                if (!wait_bar(&c.kv_empty[e], ((q / C::kEntries) & 1) ^ 1, c)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx_p(&c.kv_full[e], bytes, lane == 0 ? 1u : 0u);
                __syncwarp();
                const uint32_t dst = ring + e * C::kKvBytes + (uint32_t)(lane * box_rows * 128);
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_4d_p(dst + h * C::kBlockBytes, kind ? &p.tm_v : &p.tm_k, &c.kv_full[e], h * 64, tl.slot0,
                                  s.kvh, tl.page, tl.valid ? 1u : 0u);
                ++q;
            }
        }
    }
    if (*c.abort_flag) {  // let the copies in flight land before the CTA releases its memory
        const uint32_t first = q > (uint32_t)C::kEntries ? q - C::kEntries : 0;
        for (uint32_t k = first; k < q; ++k)
            drain_wait(&c.kv_full[k % C::kEntries], (k / C::kEntries) & 1);
    }
}

// ---------------------------------------------------------------------------
// warp 1.  The whole warp waits and runs the issue code; MMAs and commits are
// predicated on lane 0.
// ---------------------------------------------------------------------------
template <int D, bool FP8, int kTiles>
__device__ void tree_mma(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, kTiles>;
    // f32 accumulators; bf16 operands (format 1 of kind::f16) or e4m3 (format 0 of kind::f8f6f4)
    constexpr uint32_t kFmt = FP8 ? 0u : 1u;
    constexpr uint32_t kIdescS = (1u << 4) | (kFmt << 7) | (kFmt << 10) | ((uint32_t)(kKvTile >> 3) << 17) |
                                 ((uint32_t)(kQRows >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (kFmt << 7) | (kFmt << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                 ((uint32_t)(kQRows >> 4) << 24);
    const uint32_t issue = (threadIdx.x & 31) == 0 ? 1u : 0u;
    constexpr uint32_t kHi = sdesc_hi_sw128(1024);  // 8 rows x 128 B per core group
    const uint32_t q_lo = sdesc_lo(smem_u32(c.base), 16);                                   // K-major: LBO unused
    const uint32_t k_lo = sdesc_lo(smem_u32(c.base + C::kOffRing), 16);
    const uint32_t v_lo = sdesc_lo(smem_u32(c.base + C::kOffRing), C::kBlockBytes);         // MN-major: next column block
    constexpr uint32_t kEntryW = C::kKvBytes >> 4, kQTileW = C::kQBytes >> 4, kBlockW = C::kBlockBytes >> 4;

    // S of buffer `buf` = query tile t of Q buffer qb times the K in ring entry e
    auto issue_s = [&](uint32_t qb, int t, int buf, uint32_t e) {
        const uint32_t a0 = q_lo + (qb * kTiles + t) * kQTileW, b0 = k_lo + e * kEntryW;
        const uint32_t d = c.tmem + (uint32_t)(buf * kKvTile);
        if constexpr (FP8) {
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int k = 0; k < D / 32; ++k)  // 32 elements = 32 B
                    mma8_ss_wp(d, a0 + term * kBlockW + k * 2, b0 + k * 2, kHi, kIdescS, term + k > 0 ? 1u : 0u, issue);
        } else {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {  // 16 elements = 32 B
                const uint32_t off = (uint32_t)((k / 4) * kBlockW + (k % 4) * 2);
                mma_ss_wp(d, a0 + off, b0 + off, kHi, kIdescS, k > 0 ? 1u : 0u, issue);
            }
        }
    };
    // O of buffer `buf` (+)= P of that buffer times the V in ring entry e
    auto issue_pv = [&](int buf, uint32_t e, bool acc) {
        const uint32_t b0 = v_lo + e * kEntryW;
        const uint32_t d = c.tmem + (uint32_t)(C::kOCol + buf * D), a = c.tmem + (uint32_t)(buf * kKvTile);
        if constexpr (FP8) {
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int k = 0; k < kKvTile / 32; ++k)  // 32 keys: 8 columns of P, 32 rows of 128 B
                    mma8_ts_wp(d, a + (uint32_t)(term * 32 + k * 8), b0 + (uint32_t)(k * 256), kHi, kIdescO,
                               (acc || term + k > 0) ? 1u : 0u, issue);
        } else {
#pragma unroll
            for (int k = 0; k < kKvTile / 16; ++k)  // 16 keys: 8 columns of P, 16 rows of 128 B
                mma_ts_wp(d, a + (uint32_t)(k * 8), b0 + (uint32_t)(k * 128), kHi, kIdescO, (acc || k > 0) ? 1u : 0u,
                          issue);
        }
    };
    uint32_t r0 = 0;           // kv tiles before this segment; tile i's K and V are entries 2 (r0 + i), + 1
    uint32_t ready_bits = 0;   // parity of each entry's next v_ready phase
    uint32_t p_cnt[2] = {0, 0};
    bool ok = true;
    auto wait_k = [&](int i) {
        const uint32_t e = 2 * (r0 + i);
        return wait_bar(&c.kv_full[e % C::kEntries], (e / C::kEntries) & 1, c);
    };
    auto entry = [&](int i, int kind) { return (2 * (r0 + i) + kind) % C::kEntries; };
    auto wait_v = [&](const Seg& s, int i) {
        const uint32_t q = 2 * (r0 + i) + 1, e = q % C::kEntries;
        if (!wait_bar(&c.kv_full[e], (q / C::kEntries) & 1, c))
            return false;
        if (!s.mixed(s.j0 + i, p.window))
            return true;
        const uint32_t parity = ready_bits >> e & 1u;
        ready_bits ^= 1u << e;
        return wait_bar(&c.v_ready[e], parity, c);
    };
    auto wait_p = [&](int buf) {
        const bool got = wait_bar(&c.p_full[buf], p_cnt[buf] & 1, c);
        ++p_cnt[buf];
        tc_fence_after();
        return got;
    };

    if (p.inject_stall && !wait_bar(c.never, 0, c))  // failure-detection tests
        ok = false;
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const uint32_t qb = n % C::kQBufs;
        if (!wait_bar(FP8 ? &c.q_conv[qb] : &c.q_full[qb], (n / C::kQBufs) & 1, c))
            break;
        if constexpr (kTiles == 1) {
            // tile i in buffer i % 2; S runs two tiles ahead
            auto next_s = [&](int i) {
                if (!wait_k(i))
                    return false;
                issue_s(qb, 0, i & 1, entry(i, 0));
                mma_commit_p(&c.s_full[i & 1], issue);
                mma_commit_p(&c.kv_empty[entry(i, 0)], issue);
                if (i == s.tiles - 1)
                    mma_commit_p(&c.q_empty[qb], issue);
                return true;
            };
            ok = next_s(0) && (s.tiles < 2 || next_s(1));
            for (int i = 0; ok && i < s.tiles; ++i) {
                if (!wait_v(s, i) || !wait_p(i & 1)) {
                    ok = false;
                    break;
                }
                issue_pv(i & 1, entry(i, 1), i >= 2);
                mma_commit_p(&c.kv_empty[entry(i, 1)], issue);
                if (i + 2 >= s.tiles)
                    mma_commit_p(&c.o_full[i & 1], issue);
                else
                    ok = next_s(i + 2);
            }
        } else {
            // tile t's S for kv tile i + 1 follows its P V for kv tile i
            const int nq = s.toks > p.rows.tile_toks ? 2 : 1;
            auto next_s = [&](int i, int t) {
                if (t == 0 && !wait_k(i))
                    return false;
                issue_s(qb, t, t, entry(i, 0));
                mma_commit_p(&c.s_full[t], issue);
                if (t == nq - 1) {
                    mma_commit_p(&c.kv_empty[entry(i, 0)], issue);
                    if (i == s.tiles - 1)
                        mma_commit_p(&c.q_empty[qb], issue);
                }
                return true;
            };
            for (int t = 0; ok && t < nq; ++t)
                ok = next_s(0, t);
            for (int i = 0; ok && i < s.tiles; ++i) {
                if (!wait_v(s, i)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || t >= nq)
                        break;
                    if (!wait_p(t)) {
                        ok = false;
                        break;
                    }
                    issue_pv(t, entry(i, 1), i > 0);
                    if (t == nq - 1)
                        mma_commit_p(&c.kv_empty[entry(i, 1)], issue);
                    if (i == s.tiles - 1)
                        mma_commit_p(&c.o_full[t], issue);
                    else
                        ok = next_s(i + 1, t);
                }
            }
        }
        r0 += (uint32_t)s.tiles;
    }
    // every MMA this thread issued has completed once the drain barrier flips
    if (issue)
        mma_commit(c.drain);
    __syncwarp();
    drain_wait(c.drain, 0);
}

// ---------------------------------------------------------------------------
// warp 2: Q
// ---------------------------------------------------------------------------
// Two floats -> two e4m3 codes (`lo` in the low byte), and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float2 f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// One Q row of 128 bf16 values in shared memory (two column blocks of 128
// bytes, 16-byte chunks swizzled by row % 8) becomes its two e4m3 terms, in
// place: the high one in the first block, the low one in the second.  Returns
// the power of two it was scaled by, which brings its largest value to
// [2^7, 2^8).  A row that is not finite becomes NaN, which is what every score
// of it makes of the softmax.
__device__ __forceinline__ int split_q_row(uint8_t* row, int sw, int block_bytes)
{
    uint4 x[16];
    uint32_t mx = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {  // eight elements each
        x[k] = *reinterpret_cast<const uint4*>(row + (k >> 3) * block_bytes + (((k & 7) ^ sw) << 4));
        const uint32_t m = __vmaxu2(__vmaxu2(x[k].x & 0x7FFF7FFFu, x[k].y & 0x7FFF7FFFu),
                                    __vmaxu2(x[k].z & 0x7FFF7FFFu, x[k].w & 0x7FFF7FFFu));
        mx = max(mx, max(m & 0xFFFFu, m >> 16));
    }
    const int e = mx == 0 || mx >= 0x7F80u ? 0 : min(120, max(-120, 7 - ((int)(mx >> 7) - 127)));
    const float sc = __int_as_float((127 + e) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // sixteen elements each
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            hi[w] = lo[w] = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 v = x[2 * k + w / 2];
                const int word = (w % 2) * 2 + i;
                const uint32_t u = word == 0 ? v.x : word == 1 ? v.y : word == 2 ? v.z : v.w;
                const float a = __uint_as_float(u << 16) * sc, b = __uint_as_float(u & 0xFFFF0000u) * sc;
                const uint32_t h = to_e4m3x2(a, b);
                const float2 f = from_e4m3x2(h);
                hi[w] |= h << (16 * i);
                lo[w] |= to_e4m3x2(a - f.x, b - f.y) << (16 * i);
            }
            if (mx >= 0x7F80u)
                hi[w] = 0x7F7F7F7Fu;
        }
        uint8_t* to = row + ((k ^ sw) << 4);
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(to + block_bytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return e;
}

template <int D, bool FP8, int kTiles>
__device__ void tree_q(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, kTiles>;
    const int lane = threadIdx.x & 31;
    const TreeRows& r = p.rows;
    uint32_t loads = 0;
    for (uint32_t n = 0;; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const uint32_t qb = n % C::kQBufs, ph = (n / C::kQBufs) & 1;
        if (!wait_bar(&c.q_empty[qb], ph ^ 1, c))
            break;
        // lane = (tile, warp's tokens, column block): one box each
        const int t = lane / (4 * C::kQHalves), w = lane / C::kQHalves % 4, h = lane % C::kQHalves;
        const int toks = t < kTiles ? tile_tokens(r, s, t) : 0;
        const int per = r.by_warp ? (toks + 3) >> 2 : r.tile_toks;
        const bool box = toks > 0 && w * per < toks && (r.by_warp || w == 0);
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
        mbar_arrive_expect_tx_p(&c.q_full[qb], boxes * (uint32_t)(r.G * r.box_toks * 128), lane == 0 ? 1u : 0u);
        __syncwarp();
        if (box)
            tma_load_3d(smem_u32(c.base) + (qb * kTiles + t) * C::kQBytes + h * C::kBlockBytes + w * 32 * 128, &p.tm_q,
                        &c.q_full[qb], h * 64, s.kvh * r.G, s.q0 + s.tok0 + t * r.tile_toks + w * per);
        loads = n + 1;
        __syncwarp();
        if constexpr (FP8) {
            if (!wait_bar(&c.q_full[qb], ph, c))
                break;
            int8_t* exps = reinterpret_cast<int8_t*>(c.base + C::kOffExp) + qb * kTiles * kQRows;
#pragma unroll 1
            for (int k = 0; k < kTiles * 4; ++k) {
                const int row = (k & 3) * 32 + lane;
                exps[(k >> 2) * kQRows + row] = (int8_t)split_q_row(
                    c.base + (qb * kTiles + (k >> 2)) * C::kQBytes + row * 128, row & 7, C::kBlockBytes);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&c.q_conv[qb]);
        }
    }
    if (*c.abort_flag) {
        const uint32_t first = loads > (uint32_t)C::kQBufs ? loads - C::kQBufs : 0;
        for (uint32_t k = first; k < loads; ++k)
            drain_wait(&c.q_full[k % C::kQBufs], (k / C::kQBufs) & 1);
    }
}

// ---------------------------------------------------------------------------
// warp 3: V of tiles with keys that not every row sees
// ---------------------------------------------------------------------------
template <bool FP8>
__device__ __forceinline__ bool not_finite(uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (FP8)
            bad |= __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
        else
            bad |= __vcmpeq2(w[i] & 0x7F807F80u, 0x7F807F80u) != 0;
    }
    return bad;
}

template <int D, bool FP8, int kTiles>
__device__ void tree_v(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, kTiles>;
    constexpr int kChunks = 8 * C::kHalves;      // 16-byte pieces of a V row
    constexpr int kRowsAtOnce = 32 / kChunks;
    const int lane = threadIdx.x & 31;
    const int sub = lane / kChunks, chunk = lane % kChunks;
    volatile int* bad = reinterpret_cast<volatile int*>(c.base + C::kOffBad);
    uint32_t q = 0;  // ring entries seen
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        if (lane == 0)
            bad[n % kBadSlots] = 0;
        __syncwarp();
        const int lo = s.lo(p.window), lo_all = s.lo_all(p.window), ctx = s.ctx();
        // every entry is awaited and released in order, so that this warp never
        // lags a barrier by more than one phase
        for (int k = 0; k < 2 * s.tiles; ++k, ++q) {
            const uint32_t e = q % C::kEntries;
            const int i = k >> 1;
            if (!wait_bar(&c.kv_full[e], (q / C::kEntries) & 1, c)) {
                ok = false;
                break;
            }
            if (!(k & 1) || !s.mixed(s.j0 + i, p.window)) {
                mbar_arrive_p(&c.kv_empty[e], lane == 0 ? 1u : 0u);
                continue;
            }
            uint8_t* v = c.base + C::kOffRing + e * C::kKvBytes + (chunk >> 3) * C::kBlockBytes + (chunk & 7) * 16;
            const int k0 = (s.j0 + i) * kKvTile;
#pragma unroll 4
            for (int row = sub; row < kKvTile; row += kRowsAtOnce) {
                const int key = k0 + row;
                uint4* at = reinterpret_cast<uint4*>(v + row * 128);
                const bool out = key < lo || key >= s.kv_len;          // no row sees it (it may never have been loaded)
                const bool some = !out && (key < lo_all || key >= ctx);  // some rows may not
                bool zero = out;
                if (__any_sync(0xffffffffu, some)) {
                    const bool here = some && not_finite<FP8>(*at);
                    const uint32_t m = __ballot_sync(0xffffffffu, here);
                    const bool any = (m >> (sub * kChunks) & (kChunks == 32 ? 0xffffffffu : (1u << kChunks) - 1u)) != 0;
                    zero = zero || any;
                    if (m != 0 && lane == 0)
                        bad[n % kBadSlots] = 1;
                }
                if (zero)
                    *at = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&c.v_ready[e]);
                mbar_arrive(&c.kv_empty[e]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// softmax A (t = 0) and B (t = 1)
// ---------------------------------------------------------------------------
__device__ __forceinline__ float fmax3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u; }

// Which of the keys c0 .. c0 + 31 a row sees.
struct RowView {
    int lo, ctx, n;
    const unsigned* mask;  // the node's mask row
    int words;
    __device__ __forceinline__ uint32_t sees(int c0) const
    {
        uint32_t w = 0;
        if (c0 < ctx)
            w = low_bits(ctx - c0) & ~low_bits(lo - c0);
        const int node = c0 - ctx;  // bit 0's node
        if (node > -32 && node < n) {
            uint32_t bits;
            if (node < 0) {
                bits = mask[0] << -node;
            } else {
                const int at = node >> 5, sh = node & 31;
                bits = at < words ? mask[at] >> sh : 0u;
                if (sh != 0 && at + 1 < words)
                    bits |= mask[at + 1] << (32 - sh);
            }
            w |= bits & low_bits(n - node) & ~low_bits(-node);
        }
        return w;
    }
};

template <bool FP8>
__device__ __forceinline__ float kv_elem(const void* base, long long at)
{
    if (FP8)
        return from_e4m3x2(static_cast<const uint8_t*>(base)[at]).x;
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[at] << 16);
}

// Slow path: column d of the V rows that tree_v zeroed because they are not
// finite, weighted for this row, with the stabiliser m of its exponentials.
template <bool FP8>
__device__ __noinline__ float tree_bad_column(const TreeParams& p, const int* row_pages, const RowView view, int lo_all,
                                              int key0, int key1, int tok, int head, int kvh, float sl2, float m, int d)
{
    float sum = 0.f;
    const uint16_t* q = p.q + (long long)tok * p.q_st_tok + (long long)head * p.q_st_head;
    const int last = view.ctx + view.n;
    for (int key = max(key0, view.lo); key < min(key1, last); ++key) {
        if (key >= lo_all && key < view.ctx)
            key = view.ctx;  // these were not looked at
        if (key >= min(key1, last))
            break;
        if (!(view.sees(key) & 1u))
            continue;
        const int page = row_pages[key / p.page_size], slot = key % p.page_size;
        if (page < 0 || page >= p.num_pages)
            continue;
        const long long ko = (long long)page * p.k_st[0] + (long long)kvh * p.k_st[1] + (long long)slot * p.k_st[2];
        const long long vo = (long long)page * p.v_st[0] + (long long)kvh * p.v_st[1] + (long long)slot * p.v_st[2];
        bool bad = false;
        float dot = 0.f;
        for (int k = 0; k < p.D; ++k) {
            bad |= !isfinite(kv_elem<FP8>(p.v, vo + k));
            dot = fmaf(__uint_as_float((uint32_t)q[k] << 16), kv_elem<FP8>(p.k, ko + k), dot);
        }
        if (bad)
            sum += ex2_approx(fmaf(dot, sl2, -m)) * kv_elem<FP8>(p.v, vo + d);
    }
    return sum;
}

template <int D, bool FP8, int kTiles>
__device__ void tree_softmax(const TreeParams& p, const TreeCtx& c, int t)
{
    using C = TreeCfg<D, FP8, kTiles>;
    constexpr float kLog2e = 1.4426950408889634f;
    // e = 2^(x - m + kBias): e4m3 terms use their range from 2^kBias down.  The
    // stabiliser is renewed once the row's maximum has grown by kSlack.
    constexpr float kBias = FP8 ? 7.f : 0.f, kSlack = FP8 ? 1.f : 8.f;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, row = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t s_tmem = c.tmem + lane_off + (uint32_t)(t * kKvTile);
    const uint32_t o_tmem = c.tmem + lane_off + (uint32_t)C::kOCol;  // + buffer * D
    const TreeRows& rows = p.rows;
    const int G = rows.G;
    const int step = kTiles == 1 ? 2 : 1;
    float2* ml = reinterpret_cast<float2*>(c.base + C::kOffMl);
    const volatile int* bad = reinterpret_cast<const volatile int*>(c.base + C::kOffBad);

    uint32_t s_cnt = 0, o_cnt = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const uint32_t qb = n % C::kQBufs;
        // every warp awaits every segment's Q and releases it once it has read the
        // exponents it needs: the buffer and its barrier cannot run ahead of a group
        // that is still at an earlier segment
        float q_unscale = 1.f;
        const int qt = kTiles == 1 ? 0 : t;
        if constexpr (FP8) {
            if (!wait_bar(&c.q_conv[qb], (n / C::kQBufs) & 1, c)) {
                ok = false;
                break;
            }
            const int e = reinterpret_cast<const volatile int8_t*>(c.base + C::kOffExp)[(qb * kTiles + qt) * kQRows + row];
            q_unscale = __int_as_float((127 - e) << 23);
            __syncwarp();
            mbar_arrive_p(&c.q_empty[qb], lane == 0 ? 1u : 0u);
        }
        if (kTiles == 1 && n > 0 && !wait_bar(c.left, (n - 1) & 1, c)) {  // O and ml of the last segment are free
            ok = false;
            break;
        }
        if (kTiles == 2 && qt * rows.tile_toks >= s.toks)
            continue;
        const int toks = tile_tokens(rows, s, qt);
        const int per = (toks + 3) >> 2;
        const int local = rows.by_warp ? wq * per + lane / G : row / G;
        const int head = rows.by_warp ? lane % G : row % G;
        const bool valid = rows.by_warp ? lane < G * per && local < toks : row < G * toks;
        const int tok = s.q0 + s.tok0 + qt * rows.tile_toks + (valid ? local : 0);
        const bool warp_on = __any_sync(0xffffffffu, valid);
        const float sl2 = p.scale_log2 * q_unscale;
        RowView view;
        view.ctx = s.ctx();
        view.n = s.n;
        view.lo = p.window < 0 ? 0 : tree_row_lo(p.positions[tok], view.ctx, s.kv_len, p.window);
        view.mask = p.mask + (long long)tok * p.mask_stride;
        view.words = p.mask_words;

        float m_used = -INFINITY, l = 0.f;
        for (int i = kTiles == 1 ? t : 0; i < s.tiles; i += step) {
            if (!wait_bar(&c.s_full[t], s_cnt & 1, c)) {
                ok = false;
                break;
            }
            ++s_cnt;
            if (!warp_on) {  // no row of this warp is anyone's
                mbar_arrive_p(&c.p_full[t], lane == 0 ? 1u : 0u);
                continue;
            }
            tc_fence_after();
            float x[kKvTile];
            float mq[4];  // maxima of the four 32-key loads
            {
                uint32_t r[32];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tmem_ld32_max(s_tmem + (uint32_t)(q * 32), r, &mq[q]);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        x[q * 32 + k] = __uint_as_float(r[k]);
                }
                tmem_wait_ld();
            }
            const int k0 = (s.j0 + i) * kKvTile;
            // rows that are nobody's count as seeing everything; what they compute stays in their row
            if (!__all_sync(0xffffffffu, !valid || (k0 >= view.lo && k0 + kKvTile <= view.ctx))) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t w = valid ? view.sees(k0 + 32 * q) : 0xffffffffu;
                    if (__all_sync(0xffffffffu, w == 0xffffffffu))
                        continue;
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(w >> k & 1u))
                            x[32 * q + k] = -INFINITY;
                    float m0 = fmax3(x[32 * q], x[32 * q + 1], x[32 * q + 2]);
                    float m1 = fmax3(x[32 * q + 16], x[32 * q + 17], x[32 * q + 18]);
#pragma unroll
                    for (int k = 3; k < 15; k += 2) {
                        m0 = fmax3(m0, x[32 * q + k], x[32 * q + k + 1]);
                        m1 = fmax3(m1, x[32 * q + 16 + k], x[32 * q + 16 + k + 1]);
                    }
                    mq[q] = fmax3(m0, m1, fmaxf(x[32 * q + 15], x[32 * q + 31]));
                }
            }
            const float m_tile = fmax3(fmax3(mq[0], mq[1], mq[2]), mq[3], -INFINITY) * sl2;
            const bool need = valid && m_tile > m_used + kSlack;
            const float alpha = need ? ex2_approx(m_used - m_tile) : 1.f;
            l *= alpha;
            m_used = need ? m_tile : m_used;
            const float neg = m_used == -INFINITY ? 0.f : kBias - m_used;
            const float2 sc = make_float2(sl2, sl2), ng = make_float2(neg, neg);
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
            const bool rescale = __any_sync(0xffffffffu, need) && i >= step;
            if constexpr (FP8) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // 64 keys: 16 columns of each term
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int w = 0; w < 16; ++w) {
                        hi[w] = lo[w] = 0;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int k = q * 64 + w * 4 + h * 2;
                            const float2 y = __ffma2_rn(make_float2(x[k], x[k + 1]), sc, ng);
                            const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                            acc[w & 3] = __fadd2_rn(acc[w & 3], e);
                            // leading four bits, and the rest
                            const float2 f = make_float2(__uint_as_float(__float_as_uint(e.x) & 0xFFF00000u),
                                                         __uint_as_float(__float_as_uint(e.y) & 0xFFF00000u));
                            hi[w] |= to_e4m3x2(f.x, f.y) << (16 * h);
                            lo[w] |= to_e4m3x2(e.x - f.x, e.y - f.y) << (16 * h);
                        }
                    }
                    tmem_st16(s_tmem + (uint32_t)(q * 16), hi);
                    tmem_st16(s_tmem + (uint32_t)(32 + q * 16), lo);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // 32 keys: 16 columns
                    uint32_t pk[16];
#pragma unroll
                    for (int w = 0; w < 16; ++w) {
                        const int k = q * 32 + w * 2;
                        const float2 y = __ffma2_rn(make_float2(x[k], x[k + 1]), sc, ng);
                        const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                        acc[w & 3] = __fadd2_rn(acc[w & 3], e);
                        pk[w] = pack_bf16x2(e.x, e.y);
                    }
                    tmem_st16(s_tmem + (uint32_t)(q * 16), pk);
                }
            }
            if (rescale) {
                // O holds this group's sum up to its last tile (that P V precedes this S)
                const float2 ff = make_float2(alpha, alpha);
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                    uint32_t o[16];
                    tmem_ld16(o_tmem + (uint32_t)(t * D + q * 16), o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), ff);
                        o[k] = __float_as_uint(v.x);
                        o[k + 1] = __float_as_uint(v.y);
                    }
                    tmem_st16(o_tmem + (uint32_t)(t * D + q * 16), o);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_p(&c.p_full[t], lane == 0 ? 1u : 0u);
            const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
            const float2 a = __fadd2_rn(a01, a23);
            l += a.x + a.y;
        }
        if (!ok)
            break;
        const bool had = kTiles == 2 || t < s.tiles;
        if (had) {
            if (!wait_bar(&c.o_full[t], o_cnt & 1, c)) {
                ok = false;
                break;
            }
            ++o_cnt;
        }
        // from here on the stabiliser of l and O is m
        float m = m_used == -INFINITY ? m_used : m_used - kBias;
        float w0 = 1.f, w1 = 0.f;  // weights of the O buffers (kTiles 1: of A and B)
        if constexpr (kTiles == 1) {
            ml[t * kQRows + row] = make_float2(m, l);
            __syncwarp();
            mbar_arrive_p(c.met, lane == 0 ? 1u : 0u);
            if (!wait_bar(c.met, n & 1, c)) {
                ok = false;
                break;
            }
            const float2 x0 = ml[row], x1 = ml[kQRows + row];
            m = fmaxf(x0.x, x1.x);
            // (a sum that is no number keeps its weight, whatever its maximum)
            w0 = x0.x == -INFINITY && x0.y == 0.f ? 0.f : m == -INFINITY ? 1.f : ex2_approx(x0.x - m);
            w1 = x1.x == -INFINITY && x1.y == 0.f ? 0.f : m == -INFINITY ? 1.f : ex2_approx(x1.x - m);
            l = (w0 != 0.f ? w0 * x0.y : 0.f) + (w1 != 0.f ? w1 * x1.y : 0.f);
        }
        tc_fence_after();
        const int h = s.kvh * G + head;
        float out_scale = 1.f;
        if (s.whole) {
            float total = l;
            if (p.sinks != nullptr && m != -INFINITY)
                total += ex2_approx(fmaf(p.sinks[valid ? h : 0], kLog2e, -m));
            out_scale = total == 0.f ? 0.f : p.bmm2 / total;
        }
        const int d0 = kTiles == 1 ? t * (D / 2) : 0, d1 = kTiles == 1 ? d0 + D / 2 : D;
        const bool any_bad = bad[n % kBadSlots] != 0;
        const long long part = ((long long)(blockIdx.x * 2 + s.slot) * kTiles + qt) * kQRows + row;
        uint16_t* orow = p.out + (long long)tok * p.out_st_tok + (long long)h * p.out_st_head;
        if (warp_on) {
#pragma unroll 1
            for (int d = d0; d < d1; d += 32) {
                uint32_t o[32];
                if constexpr (kTiles == 1) {
                    uint32_t o1[32];
                    tmem_ld32(o_tmem + (uint32_t)d, o);
                    tmem_ld32(o_tmem + (uint32_t)(D + d), o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k)  // a buffer without weight may hold anything
                        o[k] = __float_as_uint((w0 != 0.f ? w0 * __uint_as_float(o[k]) : 0.f) +
                                               (w1 != 0.f ? w1 * __uint_as_float(o1[k]) : 0.f));
                } else {
                    tmem_ld32(o_tmem + (uint32_t)(t * D + d), o);
                    tmem_wait_ld();
                }
                if (any_bad && valid) {
                    const int* pages = p.block_tables;  // the request's row: found from its first token
                    int b = 0;
                    while (b + 1 < p.B && p.cum_q[b + 1] <= tok)
                        ++b;
                    pages += (long long)b * p.bt_stride;
                    const float raw = FP8 ? p.scale_log2 : sl2;
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) +
                                               tree_bad_column<FP8>(p, pages, view, s.lo_all(p.window), s.j0 * kKvTile,
                                                                    (s.j0 + s.tiles) * kKvTile, tok, h, s.kvh, raw, m, d + k));
                }
                if (valid && s.whole) {
                    const float2 f = make_float2(out_scale, out_scale);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t pk[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[8 * v + 2 * k]),
                                                                    __uint_as_float(o[8 * v + 2 * k + 1])),
                                                        f);
                            pk[k] = pack_bf16x2(y.x, y.y);
                        }
                        *reinterpret_cast<uint4*>(orow + d + 8 * v) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                } else if (valid) {
                    float4* to = reinterpret_cast<float4*>(p.part_o + part * D + d);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        to[v] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                            __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                }
            }
            if (valid && !s.whole && (kTiles == 2 || t == 0))
                p.part_ml[part] = make_float2(m, l);
        }
        tc_fence_before();
        if constexpr (kTiles == 1) {
            __syncwarp();
            mbar_arrive_p(c.left, lane == 0 ? 1u : 0u);
        }
    }
    tc_fence_before();
}

// ---------------------------------------------------------------------------

template <int D, bool FP8, int kTiles>
__global__ void __launch_bounds__(kTreeThreads, 1) attention_tree_kernel(const __grid_constant__ TreeParams p)
{
    using C = TreeCfg<D, FP8, kTiles>;
    extern __shared__ __align__(1024) uint8_t smem[];
    TreeCtx c;
    c.base = smem;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    c.kv_full = bars;
    c.kv_empty = c.kv_full + C::kEntries;
    c.v_ready = c.kv_empty + C::kEntries;
    c.q_full = c.v_ready + C::kEntries;
    c.q_empty = c.q_full + C::kQBufs;
    c.q_conv = c.q_empty + C::kQBufs;
    c.s_full = c.q_conv + C::kQBufs;
    c.p_full = c.s_full + 2;
    c.o_full = c.p_full + 2;
    c.met = c.o_full + 2;
    c.left = c.met + 1;
    c.drain = c.left + 1;
    c.it_full = c.drain + 1;
    c.it_empty = c.it_full + kTreeSlots;
    c.never = c.it_empty + kTreeSlots;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    c.abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    c.err = p.err;
    c.wait_limit_ns = p.wait_limit_ns;
    c.item_slot = reinterpret_cast<volatile int*>(smem + C::kOffItems);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int e = 0; e < C::kEntries; ++e) {
            mbar_init(&c.kv_full[e], 1);
            mbar_init(&c.kv_empty[e], 2);  // the MMAs that read it, and warp 3
            mbar_init(&c.v_ready[e], 1);
        }
        for (int b = 0; b < C::kQBufs; ++b) {
            mbar_init(&c.q_full[b], 1);
            mbar_init(&c.q_empty[b], FP8 ? 9 : 1);  // the MMAs that read it; e4m3: and the softmax warps
            mbar_init(&c.q_conv[b], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&c.s_full[t], 1);
            mbar_init(&c.p_full[t], 4);
            mbar_init(&c.o_full[t], 1);
        }
        mbar_init(c.met, 8);
        mbar_init(c.left, 8);
        mbar_init(c.drain, 1);
        for (int s = 0; s < kTreeSlots; ++s) {
            mbar_init(&c.it_full[s], 1);
            mbar_init(&c.it_empty[s], kTreeConsumers);
        }
        mbar_init(c.never, 1);
        *c.abort_flag = 0;
        fence_mbar_init();
    }
    if (tid == 32) {
        prefetch_tmap(&p.tm_q);
        prefetch_tmap(&p.tm_k);
        prefetch_tmap(&p.tm_v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c.tmem = *tmem_holder;

    pdl_wait();  // inputs may come from the kernel this launch follows

    // Where this CTA's run starts: kv tiles of the requests before each, by a
    // scan over the threads' contiguous shares of the requests (scratch in the
    // ring, which is empty yet).
    long long* scan = reinterpret_cast<long long*>(smem + C::kOffRing);  // 12 warp sums; [16] base, [17] request
    const int item_toks = kTiles * p.rows.tile_toks;
    const int share = (p.B + kTreeThreads - 1) / kTreeThreads;
    const int b0 = min(p.B, tid * share), b1 = min(p.B, b0 + share);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const TreeReq r = tree_request(p, b, item_toks);
        if (!r.ok && blockIdx.x == 0)
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
        mine += r.work(p.Hkv);
    }
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o)
            before += y;
    }
    if (lane == 31)
        scan[warp] = before;
    __syncthreads();
    long long total = 0, warps_before = 0;
#pragma unroll
    for (int w = 0; w < kTreeThreads / 32; ++w) {
        warps_before += w < warp ? scan[w] : 0;
        total += scan[w];
    }
    before += warps_before - mine;
    const TreeCut cut = tree_cut(total, gridDim.x);
    const bool works = (int)blockIdx.x < cut.g;
    const long long start = works ? cut.start(blockIdx.x) : 0, end = works ? cut.start(blockIdx.x + 1) : 0;
    if (works && start >= before && start < before + mine) {
        long long base = before;
        int b = b0;
        for (; b + 1 < b1; ++b) {  // this thread's requests, if it has several
            const long long w = tree_request(p, b, item_toks).work(p.Hkv);
            if (start < base + w)
                break;
            base += w;
        }
        scan[16] = base;
        scan[17] = b;
    }
    __syncthreads();
    const long long base = scan[16];
    const int first_b = works ? (int)scan[17] : 0;
    fence_proxy_async_smem();  // the ring's next writes come through the async proxy
    __syncthreads();

    // 384 threads launch with 168 registers each (104 + 200 + 200 = 504 = 3 x 168)
    if (warp < 4) {
        regs_dec<104>();
        if (warp == 0)
            tree_producer<D, FP8, kTiles>(p, c, start, end, first_b, base);
        else if (warp == 1)
            tree_mma<D, FP8, kTiles>(p, c);
        else if (warp == 2)
            tree_q<D, FP8, kTiles>(p, c);
        else
            tree_v<D, FP8, kTiles>(p, c);
    } else {
        regs_inc<200>();
        tree_softmax<D, FP8, kTiles>(p, c, (warp - 4) >> 2);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(c.tmem, C::kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// The merge of a unit that several CTAs shared: with the segments' (m_c, l_c,
// O_c) and m = max m_c, w_c = 2^(m_c - m),
//   out = bmm2 * sum_c w_c O_c / (sum_c w_c l_c + [sinks] 2^(sink log2 e - m)),
// in the order of the keys.  Block (i, y) takes the unit whose first segment is
// CTA i's, if there is one that goes on in the next CTA, and of its rows 8 y ..
// 8 y + 7, one per warp.  Latency alone: loads that do not depend on each other
// are issued together.
// ---------------------------------------------------------------------------
constexpr int kMergeRows = 8;

template <int D>
__global__ void __launch_bounds__(kMergeRows * 32) tree_merge_kernel(const __grid_constant__ TreeParams p, int tiles)
{
    constexpr float kLog2e = 1.4426950408889634f;
    constexpr int kPer = D / 32;  // dimensions per lane
    constexpr int kBatch = 8;     // segments whose rows are loaded together
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int first = blockIdx.x, r = (int)blockIdx.y * kMergeRows + (threadIdx.x >> 5);
    // the segment that opens a unit is the CTA's last; the ones after it are
    // the first of the CTAs that follow, up to the one that reaches the end
    const int4* notes = p.part_seg;
    TreePart x = TreePart::read(notes + (long long)first * 4);
    const TreePart last = TreePart::read(notes + (long long)first * 4 + 2);
    TreePart next = TreePart{};
    if (first + 1 + lane < p.grid)
        next = TreePart::read(notes + (long long)(first + 1 + lane) * 4);
    const int slot = last.all != 0 ? 1 : 0;
    if (slot)
        x = last;
    if (x.all == 0 || x.off != 0 || r >= x.toks * p.rows.G)
        return;
    int segs = 1;
    for (int c = first + 1;; c += 32) {
        if (c > first + 1)
            next = c + lane < p.grid ? TreePart::read(notes + (long long)(c + lane) * 4) : TreePart{};
        const unsigned m = __ballot_sync(0xffffffffu, next.off + next.tiles >= next.all);  // (none: 0 >= 0)
        if (m != 0) {
            segs += __ffs(m);
            break;
        }
        segs += 32;
    }
    const int tok = r / p.rows.G, head = r - tok * p.rows.G, h = x.kvh * p.rows.G + head;
    const int qt = tok / p.rows.tile_toks, in_tile = tok - qt * p.rows.tile_toks;
    const int row = tree_row(p.rows, in_tile, min(p.rows.tile_toks, x.toks - qt * p.rows.tile_toks), head);
    // segment c of the unit: slot 0 of CTA first + c, but for its first
    auto part = [&](int c) {
        return ((long long)((first + c) * 2 + (c == 0 ? slot : 0)) * tiles + qt) * kQRows + row;
    };
    const float sink = p.sinks != nullptr ? p.sinks[h] * kLog2e : -INFINITY;
    // running over groups of 32 segments, each lane holding one's (m, l)
    float m = -INFINITY, den = 0.f;
    float a[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        a[k] = 0.f;
    for (int c0 = 0; c0 < segs; c0 += 32) {
        const int n = min(32, segs - c0);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n)
            ml = p.part_ml[part(c0 + lane)];
        float w = 0.f;
        for (int b = 0; b < n; b += kBatch) {
            float v[kBatch][kPer];
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                if (b + c >= n)
                    break;
                const float* o = p.part_o + part(c0 + b + c) * D + lane * kPer;
                if constexpr (kPer == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(o);
                    v[c][0] = y.x;
                    v[c][1] = y.y;
                    v[c][2] = y.z;
                    v[c][3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(o);
                    v[c][0] = y.x;
                    v[c][1] = y.y;
                }
            }
            if (b == 0) {
                float top = fmaxf(m, ml.x);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float old = m == -INFINITY ? 1.f : ex2_approx(m - top);  // (no maximum yet: sums of 0 or NaN)
                // (a sum that is no number keeps its weight, whatever its maximum)
                w = ml.x == -INFINITY && ml.y == 0.f ? 0.f : top == -INFINITY ? 1.f : ex2_approx(ml.x - top);
                m = top;
                float s = w != 0.f ? w * ml.y : 0.f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                den = fmaf(den, old, s);
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    a[k] *= old;
            }
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const float wc = __shfl_sync(0xffffffffu, w, (b + c) & 31);
                if (b + c < n && wc != 0.f) {
#pragma unroll
                    for (int k = 0; k < kPer; ++k)
                        a[k] = fmaf(wc, v[c][k], a[k]);
                }
            }
        }
    }
    if (m != -INFINITY)
        den += ex2_approx(sink - m);
    const float f = den == 0.f ? 0.f : p.bmm2 / den;
    uint16_t* to = p.out + (long long)(x.row0 + tok) * p.out_st_tok + (long long)h * p.out_st_head + lane * kPer;
    if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(a[0] * f, a[1] * f), pack_bf16x2(a[2] * f, a[3] * f));
    else
        *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(a[0] * f, a[1] * f);
}

template <typename Kern, typename... Args>
cudaError_t launch_pdl(Kern kern, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool FP8, int kTiles>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream)
{
    using C = TreeCfg<D, FP8, kTiles>;
    auto kern = attention_tree_kernel<D, FP8, kTiles>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    // the shared-memory opt-in, once per device and instantiation (any host thread)
    static std::once_flag once[64];
    static cudaError_t err[64];
    std::call_once(once[dev], [&] {
        err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    });
    if (err[dev] != cudaSuccess)
        return err[dev];
    if ((e = launch_pdl(kern, dim3(p.grid), kTreeThreads, C::kSmemBytes, stream, p)) != cudaSuccess)
        return e;
    const int rows = min(p.max_q_len, kTiles * p.rows.tile_toks) * p.rows.G;  // of a unit, at most
    return launch_pdl(tree_merge_kernel<D>, dim3(p.grid, (rows + kMergeRows - 1) / kMergeRows), kMergeRows * 32, 0,
                      stream, p, kTiles);
}

}  // namespace

cudaError_t launch_attention_tree(const TreeParams& p, bool fp8, int tiles, cudaStream_t stream)
{
    if (fp8)
        return p.D != 128 ? cudaErrorInvalidValue
                          : tiles == 1 ? launch_tree<128, true, 1>(p, stream) : launch_tree<128, true, 2>(p, stream);
    if (p.D == 128)
        return tiles == 1 ? launch_tree<128, false, 1>(p, stream) : launch_tree<128, false, 2>(p, stream);
    if (p.D == 64)
        return tiles == 1 ? launch_tree<64, false, 1>(p, stream) : launch_tree<64, false, 2>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace b2pa
