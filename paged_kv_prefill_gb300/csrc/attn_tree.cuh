// attn_tree.cuh -- attention of a few rows per request over a paged cache on the
// 5th-generation tensor cores (tcgen05): of drafted token trees (attn_tree.cu) and
// of requests that share a prefix (attn_prefix.cu, kPrefix).
//
// For node i of a request (its q row, head h, keys as tree.cuh says):
//   out = bmm2 * sum_j e^{s_ij - m} V_j / (sum_j e^{s_ij - m} + [sinks] e^{sink_h - m}),
// s_ij = bmm1 <q_i, K_j> over the keys node i sees, 0 where it sees none.
//
// What bounds it.  A tree has few rows (nodes x G per kv head) against a long
// context, so K and V are read once for all of them: up to about 280 rows per
// kv head the time is that of the K/V stream from HBM, beyond that of the
// tensor cores and the exponentials.  Measured: 32 requests of 512 to 8192 keys,
// 9 to 16 nodes x 4 heads, D = 128: 102 us, 5.7 TB/s (0.85 of the copy rate);
// the same with e4m3, up to 16384 keys and 8 nodes: 145 us, 4.5 TB/s (0.67);
// 8 requests of up to 16384 keys, 64 nodes x 8 heads: 105 us, 1000 TFLOP/s (0.51 of
// the bf16 rate; at D = 64 76 us); one request, 8 nodes, 2048 keys: 13.9 us, latency.
//
// Work.  A unit is (request, kv head, up to kTiles query tiles of 128 rows);
// all units' kv tiles of 128 keys, laid end to end, are cut into equal runs,
// one per CTA, one CTA per SM (TreeCut; small units stay whole, tree_snap).  Every CTA finds its run from the
// lengths alone: no list, no counters, nothing that two launches or two graphs
// could share, and equal shares whatever the lengths.  A CTA thus has at most
// two segments that are parts of a unit, the first and the last of its run;
// those leave unnormalised rows with (m, l) in the workspace, which
// tree_merge_kernel puts together in a fixed order.
//
//   warp 0   producer: walks the run, posts each segment's description to the
//            other roles, and loads K/V pages (one TMA box per page and
//            128-byte column block) into a ring of K and V entries.
//   warps 1, 2   issue the MMAs; warp 1 owns TMEM.  Two issuers, since what an
//            MMA waits for takes a few hundred cycles to look at, and one warp
//            that did all of it left the tensor core idle meanwhile (512 rows per
//            kv head: 126 us with one).  kTiles 1: S = Q K^T and O += P V.
//            kTiles 2: a query tile each, in turns; at D = 64 (kPairs) all S and all P V.
//   warp 3   loads Q (a TMA box per softmax warp's tokens and column block), and
//            makes V safe where rows see different keys (see below).
//   warps 4-7, 8-11   softmax A and B: one thread per MMA row.
//   warps 12-15   (e4m3 caches only) split Q into two e4m3 terms and convert V to f16.
//
// kTiles 2 (more than one tile of rows in some request): A and B each have
// their own query tile, and K/V are read once for both.  kTiles 1: there is
// one query tile; A takes the even kv tiles and B the odd ones, of three S
// buffers in turn, into one O.  The running maximum of a row goes from one
// group to the other through shared memory as soon as a tile's own maximum is
// known, so that tensor core, both groups and loads overlap although there is
// a single tile of rows; at the end each group writes half of the columns.
//
// e4m3 caches.  K goes to the tensor core as it is (kind::f8f6f4), and Q is split
// instead: a Q row is scaled by a power of two and split into two e4m3 terms
// whose sum is exact for every element within 2^-9 of the row's largest, and off
// by at most 2^-17 of the largest below; S = Qh K^T + Ql K^T.  P V is done in f16
// (kind::f16), V being converted to f16, exactly, on its way from the ring.  A
// long tail of small probabilities is together as heavy as the row's largest, so
// that P needs its relative precision over a wide range: kept in (0, 2^15] with
// its row's largest at 2^7 or more, it is off by at most half a step of f16
// (2^-11 of itself) down to 2^-21 of the row's largest, and by 2^-32 of the largest
// below.  (P in two e4m3 terms with V as it is took 145 us for that batch when this took 160,
// but its steps end at 2^-14 of the row's largest: of a tail of 16384 keys behind a
// lead of 11 nats 0.84 was lost.)  What bounds this: the ring.  V in f16, two tiles
// of it, leaves room for 128 KB of K and V on their way (96 KB with two query tiles).
// So one Q buffer does.  The converting warps free a V entry when they have the second
// half of its rows in registers, which no longer gains anything over freeing it once all is
// converted (145 us; 143 then), and the roles' code is kept short (158 us unrolled: the
// instruction caches).
//
// bf16 caches.  P is bf16 (off by half a step, 2^-8 of itself, over all of fp32's
// range), since both operands of an MMA have one type and V's range needs bf16.
//
// V and keys that some rows of a tile do not see: their P is 0, but 0 times
// an infinity or NaN is NaN.  Keys before the item's first and past the last
// are zeroed in shared memory; keys that some rows see (tree nodes, a window's
// edge) are looked over, and one that is not finite is zeroed and added to the
// rows that see it in the epilogue, from global memory, in fp32.
//
// TMEM (512 columns).  kTiles 1: S [0,128) [128,256) [256,384), O [384,384+D).
// kTiles 2: S [0,128) [128,256), O [256,256+D) [256+D,256+2D); D = 64: three S, O at
// 384.  P overwrites the first 64 columns of its S.
//
// Every wait is bounded, as in attn_tc.cu.
#pragma once

#include <mutex>

#include "attn_common.cuh"
#include "tree.cuh"

namespace b2pa {

namespace {

constexpr int kTreeSlots = 4;     // posted segments in flight
constexpr int kBadSlots = 16;     // segments whose V was found not to be finite: a bit each

template <int D, bool FP8, int kTiles>
struct TreeCfg {
    static constexpr int kBlockBytes = kQRows * 128;        // 128 rows of one 128-byte column block
    static constexpr int kHalves = FP8 ? 1 : D / 64;        // column blocks of a K/V row
    static constexpr int kQHalves = D / 64;                 // column blocks of a Q row (bf16; e4m3: its two terms)
    static constexpr int kKvBytes = kHalves * kBlockBytes;
    static constexpr int kQBytes = kQHalves * kBlockBytes;
    static constexpr int kQBufs = D == 128 ? 1 : 2;
    static constexpr int kVBufs = FP8 ? 2 : 0;              // V tiles converted to f16
    static constexpr int kVBytes = 2 * kBlockBytes;
    static constexpr int kRing = 224 * 1024 - kQBufs * kTiles * kQBytes - kVBufs * kVBytes;
    // K and V tiles, alternating (e4m3: K in the even entries and V in the odd ones, which have other readers)
    static constexpr int kEntries = FP8 ? kRing / kKvBytes / 2 * 2 : kRing / kKvBytes;
    static constexpr int kOffRing = kQBufs * kTiles * kQBytes;
    static constexpr int kOffV = kOffRing + kEntries * kKvBytes;
    static constexpr int kOffBar = kOffV + kVBufs * kVBytes;
    // two query tiles, and TMEM has room for a third S (see tree_s_pairs)
    static constexpr bool kPairs = kTiles == 2 && D == 64;
    static constexpr int kSBufs = kTiles == 1 || kPairs ? 3 : 2;
    static constexpr int kNumBars = 3 * kEntries + 3 * kQBufs + 3 * kSBufs + 2 + 8 + 2 + 2 + 2 * kTreeSlots + 1 + 2 * kVBufs;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem address, abort flag
    static constexpr int kOffItems = kOffMisc + 16;
    static constexpr int kOffBad = kOffItems + kTreeSlots * 12 * 4;
    static constexpr int kOffExp = kOffBad + 4;  // e4m3: exponent of each Q row (int8)
    static constexpr int kOffMl = (kOffExp + (FP8 ? kQBufs * kTiles * kQRows : 0) + 15) / 16 * 16;
    static constexpr int kSmemBytes = kOffMl + (kTiles == 1 ? 2 * kQRows * 8 : 0);  // ml; its first half: the running maxima
    static constexpr int kThreads = FP8 ? 512 : 384;
    // reads of a posted segment: warps 1 and 2, twice by warp 3, the softmax and the converting warps
    static constexpr int kConsumers = FP8 ? 16 : 12;
    static constexpr int kTmemCols = 512;
    static constexpr int kOCol = kSBufs * kKvTile;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(!FP8 || D == 128, "e4m3 caches: D = 128");
    static_assert(kEntries >= 5 && kEntries <= 32, "ring");
    static_assert(kSmemBytes <= 232448, "shared memory");
};

struct TreeCtx : Ctx {
    uint64_t *kv_full, *kv_empty, *v_ready;  // [kEntries]
    uint64_t *q_full, *q_empty, *q_conv;     // [kQBufs]
    uint64_t *s_full, *p_full, *s_free;      // [kSBufs]: S there, P there, P V done
    uint64_t *o_full;                        // [2] (kTiles 1: [0])
    // kTiles 1: a warp's rows' maxima up to an even / odd tile posted ([2][4]);
    // both groups posted (m, l); both have read O
    uint64_t *m_ready, *met, *left;
    uint64_t* turn;                          // kTiles 2, [2]: this tile's MMAs next (m_ready's place)
    uint64_t* s_pair;                        // kPairs, [2][3] (there too): query tile t's S, in turn
    uint64_t *v_full, *v_empty;              // [kVBufs]: V in f16 there, its P V done
    uint64_t *drain /* [2] */, *it_full, *it_empty, *never;
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
    // the same of the segment's i-th: i < mixed0 or i >= mixed1
    __device__ __forceinline__ int mixed0(int window) const { return (lo_all(window) + kKvTile - 1) / kKvTile - j0; }
    __device__ __forceinline__ int mixed1() const { return ctx() / kKvTile - j0; }
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

// Which prefixes a CTA works on: all, those of more tokens than a query tile has, the others.
enum TreeOnly { kAll, kMore, kOneTileOnly };

// ---------------------------------------------------------------------------
// warp 0
// ---------------------------------------------------------------------------
template <typename C, int kTiles, bool kPrefix, TreeOnly kOnly>
__device__ void tree_producer(const TreeParams& p, const TreeCtx& c, long long pos, long long end, int b, long long base)
{
    const int lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(c.base + C::kOffRing);
    const int P = p.page_size, log2_p = 31 - __clz(P);  // the tensor-core path takes powers of two only
    const int box_rows = P >= kKvTile ? kKvTile : P;
    const int item_toks = kTiles * p.rows.tile_toks;
    uint32_t q = 0;  // ring entries filled
    bool ok = true;
    auto request = [&](int v) {
        TreeReq r = request_of<kPrefix>(p, v, item_toks);
        if (kOnly != kAll && v < p.prefix.groups && (r.n > p.rows.tile_toks) != (kOnly == kMore))
            r.items = 0;
        return r;
    };
    TreeReq r = pos < end ? request(b) : TreeReq{};
    int4* note = p.part_seg + (long long)blockIdx.x * 4;  // of slots 0 and 1
    if (!kPrefix && lane < 2 && !p.whole)
        TreePart{}.write(note + 2 * lane);
    __syncwarp();
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % kTreeSlots;
        if (!wait_bar(&c.it_empty[slot], ((n / kTreeSlots) & 1) ^ 1, c))
            break;
        Seg s{};
        while (pos < end && !s.on) {
            while (pos - base >= r.work(p.Hkv) && b + 1 < requests_of<kPrefix>(p)) {
                base += r.work(p.Hkv);
                r = request(++b);
            }
            const long long unit = (pos - base) / r.unit;
            const long long u0 = base + unit * r.unit;
            const int cost = kPrefix ? r.unit - r.tiles : kTreeUnitCost;
            const int off = max(0, (int)(pos - u0) - cost);
            const int to = max(0, (int)min((long long)r.unit, end - u0) - cost);
            pos = min(end, u0 + r.unit);
            if (to <= off)
                continue;  // none of its tiles
            const int it = (int)(unit % r.items);
            s.on = 1;
            s.kvh = (int)(unit / r.items);
            s.q0 = r.q0;
            s.n = r.n;
            s.kv_len = r.kv_len;
            s.tok0 = it * item_toks;
            s.toks = min(item_toks, r.n - s.tok0);
            s.j0 = r.n_lo + off;
            s.tiles = to - off;
            s.whole = s.tiles == r.tiles;
            s.slot = n == 0 ? 0 : 1;
            if constexpr (kPrefix) {
                s.n = r.kv_len - r.ctx;
                s.slot = off > 0 ? kPrefixCut : b < p.prefix.groups ? kPrefixShared : kPrefixOwn;
                if (off > 0 && lane == 0)
                    p.prefix.cut_ends[blockIdx.x] = off + s.tiles >= r.tiles;
            } else if (!s.whole && lane == 0)
                TreePart{r.tiles, off, s.tiles, s.q0 + s.tok0, s.toks, s.kvh}.write(note + 2 * s.slot);
        }
        if (lane == 0) {
            post_seg(c.item_slot + slot * 12, s);
            mbar_arrive(&c.it_full[slot]);
        }
        __syncwarp();
        if (!s.on)
            break;
        const int* row = kPrefix ? prefix_pages(p, b) : p.block_tables + (long long)b * p.bt_stride;
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
// warps 1 and 2.  The whole warp waits and runs the issue code; MMAs and
// commits are predicated on lane 0.
// ---------------------------------------------------------------------------
// f32 accumulators; bf16 operands (format 1 of kind::f16), or those of an e4m3 cache: e4m3 for
// S (format 0 of kind::f8f6f4) and f16 for O (format 0 of kind::f16); b_mn: B is MN-major (V).
__device__ __forceinline__ constexpr uint32_t tree_idesc(bool fp8, int n, bool b_mn)
{
    const uint32_t fmt = fp8 ? 0u : 1u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kQRows >> 4) << 24);
}
constexpr uint32_t kTreeDescHi = sdesc_hi_sw128(1024);  // 8 rows x 128 B per core group

// The issuers share their schedulers (and instruction caches) with two softmax
// warps each, so that every instruction of theirs costs tens of cycles: their
// loops step through ring and buffers by adding, keep barrier addresses, and
// leave the waits that take long to a call.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* err,
                                       unsigned long long limit)
{
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        const bool timed_out = global_ns() - t0 > limit;
        if (__any_sync(0xffffffffu, *abort_flag != 0 || timed_out)) {
            if (timed_out && (threadIdx.x & 31) == 0) {
                *abort_flag = 1;
                atomicOr(err, (unsigned)B2PA_DEV_TIMEOUT);
            }
            __syncwarp();
            return false;
        }
    }
    return true;
}

// wait_bar for a barrier given by its address.
__device__ __forceinline__ bool wait_at(uint32_t bar, uint32_t parity, const TreeCtx& c)
{
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, c.abort_flag, c.err, c.wait_limit_ns);
}

// The K (kind 0) or V (1) entries of the ring, in the order of the kv tiles:
// tile g's are entries 2 g and 2 g + 1.
template <int kEntries>
struct RingPos {
    uint32_t e, phase;
    __device__ __forceinline__ explicit RingPos(uint32_t kind) : e(kind), phase(0) {}
    __device__ __forceinline__ void next()
    {
        e += 2;
        if (e >= kEntries) {
            e -= kEntries;
            phase ^= 1;
        }
    }
};

// The MMAs of one query tile and kv tile.
template <int D, bool FP8, int kTiles>
struct TreeMma {
    using C = TreeCfg<D, FP8, kTiles>;
    static constexpr uint32_t kIdescS = tree_idesc(FP8, kKvTile, false), kIdescO = tree_idesc(FP8, D, true);
    static constexpr uint32_t kEntryW = C::kKvBytes >> 4, kQTileW = C::kQBytes >> 4, kBlockW = C::kBlockBytes >> 4;
    // A step of P V is 8 columns of P, 16 keys (16 rows of V).  Of a request's last
    // tile the steps behind the last key are left out.
    static constexpr int kKeys = 16, kSteps = kKvTile / kKeys;
    static constexpr uint32_t kVEntryW = (FP8 ? C::kVBytes : C::kKvBytes) >> 4;
    uint32_t tmem, q_lo, k_lo, v_lo, issue;
    __device__ __forceinline__ explicit TreeMma(const TreeCtx& c)
        : tmem(c.tmem),
          q_lo(sdesc_lo(smem_u32(c.base), 16)),                           // K-major: LBO unused
          k_lo(sdesc_lo(smem_u32(c.base + C::kOffRing), 16)),
          v_lo(sdesc_lo(smem_u32(c.base + (FP8 ? C::kOffV : C::kOffRing)), C::kBlockBytes)),  // MN-major: LBO = next column block
          issue((threadIdx.x & 31) == 0 ? 1u : 0u)
    {
    }
    // S (buffer s) = Q tile q (of all buffers') times K (ring entry e)
    __device__ __forceinline__ void scores(uint32_t s, uint32_t q, uint32_t e) const
    {
        const uint32_t a0 = q_lo + q * kQTileW, b0 = k_lo + e * kEntryW, d = tmem + s * kKvTile;
        // a step is 32 bytes of a row: 32 e4m3 elements or 16 of 16 bits; four
        // steps are a column block (e4m3: of Q's first, then second term)
#pragma unroll
        for (int k = 0; k < (FP8 ? 8 : D / 16); ++k) {
            const uint32_t step = (uint32_t)((k & 3) * 2), block = (uint32_t)(k >> 2) * kBlockW;
            if constexpr (FP8)
                mma8_ss_wp(d, a0 + block + step, b0 + step, kTreeDescHi, kIdescS, k > 0 ? 1u : 0u, issue);
            else
                mma_ss_wp(d, a0 + block + step, b0 + block + step, kTreeDescHi, kIdescS, k > 0 ? 1u : 0u, issue);
        }
    }
    // O (tile t) += P (buffer s) times V (ring entry e, or e4m3: buffer e), of which `keys` are the request's
    __device__ __forceinline__ void values(uint32_t t, uint32_t s, uint32_t e, int keys, bool first) const
    {
        const uint32_t b0 = v_lo + e * kVEntryW, a = tmem + s * kKvTile, d = tmem + (uint32_t)C::kOCol + t * D;
        auto step = [&](int k, uint32_t acc) {
            mma_ts_wp(d, a + (uint32_t)(k * 8), b0 + (uint32_t)(k * kKeys * 8), kTreeDescHi, kIdescO, acc, issue);
        };
        step(0, first ? 0u : 1u);
        if (keys >= kKvTile) {
#pragma unroll
            for (int k = 1; k < kSteps; ++k)
                step(k, 1u);
        } else {
            const int steps = (keys + kKeys - 1) / kKeys;
#pragma unroll 1
            for (int k = 1; k < steps; ++k)
                step(k, 1u);
        }
    }
};

// V of tile i of a segment there, and made safe where not every row sees its keys.
template <typename Ring>
__device__ __forceinline__ bool wait_v(const TreeCtx& c, const Ring& at, bool mixed, uint32_t& ready_bits)
{
    bool ok = wait_at(smem_u32(c.kv_full) + at.e * 8, at.phase, c);
    if (ok && mixed) {
        ok = wait_at(smem_u32(c.v_ready) + at.e * 8, ready_bits >> at.e & 1u, c);
        ready_bits ^= 1u << at.e;
    }
    return ok;
}

// Where P V finds V: a ring entry, or, e4m3, one of two buffers in f16.
template <int kEntries, bool FP8>
struct VPos {
    RingPos<kEntries> ring{1};
    uint32_t buf = 0, phase = 0;
    uint32_t ready_bits = 0;  // parity of each entry's next v_ready phase
    __device__ __forceinline__ uint32_t at() const { return FP8 ? buf : ring.e; }
    __device__ __forceinline__ bool wait(const TreeCtx& c, bool mixed)
    {
        return FP8 ? wait_at(smem_u32(c.v_full) + buf * 8, phase, c) : wait_v(c, ring, mixed, ready_bits);
    }
    // what to arrive on when its MMAs are done
    __device__ __forceinline__ uint32_t done(const TreeCtx& c) const
    {
        return FP8 ? smem_u32(c.v_empty) + buf * 8 : smem_u32(c.kv_empty) + ring.e * 8;
    }
    __device__ __forceinline__ void next()
    {
        if (FP8) {
            phase ^= buf;
            buf ^= 1;
        } else {
            ring.next();
        }
    }
};

// kTiles 1, warp 1: S of every kv tile, three buffers in turn.
template <int D, bool FP8>
__device__ void tree_s(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, 1>;
    const TreeMma<D, FP8, 1> mma(c);
    const uint32_t kv_full = smem_u32(c.kv_full), s_full = smem_u32(c.s_full), s_free = smem_u32(c.s_free);
    RingPos<C::kEntries> at(0);
    uint32_t buf = 0, turn = 0;
    bool ok = !p.inject_stall || wait_bar(c.never, 0, c);  // failure-detection tests
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const uint32_t qb = n % C::kQBufs;
        if (!wait_bar(FP8 ? &c.q_conv[qb] : &c.q_full[qb], (n / C::kQBufs) & 1, c))
            break;
        for (int i = s.tiles; i > 0; --i) {
            // K, and the buffer's last P used
            ok = wait_at(kv_full + at.e * 8, at.phase, c) && wait_at(s_free + buf * 8, turn ^ 1, c);
            if (!ok)
                break;
            tc_fence_after();
            mma.scores(buf, qb, at.e);
            mma_commit_at(s_full + buf * 8, mma.issue);  // (the softmax group releases K)
            at.next();
            if (++buf == 3) {
                buf = 0;
                turn ^= 1;
            }
        }
        if (ok)
            mma_commit_p(&c.q_empty[qb], mma.issue);
    }
    // every MMA this thread issued has completed once the drain barrier flips
    if (mma.issue)
        mma_commit(&c.drain[0]);
    __syncwarp();
    drain_wait(&c.drain[0], 0);
}

// kTiles 1, warp 2: O += P V.
template <int D, bool FP8>
__device__ void tree_pv(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, 1>;
    const TreeMma<D, FP8, 1> mma(c);
    const uint32_t p_full = smem_u32(c.p_full), s_free = smem_u32(c.s_free);
    VPos<C::kEntries, FP8> at;
    uint32_t buf = 0, turn = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const int mixed0 = s.mixed0(p.window), mixed1 = s.mixed1();
        for (int i = 0; i < s.tiles; ++i) {
            ok = at.wait(c, i < mixed0 || i >= mixed1) && wait_at(p_full + buf * 8, turn, c);
            if (!ok)
                break;
            tc_fence_after();
            mma.values(0, buf, at.at(), s.kv_len - (s.j0 + i) * kKvTile, i == 0);
            mma_commit_at(s_free + buf * 8, mma.issue);
            mma_commit_at(at.done(c), mma.issue);
            at.next();
            if (++buf == 3) {
                buf = 0;
                turn ^= 1;
            }
        }
        if (ok)
            mma_commit_p(&c.o_full[0], mma.issue);
    }
    if (mma.issue)
        mma_commit(&c.drain[1]);
    __syncwarp();
    drain_wait(&c.drain[1], 0);
}

// kTiles 2, warps 1 and 2: all MMAs of a query tile each.  P V of a kv tile and
// right behind it S of the next one into the same buffer, which is in order for
// it is one thread's, with no wait between them.  The two warps take turns, so
// that one tile's MMAs run, undivided, during the other's softmax; left alone
// they fall into step, and tensor core and softmax wait for one another (wide
// trees of 512 rows: 111 us in turns, 127 without, 118 with all S from one warp
// and all P V from the other).
template <int D, bool FP8>
__device__ void tree_tile(const TreeParams& p, const TreeCtx& c, int t)
{
    using C = TreeCfg<D, FP8, 2>;
    const TreeMma<D, FP8, 2> mma(c);
    const uint32_t kv_full = smem_u32(c.kv_full), kv_empty = smem_u32(c.kv_empty);
    const uint32_t p_full = smem_u32(c.p_full) + t * 8, s_full = smem_u32(c.s_full) + t * 8;
    const uint32_t my_turn = smem_u32(c.turn) + t * 8, your_turn = smem_u32(c.turn) + (t ^ 1) * 8;
    RingPos<C::kEntries> at_k(0);
    VPos<C::kEntries, FP8> at_v;
    uint32_t p_phase = 0, turn_phase = t ^ 1;  // (tile 0 goes first)
    bool ok = t != 0 || !p.inject_stall || wait_bar(c.never, 0, c);  // failure-detection tests
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const uint32_t qb = n % C::kQBufs;
        // (a segment of one query tile: the other's warp only passes the ring on)
        const bool two = s.toks > p.rows.tile_toks, mine = two || t == 0;
        const int mixed0 = s.mixed0(p.window), mixed1 = s.mixed1();
        ok = wait_bar(FP8 ? &c.q_conv[qb] : &c.q_full[qb], (n / C::kQBufs) & 1, c);
        for (int i = -1; i < s.tiles; ++i) {  // P V of tile i, S of tile i + 1
            const bool pv = i >= 0, sc = i + 1 < s.tiles;
            if (pv) {
                ok = ok && at_v.wait(c, i < mixed0 || i >= mixed1);
                if (mine) {
                    ok = ok && wait_at(p_full, p_phase, c);
                    p_phase ^= 1;
                }
            }
            if (sc)
                ok = ok && wait_at(kv_full + at_k.e * 8, at_k.phase, c);
            if (two) {
                ok = ok && wait_at(my_turn, turn_phase, c);
                turn_phase ^= 1;
            }
            if (!ok)
                break;
            tc_fence_after();
            if (mine && pv)
                mma.values(t, t, at_v.at(), s.kv_len - (s.j0 + i) * kKvTile, i == 0);
            if (mine && sc)
                mma.scores(t, qb * 2 + t, at_k.e);
            // before the commit, which waits for room among the MMAs
            mbar_arrive_at(your_turn, two ? mma.issue : 0u);
            if (mine && sc)
                mma_commit_at(s_full, mma.issue);
            // K and V are released by the softmax group, which hears of it all the same
            if (pv) {
                mbar_arrive_at(at_v.done(c), mine ? 0u : mma.issue);
                at_v.next();
            }
            if (sc) {
                mbar_arrive_at(kv_empty + at_k.e * 8, mine ? 0u : mma.issue);
                at_k.next();
            }
        }
        if (ok) {
            if (mine)
                mma_commit_p(&c.o_full[t], mma.issue);
            mma_commit_p(&c.q_empty[qb], mma.issue);
        }
    }
    if (mma.issue)
        mma_commit(&c.drain[t]);
    __syncwarp();
    drain_wait(&c.drain[t], 0);
}

// kPairs (kTiles 2, D = 64), warp 1: S of every (kv tile, query tile), the query tiles in
// turn, into three buffers in turn.  With one buffer more than query tiles a tile's next
// S is computed while its P V waits for P, so that a softmax group finds it when it is
// done with the last: the chain S - softmax - P V of a tile loses its first part.  8 trees
// of 64 nodes x 8 heads: 76 us, 89 with two buffers in turns as above; 16 questions of 16 to 64
// tokens behind 32768 keys 194 us, 222 with two, 254 with a warp for each query tile here
// too.  Now P V's issuer is the slowest: 8 MMAs are issued in 620 cycles of the 1150 that a
// (kv tile, query tile) takes, and a softmax group, busy for 1250 of 2300, waits for S.
template <int D, bool FP8>
__device__ void tree_s_pairs(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, 2>;
    const TreeMma<D, FP8, 2> mma(c);
    const uint32_t kv_full = smem_u32(c.kv_full), kv_empty = smem_u32(c.kv_empty);
    const uint32_t s_pair = smem_u32(c.s_pair), s_free = smem_u32(c.s_free);
    RingPos<C::kEntries> at(0);
    uint32_t buf = 0, turn = 0;
    uint32_t at0 = s_pair, at1 = s_pair + 24;  // the query tiles' next barriers
    bool ok = !p.inject_stall || wait_bar(c.never, 0, c);  // failure-detection tests
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const uint32_t qb = n % C::kQBufs;
        const int tiles = s.toks > p.rows.tile_toks ? 2 : 1;
        if (!wait_bar(&c.q_full[qb], (n / C::kQBufs) & 1, c))
            break;
        for (int i = s.tiles; ok && i > 0; --i) {
            ok = wait_at(kv_full + at.e * 8, at.phase, c);
            for (int t = 0; ok && t < tiles; ++t) {
                if (!(ok = wait_at(s_free + buf * 8, turn ^ 1, c)))  // the buffer's last P used
                    break;
                tc_fence_after();
                mma.scores(buf, qb * 2 + t, at.e);
                mma_commit_at(t == 0 ? at0 : at1, mma.issue);
                if (t == 0)
                    at0 = at0 == s_pair + 16 ? s_pair : at0 + 8;
                else
                    at1 = at1 == s_pair + 40 ? s_pair + 24 : at1 + 8;
                if (++buf == 3) {
                    buf = 0;
                    turn ^= 1;
                }
            }
            if (ok)
                mma_commit_at(kv_empty + at.e * 8, mma.issue);
            at.next();
        }
        if (ok)
            mma_commit_p(&c.q_empty[qb], mma.issue);
    }
    // every MMA this thread issued has completed once the drain barrier flips
    if (mma.issue)
        mma_commit(&c.drain[0]);
    __syncwarp();
    drain_wait(&c.drain[0], 0);
}

// kPairs, warp 2: O += P V, in the same order.
template <int D, bool FP8>
__device__ void tree_pv_pairs(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, 2>;
    const TreeMma<D, FP8, 2> mma(c);
    const uint32_t p_full = smem_u32(c.p_full), s_free = smem_u32(c.s_free);
    VPos<C::kEntries, FP8> at;
    uint32_t buf = 0, turn = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const int tiles = s.toks > p.rows.tile_toks ? 2 : 1;
        const int mixed0 = s.mixed0(p.window), mixed1 = s.mixed1();
        for (int i = 0; ok && i < s.tiles; ++i) {
            ok = at.wait(c, i < mixed0 || i >= mixed1);
            for (int t = 0; ok && t < tiles; ++t) {
                if (!(ok = wait_at(p_full + buf * 8, turn, c)))
                    break;
                tc_fence_after();
                mma.values(t, buf, at.at(), s.kv_len - (s.j0 + i) * kKvTile, i == 0);
                mma_commit_at(s_free + buf * 8, mma.issue);
                if (++buf == 3) {
                    buf = 0;
                    turn ^= 1;
                }
            }
            if (ok)
                mma_commit_at(at.done(c), mma.issue);
            at.next();
        }
        for (int t = 0; ok && t < tiles; ++t)
            mma_commit_p(&c.o_full[t], mma.issue);
    }
    if (mma.issue)
        mma_commit(&c.drain[1]);
    __syncwarp();
    drain_wait(&c.drain[1], 0);
}

// ---------------------------------------------------------------------------
// warp 3: Q, and V of tiles with keys that not every row sees
// ---------------------------------------------------------------------------
// Two e4m3 codes -> two floats.
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

// Two values |v| < 2^8, given as v 2^-8, into two e4m3 terms each: the codes
// are the high bytes of the halves of `hi` and `lo`.  In f16, v 2^-8 has e4m3's
// exponent field, subnormals included (2^-14 against 2^-6), so that a code is
// the top of the f16 bits: the leading term by cutting, its remainder (exact in
// f16) by rounding half up.
__device__ __forceinline__ void split_e4m3(float2 v, uint32_t& hi, uint32_t& lo)
{
    uint32_t f, r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f) : "f"(v.y), "f"(v.x));
    const uint32_t sign = f & 0x80008000u, mag = f & 0x7FFF7FFFu;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(mag), "r"(mag & 0x7F807F80u));
    hi = mag << 1 | sign;
    lo = r * 2u + 0x00800080u | sign;
}

// `count` Q rows of 128 bf16 values from row0 (a multiple of 16; at most 16) in
// shared memory (two column blocks of 128 bytes, 16-byte chunks swizzled by row
// % 8) become their two e4m3 terms, in place: the high one in the first block,
// the low one in the second.  exps[row] is the power of two a row was scaled
// by, which brings its largest value to [2^7, 2^8).  A row that is not finite
// becomes NaN, which is what every score of it makes of the softmax.
__device__ __forceinline__ void split_q_rows(uint8_t* tile, int block_bytes, int row0, int count, int8_t* exps)
{
    const int lane = threadIdx.x & 31;
    // a row's maximum by two lanes, a block each
    uint32_t m = 0;
    if ((lane & 15) < count) {
        const uint8_t* row = tile + (row0 + (lane & 15)) * 128 + (lane >> 4) * block_bytes;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + ((k ^ (lane & 7)) << 4));
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                     __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
        }
    }
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 16));
    m = max(m & 0xFFFFu, m >> 16);
    const int mine = m == 0 || m >= 0x7F80u ? 0 : min(120, max(-110, 7 - ((int)(m >> 7) - 127)));
    if (lane < count)
        exps[row0 + lane] = (int8_t)mine;
    __syncwarp();
    // two rows at a time, eight elements per lane (not unrolled, nor the two halves of a
    // row of V below: the roles' code competes for the instruction caches; the e4m3 batch
    // 146 us, 158 with both unrolled)
    const int c = lane & 15;
#pragma unroll 1
    for (int k = 0; k < count; k += 2) {
        const int r = k + (lane >> 4), sw = r & 7;
        const bool on = r < count;
        const int e = __shfl_sync(0xffffffffu, mine, r & 15);
        const bool nan = __shfl_sync(0xffffffffu, m, r & 15) >= 0x7F80u;
        const float sc = __int_as_float((127 - 8 + e) << 23);
        uint8_t* row = tile + (row0 + (on ? r : k)) * 128;
        const uint4 x = *reinterpret_cast<const uint4*>(row + (c >> 3) * block_bytes + (((c & 7) ^ sw) << 4));
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            split_e4m3(make_float2(__uint_as_float(u[i] << 16) * sc, __uint_as_float(u[i] & 0xFFFF0000u) * sc), hi[i], lo[i]);
        __syncwarp();  // the whole row is read
        if (on) {
            uint8_t* to = row + (((c >> 1) ^ sw) << 4) + (c & 1) * 8;
            const uint2 h = make_uint2(__byte_perm(hi[0], hi[1], 0x7531), __byte_perm(hi[2], hi[3], 0x7531));
            *reinterpret_cast<uint2*>(to) = nan ? make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu) : h;
            *reinterpret_cast<uint2*>(to + block_bytes) =
                make_uint2(__byte_perm(lo[0], lo[1], 0x7531), __byte_perm(lo[2], lo[3], 0x7531));
        }
    }
    __syncwarp();
}

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

// The Q tiles of a segment, into buffer qb.
template <int D, bool FP8, int kTiles>
__device__ __forceinline__ void load_q(const TreeParams& p, const TreeCtx& c, const Seg& s, uint32_t qb)
{
    using C = TreeCfg<D, FP8, kTiles>;
    const int lane = threadIdx.x & 31;
    const TreeRows& r = p.rows;
    // lane = (tile, warp's tokens, column block): one box each
    const int t = lane / (4 * C::kQHalves), w = lane / C::kQHalves % 4, h = lane % C::kQHalves;
    const int toks = t < kTiles ? tile_tokens(r, s, t) : 0;
    const int per = r.by_warp ? (toks + 3) / 4 : r.tile_toks;
    const int first = w * per;  // this warp's first token
    const bool box = toks > 0 && first < toks && (r.by_warp || w == 0);
    const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
    mbar_arrive_expect_tx_p(&c.q_full[qb], boxes * (uint32_t)(r.G * r.box_toks * 128), lane == 0 ? 1u : 0u);
    __syncwarp();
    if (box)
        tma_load_3d(smem_u32(c.base) + (qb * kTiles + t) * C::kQBytes + h * C::kBlockBytes + w * 32 * 128, &p.tm_q,
                    &c.q_full[qb], h * 64, s.kvh * r.G, s.q0 + s.tok0 + t * r.tile_toks + first);
    __syncwarp();
}

// V entry e, kv tile j of segment s (its n-th): keys that no row sees become
// 0, and so do keys that some rows may not see and that are not finite.
template <int D, bool FP8, int kTiles>
__device__ __noinline__ void safe_v(const TreeParams& p, const TreeCtx& c, const Seg& s, uint32_t n, int j, uint32_t e)
{
    using C = TreeCfg<D, FP8, kTiles>;
    constexpr int kChunks = 8 * C::kHalves;  // 16-byte pieces of a V row
    constexpr int kRowsAtOnce = 32 / kChunks;
    const int lane = threadIdx.x & 31;
    const int sub = lane / kChunks, chunk = lane % kChunks;
    volatile int* bad = reinterpret_cast<volatile int*>(c.base + C::kOffBad);
    const int lo = s.lo(p.window), lo_all = s.lo_all(p.window), ctx = s.ctx();
    uint8_t* v = c.base + C::kOffRing + e * C::kKvBytes + (chunk >> 3) * C::kBlockBytes + (chunk & 7) * 16;
    const int k0 = j * kKvTile;
    auto at = [&](int row) { return reinterpret_cast<uint4*>(v + row * 128); };
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // rows that no row of Q sees (they may never have been loaded)
    constexpr int kStep = 16;  // keys of an MMA: the steps after the last key are not issued
    const int seen0 = min(max(lo - k0, 0), kKvTile), seen1 = min(s.kv_len - k0, kKvTile);
    for (int row = sub; row < seen0; row += kRowsAtOnce)
        *at(row) = zero;
    for (int row = seen1 + sub; row < (seen1 + kStep - 1) / kStep * kStep; row += kRowsAtOnce)
        *at(row) = zero;
    // rows that some may not see: before the last window's edge, and the nodes
    auto look = [&](int r0, int r1) {
        constexpr int kBatch = 4;  // loads in flight
        for (int r = r0; r < r1; r += kBatch * kRowsAtOnce) {
            uint32_t hit = 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int row = r + k * kRowsAtOnce + sub;
                if (row < r1 && not_finite<FP8>(*at(row)))
                    hit |= 1u << k;
            }
            if (!__any_sync(0xffffffffu, hit != 0))
                continue;
            if (lane == 0)
                *bad = *bad | 1 << n % kBadSlots;
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t m = __ballot_sync(0xffffffffu, hit >> k & 1u);
                if (m >> (sub * kChunks) & ((1u << kChunks) - 1u))
                    *at(r + k * kRowsAtOnce + sub) = zero;
            }
        }
    };
    look(seen0, min(max(lo_all - k0, seen0), seen1));
    look(max(max(ctx, lo_all) - k0, seen0), seen1);
    fence_proxy_async_smem();
    __syncwarp();
}

// Q runs up to a segment (and a buffer) ahead of V; what is possible next is
// done, and this warp waits for neither while the other could go.
template <int D, bool FP8, int kTiles>
__device__ void tree_feed(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<D, FP8, kTiles>;
    const int lane = threadIdx.x & 31;
    volatile int* bad = reinterpret_cast<volatile int*>(c.base + C::kOffBad);
    // (decided for the whole warp, which stays converged)
    auto here = [](uint64_t* bar, uint32_t parity) { return __any_sync(0xffffffffu, mbar_test(bar, parity)) != 0; };
    Seg qs{}, vs{};
    uint32_t qn = 0, vn = 0;  // segments taken
    enum { kNext, kEmpty, kNone } q_at = kNext;  // what Q needs next: a segment, a buffer, nothing more
    uint32_t loads = 0;       // segments whose Q copies were started
    uint32_t q = 0, q_end = 0;  // ring entries seen, and those of the segments taken
    bool v_more = true, ok = true;
    uint64_t idle = 0;  // since when nothing could be done (0: something was)
    while (ok && (q_at != kNone || v_more)) {
        bool did = false;
        if (q_at == kNext && here(&c.it_full[qn % kTreeSlots], (qn / kTreeSlots) & 1)) {
            ok = take_seg(c, qn++, &qs);
            q_at = qs.on ? kEmpty : kNone;
            did = true;
        }
        const uint32_t qb = (qn - 1) % C::kQBufs, ph = ((qn - 1) / C::kQBufs) & 1;
        if (q_at == kEmpty && here(&c.q_empty[qb], ph ^ 1)) {
            load_q<D, FP8, kTiles>(p, c, qs, qb);
            loads = qn;
            q_at = kNext;
            did = true;
        }
        // every ring entry is seen and released in order, so that this warp never
        // lags a barrier by more than one phase
        uint64_t* bar = nullptr;
        uint32_t parity = 0;
        if (v_more && q == q_end) {
            bar = &c.it_full[vn % kTreeSlots];
            parity = (vn / kTreeSlots) & 1;
            if (here(bar, parity)) {
                ok = ok && take_seg(c, vn++, &vs);
                v_more = vs.on != 0;
                q_end += 2 * (uint32_t)vs.tiles;
                if (lane == 0)
                    *bad = *bad & ~(1 << (vn - 1) % kBadSlots);
                __syncwarp();
                did = true;
            }
        } else if (v_more) {
            const uint32_t e = q % C::kEntries;
            bar = &c.kv_full[e];
            parity = (q / C::kEntries) & 1;
            if (here(bar, parity)) {
                const int j = vs.j0 + vs.tiles - (int)((q_end - q + 1) >> 1);
                const bool mixed = (q & 1) && vs.mixed(j, p.window);
                if (mixed)
                    safe_v<D, FP8, kTiles>(p, c, vs, vn - 1, j, e);
                if (lane == 0) {
                    if (mixed)
                        mbar_arrive(&c.v_ready[e]);
                    mbar_arrive(&c.kv_empty[e]);
                }
                __syncwarp();
                ++q;
                did = true;
            }
        }
        if (did) {
            idle = 0;
            continue;
        }
        if (bar != nullptr)
            mbar_try_wait_ns(bar, parity, 100);
        const uint64_t now = global_ns();
        if (idle == 0)
            idle = now;
        const bool timed_out = now - idle > c.wait_limit_ns;
        if (__any_sync(0xffffffffu, *c.abort_flag != 0 || timed_out)) {
            if (timed_out && lane == 0) {
                *c.abort_flag = 1;
                atomicOr(c.err, (unsigned)B2PA_DEV_TIMEOUT);
            }
            ok = false;
        }
    }
    __syncwarp();
    if (*c.abort_flag) {
        const uint32_t first = loads > (uint32_t)C::kQBufs ? loads - C::kQBufs : 0;
        for (uint32_t k = first; k < loads; ++k)
            drain_wait(&c.q_full[k % C::kQBufs], (k / C::kQBufs) & 1);
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

// The scores of the keys k0 .. k0 + 127 that a row does not see become -inf, in TMEM.
__device__ __noinline__ void hide_keys(uint32_t s_tmem, const RowView view, int k0, bool valid)
{
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const uint32_t w = valid ? view.sees(k0 + 32 * q) : 0xffffffffu;
        if (__all_sync(0xffffffffu, w == 0xffffffffu))
            continue;
        uint32_t r[32];
        tmem_ld32(s_tmem + (uint32_t)(q * 32), r);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k)
            r[k] = w >> k & 1u ? r[k] : 0xFF800000u;
        uint32_t a[16], b[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            a[k] = r[k];
            b[k] = r[16 + k];
        }
        tmem_st16(s_tmem + (uint32_t)(q * 32), a);
        tmem_st16(s_tmem + (uint32_t)(q * 32 + 16), b);
    }
    tmem_wait_st();
}

template <bool FP8>
__device__ __forceinline__ float kv_elem(const void* base, long long at)
{
    if (FP8)
        return from_e4m3x2(static_cast<const uint8_t*>(base)[at]).x;
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[at] << 16);
}

// Slow path: column d of the V rows that safe_v zeroed because they are not
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

// ---------------------------------------------------------------------------
// warps 12-15 (e4m3 caches): a segment's Q into its two e4m3 terms, then its V,
// tile by tile, into f16; one thread per row of V
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

template <int kTiles>
__device__ void tree_convert(const TreeParams& p, const TreeCtx& c)
{
    using C = TreeCfg<128, true, kTiles>;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, row = wq * 32 + lane, sw = row & 7;
    const uint32_t lane0 = lane == 0 ? 1u : 0u;
    RingPos<C::kEntries> at(1);
    uint32_t buf = 0, phase = 1;
    uint32_t ready_bits = 0;  // parity of each entry's next v_ready phase
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            break;
        const uint32_t qb = n % C::kQBufs;
        if (!wait_bar(&c.q_full[qb], (n / C::kQBufs) & 1, c))
            break;
        // this warp's quadrant of the tiles, 16 rows at a time
#pragma unroll 1
        for (int k = 0; k < 2 * kTiles; ++k) {
            const int t = k >> 1, r0 = (k & 1) * 16, toks = tile_tokens(p.rows, s, t);
            const int per = (toks + 3) / 4;  // tokens of a quadrant
            const int count = toks <= 0             ? 0
                              : !p.rows.by_warp     ? min(32, p.rows.G * toks - wq * 32)
                              : wq * per < toks ? p.rows.G * per
                                                    : 0;
            if (count > r0)
                split_q_rows(c.base + (qb * kTiles + t) * C::kQBytes, C::kBlockBytes, wq * 32 + r0, min(16, count - r0),
                             reinterpret_cast<int8_t*>(c.base + C::kOffExp) + (qb * kTiles + t) * kQRows);
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_p(&c.q_conv[qb], lane0);
        const int mixed0 = s.mixed0(p.window), mixed1 = s.mixed1();
        for (int i = 0; i < s.tiles; ++i) {
            ok = wait_bar(&c.kv_full[at.e], at.phase, c);
            if (ok && (i < mixed0 || i >= mixed1)) {
                ok = wait_bar(&c.v_ready[at.e], ready_bits >> at.e & 1u, c);
                ready_bits ^= 1u << at.e;
            }
            if (!ok)
                break;
            const uint8_t* from = c.base + C::kOffRing + at.e * C::kKvBytes + row * 128;
            uint8_t* to = c.base + C::kOffV + buf * C::kVBytes + row * 128;
            if (!(ok = wait_bar(&c.v_empty[buf], phase, c)))
                break;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                uint4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = ld_shared_v4(smem_u32(from) + (((4 * h + k) ^ sw) << 4));
                if (h == 1) {
                    fence_proxy_async_smem();  // the loads are done before the entry's next copy
                    __syncwarp();
                    mbar_arrive_p(&c.kv_empty[at.e], lane0);
                }
                uint8_t* block = to + h * C::kBlockBytes;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ch = 2 * k;
                    *reinterpret_cast<uint4*>(block + ((ch ^ sw) << 4)) =
                        make_uint4(f16x2_of_e4m3x2(x[k].x), f16x2_of_e4m3x2(x[k].x >> 16), f16x2_of_e4m3x2(x[k].y),
                                   f16x2_of_e4m3x2(x[k].y >> 16));
                    *reinterpret_cast<uint4*>(block + (((ch + 1) ^ sw) << 4)) =
                        make_uint4(f16x2_of_e4m3x2(x[k].z), f16x2_of_e4m3x2(x[k].z >> 16), f16x2_of_e4m3x2(x[k].w),
                                   f16x2_of_e4m3x2(x[k].w >> 16));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_p(&c.v_full[buf], lane0);
            at.next();
            phase ^= buf;
            buf ^= 1;
        }
    }
}

// ---------------------------------------------------------------------------
// softmax A (t = 0) and B (t = 1)
// ---------------------------------------------------------------------------
template <int D, bool FP8, int kTiles, bool kPrefix>
__device__ void tree_softmax(const TreeParams& p, const TreeCtx& c, int t)
{
    using C = TreeCfg<D, FP8, kTiles>;
    constexpr float kLog2e = 1.4426950408889634f;
    // P = 2^(x - m + kBias), in f16 over an e4m3 cache: the bias uses its range (see
    // the top).  The stabiliser is renewed once the row's maximum has grown by kSlack.
    constexpr float kBias = FP8 ? 7.f : 0.f, kSlack = 8.f;
    // 32-key steps of the exponentials that are unrolled (see below; an e4m3 cache's kernel has one role
    // more: its batch 157 us with one step, 183 with two, before the roles' code was shortened; 512 rows per kv
    // head 136 with two, 131 with four)
    constexpr int kUnroll = kTiles == 2 ? 4 : FP8 ? 1 : 2;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, row = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t s0_tmem = c.tmem + lane_off;  // + buffer * kKvTile
    const uint32_t o_tmem = c.tmem + lane_off + (uint32_t)(C::kOCol + (kTiles == 1 ? 0 : t * D));
    const TreeRows& rows = p.rows;
    const int G = rows.G;
    volatile float* m_row = reinterpret_cast<volatile float*>(c.base + C::kOffMl) + row;  // kTiles 1: this row's running maximum
    float2* ml = reinterpret_cast<float2*>(c.base + C::kOffMl);
    const volatile int* bad = reinterpret_cast<const volatile int*>(c.base + C::kOffBad);

    // kTiles 2: what tells that the P V of tile g is done
    auto v_done = [&](uint32_t g) { return FP8 ? &c.v_empty[g & 1] : &c.kv_empty[(2 * g + 1) % C::kEntries]; };
    uint32_t g0 = 0;   // kv tiles before this segment
    uint32_t pair0 = 0;  // kPairs: (kv tile, query tile) before this segment
    uint32_t s_cnt = 0, o_cnt = 0;  // kTiles 2: S and O of this group awaited so far
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
        const bool two = kTiles == 2 && s.toks > rows.tile_toks;
        const uint32_t pairs = pair0;
        pair0 += (uint32_t)s.tiles * (two ? 2 : 1);
        if (kTiles == 2 && qt * rows.tile_toks >= s.toks) {
            g0 += (uint32_t)s.tiles;
            continue;
        }
        const int toks = tile_tokens(rows, s, qt);
        const TreeToken mine = tree_token(rows, row, toks);
        const int head = mine.head;
        const bool valid = mine.valid;
        const int tok = s.q0 + s.tok0 + qt * rows.tile_toks + (valid ? mine.tok : 0);
        const bool warp_on = __any_sync(0xffffffffu, valid);
        const float sl2 = p.scale_log2 * q_unscale;
        RowView view;
        view.ctx = s.ctx();
        view.n = s.n;
        view.lo = p.window < 0 ? 0 : tree_row_lo(p.positions[tok], view.ctx, s.kv_len, p.window);
        view.mask = p.mask + (long long)tok * p.mask_stride;
        view.words = p.mask_words;
        if constexpr (kPrefix) {  // all keys before its own, and that
            view.ctx = s.ctx() + (s.n > 0 ? s.tok0 + qt * rows.tile_toks + mine.tok + 1 : 0);
            view.n = view.lo = view.words = 0;
            view.mask = nullptr;
        }

        float m_used = -INFINITY, l = 0.f;
        // kTiles 1: the tiles of this group's parity over all segments
        for (int i = kTiles == 1 ? (int)((t ^ g0) & 1) : 0; i < s.tiles; i += kTiles == 1 ? 2 : 1) {
            const uint32_t g = g0 + (uint32_t)i;
            // kPairs: which S this is, and the one before of this query tile
            const uint32_t pair = pairs + (two ? 2 * (uint32_t)i + (uint32_t)t : (uint32_t)i), last_pair = pair - (two ? 2 : 1);
            const int buf = kTiles == 1 ? (int)(g % 3) : C::kPairs ? (int)(pair % 3) : t;
            const uint32_t s_tmem = s0_tmem + (uint32_t)(buf * kKvTile);
            const int k0 = (s.j0 + i) * kKvTile;
            // rows that are nobody's count as seeing everything; what they compute
            // stays in their row
            const bool mixed = !__all_sync(0xffffffffu, !valid || (k0 >= view.lo && k0 + kKvTile <= view.ctx));
            if (!kPrefix && mixed)  // the mask row, while S is on its way
                asm volatile("prefetch.global.L1 [%0];" ::"l"(view.mask + min(max(k0 - view.ctx, 0) >> 5, view.words - 1)));
            // (kPairs: barriers of this group's own, for it does not follow the other's segments; three,
            // for a segment of one query tile has all three buffers)
            if (!wait_bar(C::kPairs ? &c.s_pair[t * 3 + s_cnt % 3] : &c.s_full[buf],
                          kTiles == 1 ? (g / 3) & 1 : C::kPairs ? (s_cnt / 3) & 1 : s_cnt & 1, c)) {
                ok = false;
                break;
            }
            ++s_cnt;
            if (!C::kPairs && wq == 0) {  // K has been read; kTiles 2: and V of the tile before
                const uint32_t lane0 = lane == 0 ? 1u : 0u;
                mbar_arrive_p(&c.kv_empty[2 * g % C::kEntries], lane0);
                if (kTiles == 2 && i > 0)
                    mbar_arrive_p(v_done(g - 1), lane0);
            }
            if (!warp_on) {  // no row of this warp is anyone's
                if (kTiles == 1)
                    mbar_arrive_p(&c.m_ready[(g & 1) * 4 + wq], lane == 0 ? 1u : 0u);
                mbar_arrive_p(&c.p_full[buf], lane == 0 ? 1u : 0u);
                continue;
            }
            tc_fence_after();
            // Keys that a row does not see become -inf in place.  Then the scores
            // are read twice, once for the maximum and once for the exponentials, 32
            // keys at a time in a loop.  All this keeps the code short: with the 128
            // scores of a row in registers and everything unrolled over them, the
            // roles' code did not fit the instruction caches, and waits for
            // instructions were the largest stall of every kernel here.
            if (mixed)
                hide_keys(s_tmem, view, k0, valid);
            uint32_t ra[32];  // 32 scores; at first of the keys 0 .. 31
            float mx;
            {
                float mq[4];  // maxima of the four loads
#pragma unroll
                for (int q = 3; q >= 0; --q)
                    tmem_ld32_max(s_tmem + (uint32_t)(q * 32), ra, &mq[q]);
                tmem_wait_ld();
                mx = fmax3(fmax3(mq[0], mq[1], mq[2]), mq[3], -INFINITY);
            }
            const float m_tile = mx * sl2;
            // the maximum up to the tile before: the other group's (kTiles 1), which
            // posts it as early as this one does
            float m_old = m_used;
            if (kTiles == 1 && i > 0) {
                if (!wait_bar(&c.m_ready[((g - 1) & 1) * 4 + wq], ((g - 1) >> 1) & 1, c)) {
                    ok = false;
                    break;
                }
                m_old = *m_row;
            }
            const bool need = valid && m_tile > m_old + kSlack;
            const float m_new = need ? m_tile : m_old;
            if (kTiles == 1) {
                *m_row = m_new;
                __syncwarp();
                mbar_arrive_p(&c.m_ready[(g & 1) * 4 + wq], lane == 0 ? 1u : 0u);
            }
            // this group's sum is relative to its own last maximum, O to the last tile's
            if (m_used != m_new)
                l *= ex2_approx(m_used - m_new);
            const float alpha = need ? ex2_approx(m_old - m_new) : 1.f;
            m_used = m_new;
            const float neg = m_used == -INFINITY ? 0.f : kBias - m_used;
            const float2 sc = make_float2(sl2, sl2), ng = make_float2(neg, neg);
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
            const bool rescale = __any_sync(0xffffffffu, need) && i > 0;
#pragma unroll(kUnroll)
            for (int q = 0; q < 4; ++q) {
                // 32 keys' P are 16 columns, over scores already read; the next 32
                // scores are loaded behind their exponentials
                uint32_t rb[32];
                if (q < 3)
                    tmem_ld32(s_tmem + (uint32_t)(q * 32 + 32), rb);
                uint32_t pk[16];
#pragma unroll
                for (int w = 0; w < 16; ++w) {
                    const float2 y =
                        __ffma2_rn(make_float2(__uint_as_float(ra[2 * w]), __uint_as_float(ra[2 * w + 1])), sc, ng);
                    const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                    acc[w & 3] = __fadd2_rn(acc[w & 3], e);
                    if constexpr (FP8)
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[w]) : "f"(e.y), "f"(e.x));
                    else
                        pk[w] = pack_bf16x2(e.x, e.y);
                }
                tmem_st16(s_tmem + (uint32_t)(q * 16), pk);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    ra[k] = rb[k];
            }
            if (rescale) {
                // O holds the sum up to the tile before, whose P V (kTiles 2: it
                // precedes this S) has to be done, and whose successor waits for this P
                if (kTiles == 1 && !wait_bar(&c.s_free[(g - 1) % 3], ((g - 1) / 3) & 1, c)) {
                    ok = false;
                    break;
                }
                if (C::kPairs && !wait_bar(&c.s_free[last_pair % 3], (last_pair / 3) & 1, c)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float2 ff = make_float2(alpha, alpha);
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                    uint32_t o[16];
                    tmem_ld16(o_tmem + (uint32_t)(q * 16), o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), ff);
                        o[k] = __float_as_uint(v.x);
                        o[k + 1] = __float_as_uint(v.y);
                    }
                    tmem_st16(o_tmem + (uint32_t)(q * 16), o);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_p(&c.p_full[buf], lane == 0 ? 1u : 0u);
            const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
            const float2 a = __fadd2_rn(a01, a23);
            l += a.x + a.y;
        }
        g0 += (uint32_t)s.tiles;
        if (!ok)
            break;
        // the last P V of the segment (kTiles 1: one O, one wait per segment)
        if (!wait_bar(&c.o_full[kTiles == 1 ? 0 : t], kTiles == 1 ? n & 1 : o_cnt & 1, c)) {
            ok = false;
            break;
        }
        ++o_cnt;
        if (kTiles == 2 && !C::kPairs && wq == 0)
            mbar_arrive_p(v_done(g0 - 1), lane == 0 ? 1u : 0u);  // (g0: the next segment's)
        if constexpr (kTiles == 1) {
            // both groups' sums, relative to the last tile's maximum (the larger one)
            ml[t * kQRows + row] = make_float2(m_used, l);
            __syncwarp();
            mbar_arrive_p(c.met, lane == 0 ? 1u : 0u);
            if (!wait_bar(c.met, n & 1, c)) {
                ok = false;
                break;
            }
            const float2 x0 = ml[row], x1 = ml[kQRows + row];
            m_used = fmaxf(x0.x, x1.x);
            // (a sum of no keys has weight 0; one that is no number keeps its weight)
            l = (x0.x == m_used || x0.y == 0.f ? x0.y : x0.y * ex2_approx(x0.x - m_used)) +
                (x1.x == m_used || x1.y == 0.f ? x1.y : x1.y * ex2_approx(x1.x - m_used));
        }
        // from here on the stabiliser of l and O is m
        const float m = m_used == -INFINITY ? m_used : m_used - kBias;
        tc_fence_after();
        const int h = s.kvh * G + head;
        float out_scale = 1.f;
        if (!kPrefix && s.whole) {
            float total = l;
            if (p.sinks != nullptr && m != -INFINITY)
                total += ex2_approx(fmaf(p.sinks[valid ? h : 0], kLog2e, -m));
            out_scale = total == 0.f ? 0.f : p.bmm2 / total;
        }
        const int d0 = kTiles == 1 ? t * (D / 2) : 0, d1 = kTiles == 1 ? d0 + D / 2 : D;
        const bool any_bad = *bad >> n % kBadSlots & 1;
        const long long part = (long long)(blockIdx.x * 2 + s.slot) * kTiles + qt;
        uint16_t* orow = p.out + (long long)tok * p.out_st_tok + (long long)h * p.out_st_head;
        // kPrefix: the rows of a tile lie together, without those that are nobody's
        const int tile_rows = toks * G, tile_row = mine.tok * G + head;
        float4* prow = nullptr;
        if constexpr (kPrefix) {
            const long long rows0 = s.slot == kPrefixCut ? (long long)(blockIdx.x * 2 + qt) * kQRows
                                                         : ((long long)s.kvh * p.T + tok) * G + head - tile_row;
            prow = (s.slot == kPrefixCut ? p.prefix.cut_o : p.prefix.part_o[s.slot]) + rows0 * (D / 4) + tile_row;
            if (valid && (kTiles == 2 || t == 0)) {
                float4* rec = s.slot == kPrefixCut ? p.prefix.cut_rec : p.prefix.part_rec[s.slot];
                rec[rows0 + tile_row] = PrefixRow{m, l, s.whole ? -1 : (int)blockIdx.x, tile_rows, tile_row, qt}.pack();
            }
        }
        if (any_bad && warp_on) {
            // values of V that are not finite, for the rows that see them
            int b = 0;
            while (b + 1 < p.B && p.cum_q[b + 1] <= tok)
                ++b;
#pragma unroll 1
            for (int d = d0; d < d1; ++d) {
                float o = __uint_as_float(tmem_ld1(o_tmem + (uint32_t)d));
                tmem_wait_ld();
                if (valid)
                    o += tree_bad_column<FP8>(p, p.block_tables + (long long)b * p.bt_stride, view,
                                              kPrefix ? 0x7FFFFFFF : s.lo_all(p.window),
                                              kPrefix ? max(s.ctx(), s.j0 * kKvTile) : s.j0 * kKvTile,
                                              (s.j0 + s.tiles) * kKvTile, tok, h, s.kvh, p.scale_log2, m, d);
                __syncwarp();
                tmem_st1(o_tmem + (uint32_t)d, __float_as_uint(o));
            }
            tmem_wait_st();
        }
        if (warp_on) {
#pragma unroll 1
            for (int d = d0; d < d1; d += 32) {
                uint32_t o[32];
                tmem_ld32(o_tmem + (uint32_t)d, o);
                tmem_wait_ld();
                if (kPrefix && valid) {
                    float4* to = prow + (long long)(d / 4) * tile_rows;
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        to[v * tile_rows] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                        __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                } else if (valid && s.whole) {
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
                    float4* to = p.part_o + (part * (D / 4) + d / 4) * kQRows + row;
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        to[v * kQRows] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                     __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                }
            }
            if (!kPrefix && valid && !s.whole && (kTiles == 2 || t == 0))
                p.part_ml[part * kQRows + row] = make_float2(m, l);
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
__device__ __forceinline__ void tree_setup(const TreeParams& p, uint8_t* smem, TreeCtx& c)
{
    using C = TreeCfg<D, FP8, kTiles>;
    c.base = smem;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    c.kv_full = bars;
    c.kv_empty = c.kv_full + C::kEntries;
    c.v_ready = c.kv_empty + C::kEntries;
    c.q_full = c.v_ready + C::kEntries;
    c.q_empty = c.q_full + C::kQBufs;
    c.q_conv = c.q_empty + C::kQBufs;
    c.s_full = c.q_conv + C::kQBufs;
    c.p_full = c.s_full + C::kSBufs;
    c.s_free = c.p_full + C::kSBufs;
    c.o_full = c.s_free + C::kSBufs;
    c.m_ready = c.o_full + 2;
    c.turn = c.s_pair = c.m_ready;
    c.met = c.m_ready + 8;
    c.left = c.met + 1;
    c.drain = c.left + 1;
    c.it_full = c.drain + 2;
    c.it_empty = c.it_full + kTreeSlots;
    c.never = c.it_empty + kTreeSlots;
    c.v_full = c.never + 1;
    c.v_empty = c.v_full + C::kVBufs;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    c.abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    c.err = p.err;
    c.wait_limit_ns = p.wait_limit_ns;
    c.item_slot = reinterpret_cast<volatile int*>(smem + C::kOffItems);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int e = 0; e < C::kEntries; ++e) {
            mbar_init(&c.kv_full[e], 1);
            // its MMAs (kTiles 2: two tiles'; V of an e4m3 cache: the converting warps), and warp 3
            mbar_init(&c.kv_empty[e], 1 + (FP8 && (e & 1) ? 4 : C::kPairs ? 1 : kTiles));
            mbar_init(&c.v_ready[e], 1);
        }
        for (int b = 0; b < C::kQBufs; ++b) {
            mbar_init(&c.q_full[b], 1);
            mbar_init(&c.q_empty[b], (FP8 ? 8 : 0) + (C::kPairs ? 1 : kTiles));  // the MMAs that read it; e4m3: and the softmax warps
            mbar_init(&c.q_conv[b], 4);
        }
        for (int k = 0; k < C::kSBufs; ++k) {
            mbar_init(&c.s_full[k], 1);
            mbar_init(&c.p_full[k], 4);
            mbar_init(&c.s_free[k], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&c.o_full[k], 1);
            mbar_init(&c.drain[k], 1);
            if (FP8) {
                mbar_init(&c.v_full[k], 4);
                mbar_init(&c.v_empty[k], kTiles);
            }
        }
        for (int k = 0; k < 8; ++k)
            mbar_init(&c.m_ready[k], 1);
        mbar_init(c.met, 8);
        mbar_init(c.left, 8);
        for (int s = 0; s < kTreeSlots; ++s) {
            mbar_init(&c.it_full[s], 1);
            mbar_init(&c.it_empty[s], C::kConsumers);
        }
        mbar_init(c.never, 1);
        *c.abort_flag = 0;
        *reinterpret_cast<volatile int*>(smem + C::kOffBad) = 0;
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
}

// Where a CTA's run starts and ends, and the request (the sum of work before it)
// in which it starts.
struct TreeRun {
    long long start, end, base;
    int first_b;
};

// One run through all requests.  `scan`: room for 20 sums in shared memory that
// nothing else uses yet.
template <int kThreads, bool kPrefix>
__device__ __forceinline__ TreeRun tree_run(const TreeParams& p, int item_toks, long long* scan)
{
    // Where this CTA's run starts: the first request whose work, with that of the
    // requests before it, passes the run's start.  warp 0 alone needs to know; for
    // more than a request per lane all threads add up.
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_req = requests_of<kPrefix>(p);
    const bool by_all = n_req > 32;  // (of the whole grid)
    auto request = [&](int b) { return request_of<kPrefix>(p, b, item_toks); };
    TreeRun run{};
    long long &start = run.start, &end = run.end, &base = run.base;
    int& first_b = run.first_b;
    if (by_all || warp == 0) {
        const int threads = by_all ? kThreads : 32, share = (n_req + threads - 1) / threads;
        const int b0 = min(n_req, tid * share), b1 = min(n_req, b0 + share);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) {
            const TreeReq r = request(b);
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
        long long total = 0, warps_before = 0;
        if (by_all) {
            if (lane == 31)
                scan[warp] = before;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                warps_before += w < warp ? scan[w] : 0;
                total += scan[w];
            }
        } else {
            total = __shfl_sync(0xffffffffu, before, 31);
        }
        before += warps_before - mine;
        const TreeCut cut = tree_cut(total, gridDim.x);
        const bool works = (int)blockIdx.x < cut.g;
        start = works ? cut.start(blockIdx.x) : 0;
        end = works ? cut.start(blockIdx.x + 1) : 0;
        // the run's ends, moved off units that are not cut, by the threads whose
        // requests they are in
        const bool has_start = start >= before && start < before + mine, has_end = end >= before && end < before + mine;
        if (!by_all) {  // a request per lane
            const TreeReq r = request(min(b0, n_req - 1));
            const long long s0 = has_start ? tree_snap(start, before, r, cut, p.whole) : 0, e0 = has_end ? tree_snap(end, before, r, cut, p.whole) : 0;
            const unsigned ws = __ballot_sync(0xffffffffu, has_start), we = __ballot_sync(0xffffffffu, has_end);
            first_b = ws != 0 ? __ffs(ws) - 1 : 0;
            base = __shfl_sync(0xffffffffu, before, first_b);
            start = __shfl_sync(0xffffffffu, s0, first_b);
            const long long e1 = __shfl_sync(0xffffffffu, e0, we != 0 ? __ffs(we) - 1 : 0);
            end = we != 0 ? e1 : end;  // (none: it is the last)
        } else {
            for (int k = 0; k < 2; ++k) {
                if (!(k ? has_end : has_start))
                    continue;
                const long long x = k ? end : start;
                long long from = before;
                int b = b0;
                TreeReq r = request(b);
                for (; b + 1 < b1 && x >= from + r.work(p.Hkv); r = request(++b))
                    from += r.work(p.Hkv);
                scan[16 + k] = tree_snap(x, from, r, cut, p.whole);
                if (k == 0) {
                    scan[18] = from;
                    scan[19] = b;
                }
            }
            __syncthreads();
            if (works) {
                start = scan[16];
                end = end < total ? scan[17] : end;
                base = scan[18];
                first_b = (int)scan[19];
            }
            fence_proxy_async_smem();  // the ring's next writes come through the async proxy
            __syncthreads();
        }
    }
    return run;
}

template <int D, bool FP8, int kTiles, bool kPrefix, TreeOnly kOnly = kAll>
__device__ __forceinline__ void tree_roles(const TreeParams& p, const TreeCtx& c, const TreeRun& run)
{
    using C = TreeCfg<D, FP8, kTiles>;
    const int warp = threadIdx.x >> 5;
    // 384 threads launch with 168 registers each (104 + 200 + 200 = 504 = 3 x 168), 512 with 128 (96 + 160 +
    // 160 + 96 = 512 = 4 x 128)
    if (warp < 4) {
        regs_dec<FP8 ? 96 : 104>();
        if (warp == 0)
            tree_producer<C, kTiles, kPrefix, kOnly>(p, c, run.start, run.end, run.first_b, run.base);
        else if (warp == 3)
            tree_feed<D, FP8, kTiles>(p, c);
        else if constexpr (C::kPairs)
            warp == 1 ? tree_s_pairs<D, FP8>(p, c) : tree_pv_pairs<D, FP8>(p, c);
        else if constexpr (kTiles == 2)
            tree_tile<D, FP8>(p, c, warp - 1);
        else if (warp == 1)
            tree_s<D, FP8>(p, c);
        else
            tree_pv<D, FP8>(p, c);
    } else if (!FP8 || warp < 12) {
        regs_inc<FP8 ? 160 : 200>();
        tree_softmax<D, FP8, kTiles, kPrefix>(p, c, (warp - 4) >> 2);
    } else if constexpr (FP8) {
        regs_dec<96>();
        tree_convert<kTiles>(p, c);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(c.tmem, C::kTmemCols);
    }
}

template <int D, bool FP8, int kTiles, bool kPrefix>
__global__ void __launch_bounds__(TreeCfg<D, FP8, kTiles>::kThreads, 1) attention_tree_kernel(const __grid_constant__ TreeParams p)
{
    using C = TreeCfg<D, FP8, kTiles>;
    extern __shared__ __align__(1024) uint8_t smem[];
    TreeCtx c;
    tree_setup<D, FP8, kTiles>(p, smem, c);
    pdl_wait();  // inputs may come from the kernel this launch follows
    // (the ring is empty yet)
    const TreeRun run = tree_run<C::kThreads, kPrefix>(p, kTiles * p.rows.tile_toks,
                                                       reinterpret_cast<long long*>(smem + C::kOffRing));
    tree_roles<D, FP8, kTiles, kPrefix>(p, c, run);
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

// Launch a kernel of one CTA per SM; once per device and instantiation it is
// allowed its shared memory (any host thread).
template <auto kern>
cudaError_t launch_per_sm(const TreeParams& p, int threads, int smem, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    static std::once_flag once[64];
    static cudaError_t err[64];
    std::call_once(once[dev], [&] { err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (err[dev] != cudaSuccess)
        return err[dev];
    return launch_pdl(kern, dim3(p.grid), threads, smem, stream, p);
}

template <int D, bool FP8, int kTiles, bool kPrefix>
cudaError_t launch_tree_kernel(const TreeParams& p, cudaStream_t stream)
{
    using C = TreeCfg<D, FP8, kTiles>;
    return launch_per_sm<attention_tree_kernel<D, FP8, kTiles, kPrefix>>(p, C::kThreads, C::kSmemBytes, stream);
}

}  // namespace

}  // namespace b2pa
