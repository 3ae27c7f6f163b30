// attn_few.cuh -- the keys of one request for the few rows of a single token: at
// most 16 heads of a kv head (attn_prefix.cu).
//
// Bound by the stream of K and V from HBM.  The tensor cores of tcgen05 work on 128
// rows whatever there is to do, and the way from scores to values goes through
// TMEM and two hand-overs per kv tile: 3 us and more of it per unit of work, however
// short, which is what a request's own few hundred keys behind a shared prefix
// are.  Here each of eight warps takes 16 keys of every tile of 128 by itself, with
// mma.sync:
//   S^T [16 keys x rows] = K Q^T, Q being in registers;
//   its own running maxima and sums, O^T [D x rows] += V^T P^T, also in registers.
// Nothing is handed over between these warps.  At the end of a unit they leave
// their rows in shared memory and go on; two others put them together and write
// them out.  (Putting them together themselves, and fetching the next unit's Q, took
// 4000 cycles of a unit, five times the 750 that they work on a kv tile.)  All rows see
// all keys, so that there is no mask but the end.
//
//   warp 0      producer (as in attn_tree.cuh)
//   warp 1      a segment's Q, converted, in the order of the operand's registers
//   warps 2, 3  put the rows together
//   warps 4-11  compute
//
// e4m3 caches: K and V become f16 in registers, exactly; a Q row is scaled by a
// power of two so that f16 holds it exactly, as in attn_tc.cu; P is f16 with the bias of
// attn_tree.cuh.
#pragma once

#include "attn_tree.cuh"

namespace b2pa {

namespace {

constexpr int kFewWarps = 8;   // that compute
constexpr int kFewMerge = 2;   // that put their rows together

// kSets: rows, in sets of eight
template <int D, bool FP8, int kSets>
struct FewCfg {
    static constexpr int kBlockBytes = kQRows * 128;
    static constexpr int kHalves = FP8 ? 1 : D / 64;
    static constexpr int kKvBytes = kHalves * kBlockBytes;
    static constexpr int kEntries = (FP8 ? 160 : 192) * 1024 / kKvBytes;  // K and V tiles, alternating
    static constexpr int kRows = 8 * kSets;
    static constexpr int kCols = kSets == 1 ? D : 32;  // columns put together at once
    static constexpr int kOffRing = 0;
    static constexpr int kOffSum = kEntries * kKvBytes;                     // [warp][row][column] fp32
    static constexpr int kOffMl = kOffSum + kFewWarps * kRows * kCols * 4;  // [warp][row] (m, l)
    static constexpr int kOffQ = kOffMl + kFewWarps * kRows * 8;            // [set][step][half][lane]
    static constexpr int kOffScale = kOffQ + kSets * (D / 16) * 2 * 32 * 4; // [row]: power of two to take off its scores
    static constexpr int kOffBar = kOffScale + kRows * 4;
    static constexpr int kNumBars = 2 * kEntries + 2 * kTreeSlots + 5;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // abort flag
    static constexpr int kOffItems = kOffMisc + 16;
    static constexpr int kSmemBytes = kOffItems + kTreeSlots * 12 * 4;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(!FP8 || D == 128, "e4m3 caches: D = 128");
    static_assert(kSmemBytes <= 232448, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x)  // of an 8 x 8 matrix of 16-bit values
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// c [16 x 8] += a [16 x 16] b [16 x 8]: bf16, or f16 over an e4m3 cache
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1)
{
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, bool FP8, int kSets>
__device__ __forceinline__ void few_setup(const TreeParams& p, uint8_t* smem, TreeCtx& c)
{
    using C = FewCfg<D, FP8, kSets>;
    c.base = smem;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    c.kv_full = bars;
    c.kv_empty = c.kv_full + C::kEntries;
    c.it_full = c.kv_empty + C::kEntries;
    c.it_empty = c.it_full + kTreeSlots;
    c.met = c.it_empty + kTreeSlots;
    c.left = c.met + 1;
    c.q_full = c.left + 1;
    c.q_empty = c.q_full + 1;
    c.never = c.q_empty + 1;
    c.abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
    c.err = p.err;
    c.wait_limit_ns = p.wait_limit_ns;
    c.item_slot = reinterpret_cast<volatile int*>(smem + C::kOffItems);
    if (threadIdx.x == 0) {
        for (int e = 0; e < C::kEntries; ++e) {
            mbar_init(&c.kv_full[e], 1);
            mbar_init(&c.kv_empty[e], kFewWarps);
        }
        for (int s = 0; s < kTreeSlots; ++s) {
            mbar_init(&c.it_full[s], 1);
            mbar_init(&c.it_empty[s], kFewWarps + 1 + kFewMerge);
        }
        mbar_init(c.met, kFewWarps);
        mbar_init(c.left, kFewMerge);
        mbar_init(c.q_full, 1);
        mbar_init(c.q_empty, kFewWarps);
        mbar_init(c.never, 1);
        *c.abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        prefetch_tmap(&p.tm_k);
        prefetch_tmap(&p.tm_v);
    }
    __syncthreads();
}

// warp 1.  Q as the right operand: of step j (16 columns), lane (g, t) holds row g's
// columns 2 t, 2 t + 1 and 2 t + 8, 2 t + 9; over an e4m3 cache 4 t .. 4 t + 3, the order in which the
// columns of K come out of its bytes.
template <int D, bool FP8, int kSets>
__device__ void few_feed(const TreeParams& p, const TreeCtx& c)
{
    using C = FewCfg<D, FP8, kSets>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = p.rows.G;
    uint32_t* const to = reinterpret_cast<uint32_t*>(c.base + C::kOffQ) + lane;
    float* const scale = reinterpret_cast<float*>(c.base + C::kOffScale);
    for (uint32_t seg = 0;; ++seg) {
        Seg s;
        if (!take_seg(c, seg, &s) || !s.on)
            return;
        uint32_t q[kSets][D / 16][2];
        float back[kSets];
#pragma unroll
        for (int n = 0; n < kSets; ++n) {
            const int row = 8 * n + g, tok = row / G, head = row - tok * G;
            const bool valid = row < s.toks * G;
            const uint16_t* from = p.q + (long long)(s.q0 + s.tok0 + (valid ? tok : 0)) * p.q_st_tok +
                                   (long long)(s.kvh * G + (valid ? head : 0)) * p.q_st_head;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int d = 16 * j + (FP8 ? 4 * t + 2 * h : 2 * t + 8 * h);
                    q[n][j][h] = valid ? *reinterpret_cast<const uint32_t*>(from + d) : 0u;
                }
            back[n] = 1.f;
            if constexpr (FP8) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    m = __vmaxu2(m, __vmaxu2(q[n][j][0] & 0x7FFF7FFFu, q[n][j][1] & 0x7FFF7FFFu));
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
                m = max(m & 0xFFFFu, m >> 16);
                // the row's largest to [2^14, 2^15) (2^110 at most); one that is not finite stays so
                const int e = m == 0 || m >= 0x7F80u ? 0 : min(126, max(-110, 14 - ((int)(m >> 7) - 127)));
                const float sc = __int_as_float((127 + e) << 23);
                back[n] = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float lo = __uint_as_float(q[n][j][h] << 16) * sc;
                        const float hi = __uint_as_float(q[n][j][h] & 0xFFFF0000u) * sc;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(q[n][j][h]) : "f"(hi), "f"(lo));
                    }
            }
        }
        if (seg > 0 && !wait_bar(c.q_empty, (seg - 1) & 1, c))
            return;
#pragma unroll
        for (int n = 0; n < kSets; ++n) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    to[((n * (D / 16) + j) * 2 + h) * 32] = q[n][j][h];
            if (t == 0)
                scale[8 * n + g] = back[n];
        }
        __syncwarp();
        mbar_arrive_p(c.q_full, lane == 0 ? 1u : 0u);
    }
}

// Where column d of a row lies among its kCols (so that neither those who write, eight
// columns of four pairs of rows, nor those who read meet their own banks).
__device__ __forceinline__ int few_place(int row, int d) { return d ^ (row >> 1 & 3) * 8; }

// warps 2 and 3 (w = 0, 1): every other row of a unit, a lane per four columns
// (kCols / 4 lanes; more rows at once where that leaves some).
template <int D, bool FP8, int kSets>
__device__ void few_merge(const TreeParams& p, const TreeCtx& c, int w)
{
    using C = FewCfg<D, FP8, kSets>;
    constexpr float kBias = FP8 ? 7.f : 0.f;
    constexpr int kLanes = C::kCols / 4, kAtOnce = 32 / kLanes;  // of a row; rows
    const int lane = threadIdx.x & 31, d4 = lane % kLanes;
    const float* const sum = reinterpret_cast<const float*>(c.base + C::kOffSum);
    const float2* const ml = reinterpret_cast<const float2*>(c.base + C::kOffMl);
    uint32_t meets = 0;
    for (uint32_t n = 0;; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on)
            return;
        const int rows = s.toks * p.rows.G;
        const long long rows0 = s.slot == kPrefixCut ? (long long)blockIdx.x * 2 * kQRows
                                                     : ((long long)s.kvh * p.T + s.q0 + s.tok0) * p.rows.G;
        float4* const to = (s.slot == kPrefixCut ? p.prefix.cut_o : p.prefix.part_o[s.slot]) + rows0 * (D / 4);
        float4* const rec = (s.slot == kPrefixCut ? p.prefix.cut_rec : p.prefix.part_rec[s.slot]) + rows0;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += C::kCols, ++meets) {
            if (!wait_bar(c.met, meets & 1, c))
                return;
#pragma unroll 1
            for (int r0 = w * kAtOnce; r0 < rows; r0 += kFewMerge * kAtOnce) {
                const int row = min(r0 + lane / kLanes, rows - 1);
                float2 x[kFewWarps];
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kFewWarps; ++k) {
                    x[k] = ml[k * C::kRows + row];
                    top = fmaxf(top, x[k].x);
                }
                float total = 0.f;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kFewWarps; ++k) {
                    // (as in prefix_merge_kernel: what is no number stays so whatever its weight)
                    const float f = x[k].x == top ? 1.f : ex2_approx(x[k].x - top);
                    const float4 v = *reinterpret_cast<const float4*>(sum + (k * C::kRows + row) * C::kCols + few_place(row, 4 * d4));
                    total = fmaf(f, x[k].y, total);
                    y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
                }
                if (r0 + lane / kLanes < rows) {
                    to[(long long)(c0 / 4 + d4) * rows + row] = y;
                    if (c0 == 0 && d4 == 0)
                        rec[row] = PrefixRow{top == -INFINITY ? top : top - kBias, total, s.whole ? -1 : (int)blockIdx.x,
                                             rows, row, 0}.pack();
                }
            }
            __syncwarp();
            mbar_arrive_p(c.left, lane == 0 ? 1u : 0u);
        }
    }
}

// The warps that compute (w = 0 .. 7).  (No calls here, wait_at's neither: with one in a role that
// has taken registers over, setmaxnreg has no effect on the whole kernel, and roles of both
// kinds of CTA lose values to local memory.)
template <int D, bool FP8, int kSets>
__device__ void few_rows(const TreeParams& p, const TreeCtx& c, int w)
{
    using C = FewCfg<D, FP8, kSets>;
    constexpr float kBias = FP8 ? 7.f : 0.f, kSlack = 8.f;  // as in attn_tree.cuh
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t lane0 = lane == 0 ? 1u : 0u;
    const uint32_t ring = smem_u32(c.base + C::kOffRing);
    // this lane's row of a tile for the four matrices of a load, and which of two
    // neighbouring 16-byte pieces: K (bf16: keys in matrices 0 1 | 2 3, as V of an e4m3 cache and K), V bf16
    const int sw = lane & 7, j4 = lane >> 3;
    const int key_k = 16 * w + sw + 8 * (j4 & 1), piece_k = j4 >> 1;
    const int key_v = FP8 ? key_k : 16 * w + sw + 8 * (j4 >> 1), piece_v = FP8 ? piece_k : j4 & 1;
    float* const sum = reinterpret_cast<float*>(c.base + C::kOffSum);
    float2* const ml = reinterpret_cast<float2*>(c.base + C::kOffMl);

    if (p.inject_stall && !wait_bar(c.never, 0, c))  // failure-detection tests
        return;
    RingPos<C::kEntries> at_k(0), at_v(1);
    uint32_t meets = 0;
    for (uint32_t n = 0;; ++n) {
        Seg s;
        if (!take_seg(c, n, &s) || !s.on || !wait_bar(c.q_full, n & 1, c))
            return;
        uint32_t q[kSets][D / 16][2];
        float unscale[kSets][2];
#pragma unroll
        for (int a = 0; a < kSets; ++a) {
#pragma unroll
            for (int b = 0; b < D / 16; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    q[a][b][h] = reinterpret_cast<const uint32_t*>(c.base + C::kOffQ)[((a * (D / 16) + b) * 2 + h) * 32 + lane];
            const float2 u = reinterpret_cast<const float2*>(c.base + C::kOffScale)[4 * a + t];
            unscale[a][0] = p.scale_log2 * u.x;
            unscale[a][1] = p.scale_log2 * u.y;
        }
        __syncwarp();
        mbar_arrive_p(c.q_empty, lane0);
        float m[kSets][2], l[kSets][2], o[kSets][D / 16][4];
#pragma unroll
        for (int a = 0; a < kSets; ++a) {
            m[a][0] = m[a][1] = -INFINITY;
            l[a][0] = l[a][1] = 0.f;
#pragma unroll
            for (int b = 0; b < D / 16; ++b)
                o[a][b][0] = o[a][b][1] = o[a][b][2] = o[a][b][3] = 0.f;
        }
        for (int i = 0; i < s.tiles; ++i) {
            const int left = s.kv_len - (s.j0 + i) * kKvTile - 16 * w;  // keys from this warp's first on
            if (!wait_bar(&c.kv_full[at_k.e], at_k.phase, c))
                return;
            float x[kSets][4];
#pragma unroll
            for (int a = 0; a < kSets; ++a)
                x[a][0] = x[a][1] = x[a][2] = x[a][3] = 0.f;
            const uint32_t k0 = ring + at_k.e * C::kKvBytes + key_k * 128;
#pragma unroll
            for (int b = 0; b < D / 16; b += FP8 ? 2 : 1) {  // 32 bytes of a row each
                const int piece = FP8 ? b + piece_k : 2 * b + piece_k;
                uint32_t r[4];
                ldsm4(r, k0 + (piece >> 3) * C::kBlockBytes + (((piece & 7) ^ sw) << 4));
                if constexpr (FP8) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a0 = f16x2_of_e4m3x2(r[2 * h]), a1 = f16x2_of_e4m3x2(r[2 * h + 1]);
                        const uint32_t a2 = f16x2_of_e4m3x2(r[2 * h] >> 16), a3 = f16x2_of_e4m3x2(r[2 * h + 1] >> 16);
#pragma unroll
                        for (int a = 0; a < kSets; ++a)
                            mma16<true>(x[a], a0, a1, a2, a3, q[a][b + h][0], q[a][b + h][1]);
                    }
                } else {
#pragma unroll
                    for (int a = 0; a < kSets; ++a)
                        mma16<false>(x[a], r[0], r[1], r[2], r[3], q[a][b][0], q[a][b][1]);
                }
            }
            __syncwarp();
            mbar_arrive_p(&c.kv_empty[at_k.e], lane0);
            at_k.next();
            // x[a][0, 1]: key g, rows 2 t and 2 t + 1; x[a][2, 3]: key g + 8
            bool grow = false;
#pragma unroll
            for (int a = 0; a < kSets; ++a) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[a][k] *= unscale[a][k & 1];
                    if (left < 16)
                        x[a][k] = g + 8 * (k >> 1) < left ? x[a][k] : -INFINITY;
                }
                grow |= fmaxf(x[a][0], x[a][2]) > m[a][0] + kSlack || fmaxf(x[a][1], x[a][3]) > m[a][1] + kSlack;
            }
            if (__any_sync(0xffffffffu, grow)) {
                // the stabiliser of a row is renewed once its maximum has grown by kSlack
#pragma unroll
                for (int a = 0; a < kSets; ++a) {
                    float f[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float top = fmaxf(x[a][k], x[a][k + 2]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const bool need = top > m[a][k] + kSlack;
                        f[k] = need ? ex2_approx(m[a][k] - top) : 1.f;
                        m[a][k] = need ? top : m[a][k];
                        l[a][k] *= f[k];
                    }
#pragma unroll
                    for (int b = 0; b < D / 16; ++b) {
                        o[a][b][0] *= f[0];
                        o[a][b][1] *= f[1];
                        o[a][b][2] *= f[0];
                        o[a][b][3] *= f[1];
                    }
                }
            }
            uint32_t pt[kSets][2];  // P^T: keys 2 t, 2 t + 1 (and + 8) of row g
#pragma unroll
            for (int a = 0; a < kSets; ++a) {
                float e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float at = m[a][k & 1];
                    e[k] = ex2_approx(x[a][k] + (at == -INFINITY ? 0.f : kBias - at));
                    l[a][k & 1] += e[k];
                }
                uint32_t lo, hi;
                if constexpr (FP8) {
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(e[1]), "f"(e[0]));
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(e[3]), "f"(e[2]));
                } else {
                    lo = pack_bf16x2(e[0], e[1]);
                    hi = pack_bf16x2(e[2], e[3]);
                }
                pt[a][0] = transposed(lo);
                pt[a][1] = transposed(hi);
            }
            if (!wait_bar(&c.kv_full[at_v.e], at_v.phase, c))
                return;
            const uint32_t v0 = ring + at_v.e * C::kKvBytes + key_v * 128;
            // keys behind the last: whatever lies there becomes 0
            const uint32_t on_lo = (2 * t < left ? 0xFFFFu : 0u) | (2 * t + 1 < left ? 0xFFFF0000u : 0u);
            const uint32_t on_hi = (2 * t + 8 < left ? 0xFFFFu : 0u) | (2 * t + 9 < left ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int b = 0; b < D / 16; b += FP8 ? 2 : 1) {
                const int piece = FP8 ? b + piece_v : 2 * b + piece_v;
                uint32_t r[4];
                ldsm4_t(r, v0 + (piece >> 3) * C::kBlockBytes + (((piece & 7) ^ sw) << 4));
                if constexpr (FP8) {
                    // a byte pair is columns 2 g and 2 g + 1 of a key: O^T's rows g and g + 8
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a0 = f16x2_of_e4m3x2(__byte_perm(r[2 * h], 0, 0x4420)) & on_lo;
                        const uint32_t a1 = f16x2_of_e4m3x2(__byte_perm(r[2 * h], 0, 0x4431)) & on_lo;
                        const uint32_t a2 = f16x2_of_e4m3x2(__byte_perm(r[2 * h + 1], 0, 0x4420)) & on_hi;
                        const uint32_t a3 = f16x2_of_e4m3x2(__byte_perm(r[2 * h + 1], 0, 0x4431)) & on_hi;
#pragma unroll
                        for (int a = 0; a < kSets; ++a)
                            mma16<true>(o[a][b + h], a0, a1, a2, a3, pt[a][0], pt[a][1]);
                    }
                } else {
#pragma unroll
                    for (int a = 0; a < kSets; ++a)
                        mma16<false>(o[a][b], r[0] & on_lo, r[1] & on_lo, r[2] & on_hi, r[3] & on_hi, pt[a][0], pt[a][1]);
                }
            }
            __syncwarp();
            mbar_arrive_p(&c.kv_empty[at_v.e], lane0);
            at_v.next();
        }
#pragma unroll
        for (int a = 0; a < kSets; ++a)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                l[a][k] += __shfl_xor_sync(0xffffffffu, l[a][k], 4);
                l[a][k] += __shfl_xor_sync(0xffffffffu, l[a][k], 8);
                l[a][k] += __shfl_xor_sync(0xffffffffu, l[a][k], 16);
            }
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += C::kCols, ++meets) {
            if (meets > 0 && !wait_bar(c.left, (meets - 1) & 1, c))  // what was there before has been read
                return;
            if (c0 == 0 && g == 0)
#pragma unroll
                for (int a = 0; a < kSets; ++a) {
                    ml[w * C::kRows + 8 * a + 2 * t] = make_float2(m[a][0], l[a][0]);
                    ml[w * C::kRows + 8 * a + 2 * t + 1] = make_float2(m[a][1], l[a][1]);
                }
#pragma unroll
            for (int a = 0; a < kSets; ++a)
#pragma unroll
                for (int b = c0 / 16; b < (c0 + C::kCols) / 16; ++b)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {  // row 2 t + k
                        float* at = sum + (w * C::kRows + 8 * a + 2 * t + k) * C::kCols;
                        const int d = 16 * b - c0;
                        if constexpr (FP8) {
                            *reinterpret_cast<float2*>(at + few_place(2 * t, d + 2 * g)) = make_float2(o[a][b][k], o[a][b][k + 2]);
                        } else {
                            at[few_place(2 * t, d + g)] = o[a][b][k];
                            at[few_place(2 * t, d + g + 8)] = o[a][b][k + 2];
                        }
                    }
            __syncwarp();
            mbar_arrive_p(c.met, lane0);
        }
    }
}

template <int D, bool FP8, int kSets>
__device__ __forceinline__ void few_roles(const TreeParams& p, const TreeCtx& c, const TreeRun& run)
{
    using C = FewCfg<D, FP8, kSets>;
    const int warp = threadIdx.x >> 5;
    // (registers as in tree_roles)
    if (warp < 4) {
        regs_dec<FP8 ? 96 : 104>();
        if (warp == 0)
            tree_producer<C, 1, true, kAll>(p, c, run.start, run.end, run.first_b, run.base);
        else if (warp == 1)
            few_feed<D, FP8, kSets>(p, c);
        else
            few_merge<D, FP8, kSets>(p, c, warp - 2);
    } else if (!FP8 || warp < 12) {
        regs_inc<FP8 ? 160 : 200>();
        few_rows<D, FP8, kSets>(p, c, warp - 4);
    } else if constexpr (FP8) {
        regs_dec<96>();
    }
    __syncthreads();
}

}  // namespace

}  // namespace b2pa
