// rope.cu -- RMS norm of each query and key head with the rotary position
// rotation, in one pass over the data.
//
// For a row x (token t, head h) of D elements, with w its norm weight,
//
//   y = w * x / sqrt(mean(x^2) + eps)                 (no weight: y = x)
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i)          for i < R / 2
//
// with (a, b) = (y_2i, y_2i+1) (interleaved) or (y_i, y_i+R/2), and c_i, s_i
// row `pos` of the caller's table, pos being the token's position on the axis
// that frequency i belongs to.  Elements from R on pass through.  All of it
// in fp32, rounded to bf16 once.
//
// Bound by HBM: 4 bytes move per element and a handful of operations are done
// on it.  A group of lanes (a power of two) holds one row, 16 elements per
// lane, so that both elements of every pair are in one lane and the norm's
// sum takes log2(lanes) shuffles.  A lane's two 16-byte chunks are
// (c, c + R/16) when pairs lie R/2 apart and R/2 is a multiple of 8, and
// neighbours otherwise; pairs R/2 apart with another R/2 go through a row of
// shared memory.
//
// Two kernels.  rope_rows_kernel: one row per group, for calls of one or
// two waves, whose time is latency, and for the rare pairing.  rope_staged_kernel,
// for the others: the table row must be read before the rotation and its
// place is known only from the positions, and a group that does this for a few
// rows at a time keeps too few loads in flight.  So all tokens' rows, laid end
// to end in sets of kSetRows heads, are cut into equal runs, one per group, and
// each thread copies its own pieces of the rows and of the table into its own
// places of a ring in shared memory with cp.async, kStages - 1 sets ahead; no
// thread reads another's pieces, so the ring needs no barrier.  A run goes
// through a token's heads one after the other, so that positions, table row
// and the weights times the table are taken once per token and tensor and not
// once per set, which was most of the instructions.  11750 tokens x (32 + 8)
// heads x 128: 75 us with one row per group, 60 us with four in registers,
// 45.4 us so (5.4 TB/s, 0.80 of the copy rate); 16384 tokens x 72 heads with
// three axes 101 us (6.0 TB/s, 0.89; 123 with the table per set).  Sets of one and
// three rows 103 and 104 us, of four and eight 115; three blocks of 128 threads
// per SM 112, five 112, six 123; eight of 64 the same as four of 128.
#include "rope.cuh"

#include "../../include/b2pa.h"
#include "ptx.cuh"

namespace b2pa {

namespace {

constexpr int kRopeThreads = 128;

enum RopeMode { kInterleaved, kHalvesInLane, kHalvesInSmem };

// Eight consecutive elements as four packed pairs (the packed fp32 operations
// do two at once).
__device__ __forceinline__ void unpack8(uint4 v, float2* f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2* f)
{
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}

__device__ __forceinline__ void load4(const float* p, float2* f)
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
}

__device__ __forceinline__ void load_weight8(const RopeTensor& x, int d, float2* w)
{
    if (x.weight_f32) {
        load4(static_cast<const float*>(x.weight) + d, w);
        load4(static_cast<const float*>(x.weight) + d + 4, w + 2);
    } else
        unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x.weight) + d)), w);
}

// This lane's two chunks of a row (-1: none) and whether its pairs rotate.
struct Chunks {
    int a, b;
    bool turns;
};

template <RopeMode kMode>
__device__ __forceinline__ Chunks chunks_of(const RopeParams& p, int lane)
{
    Chunks c{2 * lane, 2 * lane + 1, 16 * lane < p.R};
    if (kMode == kHalvesInLane) {
        const int hc = p.R >> 4;  // chunks of one half
        c.turns = lane < hc;
        c.a = c.turns ? lane : 2 * hc + 2 * (lane - hc);
        c.b = c.turns ? lane + hc : c.a + 1;
    }
    if (c.a >= p.D >> 3)
        c.a = -1;
    if (c.b >= p.D >> 3)
        c.b = -1;
    return c;
}

// A token's positions; ok = false, and the first row of the table, if one is
// outside it.
struct Places {
    int pos[kRopeMaxAxes];
    bool ok;
    __device__ __forceinline__ int at(int axis) const
    {
        return axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
    }
    __device__ __forceinline__ const float* row(const RopeParams& p, int axis) const
    {
        return p.cos_sin + (long long)at(axis) * p.cs_stride;
    }
};

__device__ __forceinline__ Places places_of(const RopeParams& p, long long t, bool on)
{
    Places x;
    x.ok = on;
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes; ++a) {
        x.pos[a] = 0;
        if (on && a < p.axes)
            x.pos[a] = p.positions[a * p.pos_stride + t];
    }
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes; ++a)
        if (x.pos[a] < 0 || x.pos[a] >= p.max_pos)
            x.ok = false;
    if (!x.ok)
        x.pos[0] = x.pos[1] = x.pos[2] = x.pos[3] = 0;
    return x;
}

__device__ __forceinline__ void load_weights(const RopeTensor& x, const Chunks& ch, float2 (&wa)[4], float2 (&wb)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        wa[i] = wb[i] = make_float2(1.f, 1.f);
    if (x.weight != nullptr && ch.a >= 0)
        load_weight8(x, 8 * ch.a, wa);
    if (x.weight != nullptr && ch.b >= 0)
        load_weight8(x, 8 * ch.b, wb);
}

// x / sqrt(mean(x^2) + eps) over the row that kLanes lanes hold (norm false:
// x; the lanes of a warp may differ in it, so all take part in the sum).
template <int kLanes>
__device__ __forceinline__ void norm_row(const RopeParams& p, bool norm, float2 (&a)[4], float2 (&b)[4])
{
    float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum2 = __ffma2_rn(a[i], a[i], __ffma2_rn(b[i], b[i], sum2));
    float sum = sum2.x + sum2.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = norm ? rsqrtf(fmaf(sum, p.inv_d, p.eps)) : 1.f;
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = __fmul2_rn(a[i], inv2);
        b[i] = __fmul2_rn(b[i], inv2);
    }
}

// Weight and rotation of a lane's 16 elements as one linear map, formed once
// for all rows that share it:  halves: a' = m0 a + m1 b, b' = m2 b + m3 a with
// m = (wa c, -wb s, wb c, wa s).  Interleaved, per packed pair (x, y): x' =
// m.x x + n.x y, y' = m.y y + n.y x with m = (wx c, wy c), n = (-wy s, wx s);
// m0, n = m1 for a and m2, n = m3 for b.  A pair that does not turn has c = 1,
// s = 0 and skips the cross terms (an infinity times 0 is no 0).
struct Turn {
    float2 m[4][4];
};

template <RopeMode kMode>
__device__ __forceinline__ Turn turn_of(const RopeParams& p, int lane, const float2 (&c)[4], const float2 (&s)[4],
                                        const float2 (&wa)[4], const float2 (&wb)[4])
{
    Turn t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kMode == kHalvesInLane) {
            t.m[0][i] = __fmul2_rn(wa[i], c[i]);
            t.m[1][i] = __fmul2_rn(wb[i], make_float2(-s[i].x, -s[i].y));
            t.m[2][i] = __fmul2_rn(wb[i], c[i]);
            t.m[3][i] = __fmul2_rn(wa[i], s[i]);
        } else {
            const float ca = i & 1 ? c[i / 2].y : c[i / 2].x, sa = i & 1 ? s[i / 2].y : s[i / 2].x;
            const float cb = i & 1 ? c[2 + i / 2].y : c[2 + i / 2].x, sb = i & 1 ? s[2 + i / 2].y : s[2 + i / 2].x;
            t.m[0][i] = __fmul2_rn(wa[i], make_float2(ca, ca));
            t.m[1][i] = make_float2(-wa[i].y * sa, wa[i].x * sa);
            t.m[2][i] = __fmul2_rn(wb[i], make_float2(cb, cb));
            t.m[3][i] = make_float2(-wb[i].y * sb, wb[i].x * sb);
        }
    }
    return t;
}

template <RopeMode kMode>
__device__ __forceinline__ void turn_row(const RopeParams& p, int lane, bool turns, const Turn& t, float2 (&a)[4],
                                         float2 (&b)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = a[i], v = b[i];
        a[i] = __fmul2_rn(u, t.m[0][i]);
        b[i] = __fmul2_rn(v, t.m[2][i]);
        if (kMode == kHalvesInLane) {
            if (turns) {
                a[i] = __ffma2_rn(v, t.m[1][i], a[i]);
                b[i] = __ffma2_rn(u, t.m[3][i], b[i]);
            }
        } else {
            if (16 * lane + 2 * i < p.R)
                a[i] = __ffma2_rn(make_float2(u.y, u.x), t.m[1][i], a[i]);
            if (16 * lane + 8 + 2 * i < p.R)
                b[i] = __ffma2_rn(make_float2(v.y, v.x), t.m[3][i], b[i]);
        }
    }
}

__device__ __forceinline__ void store_row(const RopeTensor& x, long long t, int h, const Chunks& ch, const float2 (&a)[4],
                                          const float2 (&b)[4])
{
    uint16_t* row = x.out + t * x.out_tok + (long long)h * x.out_head;
    if (ch.a >= 0)
        *reinterpret_cast<uint4*>(row + 8 * ch.a) = pack8(a);
    if (ch.b >= 0)
        *reinterpret_cast<uint4*>(row + 8 * ch.b) = pack8(b);
}

// The common axis of the frequencies 4 g .. 4 g + 3 if their table entries can
// be read as a float4, else 255.
__device__ __forceinline__ int vector_axis(const RopeParams& p, int g)
{
    return p.vec_table && 4 * g < p.R >> 1 ? p.axis_of4[g] : 255;
}

// kLanes lanes per row, each holding two chunks of 8 elements; one row per group.
template <RopeMode kMode, int kLanes>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kGroups = kRopeThreads / kLanes;
    __shared__ __align__(16) float pair_rows[kMode == kHalvesInSmem ? kGroups * kLanes * 16 : 1];
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const unsigned heads = (unsigned)(p.x[0].heads + p.x[1].heads);
    const unsigned long long id = (unsigned long long)blockIdx.x * kGroups + group;
    // (a 32-bit division where the number allows it)
    const long long t = id <= 0xFFFFFFFFull ? (long long)((unsigned)id / heads) : (long long)(id / heads);
    const bool on = t < p.T;  // every lane stays for the shuffles
    const int hh = (int)((long long)id - t * heads);
    const bool is_k = hh >= p.x[0].heads;
    const RopeTensor& x = p.x[is_k ? 1 : 0];
    const int h = is_k ? hh - p.x[0].heads : hh;
    const int half = p.R >> 1;
    const Chunks ch = chunks_of<kMode>(p, lane);

    uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va;
    if (on) {
        const uint16_t* row = x.in + t * x.in_tok + (long long)h * x.in_head;
        if (ch.a >= 0)
            va = *reinterpret_cast<const uint4*>(row + 8 * ch.a);
        if (ch.b >= 0)
            vb = *reinterpret_cast<const uint4*>(row + 8 * ch.b);
    }
    float2 wa[4], wb[4];
    load_weights(x, ch, wa, wb);
    const Places at = places_of(p, t, on);
    if (on && !at.ok && hh == 0 && lane == 0)
        atomicOr(p.err, (unsigned)B2PA_DEV_BAD_POSITION);

    float2 c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = make_float2(1.f, 1.f);
        s[i] = make_float2(0.f, 0.f);
    }
    if (kMode != kHalvesInSmem && ch.turns) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {  // four of its eight frequencies
            const int f = 8 * lane + 4 * v, axis = vector_axis(p, 2 * lane + v);
            if (axis != 255) {
                load4(at.row(p, axis) + f, &c[2 * v]);
                load4(at.row(p, axis) + half + f, &s[2 * v]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (f + i >= half)
                        break;
                    const float* e = at.row(p, p.axis_of[f + i]) + f + i;
                    (i & 1 ? c[2 * v + i / 2].y : c[2 * v + i / 2].x) = __ldg(e);
                    (i & 1 ? s[2 * v + i / 2].y : s[2 * v + i / 2].x) = __ldg(e + half);
                }
            }
        }
    }
    float2 a[4], b[4];
    unpack8(va, a);
    unpack8(vb, b);
    norm_row<kLanes>(p, x.weight != nullptr, a, b);
    if (kMode != kHalvesInSmem) {
        turn_row<kMode>(p, lane, ch.turns, turn_of<kMode>(p, lane, c, s, wa, wb), a, b);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __fmul2_rn(a[i], wa[i]);
            b[i] = __fmul2_rn(b[i], wb[i]);
        }
        float* row = pair_rows + group * kLanes * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            reinterpret_cast<float2*>(row + 16 * lane)[i] = a[i];
            reinterpret_cast<float2*>(row + 16 * lane + 8)[i] = b[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = 16 * lane + i;
            if (e < p.R) {
                const int f = e < half ? e : e - half;
                const float* cs = at.row(p, p.axis_of[f]) + f;
                const float cc = __ldg(cs), ss = __ldg(cs + half);
                const float u = row[e], v = row[e < half ? e + half : e - half];
                const float y = e < half ? u * cc - v * ss : u * cc + v * ss;
                float2& to = i < 8 ? a[(i & 7) / 2] : b[(i & 7) / 2];
                (i & 1 ? to.y : to.x) = y;
            }
        }
    }
    if (at.ok)
        store_row(x, t, h, ch, a, b);
}

// ---------------------------------------------------------------- the staged kernel

constexpr int kSetRows = 2;
constexpr int kStages = 2;
// a thread's pieces of 16 bytes: 2 per row, 4 of a table row
constexpr int kStagedSmem = (kStages * 2 * kSetRows + 2 * 4) * 16 * kRopeThreads;  // rows; two tokens' table rows

__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Through L1: the table's row is the same for all sets of a token, most of
// which one block has in flight at once.
__device__ __forceinline__ void copy16_l1(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4_l1(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <RopeMode kMode, int kLanes>
__global__ void __launch_bounds__(kRopeThreads) rope_staged_kernel(const __grid_constant__ RopeParams p, unsigned total)
{
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int kGroups = kRopeThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int half = p.R >> 1, f0 = 8 * lane;
    const Chunks ch = chunks_of<kMode>(p, lane);
    const int axis0 = vector_axis(p, 2 * lane), axis1 = vector_axis(p, 2 * lane + 1);
    // sets of kSetRows rows of a token: those of the queries, then those of the
    // keys; all tokens' sets, one after the other, are cut into equal runs
    const unsigned sets_q = (unsigned)(p.x[0].heads + kSetRows - 1) / kSetRows;
    const unsigned sets = sets_q + (unsigned)(p.x[1].heads + kSetRows - 1) / kSetRows;
    const unsigned groups = gridDim.x * kGroups, me = blockIdx.x * kGroups + threadIdx.x / kLanes;
    const unsigned share = total / groups, more = total % groups;
    const unsigned first = me * share + min(me, more), count = share + (me < more ? 1 : 0);
    const unsigned rounds = share + (more > 0 ? 1 : 0);  // the same for every thread: the shuffles need whole warps
    const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
    // this thread's pieces of a set's rows and of a token's table row
    auto piece = [&](unsigned stage, int k) { return mine + (stage * 2 * kSetRows + k) * (kRopeThreads * 16); };
    auto table = [&](unsigned which, int k) { return mine + ((kStages * kSetRows + which * 2) * 2 + k) * (kRopeThreads * 16); };

    struct Set {
        unsigned n;     // of this group's
        unsigned t, r;  // token, set of the token
        unsigned tab;   // where the token's table row is
        bool opens;     // the group's first set of this token
    };
    auto next = [&](Set& z) {
        ++z.n;
        z.opens = ++z.r == sets;
        if (z.opens) {
            z.r = 0;
            ++z.t;
            z.tab ^= 1;
        }
    };
    auto is_k = [&](const Set& z) { return z.r >= sets_q; };
    auto head0 = [&](const Set& z) { return (int)(is_k(z) ? z.r - sets_q : z.r) * kSetRows; };

    // `use` is the set whose rows are computed, `copied` the one whose copies
    // start next; `at` are the positions of the token it opens next
    Set use{0, first / sets, first % sets, 0, true}, copied = use;
    Places at = places_of(p, copied.t, count > 0);
    uint32_t ok_bits = 0;  // bit of a table row: its token's positions are inside the table
    unsigned to = 0, from = 0;  // stages
    auto advance = [&] {
        if (copied.n < count) {
            const RopeTensor& x = p.x[is_k(copied) ? 1 : 0];
            const int h0 = head0(copied);
            const uint16_t* row = x.in + (long long)copied.t * x.in_tok + (long long)h0 * x.in_head;
#pragma unroll
            for (int r = 0; r < kSetRows; ++r, row += x.in_head)
                if (h0 + r < x.heads) {
                    if (ch.a >= 0)
                        copy16(piece(to, 2 * r), row + 8 * ch.a);
                    if (ch.b >= 0)
                        copy16(piece(to, 2 * r + 1), row + 8 * ch.b);
                }
            if (copied.opens) {  // (behind the rows, which need no position)
                if (!at.ok && lane == 0)
                    atomicOr(p.err, (unsigned)B2PA_DEV_BAD_POSITION);
                ok_bits = (ok_bits & ~(1u << copied.tab)) | ((at.ok ? 1u : 0u) << copied.tab);
                if (ch.turns) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int axis = v ? axis1 : axis0, f = f0 + 4 * v;
                        const uint32_t cos = table(copied.tab, v), sin = table(copied.tab, 2 + v);
                        if (axis != 255) {
                            const float* e = at.row(p, axis) + f;
                            copy16_l1(cos, e);
                            copy16_l1(sin, e + half);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int fi = min(f + i, half - 1);  // (a frequency past the last one turns no pair)
                                const float* e = at.row(p, p.axis_of[fi]) + fi;
                                copy4_l1(cos + 4 * i, e);
                                copy4_l1(sin + 4 * i, e + half);
                            }
                        }
                    }
                }
                at = places_of(p, copied.t + 1, copied.t + 1 < (unsigned)p.T);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next(copied);
        to = to + 1 == kStages ? 0 : to + 1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        advance();
    Turn turn;
    for (unsigned round = 0; round < rounds; ++round) {
        advance();
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        const RopeTensor& x = p.x[is_k(use) ? 1 : 0];
        const int h0 = head0(use);
        // another token, or its keys after its queries (for the whole warp: what a
        // group has already it forms again)
        if (__any_sync(0xffffffffu, use.opens || use.r == sets_q)) {
            float2 wa[4], wb[4], c[4], s[4];
            load_weights(x, ch, wa, wb);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 u = make_uint4(0x3F800000u, 0x3F800000u, 0x3F800000u, 0x3F800000u), v = make_uint4(0u, 0u, 0u, 0u);
                if (ch.turns) {
                    u = ld_shared_v4(table(use.tab, i));
                    v = ld_shared_v4(table(use.tab, 2 + i));
                }
                c[2 * i] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
                c[2 * i + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
                s[2 * i] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
                s[2 * i + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
            }
            if (kMode == kInterleaved) {
                // pairs past R in a lane that turns others keep their value
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (f0 + i >= half)
                        (i & 1 ? c[i / 2].y : c[i / 2].x) = 1.f;
            }
            turn = turn_of<kMode>(p, lane, c, s, wa, wb);
        }
        const bool ok = use.n < count && (ok_bits >> use.tab & 1u);
#pragma unroll
        for (int r = 0; r < kSetRows; ++r) {
            const bool there = h0 + r < x.heads;
            uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va;
            if (there && ch.a >= 0)
                va = ld_shared_v4(piece(from, 2 * r));
            if (there && ch.b >= 0)
                vb = ld_shared_v4(piece(from, 2 * r + 1));
            float2 a[4], b[4];
            unpack8(va, a);
            unpack8(vb, b);
            norm_row<kLanes>(p, x.weight != nullptr, a, b);
            turn_row<kMode>(p, lane, ch.turns, turn, a, b);
            if (ok && there)
                store_row(x, use.t, h0 + r, ch, a, b);
        }
        next(use);
        from = from + 1 == kStages ? 0 : from + 1;
    }
}

template <RopeMode kMode, int kLanes>
cudaError_t launch_lanes(const RopeParams& p, int sms, cudaStream_t stream)
{
    constexpr int kGroups = kRopeThreads / kLanes;
    const long long rows = (long long)p.T * (p.x[0].heads + p.x[1].heads);
    if constexpr (kMode != kHalvesInSmem) {
        // Where the copies ahead pay: 40 heads x 128, 430 tokens 3.9 us by rows and 4.2
        // staged, 600 tokens 5.4 and 5.5, 900 tokens 6.8 and 6.4, 3000 tokens 17.8 and 15.
        const long long sets = (long long)p.T * ((p.x[0].heads + kSetRows - 1) / kSetRows + (p.x[1].heads + kSetRows - 1) / kSetRows);
        const int grid = sms * 4;  // (see the top)
        if (rows > (long long)sms * 10 * kGroups && sets + (long long)grid * kGroups * (kStages + 1) <= 0xFFFFFFFFLL) {
            auto kern = rope_staged_kernel<kMode, kLanes>;
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedSmem);
            if (e != cudaSuccess)
                return e;
            kern<<<grid, kRopeThreads, kStagedSmem, stream>>>(p, (unsigned)sets);
            return cudaGetLastError();
        }
    }
    const long long blocks = (rows + kGroups - 1) / kGroups;
    if (blocks > 0x7FFFFFFFLL)
        return cudaErrorInvalidConfiguration;
    rope_rows_kernel<kMode, kLanes><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <RopeMode kMode>
cudaError_t launch_mode(const RopeParams& p, int sms, cudaStream_t stream)
{
    // 16 elements per lane.  Halves in one lane: R / 16 lanes turn, the rest pass
    const int need = kMode == kHalvesInLane ? p.R / 16 + (p.D - p.R + 15) / 16 : (p.D + 15) / 16;
    if (need <= 4)
        return launch_lanes<kMode, 4>(p, sms, stream);
    if (need <= 8)
        return launch_lanes<kMode, 8>(p, sms, stream);
    return launch_lanes<kMode, 16>(p, sms, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, bool interleaved, int sms, cudaStream_t stream)
{
    if (p.T == 0)
        return cudaSuccess;
    if (interleaved)
        return launch_mode<kInterleaved>(p, sms, stream);
    return p.R % 16 == 0 ? launch_mode<kHalvesInLane>(p, sms, stream) : launch_mode<kHalvesInSmem>(p, sms, stream);
}

}  // namespace b2pa
