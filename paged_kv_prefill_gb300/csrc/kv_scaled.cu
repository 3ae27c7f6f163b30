// kv_scaled.cu -- an e4m3 cache with one scale per (token, kv head) row: the
// quantising write and the read back.
//
// Write: a row x of D bf16 values gets scale = 2^e, the smallest power of two
// with max|x| / 2^e <= 448 (the largest e4m3 value), and codes
// e4m3(x / 2^e), rounded to nearest even.  Dividing by a power of two is
// exact, so each code is x's nearest; e4m3 being a floating-point format, a
// power of two loses none of its precision against max|x| / 448.
// Read: code * 2^e has four significant bits and is exact in bf16 (with
// scales of the caller's own, one rounding).
//
// Both are bound by HBM: 2 bytes of bf16 and 1 of e4m3 per element, 4 bytes
// per row for the scale, no reuse; behind that by the instructions per
// element.  A group of lanes (a power of two) takes the K and the V row of one
// (token, kv head), kChunks 16-byte pieces of bf16 per lane and tensor, and
// the maxima of the two rows ride in the two halves of one word, through one
// chain of log2(lanes) shuffles.  More rows per group, with their loads issued
// together, were slower: the registers they take cost more loads in flight
// than they add (write of 32768 tokens x 8 heads x 128: 35 us with one row, 37
// with two or four, 47 with eight; read of 131072 x 8 x 64: 68, 72, 78, 83).
// Blocks of 128 threads: 35.6 and 68.7 us (5.7 and 6.0 TB/s, 0.84 and 0.88 of
// the copy rate); of 256: 36.8 and 70.9.
#include "kv_scaled.cuh"

#include "../../include/b2pa.h"
#include "ptx.cuh"

namespace b2pa {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ uint32_t two_e4m3(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight bf16 values times 2^-e, as e4m3.
__device__ __forceinline__ uint2 quantise8(uint4 v, float inv)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = two_e4m3(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xFFFF0000u) * inv);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Largest finite magnitude of kChunks x 8 bf16 values, as bf16 bits.
template <int kChunks>
__device__ __forceinline__ uint32_t top_of(const uint4* v)
{
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu),
                                 __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu)));
    m = max(m & 0xFFFFu, m >> 16);
    if (m >= 0x7F80u) {  // an infinity or NaN among them: again, without those
        m = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
                m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
        }
    }
    return m;
}

// e of a row whose largest finite magnitude has these bf16 bits: with the
// value m 2^E, 1 <= m < 2, and 448 = 1.75 * 2^8, it is E - 8 for m <= 1.75,
// else E - 7; at least -126, so that 2^e and 2^-e are normal floats.  A row of
// zeros has scale 1.
__device__ __forceinline__ int scale_exponent(uint32_t top)
{
    if (top == 0)
        return 0;
    const int e = (int)(top >> 7) - 127 - ((top & 0x7Fu) <= 0x60u ? 8 : 7);
    return max(e, -126);
}

// The (token, kv head) of a lane group and its slot.
struct Row {
    bool on;
    long long n;     // token
    int h;           // kv head
    long long page;  // -1: a slot outside the pool
    int slot;
};

template <int kLanes>
__device__ __forceinline__ Row row_of(const ScaledKvParams& p)
{
    const unsigned long long id = (unsigned long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const unsigned heads = (unsigned)p.Hkv;
    Row s;
    // (a 32-bit division where the number allows it)
    s.n = id <= 0xFFFFFFFFull ? (long long)((unsigned)id / heads) : (long long)(id / heads);
    s.h = (int)((long long)id - s.n * heads);
    s.on = s.n < p.T;
    s.page = s.slot = 0;
    if (s.on) {
        const int loc = p.cache_loc[s.n];
        const int page = loc / p.page_size;
        s.page = page;
        s.slot = loc - page * p.page_size;
        if (loc < 0 || page >= p.num_pages) {
            s.page = -1;
            if (s.h == 0 && threadIdx.x % kLanes == 0)
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_SLOT);
        }
    }
    return s;
}

__device__ __forceinline__ long long place(const long long st[3], const Row& s)
{
    return s.page * st[0] + s.h * st[1] + s.slot * st[2];
}

template <int kChunks, int kLanes>
__global__ void __launch_bounds__(kThreads) append_scaled_kernel(const __grid_constant__ ScaledKvParams p)
{
    const int lane = threadIdx.x % kLanes, d = 8 * kChunks * lane;
    const Row s = row_of<kLanes>(p);
    const bool on = s.on && s.page >= 0, mine = on && d < p.D;  // every lane stays for the shuffles
    uint4 v[2][kChunks];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            v[i][c] = make_uint4(0u, 0u, 0u, 0u);
            if (mine)
                v[i][c] = reinterpret_cast<const uint4*>(p.x[i] + s.n * p.tok[i] + s.h * p.head[i] + d)[c];
        }
    uint32_t top = top_of<kChunks>(v[0]) | top_of<kChunks>(v[1]) << 16;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = scale_exponent(i ? top >> 16 : top & 0xFFFFu);
        const float inv = __int_as_float((127 - e) << 23);
        if (mine) {
            uint8_t* to = p.pool[i] + place(p.pool_st[i], s) + d;
            if constexpr (kChunks == 2) {
                const uint2 a = quantise8(v[i][0], inv), b = quantise8(v[i][1], inv);
                *reinterpret_cast<uint4*>(to) = make_uint4(a.x, a.y, b.x, b.y);
            } else {
                *reinterpret_cast<uint2*>(to) = quantise8(v[i][0], inv);
            }
        }
        if (on && lane == 0)
            p.scale[i][place(p.scale_st[i], s)] = __int_as_float((127 + e) << 23);
    }
}

// Eight codes times a scale, as bf16.
__device__ __forceinline__ uint4 restore8(uint32_t c0, uint32_t c1, float scale)
{
    const uint32_t w[4] = {c0 & 0xFFFFu, c0 >> 16, c1 & 0xFFFFu, c1 >> 16};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w[i]));
        float lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        const float2 y = __fmul2_rn(make_float2(lo, hi), make_float2(scale, scale));
        o[i] = pack_bf16x2(y.x, y.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int kChunks, int kLanes>
__global__ void __launch_bounds__(kThreads) read_scaled_kernel(const __grid_constant__ ScaledKvParams p)
{
    const int d = 8 * kChunks * (int)(threadIdx.x % kLanes);
    const Row s = row_of<kLanes>(p);
    if (!s.on || d >= p.D)
        return;
    uint32_t c[2][2 * kChunks];
    float unit[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < 2 * kChunks; ++k)
            c[i][k] = 0u;  // a slot outside the pool reads as zeros
        unit[i] = 1.f;
        if (s.page >= 0) {
            const uint8_t* from = p.pool[i] + place(p.pool_st[i], s) + d;
            if constexpr (kChunks == 2) {
                const uint4 x = *reinterpret_cast<const uint4*>(from);
                c[i][0] = x.x;
                c[i][1] = x.y;
                c[i][2] = x.z;
                c[i][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(from);
                c[i][0] = x.x;
                c[i][1] = x.y;
            }
            unit[i] = p.scale[i][place(p.scale_st[i], s)];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
            reinterpret_cast<uint4*>(p.y[i] + s.n * p.tok[i] + s.h * p.head[i] + d)[k] =
                restore8(c[i][2 * k], c[i][2 * k + 1], unit[i]);
}

template <bool kWrite, int kChunks, int kLanes>
cudaError_t launch_lanes(const ScaledKvParams& p, cudaStream_t stream)
{
    constexpr int kGroups = kThreads / kLanes;
    const long long blocks = ((long long)p.T * p.Hkv + kGroups - 1) / kGroups;
    if (blocks > 0x7FFFFFFFLL)
        return cudaErrorInvalidConfiguration;
    if (kWrite)
        append_scaled_kernel<kChunks, kLanes><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    else
        read_scaled_kernel<kChunks, kLanes><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <bool kWrite>
cudaError_t launch(const ScaledKvParams& p, cudaStream_t stream)
{
    if (p.T == 0)
        return cudaSuccess;
    // 16 elements per lane where every row of the pools can be taken in 16-byte pieces
    uintptr_t at = p.D % 16 == 0 ? 0 : 8;
    for (int i = 0; i < 2; ++i)
        at |= reinterpret_cast<uintptr_t>(p.pool[i]) | (uintptr_t)p.pool_st[i][0] | (uintptr_t)p.pool_st[i][1] |
              (uintptr_t)p.pool_st[i][2];
    if (at % 16 == 0) {
        const int need = p.D >> 4;
        if (need <= 4)
            return launch_lanes<kWrite, 2, 4>(p, stream);
        if (need <= 8)
            return launch_lanes<kWrite, 2, 8>(p, stream);
        return launch_lanes<kWrite, 2, 16>(p, stream);
    }
    const int need = p.D >> 3;
    if (need <= 8)
        return launch_lanes<kWrite, 1, 8>(p, stream);
    if (need <= 16)
        return launch_lanes<kWrite, 1, 16>(p, stream);
    return launch_lanes<kWrite, 1, 32>(p, stream);
}

}  // namespace

cudaError_t launch_append_scaled(const ScaledKvParams& p, cudaStream_t stream)
{
    return launch<true>(p, stream);
}
cudaError_t launch_read_scaled(const ScaledKvParams& p, cudaStream_t stream)
{
    return launch<false>(p, stream);
}

}  // namespace b2pa
