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
// per row for the scale, no reuse.  A group of lanes (a power of two) holds a
// row, 8 elements (one 16-byte chunk of bf16) per lane, so that the row's
// maximum takes log2(lanes) shuffles.  A group takes the K and the V row of
// kRows (token, kv head) pairs and issues all their loads before the first
// store.
#include "kv_scaled.cuh"

#include "../../include/b2pa.h"
#include "ptx.cuh"

namespace b2pa {

namespace {

constexpr int kThreads = 256;

struct Row {
    bool on;      // a row to move
    long long n;  // token
    int h;        // kv head
    long long page, slot;
};

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

// Largest finite magnitude of eight bf16 values, as bf16 bits.
__device__ __forceinline__ uint32_t top8(uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
        m = max(m, lo < 0x7F80u ? lo : 0u);
        m = max(m, hi < 0x7F80u ? hi : 0u);
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

template <int kLanes, int kRows, typename Idx>
__device__ __forceinline__ Row row_of(const ScaledKvParams& p, int r)
{
    constexpr int kGroups = kThreads / kLanes;
    const Idx id = ((Idx)blockIdx.x * kRows + r) * kGroups + threadIdx.x / kLanes;
    Row w;
    const Idx n = id / (Idx)p.Hkv;
    w.n = (long long)n;
    w.h = (int)(id - n * (Idx)p.Hkv);
    w.on = n < (Idx)p.T;
    w.page = w.slot = 0;
    if (w.on) {
        const int loc = p.cache_loc[w.n];
        w.page = loc / p.page_size;
        w.slot = loc - w.page * p.page_size;
        if (loc < 0 || w.page >= p.num_pages) {
            w.page = -1;
            if (w.h == 0 && threadIdx.x % kLanes == 0)
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_SLOT);
        }
    }
    return w;
}

template <int kLanes, int kRows, typename Idx>
__global__ void __launch_bounds__(kThreads) append_scaled_kernel(const __grid_constant__ ScaledKvParams p)
{
    const int lane = threadIdx.x % kLanes;
    const bool mine = 8 * lane < p.D;
    Row row[kRows];
    uint4 v[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        row[r] = row_of<kLanes, kRows, Idx>(p, r);
        row[r].on = row[r].on && row[r].page >= 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[r][i] = make_uint4(0u, 0u, 0u, 0u);
            if (row[r].on && mine)
                v[r][i] = *reinterpret_cast<const uint4*>(p.x[i] + row[r].n * p.tok[i] + row[r].h * p.head[i] + 8 * lane);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t top = top8(v[r][i]);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e = scale_exponent(top);
            if (!row[r].on)
                continue;
            const uint2 c = quantise8(v[r][i], __int_as_float((127 - e) << 23));
            if (mine)
                *reinterpret_cast<uint2*>(p.pool[i] + row[r].page * p.pool_st[i][0] + row[r].h * p.pool_st[i][1] +
                                          row[r].slot * p.pool_st[i][2] + 8 * lane) = c;
            if (lane == 0)
                p.scale[i][row[r].page * p.scale_st[i][0] + row[r].h * p.scale_st[i][1] +
                           row[r].slot * p.scale_st[i][2]] = __int_as_float((127 + e) << 23);
        }
}

// Eight codes times a scale, as bf16.
__device__ __forceinline__ uint4 restore8(uint2 c, float scale)
{
    const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w[i]));
        float lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        o[i] = pack_bf16x2(lo * scale, hi * scale);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int kLanes, int kRows, typename Idx>
__global__ void __launch_bounds__(kThreads) read_scaled_kernel(const __grid_constant__ ScaledKvParams p)
{
    const int lane = threadIdx.x % kLanes;
    const bool mine = 8 * lane < p.D;
    Row row[kRows];
    uint2 c[kRows][2];
    float s[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        row[r] = row_of<kLanes, kRows, Idx>(p, r);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[r][i] = make_uint2(0u, 0u);  // a slot outside the pool reads as zeros
            s[r][i] = 1.f;
            if (row[r].on && mine && row[r].page >= 0) {
                c[r][i] = *reinterpret_cast<const uint2*>(p.pool[i] + row[r].page * p.pool_st[i][0] +
                                                          row[r].h * p.pool_st[i][1] + row[r].slot * p.pool_st[i][2] +
                                                          8 * lane);
                s[r][i] = p.scale[i][row[r].page * p.scale_st[i][0] + row[r].h * p.scale_st[i][1] +
                                     row[r].slot * p.scale_st[i][2]];
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (row[r].on && mine)
                *reinterpret_cast<uint4*>(p.y[i] + row[r].n * p.tok[i] + row[r].h * p.head[i] + 8 * lane) =
                    restore8(c[r][i], s[r][i]);
}

template <bool kWrite, int kLanes, int kRows>
cudaError_t launch_rows(const ScaledKvParams& p, cudaStream_t stream)
{
    constexpr long long kPerBlock = (long long)kThreads / kLanes * kRows;
    const long long rows = (long long)p.T * p.Hkv;
    const long long blocks = (rows + kPerBlock - 1) / kPerBlock;
    if (blocks > 0x7FFFFFFFLL)
        return cudaErrorInvalidConfiguration;
    if (rows <= 0x7FFFFFFFLL - kPerBlock) {
        if (kWrite)
            append_scaled_kernel<kLanes, kRows, unsigned><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
        else
            read_scaled_kernel<kLanes, kRows, unsigned><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    } else {
        if (kWrite)
            append_scaled_kernel<kLanes, kRows, unsigned long long><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
        else
            read_scaled_kernel<kLanes, kRows, unsigned long long><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

template <bool kWrite, int kLanes>
cudaError_t launch_lanes(const ScaledKvParams& p, int sms, cudaStream_t stream)
{
    // several rows per group once one per group would need more than one wave
    // of blocks (8 blocks of 256 threads per SM)
    const long long wave = (long long)sms * 8 * (kThreads / kLanes);
    return (long long)p.T * p.Hkv > wave ? launch_rows<kWrite, kLanes, 4>(p, stream)
                                         : launch_rows<kWrite, kLanes, 1>(p, stream);
}

template <bool kWrite>
cudaError_t launch(const ScaledKvParams& p, int sms, cudaStream_t stream)
{
    if (p.T == 0)
        return cudaSuccess;
    const int need = p.D >> 3;
    if (need <= 8)
        return launch_lanes<kWrite, 8>(p, sms, stream);
    if (need <= 16)
        return launch_lanes<kWrite, 16>(p, sms, stream);
    return launch_lanes<kWrite, 32>(p, sms, stream);
}

}  // namespace

cudaError_t launch_append_scaled(const ScaledKvParams& p, int sms, cudaStream_t stream)
{
    return launch<true>(p, sms, stream);
}
cudaError_t launch_read_scaled(const ScaledKvParams& p, int sms, cudaStream_t stream)
{
    return launch<false>(p, sms, stream);
}

}  // namespace b2pa
