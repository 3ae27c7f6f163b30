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
// shared memory.  A group takes kRows rows of one token, whose cosines and
// sines it reads once, and issues all their loads first.
#include "rope.cuh"

#include "../../include/b2pa.h"
#include "ptx.cuh"

namespace b2pa {

namespace {

constexpr int kRopeThreads = 128;

enum RopeMode { kInterleaved, kHalvesInLane, kHalvesInSmem };

__device__ __forceinline__ void unpack8(uint4 v, float* f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float* f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void load_weight8(const RopeTensor& x, int d, float* w)
{
    if (x.weight_f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x.weight) + d);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
        unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x.weight) + d)), w);
    }
}

// kLanes: lanes per row, each holding two chunks of 8 elements.
template <RopeMode kMode, int kLanes, int kRows>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kGroups = kRopeThreads / kLanes;
    __shared__ float pair_rows[kMode == kHalvesInSmem ? kGroups * kLanes * 16 : 1];
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    // sets of kRows rows: those of the queries, then those of the keys
    const int sets_q = (p.x[0].heads + kRows - 1) / kRows, sets = sets_q + (p.x[1].heads + kRows - 1) / kRows;
    const unsigned long long id = (unsigned long long)blockIdx.x * kGroups + group;
    // (a 32-bit division where the number allows it)
    const long long t = id <= 0xFFFFFFFFull ? (long long)((unsigned)id / (unsigned)sets) : (long long)(id / sets);
    const bool on = t < p.T;  // every lane stays for the shuffles
    const int set = (int)((long long)id - t * sets);
    const bool is_k = set >= sets_q;
    const RopeTensor& x = p.x[is_k ? 1 : 0];
    const int h0 = (is_k ? set - sets_q : set) * kRows;
    const int half = p.R >> 1, chunks = p.D >> 3;

    // this lane's two chunks (-1: none) and whether its pairs rotate
    int ca = 2 * lane, cb = 2 * lane + 1;
    bool turns = 8 * ca < p.R;
    if (kMode == kHalvesInLane) {
        const int hc = half >> 3;  // chunks of one half
        turns = lane < hc;
        ca = turns ? lane : 2 * hc + 2 * (lane - hc);
        cb = turns ? lane + hc : ca + 1;
    }
    if (!on || ca >= chunks)
        ca = -1;
    if (!on || cb >= chunks)
        cb = -1;

    uint4 va[kRows], vb[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        va[r] = vb[r] = make_uint4(0u, 0u, 0u, 0u);
        if (h0 + r < x.heads) {
            const uint16_t* row = x.in + t * x.in_tok + (long long)(h0 + r) * x.in_head;
            if (ca >= 0)
                va[r] = *reinterpret_cast<const uint4*>(row + 8 * ca);
            if (cb >= 0)
                vb[r] = *reinterpret_cast<const uint4*>(row + 8 * cb);
        }
    }

    int pos[kRopeMaxAxes];
    bool ok = on;
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes; ++a) {
        pos[a] = 0;
        if (on && a < p.axes) {
            pos[a] = p.positions[a * p.pos_stride + t];
            if (pos[a] < 0 || pos[a] >= p.max_pos)
                ok = false;
        }
    }
    if (on && !ok && set == 0 && lane == 0)
        atomicOr(p.err, (unsigned)B2PA_DEV_BAD_POSITION);
    if (!ok)
        pos[0] = pos[1] = pos[2] = pos[3] = 0;
    auto place = [&](int axis) {
        return axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
    };
    auto entry = [&](int f) { return p.cos_sin + (long long)place(p.axis_of[f]) * p.cs_stride + f; };

    // cosines and sines of this lane's eight frequencies (pairs in one lane)
    float c[8], s[8];
    if (kMode != kHalvesInSmem) {
        const int f0 = 8 * lane;  // interleaved: elements 16 lane ..; halves: elements 8 lane .. of each half
        const int a8 = turns && f0 + 8 <= half ? p.axis_of8[lane] : 255;
        if (p.vec_table && a8 != 255) {
            const float* e = p.cos_sin + (long long)place(a8) * p.cs_stride + f0;
            const float4 c0 = __ldg(reinterpret_cast<const float4*>(e)), c1 = __ldg(reinterpret_cast<const float4*>(e) + 1);
            const float4 s0 = __ldg(reinterpret_cast<const float4*>(e + half)), s1 = __ldg(reinterpret_cast<const float4*>(e + half) + 1);
            c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
            s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = 1.f;
                s[i] = 0.f;
                if (turns && f0 + i < half) {
                    const float* e = entry(f0 + i);
                    c[i] = __ldg(e);
                    s[i] = __ldg(e + half);
                }
            }
        }
    }
    const bool norm = x.weight != nullptr;
    float wa[8], wb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        wa[i] = wb[i] = 1.f;
    if (norm && ca >= 0)
        load_weight8(x, 8 * ca, wa);
    if (norm && cb >= 0)
        load_weight8(x, 8 * cb, wb);

#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float a[8], b[8];
        unpack8(va[r], a);
        unpack8(vb[r], b);
        if (norm) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(sum / (float)p.D + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] *= inv * wa[i];
                b[i] *= inv * wb[i];
            }
        }
        if (kMode == kHalvesInLane) {
            if (turns) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = a[i], v = b[i];
                    a[i] = u * c[i] - v * s[i];
                    b[i] = v * c[i] + u * s[i];
                }
            }
        } else if (kMode == kInterleaved) {
            // a pair past R has c = 1, s = 0
            if (turns) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = a[2 * i], v = a[2 * i + 1], y = b[2 * i], z = b[2 * i + 1];
                    if (16 * lane + 2 * i < p.R) {
                        a[2 * i] = u * c[i] - v * s[i];
                        a[2 * i + 1] = v * c[i] + u * s[i];
                    }
                    if (16 * lane + 8 + 2 * i < p.R) {
                        b[2 * i] = y * c[4 + i] - z * s[4 + i];
                        b[2 * i + 1] = z * c[4 + i] + y * s[4 + i];
                    }
                }
            }
        } else {
            float* row = pair_rows + group * kLanes * 16;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                row[16 * lane + i] = a[i];
                row[16 * lane + 8 + i] = b[i];
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = 16 * lane + i;
                if (e < p.R && on) {
                    const int f = e < half ? e : e - half;
                    const float* cs = entry(f);
                    const float cc = __ldg(cs), ss = __ldg(cs + half);
                    const float u = row[e], v = row[e < half ? e + half : e - half];
                    const float y = e < half ? u * cc - v * ss : u * cc + v * ss;
                    if (i < 8)
                        a[i] = y;
                    else
                        b[i - 8] = y;
                }
            }
        }
        if (ok && h0 + r < x.heads) {
            uint16_t* row = x.out + t * x.out_tok + (long long)(h0 + r) * x.out_head;
            if (ca >= 0)
                *reinterpret_cast<uint4*>(row + 8 * ca) = pack8(a);
            if (cb >= 0)
                *reinterpret_cast<uint4*>(row + 8 * cb) = pack8(b);
        }
    }
}

template <RopeMode kMode, int kLanes, int kRows>
cudaError_t launch_rows(const RopeParams& p, cudaStream_t stream)
{
    constexpr int kGroups = kRopeThreads / kLanes;
    const long long sets = (p.x[0].heads + kRows - 1) / kRows + (p.x[1].heads + kRows - 1) / kRows;
    const long long blocks = (p.T * sets + kGroups - 1) / kGroups;
    if (blocks > 0x7FFFFFFFLL)
        return cudaErrorInvalidConfiguration;
    qk_norm_rope_kernel<kMode, kLanes, kRows><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <RopeMode kMode, int kLanes>
cudaError_t launch_lanes(const RopeParams& p, int sms, cudaStream_t stream)
{
    // four rows per group once one row per group would need more than one
    // wave of blocks (12 blocks of 128 threads fit an SM's registers)
    const long long groups = (long long)p.T * (p.x[0].heads + p.x[1].heads);
    const long long wave = (long long)sms * 12 * (kRopeThreads / kLanes);
    return groups > wave ? launch_rows<kMode, kLanes, 4>(p, stream) : launch_rows<kMode, kLanes, 1>(p, stream);
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
