// verify.cu -- which drafted nodes a target model accepts, and the token after
// them, from given random numbers.
//
// At an accepted node with target row p, draft row q and children c_1, c_2, ..
// (in the order of their numbers, tokens x_r drawn from q, independently):
//   R_1 = p, M_1 = 1
//   c_r is accepted if R_r(x_r) > 0 and u_r q(x_r) M_r < R_r(x_r)
//   else R_{r+1} = max(R_r - M_r q, 0), M_{r+1} = sum R_{r+1}
// where all R_r here are M_r times the distributions that the rule is about, so
// that nothing is divided.  R_{r+1} = max(p - a q, 0) with a = M_1 + .. + M_r: a
// refusal takes one pass over the rows p and q, with nothing kept from the pass
// before.  Without draft rows each child is a token that the draft chose for sure:
// q is 1 at x_r, so R_{r+1} is R_r with x_r left out, M_{r+1} = M_r - R_r(x_r), and
// no pass is needed.
// The path ends at a node none of whose children was accepted; the next token
// is the first i with R(0) + .. + R(i) > v sum R.
//
// What bounds it: the last node's row of V values is read once (p, and q where
// a child was refused), and every refusal that another child follows is a pass
// more, from L2; else it is latency.  Which token a random number picks depends on
// sums of V values to far more bits than fp32 has (a border between two of
// 131072 tokens is hit by an error of 2^-24 once in a hundred calls), and fp64
// is slow here (sums over threads in fp64 took half of the time, 5000 cycles for each
// pass), so that values and sums are pairs of floats, about 2^-46 exact.
//
// A cluster of CTAs per request: each goes over its part of the row, and they add
// up their sums through one another's shared memory.  All of them walk the tree,
// alike, so that nothing else has to be passed on.  8 nodes over 32000 tokens 6.9 us;
// 32 trees of up to 32 nodes over 131072 tokens 12.9 (four CTAs each 20.0, one of 512
// threads 53); 64 drawn trees, whose slowest has five passes, 27.2 (four CTAs 36.6; CTAs of
// 128 threads 35.0, of 512 34.5; two loads of a row in flight instead of four 33.2,
// eight 29.4).
#include "verify.cuh"

#include <cooperative_groups.h>

#include "../../include/b2pa.h"
#include "ptx.cuh"

namespace b2pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 128;  // values that a warp reads at once
constexpr int kMaxCtas = 8; // of a cluster

// A number as a sum of two floats, the first of which is the nearest to it: about
// 2^-47 exact.
struct Pair {
    float h = 0.f, l = 0.f;
    static __device__ __forceinline__ Pair of(float h, float l)  // |h| >= |l|
    {
        const float t = h + l;
        return Pair{t, l - (t - h)};
    }
    __device__ __forceinline__ Pair operator+(Pair b) const
    {
        const float t = h + b.h, z = t - h;
        return of(t, ((h - (t - z)) + (b.h - z)) + (l + b.l));
    }
    __device__ __forceinline__ Pair operator*(Pair b) const
    {
        const float t = h * b.h;
        return of(t, fmaf(h, b.h, -t) + fmaf(h, b.l, l * b.h));
    }
    __device__ __forceinline__ Pair operator-() const { return Pair{-h, -l}; }
    __device__ __forceinline__ bool operator<(Pair b) const { return h < b.h || (h == b.h && l < b.l); }
    __device__ __forceinline__ bool positive() const { return h > 0.f; }
    __device__ __forceinline__ Pair shfl_xor(int o) const
    {
        return Pair{__shfl_xor_sync(0xffffffffu, h, o), __shfl_xor_sync(0xffffffffu, l, o)};
    }
    __device__ __forceinline__ Pair shfl(int from) const
    {
        return Pair{__shfl_sync(0xffffffffu, h, from), __shfl_sync(0xffffffffu, l, from)};
    }
    // the sums of the lanes up to each one
    __device__ __forceinline__ Pair scan() const
    {
        Pair x = *this;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Pair y{__shfl_up_sync(0xffffffffu, x.h, o), __shfl_up_sync(0xffffffffu, x.l, o)};
            if ((int)(threadIdx.x & 31) >= o)
                x = y + x;
        }
        return x;
    }
};

// Two running sums: the floats, and what rounding took from them (exactly,
// whichever of the summands is larger).
struct Sums {
    float2 s = {0.f, 0.f}, c = {0.f, 0.f};
    __device__ __forceinline__ void add(float2 hi)
    {
        const float2 t = __fadd2_rn(s, hi), b = sub2(t, s);
        c = __fadd2_rn(c, __fadd2_rn(sub2(s, sub2(t, b)), sub2(hi, b)));
        s = t;
    }
    __device__ __forceinline__ void add(float2 hi, float2 lo)
    {
        add(hi);
        c = __fadd2_rn(c, lo);
    }
    __device__ __forceinline__ Pair value() const { return Pair::of(s.x, c.x) + Pair::of(s.y, c.y); }
    static __device__ __forceinline__ float2 sub2(float2 a, float2 b)
    {
        return __ffma2_rn(b, make_float2(-1.f, -1.f), a);
    }
};

// Negative values, infinities and NaN count as 0.
__device__ __forceinline__ float sane(float x) { return __float_as_uint(x) < 0x7F800000u ? x : 0.f; }
__device__ __forceinline__ float4 sane(float4 x) { return make_float4(sane(x.x), sane(x.y), sane(x.z), sane(x.w)); }

// max(p - a q, 0) as pairs; a = ah + al.
__device__ __forceinline__ void rest_of(float2 p, float2 q, float2 ah, float2 al, float2* hi, float2* lo)
{
    const float2 h = __fmul2_rn(ah, q);
    const float2 l = __ffma2_rn(al, q, __ffma2_rn(ah, q, make_float2(-h.x, -h.y)));  // a q = h + l
    const float2 d = Sums::sub2(p, h);
    const float2 e = Sums::sub2(Sums::sub2(Sums::sub2(p, d), h), l);  // (what is above 0 has p >= h - l)
    const float2 r = __fadd2_rn(d, e);
    *hi = make_float2(r.x > 0.f ? d.x : 0.f, r.y > 0.f ? d.y : 0.f);
    *lo = make_float2(r.x > 0.f ? e.x : 0.f, r.y > 0.f ? e.y : 0.f);
}

// What the threads of a request are to go over: a row, what is taken from it.
struct Pass {
    const float *p, *q;  // q: null where a = 0
    float ah, al;
    int outs;            // tokens left out (in shared memory)
    int last;            // the last pass: the token is wanted too
};

// Four values of a row from i on; beyond `end`: 0.
__device__ __forceinline__ float4 load4(const float* row, int i, int end, bool aligned)
{
    if (aligned && i + 4 <= end)
        return *reinterpret_cast<const float4*>(row + i);
    return make_float4(i < end ? row[i] : 0.f, i + 1 < end ? row[i + 1] : 0.f, i + 2 < end ? row[i + 2] : 0.f,
                       i + 3 < end ? row[i + 3] : 0.f);
}

// The four values R(i ..) from those of p and q.
template <bool kDraft>
__device__ __forceinline__ void rest4(const Pass& w, const int* out, bool outs, int i, float4 p4, float4 q4, float2 hi[2],
                                      float2 lo[2])
{
    p4 = sane(p4);
    hi[0] = make_float2(p4.x, p4.y);
    hi[1] = make_float2(p4.z, p4.w);
    lo[0] = lo[1] = make_float2(0.f, 0.f);
    if (kDraft) {
        q4 = sane(q4);
        const float2 ah = make_float2(w.ah, w.ah), al = make_float2(w.al, w.al);
        rest_of(hi[0], make_float2(q4.x, q4.y), ah, al, hi, lo);
        rest_of(hi[1], make_float2(q4.z, q4.w), ah, al, hi + 1, lo + 1);
    } else if (outs) {
        for (int o = 0; o < w.outs; ++o) {
            const int k = out[o] - i;
            hi[0].x = k == 0 ? 0.f : hi[0].x;
            hi[0].y = k == 1 ? 0.f : hi[0].y;
            hi[1].x = k == 2 ? 0.f : hi[1].x;
            hi[1].y = k == 3 ? 0.f : hi[1].y;
        }
    }
}

// Sum of R over values i, i + step, .. < end, four at a time, by one lane (end: the
// row's or a run's; `aligned`: rows can be read in 16-byte pieces).  All loads of a
// batch are under way together.
template <bool kDraft>
__device__ __forceinline__ Pair sum_rest(const Pass& w, const int* out, bool outs, int i, int end, int step, bool aligned)
{
    constexpr int kBatch = 4;
    Sums s[2];
    float2 hi[2], lo[2];
    if (aligned)
        for (; i + (kBatch - 1) * step + 4 <= end; i += kBatch * step) {
            float4 p4[kBatch], q4[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                p4[k] = *reinterpret_cast<const float4*>(w.p + i + k * step);
                q4[k] = kDraft ? *reinterpret_cast<const float4*>(w.q + i + k * step) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                rest4<kDraft>(w, out, outs, i + k * step, p4[k], q4[k], hi, lo);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    kDraft ? s[j].add(hi[j], lo[j]) : s[j].add(hi[j]);
            }
        }
    for (; i < end; i += step) {
        const float4 p4 = load4(w.p, i, end, aligned);
        const float4 q4 = kDraft ? load4(w.q, i, end, aligned) : make_float4(0.f, 0.f, 0.f, 0.f);
        rest4<kDraft>(w, out, outs, i, p4, q4, hi, lo);
        s[0].add(hi[0], lo[0]);
        s[1].add(hi[1], lo[1]);
    }
    return s[0].value() + s[1].value();
}

__device__ __forceinline__ Pair sum_rest(const Pass& w, const int* out, bool outs, int i, int end, int step, bool aligned)
{
    return w.q != nullptr ? sum_rest<true>(w, out, outs, i, end, step, aligned)
                          : sum_rest<false>(w, out, outs, i, end, step, aligned);
}

__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    extern __shared__ int nodes[];  // parents, tokens, left-out tokens, u, p and q at the tokens: [max_q] each
    __shared__ Pass pass;
    __shared__ Pair sums[kWarps];
    __shared__ Pair cta_sums[2][kMaxCtas];  // of this pass, and of the one before, which may still be read
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = (int)(blockIdx.x / (unsigned)ctas);
    int *par = nodes, *tok = par + p.max_q, *out = tok + p.max_q;
    float *u = reinterpret_cast<float*>(out + p.max_q), *pt = u + p.max_q, *qt = pt + p.max_q;
    if (ctas > 1)
        cluster.barrier_arrive();  // (awaited before CTAs write one another's shared memory: all have to be there)
    pdl_wait();
    const int q0 = p.cum_q[b], n = p.cum_q[b + 1] - q0;
    bool bad = n < 0 || n > p.max_q || q0 < 0 || q0 > p.T - n;
    int* acc = p.accepted + (long long)b * p.acc_st;
    if (rank == 0)
        for (int i = tid; i < p.width; i += kThreads)
            acc[i] = -1;
    if (!bad)
        for (int i = tid; i < n; i += kThreads) {
            const int up = i > 0 ? p.parents[q0 + i] : -1, t = p.tokens[q0 + i];
            par[i] = up;
            tok[i] = t;
            u[i] = p.uniforms[q0 + i];
            const bool in = up >= 0 && up < i && t >= 0 && t < p.V;
            bad = bad || (i > 0 && (up < 0 || up >= i));
            pt[i] = in ? sane(p.target[(long long)(q0 + up) * p.target_st + t]) : 0.f;
            qt[i] = in && p.draft != nullptr ? sane(p.draft[(long long)(q0 + up) * p.draft_st + t]) : 0.f;
        }
    bad = __syncthreads_or(bad);  // (and acc is filled)
    if (ctas > 1)
        cluster.barrier_wait();
    if (bad || n == 0) {
        if (tid == 0 && rank == 0) {
            p.counts[b] = 0;
            p.next[b] = -1;
            if (bad)
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
        }
        return;  // (all CTAs of the request do)
    }
    const float v = p.last[b];
    // the run of values of a warp, of the request's ctas * kWarps
    const int all_warps = ctas * kWarps;
    const int per = ((p.V + all_warps - 1) / all_warps + kTile - 1) / kTile * kTile;
    const int i0 = (int)min((long long)p.V, (long long)(rank * kWarps + warp) * per), i1 = min(p.V, i0 + per);
    // warp 0 walks; the others go over rows when it needs a sum
    int node = 0, at = 1, count = 1, outs = 0;  // the last accepted node, where its next child may be
    Pair a, mass{1.f, 0.f};
    bool from_p = false;  // nothing was left of the last row: it is taken whole
    if (tid == 0 && rank == 0)
        acc[0] = 0;
    for (int turn = 0;; turn ^= 1) {
        if (warp == 0) {
            bool ask = false;
            while (true) {
                // the next child of `node`
                int child = n;
                for (int i = at; i < n; i += 32) {
                    const unsigned m = __ballot_sync(0xffffffffu, i + lane < n && par[i + lane] == node);
                    if (m != 0) {
                        child = i + __ffs(m) - 1;
                        break;
                    }
                }
                at = child;
                if (child == n || ask)
                    break;
                bool yes;
                if (p.draft != nullptr) {
                    const Pair q{qt[child], 0.f}, r = Pair{pt[child], 0.f} + -(a * q);
                    yes = r.positive() && Pair{u[child], 0.f} * q * mass < r;
                } else {
                    bool twin = false;  // refused already
                    for (int i = lane; i < outs; i += 32)
                        twin = twin || out[i] == tok[child];
                    const Pair r{__any_sync(0xffffffffu, twin) ? 0.f : pt[child], 0.f};
                    yes = r.positive() && Pair{u[child], 0.f} * mass < r;
                    if (!yes) {
                        mass = mass + -r;
                        if (lane == 0)
                            out[outs] = tok[child];
                        ++outs;
                        __syncwarp();
                    }
                }
                at = child + 1;
                if (yes) {
                    node = child;
                    if (lane == 0 && rank == 0 && count < p.width)
                        acc[count] = node;
                    ++count;
                    a = Pair{};
                    mass = Pair{1.f, 0.f};
                    outs = 0;
                } else if (p.draft != nullptr && mass.positive()) {
                    a = a + mass;
                    ask = true;  // a sum, if another child follows
                }
            }
            if (lane == 0) {
                Pass w;
                w.p = p.target + (long long)(q0 + node) * p.target_st;
                w.q = a.positive() ? p.draft + (long long)(q0 + node) * p.draft_st : nullptr;
                w.ah = a.h;
                w.al = a.l;
                w.outs = outs;
                w.last = at >= n;
                pass = w;
            }
        }
        __syncthreads();
        const Pass w = pass;
        // R summed up
        bool here = false;
        for (int o = lane; o < w.outs; o += 32)
            here = here || (out[o] >= i0 && out[o] < i1);
        here = __any_sync(0xffffffffu, here);
        Pair mine = sum_rest(w, out, here, i0 + 4 * lane, i1, kTile, p.aligned);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mine = mine + mine.shfl_xor(o);
        if (lane == 0)
            sums[warp] = mine;
        __syncthreads();
        // sums up to this warp's run and its end, added in one order, so that one's
        // end is the next one's beginning
        Pair total, before, end;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            before = i == warp ? total : before;
            total = total + sums[i];
            end = i == warp ? total : end;
        }
        if (ctas > 1) {
            if (tid < ctas)
                *cluster.map_shared_rank(&cta_sums[turn][rank], tid) = total;  // to each of them
            cluster.sync();
            Pair all, below;
            for (int i = 0; i < ctas; ++i) {
                below = i == rank ? all : below;
                all = all + cta_sums[turn][i];
            }
            before = below + before;
            end = below + end;
            total = all;
        } else {
            __syncthreads();  // `sums` and `pass` have been read
        }
        if (!w.last) {
            mass = total;
            continue;
        }
        if (!total.positive() && !from_p) {
            from_p = true;  // (of every thread)
            a = Pair{};
            outs = 0;
            continue;
        }
        if (tid == 0 && rank == 0) {
            p.counts[b] = count;
            if (!total.positive()) {
                p.next[b] = -1;
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PROBS);
            }
        }
        // the warp in whose run the sum passes v times the whole (v = 1 is not allowed,
        // and takes the one in which it gets there)
        const Pair want = Pair{v > 0.f ? v : 0.f, 0.f} * total;
        if (total.positive() && (want < total ? !(want < before) && want < end : before < total && !(end < total))) {
            // a run of values for each lane; then one value each of the lucky lane's
            const int chunk = per / 32, c0 = i0 + lane * chunk, c1 = min(i1, c0 + chunk);
            const Pair own = sum_rest(w, out, here, c0, c1, 4, p.aligned), upto = before + own.scan();
            const unsigned over = __ballot_sync(0xffffffffu, own.positive() && want < upto);
            const unsigned some = __ballot_sync(0xffffffffu, own.positive());
            const int lucky = over != 0 ? __ffs(over) - 1 : max(31 - __clz(some), 0);
            Pair run = lucky > 0 ? upto.shfl(max(lucky - 1, 0)) : before;
            const int f0 = i0 + lucky * chunk, f1 = min(i1, f0 + chunk);
            int token = -1;
            for (int f = f0; f < f1; f += 32) {
                const int i = f + lane;
                const Pair r = i < f1 ? sum_rest(w, out, here, i, i + 1, 4, false) : Pair{};  // (one value)
                const Pair c = run + r.scan();
                const unsigned hit = __ballot_sync(0xffffffffu, r.positive() && want < c);
                const unsigned any = __ballot_sync(0xffffffffu, r.positive());
                if (hit != 0) {
                    token = f + __ffs(hit) - 1;
                    break;
                }
                if (any != 0)
                    token = f + 31 - __clz(any);  // in case that none passes
                run = c.shfl(31);
            }
            if (lane == 0)
                p.next[b] = token;
        }
        return;
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int sms, cudaStream_t stream)
{
    const size_t smem = (size_t)p.max_q * 6 * sizeof(int);
    // as many CTAs for a request as find a place at once (eight of 256 threads on an SM)
    int ctas = kMaxCtas;
    while (ctas > 1 && ((long long)p.B * ctas > 8LL * sms || p.V <= (ctas / 2) * kWarps * kTile))
        ctas /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kVerifyMaxNodes * 6 * (int)sizeof(int));
        if (e != cudaSuccess)
            return e;
    }
    return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace b2pa
