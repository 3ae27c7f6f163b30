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
// is slow here, so that values and sums are pairs of floats, about 2^-46 exact,
// and fp64 is left to sums over threads.
#include "verify.cuh"

#include "../../include/b2pa.h"
#include "ptx.cuh"

namespace b2pa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 128;  // values that a warp reads at once

// A sum of values >= 0, as a pair: the float and what rounding took from it.
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float hi, float lo)
    {
        const float t = s + hi, big = fmaxf(s, hi), small = fminf(s, hi);
        c += (small - (t - big)) + lo;
        s = t;
    }
    __device__ __forceinline__ double value() const { return (double)s + (double)c; }
};

// Negative values, infinities and NaN count as 0.
__device__ __forceinline__ float sane(float x) { return x > 0.f && x <= 3.402823466e38f ? x : 0.f; }

// max(p - a q, 0) as a pair; a = ah + al.
__device__ __forceinline__ void rest_of(float p, float q, float ah, float al, float* hi, float* lo)
{
    const float h = ah * q, l = fmaf(al, q, fmaf(ah, q, -h));  // a q = h + l
    const float d = p - h;
    const float e = ((p - d) - h) - l;  // (what is above 0 has p >= h - l)
    const bool on = d + e > 0.f;
    *hi = on ? d : 0.f;
    *lo = on ? e : 0.f;
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

// The four values R(i ..) of a lane.
__device__ __forceinline__ void rest4(const Pass& w, const int* out, bool outs, int i, int end, bool aligned, float hi[4],
                                      float lo[4])
{
    const float4 p4 = load4(w.p, i, end, aligned);
    const float p[4] = {p4.x, p4.y, p4.z, p4.w};
    if (w.q != nullptr) {
        const float4 q4 = load4(w.q, i, end, aligned);
        const float q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            rest_of(sane(p[k]), sane(q[k]), w.ah, w.al, hi + k, lo + k);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        hi[k] = sane(p[k]);
        lo[k] = 0.f;
    }
    if (outs)
        for (int o = 0; o < w.outs; ++o)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (out[o] == i + k)
                    hi[k] = 0.f;
}

__device__ __forceinline__ double warp_sum(double x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p)
{
    extern __shared__ int nodes[];  // parents, tokens, left-out tokens, u, p and q at the tokens: [max_q] each
    __shared__ Pass pass;
    __shared__ double sums[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
    int *par = nodes, *tok = par + p.max_q, *out = tok + p.max_q;
    float *u = reinterpret_cast<float*>(out + p.max_q), *pt = u + p.max_q, *qt = pt + p.max_q;
    pdl_wait();
    const int q0 = p.cum_q[b], n = p.cum_q[b + 1] - q0;
    bool bad = n < 0 || n > p.max_q || q0 < 0 || q0 > p.T - n;
    int* acc = p.accepted + (long long)b * p.acc_st;
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
    if (bad || n == 0) {
        if (tid == 0) {
            p.counts[b] = 0;
            p.next[b] = -1;
            if (bad)
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
        }
        return;
    }
    // warp 0 walks; the others go over rows when it needs a sum
    int node = 0, at = 1, count = 1, outs = 0;  // the last accepted node, where its next child may be
    double a = 0., mass = 1.;
    bool from_p = false;  // nothing was left of the last row: it is taken whole
    if (warp == 0 && lane == 0)
        acc[0] = 0;
    while (true) {
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
                    const double r = (double)pt[child] - a * (double)qt[child];
                    yes = r > 0. && (double)u[child] * (double)qt[child] * mass < r;
                } else {
                    bool twin = false;  // refused already
                    for (int i = lane; i < outs; i += 32)
                        twin = twin || out[i] == tok[child];
                    const double r = __any_sync(0xffffffffu, twin) ? 0. : (double)pt[child];
                    yes = r > 0. && (double)u[child] * mass < r;
                    if (!yes) {
                        mass -= r;
                        if (lane == 0)
                            out[outs] = tok[child];
                        ++outs;
                        __syncwarp();
                    }
                }
                at = child + 1;
                if (yes) {
                    node = child;
                    if (lane == 0 && count < p.width)
                        acc[count] = node;
                    ++count;
                    a = 0.;
                    mass = 1.;
                    outs = 0;
                } else if (p.draft != nullptr && mass > 0.) {
                    a += mass;
                    ask = true;  // a sum, if another child follows
                }
            }
            if (lane == 0) {
                Pass w;
                w.p = p.target + (long long)(q0 + node) * p.target_st;
                w.q = a > 0. ? p.draft + (long long)(q0 + node) * p.draft_st : nullptr;
                w.ah = (float)a;
                w.al = (float)(a - (double)w.ah);
                w.outs = outs;
                w.last = at >= n;
                pass = w;
            }
        }
        __syncthreads();
        const Pass w = pass;
        // R summed up: a run of values for each warp
        const int per = ((p.V + kWarps - 1) / kWarps + kTile - 1) / kTile * kTile;
        const int i0 = min(p.V, warp * per), i1 = min(p.V, i0 + per);
        bool here = false;
        for (int o = lane; o < w.outs; o += 32)
            here = here || (out[o] >= i0 && out[o] < i1);
        here = __any_sync(0xffffffffu, here);
        Sum s;
#pragma unroll 4
        for (int i = i0 + 4 * lane; i < i1; i += kTile) {
            float hi[4], lo[4];
            rest4(w, out, here, i, i1, p.aligned, hi, lo);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s.add(hi[k], lo[k]);
        }
        const double mine = warp_sum(s.value());
        if (lane == 0)
            sums[warp] = mine;
        __syncthreads();
        double total = 0., before = 0.;
        for (int i = 0; i < kWarps; ++i) {
            before += i < warp ? sums[i] : 0.;
            total += sums[i];
        }
        __syncthreads();  // `sums` and `pass` have been read
        if (!w.last) {
            mass = total;
            continue;
        }
        if (!(total > 0.) && !from_p) {
            from_p = true;  // (of every thread)
            a = 0.;
            outs = 0;
            continue;
        }
        if (tid == 0) {
            p.counts[b] = count;
            if (!(total > 0.)) {
                p.next[b] = -1;
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PROBS);
            }
        }
        // the warp in whose run the sum passes v times the whole
        const double v = p.last[b], want = (v > 0. ? v : 0.) * total;
        int lucky = kWarps;
        double sum = 0.;
        int positive = -1;
        for (int i = 0; i < kWarps; ++i) {
            sum += sums[i];
            if (sums[i] > 0.)
                positive = i;
            if (lucky == kWarps && sum > want)
                lucky = i;
        }
        if (lucky == kWarps)
            lucky = positive;  // v is 1, nearly or more
        if (warp != lucky)
            return;
        double run = before;
        int token = -1;
        for (int j = i0; j < i1; j += kTile) {
            float hi[4], lo[4];
            rest4(w, out, here, j + 4 * lane, i1, p.aligned, hi, lo);
            double r[4], mine4 = 0.;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                r[k] = (double)hi[k] + (double)lo[k];
                mine4 += r[k];
            }
            double upto = mine4;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, upto, o);
                upto += lane >= o ? y : 0.;
            }
            // a lane's first value that passes; its last positive one
            double c = run + upto - mine4;
            int first = -1, final_ = -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                c += r[k];
                if (r[k] > 0.) {
                    final_ = j + 4 * lane + k;
                    if (first < 0 && c > want)
                        first = final_;
                }
            }
            const unsigned hit = __ballot_sync(0xffffffffu, first >= 0), any = __ballot_sync(0xffffffffu, final_ >= 0);
            if (hit != 0) {
                token = __shfl_sync(0xffffffffu, first, __ffs(hit) - 1);
                break;
            }
            if (any != 0)
                token = __shfl_sync(0xffffffffu, final_, 31 - __clz(any));  // in case that none passes
            run += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0)
            p.next[b] = token;
        return;
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int sms, cudaStream_t stream)
{
    (void)sms;
    const size_t smem = (size_t)p.max_q * 6 * sizeof(int);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kVerifyMaxNodes * 6 * (int)sizeof(int));
        if (e != cudaSuccess)
            return e;
    }
    return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace b2pa
