// From logits to the tokens that count: probabilities of a row of logits, and
// the verification of drafted tokens with the draw of the next one.
#include <stdint.h>

#include "ssd_layer_device.h"
#include "ssd_step.h"

namespace ssd {

// ---------------------------------------------------------------------------
// Probabilities.

struct Peak {
    float m;    // the largest logit so far (-infinity: none)
    float s;    // sum of exp((x - m) / T)
    int at;     // first place of the largest
};

// exp(d / T) of d <= 0, with c = log2(e) / T in two parts: the product's
// rounding, which would be d 2^-24 in the exponent, is put back.
struct InvTemp {
    float hi, lo;
    __device__ __forceinline__ explicit InvTemp(float t) {
        const double c = 1.4426950408889634 / (double)t;
        hi = (float)c;
        lo = (float)(c - (double)hi);
        if (!(fabsf(hi) < __builtin_inff())) lo = 0.0f;
    }
    __device__ __forceinline__ float operator()(float d) const {
        const float y = d * hi;
        const float rest = fmaf(d, hi, -y) + d * lo;
        const float e = __builtin_amdgcn_exp2f(y);
        const float r = e + e * (rest * kLn2);
        return fabsf(y) < 1000.0f ? r : e;
    }
};

template <typename T>
__global__ __launch_bounds__(1024) void probs_kernel(int V, int per_req, const T *__restrict__ logits,
                                                     int64_t ls, const float *__restrict__ temperature,
                                                     float *__restrict__ probs, int64_t ps)
{
    __shared__ Peak part[16];
    const int64_t row = blockIdx.x;
    const T *const x = logits + row * ls;
    float *const p = probs + row * ps;
    const float t = temperature ? temperature[row / per_req] : 1.0f;
    const bool greedy = !(t > 0.0f);
    const InvTemp inv(greedy ? 1.0f : t);
    Peak k{-__builtin_inff(), 0.0f, V};
    for (int i = (int)threadIdx.x; i < V; i += 1024) {
        const float v = to_f32(x[i]);
        if (v > k.m) {
            k.m = v;
            k.at = i;
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const float m = __shfl_xor(k.m, off, kWave);
        const int at = __shfl_xor(k.at, off, kWave);
        if (m > k.m || (m == k.m && at < k.at)) {
            k.m = m;
            k.at = at;
        }
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = k;
    __syncthreads();
    for (int i = 0; i < 16; ++i) {
        const Peak o = part[i];
        if (o.m > k.m || (o.m == k.m && o.at < k.at)) k = o;
    }
    __syncthreads();
    if (greedy) {
        for (int i = (int)threadIdx.x; i < V; i += 1024) p[i] = i == k.at ? 1.0f : 0.0f;
        return;
    }
    const float top = k.m == -__builtin_inff() ? 0.0f : k.m;
    float s = 0.0f;
    for (int i = (int)threadIdx.x; i < V; i += 1024) {
        const float v = to_f32(x[i]);
        s += v == -__builtin_inff() ? 0.0f : inv(v - top);
    }
    s = group_sum(s, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6].s = s;
    __syncthreads();
    s = 0.0f;
    for (int i = 0; i < 16; ++i) s += part[i].s;
    const float r = s == 0.0f ? 0.0f : 1.0f / s;
    for (int i = (int)threadIdx.x; i < V; i += 1024) {
        const float v = to_f32(x[i]);
        p[i] = v == -__builtin_inff() ? 0.0f * s : inv(v - top) * r;
    }
}

size_t probs_workspace(const ProbsDims &) { return 0; }

void launch_probs(const ProbsDims &d, const void *logits, const float *temperature, float *probs,
                  void *, void *stream)
{
    const int rows = d.R * d.T;
    if (rows <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d.bf16)
        hipLaunchKernelGGL(probs_kernel<bf16>, dim3((unsigned)rows), dim3(1024), 0, st, d.V, d.T,
                           static_cast<const bf16 *>(logits), d.ls, temperature, probs, d.ps);
    else
        hipLaunchKernelGGL(probs_kernel<float>, dim3((unsigned)rows), dim3(1024), 0, st, d.V, d.T,
                           static_cast<const float *>(logits), d.ls, temperature, probs, d.ps);
}

// ---------------------------------------------------------------------------
// Verification.
//
// Float32 probabilities make everything behind them exact enough that a token
// does not hang on the order of a sum: u q has 48 bits, p - q at most a few
// more than 53, and a sum of V of them in 64 bits is off by 2^-53 of itself a
// step, far less than the distance of a uniform number of 24 bits from a
// border that it does not lie on.
//
// Two launches: the weights of each segment of 4096 entries are summed (one
// block a segment and request), then one block a request finds the segment
// that the draw falls into and goes through its entries. Bound by the rows'
// bytes, for few requests by the chain draft -> its probabilities -> row.

constexpr int kSeg = 4096, kSegThreads = 256, kPerThread = kSeg / kSegThreads;

struct Decision {
    int count, accepted;     // drafts of the request, and how many of them stand
};

// Every wave of the block comes to the same answer: lane i tests draft i.
__device__ __forceinline__ Decision decide(const VerifyDims &d, const VerifyArgs &a, int r) {
    const int lane = threadIdx.x & 63, most = d.T - 1;
    int n = a.count ? a.count[r] : most;
    n = n < 0 ? 0 : (n > most ? most : n);
    bool ok = false;
    if (lane < n) {
        const int tok = a.tokens[(int64_t)r * most + lane];
        if (tok >= 0 && tok < d.V) {
            const float p = a.target[((int64_t)r * d.T + lane) * d.ts + tok];
            const float q = a.draft ? a.draft[((int64_t)r * most + lane) * d.ds + tok] : 1.0f;
            const float u = a.uniform[(int64_t)r * d.T + lane];
            // (an exact product; a draft probability that counts as zero is zero)
            ok = (double)u * (double)(q > 0.0f ? q : 0.0f) < (double)p;
        }
    }
    const uint64_t no = ~__ballot(ok);
    const int first = no ? __ffsll((unsigned long long)no) - 1 : 64;
    return Decision{n, first < n ? first : n};
}

// What the entry v of the next token's row weighs: w against the draft, and p.
struct Row {
    const float *p, *q;
    int gone;                // the certain draft that was turned down (-1: none)
    __device__ __forceinline__ Row(const VerifyDims &d, const VerifyArgs &a, int r, Decision k) {
        const int most = d.T - 1;
        const bool cut = k.accepted < k.count;
        p = a.target + ((int64_t)r * d.T + k.accepted) * d.ts;
        q = cut && a.draft ? a.draft + ((int64_t)r * most + k.accepted) * d.ds : nullptr;
        gone = cut && !a.draft ? a.tokens[(int64_t)r * most + k.accepted] : -1;
    }
    __device__ __forceinline__ void weigh(int v, float pv, float qv, double &w, double &plain) const {
        const double pd = pv > 0.0f ? (double)pv : 0.0;
        const double left = pd - (qv > 0.0f ? (double)qv : 0.0);
        plain = pd;
        w = v == gone || !(left > 0.0) ? 0.0 : left;
    }
};

__device__ __forceinline__ double shfl_xor64(double v, int off) { return __shfl_xor(v, off, kWave); }

__global__ __launch_bounds__(kSegThreads) void verify_sums_kernel(VerifyDims d, VerifyArgs a, int segs,
                                                                  double *__restrict__ sums)
{
    __shared__ double part[2][kSegThreads / 64];
    const int seg = blockIdx.x, r = blockIdx.y;
    const Decision k = decide(d, a, r);
    const Row row(d, a, r, k);
    double sw = 0.0, sp = 0.0;
    for (int j = 0; j < kPerThread; ++j) {
        const int v = seg * kSeg + j * kSegThreads + (int)threadIdx.x;
        if (v < d.V) {
            double w, p;
            row.weigh(v, row.p[v], row.q ? row.q[v] : 0.0f, w, p);
            sw += w;
            sp += p;
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        sw += shfl_xor64(sw, off);
        sp += shfl_xor64(sp, off);
    }
    if ((threadIdx.x & 63) == 0) {
        part[0][threadIdx.x >> 6] = sw;
        part[1][threadIdx.x >> 6] = sp;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double s = 0.0;
        for (int i = 0; i < kSegThreads / 64; ++i) s += part[threadIdx.x][i];
        sums[((int64_t)r * segs + seg) * 2 + threadIdx.x] = s;
    }
    if (seg == 0) {
        if (threadIdx.x == 0) a.accepted[r] = k.accepted;
        for (int i = (int)threadIdx.x; i < d.T; i += kSegThreads)
            if (i != k.accepted)
                a.out[(int64_t)r * d.T + i] = i < k.accepted ? a.tokens[(int64_t)r * (d.T - 1) + i] : -1;
    }
}

__global__ __launch_bounds__(kSegThreads) void verify_pick_kernel(VerifyDims d, VerifyArgs a, int segs,
                                                                  const double *__restrict__ sums)
{
    __shared__ double incl[kSegThreads];
    __shared__ int found, last;
    const int r = blockIdx.x, tid = threadIdx.x;
    const Decision k = decide(d, a, r);
    const Row row(d, a, r, k);
    const double *const s = sums + (int64_t)r * segs * 2;
    // every thread adds the segments up in the same order
    double tw = 0.0, tp = 0.0;
    for (int i = 0; i < segs; ++i) {
        tw += s[2 * i];
        tp += s[2 * i + 1];
    }
    const int which = tw > 0.0 ? 0 : 1;
    const double total = which ? tp : tw, want = total * (double)a.uniform[(int64_t)r * d.T + d.T - 1];
    double before = 0.0;
    int seg = -1;
    double seg_before = 0.0;
    for (int i = 0; i < segs; ++i) {
        const double w = s[2 * i + which];
        if (w > 0.0) {                       // (the last one of positive weight, if none passes)
            seg = i;
            seg_before = before;
            if (before + w > want) break;
        }
        before += w;
    }
    int token = -1;
    if (seg >= 0) {                          // (the same in every thread)
        double w[kPerThread], mine = 0.0;
        const int v0 = seg * kSeg + tid * kPerThread;
        int lastpos = -1;
#pragma unroll
        for (int j = 0; j < kPerThread; ++j) {
            const int v = v0 + j;
            double x = 0.0, p = 0.0;
            if (v < d.V) row.weigh(v, row.p[v], row.q ? row.q[v] : 0.0f, x, p);
            w[j] = which ? p : x;
            mine += w[j];
            if (w[j] > 0.0) lastpos = v;
        }
        if (tid == 0) {
            found = 0x7fffffff;
            last = -1;
        }
        incl[tid] = mine;
        __syncthreads();
        for (int off = 1; off < kSegThreads; off <<= 1) {
            const double o = tid >= off ? incl[tid - off] : 0.0;
            __syncthreads();
            incl[tid] += o;
            __syncthreads();
        }
        double c = seg_before + (tid ? incl[tid - 1] : 0.0);
        int hit = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < kPerThread; ++j) {
            c += w[j];
            if (w[j] > 0.0 && c > want && hit == 0x7fffffff) hit = v0 + j;
        }
        if (hit != 0x7fffffff) atomicMin(&found, hit);
        if (lastpos >= 0) atomicMax(&last, lastpos);
        __syncthreads();
        token = found != 0x7fffffff ? found : last;
    }
    if (tid == 0) a.out[(int64_t)r * d.T + k.accepted] = token;
}

static int segments(const VerifyDims &d) { return (d.V + kSeg - 1) / kSeg; }
size_t verify_workspace(const VerifyDims &d) { return (size_t)d.R * segments(d) * 2 * sizeof(double); }

void launch_verify(const VerifyDims &d, const VerifyArgs &a, void *workspace, void *stream)
{
    if (d.R <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const int segs = segments(d);
    double *const sums = static_cast<double *>(workspace);
    hipLaunchKernelGGL(verify_sums_kernel, dim3((unsigned)segs, (unsigned)d.R), dim3(kSegThreads), 0, st, d, a,
                       segs, sums);
    hipLaunchKernelGGL(verify_pick_kernel, dim3((unsigned)d.R), dim3(kSegThreads), 0, st, d, a, segs, sums);
}

}  // namespace ssd
