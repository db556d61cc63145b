// From logits to the tokens that count: probabilities of a row of logits, and
// the verification of drafted tokens with the draw of the next one.
#include <stdint.h>

#include "ssd_layer_device.h"
#include "ssd_step.h"

namespace ssd {

// ---------------------------------------------------------------------------
// Probabilities.

// A row (short ones) or a part of a row by one block, its logits kept in
// registers from their only load. A row that one block cannot hold is cut into
// parts: the first launch leaves each part's largest logit and sum, the second
// joins them and writes. Bound by the bytes of logits (in parts read twice, the
// second time from the last-level cache as far as it holds them) and
// probabilities: 4096 rows of 32000 bfloat16 156 us, 5.0 TB/s; 384 of 131072 85 us as a pass
// among others, 3.6 TB/s of what has to be moved, and 74 on inputs that the last pass left in the
// last-level cache.
struct Peak {
    float m;    // the largest logit (-infinity: none)
    float s;    // sum of exp((x - m) / T)
    int at;     // first place of the largest
    int pad;
};
__device__ __forceinline__ void take_larger(Peak &k, float m, int at) {
    if (m > k.m || (m == k.m && at < k.at)) {
        k.m = m;
        k.at = at;
    }
}

// exp(d / T) of d <= 0, with c = log2(e) / T in two parts: the product's
// rounding, which would be d 2^-24 in the exponent, is put back.
struct InvTemp {
    float hi, lo, far;      // far: a d whose exponential is zero, and so is that of all below it
    __device__ __forceinline__ explicit InvTemp(float t) {
        const double c = 1.4426950408889634 / (double)t;
        hi = c < 3.0e38 ? (float)c : 3.0e38f;          // (a difference of 0 times infinity is no number)
        lo = c < 3.0e38 ? (float)(c - (double)hi) : 0.0f;
        far = -300.0f / hi;
    }
    // (else the largest float is nearer than `far`, and masked logits are looked for one by one)
    __device__ __forceinline__ bool usual() const { return hi > 1.0e-36f; }
    // exp(d / T) for a sum: off by the exponent's rounding, d / T 2^-24 of itself, which over a row's
    // probabilities comes to at most the logarithm of their number times 2^-24 (their entropy's bound)
    __device__ __forceinline__ float summand(float d) const {
        d = fmaxf(d, far);
        return __builtin_amdgcn_exp2f(fmaf(d, hi, d * lo));
    }
    // exp(d / T) = e (1 + rest ln 2); a d that is NaN or -infinity has e = 0
    __device__ __forceinline__ float split(float d, float &rest) const {
        d = fmaxf(d, far);
        const float y = d * hi;
        rest = fmaf(d, lo, fmaf(d, hi, -y));
        return __builtin_amdgcn_exp2f(y);
    }
    // exp((v - top) / T) of v that is not -infinity, at any T (the halves' difference is a float where
    // v - top is past the largest, and at temperatures that are not usual their exponential counts)
    __device__ __forceinline__ float operator()(float v, float top) const {
        const float d = 0.5f * v - 0.5f * top, y = 2.0f * (d * hi);
        const float rest = 2.0f * (fmaf(d, hi, -0.5f * y) + d * lo);
        const float e = __builtin_amdgcn_exp2f(y);
        return y > -1000.0f ? fmaf(e, rest * kLn2, e) : e;      // (NaN passes through e)
    }
};

// A thread's N vectors of 16 bytes, `threads` vectors apart; elements past the row's end are
// -infinity. Rows start on their element.
template <typename T, int N> struct Logits {
    static constexpr int E = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(E)));
    typedef vec any __attribute__((aligned(sizeof(T))));
    vec v[N];
    __device__ __forceinline__ void load(const T *x, int from, int end, int threads) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = from + (j * threads + (int)threadIdx.x) * E;
            if (i + E <= end) v[j] = *reinterpret_cast<const any *>(x + i);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) v[j][e] = i + e < end ? x[i + e] : from_f32<T>(-__builtin_inff());
        }
    }
    // (unpacked by hand: the compiler rounds a maximum of widened bfloat16 back to bfloat16 and widens it again)
    __device__ __forceinline__ float at(int j, int e) const {
        if constexpr (sizeof(T) == 4) return v[j][e];
        else {
            typedef uint32_t words __attribute__((ext_vector_type(4)));
            const uint32_t w = __builtin_bit_cast(words, v[j])[e / 2];
            return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
        }
    }
    template <typename F> __device__ __forceinline__ void each(int from, int threads, F f) const {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) f(from + (j * threads + (int)threadIdx.x) * E + e, at(j, e));
    }
};

__device__ __forceinline__ float wave_max(float v) {
    v = larger(v, dpp<0xb1>(v));       // quad_perm [1,0,3,2]
    v = larger(v, dpp<0x4e>(v));       // quad_perm [2,3,0,1]
    v = larger(v, dpp<0x141>(v));      // row_half_mirror
    v = larger(v, dpp<0x140>(v));      // row_mirror
    return across32(across16(v, larger), larger);
}

// The part's peak and sum, the same in every thread of the block. Vector work next to the loads: of
// rows whose place of the largest nobody asks for, maxima alone (3 logits an instruction, NaN kept), and
// no look at masked logits (16 rows of 131072 bfloat16 12.8 -> 10.0 us, 384 of them 82.8 -> 79.3).
template <typename T, int N, int W>
__device__ __forceinline__ Peak block_peak(const Logits<T, N> &l, int from, const InvTemp &inv, bool greedy) {
    __shared__ Peak part[W];
    __shared__ float sums[W];
    const bool usual = !greedy && inv.usual();              // (the same in the block)
    const int wave = (int)threadIdx.x >> 6, lane = threadIdx.x & 63;
    Peak k{-__builtin_inff(), 0.0f, 0x7fffffff, 0};
    float own = -__builtin_inff();
    if (usual) {
        l.each(from, 64 * W, [&](int, float v) { own = __builtin_elementwise_maximum(own, v); });
        k.m = wave_max(own);
    } else {
        l.each(from, 64 * W, [&](int i, float v) {
            // (places rise: an equal one later does not replace)
            k.at = v > k.m ? i : k.at;
            k.m = v > k.m ? v : k.m;
        });
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) take_larger(k, __shfl_xor(k.m, off, kWave), __shfl_xor(k.at, off, kWave));
    }
    if (lane == 0) part[wave] = k;
    __syncthreads();
    k = Peak{-__builtin_inff(), 0.0f, 0x7fffffff, 0};
#pragma unroll
    for (int i = 0; i < W; ++i) take_larger(k, part[i].m, part[i].at);
    const float top = k.m == -__builtin_inff() ? 0.0f : k.m;
    float s = 0.0f;
    if (usual) {
        l.each(from, 64 * W, [&](int, float v) { s += inv.summand(v - top); });
        // (a logit of NaN or +infinity makes the sum NaN)
        s += own == -__builtin_inff() ? 0.0f : own - own;
    } else
        l.each(from, 64 * W, [&](int, float v) { s += v == -__builtin_inff() ? 0.0f : inv(v, top); });
    s = group_sum(s, 64);
    if (lane == 0) sums[wave] = s;
    __syncthreads();
    k.s = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) k.s += sums[i];
    return k;
}

template <typename T, int N, int W>
__device__ __forceinline__ void write_probs(const Logits<T, N> &l, int from, int end, const Peak &k, bool greedy,
                                            const InvTemp &inv, float *p) {
    constexpr int E = Logits<T, N>::E;
    typedef float vec4 __attribute__((ext_vector_type(4)));
    typedef vec4 any4 __attribute__((aligned(4)));
    const float top = k.m == -__builtin_inff() ? 0.0f : k.m, r = k.s == 0.0f ? 0.0f : 1.0f / k.s;
    const float none = 0.0f * k.s;                  // what a masked logit gets: 0, or NaN with its row
    const bool usual = !greedy && inv.usual();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int i = from + (j * 64 * W + (int)threadIdx.x) * E;
        float y[E];
        if (usual)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float rest;
                const float p1 = inv.split(l.at(j, e) - top, rest) * r;
                y[e] = fmaf(p1, rest * kLn2, p1);
            }
        else
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float v = l.at(j, e);
                y[e] = greedy ? (i + e == k.at ? 1.0f : 0.0f) : v == -__builtin_inff() ? none : inv(v, top) * r;
            }
        if (i + E <= end)
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const vec4 o = {y[e], y[e + 1], y[e + 2], y[e + 3]};
                *reinterpret_cast<any4 *>(p + i + e) = o;
            }
        else
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (i + e < end) p[i + e] = y[e];
    }
}

// STEP 0: whole rows; 1: the parts' peaks; 2: parts joined and written.
template <typename T, int N, int W, int STEP>
__global__ __launch_bounds__(64 * W, W == 8 ? 4 : 1) void probs_kernel(int V, int per_req, const T *__restrict__ logits, int64_t ls,
                                                       const float *__restrict__ temperature,
                                                       float *__restrict__ probs, int64_t ps, int parts,
                                                       Peak *__restrict__ peaks)
{
    constexpr int SPAN = 64 * W * Logits<T, N>::E * N;
    const int part = STEP == 0 ? 0 : (int)blockIdx.x % parts;
    const int64_t row = STEP == 0 ? blockIdx.x : blockIdx.x / parts;
    const int from = part * SPAN, end = V - from < SPAN ? V : from + SPAN;
    Logits<T, N> l;
    l.load(logits + row * ls, from, end, 64 * W);
    const float t = temperature ? temperature[row / per_req] : 1.0f;
    const bool greedy = !(t > 0.0f);
    const InvTemp inv(greedy ? 1.0f : t);
    Peak k;
    if constexpr (STEP < 2) {
        k = block_peak<T, N, W>(l, from, inv, greedy);
        if constexpr (STEP == 1) {
            if (threadIdx.x == 0) peaks[blockIdx.x] = k;
            return;
        }
    } else {
        // every wave joins the row's parts by itself
        const int lane = threadIdx.x & 63;
        const Peak *const mine = peaks + row * parts;
        k = Peak{-__builtin_inff(), 0.0f, 0x7fffffff, 0};
        for (int i = lane; i < parts; i += 64) take_larger(k, mine[i].m, mine[i].at);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) take_larger(k, __shfl_xor(k.m, off, kWave), __shfl_xor(k.at, off, kWave));
        float s = 0.0f;
        for (int i = lane; i < parts; i += 64) {
            const Peak o = mine[i];
            s += o.m == -__builtin_inff() ? o.s : o.s * inv(o.m, k.m);
        }
        k.s = group_sum(s, 64);
    }
    write_probs<T, N, W>(l, from, end, k, greedy, inv, probs + row * ps);
}

// Rows of up to 16 K logits (bfloat16: 32 K) are taken whole, others in parts of 4 K (8 K): 512 rows
// of 32000 bfloat16 26 us whole and 33 in parts, of 50257 52 and 48; 1024 of 34000 79 and 58.
template <typename T> static constexpr int probs_span() { return 256 * Logits<T, 4>::E * 4; }
static int probs_parts(const ProbsDims &d) {
    const int span = d.bf16 ? probs_span<bf16>() : probs_span<float>();
    return d.V <= 4 * span ? 0 : (d.V + span - 1) / span;
}
size_t probs_workspace(const ProbsDims &d) { return (size_t)d.R * d.T * probs_parts(d) * sizeof(Peak); }

template <typename T>
static void probs_t(const ProbsDims &d, const void *logits, const float *temperature, float *probs, Peak *peaks,
                    hipStream_t st)
{
    const unsigned rows = (unsigned)(d.R * d.T);
    const T *const x = static_cast<const T *>(logits);
    constexpr int E = Logits<T, 1>::E;
    const int parts = probs_parts(d);
    if (parts) {
        hipLaunchKernelGGL((probs_kernel<T, 4, 4, 1>), dim3(rows * parts), dim3(256), 0, st, d.V, d.T, x, d.ls,
                           temperature, probs, d.ps, parts, peaks);
        hipLaunchKernelGGL((probs_kernel<T, 4, 4, 2>), dim3(rows * parts), dim3(256), 0, st, d.V, d.T, x, d.ls,
                           temperature, probs, d.ps, parts, peaks);
    } else {
        // (few threads with many logits each: they share a sum and a maximum, which costs the same for
        // 256 threads and 1024, and leave less of a row's end idle; 4096 rows of 4000 bfloat16 24 us, of
        // 8000 44, and 77 and 80 by 1024 threads)
        auto whole = [&](auto N, auto W) {
            hipLaunchKernelGGL((probs_kernel<T, decltype(N)::value, decltype(W)::value, 0>), dim3(rows),
                               dim3(64 * decltype(W)::value), 0, st, d.V, d.T, x, d.ls, temperature, probs, d.ps, 1, peaks);
        };
        using std::integral_constant;
        if (d.V <= 256 * E) whole(integral_constant<int, 1>{}, integral_constant<int, 4>{});
        else if (d.V <= 512 * E) whole(integral_constant<int, 2>{}, integral_constant<int, 4>{});
        else if (d.V <= 1024 * E) whole(integral_constant<int, 4>{}, integral_constant<int, 4>{});
        else if (d.V <= 2048 * E) whole(integral_constant<int, 4>{}, integral_constant<int, 8>{});
        else whole(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    }
}

void launch_probs(const ProbsDims &d, const void *logits, const float *temperature, float *probs,
                  void *workspace, void *stream)
{
    if ((int64_t)d.R * d.T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d.bf16) probs_t<bf16>(d, logits, temperature, probs, static_cast<Peak *>(workspace), st);
    else probs_t<float>(d, logits, temperature, probs, static_cast<Peak *>(workspace), st);
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
// Rows of up to 12 K entries are one block's work. Longer ones take two launches: the
// weights of every 2048 entries are summed (a wave each), then one block a request
// finds the 2048 that the draw falls into and goes through their entries. Bound by the
// rows' bytes (128 requests of 131072: 29 us, 4.6 TB/s), for few requests by two launches and
// the chain draft -> its probabilities -> row -> sums -> entries (one: 13 us).

constexpr int kGrain = 2048, kPickThreads = 256, kPerThread = kGrain / kPickThreads;

struct Decision {
    int count, accepted;     // drafts of the request, and how many of them stand
};

// Moves of both halves of a double between lanes (lanes without a source, or outside ROWS, get 0).
template <int CTRL, int ROWS = 15> __device__ __forceinline__ double dpp64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 15, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 15, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Inclusive sums over the lanes of a wave, in their order. (Moves by the registers' own paths, not
// through LDS: one request of 6 tokens of 50257 12.8 -> 12.0 us.)
__device__ __forceinline__ double wave_scan(double v) {
    v += dpp64<0x111>(v);              // row_shr 1, 2, 4, 8: within 16 lanes
    v += dpp64<0x112>(v);
    v += dpp64<0x114>(v);
    v += dpp64<0x118>(v);
    v += dpp64<0x142, 0xa>(v);         // lane 15's to the second and lane 47's to the fourth 16
    v += dpp64<0x143, 0xc>(v);         // lane 31's to the upper 32
    return v;
}

// Every wave of the block comes to the same answer: lane i tests draft i.
__device__ __forceinline__ Decision decide(const VerifyDims &d, const VerifyArgs &a, int r) {
    const int lane = threadIdx.x & 63, most = d.T - 1;
    int n = a.count ? a.count[r] : most;
    bool ok = false;
    // (all drafts, whatever the count: it is not waited for)
    if (lane < most) {
        const int tok = a.tokens[(int64_t)r * most + lane];
        const float u = a.uniform[(int64_t)r * d.T + lane];
        if (tok >= 0 && tok < d.V) {
            const float p = a.target[((int64_t)r * d.T + lane) * d.ts + tok];
            const float q = a.draft ? a.draft[((int64_t)r * most + lane) * d.ds + tok] : 1.0f;
            // (an exact product; a draft probability that counts as zero is zero)
            ok = (double)u * (double)(q > 0.0f ? q : 0.0f) < (double)p;
        }
    }
    n = n < 0 ? 0 : (n > most ? most : n);
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

// 4 entries from v on (zeros past the row's end); rows start on their element.
__device__ __forceinline__ void load_entries(const float *row, int v, int V, float *x) {
    typedef float vec4 __attribute__((ext_vector_type(4)));
    typedef vec4 any4 __attribute__((aligned(4)));
    if (v + 4 <= V) {
        const vec4 q = *reinterpret_cast<const any4 *>(row + v);
        x[0] = q[0]; x[1] = q[1]; x[2] = q[2]; x[3] = q[3];
    } else
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = v + i < V ? row[v + i] : 0.0f;
}

__global__ __launch_bounds__(256) void verify_sums_kernel(VerifyDims d, VerifyArgs a, int grains,
                                                          double *__restrict__ sums)
{
    const int lane = threadIdx.x & 63, grain = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6), r = blockIdx.y;
    if (grain >= grains) return;
    const Decision k = decide(d, a, r);
    const Row row(d, a, r, k);
    constexpr int VECS = kGrain / 256;
    float p[VECS][4], q[VECS][4] = {};
#pragma unroll
    for (int j = 0; j < VECS; ++j) load_entries(row.p, grain * kGrain + (j * 64 + lane) * 4, d.V, p[j]);
    if (row.q)
#pragma unroll
        for (int j = 0; j < VECS; ++j) load_entries(row.q, grain * kGrain + (j * 64 + lane) * 4, d.V, q[j]);
    double sw = 0.0, sp = 0.0;
#pragma unroll
    for (int j = 0; j < VECS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            double w, pl;
            row.weigh(grain * kGrain + (j * 64 + lane) * 4 + i, p[j][i], q[j][i], w, pl);
            sw += w;
            sp += pl;
        }
    sw = wave_scan(sw);
    sp = wave_scan(sp);
    if (lane == 63) {
        sums[((int64_t)r * grains + grain) * 2] = sw;
        sums[((int64_t)r * grains + grain) * 2 + 1] = sp;
    }
    if (grain == 0) {
        if (lane == 0) a.accepted[r] = k.accepted;
        for (int i = lane; i < d.T; i += 64)
            if (i != k.accepted)
                a.out[(int64_t)r * d.T + i] = i < k.accepted ? a.tokens[(int64_t)r * (d.T - 1) + i] : -1;
    }
}

// Inclusive sums over the block's threads, in their order, of N values each, and the sums of all.
template <int N> struct BlockScan {
    double part[N][16];
    __device__ __forceinline__ void run(double *v, double *all) {
        const int lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6, waves = (int)blockDim.x >> 6;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = wave_scan(v[k]);
            if (lane == 63) part[k][wave] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            double before = 0.0;
            all[k] = 0.0;
            for (int i = 0; i < waves; ++i) {
                if (i < wave) before += part[k][i];
                all[k] += part[k][i];
            }
            v[k] += before;
        }
    }
};

// The first place that passes `want` and the last of positive weight, over the block.
struct Pick {
    int found, last;
    __device__ __forceinline__ void clear() {
        found = 0x7fffffff;
        last = -1;
    }
    __device__ __forceinline__ int place() const { return found != 0x7fffffff ? found : last; }
};
// A thread's N weights from place v0 on, behind weights of `before`.
template <int N>
__device__ __forceinline__ void pick_among(const double *w, int v0, double before, double want, Pick *p) {
    int hit = 0x7fffffff, last = -1;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        before += w[j];
        if (w[j] > 0.0) {
            last = v0 + j;
            if (hit == 0x7fffffff && before > want) hit = v0 + j;
        }
    }
    if (hit != 0x7fffffff) atomicMin(&p->found, hit);
    if (last >= 0) atomicMax(&p->last, last);
}

// A thread's N entries of the row: its weights against the draft, and the target's own.
template <int N>
__device__ __forceinline__ void weigh_run(const Row &row, int v0, int V, double *w, double *plain) {
    float p[N], q[N] = {};
#pragma unroll
    for (int j = 0; j < N; j += 4) load_entries(row.p, v0 + j, V, p + j);
    if (row.q)
#pragma unroll
        for (int j = 0; j < N; j += 4) load_entries(row.q, v0 + j, V, q + j);
#pragma unroll
    for (int j = 0; j < N; ++j) row.weigh(v0 + j, p[j], q[j], w[j], plain[j]);
}

// Rows of up to 12 K entries: all in one block a request, 16 entries a thread. (One launch and two, in a
// captured graph: 128 requests of 8000 11.1 and 13.6 us, of 12000 12.7 and 13.7, of 16384 14.3 and 13.7; one
// request of 12000 11.1 and 12.3, of 16384 12.5 and 12.2; 512 of 8000 14.6 and 16.1, of 12000 25.6 and 19.7.)
constexpr int kWholePer = 16, kWholeThreads = 768, kWholeMost = kWholeThreads * kWholePer;
__global__ __launch_bounds__(kWholeThreads) void verify_whole_kernel(VerifyDims d, VerifyArgs a) {
    __shared__ BlockScan<2> scan;
    __shared__ Pick pick;
    const int r = blockIdx.x, tid = threadIdx.x, v0 = tid * kWholePer;
    const double uniform = (double)a.uniform[(int64_t)r * d.T + d.T - 1];
    const Decision k = decide(d, a, r);
    const Row row(d, a, r, k);
    if (tid == 0) pick.clear();
    double w[kWholePer], plain[kWholePer], sw = 0.0, sp = 0.0, t[2];
    weigh_run<kWholePer>(row, v0, d.V, w, plain);
#pragma unroll
    for (int j = 0; j < kWholePer; ++j) {
        sw += w[j];
        sp += plain[j];
    }
    double i[2] = {sw, sp};
    scan.run(i, t);
    if (t[0] > 0.0) pick_among<kWholePer>(w, v0, i[0] - sw, t[0] * uniform, &pick);
    else pick_among<kWholePer>(plain, v0, i[1] - sp, t[1] * uniform, &pick);
    __syncthreads();
    if (tid == 0) a.accepted[r] = k.accepted;
    for (int j = tid; j < d.T; j += (int)blockDim.x)
        a.out[(int64_t)r * d.T + j] = j < k.accepted ? a.tokens[(int64_t)r * (d.T - 1) + j]
                                      : j == k.accepted ? pick.place() : -1;
}

__global__ __launch_bounds__(kPickThreads) void verify_pick_kernel(VerifyDims d, VerifyArgs a, int grains,
                                                                   const double *__restrict__ sums)
{
    __shared__ BlockScan<2> scan;
    __shared__ BlockScan<1> scan1;
    __shared__ double start;
    __shared__ Pick pick[2];
    const int r = blockIdx.x, tid = threadIdx.x;
    if (tid < 2) pick[tid].clear();
    const double uniform = (double)a.uniform[(int64_t)r * d.T + d.T - 1];
    // the first launch's decision
    int n = a.count ? a.count[r] : d.T - 1;
    n = n < 0 ? 0 : (n > d.T - 1 ? d.T - 1 : n);
    const Decision k{n, a.accepted[r]};
    const Row row(d, a, r, k);
    const double *const s = sums + (int64_t)r * grains * 2;
    // a thread's grains follow one another
    const int per = (grains + kPickThreads - 1) / kPickThreads, g0 = tid * per;
    const int g1 = g0 + per < grains ? g0 + per : grains;
    double mw = 0.0, mp = 0.0, t[2];
    for (int i = g0; i < g1; ++i) {
        mw += s[2 * i];
        mp += s[2 * i + 1];
    }
    double in[2] = {mw, mp};
    scan.run(in, t);
    const int which = t[0] > 0.0 ? 0 : 1;
    const double want = (which ? t[1] : t[0]) * uniform, before = which ? in[1] - mp : in[0] - mw;
    // the first grain that passes `want`, or the last of positive weight
    double c = before;
    for (int i = g0; i < g1; ++i) {
        const double w = s[2 * i + which];
        pick_among<1>(&w, i, c, want, &pick[0]);
        c += w;
    }
    __syncthreads();
    const int grain = pick[0].place();
    if (grain < 0) {                         // (the same in every thread)
        if (tid == 0) a.out[(int64_t)r * d.T + k.accepted] = -1;
        return;
    }
    if (grain >= g0 && grain < g1) {
        double b = before;
        for (int i = g0; i < grain; ++i) b += s[2 * i + which];
        start = b;
    }
    const int v0 = grain * kGrain + tid * kPerThread;
    double w[kPerThread], plain[kPerThread], mine = 0.0, all;
    weigh_run<kPerThread>(row, v0, d.V, w, plain);
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        w[j] = which ? plain[j] : w[j];
        mine += w[j];
    }
    double incl = mine;
    scan1.run(&incl, &all);                                      // (start is written by now)
    pick_among<kPerThread>(w, v0, start + (incl - mine), want, &pick[1]);
    __syncthreads();
    if (tid == 0) a.out[(int64_t)r * d.T + k.accepted] = pick[1].place();
}

static int grains_of(const VerifyDims &d) { return (d.V + kGrain - 1) / kGrain; }
size_t verify_workspace(const VerifyDims &d)
{
    return d.V <= kWholeMost ? 0 : (size_t)d.R * grains_of(d) * 2 * sizeof(double);
}

void launch_verify(const VerifyDims &d, const VerifyArgs &a, void *workspace, void *stream)
{
    if (d.R <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d.V <= kWholeMost) {
        const int threads = ((d.V + kWholePer - 1) / kWholePer + 63) / 64 * 64;
        hipLaunchKernelGGL(verify_whole_kernel, dim3((unsigned)d.R), dim3((unsigned)threads), 0, st, d, a);
        return;
    }
    const int grains = grains_of(d);
    double *const sums = static_cast<double *>(workspace);
    hipLaunchKernelGGL(verify_sums_kernel, dim3((unsigned)((grains + 3) / 4), (unsigned)d.R), dim3(256), 0, st, d, a,
                       grains, sums);
    hipLaunchKernelGGL(verify_pick_kernel, dim3((unsigned)d.R), dim3(kPickThreads), 0, st, d, a, grains, sums);
}

}  // namespace ssd
