// Channel-wise selective scan over packed sequences (prompts) and for the few
// tokens of a verify step.
//
//     h_t[c,n] = exp(dt_t[c] A[c,n]) h_{t-1}[c,n] + dt_t[c] x_t[c] B_t[g,n]
//     y_t[c]   = (sum over n of h_t[c,n] C_t[g,n] + D[c] x_t[c]) silu(z_t[c])
//
// Every (channel, state) has a decay of its own, so the recurrence has no
// matrix product in it: each token costs one exponential, two products and two
// multiply-adds per (channel, state) on the vector units, which bound the
// prompt form. The single-token form is bound by the states it reads and writes.
#include "ssd_layer.h"
#include "ssd_layer_device.h"

namespace ssd {

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) <= 1, with
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, summed to s^13 (the next
// term is under 2^-25 of the sum): accurate relative to the result also where
// e is small, which a logarithm of the rounded 1 + e is not.
__device__ __forceinline__ float softplus(float v) {
    const float e = __expf(-fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
    const float q = s * s;
    float p = 2.0f / 13.0f;
    p = p * q + 2.0f / 11.0f;
    p = p * q + 2.0f / 9.0f;
    p = p * q + 2.0f / 7.0f;
    p = p * q + 2.0f / 5.0f;
    p = p * q + 2.0f / 3.0f;
    p = p * q + 2.0f;
    return fmaxf(v, 0.0f) + p * s;
}
// (NaN steps stay NaN: fminf and fmaxf would drop them)
__device__ __forceinline__ float step_size(const DtTf &tf, float raw, float bias) {
    if (!tf.on) return raw;
    const float sp = softplus(raw + bias);
    return sp != sp ? sp : fminf(fmaxf(sp, tf.lo), tf.hi);
}
__device__ __forceinline__ float silu(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// Lane J's value of a group of L lanes (4: a quad; 16: a row).
template <int L, int J> __device__ __forceinline__ float from_lane(float v) {
    if constexpr (L == 4) return dpp<0x55 * J>(v);       // quad_perm [J,J,J,J]
    else return dpp<0x150 + J>(v);                       // row_newbcast J
}

// v[j], j < L: every lane's share of token j's sum. Returns the whole sum of
// the lane's own token (lane j of the group: token j). Halves of the group
// swap the tokens that they do not keep (L/2 + L/4 + ... + 1 exchanges in
// place of log2 L for each token).
template <int L> __device__ __forceinline__ float sum_own(float *v, int lane) {
    if constexpr (L == 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float keep = (lane & 8) ? v[j + 8] : v[j], send = (lane & 8) ? v[j] : v[j + 8];
            v[j] = keep + dpp<0x140>(send);              // row_mirror: lane 15 - i
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float keep = (lane & 4) ? v[j + 4] : v[j], send = (lane & 4) ? v[j] : v[j + 4];
            v[j] = keep + dpp<0x141>(send);              // row_half_mirror: 7 - i of 8
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float keep = (lane & 2) ? v[j + 2] : v[j], send = (lane & 2) ? v[j] : v[j + 2];
        v[j] = keep + dpp<0x4e>(send);                   // quad_perm [2,3,0,1]
    }
    const float keep = (lane & 1) ? v[1] : v[0], send = (lane & 1) ? v[0] : v[1];
    return keep + dpp<0xb1>(send);                       // quad_perm [1,0,3,2]
}

template <int N, typename F> __device__ __forceinline__ void unrolled(F f) {
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>());
    }
}

template <typename T, int M> __device__ __forceinline__ void load_state(const T *p, float *v) {
    if constexpr (M % 4 == 0) {
#pragma unroll
        for (int i = 0; i < M; i += 4) load4<T>(p + i, v + i);
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] = to_f32(p[i]);
    }
}
template <typename T, int M> __device__ __forceinline__ void store_state(T *p, const float *v) {
    if constexpr (M % 4 == 0) {
#pragma unroll
        for (int i = 0; i < M; i += 4) store4<T>(p + i, v + i);
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i) p[i] = from_f32<T>(v[i]);
    }
}

// Prompt form. L lanes per channel hold SPL = N / L states each, in registers
// for the whole sequence; a block of 4 waves takes 256 / L channels of one
// group and one sequence. The tokens are taken in groups of L: lane j of a
// channel reads x, dt and z of the group's token j, prepares its step size and
// gate once, and the group's L tokens are then run through one after the
// other, each lane taking token j's values from lane j. B and C of a stage of
// ST tokens are widened to float in LDS by the whole block (two buffers, one
// barrier a stage); the next stage's loads are in flight meanwhile.
template <typename TX, typename TS, int N, int L>
__global__ __launch_bounds__(256) void scan_kernel(
    int T, int S, int C, int G, int num_slots, int chb, ScanArgs a, int64_t xs, int64_t dts,
    int64_t zs, int64_t bs, int64_t cs, int64_t ys, DtTf tf)
{
    constexpr int SPL = N / L, CB = 256 / L;
    constexpr int GROUPS = L == 16 ? 4 : 8;      // groups of L tokens in a stage
    constexpr int ST = L * GROUPS;
    constexpr int BCV = ST * N * 2 / 256;        // B, C values a thread stages
    __shared__ __align__(16) float bc[2][2][ST][N];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), j0 = tid % L;
    const int per = C / G, gblocks = chb / G;
    const int s = (int)(blockIdx.x / (unsigned)chb), cb = (int)(blockIdx.x % (unsigned)chb);
    const int g = cb / gblocks;
    const int in_g = (cb % gblocks) * CB + tid / L;
    const bool live = in_g < per;
    const int c = g * per + (live ? in_g : per - 1);

    int start = a.cu[s], end = a.cu[s + 1];
    start = start < 0 ? 0 : (start > T ? T : start);
    end = end < 0 ? 0 : (end > T ? T : end);
    const int len = end > start ? end - start : 0;
    const int slot = a.idx[s];
    const bool slot_ok = slot >= 0 && slot < num_slots;
    const int64_t so = ((int64_t)(slot_ok ? slot : 0) * C + c) * N + j0 * SPL;
    TS *const cache = static_cast<TS *>(a.cache) + so;

    float A2[SPL], h[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        A2[i] = a.A[(int64_t)c * N + j0 * SPL + i] * kLog2e;
        h[i] = 0.0f;
    }
    if (slot_ok && a.has && a.has[s]) load_state<TS, SPL>(cache, h);
    const float Dc = a.D ? a.D[c] : 0.0f, bias = tf.bias ? tf.bias[c] : 0.0f;
    const TX *const xp = static_cast<const TX *>(a.x) + (int64_t)start * xs + c;
    const TX *const dp = static_cast<const TX *>(a.dt) + (int64_t)start * dts + c;
    const TX *const zp = a.z ? static_cast<const TX *>(a.z) + (int64_t)start * zs + c : nullptr;
    TX *const yp = static_cast<TX *>(a.y) + (int64_t)start * ys + c;
    const TX *const Bp = static_cast<const TX *>(a.B) + (int64_t)start * bs + (int64_t)g * N;
    const TX *const Cp = static_cast<const TX *>(a.C) + (int64_t)start * cs + (int64_t)g * N;

    TX xv[GROUPS], dv[GROUPS], zv[GROUPS], bv[BCV];
    auto request = [&](int t0) {
#pragma unroll
        for (int m = 0; m < GROUPS; ++m) {
            const int t = t0 + m * L + j0;
            const int64_t r = t < len ? t : len - 1;
            xv[m] = xp[r * xs];
            dv[m] = dp[r * dts];
            if (zp) zv[m] = zp[r * zs];
        }
        // value e of the stage: state e % N of token (e / N) % ST, of B then C
#pragma unroll
        for (int k = 0; k < BCV; ++k) {
            const int e = tid + 256 * k, n = e % N, t = t0 + (e / N) % ST;
            const int64_t r = t < len ? t : len - 1;
            bv[k] = e < ST * N ? Bp[r * bs + n] : Cp[r * cs + n];
        }
    };
    if (len > 0) request(0);
    int buf = 0;
    for (int t0 = 0; t0 < len; t0 += ST, buf ^= 1) {
        // tokens past the end: B, C zero here and a step of zero below
#pragma unroll
        for (int k = 0; k < BCV; ++k) {
            const int e = tid + 256 * k, t = (e / N) % ST;
            (&bc[buf][0][0][0])[e] = t0 + t < len ? to_f32(bv[k]) : 0.0f;
        }
        float x[GROUPS], dt[GROUPS], gate[GROUPS];
#pragma unroll
        for (int m = 0; m < GROUPS; ++m) {
            const bool in = t0 + m * L + j0 < len;
            x[m] = in ? to_f32(xv[m]) : 0.0f;
            dt[m] = in ? step_size(tf, to_f32(dv[m]), bias) : 0.0f;
            gate[m] = zp ? silu(to_f32(zv[m])) : 1.0f;
        }
        __syncthreads();
        if (t0 + ST < len) request(t0 + ST);
#pragma unroll
        for (int m = 0; m < GROUPS; ++m) {
            if (t0 + m * L >= len) break;
            const float dtx = dt[m] * x[m];
            float part[L];
            unrolled<L>([&](auto J) {
                constexpr int j = decltype(J)::value;
                const float d = from_lane<L, j>(dt[m]), u = from_lane<L, j>(dtx);
                const float *const Bt = &bc[buf][0][m * L + j][j0 * SPL];
                const float *const Ct = &bc[buf][1][m * L + j][j0 * SPL];
                float p = 0.0f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    h[i] = __builtin_amdgcn_exp2f(d * A2[i]) * h[i] + u * Bt[i];
                    p = i == 0 ? h[i] * Ct[i] : p + h[i] * Ct[i];
                }
                part[j] = p;
            });
            const float y = (sum_own<L>(part, lane) + Dc * x[m]) * gate[m];
            const int t = t0 + m * L + j0;
            if (live && t < len) yp[(int64_t)t * ys] = from_f32<TX>(y);
        }
    }
    if (slot_ok && live) store_state<TS, SPL>(cache, h);
}

size_t scan_workspace(const ScanDims &) { return 0; }

template <typename TX, typename TS, int N>
static void launch_scan_n(const ScanDims &d, const ScanArgs &a, hipStream_t st)
{
    constexpr int L = 4;
    const int per = d.C / d.G, chb = d.G * ((per + 256 / L - 1) / (256 / L));
    hipLaunchKernelGGL((scan_kernel<TX, TS, N, L>), dim3((unsigned)((int64_t)chb * d.S)), dim3(256),
                       0, st, d.T, d.S, d.C, d.G, d.num_slots, chb, a, d.xs, d.dts, d.zs, d.bs,
                       d.cs, d.ys, d.tf);
}

// Verify-step form: L = 4 lanes per channel, N / 4 states each; a block takes 64
// channels of one request. The state and the tokens' inputs, TM tokens at a
// time, are all requested before the first wait.
template <typename TX, typename TS, int N, int TM>
__global__ __launch_bounds__(256) void scan_update_kernel(
    int Tr, int C, int G, int num_slots, int chb, ScanArgs a, int64_t xs, int64_t dts, int64_t zs,
    int64_t bs, int64_t cs, int64_t ys, DtTf tf, TS *__restrict__ inter)
{
    constexpr int L = 4, SPL = N / L, CB = 256 / L;
    const int tid = threadIdx.x, j0 = tid % L;
    const int r = (int)(blockIdx.x / (unsigned)chb);
    const int c = (int)(blockIdx.x % (unsigned)chb) * CB + tid / L;
    if (c >= C) return;      // (whole quads)
    const int g = c / (C / G);
    const int slot = a.idx[r];
    const bool slot_ok = slot >= 0 && slot < num_slots;
    TS *const cache = static_cast<TS *>(a.cache) +
                      ((int64_t)(slot_ok ? slot : 0) * C + c) * N + j0 * SPL;
    const TX *const xp = static_cast<const TX *>(a.x) + (int64_t)r * Tr * xs + c;
    const TX *const dp = static_cast<const TX *>(a.dt) + (int64_t)r * Tr * dts + c;
    const TX *const zp = a.z ? static_cast<const TX *>(a.z) + (int64_t)r * Tr * zs + c : nullptr;
    TX *const yp = static_cast<TX *>(a.y) + (int64_t)r * Tr * ys + c;
    const TX *const Bp = static_cast<const TX *>(a.B) + (int64_t)r * Tr * bs + g * N + j0 * SPL;
    const TX *const Cp = static_cast<const TX *>(a.C) + (int64_t)r * Tr * cs + g * N + j0 * SPL;

    TX xv[TM], dv[TM], zv[TM], Bv[TM][SPL], Cv[TM][SPL];
    auto request = [&](int t0) {
#pragma unroll
        for (int m = 0; m < TM; ++m) {
            const int64_t t = t0 + m < Tr ? t0 + m : Tr - 1;
            xv[m] = xp[t * xs];
            dv[m] = dp[t * dts];
            if (zp) zv[m] = zp[t * zs];
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                Bv[m][i] = Bp[t * bs + i];
                Cv[m][i] = Cp[t * cs + i];
            }
        }
    };
    float h[SPL], A2[SPL];
    if (Tr > 0) request(0);
    load_state<TS, SPL>(cache, h);
#pragma unroll
    for (int i = 0; i < SPL; ++i) A2[i] = a.A[(int64_t)c * N + j0 * SPL + i] * kLog2e;
    const float Dc = a.D ? a.D[c] : 0.0f, bias = tf.bias ? tf.bias[c] : 0.0f;
    if (!slot_ok) {
#pragma unroll
        for (int i = 0; i < SPL; ++i) h[i] = 0.0f;
    }
    for (int t0 = 0; t0 < Tr; t0 += TM) {
        if (t0 > 0) request(t0);
#pragma unroll
        for (int m = 0; m < TM; ++m) {
            const int t = t0 + m;
            if (t >= Tr) break;
            const float x = to_f32(xv[m]), dt = step_size(tf, to_f32(dv[m]), bias), u = dt * x;
            float p = 0.0f;
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                h[i] = __builtin_amdgcn_exp2f(dt * A2[i]) * h[i] + u * to_f32(Bv[m][i]);
                p += h[i] * to_f32(Cv[m][i]);
            }
            p += dpp<0xb1>(p);
            p += dpp<0x4e>(p);
            const float y = (p + Dc * x) * (zp ? silu(to_f32(zv[m])) : 1.0f);
            if (j0 == 0) yp[(int64_t)t * ys] = from_f32<TX>(y);
            if (inter)
                store_state<TS, SPL>(inter + (((int64_t)r * Tr + t) * C + c) * N + j0 * SPL, h);
        }
    }
    if (!inter && slot_ok) store_state<TS, SPL>(cache, h);
}

template <typename TX, typename TS, int N>
static void launch_update_n(const ScanDims &d, const ScanArgs &a, void *inter, hipStream_t st)
{
    const int Tr = d.T / d.S, chb = (d.C + 63) / 64;
    const dim3 grid((unsigned)((int64_t)chb * d.S));
#define SSD_UPD(TM)                                                                              \
    hipLaunchKernelGGL((scan_update_kernel<TX, TS, N, TM>), grid, dim3(256), 0, st, Tr, d.C, d.G, \
                       d.num_slots, chb, a, d.xs, d.dts, d.zs, d.bs, d.cs, d.ys, d.tf,           \
                       static_cast<TS *>(inter))
    if (Tr <= 1) SSD_UPD(1);
    else SSD_UPD(4);
#undef SSD_UPD
}

#define SSD_BY_N(FN, TX, TS, ...)                                    \
    do {                                                             \
        if (d.N == 16) FN<TX, TS, 16>(d, a, __VA_ARGS__);            \
        else if (d.N == 32) FN<TX, TS, 32>(d, a, __VA_ARGS__);       \
        else FN<TX, TS, 64>(d, a, __VA_ARGS__);                      \
    } while (0)
#define SSD_BY_TYPE(FN, ...)                                             \
    do {                                                                 \
        if (d.in_bf16) {                                                 \
            if (d.state_dtype == 0) SSD_BY_N(FN, bf16, float, __VA_ARGS__); \
            else if (d.state_dtype == 1) SSD_BY_N(FN, bf16, bf16, __VA_ARGS__); \
            else SSD_BY_N(FN, bf16, f16, __VA_ARGS__);                   \
        } else {                                                         \
            if (d.state_dtype == 0) SSD_BY_N(FN, float, float, __VA_ARGS__); \
            else if (d.state_dtype == 1) SSD_BY_N(FN, float, bf16, __VA_ARGS__); \
            else SSD_BY_N(FN, float, f16, __VA_ARGS__);                  \
        }                                                                \
    } while (0)

void launch_scan(const ScanDims &d, const ScanArgs &a, void *, void *stream)
{
    if (d.S <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    SSD_BY_TYPE(launch_scan_n, st);
}

void launch_scan_update(const ScanDims &d, const ScanArgs &a, void *inter, void *stream)
{
    if (d.S <= 0 || d.T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    SSD_BY_TYPE(launch_update_n, inter, st);
}

}  // namespace ssd
