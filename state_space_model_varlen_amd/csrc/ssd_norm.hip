// Root-mean-square norm, with the residual's addition or a gate in front of it
// and 16-, 32- or 8-bit rows behind it.
//
// out = v rsqrt(mean(v^2) + eps) w: a row (or a group of one) is read once,
// kept in registers as float while its squares are summed over the block, and
// written once: bound by its bytes (4096 rows of 2560 with their float32 sum in
// place 26.7 us, 4.7 TB/s), or for few rows by the latency of one load, one sum
// over the block and one store (one row 2.1 us, a call 6.9).
#include <stdint.h>

#include "ssd_layer_device.h"
#include "ssd_step.h"

namespace ssd {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
struct e4m3 {
    uint8_t code;
};

enum NormMode { kPlain, kAdd, kGate };

struct NormArgs {
    const void *x, *other;      // other: residual or gate
    const float *weight;
    void *out, *sum;            // sum: residual_out
    uint8_t *scale;
    int64_t xs, others, sums, os;
    int64_t segments;           // rows * groups
    int groups, per, hidden;    // per: elements a group
    float eps;
};

// The exponent byte of elements whose largest finite magnitude is `top`: top =
// 1.m 2^e and 448 = 1.75 2^8, so the least s with top <= 448 2^s is e - 8, one
// more where 1.m > 1.75.
__device__ __forceinline__ int scale_byte(float top) {
    const uint32_t bits = __float_as_uint(top);
    const int b = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return b < 1 ? 1 : b;
}
__device__ __forceinline__ float finite_size(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;
}
__device__ __forceinline__ float silu(float z) { return z / (1.0f + __expf(-z)); }

__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xb1>(v);       // quad_perm [1,0,3,2]
    v += dpp<0x4e>(v);       // quad_perm [2,3,0,1]
    v += dpp<0x141>(v);      // row_half_mirror
    v += dpp<0x140>(v);      // row_mirror
    return across32(across16(v, added), added);
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float *part) {
    v = wave_sum(v);
    const int waves = (int)blockDim.x >> 6;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < waves; ++i) s += part[i];
    return s;
}

// 8 elements of a row, the first `n` of them if it ends there; rows start on their element.
template <typename T> struct Run8 {
    typedef T vec __attribute__((ext_vector_type(8)));
    typedef vec any __attribute__((aligned(sizeof(T))));
    vec v;
    __device__ __forceinline__ void load(const T *p, int n) {
        if (n >= 8) v = *reinterpret_cast<const any *>(p);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : from_f32<T>(0.0f);
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_f32(v[i]);
    }
    __device__ __forceinline__ static void store(T *p, const float *f, int n) {
        vec o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = from_f32<T>(f[i]);
        if (n >= 8) *reinterpret_cast<any *>(p) = o;
        else
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = o[i];
    }
};

// The row and first element of group `seg`.
__device__ __forceinline__ int64_t group_of(const NormArgs &a, unsigned seg, int &at) {
    if (a.groups == 1) {
        at = 0;
        return seg;
    }
    const unsigned row = seg / (unsigned)a.groups;
    at = (int)(seg - row * (unsigned)a.groups) * a.per;
    return row;
}

// 8 normed elements from `at` of a row on, the first n of them.
template <typename TO> __device__ __forceinline__ void write_run(const NormArgs &a, int64_t row, int at, float *v, int n) {
    if constexpr (std::is_same<TO, e4m3>::value) {
        // (32 elements are 4 neighbouring lanes' and end with the group: all in or all out)
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_size(v[e]));
        top = fmaxf(top, dpp<0xb1>(top));
        top = fmaxf(top, dpp<0x4e>(top));
        const int b = scale_byte(top);
        const float inv = __uint_as_float((254u - (uint32_t)b) << 23);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = fabsf(v[e]) < __builtin_inff() ? v[e] * inv : __builtin_nanf("");
        u32x2 c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j], v[4 * j + 1], 0, false);
            c[j] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2], v[4 * j + 3], lo, true);
        }
        if (n > 0) {
            typedef u32x2 any2 __attribute__((aligned(1)));
            *reinterpret_cast<any2 *>(static_cast<uint8_t *>(a.out) + row * a.os + at) = c;
            if ((threadIdx.x & 3) == 0) a.scale[row * (a.hidden / 32) + at / 32] = (uint8_t)b;
        }
    } else
        Run8<TO>::store(static_cast<TO *>(a.out) + row * a.os + at, v, n);
}

// One group by one block (LANES 0) or by LANES lanes of a block of 256 threads, VPT vectors of 8
// elements a thread.
template <typename TX, typename TR, typename TO, int MODE, int VPT, int LANES>
__global__ __launch_bounds__(LANES ? 256 : 1024) void norm_kernel(NormArgs a) {
    __shared__ float part[16];
    const int lane = LANES ? (int)threadIdx.x % (LANES ? LANES : 1) : (int)threadIdx.x;   // of the group's
    const int lanes = LANES ? LANES : (int)blockDim.x;
    const unsigned seg = LANES ? blockIdx.x * (256u / (LANES ? LANES : 1)) + threadIdx.x / (LANES ? LANES : 1) : blockIdx.x;
    if (LANES && seg >= a.segments) return;                 // (all of a group's lanes)
    int at;
    const int64_t row = group_of(a, seg, at);
    const TX *const x = static_cast<const TX *>(a.x) + row * a.xs + at;
    const TR *const other = static_cast<const TR *>(a.other) + (MODE == kPlain ? 0 : row * a.others + at);
    Run8<TX> rx[VPT];
    Run8<TR> ro[VPT];
    Run8<float> rw[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = (k * lanes + lane) * 8, n = a.per - i;
        rx[k].load(x + i, n);
        if constexpr (MODE != kPlain) ro[k].load(other + i, n);
        if (a.weight) rw[k].load(a.weight + at + i, n);
    }
    float v[VPT][8], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = (k * lanes + lane) * 8, n = a.per - i;
        rx[k].get(v[k]);
        if constexpr (MODE != kPlain) {
            float o[8];
            ro[k].get(o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = MODE == kAdd ? v[k][e] + o[e] : v[k][e] * silu(o[e]);
        }
        if constexpr (MODE == kAdd)
            if (a.sum) Run8<TR>::store(static_cast<TR *>(a.sum) + row * a.sums + at + i, v[k], n);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[k][e], v[k][e], sum);
    }
    if constexpr (LANES == 16) {
        sum += dpp<0xb1>(sum);
        sum += dpp<0x4e>(sum);
        sum += dpp<0x141>(sum);
        sum += dpp<0x140>(sum);
    } else if constexpr (LANES == 64)
        sum = wave_sum(sum);
    else
        sum = block_sum(sum, part);
    const float r = rsqrtf(sum / (float)a.per + a.eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = (k * lanes + lane) * 8, n = a.per - i;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] *= r;
        if (a.weight) {
            float w[8];
            rw[k].get(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= w[e];
        }
        write_run<TO>(a, row, at + i, v[k], n);
    }
}

// The same for rows that no block can keep: read a second time instead (64 rows of 40000 10.1 us,
// 512 37.5, 4.4 TB/s of what has to be moved). A thread adds up to 2^20 squares, 8 of them in float32
// and their sums in 64 bits: equal squares would all round one way (2^26 elements of 1.1 were off by 3e-4).
template <typename TX, typename TR, typename TO, int MODE>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
    __shared__ float part[16];
    int at;
    const int64_t row = group_of(a, blockIdx.x, at);
    const TX *const x = static_cast<const TX *>(a.x) + row * a.xs + at;
    const TR *const other = static_cast<const TR *>(a.other) + (MODE == kPlain ? 0 : row * a.others + at);
    constexpr int STEP = 1024 * 8;
    auto values = [&](int i, float *v) {
        Run8<TX> rx;
        rx.load(x + i, a.per - i);
        rx.get(v);
        if constexpr (MODE != kPlain) {
            Run8<TR> ro;
            float o[8];
            ro.load(other + i, a.per - i);
            ro.get(o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = MODE == kAdd ? v[e] + o[e] : v[e] * silu(o[e]);
        }
    };
    double squares = 0.0;
#pragma unroll 4
    for (int i = (int)threadIdx.x * 8; i < a.per; i += STEP) {
        float v[8], eight = 0.0f;
        values(i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) eight = fmaf(v[e], v[e], eight);
        squares += (double)eight;
    }
    const float sum = block_sum((float)squares, part);
    const float r = rsqrtf(sum / (float)a.per + a.eps);
    for (int i = (int)threadIdx.x * 8; i < a.per; i += STEP) {
        float v[8];
        values(i, v);
        if constexpr (MODE == kAdd)
            // (behind the last read of the residual: it may be the same array)
            if (a.sum) Run8<TR>::store(static_cast<TR *>(a.sum) + row * a.sums + at + i, v, a.per - i);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r;
        if (a.weight) {
            Run8<float> rw;
            float w[8];
            rw.load(a.weight + at + i, a.per - i);
            rw.get(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= w[e];
        }
        write_run<TO>(a, row, at + i, v, a.per - i);
    }
}

template <typename TX, typename TR, typename TO, int MODE>
static void norm_t(const NormArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)a.segments);
    const int vecs = (a.per + 7) / 8;
    if (vecs > 4096) {
        hipLaunchKernelGGL((norm_long_kernel<TX, TR, TO, MODE>), grid, dim3(1024), 0, st, a);
        return;
    }
    // (32768 groups of 125: 18.8 us with a block each, 9.5 with 16 lanes)
    if (vecs <= 64) {
        const int per = vecs <= 16 ? 16 : 4;                // groups a block
        const dim3 blocks((unsigned)((a.segments + per - 1) / per));
        if (vecs <= 16) hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 1, 16>), blocks, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 1, 64>), blocks, dim3(256), 0, st, a);
        return;
    }
    // (512 rows, 1, 2 and 4 vectors a thread: of 2560 elements 4.1, 4.7 and 6.0 us, of 8192 6.8, 6.6 and 6.9, of
    // 16384 10.4 by 2 and by 4; 32768 22.8 by 4 and 30.3 read twice)
    const int vpt = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    const dim3 block((unsigned)(((vecs + vpt - 1) / vpt + 63) / 64 * 64));
    if (vpt == 1) hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 1, 0>), grid, block, 0, st, a);
    else if (vpt == 2) hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 2, 0>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 4, 0>), grid, block, 0, st, a);
}
template <typename TX, typename TO>
static void norm_by_mode(const NormArgs &a, NormMode mode, bool residual_bf16, hipStream_t st) {
    if (mode == kPlain) norm_t<TX, TX, TO, kPlain>(a, st);
    else if (mode == kGate) norm_t<TX, TX, TO, kGate>(a, st);
    else if (residual_bf16) norm_t<TX, bf16, TO, kAdd>(a, st);
    else norm_t<TX, float, TO, kAdd>(a, st);
}

void launch_rms_norm(const NormDims &d, const void *x, const void *gate, const void *residual,
                     const float *weight, void *out, uint8_t *out_scale, void *residual_out,
                     void *stream)
{
    if (d.rows <= 0) return;
    const NormMode mode = residual ? kAdd : gate ? kGate : kPlain;
    const NormArgs a{x, residual ? residual : gate, weight, out, residual_out, out_scale,
                     d.xs, residual ? d.rs : d.gs, d.ros, d.os, d.rows * d.groups,
                     d.groups, d.hidden / d.groups, d.hidden, d.eps};
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const bool rb = d.residual == Elem::bf16;
    if (d.in == Elem::bf16) {
        if (d.out == Elem::f32) norm_by_mode<bf16, float>(a, mode, rb, st);
        else if (d.out == Elem::bf16) norm_by_mode<bf16, bf16>(a, mode, rb, st);
        else norm_by_mode<bf16, e4m3>(a, mode, rb, st);
    } else {
        if (d.out == Elem::f32) norm_by_mode<float, float>(a, mode, rb, st);
        else if (d.out == Elem::bf16) norm_by_mode<float, bf16>(a, mode, rb, st);
        else norm_by_mode<float, e4m3>(a, mode, rb, st);
    }
}

}  // namespace ssd
