// Root-mean-square norm, with the residual's addition or a gate in front of it
// and 16-, 32- or 8-bit rows behind it.
//
// out = v rsqrt(mean(v^2) + eps) w: a row (or a group of one) is read once,
// kept in registers as float while its squares are summed over the block, and
// written once: bound by its bytes, or for few rows by the latency of one load,
// one sum over the block and one store.
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

// One group by one block, VPT vectors of 8 elements a thread; every row on 16
// bytes (out: 8 for 8-bit rows).
template <typename TX, typename TR, typename TO, int MODE, int VPT>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
    __shared__ float part[16];
    const int64_t seg = blockIdx.x;
    const int64_t row = seg / a.groups;
    const int at = (int)(seg - row * a.groups) * a.per;
    const TX *const x = static_cast<const TX *>(a.x) + row * a.xs + at;
    const TR *const other = static_cast<const TR *>(a.other) + (MODE == kPlain ? 0 : row * a.others + at);
    RawV<TX, 8> rx[VPT];
    RawV<TR, 8> ro[VPT];
    RawV<float, 8> rw[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = (k * (int)blockDim.x + (int)threadIdx.x) * 8;
        rx[k].zero();
        if (i < a.per) {
            rx[k].load(x + i);
            if constexpr (MODE != kPlain) ro[k].load(other + i);
            if (a.weight) rw[k].load(a.weight + at + i);
        }
    }
    float v[VPT][8], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = (k * (int)blockDim.x + (int)threadIdx.x) * 8;
        rx[k].get(v[k]);
        if (i < a.per) {
            if constexpr (MODE != kPlain) {
                float o[8];
                ro[k].get(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k][e] = MODE == kAdd ? v[k][e] + o[e] : v[k][e] * silu(o[e]);
            }
            if constexpr (MODE == kAdd) {
                if (a.sum) {
                    RawV<TR, 8> s;
                    s.set(v[k]);
                    s.store(static_cast<TR *>(a.sum) + row * a.sums + at + i);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[k][e], v[k][e], sum);
    }
    sum = block_sum(sum, part);
    const float r = rsqrtf(sum / (float)a.per + a.eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = (k * (int)blockDim.x + (int)threadIdx.x) * 8;
        float w[8];
        if (a.weight && i < a.per) rw[k].get(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = a.weight && i < a.per ? v[k][e] * r * w[e] : v[k][e] * r;
        if constexpr (std::is_same<TO, e4m3>::value) {
            // (32 elements are 4 neighbouring lanes' and end with the group: all in or all out)
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_size(v[k][e]));
            top = fmaxf(top, dpp<0xb1>(top));
            top = fmaxf(top, dpp<0x4e>(top));
            const int b = scale_byte(top);
            const float inv = __uint_as_float((254u - (uint32_t)b) << 23);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[k][e] = fabsf(v[k][e]) < __builtin_inff() ? v[k][e] * inv : __builtin_nanf("");
            u32x2 c;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * j], v[k][4 * j + 1], 0, false);
                c[j] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * j + 2], v[k][4 * j + 3], lo, true);
            }
            if (i < a.per) {
                *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + row * a.os + at + i) = c;
                if ((threadIdx.x & 3) == 0) a.scale[row * (a.hidden / 32) + (at + i) / 32] = (uint8_t)b;
            }
        } else if (i < a.per) {
            RawV<TO, 8> o;
            o.set(v[k]);
            o.store(static_cast<TO *>(a.out) + row * a.os + at + i);
        }
    }
}

// The same for rows of any alignment and length: an element a thread and step,
// read a second time instead of kept.
template <typename TX, typename TR, typename TO, int MODE>
__global__ __launch_bounds__(256) void norm_any_kernel(NormArgs a) {
    __shared__ float part[4];
    const int64_t seg = blockIdx.x;
    const int64_t row = seg / a.groups;
    const int at = (int)(seg - row * a.groups) * a.per;
    const TX *const x = static_cast<const TX *>(a.x) + row * a.xs + at;
    const TR *const other = static_cast<const TR *>(a.other) + (MODE == kPlain ? 0 : row * a.others + at);
    auto value = [&](int i) {
        const float v = to_f32(x[i]);
        if constexpr (MODE == kAdd) return v + to_f32(other[i]);
        else if constexpr (MODE == kGate) return v * silu(to_f32(other[i]));
        else return v;
    };
    float sum = 0.0f;
    for (int i = (int)threadIdx.x; i < a.per; i += 256) {
        const float v = value(i);
        sum = fmaf(v, v, sum);
    }
    sum = block_sum(sum, part);
    const float r = rsqrtf(sum / (float)a.per + a.eps);
    for (int i = (int)threadIdx.x; i < a.per; i += 256) {
        const float v = value(i);
        if constexpr (MODE == kAdd)
            // (behind the last read of the residual: it may be the same array)
            if (a.sum) static_cast<TR *>(a.sum)[row * a.sums + at + i] = from_f32<TR>(v);
        float y = v * r;
        if (a.weight) y *= a.weight[at + i];
        if constexpr (std::is_same<TO, e4m3>::value) {
            // (groups are whole blocks of 32: half a wave is in or out together)
            float top = finite_size(y);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
            const int b = scale_byte(top);
            y = fabsf(y) < __builtin_inff() ? y * __uint_as_float((254u - (uint32_t)b) << 23)
                                            : __builtin_nanf("");
            static_cast<uint8_t *>(a.out)[row * a.os + at + i] =
                (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false);
            if ((threadIdx.x & 31) == 0) a.scale[row * (a.hidden / 32) + (at + i) / 32] = (uint8_t)b;
        } else
            static_cast<TO *>(a.out)[row * a.os + at + i] = from_f32<TO>(y);
    }
}

template <typename TX, typename TR, typename TO, int MODE>
static void norm_t(const NormArgs &a, bool wide, hipStream_t st) {
    const dim3 grid((unsigned)a.segments);
    const int vecs = (a.per + 7) / 8;
    if (!wide || vecs > 4096) {
        hipLaunchKernelGGL((norm_any_kernel<TX, TR, TO, MODE>), grid, dim3(256), 0, st, a);
        return;
    }
    const int vpt = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    const dim3 block((unsigned)(((vecs + vpt - 1) / vpt + 63) / 64 * 64));
    if (vpt == 1) hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 1>), grid, block, 0, st, a);
    else if (vpt == 2) hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 2>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((norm_kernel<TX, TR, TO, MODE, 4>), grid, block, 0, st, a);
}
template <typename TX, typename TO>
static void norm_by_mode(const NormArgs &a, NormMode mode, bool residual_bf16, bool wide, hipStream_t st) {
    if (mode == kPlain) norm_t<TX, TX, TO, kPlain>(a, wide, st);
    else if (mode == kGate) norm_t<TX, TX, TO, kGate>(a, wide, st);
    else if (residual_bf16) norm_t<TX, bf16, TO, kAdd>(a, wide, st);
    else norm_t<TX, float, TO, kAdd>(a, wide, st);
}

static size_t bytes_of(Elem e) { return e == Elem::f32 ? 4 : e == Elem::bf16 ? 2 : 1; }

void launch_rms_norm(const NormDims &d, const void *x, const void *gate, const void *residual,
                     const float *weight, void *out, uint8_t *out_scale, void *residual_out,
                     void *stream)
{
    if (d.rows <= 0) return;
    const NormMode mode = residual ? kAdd : gate ? kGate : kPlain;
    const NormArgs a{x, residual ? residual : gate, weight, out, residual_out, out_scale,
                     d.xs, residual ? d.rs : d.gs, d.ros, d.os, d.rows * d.groups,
                     d.groups, d.hidden / d.groups, d.hidden, d.eps};
    auto on = [](const void *p, int64_t stride, size_t e, size_t n) {
        return reinterpret_cast<uintptr_t>(p) % n == 0 && (uint64_t)stride * e % n == 0;
    };
    const size_t ei = bytes_of(d.in), er = bytes_of(d.residual), eo = bytes_of(d.out);
    const bool wide = a.per % 8 == 0 && on(x, d.xs, ei, 16) && on(gate, gate ? d.gs : 0, ei, 16) &&
                      on(residual, residual ? d.rs : 0, er, 16) &&
                      on(residual_out, residual_out ? d.ros : 0, er, 16) && on(weight, 0, 4, 16) &&
                      on(out, d.os, eo, eo == 1 ? 8 : 16);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const bool rb = d.residual == Elem::bf16;
    if (d.in == Elem::bf16) {
        if (d.out == Elem::f32) norm_by_mode<bf16, float>(a, mode, rb, wide, st);
        else if (d.out == Elem::bf16) norm_by_mode<bf16, bf16>(a, mode, rb, wide, st);
        else norm_by_mode<bf16, e4m3>(a, mode, rb, wide, st);
    } else {
        if (d.out == Elem::f32) norm_by_mode<float, float>(a, mode, rb, wide, st);
        else if (d.out == Elem::bf16) norm_by_mode<float, bf16>(a, mode, rb, wide, st);
        else norm_by_mode<float, e4m3>(a, mode, rb, wide, st);
    }
}

}  // namespace ssd
