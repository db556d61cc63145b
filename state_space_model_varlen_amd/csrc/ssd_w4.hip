// Products with 4-bit weights: y[t,n] = sum over k of x[t,k] w[n,k] + bias[n].
//
// The matrix instructions take the weights as their first operand (16 weight
// rows) and the tokens as their second (16 tokens), so that a lane's results
// are 4 neighbouring outputs of one token. K goes in steps of 128: lane l of
// a wave reads 16 bytes of weight row l % 16, the 32 codes of block l / 16 of
// the step, as they lie in memory.
//   8-bit rows: one 16 x 16 x 128 instruction takes codes, 8-bit values and the
//   exponent bytes of both. It expects of a lane's 32 token values the first 16
//   from K = 16 (l / 16) and the others from 64 + 16 (l / 16), while a lane's
//   exponent byte belongs to block l / 16 of either operand.
//   bfloat16 rows: the codes are widened to bfloat16 with their block's power of
//   two (exact), and four 16 x 16 x 32 instructions each take 8 of them; the
//   order of K inside the step does not matter as long as both operands keep it.
#include <stdint.h>

#include "ssd_layer_device.h"
#include "ssd_step.h"

namespace ssd {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Byte offset of a lane that has nothing to read: past every resource's end.
constexpr uint32_t kNothing = 0x80000000u;

// (`at`, the same in every lane, is added to the address; that a lane's own offset lies past the
// end is seen with and without it)
__device__ __forceinline__ i32x4 buf16(rsrc_t r, uint32_t off, uint32_t at = 0) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, (int)at, 0));
}
__device__ __forceinline__ int buf1(rsrc_t r, uint32_t off, uint32_t at = 0) {
    return (int)__builtin_amdgcn_raw_buffer_load_b8(r, (int)off, (int)at, 0);
}

// 8 codes (one word) widened to bfloat16 and scaled by 2^(byte - 127).
__device__ __forceinline__ bf16x8 widen_codes(uint32_t w, uint32_t byte) {
    const float s = __uint_as_float(byte << 23);
    bf16x8 r;
    bf16x2 p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = p[i][0];
        r[2 * i + 1] = p[i][1];
    }
    return r;
}

__device__ __forceinline__ f32x4 mma_8bit(i32x4 w, int ws, i32x4 x0, i32x4 x1, int xs, f32x4 c) {
    const i32x8 a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    const i32x8 b = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
    // (first operand 4-bit, second e4m3; exponents from the lowest byte)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 0, 0, ws, 0, xs);
}

// What a block of 4 waves works on: 16 RT weight rows, 16 TT tokens; the waves
// take the K steps in turn and are joined in LDS.
template <bool E4M3, int TT, int RT, typename TO>
__global__ __launch_bounds__(256) void linear_kernel(LinearDims d, LinearArgs a)
{
    __shared__ f32x4 part[4][RT * TT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), n16 = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * 16 * RT, t0 = (int)blockIdx.y * 16 * TT;
    const int blocks = d.K / 32;                                  // of 32 in a row
    constexpr int EX = E4M3 ? 1 : 2;
    const int nrows = d.N - n0 < 16 * RT ? d.N - n0 : 16 * RT, ntok = d.T - t0 < 16 * TT ? d.T - t0 : 16 * TT;
    const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * (d.K / 2), (uint32_t)nrows * (uint32_t)(d.K / 2));
    const rsrc_t rs = make_rsrc(a.w_scale + (int64_t)n0 * blocks, (uint32_t)nrows * (uint32_t)blocks);
    const rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + (int64_t)t0 * d.xs * EX,
                                (uint32_t)((ntok - 1) * d.xs + d.K) * EX);
    const rsrc_t rxs = make_rsrc(a.x_scale + (int64_t)t0 * blocks, E4M3 ? (uint32_t)ntok * (uint32_t)blocks : 0);
    f32x4 acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = zero4();

    for (int s = wave; s * 4 < blocks; s += 4) {
        const int b = 4 * s + g;                                  // this lane's block of 32
        const bool in = b < blocks;
        i32x4 w[RT];
        int ws[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = 16 * r + n16;
            w[r] = buf16(rw, in ? (uint32_t)row * (uint32_t)(d.K / 2) + 16u * b : kNothing);
            ws[r] = buf1(rs, in ? (uint32_t)row * (uint32_t)blocks + b : kNothing);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int tok = 16 * t + n16;
            const bool live = tok < ntok;
            const uint32_t at = (uint32_t)tok * (uint32_t)d.xs * EX;
            if constexpr (E4M3) {
                const uint32_t k0 = 128u * s + 16u * g, k1 = k0 + 64u;
                const i32x4 x0 = buf16(rx, live && k0 < (uint32_t)d.K ? at + k0 : kNothing);
                const i32x4 x1 = buf16(rx, live && k1 < (uint32_t)d.K ? at + k1 : kNothing);
                const int xs = buf1(rxs, live && in ? (uint32_t)tok * (uint32_t)blocks + b : kNothing);
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r][t] = mma_8bit(w[r], ws[r], x0, x1, xs, acc[r][t]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t k = 128u * s + 32u * g + 8u * i;
                    const bf16x8 x = __builtin_bit_cast(bf16x8, buf16(rx, live && in ? at + 2u * k : kNothing));
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        acc[r][t] = Mma<bf16>::run(widen_codes((uint32_t)w[r][i], (uint32_t)ws[r]), x, acc[r][t]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) part[wave][r * TT + t][lane] = acc[r][t];
    __syncthreads();
    TO *const out = static_cast<TO *>(a.out);
    for (int i = wave; i < RT * TT; i += 4) {
        f32x4 y = part[0][i][lane];
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            const f32x4 o = part[k][i][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] += o[e];
        }
        const int tok = t0 + 16 * (i % TT) + n16, n = n0 + 16 * (i / TT) + 4 * g;
        if (tok < d.T)
            for (int e = 0; e < 4; ++e)
                if (n + e < d.N)
                    out[(int64_t)tok * d.os + n + e] = from_f32<TO>(y[e] + (a.bias ? a.bias[n + e] : 0.0f));
    }
}

// ---------------------------------------------------------------------------
// Many tokens: a block of 4 waves takes 16 TT tokens and 64 RT weight rows, 16 RT
// of them a wave. The weights go straight from memory to registers, where they
// are operands as they lie, each read by one wave; the tokens' rows are shared
// and go through LDS, 128 of their values a stage, written there by the loads
// themselves. While a stage is multiplied the next one is on its way.
//
// A row's 16-byte chunk c lies in place c ^ row % 16 (of 16) or c ^ row / 2 % 8
// (of 8), so that the 16 rows that a fragment reads together touch all banks.
//
// Rows of a fragment are dealt such that a lane's results of its RT fragments
// are 4 RT neighbouring outputs.
enum LinearMode {
    kEight,      // 8-bit rows, scaled 8-bit instruction
    kSixteen,    // bfloat16 rows
    kWidened     // 8-bit rows widened to bfloat16
};

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ bf16x8 widen_8bit(u32x2 w, float s) {
    bf16x8 r;
    bf16x2 p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], s, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], s, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], s, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], s, true);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = p[i][0];
        r[2 * i + 1] = p[i][1];
    }
    return r;
}

template <int MODE, int TT, int RT, typename TO>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(LinearDims d, LinearArgs a, int ttiles, int ntiles)
{
    constexpr int EX = MODE == kSixteen ? 2 : 1;
    constexpr int TOK = 16 * TT, CH = 8 * EX;             // CH: 16-byte chunks of a token a stage
    constexpr int PITCH = 16 * CH, LOADS = TOK * CH / 256;
    static_assert(TOK * CH % 256 == 0, "whole loads");
    __shared__ __align__(16) char xa[TOK * PITCH], xb[TOK * PITCH];
    // (scales of 8-bit rows: 4 a token)
    __shared__ uint8_t sa[MODE == kSixteen ? 1 : 4 * TOK], sb[MODE == kSixteen ? 1 : 4 * TOK];
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), n16 = lane & 15, g = lane >> 4;

    // tiles in groups of 8 token tiles, so that the blocks of one L2 share rows and weights
    constexpr int kGroup = 8;
    const int id = xcd_logical_block((int)blockIdx.x, ttiles * ntiles);
    const int grp = id / (kGroup * ntiles), in = id - grp * (kGroup * ntiles);
    const int gm = ttiles - grp * kGroup < kGroup ? ttiles - grp * kGroup : kGroup;
    const int nt = in / gm, t0 = (grp * kGroup + in - nt * gm) * TOK, n0 = nt * 64 * RT;

    const int blocks = d.K / 32, stages = (blocks + 3) / 4;
    const int nrows = d.N - n0 < 64 * RT ? d.N - n0 : 64 * RT, ntok = d.T - t0 < TOK ? d.T - t0 : TOK;
    const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * (d.K / 2), (uint32_t)nrows * (uint32_t)(d.K / 2));
    const rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + (int64_t)t0 * d.xs * EX,
                                (uint32_t)((ntok - 1) * d.xs + d.K) * EX);
    const rsrc_t rs = make_rsrc(a.w_scale + (int64_t)n0 * blocks, (uint32_t)nrows * (uint32_t)blocks);
    const rsrc_t rxs = make_rsrc(a.x_scale + (int64_t)t0 * blocks,
                                 MODE == kSixteen ? 0 : (uint32_t)ntok * (uint32_t)blocks);

    // this lane's first weight row (the others follow 4 rows apart), and the chunks and scales that
    // this thread brings to LDS
    const int row0 = wave * 16 * RT + 4 * RT * (n16 >> 2) + (n16 & 3);
    const uint32_t srow = (uint32_t)row0 * (uint32_t)blocks + g, sstep = 4u * (uint32_t)blocks;
    // (row / CH of a chunk's place: the same for all of a thread's chunks)
    const int turn = CH == 16 ? n16 : n16 >> 1;
    const uint32_t chunk = 16u * ((tid % CH) ^ ((tid >> 4) & (CH - 1)));
    const uint32_t xrow = (uint32_t)(tid / CH) * (uint32_t)d.xs * EX + chunk;
    const uint32_t xstep = (256u / CH) * (uint32_t)d.xs * EX;
    const uint32_t xsrow = (uint32_t)(tid >> 2) * (uint32_t)blocks + (tid & 3), xsstep = 64u * (uint32_t)blocks;
    constexpr int XS = MODE == kSixteen ? 0 : (TT + 3) / 4;      // scale loads of a thread

    struct Stage {
        i32x4 w[RT];
        int s[RT], xs[XS ? XS : 1];
    };
    f32x4 acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = zero4();

    // everything of stage s on its way: tokens to LDS, the rest to registers; what lies past a row's
    // or the tile's end comes back as zeros
    auto request = [&](int s, char *x, Stage &w) {
        const uint32_t xo = xrow + (chunk + (uint32_t)PITCH * s < (uint32_t)d.K * EX ? 0u : kNothing);
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void *)(x + (q * 256 + wave * 64) * 16), 16,
                                                     xo + q * xstep, PITCH * s, 0, 0);
        // (a scale byte for 16 bytes of weights)
        const uint32_t so = srow + (4 * s + g < blocks ? 0u : kNothing / 16), wo = 16u * so;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            w.w[r] = buf16(rw, wo + r * (16u * sstep), 64u * s);
            w.s[r] = buf1(rs, so + r * sstep, 4u * s);
        }
#pragma unroll
        for (int q = 0; q < XS; ++q)
            w.xs[q] = buf1(rxs, xsrow + (4 * s + (tid & 3) < blocks ? 0u : kNothing) + q * xsstep, 4u * s);
    };
    // the tokens' scales next to their values
    auto deposit = [&](const Stage &w, uint8_t *xs) {
#pragma unroll
        for (int q = 0; q < XS; ++q)
            if (TT % 4 == 0 || tid < 4 * TOK) xs[q * 256 + tid] = (uint8_t)w.xs[q];
    };
    auto multiply = [&](const char *x, const uint8_t *xs, const Stage &wt) {
        const char *const xl = x + n16 * PITCH;
        if constexpr (MODE == kEight) {
            i32x4 f[2][2];
            int b[2];
            auto take = [&](int t) {
                f[t & 1][0] = *reinterpret_cast<const i32x4 *>(xl + 16 * t * PITCH + 16 * (g ^ turn));
                f[t & 1][1] = *reinterpret_cast<const i32x4 *>(xl + 16 * t * PITCH + 16 * ((4 + g) ^ turn));
                b[t & 1] = xs[4 * (16 * t + n16) + g];
            };
            take(0);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (t + 1 < TT) take(t + 1);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r][t] = mma_8bit(wt.w[r], wt.s[r], f[t & 1][0], f[t & 1][1], b[t & 1], acc[r][t]);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bf16x8 w[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) w[r] = widen_codes((uint32_t)wt.w[r][i], (uint32_t)wt.s[r]);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    bf16x8 v;
                    if constexpr (MODE == kSixteen)
                        v = *reinterpret_cast<const bf16x8 *>(xl + 16 * t * PITCH + 16 * ((4 * g + i) ^ turn));
                    else {
                        const uint32_t b = xs[4 * (16 * t + n16) + g];
                        v = widen_8bit(*reinterpret_cast<const u32x2 *>(
                                           xl + 16 * t * PITCH + 16 * ((2 * g + (i >> 1)) ^ turn) + 8 * (i & 1)),
                                       __uint_as_float(b << 23));
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) acc[r][t] = Mma<bf16>::run(w[r], v, acc[r][t]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    Stage wa, wb;
    request(0, xa, wa);
    deposit(wa, sa);
    __syncthreads();
    int s = 0;
    for (; s + 2 <= stages; s += 2) {
        request(s + 1, xb, wb);
        multiply(xa, sa, wa);
        deposit(wb, sb);
        __syncthreads();
        request(s + 2, xa, wa);
        multiply(xb, sb, wb);
        deposit(wa, sa);
        __syncthreads();
    }
    if (s < stages) multiply(xa, sa, wa);

    TO *const out = static_cast<TO *>(a.out);
    const int n = n0 + wave * 16 * RT + 4 * RT * g;
    float bias[4 * RT];
#pragma unroll
    for (int e = 0; e < 4 * RT; ++e) bias[e] = a.bias && n + e < d.N ? a.bias[n + e] : 0.0f;
    constexpr int VE = 4 * RT * sizeof(TO) >= 16 ? 16 / sizeof(TO) : 4 * RT;      // elements a store
    const bool wide = n + 4 * RT <= d.N && ((uintptr_t)out | (uint64_t)d.os * sizeof(TO) | n * sizeof(TO)) %
                                                (VE * sizeof(TO)) == 0;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int tok = t0 + 16 * t + n16;
        if (tok >= d.T) continue;
        float y[4 * RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[4 * r + e] = acc[r][t][e] + bias[4 * r + e];
        TO *const to = out + (int64_t)tok * d.os + n;
        if (wide) {
#pragma unroll
            for (int e = 0; e < 4 * RT; e += VE) {
                RawV<TO, VE> o;
                o.set(y + e);
                o.store(to + e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4 * RT; ++e)
                if (n + e < d.N) to[e] = from_f32<TO>(y[e]);
        }
    }
}

size_t linear_workspace(const LinearDims &) { return 0; }

// Which kernel, and its tile.
struct LinearPlan {
    bool tile;
    int mode;
    const char *name;
};
static LinearPlan linear_plan(const LinearDims &d) {
    LinearPlan p;
    // float32 results of 8-bit rows come from widened values
    p.mode = !d.e4m3 ? kSixteen : d.out_bf16 ? kEight : kWidened;
    p.tile = d.T > 64;
    p.name = p.tile ? "tile" : "split";
    return p;
}
const char *linear_kernel_name(const LinearDims &d) { return linear_plan(d).name; }

template <int MODE, int TT, int RT, typename TO>
static void linear_tile(const LinearDims &d, const LinearArgs &a, hipStream_t st) {
    const int tt = (d.T + 16 * TT - 1) / (16 * TT), nt = (d.N + 64 * RT - 1) / (64 * RT);
    hipLaunchKernelGGL((linear_tile_kernel<MODE, TT, RT, TO>), dim3((unsigned)(tt * nt)), dim3(256), 0, st, d, a, tt,
                       nt);
}
template <bool E4M3, typename TO>
static void linear_split(const LinearDims &d, const LinearArgs &a, hipStream_t st) {
    const unsigned nb = (unsigned)((d.N + 15) / 16);
    if (d.T <= 16)
        hipLaunchKernelGGL((linear_kernel<E4M3, 1, 1, TO>), dim3(nb, 1), dim3(256), 0, st, d, a);
    else
        hipLaunchKernelGGL((linear_kernel<E4M3, 4, 2, TO>), dim3((unsigned)((d.N + 31) / 32), (unsigned)((d.T + 63) / 64)),
                           dim3(256), 0, st, d, a);
}
template <int MODE, typename TO>
static void linear_t(const LinearDims &d, const LinearArgs &a, const LinearPlan &p, hipStream_t st) {
    if (p.tile) linear_tile<MODE, 8, 4, TO>(d, a, st);
    else linear_split<MODE != kSixteen, TO>(d, a, st);
}

void launch_linear(const LinearDims &d, const LinearArgs &a, void *, void *stream)
{
    if (d.T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const LinearPlan p = linear_plan(d);
    if (p.mode == kEight) linear_t<kEight, bf16>(d, a, p, st);
    else if (p.mode == kWidened) linear_t<kWidened, float>(d, a, p, st);
    else if (d.out_bf16) linear_t<kSixteen, bf16>(d, a, p, st);
    else linear_t<kSixteen, float>(d, a, p, st);
}

// ---------------------------------------------------------------------------
// Weights to codes: 32 of a row a thread, once for a model.
template <typename T>
__global__ __launch_bounds__(256) void encode_kernel(int64_t blocks, const T *__restrict__ w,
                                                     uint8_t *__restrict__ codes, uint8_t *__restrict__ scale)
{
    const int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (b >= blocks) return;
    float v[32], top = 0.0f;
    load_run<T, 32>(w + b * 32, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fabsf(v[i]) < __builtin_inff() ? fmaxf(top, fabsf(v[i])) : top;
    // top = 1.m 2^e and 6 = 1.5 2^2: the least s with top <= 6 2^s is e - 2, one more where
    // 1.m > 1.5
    const uint32_t bits = __float_as_uint(top);
    int e = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);
    e = e < 1 ? 1 : e;
    const float inv = __uint_as_float((254u - (uint32_t)e) << 23);
    uint32_t word[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        // scaling by a power of two is exact (what it flushes is far below 0.25); between two
        // values the even code takes the middle
        const float m = fabsf(v[i]) * inv;
        uint32_t c = (m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) + (m >= 3.5f) + (m > 5.0f);
        c |= v[i] < 0.0f ? 8u : 0u;
        word[i / 8] |= c << (4 * (i % 8));
    }
    *reinterpret_cast<uint4 *>(codes + b * 16) = make_uint4(word[0], word[1], word[2], word[3]);
    scale[b] = (uint8_t)e;
}

void launch_linear_encode(int N, int K, bool is_bf16, const void *w, uint8_t *codes, uint8_t *scale,
                          void *stream)
{
    const int64_t blocks = (int64_t)N * (K / 32);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)((blocks + 255) / 256));
    if (is_bf16)
        hipLaunchKernelGGL(encode_kernel<bf16>, grid, dim3(256), 0, st, blocks, static_cast<const bf16 *>(w), codes,
                           scale);
    else
        hipLaunchKernelGGL(encode_kernel<float>, grid, dim3(256), 0, st, blocks, static_cast<const float *>(w), codes,
                           scale);
}

}  // namespace ssd
