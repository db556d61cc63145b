// Products with 4-bit weights: y[t,n] = sum over k of x[t,k] w[n,k] + bias[n].
//
// The matrix instructions take the weights as their first operand (16 weight
// rows) and the tokens as their second (16 tokens), so that a lane's results
// are 4 neighbouring outputs of one token. K goes in steps of 128: lane l of
// a wave reads 16 bytes of weight row l % 16, the 32 codes of block l / 16 of
// the step, as they lie in memory.
//   The codes are widened to bfloat16 with their block's power of two (exact),
//   8-bit rows too, and four 16 x 16 x 32 instructions each take 8 of them; the
//   order of K inside the step does not matter as long as both operands keep it.
//   8-bit rows whose products may be cut (cut_products): one 16 x 16 x 128
//   instruction takes codes, 8-bit values and the exponent bytes of both. It
//   expects of a lane's 32 token values the first 16 from K = 16 (l / 16) and the
//   others from 64 + 16 (l / 16), while a lane's exponent byte belongs to block
//   l / 16 of either operand.
#include <stdint.h>

#include "ssd_layer_device.h"
#include "ssd_step.h"

namespace ssd {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

enum LinearMode {
    kEight,      // 8-bit rows, scaled 8-bit instruction: products cut
    kSixteen,    // bfloat16 rows
    kWidened     // 8-bit rows widened to bfloat16
};


// Byte offset of a lane that has nothing to read: past every resource's end.
constexpr uint32_t kNothing = 0x40000000u;     // (twice it is still past the end)

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

// 8 values of 8 bits widened to bfloat16 and scaled by s, a power of two.
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

__device__ __forceinline__ f32x4 mma_8bit(i32x4 w, int ws, i32x4 x0, i32x4 x1, int xs, f32x4 c) {
    const i32x8 a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    const i32x8 b = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
    // (first operand 4-bit, second e4m3; exponents from the lowest byte)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 0, 0, ws, 0, xs);
}

// ---------------------------------------------------------------------------
// Very few tokens: a block of 4 waves takes 16 weight rows, all tokens (at most
// 16) and all of K. The tokens go to LDS once; the waves take K in turn, 256
// values at a time, their weights straight to registers, all of a wave's first
// UNITS turns on their way before the tokens are waited for, and are joined in
// LDS. Bound by the weights' bytes (4 tokens, 4096 to 18560: 16.5 us, 2.5 TB/s) and, for small
// ones, by the chain of loads, products and join (one, 2560 to 10576: 6.3 us). What counts is few loads,
// whatever each brings: two of weights and, where rows of scales are whole words (WORDS), one of scales
// for 4 K of products.
template <int MODE, bool WORDS, typename TO>
__global__ __launch_bounds__(256) void linear_few_kernel(LinearDims d, LinearArgs a, int pitch)
{
    constexpr int EX = MODE == kSixteen ? 2 : 1, W = 4, UNITS = 3;
    extern __shared__ __align__(16) char xs_[];           // T rows of `pitch` bytes, then their scales
    __shared__ f32x4 part[W][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), n16 = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * 16, blocks = d.K / 32, units = (blocks + 7) / 8;
    const int nrows = d.N - n0 < 16 ? d.N - n0 : 16;
    const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * (d.K / 2), (uint32_t)nrows * (uint32_t)(d.K / 2));
    const rsrc_t rs = make_rsrc(a.w_scale + (int64_t)n0 * blocks, (uint32_t)nrows * (uint32_t)blocks);

    struct Unit {
        i32x4 w[2];
        uint32_t s[2];
    };
    // (what lies past a row's or the tile's end, or past the last unit, comes back as zeros)
    auto request = [&](int u, Unit &t) {
        const uint32_t row = (uint32_t)n16 * (uint32_t)blocks;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t off = 8 * u + 4 * h + g < blocks ? 0u : kNothing;
            t.w[h] = buf16(rw, 16u * row + 16u * g + off, 128u * u + 64u * h);
            if constexpr (!WORDS) t.s[h] = (uint32_t)buf1(rs, row + g + off, 8u * u + 4u * h);
        }
        if constexpr (WORDS) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)(row + (u < units ? 0u : kNothing)), 8 * u, 0);
            t.s[0] = (uint32_t)v[0];          // (the lane's byte is taken out where it is used)
            t.s[1] = (uint32_t)v[1];
        }
    };
    Unit t[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) request(wave + W * i, t[i]);

    // tokens, filled up with zeros to whole units
    const int chunks = d.K * EX / 16, all = pitch / 16;
    for (int tok = 0; tok < d.T; ++tok) {
        const i32x4 *const from = reinterpret_cast<const i32x4 *>(static_cast<const char *>(a.x) + (int64_t)tok * d.xs * EX);
        for (int c = tid; c < all; c += 256)
            *reinterpret_cast<i32x4 *>(xs_ + tok * pitch + 16 * c) = c < chunks ? from[c] : i32x4{0, 0, 0, 0};
    }
    char *const xscale = xs_ + d.T * pitch;
    if (MODE != kSixteen)
        for (int i = tid; i < d.T * 8 * units; i += 256) {
            const int tok = i / (8 * units), b = i - tok * 8 * units;
            xscale[i] = b < blocks ? (char)a.x_scale[(int64_t)tok * blocks + b] : 0;
        }
    __syncthreads();

    const int tok = n16 < d.T ? n16 : d.T - 1;             // (columns past the last token are not stored)
    const char *const x = xs_ + tok * pitch;
    f32x4 acc = zero4();
    for (int u0 = wave; u0 < units; u0 += W * UNITS) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int u = u0 + W * i;
            if (u < units) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const char *const xk = x + (256 * u + 128 * h) * EX;
                    const uint32_t ws = WORDS ? t[i].s[h] >> (8 * g) & 255u : t[i].s[h];
                    if constexpr (MODE == kSixteen) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc = Mma<bf16>::run(widen_codes((uint32_t)t[i].w[h][j], ws),
                                                 *reinterpret_cast<const bf16x8 *>(xk + 64 * g + 16 * j), acc);
                    } else {
                        const uint32_t b = (uint8_t)xscale[tok * 8 * units + 8 * u + 4 * h + g];
                        if constexpr (MODE == kEight)
                            acc = mma_8bit(t[i].w[h], (int)ws, *reinterpret_cast<const i32x4 *>(xk + 16 * g),
                                           *reinterpret_cast<const i32x4 *>(xk + 64 + 16 * g), (int)b, acc);
                        else
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc = Mma<bf16>::run(widen_codes((uint32_t)t[i].w[h][j], ws),
                                                     widen_8bit(*reinterpret_cast<const u32x2 *>(xk + 32 * g + 8 * j),
                                                                __uint_as_float(b << 23)), acc);
                    }
                }
            }
            if (u + W * UNITS < units) request(u + W * UNITS, t[i]);
        }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int k = 1; k < W; ++k) {
        const f32x4 o = part[k][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += o[e];
    }
    TO *const out = static_cast<TO *>(a.out);
    if (n16 < d.T)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = n0 + 4 * g + e;
            if (n < d.N) out[(int64_t)n16 * d.os + n] = from_f32<TO>(acc[e] + (a.bias ? a.bias[n] : 0.0f));
        }
}

// ---------------------------------------------------------------------------
// Many tokens: a block of WT x WN waves takes 16 TT WT tokens and 16 RT WN weight
// rows, 16 TT by 16 RT a wave. Tokens, weights and scales go to LDS by the loads
// themselves, a stage of K (128 values of 8-bit rows, 64 of bfloat16) in one of
// NBUF buffers: while a stage is multiplied the next NBUF - 1 are on their way.
// Bound by the matrix units with what feeds them: 4096 tokens, 2560 to 10576 186 us in
// bfloat16 and in widened 8 bits (1190 TFLOP/s; 8192 each way 758 and 749, 1450 and 1470), 100 with
// cut products (2210; 381, 2880).
// With cut products and the loads taken out a 128 x 256 stage goes from 0.95 to 0.6 us, with the products
// taken out it stays at 0.9. Where in a load's way that time goes is not known: the address units
// are busy for 32 % of this tile's time and 52 % of that of 192 x 256 (TA_BUSY_avr).
//
// A token's 128 bytes of a stage are 8 chunks, chunk c in place c ^ token / 2 % 8,
// so that the 16 tokens that a fragment reads together touch all banks. Weight
// rows lie in the order in which the fragments take them, which is such that a
// lane's results of its RT fragments are 4 RT neighbouring outputs.
//
// Scales take a word each: of kWords the 4 bytes of a stage in one (their arrays' rows are whole words
// then), of kBytes one byte. kQuads (rows are whole 16 bytes) loads them for four stages at once, to
// one of two places of their own: a row's scales are in a line of their own, which takes a load
// whatever is used of it. For 128 x 256 with cut products, which is bound by its loads: 384 tokens, 4096 to
// 18560 35.2 -> 33.3 us; the larger tiles have fewer of them and lose by reading the bytes apart (192 x 256,
// 4096 tokens, 5120 to 2560: 54.2 -> 56.8).
enum Scales { kBytes, kWords, kQuads };
typedef __attribute__((address_space(3))) void lds_void;

// Loads of 16, 4 or 1 bytes a lane straight to LDS, the lanes' one behind the other from `to` on (a
// word each for 4 and 1), written as instructions that the compiler does not count: it would wait for
// all of them before it reads any other LDS. What waits for them is wait_and_meet(). They have no
// result register, and the address is taken when they are issued. (m0 has no other user here.)
struct LdsSource {
    i32x4 r;
    __device__ __forceinline__ LdsSource(const void *base, uint32_t bytes) {
        const uint64_t b = (uint64_t)base;
        r = i32x4{(int)(uint32_t)b, (int)(uint32_t)(b >> 32) & 0xffff, (int)bytes, 0x00020000};
    }
};
__device__ __forceinline__ uint32_t lds_address(const void *p) { return (uint32_t)(uintptr_t)(const lds_void *)p; }
__device__ __forceinline__ void to_lds16(i32x4 r, uint32_t to, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(off),
                 "s"(r), "s"(at) : "memory");
}
__device__ __forceinline__ void to_lds4(i32x4 r, uint32_t to, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(to), "v"(off),
                 "s"(r), "s"(at) : "memory");
}
__device__ __forceinline__ void to_lds1(i32x4 r, uint32_t to, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds" ::"s"(to), "v"(off),
                 "s"(r), "s"(at) : "memory");
}

// Every wave waits for all but its newest `N` loads and for its own LDS reads, then for the others.
template <int N> __device__ __forceinline__ void wait_and_meet() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The same where a load came before the newest `N` and is not waited for either if `more` is 0, and
// such a load. (The compiler does not see the branches: with its own it lost the products' registers.)
template <int N> __device__ __forceinline__ void wait_and_meet(int more) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_cmp_eq_u32 %2, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(%0)\n1:\n\t"
                 "s_waitcnt vmcnt(%1) lgkmcnt(0)\n\ts_barrier" ::"n"(N), "n"(N + 1), "s"(more) : "memory", "scc");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void to_lds16_if0(int more, i32x4 r, uint32_t to, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_cmp_eq_u32 %4, 0\n\ts_cbranch_scc0 1f\n\t"
                 "buffer_load_dwordx4 %1, %2, %3 offen lds\n1:" ::"s"(to), "v"(off), "s"(r), "s"(at), "s"(more)
                 : "memory", "scc");
}

// Buffer I of a block (objects of their own: the compiler then sees that a read of one does not
// depend on loads on their way to another).
template <typename B, int I> __device__ __forceinline__ B &buffer() {
    __shared__ __align__(16) B b;
    return b;
}
template <int N, int I = 0, typename F> __device__ __forceinline__ void each(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<N, I + 1>(f);
    }
}

template <int MODE, int WT, int WN, int WK, int TT, int RT, int NSUB, int NBUF, Scales SCALES, int PERCU, typename TO>
__global__ __launch_bounds__(64 * WT * WN * WK, (WT * WN * WK * PERCU + 3) / 4) void linear_tile_kernel(LinearDims d, LinearArgs a,
                                                                                           int ttiles, int ntiles)
{
    constexpr int THREADS = 64 * WT * WN * WK, TOK = 16 * TT * WT, ROWS = 16 * RT * WN;
    constexpr int EX = MODE == kSixteen ? 2 : 1, KS = 128 / EX, BS = KS / 32;    // values, blocks a stage
    constexpr int CW = KS / 32;                                                 // chunks of a weight row a stage
    constexpr int LX = (TOK * 8 + THREADS - 1) / THREADS, LW = (ROWS * CW + THREADS - 1) / THREADS;     // loads of a thread
    // words of scales: the tokens' and, from a whole wave's on, the weights'
    constexpr bool WORDS = SCALES != kBytes, QUADS = SCALES == kQuads;
    constexpr int SX = MODE == kSixteen ? 0 : WORDS ? TOK : TOK * BS, SO = (SX + 63) / 64 * 64;
    constexpr int SW = WORDS && MODE != kSixteen ? ROWS : ROWS * BS;
    constexpr int LS = (SO + SW + THREADS - 1) / THREADS;
    constexpr int LOADS = LX + LW + (QUADS ? 0 : LS);
    static_assert(!QUADS || (MODE != kSixteen && NSUB == 1 && NBUF == 3 && LS == 1), "one load of scales");
    static_assert(RT == 1 || RT == 2 || RT == 4 || RT == 8, "whole stores");
    static_assert(LX == 1 || TOK * 8 % THREADS == 0, "loads that are all of the tile's tokens");
    static_assert(NSUB % WK == 0 && LOADS * NSUB * (NBUF - 2) < 64, "waits that can be counted");
    // chunks and words of a step, rounded up to a wave's load; every wave makes the same number of
    // loads, those that have nothing to bring into `spare`
    constexpr int NX = (TOK * 8 + 63) / 64 * 64, NW = (ROWS * CW + 63) / 64 * 64, NS = (SO + SW + 63) / 64 * 64;
    struct Rows {
        char x[NX * 16], w[NW * 16];
    };
    struct RowsAndScales : Rows {
        uint32_t s[NS];
    };
    struct Fours {
        uint32_t s[2][NS][4];
    };
    using Step = std::conditional_t<QUADS, Rows, RowsAndScales>;
    struct Buffer {
        Step step[NSUB];
    };
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), n16 = lane & 15, g = lane >> 4;
    constexpr bool EXACT = LX * THREADS == NX && LW * THREADS == NW && LS * THREADS == NS;
    uint32_t nowhere = 0;
    if constexpr (!EXACT) {
        __shared__ __align__(16) char spare[1024];
        nowhere = lds_address(spare);
    }
    auto &fours = buffer<std::conditional_t<QUADS, Fours, uint32_t>, NBUF>();        // (nothing without QUADS)
    const int wt = wave / WN % WT, wn = wave % WN, wk = wave / (WN * WT);

    // tiles in groups of token tiles, so that the blocks of one L2 share rows and weights
    constexpr int kGroup = 1024 / TOK;
    const int id = xcd_logical_block((int)blockIdx.x, ttiles * ntiles);
    const int grp = id / (kGroup * ntiles), in = id - grp * (kGroup * ntiles);
    const int gm = ttiles - grp * kGroup < kGroup ? ttiles - grp * kGroup : kGroup;
    const int nt = in / gm, t0 = (grp * kGroup + in - nt * gm) * TOK, n0 = nt * ROWS;

    const int blocks = d.K / 32, stages = (blocks + BS * NSUB - 1) / (BS * NSUB);
    const int nrows = d.N - n0 < ROWS ? d.N - n0 : ROWS, ntok = d.T - t0 < TOK ? d.T - t0 : TOK;
    const LdsSource rw(a.w + (int64_t)n0 * (d.K / 2), (uint32_t)nrows * (uint32_t)(d.K / 2));
    const LdsSource rx(static_cast<const char *>(a.x) + (int64_t)t0 * d.xs * EX,
                                (uint32_t)((ntok - 1) * d.xs + d.K) * EX);
    const LdsSource rs(a.w_scale + (int64_t)n0 * blocks, (uint32_t)nrows * (uint32_t)blocks);
    const LdsSource rxs(a.x_scale + (int64_t)t0 * blocks,
                                 MODE == kSixteen ? 0 : (uint32_t)ntok * (uint32_t)blocks);

    // the weight row in place p of the tile
    auto row_in = [](int p) {
        const int m = p & 15, r = (p >> 4) % RT, w = p / (16 * RT);
        return w * 16 * RT + 4 * RT * (m >> 2) + 4 * r + (m & 3);
    };
    // what this thread brings to LDS: offsets in the tile, and the block in the stage
    const uint32_t chunk = 16u * ((tid & 7) ^ ((tid >> 4) & 7));
    const uint32_t xrow = tid < TOK * 8 ? (uint32_t)(tid >> 3) * (uint32_t)d.xs * EX + chunk : kNothing;
    const uint32_t xstep = (THREADS / 8u) * (uint32_t)d.xs * EX;
    uint32_t wrow[LW], srow[LS];
    int sblk[LS];
#pragma unroll
    for (int q = 0; q < LW; ++q) {
        const int c = q * THREADS + tid;
        wrow[q] = c < ROWS * CW ? (uint32_t)row_in(c / CW) * (uint32_t)(d.K / 2) + 16u * (c % CW) : kNothing;
    }
#pragma unroll
    for (int q = 0; q < LS; ++q) {
        const int e = q * THREADS + tid;
        constexpr bool one = WORDS && MODE != kSixteen;
        const int f = e < SO ? e : e - SO, at = one ? f : f / BS;
        sblk[q] = one ? 0 : f % BS;
        srow[q] = f < (e < SO ? SX : SW) ? (uint32_t)(e < SO ? at : row_in(at)) * (uint32_t)blocks + sblk[q] : kNothing;
    }

    f32x4 acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = zero4();

    // load q of step s on its way; what lies past a row's or the tile's end comes as zeros
    auto load_one = [&](auto Q, int s, const Step &b) __attribute__((always_inline)) {
        constexpr int q = decltype(Q)::value;
        const uint32_t bx = lds_address(b.x), bw = bx + sizeof(b.x);
        if constexpr (q < LX) {
            const uint32_t xo = xrow + (chunk + 128u * s < (uint32_t)d.K * EX ? 0u : kNothing);
            const int c = q * THREADS + wave * 64;
            to_lds16(rx.r, c < NX ? bx + 16 * c : nowhere, xo + q * xstep, 128u * s);
        } else if constexpr (q < LX + LW) {
            const uint32_t wo = BS * s + tid % CW < blocks ? 0u : kNothing;
            const int c = (q - LX) * THREADS + wave * 64;
            to_lds16(rw.r, c < NW ? bw + 16 * c : nowhere, wrow[q - LX] + wo, 16u * BS * s);
        } else {
            constexpr int i = q - LX - LW;
            const int e = i * THREADS + wave * 64;
            const uint32_t so = srow[i] + (BS * s + sblk[i] < blocks ? 0u : kNothing);
            const i32x4 r = e < SO ? rxs.r : rs.r;                               // (the same in a wave)
            const uint32_t to = e < NS ? bw + (uint32_t)sizeof(b.w) + 4 * e : nowhere;
            if constexpr (WORDS && MODE != kSixteen) to_lds4(r, to, so, BS * s);
            else to_lds1(r, to, so, BS * s);
        }
    };
    // the scales of stages s .. s + 3, where s is a multiple of 4
    auto load_four = [&](int s) __attribute__((always_inline)) {
        if constexpr (QUADS) {
            const int e = wave * 64;
            to_lds16_if0(s & 3, e < SO ? rxs.r : rs.r, e < NS ? lds_address(fours.s[(s >> 2) & 1]) + 16 * e : nowhere,
                         srow[0] + (BS * s < blocks ? 0u : kNothing), (uint32_t)(BS * s));
        }
    };
    // a share of a stage's loads: those of turn t of `turns`
    auto request_share = [&](auto T_, auto N_, int s, const Buffer &b) __attribute__((always_inline)) {
        constexpr int t = decltype(T_)::value, turns = decltype(N_)::value, all = LOADS * NSUB;
        constexpr int from = all * t / turns, to = all * (t + 1) / turns;
        if constexpr (t == 0) load_four(s);
        each<to - from>([&](auto I) __attribute__((always_inline)) {
            constexpr int l = from + decltype(I)::value;
            load_one(std::integral_constant<int, l % LOADS>{}, s * NSUB + l / LOADS, b.step[l / LOADS]);
        });
    };
    auto request = [&](int s, const Buffer &b) __attribute__((always_inline)) {
        request_share(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, s, b);
    };
    // scale of block `blk` of token (from 0) or weight row (from SO) `at` in stage s
    auto scale_of = [&](const Step &b, int s, int from, int at, int blk) __attribute__((always_inline)) -> uint32_t {
        if constexpr (QUADS)
            return reinterpret_cast<const uint8_t *>(fours.s[(s >> 2) & 1][from + at])[4 * (s & 3) + blk];
        else if constexpr (WORDS && MODE != kSixteen) return reinterpret_cast<const uint8_t *>(b.s + from)[4 * at + blk];
        else return b.s[from + at * BS + blk];
    };
    // (between(turn, turns) is called as the products go)
    auto multiply_step = [&](const Step &b, int s, auto between) __attribute__((always_inline)) {
        const char *const x = b.x + (wt * 16 * TT + n16) * 128;
        const char *const w = b.w + (wn * 16 * RT + n16) * (CW * 16);
        const int turn = n16 >> 1;
        uint32_t ws[RT][MODE == kSixteen ? 2 : 1];      // (by block: a lane group's own, or both)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < (MODE == kSixteen ? 2 : 1); ++i)
                ws[r][i] = scale_of(b, s, SO, wn * 16 * RT + 16 * r + n16, MODE == kSixteen ? i : g);
        if constexpr (MODE == kEight) {
            i32x4 wf[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                wf[r] = *reinterpret_cast<const i32x4 *>(w + r * (256 * CW) + 16 * g);
            constexpr int AHEAD = TT > 1 ? 1 : 0, RING = AHEAD + 1;
            i32x4 f[RING][2];
            int xs[RING];
            auto take = [&](int t) __attribute__((always_inline)) {
                f[t % RING][0] = *reinterpret_cast<const i32x4 *>(x + t * 2048 + 16 * (g ^ turn));
                f[t % RING][1] = *reinterpret_cast<const i32x4 *>(x + t * 2048 + 16 * ((4 + g) ^ turn));
                xs[t % RING] = (int)scale_of(b, s, 0, wt * 16 * TT + 16 * t + n16, g);
            };
#pragma unroll
            for (int t = 0; t < AHEAD; ++t) take(t);
            each<TT>([&](auto I) __attribute__((always_inline)) {
                constexpr int t = decltype(I)::value;
                if constexpr (t + AHEAD < TT) take(t + AHEAD);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r][t] = mma_8bit(wf[r], (int)ws[r][0], f[t % RING][0], f[t % RING][1], xs[t % RING], acc[r][t]);
                __builtin_amdgcn_sched_barrier(0);
                between(I, std::integral_constant<int, TT>{});
                __builtin_amdgcn_sched_barrier(0);
            });
        } else if constexpr (MODE == kSixteen) {
            // lane group g takes K = 8 g .. 8 g + 7 of a block, a block an instruction
            uint32_t wf[RT][2];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) wf[r][i] = *reinterpret_cast<const uint32_t *>(w + r * (256 * CW) + 16 * i + 4 * g);
            // (fragments of the tokens are read AHEAD before they are multiplied)
            constexpr int AHEAD = 3;
            bf16x8 f[AHEAD + 1];
            auto take = [&](int k) __attribute__((always_inline)) {
                f[k % (AHEAD + 1)] = *reinterpret_cast<const bf16x8 *>(x + k % TT * 2048 + 16 * ((4 * (k / TT) + g) ^ turn));
            };
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) take(k);
            bf16x8 wv[RT];
            each<2 * TT>([&](auto I) __attribute__((always_inline)) {
                constexpr int k = decltype(I)::value;
                if constexpr (k + AHEAD < 2 * TT) take(k + AHEAD);
                if constexpr (k % TT == 0)
#pragma unroll
                    for (int r = 0; r < RT; ++r) wv[r] = widen_codes(wf[r][k / TT], ws[r][k / TT]);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r][k % TT] = Mma<bf16>::run(wv[r], f[k % (AHEAD + 1)], acc[r][k % TT]);
                __builtin_amdgcn_sched_barrier(0);
                between(I, std::integral_constant<int, 2 * TT>{});
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
            // lane group g takes block g, 8 values an instruction
            i32x4 wf[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                wf[r] = *reinterpret_cast<const i32x4 *>(w + r * (256 * CW) + 16 * g);
            each<4>([&](auto I) __attribute__((always_inline)) {
                constexpr int i = decltype(I)::value;
                bf16x8 wv[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) wv[r] = widen_codes((uint32_t)wf[r][i], ws[r][0]);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const uint32_t xs = scale_of(b, s, 0, wt * 16 * TT + 16 * t + n16, g);
                    const bf16x8 v = widen_8bit(*reinterpret_cast<const u32x2 *>(
                                                    x + t * 2048 + 16 * ((2 * g + (i >> 1)) ^ turn) + 8 * (i & 1)),
                                                __uint_as_float(xs << 23));
#pragma unroll
                    for (int r = 0; r < RT; ++r) acc[r][t] = Mma<bf16>::run(wv[r], v, acc[r][t]);
                }
                __builtin_amdgcn_sched_barrier(0);
                between(I, std::integral_constant<int, 4>{});
                __builtin_amdgcn_sched_barrier(0);
            });
        }
    };

    // the products of one buffer's stage, with the loads of stage `next` into another between them
    // (asked for all at once they hold the products up; with two buffers they have to be on their way
    // first: 4096 tokens, 5120 to 2560 with cut products 65 -> 59 us, with two buffers in bfloat16 118 -> 132)
    auto multiply = [&](const Buffer &b, int next, const Buffer &into) __attribute__((always_inline)) {
        if constexpr (NBUF == 2) {
            request(next, into);
            each<NSUB / WK>([&](auto U) __attribute__((always_inline)) { multiply_step(b.step[decltype(U)::value * WK + wk], next - NBUF + 1, [](auto, auto) __attribute__((always_inline)) {}); });
        } else
            each<NSUB / WK>([&](auto U) __attribute__((always_inline)) {
                constexpr int u = decltype(U)::value;
                multiply_step(b.step[u * WK + wk], next - NBUF + 1, [&](auto T_, auto N_) __attribute__((always_inline)) {
                    request_share(std::integral_constant<int, u * decltype(N_)::value + decltype(T_)::value>{},
                                  std::integral_constant<int, decltype(N_)::value * (NSUB / WK)>{}, next, into);
                });
            });
    };
    auto multiply_last = [&](const Buffer &b, int s) __attribute__((always_inline)) {
        each<NSUB / WK>([&](auto U) __attribute__((always_inline)) { multiply_step(b.step[decltype(U)::value * WK + wk], s, [](auto, auto) __attribute__((always_inline)) {}); });
    };

    // the stage in buffer I of a round of NBUF from `s` on
    int s = 0;
    auto stage = [&](auto I) __attribute__((always_inline)) {
        constexpr int i = decltype(I)::value;
        multiply(buffer<Buffer, i>(), s + i + NBUF - 1, buffer<Buffer, (i + NBUF - 1) % NBUF>());
        // (all but the loads that have just been asked for)
        if constexpr (QUADS) wait_and_meet<LOADS>((s + i + NBUF - 1) & 3);
        else wait_and_meet<(NBUF - 2) * NSUB * LOADS>();
    };
    auto last = [&](auto I) __attribute__((always_inline)) {
        if (s + decltype(I)::value < stages) multiply_last(buffer<Buffer, decltype(I)::value>(), s + decltype(I)::value);
    };
    each<NBUF - 1>([&](auto I) __attribute__((always_inline)) { request(decltype(I)::value, buffer<Buffer, decltype(I)::value>()); });
    wait_and_meet<(NBUF - 2) * NSUB * LOADS>();
    for (; s + NBUF <= stages; s += NBUF) each<NBUF>(stage);
    wait_and_meet<0>();
    each<NBUF - 1>(last);

    if constexpr (WK > 1) {
        // the waves that took other steps of the same tile, in order
        __shared__ f32x4 part[WK - 1][WT * WN][RT * TT][64];
        if (wk > 0)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t) part[wk - 1][wave % (WT * WN)][r * TT + t][lane] = acc[r][t];
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int k = 0; k < WK - 1; ++k)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const f32x4 o = part[k][wave % (WT * WN)][r * TT + t][lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][t][e] += o[e];
                }
    }

    TO *const out = static_cast<TO *>(a.out);
    const int n = n0 + wn * 16 * RT + 4 * RT * g;
    float bias[4 * RT];
#pragma unroll
    for (int e = 0; e < 4 * RT; ++e) bias[e] = a.bias && n + e < d.N ? a.bias[n + e] : 0.0f;
    constexpr int VE = 4 * RT * sizeof(TO) >= 16 ? 16 / sizeof(TO) : 4 * RT;      // elements a store
    const bool wide = n + 4 * RT <= d.N && ((uintptr_t)out | (uint64_t)d.os * sizeof(TO) | n * sizeof(TO)) %
                                                (VE * sizeof(TO)) == 0;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int tok = t0 + wt * 16 * TT + 16 * t + n16;
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

static LinearMode linear_mode(const LinearDims &d) {
    // The 8-bit instruction cuts the 32 products of a block off at 2^-13 of the largest: where a product of
    // 2688 was cancelled by another, results of up to 0.6 came out as 0. It is a caller's choice, for
    // bfloat16 results; others come from widened values.
    return !d.e4m3 ? kSixteen : d.cut && d.out_bf16 ? kEight : kWidened;
}

// The tiles that are built. One is taken by its estimated time on the CU that gets the most of
// them: its bytes, its products at a share of the rate that the tile reached on long prompts
// (TFLOP/s; the whole chip), or its stages at the time of one; and a time a round of blocks. On 185
// sizes (1 to 4096 tokens, 256 to 8192 values, 300 to 50257 outputs) the tile so taken was on average 1.0 %
// (bfloat16 rows) and 2.3 % (cut products) slower than the best of them, on 280 sizes of widened 8-bit rows
// 1.9 %, at most 30, 37 and 36 %. (Widened rows by the cut products' figures: 5.2 %, at most 71.)
// 192 x 256 is for sizes whose tiles of 256 leave CUs without one: 4096 tokens, 5120 to 2560 are 220 of
// them, not 160 (bfloat16 119.9 -> 104.2 us); 2048 tokens, 2560 to 10576: 128.8 -> 114.8.
struct Tile {
    int tokens, rows, threads, per_cu, steps;      // steps of 128 (bfloat16: 64) values a stage
    double rate[3];                                // by LinearMode
};
static constexpr Tile kTiles[] = {
    {16, 16, 256, 2, 4, {224, 103, 198}},       {16, 32, 128, 2, 1, {369, 191, 349}},
    {32, 32, 256, 1, 4, {385, 246, 307}},       {64, 64, 256, 2, 2, {898, 576, 547}},
    {128, 128, 512, 2, 1, {1793, 1014, 1054}},  {256, 256, 512, 1, 1, {2507, 1341, 1247}},
    {192, 256, 512, 1, 1, {2250, 1200, 1127}},  {128, 256, 512, 1, 1, {1850, 0, 1058}}};
// Bytes a microsecond of a CU, share of the rate, microseconds of a stage and what a further step of it adds,
// microseconds of a round.
struct TileTimes {
    double bytes, products, stage, step, round;
};
static constexpr TileTimes kTileTimes[3] = {
    {2.75e4, 0.944, 0.162, 0.267, 1.43}, {6.05e4, 0.531, 0.269, 0.264, 0.947}, {1.87e4, 0.501, 0.27, 0.261, 1.15}};
static const char *const kTileNames[] = {"16x16",   "16x32",   "32x32",   "64x64",
                                         "128x128", "256x256", "192x256", "128x256"};

static int linear_tile_of(const LinearDims &d) {
    const LinearMode mode = linear_mode(d);
    const TileTimes &c = kTileTimes[mode];
    const bool wide = mode == kSixteen;
    int best = -1;
    double least = 0;
    for (int i = 0; i < (wide ? 7 : 8); ++i) {
        const Tile &t = kTiles[i];
        const int64_t blocks = (int64_t)((d.T + t.tokens - 1) / t.tokens) * ((d.N + t.rows - 1) / t.rows);
        if (blocks > 0xffffffffLL / t.threads) continue;      // (more than a launch takes; of the largest never)
        const int64_t most = (blocks + 255) / 256, rounds = (most + t.per_cu - 1) / t.per_cu;     // of a CU
        const double bytes = (double)d.K * ((d.T < t.tokens ? d.T : t.tokens) * (wide ? 2 : 1) + t.rows * 0.53);
        const double flops = 2.0 * t.tokens * t.rows * d.K;
        const double stages = d.K / (wide ? 64.0 : 128.0) / t.steps;
        // microseconds
        const double by_bytes = most * bytes / c.bytes;
        const double by_products = most * flops * 256e-6 / (t.rate[mode] * c.products);
        const double by_stages = rounds * stages * c.stage * (1 + c.step * t.steps);
        double time = by_bytes > by_products ? by_bytes : by_products;
        time = (time > by_stages ? time : by_stages) + rounds * c.round;
        if (best < 0 || time < least) {
            least = time;
            best = i;
        }
    }
    return best;
}

// Up to 4 tokens: a block of every 16 weight rows reads them all; with more of them the tiles, which
// share them, are faster. On 8 sizes of 1 to 8 tokens this limit was on average 3.5 % (bfloat16 rows), 3.0 %
// (widened) and 3.9 % (cut) slower than the faster of the two ways; a limit of 8 3.9, 6.0 and 10.9 %, of 2
// 8.1, 4.2 and 2.6 % (8 tokens of 8 bits, 4096 to 18560: 19.8 us here and 14.9 by the tiles; 2560 to 10576:
// 8.5 and 9.9).
static bool linear_few(const LinearDims &d) {
    const int64_t bytes = (int64_t)d.T * (d.K + 255) / 256 * 256 * (d.e4m3 ? 1 : 2);
    return d.T <= 4 && bytes <= 48 << 10;
}
const char *linear_kernel_name(const LinearDims &d) { return linear_few(d) ? "few" : kTileNames[linear_tile_of(d)]; }

template <int MODE, int WT, int WN, int WK, int TT, int RT, int NSUB, int NBUF, Scales SCALES, int PERCU, typename TO>
static void linear_tile(const LinearDims &d, const LinearArgs &a, hipStream_t st) {
    const int tt = (d.T + 16 * TT * WT - 1) / (16 * TT * WT), nt = (d.N + 16 * RT * WN - 1) / (16 * RT * WN);
    hipLaunchKernelGGL((linear_tile_kernel<MODE, WT, WN, WK, TT, RT, NSUB, NBUF, SCALES, PERCU, TO>),
                       dim3((unsigned)(tt * nt)), dim3(64 * WT * WN * WK), 0, st, d, a, tt, nt);
}
template <int MODE, bool WORDS, typename TO>
static void linear_few_t(const LinearDims &d, const LinearArgs &a, hipStream_t st) {
    const int units = (d.K + 255) / 256, pitch = units * 256 * (MODE == kSixteen ? 2 : 1) + 16;
    const int scales = MODE == kSixteen ? 0 : d.T * 8 * units;
    hipLaunchKernelGGL((linear_few_kernel<MODE, WORDS, TO>), dim3((unsigned)((d.N + 15) / 16)), dim3(256),
                       d.T * pitch + scales, st, d, a, pitch);
}
template <int MODE, Scales W, typename TO>
static void linear_t(const LinearDims &d, const LinearArgs &a, hipStream_t st) {
    if (linear_few(d)) {
        if (d.K % 256 == 0 && (uintptr_t)a.w_scale % 8 == 0) linear_few_t<MODE, true, TO>(d, a, st);
        else linear_few_t<MODE, false, TO>(d, a, st);
        return;
    }
    // (blocks a CU that the buffers leave room for)
    constexpr int two = W == kWords || MODE == kSixteen ? 2 : 1;
    switch (linear_tile_of(d)) {
    case 0: return linear_tile<MODE, 1, 1, 4, 1, 1, 4, 3, W, 2, TO>(d, a, st);
    case 1: return linear_tile<MODE, 1, 2, 1, 1, 1, 1, 8, W, 2, TO>(d, a, st);
    case 2: return linear_tile<MODE, 1, 1, 4, 2, 2, 4, 3, W, 1, TO>(d, a, st);
    case 3: return linear_tile<MODE, 1, 4, 1, 4, 1, 2, 3, W, two, TO>(d, a, st);
    case 4: return linear_tile<MODE, 2, 4, 1, 4, 2, 1, 3, W, two, TO>(d, a, st);
    case 5:
        // (scales of a byte a word leave room for two buffers)
        return linear_tile<MODE, 2, 4, 1, 8, 4, 1, W == kWords || MODE == kSixteen ? 3 : 2, W, 1, TO>(d, a, st);
    case 6: return linear_tile<MODE, 2, 4, 1, 6, 4, 1, 3, W, 1, TO>(d, a, st);
    default:
        if constexpr (MODE == kEight && W == kWords)
            if (d.K % 512 == 0 && ((uintptr_t)a.x_scale | (uintptr_t)a.w_scale) % 16 == 0)
                return linear_tile<MODE, 2, 4, 1, 4, 4, 1, 3, kQuads, 1, TO>(d, a, st);
        if constexpr (MODE != kSixteen) linear_tile<MODE, 2, 4, 1, 4, 4, 1, 3, W, 1, TO>(d, a, st);
    }
}
void launch_linear(const LinearDims &d, const LinearArgs &a, void *stream)
{
    if (d.T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const LinearMode m = linear_mode(d);
    const bool words = d.K % 128 == 0 && ((uintptr_t)a.x_scale | (uintptr_t)a.w_scale) % 4 == 0;
    if (m == kEight) words ? linear_t<kEight, kWords, bf16>(d, a, st) : linear_t<kEight, kBytes, bf16>(d, a, st);
    else if (m == kWidened && d.out_bf16) words ? linear_t<kWidened, kWords, bf16>(d, a, st) : linear_t<kWidened, kBytes, bf16>(d, a, st);
    else if (m == kWidened) words ? linear_t<kWidened, kWords, float>(d, a, st) : linear_t<kWidened, kBytes, float>(d, a, st);
    else if (d.out_bf16) linear_t<kSixteen, kBytes, bf16>(d, a, st);
    else linear_t<kSixteen, kBytes, float>(d, a, st);
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
    // 1.m > 1.5; 6 2^125 = 1.5 2^127 is the largest whose codes all stay in bfloat16's range
    const uint32_t bits = __float_as_uint(top);
    int e = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);
    e = e < 1 ? 1 : e > 252 ? 252 : e;
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
