// Channel-wise selective scan over packed sequences (prompts) and for the few
// tokens of a verify step.
//
//     h_t[c,n] = exp(dt_t[c] A[c,n]) h_{t-1}[c,n] + dt_t[c] x_t[c] B_t[g,n]
//     y_t[c]   = (sum over n of h_t[c,n] C_t[g,n] + D[c] x_t[c]) silu(z_t[c])
//
// Every (channel, state) has a decay of its own, so the recurrence has no
// matrix product in it: each token costs one exponential, two products and two
// multiply-adds per (channel, state) on the vector units, which bound the
// prompt form: a wave issues 38 instructions for a token of its 16 channels (N =
// 16), 20 of which are those five for its 4 states a lane; the rest prepares step
// sizes and gates, moves rows and joins lanes. At 4 cycles each (8 an exponential)
// the 8192 tokens x 4096 channels of 1 prompt, run twice for their segments, take
// 256 us of issue alone; measured 262 us. The single-token form is bound by the
// states it reads and writes.
#include "ssd_layer.h"
#include "ssd_layer_device.h"
#include <cmath>

namespace ssd {

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) <= 1, with
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3: s times a polynomial in s^2,
// fitted on [0, 1/9] at Chebyshev's points, good to 8e-9 relative. Accurate relative
// to the result also where e is small, which a logarithm of the rounded 1 + e
// is not, and half the operations of the library's log1p.
__device__ __forceinline__ float softplus(float v) {
    const float e = __expf(-fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
    const float q = s * s;
    float p = 0.28174657f;
    p = p * q + 0.27961418f;
    p = p * q + 0.40024853f;
    p = p * q + 0.66666317f;
    p = p * q + 2.0f;
    return fmaxf(v, 0.0f) + p * s;
}
// (a NaN stays one: the median instruction would turn it into a bound)
__device__ __forceinline__ float transformed(const DtTf &tf, float raw, float bias) {
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(softplus(raw + bias), tf.lo), tf.hi);
}
__device__ __forceinline__ float step_size(const DtTf &tf, float raw, float bias) {
    return tf.on ? transformed(tf, raw, bias) : raw;
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
// for as long as the block runs; a block of 4 waves takes 256 / L channels of
// one group and one sequence, or one segment of it. The tokens are taken in
// groups of L: lane j of a channel reads x, dt and z of the group's token j,
// prepares its step size and gate once, and the group's L tokens are then run
// through one after the other, each lane taking token j's values from lane j.
// B and C of a stage of ST tokens are widened to float in LDS by the whole
// block (two buffers, one barrier a stage); the next stage's loads are in
// flight meanwhile. Rows are read through buffer resources that end with the
// sequence, so tokens past it come as zeros and are dropped on the way out.
//
// Segments. One sequence is a chain, and few channels leave most of the chip
// idle; then sequences are cut into segments of `seg` tokens. The recurrence
// is linear in its starting state: a first launch runs every segment but the
// last from zero (the first one from its cached state, finished at once) and
// keeps its final state and the sum of its steps; a second one chains those in
// front of it, exp(A sum dt) state + final, and runs each later segment again,
// with outputs. `cur` says which launch this is: 0 the only one, 1 and 2. Every
// later segment reads the final states of all before it, which grows with the
// square of their number: nothing at 8192 tokens, an eighth of the time at 262144
// (2048 channels, 512 segments of 512: 4551 us, where 16 times the 8192 tokens x 4096
// channels are 4040), and more beyond.
struct ScanSegs {
    int seg, cur;
    float *fin, *sum;   // [segments][C][N] final states, [segments][C] sums of steps
};

// One element through a resource, `row` bytes (a scalar, counted by the range check) and `off`
// into it; a register of its own until it is widened.
template <typename TX> __device__ __forceinline__ uint32_t buf_one(rsrc_t r, int off, int row) {
    if constexpr (sizeof(TX) == 2)
        return (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, off, row, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b32(r, off, row, 0);
}
template <typename TX> __device__ __forceinline__ float widen_one(uint32_t w) {
    return __uint_as_float(sizeof(TX) == 2 ? w << 16 : w);
}
template <typename TX> __device__ __forceinline__ void buf_put(rsrc_t r, float v, int off, int row) {
    const TX t = from_f32<TX>(v);
    if constexpr (sizeof(TX) == 2)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, t), r, off, row, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(t), r, off, row, 0);
}

template <typename TX, typename TS, int N, int L>
__global__ __launch_bounds__(256) void scan_kernel(
    int T, int S, int C, int G, int num_slots, int chb, ScanArgs a, int64_t xs, int64_t dts,
    int64_t zs, int64_t bs, int64_t cs, int64_t ys, DtTf tf, ScanSegs sg)
{
    constexpr int SPL = N / L, CB = 256 / L;
    constexpr int GROUPS = L == 16 ? 4 : 8;      // groups of L tokens in a stage
    constexpr int ST = L * GROUPS;
    constexpr int BCV = ST * N * 2 / 256;        // B, C values a thread stages
    constexpr int E = (int)sizeof(TX);
    __shared__ __align__(16) float bc[2][2][ST][N];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), j0 = tid % L;
    // Blocks go to the 8 XCDs in turn; the 4 blocks of L = 16 that share a row's 128
    // bytes are dealt to one XCD, whose L2 then fetches the line once.
    unsigned id = blockIdx.x;
    if (L == 16 && (id | 31u) < gridDim.x) id = (id & ~31u) | (id & 7u) << 2 | (id >> 3 & 3u);
    const int b = (int)(id / (unsigned)chb), cb = (int)(id % (unsigned)chb);
    const SeqTile tile = S > 1 && S <= kWave
                             ? heaviest_first(lane_seqs(a.cu, S, T, sg.seg, 1), S, sg.seg, b)
                             : find_tile(a.cu, S, T, sg.seg, 1, b);
    if (tile.seq < 0) return;
    const bool first = tile.t0 == 0, last = tile.t0 >= tile.len - sg.seg;
    if (sg.cur == 1 ? !first && last : sg.cur == 2 && first) return;
    const int per = C / G, gblocks = chb / G;
    const int g = cb / gblocks, c_first = (cb % gblocks) * CB;
    const bool live = c_first + tid / L < per;
    const int c = g * per + (live ? c_first + tid / L : per - 1);
    const int len = tile.len - tile.t0 < sg.seg ? tile.len - tile.t0 : sg.seg;
    const int64_t row0 = tile.start + tile.t0;
    const int slot = scalar(a.idx[tile.seq]);
    const bool slot_ok = slot >= 0 && slot < num_slots;
    const int64_t so = (int64_t)c * N + j0 * SPL;
    TS *const cache = static_cast<TS *>(a.cache) + (int64_t)(slot_ok ? slot : 0) * C * N + so;

    float A2[SPL], h[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        A2[i] = a.A[so + i] * kLog2e;
        h[i] = 0.0f;
    }
    if (first) {
        if (slot_ok && a.has && a.has[tile.seq]) load_state<TS, SPL>(cache, h);
    } else if (sg.cur == 2) {
        const int f = b - tile.t0 / sg.seg;
        load_state<float, SPL>(sg.fin + (int64_t)f * C * N + so, h);
        constexpr int AT = 32 / SPL;          // segments requested at once
        for (int k = f + 1; k < b; k += AT) {
            float add[AT][SPL], d[AT];
#pragma unroll
            for (int u = 0; u < AT; ++u) {
                const int64_t at = k + u < b ? k + u : b - 1;
                load_state<float, SPL>(sg.fin + at * C * N + so, add[u]);
                d[u] = sg.sum[at * C + c];
            }
#pragma unroll
            for (int u = 0; u < AT; ++u)
                if (k + u < b)
#pragma unroll
                    for (int i = 0; i < SPL; ++i)
                        h[i] = fmaf(__builtin_amdgcn_exp2f(d[u] * A2[i]), h[i], add[u][i]);
        }
    }
    const bool out = sg.cur != 1 || first;       // outputs wanted, not the final state alone
    const float Dc = a.D ? a.D[c] : 0.0f, bias = tf.bias ? tf.bias[c] : 0.0f;
    const bool gated = a.z != nullptr;
    const TX *const xb = static_cast<const TX *>(a.x) + row0 * xs;
    const TX *const db = static_cast<const TX *>(a.dt) + row0 * dts;
    const TX *const zb = static_cast<const TX *>(gated ? a.z : a.x) + row0 * zs;
    TX *const yb = static_cast<TX *>(a.y) + row0 * ys;
    const TX *const Bb = static_cast<const TX *>(a.B) + row0 * bs + (int64_t)g * N;
    const TX *const Cb = static_cast<const TX *>(a.C) + row0 * cs + (int64_t)g * N;
    // a lane's place in a stage's rows: its token of the first group, its channel
    const int xo = (j0 * (int)xs + c) * E, dto = (j0 * (int)dts + c) * E;
    const int zo = (j0 * (int)zs + c) * E;
    // (a lane without a channel writes past the end: dropped)
    const int yo = live ? (j0 * (int)ys + c) * E : 0x40000000;

    uint32_t xv[GROUPS], dv[GROUPS], zv[GROUPS], bv[BCV];
    auto request = [&](int t0) {
        const int n = len - t0 < ST ? len - t0 : ST;
        const rsrc_t rx = make_rsrc(xb + t0 * xs, (uint32_t)((n - 1) * (int)xs + C) * E);
        const rsrc_t rd = make_rsrc(db + t0 * dts, (uint32_t)((n - 1) * (int)dts + C) * E);
        const rsrc_t rz = make_rsrc(zb + t0 * zs, gated ? (uint32_t)((n - 1) * (int)zs + C) * E : 0);
        const rsrc_t rb = make_rsrc(Bb + t0 * bs, (uint32_t)((n - 1) * (int)bs + N) * E);
        const rsrc_t rc = make_rsrc(Cb + t0 * cs, (uint32_t)((n - 1) * (int)cs + N) * E);
#pragma unroll
        for (int m = 0; m < GROUPS; ++m) {
            xv[m] = buf_one<TX>(rx, xo, m * L * (int)xs * E);
            dv[m] = buf_one<TX>(rd, dto, m * L * (int)dts * E);
            zv[m] = buf_one<TX>(rz, zo, m * L * (int)zs * E);   // (no gate: an empty resource)
        }
        // value e of the stage: state e % N of token (e / N) % ST, of B then C
#pragma unroll
        for (int k = 0; k < BCV; ++k) {
            const int e = tid + 256 * k, n_ = e % N, t = (e / N) % ST;
            if (256 * k < ST * N) bv[k] = buf_one<TX>(rb, (t * (int)bs + n_) * E, 0);
            else bv[k] = buf_one<TX>(rc, (t * (int)cs + n_) * E, 0);
        }
    };
    float steps = 0.0f;       // of the lane's own tokens
    if (len > 0) request(0);
    int buf = 0;
    for (int t0 = 0; t0 < len; t0 += ST, buf ^= 1) {
#pragma unroll
        for (int k = 0; k < BCV; ++k) (&bc[buf][0][0][0])[tid + 256 * k] = widen_one<TX>(bv[k]);
        // (each choice once for all groups, so that their chains of dependent steps run
        // side by side)
        float x[GROUPS], dt[GROUPS], gate[GROUPS];
#pragma unroll
        for (int m = 0; m < GROUPS; ++m) {
            x[m] = widen_one<TX>(xv[m]);
            dt[m] = widen_one<TX>(dv[m]);
            gate[m] = 1.0f;
        }
        if (tf.on) {
#pragma unroll
            for (int m = 0; m < GROUPS; ++m) dt[m] = transformed(tf, dt[m], bias);
        }
        if (gated && out) {
#pragma unroll
            for (int m = 0; m < GROUPS; ++m) gate[m] = silu(widen_one<TX>(zv[m]));
        }
        if (t0 + ST > len) {          // tokens past the end take no step: the state stays
#pragma unroll
            for (int m = 0; m < GROUPS; ++m)
                if (t0 + m * L + j0 >= len) dt[m] = 0.0f;
            // (also where A is -infinity, whose product with 0 is NaN)
#pragma unroll
            for (int i = 0; i < SPL; ++i) A2[i] = __builtin_elementwise_maximum(A2[i], -3.4e38f);
        }
        __syncthreads();
        if (t0 + ST < len) request(t0 + ST);
        if (sg.cur == 1) {
#pragma unroll
            for (int m = 0; m < GROUPS; ++m) steps += dt[m];
        }
        if (out) {
            const int n = len - t0 < ST ? len - t0 : ST;
            const rsrc_t ry = make_rsrc(yb + t0 * ys, (uint32_t)((n - 1) * (int)ys + C) * E);
            // With few states a lane, B and C of a group are read from LDS while the group
            // before is worked on
            constexpr int AHEAD = L == 16 && SPL <= 2 ? 1 : 0;
            float Bn[2][L][SPL], Cn[2][L][SPL];
            auto fetch = [&](int m) {
#pragma unroll
                for (int j = 0; j < L; ++j)
#pragma unroll
                    for (int i = 0; i < SPL; ++i) {
                        Bn[m & 1][j][i] = bc[buf][0][m * L + j][j0 * SPL + i];
                        Cn[m & 1][j][i] = bc[buf][1][m * L + j][j0 * SPL + i];
                    }
            };
            if (AHEAD) fetch(0);
#pragma unroll
            for (int m = 0; m < GROUPS; ++m) {
                if (m + AHEAD < GROUPS) fetch(m + AHEAD);
                const float dtx = dt[m] * x[m];
                float part[L];
                unrolled<L>([&](auto J) {
                    constexpr int j = decltype(J)::value;
                    const float d = from_lane<L, j>(dt[m]), u = from_lane<L, j>(dtx);
                    float p = 0.0f;
#pragma unroll
                    for (int i = 0; i < SPL; ++i) {
                        h[i] = fmaf(__builtin_amdgcn_exp2f(d * A2[i]), h[i], u * Bn[m & 1][j][i]);
                        p = i == 0 ? h[i] * Cn[m & 1][j][i] : fmaf(h[i], Cn[m & 1][j][i], p);
                    }
                    part[j] = p;
                });
                const float y = (sum_own<L>(part, lane) + Dc * x[m]) * gate[m];
                buf_put<TX>(ry, y, yo, m * L * (int)ys * E);
            }
        } else {
#pragma unroll
            for (int m = 0; m < GROUPS; ++m) {
                const float dtx = dt[m] * x[m];
                unrolled<L>([&](auto J) {
                    constexpr int j = decltype(J)::value;
                    const float d = from_lane<L, j>(dt[m]), u = from_lane<L, j>(dtx);
                    const float *const Bt = &bc[buf][0][m * L + j][j0 * SPL];
#pragma unroll
                    for (int i = 0; i < SPL; ++i)
                        h[i] = fmaf(__builtin_amdgcn_exp2f(d * A2[i]), h[i], u * Bt[i]);
                });
            }
        }
    }
    if (!live) return;
    if (last) {
        if (slot_ok) store_state<TS, SPL>(cache, h);
    } else if (sg.cur == 1) {
        store_state<float, SPL>(sg.fin + (int64_t)b * C * N + so, h);
        // the channel's lanes hold the steps of their own tokens
        steps += dpp<0xb1>(steps);
        steps += dpp<0x4e>(steps);
        if constexpr (L == 16) {
            steps += dpp<0x141>(steps);
            steps += dpp<0x140>(steps);
        }
        if (j0 == 0) sg.sum[(int64_t)b * C + c] = steps;
    }
}

// Lanes a channel (4 or 16) and tokens a segment (0: whole sequences), from an
// estimate of each way's time in cycles of a SIMD (1024 of them). Measured with
// N = 16: a wave alone on its SIMD takes 280 cycles a token with 4 lanes a
// channel (16 channels a wave) and 117 with 16 (4 channels); waves that share
// a SIMD 175 and 90 each; both launches of the segmented form together 325.
//   2 prompts of 100 and 156 tokens, 64 channels: 16 lanes 24 us, 4 lanes 34 us
//   1 of 8192, 4096 channels: 830 us with 4 lanes, 438 us with 16, 262 us in
//   segments of 256 (271 us of 128, 280 us of 512)
//   8 of 1 to 1600, 5120 channels: 184 us with 4 lanes, the longest first (274 us
//   in the order given), 224 us with 16, 209 us in segments of 256
//   1 of 1024, 5120 channels: 62 us in segments of 128, 92 us with 16 lanes (1280
//   waves), 109 us with 4
//   2 of 717 and 1508, 72 channels: 20 us in segments with 16 lanes, 37 us with 4
// The longest sequence is not known here: 2.5 times the mean stands for it (prompt
// attention, whose rule was measured by itself, takes twice). With N = 32 and 64 a
// wave has 2 and 4 times the states, which `waves` counts and the cycles of a wave
// alone do not: 265 us for the 8 of 1 to 1600 with N = 32, 544 us for 2560 channels
// with N = 64, both in whole sequences; other ways were not measured there.
struct ScanPlan {
    int lanes, seg;
};
static ScanPlan scan_plan(const ScanDims &d)
{
    ScanPlan best{4, 0};
    if (d.S <= 0) return best;
    const double T = d.T, waves = (double)d.C * d.N / 16 / 16;
    const double longest = d.S == 1 ? T : fmin(T, 2.5 * T / d.S), share = T * waves / 1024;
    // one sequence's waves are all as long: the SIMDs that get one more set the time
    const double on4 = d.S == 1 ? ceil(waves / 1024) : 1, on16 = d.S == 1 ? ceil(waves * 4 / 1024) : 1;
    double least = fmax(longest * fmax(280, on4 * 175), share * 175);
    const double e16 = fmax(longest * fmax(117, on16 * 90), share * 4 * 90);
    if (e16 < least) {
        least = e16;
        best = ScanPlan{16, 0};
    }
    for (int seg = 128; seg <= 512; seg *= 2) {
        const double joins = 12000 + longest / seg * 250 + seg * 50.0;
        const double s4 = fmax(2.0 * seg * 280, share * 325) + joins;
        const double s16 = fmax(2.0 * seg * 117, share * 4 * 165) + joins;
        if (longest > seg && fmin(s4, s16) < least) {
            least = fmin(s4, s16);
            best = ScanPlan{s16 < s4 ? 16 : 4, seg};
        }
    }
    return best;
}
static int64_t scan_segments(const ScanDims &d, const ScanPlan &p)
{
    return p.seg ? (int64_t)d.T / p.seg + d.S : 0;
}

const char *scan_kernel_name(const ScanDims &d)
{
    static const char *const name[2][4] = {
        {"4 lanes", "4 lanes, segments of 128", "4 lanes, segments of 256", "4 lanes, segments of 512"},
        {"16 lanes", "16 lanes, segments of 128", "16 lanes, segments of 256",
         "16 lanes, segments of 512"}};
    const ScanPlan p = scan_plan(d);
    return name[p.lanes == 16][p.seg / 128 - p.seg / 512];
}

size_t scan_workspace(const ScanDims &d)
{
    return (size_t)scan_segments(d, scan_plan(d)) * d.C * (d.N + 1) * sizeof(float);
}

template <typename TX, typename TS, int N, int L>
static void launch_scan_l(const ScanDims &d, const ScanArgs &a, int seg, void *workspace,
                          hipStream_t st)
{
    const int per = d.C / d.G, chb = d.G * ((per + 256 / L - 1) / (256 / L));
    ScanSegs sg{0x7fffffff, 0, nullptr, nullptr};
    const int64_t n = seg ? (int64_t)d.T / seg + d.S : d.S;
    if (seg) {
        sg.seg = seg;
        sg.cur = 1;
        sg.fin = static_cast<float *>(workspace);
        sg.sum = sg.fin + n * d.C * d.N;
    }
    for (; sg.cur <= 2; ++sg.cur) {
        hipLaunchKernelGGL((scan_kernel<TX, TS, N, L>), dim3((unsigned)(n * chb)), dim3(256), 0, st,
                           d.T, d.S, d.C, d.G, d.num_slots, chb, a, d.xs, d.dts, d.zs, d.bs, d.cs,
                           d.ys, d.tf, sg);
        if (!seg) break;
    }
}

template <typename TX, typename TS, int N>
static void launch_scan_n(const ScanDims &d, const ScanArgs &a, void *workspace, hipStream_t st)
{
    const ScanPlan p = scan_plan(d);
    if (p.lanes == 16) launch_scan_l<TX, TS, N, 16>(d, a, p.seg, workspace, st);
    else launch_scan_l<TX, TS, N, 4>(d, a, p.seg, workspace, st);
}

// Verify-step form, bound by the states: a lane holds 16 bytes of them (4 float
// or 8 two-byte states), N of them a channel's L lanes, a block 256 / L channels
// of one group and one request. The state and the inputs of TM tokens are all
// requested before the first wait; B and C go through LDS, widened once for all
// of the block's channels. States after a token leave past the caches: a
// rollback reads one of them, later.
template <typename TS, int M> __device__ __forceinline__ void store_state_nt(TS *p, const float *v) {
    RawV<TS, M> r;
    r.set(v);
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    static_assert(sizeof(r.v) == 16, "16 bytes a lane");
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, r.v), reinterpret_cast<u32x4 *>(p));
}

template <typename TX, typename TS, int N, int TM>
__global__ __launch_bounds__(256) void scan_update_kernel(
    int Tr, int C, int G, int num_slots, int chb, ScanArgs a, int64_t xs, int64_t dts, int64_t zs,
    int64_t bs, int64_t cs, int64_t ys, DtTf tf, TS *__restrict__ inter)
{
    constexpr int SPL = 16 / (int)sizeof(TS), L = N / SPL, CB = 256 / L;
    constexpr int BCV = (TM * N * 2 + 255) / 256;
    __shared__ __align__(16) float bc[2][TM][N];
    const int tid = threadIdx.x, j0 = tid % L;
    const int r = (int)(blockIdx.x / (unsigned)chb), cb = (int)(blockIdx.x % (unsigned)chb);
    const int per = C / G, gblocks = chb / G, g = cb / gblocks;
    const int in_g = cb % gblocks * CB + tid / L;
    const bool live = in_g < per;
    const int c = g * per + (live ? in_g : per - 1);
    const int64_t row0 = (int64_t)r * Tr;
    const TX *const xp = static_cast<const TX *>(a.x) + row0 * xs + c;
    const TX *const dp = static_cast<const TX *>(a.dt) + row0 * dts + c;
    const TX *const zp = a.z ? static_cast<const TX *>(a.z) + row0 * zs + c : nullptr;
    TX *const yp = static_cast<TX *>(a.y) + row0 * ys + c;
    const TX *const Bp = static_cast<const TX *>(a.B) + row0 * bs + (int64_t)g * N;
    const TX *const Cp = static_cast<const TX *>(a.C) + row0 * cs + (int64_t)g * N;

    TX xv[TM], dv[TM], zv[TM], bv[BCV];
    auto request = [&](int t0) {
        // value e: state e % N of token e / N, of B and then of C
#pragma unroll
        for (int k = 0; k < BCV; ++k) {
            const int e = tid + 256 * k, t = t0 + e / N % TM;
            const int64_t tr = t < Tr ? t : Tr - 1;
            if (e < 2 * TM * N) bv[k] = e < TM * N ? Bp[tr * bs + e % N] : Cp[tr * cs + e % N];
        }
#pragma unroll
        for (int m = 0; m < TM; ++m) {
            const int64_t t = t0 + m < Tr ? t0 + m : Tr - 1;
            xv[m] = xp[t * xs];
            dv[m] = dp[t * dts];
            zv[m] = zp ? zp[t * zs] : xv[m];
        }
    };
    if (Tr > 0) request(0);
    const int slot = a.idx[r];
    const bool slot_ok = slot >= 0 && slot < num_slots;
    const int64_t so = (int64_t)c * N + j0 * SPL;
    TS *const cache = static_cast<TS *>(a.cache) + (int64_t)(slot_ok ? slot : 0) * C * N + so;
    RawV<TS, SPL> raw;
    raw.load(cache);
    float h[SPL], A2[SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) A2[i] = a.A[so + i] * kLog2e;
    const float Dc = a.D ? a.D[c] : 0.0f, bias = tf.bias ? tf.bias[c] : 0.0f;
    raw.get(h);
    if (!slot_ok) {
#pragma unroll
        for (int i = 0; i < SPL; ++i) h[i] = 0.0f;
    }
    for (int t0 = 0; t0 < Tr; t0 += TM) {
        if (t0 > 0) {
            __syncthreads();       // the last tokens' B and C are done with
            request(t0);
        }
#pragma unroll
        for (int k = 0; k < BCV; ++k)
            if (tid + 256 * k < 2 * TM * N) (&bc[0][0][0])[tid + 256 * k] = to_f32(bv[k]);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < TM; ++m) {
            const int t = t0 + m;
            if (t >= Tr) break;
            const float x = to_f32(xv[m]), dt = step_size(tf, to_f32(dv[m]), bias), u = dt * x;
            float p = 0.0f;
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                h[i] = fmaf(__builtin_amdgcn_exp2f(dt * A2[i]), h[i], u * bc[0][m][j0 * SPL + i]);
                p = fmaf(h[i], bc[1][m][j0 * SPL + i], p);
            }
            // the sum over the channel's L = 2, 4, 8 or 16 lanes
            p += dpp<0xb1>(p);
            if constexpr (L >= 4) p += dpp<0x4e>(p);
            if constexpr (L >= 8) p += dpp<0x141>(p);
            if constexpr (L >= 16) p += dpp<0x140>(p);
            const float y = (p + Dc * x) * (zp ? silu(to_f32(zv[m])) : 1.0f);
            if (live && j0 == 0) yp[(int64_t)t * ys] = from_f32<TX>(y);
            if (inter && live) store_state_nt<TS, SPL>(inter + (row0 + t) * C * N + so, h);
        }
    }
    if (!inter && slot_ok && live) store_state<TS, SPL>(cache, h);
}

template <typename TX, typename TS, int N>
static void launch_update_n(const ScanDims &d, const ScanArgs &a, void *inter, hipStream_t st)
{
    constexpr int CB = 256 * 16 / (int)sizeof(TS) / N;
    const int Tr = d.T / d.S, per = d.C / d.G, chb = d.G * ((per + CB - 1) / CB);
    const dim3 grid((unsigned)((int64_t)chb * d.S));
#define SSD_UPD(TM)                                                                              \
    hipLaunchKernelGGL((scan_update_kernel<TX, TS, N, TM>), grid, dim3(256), 0, st, Tr, d.C, d.G, \
                       d.num_slots, chb, a, d.xs, d.dts, d.zs, d.bs, d.cs, d.ys, d.tf,           \
                       static_cast<TS *>(inter))
    // tokens requested at once: the whole request when it has up to 4
    if (Tr <= 1) SSD_UPD(1);
    else if (Tr <= 2) SSD_UPD(2);
    else if (Tr <= 3) SSD_UPD(3);
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

void launch_scan(const ScanDims &d, const ScanArgs &a, void *workspace, void *stream)
{
    if (d.S <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    SSD_BY_TYPE(launch_scan_n, workspace, st);
}

void launch_scan_update(const ScanDims &d, const ScanArgs &a, void *inter, void *stream)
{
    if (d.S <= 0 || d.T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    SSD_BY_TYPE(launch_update_n, inter, st);
}

}  // namespace ssd
