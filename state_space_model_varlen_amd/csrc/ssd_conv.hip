// Short causal convolution over packed sequences, with the last inputs of
// every sequence kept in a cache by slot (the layer piece in front of the
// selective scan), its single-token form and the commit after a verify step.
//
//     y[t,c] = act(bias[c] + sum over k < W of weight[c,k] x[t - (W-1) + k, c])
//
// Bandwidth-bound: 2 W + 4 operations for every element read and written.
#include "ssd_layer.h"
#include "ssd_layer_device.h"

namespace ssd {

struct ConvOut {
    void *p[3];
    int64_t s[3];
    int end0, end1;   // channels [0, end0) go to p[0], [end0, end1) to p[1], the rest to p[2]
};

// One wave per (tile of TT tokens of one sequence, 64 VEC channels), VEC
// channels a lane: a tile's TT rows and the W - 1 before them are requested at
// once, then a window of W rows slides over them in registers. Tiles start at
// the sequence's first token, so the tokens that look into the cache slot all
// belong to the sequence's first tile; that block alone reads the slot and
// then writes it, each lane its own channels, and no other block can see a
// slot half way.
template <typename TX, typename TS, int W, int VEC, int TT>
__global__ __launch_bounds__(64) void conv_kernel(
    int T, int S, int C, int num_slots, int chb, const TX *__restrict__ x, int64_t xs,
    const float *__restrict__ weight, const float *__restrict__ bias,
    const int32_t *__restrict__ cu, TS *cache, const int32_t *__restrict__ idx,
    const uint8_t *__restrict__ has, int all_init, ConvOut out, int silu, int write_state)
{
    const int b = (int)(blockIdx.x / (unsigned)chb);
    const int c0 = ((int)(blockIdx.x % (unsigned)chb) * kWave + (int)threadIdx.x) * VEC;
    const SeqTile t = cu ? find_tile(cu, S, T, TT, 1, b) : uniform_tile(S, T / S, TT, b);
    if (t.seq < 0) return;
    // A lane's 8 channels x 4 taps are 128 bytes; read as they lie, every load of
    // theirs would touch 64 lines, more than all the rows together. They come in
    // whole lines and change lanes through LDS (the channel's place turned by the
    // lane, so that neither side meets bank conflicts).
    const int lane = threadIdx.x;
    __shared__ f32x4 wl[VEC == 8 && W == 4 ? 512 : 1];
    if constexpr (VEC == 8 && W == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int q = i * kWave + lane, ch = c0 - lane * 8 + q;
            if (ch < C) wl[(q & ~7) | ((q ^ (q >> 3)) & 7)] = *reinterpret_cast<const f32x4 *>(weight + (int64_t)ch * 4);
        }
    }
    if (c0 >= C) return;
    const TX *const xr = x + (int64_t)t.start * xs + c0;
    const bool first = t.t0 == 0;
    const int n = t.len - t.t0 < TT ? t.len - t.t0 : TT;

    // requested in this order: the tile's rows, those before it (a later tile: places
    // t0 - (W-1) ..; the first tile: the slot's rows, once its number is there)
    RawV<TX, VEC> row[TT], hist[W - 1];
    RawV<TS, VEC> old[W - 1];
    if (n > 0) {
#pragma unroll
        for (int j = 0; j < TT; ++j) row[j].load(xr + (int64_t)(t.t0 + (j < n ? j : n - 1)) * xs);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        hist[k].zero();
        old[k].zero();
    }
    const int slot = idx[t.seq];
    const bool slot_ok = slot >= 0 && slot < num_slots;
    TS *const cs = cache + (int64_t)(slot_ok ? slot : 0) * (W - 1) * C + c0;
    if (!first) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) hist[k].load(xr + (int64_t)(t.t0 - (W - 1) + k) * xs);
    } else if (slot_ok && (all_init || (has && has[t.seq]))) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) old[k].load(cs + (int64_t)k * C);
    }
    if (n > 0) {
        float w[VEC][W], bs[VEC];
        if constexpr (VEC == 8 && W == 4) wave_lds_sync();
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (VEC == 8 && W == 4) {
                const f32x4 v = wl[lane * 8 + (i ^ (lane & 7))];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i][k] = v[k];
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) w[i][k] = weight[(int64_t)(c0 + i) * W + k];
            }
            bs[i] = bias ? bias[c0 + i] : 0.0f;
        }
        const int seg = c0 < out.end0 ? 0 : (c0 < out.end1 ? 1 : 2);
        const int64_t ys = out.s[seg];
        TX *yr = static_cast<TX *>(out.p[seg]) + (int64_t)(t.start + t.t0) * ys + c0 -
                 (seg == 0 ? 0 : (seg == 1 ? out.end0 : out.end1));
        float win[W][VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            if (first) old[k].get(win[k]);
            else hist[k].get(win[k]);
        }
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            if (j >= n) continue;   // (a break would keep the loop rolled and the rows in memory)
            row[j].get(win[W - 1]);
            float acc[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                acc[i] = bs[i];
#pragma unroll
                for (int k = 0; k < W; ++k) acc[i] += w[i][k] * win[k][i];
                if (silu) acc[i] *= __builtin_amdgcn_rcpf(1.0f + __expf(-acc[i]));
            }
            RawV<TX, VEC> o;
            o.set(acc);
            o.store(yr + (int64_t)j * ys);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) win[k][i] = win[k + 1][i];
        }
    }
    if (!first || !write_state || !slot_ok) return;
    // row k of the new slot is row len + k of (the old rows, the sequence)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        RawV<TS, VEC> o;
        if (t.len + k >= W - 1) {
            RawV<TX, VEC> v;
            v.load(xr + (int64_t)(t.len + k - (W - 1)) * xs);
            float f[VEC];
            v.get(f);
            o.set(f);
        } else {
            o = old[k];
#pragma unroll
            for (int m = 0; m < W - 1; ++m)
                if (m == t.len + k) o = old[m];
        }
        o.store(cs + (int64_t)k * C);
    }
}

// Request r's slot takes 1 + accepted[r] tokens in: row k becomes row
// 1 + accepted + k of (the old rows, the request's tokens).
template <typename TX, typename TS, int W>
__global__ __launch_bounds__(256) void conv_commit_kernel(int Tr, int C, int num_slots,
                                                          const TX *__restrict__ x, int64_t xs,
                                                          TS *cache, const int32_t *__restrict__ idx,
                                                          const int32_t *__restrict__ accepted)
{
    const int chb = (C + 255) / 256;
    const int r = (int)(blockIdx.x / (unsigned)chb);
    const int c = (int)(blockIdx.x % (unsigned)chb) * 256 + (int)threadIdx.x;
    const int slot = idx[r], a = accepted[r];
    if (c >= C || slot < 0 || slot >= num_slots || a < 0 || a >= Tr) return;
    TS *const cs = cache + (int64_t)slot * (W - 1) * C + c;
    TS v[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int at = a + 1 + k;
        v[k] = at < W - 1 ? cs[(int64_t)at * C]
                          : from_f32<TS>(to_f32(x[((int64_t)r * Tr + at - (W - 1)) * xs + c]));
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) cs[(int64_t)k * C] = v[k];
}

template <typename TX, typename TS, int W, int VEC, int TT>
static void launch_conv_t(const ConvDims &d, const void *x, const float *w, const float *bias,
                          const int32_t *cu, void *cache, const int32_t *idx, const uint8_t *has,
                          bool all_init, const ConvOut &o, bool write_state, hipStream_t st)
{
    const int chb = (d.C + kWave * VEC - 1) / (kWave * VEC);
    int64_t tiles = (int64_t)d.T / TT + d.S;
    if (!cu) {
        const int len = d.T / d.S;
        tiles = (int64_t)d.S * (len > 0 ? (len - 1) / TT + 1 : 1);
    }
    hipLaunchKernelGGL((conv_kernel<TX, TS, W, VEC, TT>), dim3((unsigned)(tiles * chb)), dim3(64),
                       0, st, d.T, d.S, d.C, d.num_slots, chb, static_cast<const TX *>(x), d.xs, w,
                       bias, cu, static_cast<TS *>(cache), idx, has, all_init ? 1 : 0, o,
                       d.silu ? 1 : 0, write_state ? 1 : 0);
}

template <typename TX, typename TS, int W>
static void launch_conv_w(const ConvDims &d, const void *x, const float *w, const float *bias,
                          const int32_t *cu, void *cache, const int32_t *idx, const uint8_t *has,
                          bool all_init, const ConvOut &o, bool write_state, hipStream_t st)
{
    // 8 channels a lane where every run of 8 lies in one output and on 16 bytes
    auto on16 = [](const void *p, int64_t stride, size_t e) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (uint64_t)stride * e % 16 == 0;
    };
    bool wide = d.C % 8 == 0 && o.end0 % 8 == 0 && o.end1 % 8 == 0 && on16(x, d.xs, sizeof(TX)) &&
                on16(cache, d.C, sizeof(TS)) && on16(w, 0, 4);
    for (int i = 0; i < 3; ++i)
        if (d.yc[i] > 0) wide = wide && on16(o.p[i], o.s[i], sizeof(TX));
    // a verify step's few tokens need no 16-row tile (and its registers)
    const bool few = !cu && d.T / d.S <= 4;
#define SSD_CONV(VEC, TT) \
    launch_conv_t<TX, TS, W, VEC, TT>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st)
    if (wide) { if (few) SSD_CONV(8, 4); else SSD_CONV(8, 16); }
    else      { if (few) SSD_CONV(1, 4); else SSD_CONV(1, 16); }
#undef SSD_CONV
}

template <typename TX, typename TS>
static void launch_conv_x(const ConvDims &d, const void *x, const float *w, const float *bias,
                          const int32_t *cu, void *cache, const int32_t *idx, const uint8_t *has,
                          bool all_init, const ConvOut &o, bool write_state, hipStream_t st)
{
    if (d.W == 4) launch_conv_w<TX, TS, 4>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st);
    else if (d.W == 3) launch_conv_w<TX, TS, 3>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st);
    else launch_conv_w<TX, TS, 2>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st);
}

void launch_conv(const ConvDims &d, const void *x, const float *w, const float *bias,
                 const int32_t *cu, void *cache, const int32_t *idx, const uint8_t *has,
                 bool all_init, void *const y[3], bool write_state, void *stream)
{
    if (d.S <= 0) return;
    ConvOut o;
    for (int i = 0; i < 3; ++i) {
        o.p[i] = y[i];
        o.s[i] = d.ys[i];
    }
    o.end0 = d.yc[0];
    o.end1 = d.yc[0] + d.yc[1];
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (d.in_bf16) {
        if (d.state_bf16) launch_conv_x<bf16, bf16>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st);
        else launch_conv_x<bf16, float>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st);
    } else {
        if (d.state_bf16) launch_conv_x<float, bf16>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st);
        else launch_conv_x<float, float>(d, x, w, bias, cu, cache, idx, has, all_init, o, write_state, st);
    }
}

void launch_conv_commit(const ConvDims &d, const void *x, void *cache, const int32_t *idx,
                        const int32_t *accepted, void *stream)
{
    if (d.S <= 0 || d.T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)((int64_t)d.S * ((d.C + 255) / 256)));
#define SSD_COMMIT(TX, TS, W)                                                                     \
    hipLaunchKernelGGL((conv_commit_kernel<TX, TS, W>), grid, dim3(256), 0, st, d.T / d.S, d.C,   \
                       d.num_slots, static_cast<const TX *>(x), d.xs, static_cast<TS *>(cache),   \
                       idx, accepted)
#define SSD_COMMIT_W(TX, TS)                    \
    do {                                        \
        if (d.W == 4) SSD_COMMIT(TX, TS, 4);    \
        else if (d.W == 3) SSD_COMMIT(TX, TS, 3); \
        else SSD_COMMIT(TX, TS, 2);             \
    } while (0)
    if (d.in_bf16) {
        if (d.state_bf16) SSD_COMMIT_W(bf16, bf16);
        else SSD_COMMIT_W(bf16, float);
    } else {
        if (d.state_bf16) SSD_COMMIT_W(float, bf16);
        else SSD_COMMIT_W(float, float);
    }
#undef SSD_COMMIT_W
#undef SSD_COMMIT
}

}  // namespace ssd
