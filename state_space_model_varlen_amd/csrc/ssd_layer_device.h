// Device helpers shared by the operators around the scan: runs of elements
// kept as loaded, the tile of packed sequences that a block works on.
#pragma once

#include <type_traits>

#include "ssd_device.h"

namespace ssd {

// VEC consecutive elements kept as loaded: one 16-byte (bf16) or two (float)
// vector loads for VEC = 8, one element for VEC = 1 (rows of any alignment).
template <typename T, int VEC> struct RawV {
    typedef T vec __attribute__((ext_vector_type(VEC)));
    vec v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const vec *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<vec *>(p) = v; }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(0.0f);
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = to_f32(v[i]);
    }
    __device__ __forceinline__ void set(const float *f) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(f[i]);
    }
};
template <typename T> struct RawV<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ void zero() { v = from_f32<T>(0.0f); }
    __device__ __forceinline__ void get(float *f) const { f[0] = to_f32(v); }
    __device__ __forceinline__ void set(const float *f) { v = from_f32<T>(f[0]); }
};

// Lane moves inside a row of 16 lanes, an operand of the instruction that uses
// the value.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                                 0xf, 0xf, true));
}
// Exchanges across the rows of a wave: every lane gets f(own, the lane 32, or
// 16, away) (the swap instructions leave one half's values in the first
// register and the other's in the second).
template <typename F> __device__ __forceinline__ float across32(float v, F f) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v),
                                                    __builtin_bit_cast(unsigned, v), false, false);
    return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <typename F> __device__ __forceinline__ float across16(float v, F f) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v),
                                                    __builtin_bit_cast(unsigned, v), false, false);
    return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float added(float a, float b) { return a + b; }

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// One value, the same in every lane, kept in a scalar register.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The tile of a packed batch that a block works on: sequence `seq` owns rows
// start .. start + len - 1 (clamped to [0, total)), the tile begins at its
// token t0. seq is -1 past the last tile.
struct SeqTile {
    int seq, start, len, t0;
};

// Tile b of the batch, when every sequence is cut into tiles of `tile` tokens
// from its own first token and an empty one has `of_empty` tiles: the batch
// has at most total / tile + S tiles. Every lane of the wave takes part (64
// sequences at a time: counted, summed over the wave, and the first whose
// running count passes b found by a ballot).
__device__ __forceinline__ SeqTile find_tile(const int32_t *__restrict__ cu, int S, int total,
                                             int tile, int of_empty, int b) {
    const int lane = threadIdx.x & (kWave - 1);
    int before = 0;
    for (int base = 0; base < S; base += kWave) {
        const int s = base + lane;
        int a = 0, len = 0, n = 0;
        if (s < S) {
            a = cu[s];
            const int e = cu[s + 1];
            a = a < 0 ? 0 : (a > total ? total : a);
            const int ec = e < 0 ? 0 : (e > total ? total : e);
            len = ec > a ? ec - a : 0;
            n = len > 0 ? (len - 1) / tile + 1 : of_empty;
        }
        int incl = n;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int o = __shfl_up(incl, off, kWave);
            if (lane >= off) incl += o;
        }
        const uint64_t past = __ballot(before + incl > b);
        if (past) {
            const int src = __ffsll((unsigned long long)past) - 1;
            SeqTile r;
            r.seq = base + src;
            r.start = scalar(__shfl(a, src, kWave));
            r.len = scalar(__shfl(len, src, kWave));
            r.t0 = (b - before - scalar(__shfl(incl - n, src, kWave))) * tile;
            return r;
        }
        before += scalar(__shfl(incl, kWave - 1, kWave));
    }
    return SeqTile{-1, 0, 0, 0};
}

// A lane's sequence of up to 64: its rows, its tiles and what orders it.
struct LaneSeqs {
    int start, len, tiles, weight;
};
__device__ __forceinline__ LaneSeqs lane_seqs(const int32_t *__restrict__ cu, int S, int total,
                                              int tile, int of_empty) {
    const int s = threadIdx.x & (kWave - 1);
    LaneSeqs r{0, 0, 0, -1};
    if (s < S) {
        const int a = cu[s], e = cu[s + 1];
        r.start = a < 0 ? 0 : (a > total ? total : a);
        const int ec = e < 0 ? 0 : (e > total ? total : e);
        r.len = ec > r.start ? ec - r.start : 0;
        r.tiles = r.len > 0 ? (r.len - 1) / tile + 1 : of_empty;
        r.weight = r.len;
    }
    return r;
}
// Tile b of them when the sequences are taken by falling weight (of equal ones
// the first): blocks start in order, so the longest work starts first and the
// short ends fill the gaps. Every lane of the wave takes part.
__device__ __forceinline__ SeqTile heaviest_first(const LaneSeqs &r, int S, int tile, int b) {
    const int s = threadIdx.x & (kWave - 1);
    int before = 0;
    for (int j = 0; j < S; ++j) {
        const int w = __builtin_amdgcn_readlane(r.weight, j), n = __builtin_amdgcn_readlane(r.tiles, j);
        before += w > r.weight || (w == r.weight && j < s) ? n : 0;
    }
    const uint64_t mine = __ballot(b >= before && b < before + r.tiles);
    if (!mine) return SeqTile{-1, 0, 0, 0};
    const int src = __ffsll((unsigned long long)mine) - 1;
    return SeqTile{src, __builtin_amdgcn_readlane(r.start, src), __builtin_amdgcn_readlane(r.len, src),
                   (b - __builtin_amdgcn_readlane(before, src)) * tile};
}

// The same for a batch whose sequences all have `len` tokens.
__device__ __forceinline__ SeqTile uniform_tile(int S, int len, int tile, int b) {
    const int per = len > 0 ? (len - 1) / tile + 1 : 1;
    const int s = b / per;
    return SeqTile{s < S ? s : -1, s * len, len, (b - s * per) * tile};
}

}  // namespace ssd
