// Paged key / value cache: rows quantised as they are written, read back into
// packed rows, and attended to by single tokens.
//
// An 8-bit row holds codes c (4 exponent, 3 mantissa bits) and one byte b, and
// stands for c 2^(b - 127). The scale is a power of two, so dividing by it is
// exact and a value is rounded once; widening a code and scaling it is exact in
// bf16 as well, so the matrix products see exactly what the cache holds.
#include "ssd_layer.h"
#include "ssd_layer_device.h"

namespace ssd {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float pow2_of_byte(uint32_t b) { return __uint_as_float(b << 23); }

// The larger of v over each aligned group of W = 8 or 16 lanes.
template <int W> __device__ __forceinline__ float group_max(float v) {
    if constexpr (W == 16) v = fmaxf(v, dpp<0x140>(v));   // row_mirror
    v = fmaxf(v, dpp<0x141>(v));                          // row_half_mirror
    v = fmaxf(v, dpp<0x4e>(v));                           // quad_perm [2,3,0,1]
    return fmaxf(v, dpp<0xb1>(v));                        // quad_perm [1,0,3,2]
}

// 8 codes of 8 scaled values (|v| <= 448 or NaN), rounded to nearest even.
__device__ __forceinline__ u32x2 codes8(const float *v) {
    u32x2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
        r[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true);
    }
    return r;
}

// One row (token, head) of k (blockIdx.y 0) or v (1) by D / 8 lanes, 8 elements
// a lane; the scale from the row's largest finite magnitude. Bound by the rows'
// bytes.
template <typename T, bool E4M3, int D>
__global__ __launch_bounds__(256) void kv_store_kernel(
    int rows, int Hkv, int log_page, int64_t positions, const T *__restrict__ k,
    const T *__restrict__ v, int64_t ks, int64_t vs, const int64_t *__restrict__ slots, KvCache c)
{
    constexpr int LPR = D / 8;
    const int row = (int)blockIdx.x * (256 / LPR) + (int)threadIdx.x / LPR;
    if (row >= rows) return;
    const int t = row / Hkv, h = row - t * Hkv, d0 = (int)threadIdx.x % LPR * 8;
    const int64_t pos = slots[t];
    if (pos < 0 || pos >= positions) return;
    const bool is_v = blockIdx.y != 0;
    float f[8];
    RawV<T, 8> raw;
    raw.load((is_v ? v + (int64_t)t * vs : k + (int64_t)t * ks) + (int64_t)h * D + d0);
    raw.get(f);
    const int64_t to = (((pos >> log_page) * Hkv + h) << log_page) + (pos & ((1 << log_page) - 1));
    if constexpr (E4M3) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = fabsf(f[i]);
            top = a < __builtin_inff() ? fmaxf(top, a) : top;
        }
        top = group_max<LPR>(top);
        // top = 1.m 2^e; 448 = 1.75 2^8: the least s with top <= 448 2^s is e - 8,
        // one more where 1.m > 1.75
        const uint32_t bits = __float_as_uint(top);
        int b = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        b = b < 1 ? 1 : b;
        const float inv = pow2_of_byte(254u - (uint32_t)b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = fabsf(f[i]) < __builtin_inff() ? f[i] * inv : __builtin_nanf("");
        uint8_t *const cache = static_cast<uint8_t *>(is_v ? c.v : c.k);
        *reinterpret_cast<u32x2 *>(cache + to * D + d0) = codes8(f);
        if (d0 == 0) (is_v ? c.vsc : c.ksc)[to] = (uint8_t)b;
    } else {
        RawV<bf16, 8> o;
        o.set(f);
        o.store(static_cast<bf16 *>(is_v ? c.v : c.k) + to * D + d0);
    }
}

// 16 consecutive cache elements as floats.
template <bool E4M3> __device__ __forceinline__ void cache16(const void *cache, int64_t at, float sc,
                                                             float *f) {
    if constexpr (E4M3) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(cache) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            f[4 * i] = lo[0] * sc;
            f[4 * i + 1] = lo[1] * sc;
            f[4 * i + 2] = hi[0] * sc;
            f[4 * i + 3] = hi[1] * sc;
        }
    } else
        load_run<bf16, 16>(static_cast<const bf16 *>(cache) + at, f);
}

// A tile of 16 tokens of one sequence, all heads, of k (blockIdx.y 0) or v: 16
// elements a thread and step, consecutive threads along the packed row.
constexpr int kLoadTile = 16;
template <typename T, bool E4M3, int D>
__global__ __launch_bounds__(256) void kv_load_kernel(
    int T_, int S, int max_pages, int pages, int log_page, int Hkv, const int32_t *__restrict__ cu,
    const int32_t *__restrict__ table, KvCache c, T *__restrict__ k, T *__restrict__ v, int64_t ks,
    int64_t vs)
{
    const SeqTile t = find_tile(cu, S, T_, kLoadTile, 0, (int)blockIdx.x);
    if (t.seq < 0) return;
    const bool is_v = blockIdx.y != 0;
    const int n = t.len - t.t0 < kLoadTile ? t.len - t.t0 : kLoadTile;
    const int chunks = Hkv * (D / 16);
    for (int e = (int)threadIdx.x; e < n * chunks; e += 256) {
        const int j = e / chunks, o = (e - j * chunks) * 16, h = o / D, pos = t.t0 + j;
        const int pi = pos >> log_page;
        const int pg = pi < max_pages ? table[(int64_t)t.seq * max_pages + pi] : -1;
        float f[16] = {};
        if (pg >= 0 && pg < pages) {
            const int64_t row = (((int64_t)pg * Hkv + h) << log_page) + (pos & ((1 << log_page) - 1));
            const float sc = E4M3 ? pow2_of_byte((is_v ? c.vsc : c.ksc)[row]) : 1.0f;
            cache16<E4M3>(is_v ? c.v : c.k, row * D + o % D, sc, f);
        }
        T *const to = is_v ? v + (int64_t)(t.start + pos) * vs : k + (int64_t)(t.start + pos) * ks;
        store_run<T, 16>(to + o, f);
    }
}

template <typename T, bool E4M3, int D>
static void store_t(const KvDims &d, int n, const void *k, const void *v, const int64_t *slots,
                    const KvCache &c, hipStream_t st)
{
    const int64_t rows = (int64_t)n * d.Hkv;
    const int per = 256 / (D / 8);
    hipLaunchKernelGGL((kv_store_kernel<T, E4M3, D>), dim3((unsigned)((rows + per - 1) / per), 2),
                       dim3(256), 0, st, (int)rows, d.Hkv, __builtin_ctz(d.page), (int64_t)d.pages * d.page,
                       static_cast<const T *>(k), static_cast<const T *>(v), d.ks, d.vs, slots, c);
}
template <typename T, bool E4M3, int D>
static void load_t(const KvDims &d, int n, int S, int max_pages, const int32_t *cu,
                   const int32_t *table, const KvCache &c, void *k, void *v, hipStream_t st)
{
    hipLaunchKernelGGL((kv_load_kernel<T, E4M3, D>), dim3((unsigned)(n / kLoadTile + S), 2),
                       dim3(256), 0, st, n, S, max_pages, d.pages, __builtin_ctz(d.page), d.Hkv, cu, table, c,
                       static_cast<T *>(k), static_cast<T *>(v), d.ks, d.vs);
}

#define SSD_KV_BY_TYPE(FN, ...)                                        \
    do {                                                               \
        if (d.in_bf16) {                                               \
            if (d.e4m3) {                                              \
                if (d.D == 128) FN<bf16, true, 128>(__VA_ARGS__);      \
                else FN<bf16, true, 64>(__VA_ARGS__);                  \
            } else {                                                   \
                if (d.D == 128) FN<bf16, false, 128>(__VA_ARGS__);     \
                else FN<bf16, false, 64>(__VA_ARGS__);                 \
            }                                                          \
        } else {                                                       \
            if (d.e4m3) {                                              \
                if (d.D == 128) FN<float, true, 128>(__VA_ARGS__);     \
                else FN<float, true, 64>(__VA_ARGS__);                 \
            } else {                                                   \
                if (d.D == 128) FN<float, false, 128>(__VA_ARGS__);    \
                else FN<float, false, 64>(__VA_ARGS__);                \
            }                                                          \
        }                                                              \
    } while (0)

void launch_kv_store(const KvDims &d, int T, const void *k, const void *v, const int64_t *slots,
                     const KvCache &c, void *stream)
{
    if (T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    SSD_KV_BY_TYPE(store_t, d, T, k, v, slots, c, st);
}

void launch_kv_load(const KvDims &d, int T, int S, int max_pages, const int32_t *cu,
                    const int32_t *table, const KvCache &c, void *k, void *v, void *stream)
{
    if (T <= 0 || S <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    SSD_KV_BY_TYPE(load_t, d, T, S, max_pages, cu, table, c, k, v, st);
}

// ---------------------------------------------------------------------------
// Attention of single tokens over the cache.
//
// A block of 4 waves takes one request, one key head, one span of its keys and
// 16 NRT of the T H / Hkv query rows that share the head; the waves take the
// span's tiles of 32 keys in turn, each with a running maximum and sum of its
// own, and are joined in LDS at the end. Bound by the cache's bytes: the next
// tile's keys and values are in flight while a tile is worked on.
//
// Scores are formed transposed (keys x rows), so that a lane holds scores of
// one query row and its probabilities are, as they stand, the operand of the
// second product (dims x rows); the values' tile goes through LDS for the
// transposed operand. A key row's 32-byte (or 64-byte) pieces are dealt to the
// lanes as they load fastest: the order of the head's dimensions in the sum
// does not matter as long as q's registers are filled in the same order.
template <bool E4M3, int D> struct Tile {
    static constexpr int EB = E4M3 ? 1 : 2;               // bytes an element
    static constexpr int KL = D * EB / 64;                // 16-byte loads of a lane for 16 keys
    static constexpr int VL = 32 * D * EB / 1024;         // 16-byte loads of a lane for 32 value rows
    static constexpr int LPV = D * EB / 16;               // lanes a value row
    u32x4 k[2][KL], v[VL];
    uint32_t ksc[2], vsc[VL];
};

// first head dimension of the 8 that lane group g multiplies in step s
template <bool E4M3> __device__ __forceinline__ int dim_of(int s, int g) {
    return E4M3 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
}

// 8 codes (two words) as bf16 times the power of two `sc` (exact).
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi, float sc) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? lo : hi;
        const bf16x2 p = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, true)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, false);
        r[2 * i] = p[0];
        r[2 * i + 1] = p[1];
    }
    return r;
}

// Non-finite elements of 16 bytes set to zero; whether there were any.
template <bool E4M3> __device__ __forceinline__ bool take_out(u32x4 &w) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t bad;
        if constexpr (E4M3) {      // codes 0x7f and 0xff
            bad = (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
            bad *= 0xffu;
        } else                     // exponents of all ones
            bad = ((w[i] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
                  ((w[i] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
        w[i] &= ~bad;
        any |= bad != 0;
    }
    return any;
}

struct DecodePart {
    float *o, *ml;     // [rows of all requests][splits][D], [..][2] (maximum, sum)
    int splits, span;  // span: keys a split
};

template <bool E4M3, int D, int NRT>
__global__ __launch_bounds__(256, 2) void decode_attn_kernel(
    int T, int H, int Hkv, int pages, int log_page, int max_pages, float scale2,
    const bf16 *__restrict__ q, int64_t qs, KvCache c, const int32_t *__restrict__ table,
    const int32_t *__restrict__ lens, bf16 *__restrict__ out, int64_t os, float *__restrict__ lse,
    DecodePart part)
{
    typedef Tile<E4M3, D> TL;
    constexpr int STEPS = D / 32, DT = D / 16, VP = D + 16;   // VP: row pitch of a value tile
    constexpr int OP = D + 4;
    static_assert(16 * OP * 4 <= 32 * VP * 2, "a row tile's result fits the value tile");
    __shared__ __align__(16) bf16 vt[4][32 * VP];
    __shared__ float ml[4][2][NRT * 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), n16 = lane & 15, g = lane >> 4;
    const int split = (int)blockIdx.x % part.splits, r0 = (int)blockIdx.x / part.splits * NRT * 16;
    const int kvh = blockIdx.y, r = blockIdx.z;
    const int group = H / Hkv, rows = T * group;
    int L = scalar(lens[r]);
    const int most = max_pages << log_page;
    L = L < 0 ? 0 : (L > most ? most : L);
    const int k0 = split * part.span;
    const int k1 = L - k0 < part.span ? L : k0 + part.span;
    if (k0 >= k1 && split > 0) return;         // (the join reads no such split)
    const int32_t *const tab = table + (int64_t)r * max_pages;
    const int shared = L - T + 1;              // keys that all of the request's tokens see

    // q of row n16 of every row tile, and how many keys the row sees
    bf16x8 qf[NRT][STEPS];
    int sees[NRT];
#pragma unroll
    for (int m = 0; m < NRT; ++m) {
        const int row = r0 + m * 16 + n16, rc = row < rows ? row : rows - 1;
        const int t = rc / group, h = kvh * group + rc % group;
        const bf16 *const qp = q + ((int64_t)r * T + t) * qs + (int64_t)h * D;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            qf[m][s] = *reinterpret_cast<const bf16x8 *>(qp + dim_of<E4M3>(s, g));
        sees[m] = row < rows ? shared + t : 0;
    }

    const char *const kc = static_cast<const char *>(c.k), *const vc = static_cast<const char *>(c.v);
    // the first row in the cache of 16 keys from `key` on (a multiple of 16), or -1
    auto base_of = [&](int key) -> int64_t {
        if (key >= k1) return -1;
        const int pg = scalar(tab[key >> log_page]);
        return pg >= 0 && pg < pages
                   ? (((int64_t)pg * Hkv + kvh) << log_page) + (key & ((1 << log_page) - 1)) : -1;
    };
    auto request = [&](TL &t, int key, int64_t b0, int64_t b1) {
        // (scalar bases, one offset a lane; a load of the values stays in one half)
        const int64_t base[2] = {b0 < 0 ? 0 : b0, b1 < 0 ? 0 : b1};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const char *const p = kc + base[i] * (D * TL::EB);
#pragma unroll
            for (int l = 0; l < TL::KL; ++l)
                t.k[i][l] = *reinterpret_cast<const u32x4 *>(p + (n16 * (D * TL::EB) + g * 16 + 64 * l));
            if (E4M3) t.ksc[i] = (c.ksc + base[i])[n16];
        }
        constexpr int RV = 64 / TL::LPV;          // value rows a load covers: 4, 8 or 16
#pragma unroll
        for (int l = 0; l < TL::VL; ++l) {
            const int64_t half = base[l * RV / 16];
            const int vr = l * RV % 16 + lane / TL::LPV;
            t.v[l] = *reinterpret_cast<const u32x4 *>(
                vc + half * (D * TL::EB) + (vr * (D * TL::EB) + lane % TL::LPV * 16));
            if (E4M3) t.vsc[l] = (c.vsc + half)[vr];
        }
    };

    f32x4 o[NRT][DT];
    float mx[NRT], sum[NRT];
    bool odd = false;                          // values were taken out
#pragma unroll
    for (int m = 0; m < NRT; ++m) {
        mx[m] = -__builtin_inff();
        sum[m] = 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[m][i] = zero4();
    }
    bf16 *const vw = vt[wave];
    TL cur, next;
    int key = k0 + wave * 32;
    int64_t b0 = base_of(key), b1 = base_of(key + 16);
    if (key < k1) request(cur, key, b0, b1);
    for (; key < k1; key += 128) {
        const int64_t n0 = base_of(key + 128), n1 = base_of(key + 144);
        if (key + 128 < k1) request(next, key + 128, n0, n1);
        // scores of 32 keys x 16 rows: keys 4 g + v and 16 + 4 g + v of row n16
        f32x4 s[NRT][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int m = 0; m < NRT; ++m) s[m][i] = zero4();
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
                bf16x8 kf;
                if constexpr (E4M3) {
                    const u32x4 w = cur.k[i][st >> 1];
                    kf = (st & 1) ? widen8(w[2], w[3], pow2_of_byte(cur.ksc[i]))
                                  : widen8(w[0], w[1], pow2_of_byte(cur.ksc[i]));
                } else
                    kf = __builtin_bit_cast(bf16x8, cur.k[i][st]);
#pragma unroll
                for (int m = 0; m < NRT; ++m) s[m][i] = Mma<bf16>::run(kf, qf[m][st], s[m][i]);
            }
        }
        // the values' tile, rows that do not count as zeros (whatever lies there). Where
        // some of the request's tokens do not see all of its keys, a masked weight is
        // zero but zero times an infinity is not: non-finite values stay out of the
        // product and are added below to the rows that see them.
        const bool partial = key + 32 > shared;
#pragma unroll
        for (int l = 0; l < TL::VL; ++l) {
            const int vr = l * (64 / TL::LPV) + lane / TL::LPV;
            const bool in = key + vr < k1 && (l * (64 / TL::LPV) < 16 ? b0 : b1) >= 0;
            const uint32_t keep = in ? 0xffffffffu : 0u;
            u32x4 w = cur.v[l] & keep;
            if (partial) odd |= take_out<E4M3>(w);
            bf16 *const to = vw + vr * VP + lane % TL::LPV * (16 / TL::EB);
            if constexpr (E4M3) {
                const float sc = in ? pow2_of_byte(cur.vsc[l]) : 1.0f;
                *reinterpret_cast<bf16x8 *>(to) = widen8(w[0], w[1], sc);
                *reinterpret_cast<bf16x8 *>(to + 8) = widen8(w[2], w[3], sc);
            } else
                *reinterpret_cast<u32x4 *>(to) = w;
        }
        wave_lds_sync();
        // The matrix products take bf16. A weight goes in as its rounded value and what the
        // rounding left: two products in place of one, on matrix units that are a twentieth
        // busy (128 requests of 1 K to 4 K keys in 8 bits 151 -> 155 us, one of 32769 in bf16
        // 33.5 -> 34.1), against an eighth bit rounded (a result's error 1.25 times its own
        // rounding's).
        bf16x8 pf[NRT], pr[NRT];
#pragma unroll
        for (int m = 0; m < NRT; ++m) {
            float sc[8], top = -__builtin_inff();
            const int end = sees[m] < k1 ? sees[m] : k1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = key + (e >> 2) * 16 + 4 * g + (e & 3);
                const bool in = at < end && ((e >> 2) ? b1 : b0) >= 0;
                sc[e] = in ? s[m][e >> 2][e & 3] * scale2 : -__builtin_inff();
                top = fmaxf(top, sc[e]);
            }
            top = across32(across16(top, larger), larger);
            const float was = mx[m];
            mx[m] = fmaxf(was, top);
            // (a row that has seen nothing yet: subtract 0, its terms are exp2(-inf))
            const float ref = mx[m] == -__builtin_inff() ? 0.0f : mx[m];
            const float f = __builtin_amdgcn_exp2f(was - ref);
            sum[m] *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = __builtin_amdgcn_exp2f(sc[e] - ref);
                sum[m] += p;
                pf[m][e] = static_cast<bf16>(p);
                pr[m][e] = static_cast<bf16>(p - to_f32(pf[m][e]));
            }
            if (__any(top > was))
#pragma unroll
                for (int i = 0; i < DT; ++i) o[m][i] *= f;
        }
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            const bf16x8 vf = mfma_frag_tr_split(vw, VP, 0, 16 * i, lane);
#pragma unroll
            for (int m = 0; m < NRT; ++m)
                o[m][i] = Mma<bf16>::run(vf, pr[m], Mma<bf16>::run(vf, pf[m], o[m][i]));
        }
        wave_lds_sync();
        cur = next;
        b0 = n0;
        b1 = n1;
    }

    // Values that are not finite go back to the rows that see them, from the wave that had
    // their tile: those taken out, from the tile that `shared` is in on; and all of them where
    // a sum came out as NaN, because an infinity times a weight's remainder has either sign, or
    // is NaN (8 bits hold no infinities).
    bool lost = false;
#pragma unroll
    for (int m = 0; m < NRT; ++m) {
        sum[m] = across32(across16(sum[m], added), added);
        if constexpr (!E4M3) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) nan |= o[m][i][e] != o[m][i][e];
            lost |= nan && sum[m] == sum[m];
        }
    }
    lost = __any(lost);
    if (lost || __any(odd)) {
        const int from = shared > k0 && !lost ? (shared - k0) / 32 * 32 : 0, mine = wave * 32;
        const int first = k0 + mine + (from > mine ? (from - mine + 127) / 128 * 128 : 0);
        for (int i = 0; i < DT; ++i) {
            f32x4 back[NRT];
#pragma unroll
            for (int m = 0; m < NRT; ++m) back[m] = zero4();
            for (int half = first; half < k1; half += half & 16 ? 112 : 16) {
                const int64_t b = base_of(half);
                if (b < 0) continue;
                const char *const row = vc + (b * D + 16 * i + 4 * g) * TL::EB;
#pragma unroll 4
                for (int u = 0; u < 16; ++u) {
                    float v[4];
                    if constexpr (E4M3) {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(row + u * D);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = (w >> (8 * e) & 0x7f) == 0x7f ? __builtin_nanf("") : 0.0f;
                    } else
                        load4<bf16>(reinterpret_cast<const bf16 *>(row) + u * D, v);
#pragma unroll
                    for (int m = 0; m < NRT; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (half + u < sees[m] && !(fabsf(v[e]) < __builtin_inff())) back[m][e] += v[e];
                }
            }
#pragma unroll
            for (int k = 0; k < DT; ++k)
#pragma unroll
                for (int m = 0; m < NRT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float was = o[m][k][e], v = back[m][e];
                        if (k == i) o[m][k][e] = was != was && v != 0.0f ? v : was + v;
                    }
        }
    }

    // join the waves: common maximum, then the four results summed through LDS
#pragma unroll
    for (int m = 0; m < NRT; ++m)
        if (g == 0) {
            ml[wave][0][m * 16 + n16] = mx[m];
            ml[wave][1][m * 16 + n16] = sum[m];
        }
    __syncthreads();
    for (int m = 0; m < NRT; ++m) {
        const int at = m * 16 + n16;
        const float top = fmaxf(fmaxf(ml[0][0][at], ml[1][0][at]), fmaxf(ml[2][0][at], ml[3][0][at]));
        const float ref = top == -__builtin_inff() ? 0.0f : top;
        float *const ow = reinterpret_cast<float *>(vt[wave]);
        float f = 0.0f;
#pragma unroll
        for (int k = 0; k < NRT; ++k)
            if (k == m) f = __builtin_amdgcn_exp2f(mx[k] - ref);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            f32x4 v = zero4();
#pragma unroll
            for (int k = 0; k < NRT; ++k)
                if (k == m) v = o[k][i] * f;
            *reinterpret_cast<f32x4 *>(ow + n16 * OP + 16 * i + 4 * g) = v;
        }
        __syncthreads();
        constexpr int PER = D / 16;                  // elements a thread: 16 threads a row
        const int row = r0 + m * 16 + tid / 16, d0 = tid % 16 * PER, rl = m * 16 + tid / 16;
        float acc[PER] = {};
        float all = 0.0f, top2 = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < 4; ++w) top2 = fmaxf(top2, ml[w][0][rl]);
        const float ref2 = top2 == -__builtin_inff() ? 0.0f : top2;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            all += ml[w][1][rl] * __builtin_amdgcn_exp2f(ml[w][0][rl] - ref2);
            const float *const from = reinterpret_cast<const float *>(vt[w]) + tid / 16 * OP + d0;
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] += from[e];
        }
        if (row < rows) {
            const int t = row / group, h = kvh * group + row % group;
            const int64_t qr = (int64_t)r * T + t;
            if (part.splits == 1) {
                const float inv = all > 0.0f || all != all ? 1.0f / all : 0.0f;
                RawV<bf16, PER> res;
#pragma unroll
                for (int e = 0; e < PER; ++e) acc[e] *= inv;
                res.set(acc);
                res.store(out + qr * os + (int64_t)h * D + d0);
                if (lse && d0 == 0) lse[qr * H + h] = (ref2 + __builtin_amdgcn_logf(all)) * kLn2;
            } else {
                const int64_t at2 = (qr * H + h) * part.splits + split;
#pragma unroll
                for (int e = 0; e < PER; ++e) part.o[at2 * D + d0 + e] = acc[e];
                if (d0 == 0) {
                    part.ml[at2 * 2] = top2;
                    part.ml[at2 * 2 + 1] = all;
                }
            }
        }
        __syncthreads();
    }
}

// Joins the splits of a (token, head): one block, its threads in groups of D / 4
// lanes that take the splits in turn, 4 elements a lane and the loads of 4
// splits at once, and are summed through LDS. (One wave that walked 86 splits
// took 28 us, this takes 5.)
template <int D>
__global__ __launch_bounds__(256) void decode_join_kernel(int T, int H, int most,
                                                          const int32_t *__restrict__ lens,
                                                          DecodePart part, bf16 *__restrict__ out,
                                                          int64_t os, float *__restrict__ lse)
{
    constexpr int LANES = D / 4, GRP = 256 / LANES;
    __shared__ __align__(16) float acc_l[GRP][D];
    __shared__ float red[2][4];
    const int tid = threadIdx.x, grp = tid / LANES, d0 = tid % LANES * 4;
    const int64_t row = blockIdx.x, qr = row / H;
    int L = lens[qr / T];
    L = L < 0 ? 0 : (L > most ? most : L);
    int ns = (L + part.span - 1) / part.span;
    ns = ns < 1 ? 1 : ns;
    const float *const ml = part.ml + row * part.splits * 2;
    const float *const o = part.o + row * part.splits * D + d0;
    float top = -__builtin_inff();
    for (int s = tid; s < ns; s += 256) top = fmaxf(top, ml[2 * s]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if ((tid & 63) == 0) red[0][tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    float all = 0.0f;
    for (int s = tid; s < ns; s += 256) all += __builtin_amdgcn_exp2f(ml[2 * s] - ref) * ml[2 * s + 1];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) all += __shfl_xor(all, off, 64);
    if ((tid & 63) == 0) red[1][tid >> 6] = all;
    f32x4 acc = zero4();
    for (int s0 = grp; s0 < ns; s0 += 4 * GRP) {
        f32x4 v[4];
        float f[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int s = s0 + u * GRP < ns ? s0 + u * GRP : ns - 1;
            v[u] = *reinterpret_cast<const f32x4 *>(o + (int64_t)s * D);
            f[u] = ml[2 * s];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (s0 + u * GRP < ns) acc += v[u] * __builtin_amdgcn_exp2f(f[u] - ref);
    }
    *reinterpret_cast<f32x4 *>(&acc_l[grp][d0]) = acc;
    __syncthreads();
    all = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    const float inv = all > 0.0f || all != all ? 1.0f / all : 0.0f;
    const int h = (int)(row - qr * H);
    if (tid < D) {
        float v = 0.0f;
#pragma unroll
        for (int g = 0; g < GRP; ++g) v += acc_l[g][tid];
        out[qr * os + (int64_t)h * D + tid] = static_cast<bf16>(v * inv);
    }
    if (lse && tid == 0) lse[row] = (ref + __builtin_amdgcn_logf(all)) * kLn2;
}

// Row tiles a block holds: all of a head group's rows where they fit in two.
static int row_tiles(const DecodeAttnDims &d)
{
    return d.T * (d.H / d.kv.Hkv) <= 16 ? 1 : 2;
}
// How the contexts are split over blocks. Splits cost their partial results
// (twice, written and read) and the join's launch, so there are no more than
// bring 1024 blocks, of at least 512 keys; but with few requests a block's
// chain of key tiles is what takes time, and up to 512 blocks of at least 128
// keys are made. (128 requests of 1 K to 4 K keys, 8 key heads, 8 bits: 164 us
// unsplit, 190 us in two, 198 us in four. One request of 32769 keys in bf16: 31
// us in 65 splits of 512, 33 us in 128 of 256.) The contexts are not known here,
// their table's width is: a table far wider than they are makes few, long splits
// (8 requests of 1500 keys: 13 us with a table for 1536, 53 us with one for 32768).
static DecodePart plan(const DecodeAttnDims &d)
{
    DecodePart p{nullptr, nullptr, 1, 128};
    const int64_t most = (int64_t)d.max_pages * d.kv.page;
    const int rows = d.T * (d.H / d.kv.Hkv), in_block = 16 * row_tiles(d);
    const int64_t blocks = (int64_t)d.R * d.kv.Hkv * ((rows + in_block - 1) / in_block);
    if (blocks <= 0 || most <= 128) {
        p.span = most > 128 ? (int)((most + 127) / 128 * 128) : 128;
        return p;
    }
    auto most_splits = [&](int64_t target, int64_t keys) {
        const int64_t n = (most + keys - 1) / keys;
        return target / blocks < n ? target / blocks : n;
    };
    int64_t splits = most_splits(1024, 512);
    if (splits * blocks < 512) splits = most_splits(512, 128);
    if (splits < 1) splits = 1;
    const int64_t span = ((most + splits - 1) / splits + 127) / 128 * 128;
    p.span = (int)span;
    p.splits = (int)((most + span - 1) / span);
    return p;
}

size_t decode_attn_workspace(const DecodeAttnDims &d)
{
    const DecodePart p = plan(d);
    if (p.splits == 1) return 0;
    return (size_t)d.R * d.T * d.H * p.splits * (d.kv.D + 2) * sizeof(float);
}

template <bool E4M3, int D, int NRT>
static void decode_t(const DecodeAttnDims &d, const void *q, const KvCache &c, const int32_t *table,
                     const int32_t *lens, void *out, float *lse, const DecodePart &p, hipStream_t st)
{
    const int rows = d.T * (d.H / d.kv.Hkv);
    const dim3 grid((unsigned)(p.splits * ((rows + 16 * NRT - 1) / (16 * NRT))), d.kv.Hkv, d.R);
    hipLaunchKernelGGL((decode_attn_kernel<E4M3, D, NRT>), grid, dim3(256), 0, st, d.T, d.H,
                       d.kv.Hkv, d.kv.pages, __builtin_ctz(d.kv.page), d.max_pages, d.scale * kLog2e,
                       static_cast<const bf16 *>(q), d.qs, c, table, lens, static_cast<bf16 *>(out),
                       d.os, lse, p);
    if (p.splits > 1) {
        const int64_t n = (int64_t)d.R * d.T * d.H;
        hipLaunchKernelGGL((decode_join_kernel<D>), dim3((unsigned)n), dim3(256), 0, st, d.T, d.H,
                           d.max_pages * d.kv.page, lens, p, static_cast<bf16 *>(out), d.os, lse);
    }
}

void launch_decode_attn(const DecodeAttnDims &d, const void *q, const KvCache &c,
                        const int32_t *table, const int32_t *lens, void *out, float *lse,
                        void *workspace, void *stream)
{
    if (d.R <= 0 || d.T <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    DecodePart p = plan(d);
    const int nrt = row_tiles(d);
    if (p.splits > 1) {
        p.o = static_cast<float *>(workspace);
        p.ml = p.o + (int64_t)d.R * d.T * d.H * p.splits * d.kv.D;
    }
#define SSD_DEC(E, D)                                                                         \
    do {                                                                                      \
        if (nrt == 1) decode_t<E, D, 1>(d, q, c, table, lens, out, lse, p, st);               \
        else decode_t<E, D, 2>(d, q, c, table, lens, out, lse, p, st);                        \
    } while (0)
    if (d.kv.e4m3) { if (d.kv.D == 128) SSD_DEC(true, 128); else SSD_DEC(true, 64); }
    else           { if (d.kv.D == 128) SSD_DEC(false, 128); else SSD_DEC(false, 64); }
#undef SSD_DEC
}

}  // namespace ssd
