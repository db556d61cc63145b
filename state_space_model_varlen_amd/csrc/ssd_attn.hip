// Softmax attention over packed prompts: causal or full, grouped heads, more
// keys than queries where a sequence continues a cached prefix.
//
// One pass over a sequence's keys per block of queries, with a running maximum
// and sum in float32. For query row i and the keys seen so far,
//     m = max_j s_ij,  l = sum_j exp2(s_ij - m),  o = sum_j exp2(s_ij - m) v_j
// (scores in units of log 2), o and l being rescaled when m grows; the result
// is o / l. 4 D operations for every visible pair, against a few bytes: bound
// by the matrix units on any but the shortest prompts.
#include "ssd_layer.h"
#include "ssd_layer_device.h"

namespace ssd {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct AttnArgs {
    const void *q, *k, *v;
    const int32_t *cuq, *cuk;
    void *out;
    float *lse;
    int64_t qs, ks, vs, os;
    int Tq, Tk, S, H, Hkv, causal;
    float scale2;   // scale log2(e)
};

// The block's queries: tile of BM queries of one sequence, the first of its
// heads (HPB of one key head's group) and the head past them, the key head, the
// sequence's key rows, and `off`: query i sees keys up to i + off.
struct AttnBlock {
    int seq, q0, lq, qrow, head, head_end, kvh, krow, lk, off;
};
// Heads run fastest over the blocks, the key head innermost, so that the 8
// XCDs, which take blocks in turn, each see few key heads. The sequences with
// the most keys come first (up to 64 of them), and within a sequence the last
// tile, which sees the most.
__device__ __forceinline__ AttnBlock attn_block(const AttnArgs &a, int BM, int HPB = 1) {
    AttnBlock r;
    const int group = a.H / a.Hkv, hb = a.Hkv * ((group + HPB - 1) / HPB);
    const int hh = (int)(blockIdx.x % (unsigned)hb), b = (int)(blockIdx.x / (unsigned)hb);
    SeqTile t;
    if (a.S > 1 && a.S <= kWave) {
        LaneSeqs l = lane_seqs(a.cuq, a.S, a.Tq, BM, 0);
        const int s = threadIdx.x & (kWave - 1);
        if (s < a.S) l.weight = a.cuk[s + 1] - a.cuk[s];
        t = heaviest_first(l, a.S, BM, b);
    } else
        t = find_tile(a.cuq, a.S, a.Tq, BM, 0, b);
    r.seq = t.seq;
    if (t.seq < 0) return r;
    r.kvh = hh % a.Hkv;
    r.head = r.kvh * group + hh / a.Hkv * HPB;
    r.head_end = (r.kvh + 1) * group;
    r.lq = t.len;
    r.qrow = t.start;
    r.q0 = (t.len - 1) / BM * BM - t.t0;
    int k0 = scalar(a.cuk[t.seq]), k1 = scalar(a.cuk[t.seq + 1]);
    k0 = k0 < 0 ? 0 : (k0 > a.Tk ? a.Tk : k0);
    k1 = k1 < 0 ? 0 : (k1 > a.Tk ? a.Tk : k1);
    r.krow = k0;
    r.lk = k1 > k0 ? k1 - k0 : 0;
    r.off = a.causal ? r.lk - r.lq : 0x3fffffff;
    return r;
}
// Keys that query i (clamped: i + off may pass 2^31 where there is no mask) sees.
__device__ __forceinline__ int keys_seen(const AttnBlock &b, int i) {
    const int n = b.off >= b.lk ? b.lk : i + b.off + 1;
    return n < 0 ? 0 : (n > b.lk ? b.lk : n);
}

// A masked probability is zero, and zero times an infinity or a NaN among the
// values is not. In a tile that hides some of its keys from some of the block's
// queries, non-finite values are therefore taken out of the product and added
// afterwards to the queries that do see them (any positive weight gives the
// same infinity or NaN).
__device__ __forceinline__ bool bad16(uint32_t w) { return (w & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool take_out(u32x4 &w, bf16) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool lo = bad16(w[i]), hi = bad16(w[i] >> 16);
        w[i] &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
        any |= lo | hi;
    }
    return any;
}
// Whether an element of a query's sum of values came out as NaN for no fault of its
// weights. (A weight goes into the products as two parts, its rounded value and the
// rest; an infinity times the rest has either sign, or is NaN.)
template <int D> __device__ __forceinline__ bool lost_sums(const f32x16 (&o)[D / 32], float sum) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) nan |= o[i][e] != o[i][e];
    return __any(nan && sum == sum);
}
// Adds the non-finite values among keys from .. kend - 1 (whole tiles of 32 that the
// wave answers for) to the sums of the queries that see them; a sum that is NaN is
// replaced by theirs. A tile is looked through as it lies first: most have none.
template <int D, typename F>
__device__ __forceinline__ void give_back(const bf16 *V, int64_t vs, int from, int kend, int seen,
                                          f32x16 (&o)[D / 32], F mine) {
    constexpr int LPV = D / 8, RV = 64 / LPV;                      // lanes a row, rows a load
    const int lane = threadIdx.x & 63, hf = lane >> 5;
    f32x16 back[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) back[i][e] = 0.0f;
    for (int j = from; j < kend; j += 32) {
        if (!mine(j)) continue;
        bool any = false;
#pragma unroll
        for (int r = 0; r < 32; r += RV) {
            const int k = j + r + lane / LPV;
            u32x4 w = *reinterpret_cast<const u32x4 *>(V + (int64_t)(k < kend ? k : kend - 1) * vs +
                                                       lane % LPV * 8);
            any |= take_out(w, bf16());
        }
        if (!__any(any)) continue;
        const int end = j + 32 < kend ? j + 32 : kend;
        for (int k = j; k < end; ++k)
            if (k < seen)
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        float v[4];
                        load4<bf16>(V + (int64_t)k * vs + 32 * i + 2 * e + 4 * hf, v);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (!(fabsf(v[u]) < __builtin_inff())) back[i][e + u] += v[u];
                    }
        bool more = false;                                         // (all NaN: no need to go on)
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) more |= o[i][e] == o[i][e] || back[i][e] == back[i][e];
        if (!__any(more)) break;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float was = o[i][e], v = back[i][e];
            o[i][e] = was != was && v != 0.0f ? v : was + v;
        }
}

// bf16 heads of D. A block of 4 waves takes 32 queries of one head a wave: of HPB
// heads that share a key head, BM = 128 / HPB queries of each (fewer queries
// mean less work beyond the diagonal, and short sequences fill the block),
// against tiles of 64 keys in LDS, worked on in two steps of 32 keys.
//
// Scores are formed transposed, S^T = K Q^T (keys x queries), so that a lane
// holds 16 of every 32 scores of one query (its partner 32 lanes away the
// rest): the row maximum and the rescaling are per lane, and the weights, in
// bf16, are as they stand the operand of O^T = V^T P^T. The values'
// transposed operand comes through the LDS transpose read. Row pitches keep
// both kinds of reads free of bank conflicts (K: 4 dwords past a multiple of
// 64 dwords; V: 16 past).
//
// The products take bf16, so a weight goes into the second one as its rounded value
// and, rounded in turn, what that left (off by 2^-16 of it: the result's error is its
// own rounding's; with the rounded value alone, BF16W, a caller's choice, it is 1.25
// times that, and 16384 tokens of 32 heads of 128 take 2181 us instead of 2938).
//
// The matrix and the vector work of a step are about equally long (D = 128: 768
// cycles of MFMA, 512 with BF16W; 520 and 360 of exponentials, maxima, sums and
// parts), and a wave that takes one after the other leaves each unit idle half the
// time. So a step forms the scores of the step after it, adds the values of the step
// before it, and does the softmax of its own: three pieces that do not depend on one
// another and are issued interleaved. Keys are therefore needed a step early and
// values a step late; with two buffers of each, one barrier a tile, between its
// steps, lets K of the next tile and V of this one be written before it and used
// after it. Heads of 128 take 250 registers (with BF16W 256, and 16 bytes of scratch),
// two waves a SIMD; heads of 64 161, three.
template <int D> struct AttnSmem {
    static constexpr int BN = 64, KP = D + 8, VP = D + 32;
    __align__(16) bf16 k[2][BN * KP];
    __align__(16) bf16 v[2][BN * VP];
    int hidden;                      // a partly masked tile has non-finite values
};

template <int D, int HPB, bool BF16W>
__global__ __launch_bounds__(256, 2) void attn_kernel(AttnArgs a)
{
    typedef AttnSmem<D> SM;
    constexpr int BM = 128 / HPB, BN = SM::BN, KP = SM::KP, VP = SM::VP;
    constexpr int VEC = BN * D / 8 / 256;       // 16-byte vectors a thread stages of K, and of V
    constexpr int RPT = D / 8;                  // threads a row
    __shared__ SM sm;
    const AttnBlock b = attn_block(a, BM, HPB);
    if (b.seq < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), qi = lane & 31, hf = lane >> 5;
    const int q = b.q0 + wave / HPB * 32 + qi;                 // the lane's query
    const int qc = q < b.lq ? q : b.lq - 1;
    const int head = b.head + wave % HPB, hc = head < b.head_end ? head : b.head;
    const bf16 *const Q = static_cast<const bf16 *>(a.q) + (int64_t)(b.qrow + qc) * a.qs +
                          (int64_t)hc * D + hf * 8;
    bf16x8 qf[D / 16];
#pragma unroll
    for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const bf16x8 *>(Q + 16 * s);
    const int seen = q < b.lq ? keys_seen(b, q) : 0;
    const int qlast = b.q0 + BM - 1 < b.lq - 1 ? b.q0 + BM - 1 : b.lq - 1;
    const int kend = keys_seen(b, qlast);                      // keys the block needs
    const int kfull = keys_seen(b, b.q0);                      // keys that all its queries see

    const bf16 *const K = static_cast<const bf16 *>(a.k) + (int64_t)b.krow * a.ks + (int64_t)b.kvh * D;
    const bf16 *const V = static_cast<const bf16 *>(a.v) + (int64_t)b.krow * a.vs + (int64_t)b.kvh * D;
    u32x4 kr[VEC], vr[VEC];
    // a tile's rows from key j0 on; rows past the sequence's end come back as zeros
    auto request = [&](u32x4 (&r)[VEC], const bf16 *base, int stride, int j0) __attribute__((always_inline)) {
        const int rows = b.lk - j0 < BN ? b.lk - j0 : BN;
        const rsrc_t rs = make_rsrc(base + (int64_t)j0 * stride,
                                    rows > 0 ? (uint32_t)((rows - 1) * stride + D) * 2 : 0u);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            r[i] = __builtin_bit_cast(u32x4, buf_ld16(rs, (uint32_t)((tid + 256 * i) / RPT * stride +
                                                                     8 * (tid % RPT)) * 2));
    };
    auto stage_k = [&](int t) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            *reinterpret_cast<u32x4 *>(&sm.k[t & 1][(tid + 256 * i) / RPT * KP + 8 * (tid % RPT)]) = kr[i];
    };
    auto stage_v = [&](int t) __attribute__((always_inline)) {
        if ((t + 1) * BN > kfull) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < VEC; ++i) any |= take_out(vr[i], bf16());
            if (any) sm.hidden = 1;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            *reinterpret_cast<u32x4 *>(&sm.v[t & 1][(tid + 256 * i) / RPT * VP + 8 * (tid % RPT)]) = vr[i];
    };

    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float m = -__builtin_inff(), sum = 0.0f;

    // scores of 32 keys: element e is key 8 (e / 4) + 4 hf + e % 4 of them
    auto scores = [&](int buf, int sub) __attribute__((always_inline)) {
        f32x16 s;
        const bf16 *const kl = &sm.k[buf][(sub * 32 + qi) * KP + hf * 8];
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
        for (int st = 0; st < D / 16; ++st)
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                *reinterpret_cast<const bf16x8 *>(kl + 16 * st), qf[st], s, 0, 0, 0);
        return s;
    };
    // adds 32 keys' values: the operand of dims 32 i .. and keys 16 w .., of which the
    // lanes of a half hold the keys 4 hf + v and 8 + 4 hf + v that their weights belong to
    const int jl = lane & 15;
    const int vo = (4 * hf + (jl >> 2)) * VP + ((lane >> 4) & 1) * 16 + 4 * (jl & 3);
    auto add_values = [&](int buf, int sub, const bf16x8 (&p)[2], const bf16x8 (&r)[2]) __attribute__((always_inline)) {
        const bf16 *const vl = &sm.v[buf][sub * 32 * VP + vo];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const v4i16 lo = lds_read_tr16(vl + 16 * w * VP + 32 * i);
                const v4i16 hi = lds_read_tr16(vl + (16 * w + 8) * VP + 32 * i);
                typedef short v8i16 __attribute__((ext_vector_type(8)));
                const v8i16 both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, both), p[w],
                                                               o[i], 0, 0, 0);
                if constexpr (!BF16W)
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, both), r[w],
                                                                   o[i], 0, 0, 0);
            }
    };
    // softmax weights of the 32 keys from key j on; returns what the result so far has
    // to be scaled by, and whether any lane's maximum rose
    auto weights = [&](f32x16 &s, int j, bool masked, bf16x8 (&p)[2], bf16x8 (&r)[2], bool &rose) __attribute__((always_inline)) {
        if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (j + 8 * (e >> 2) + 4 * hf + (e & 3) >= seen) s[e] = -__builtin_inff();
        }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
        top = across32(top, larger) * a.scale2;
        const float was = m;
        m = fmaxf(m, top);
        // (a row that has seen nothing yet: subtract 0, its terms are exp2(-inf))
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        const float f = __builtin_amdgcn_exp2f(was - ref);
        sum *= f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float w = __builtin_amdgcn_exp2f(s[e] * a.scale2 - ref);
            sum += w;
            p[e >> 3][e & 7] = static_cast<bf16>(w);
            if constexpr (!BF16W) r[e >> 3][e & 7] = static_cast<bf16>(w - to_f32(p[e >> 3][e & 7]));
        }
        rose = top > was;
        return f;
    };
    // (the empty statements keep the weights in front of the branch, where the matrix
    // products they run beside are, and the products with f behind it)
    auto rescale = [&](float f, bool rose, bf16x8 (&p)[2], bf16x8 (&r)[2]) __attribute__((always_inline)) {
        asm volatile("" : "+v"(p[0]), "+v"(p[1]), "+v"(sum));
        if constexpr (!BF16W) asm volatile("" : "+v"(r[0]), "+v"(r[1]));
        if (__any(rose)) {
            asm volatile("" : "+v"(f));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] *= f;
        }
    };
    const int tiles = (kend + BN - 1) / BN;
    f32x16 s0, s1;
    bf16x8 p0[2], p1[2], r0[2], r1[2];
    if (tid == 0) sm.hidden = 0;
    // (the values "before the first tile": zeros with zero weights)
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) p1[w][e] = r1[w][e] = static_cast<bf16>(0.0f);
    for (int i = tid; i < BN * VP / 8; i += 256) reinterpret_cast<u32x4 *>(sm.v[1])[i] = u32x4{0, 0, 0, 0};
    if (tiles > 0) {
        request(kr, K, (int)a.ks, 0);
        stage_k(0);
        request(kr, K, (int)a.ks, BN);
        request(vr, V, (int)a.vs, 0);
    }
    __syncthreads();
    if (tiles > 0) s0 = scores(0, 0);
    auto tile = [&](int t, auto with_mask) __attribute__((always_inline)) {
        constexpr bool masked = decltype(with_mask)::value;
        const int j = t * BN, buf = t & 1;
        bool rose;
        s1 = scores(buf, 1);
        add_values(buf ^ 1, 1, p1, r1);
        float f = weights(s0, j, masked, p0, r0, rose);
        rescale(f, rose, p0, r0);
        stage_k(t + 1);
        stage_v(t);
        __syncthreads();
        request(kr, K, (int)a.ks, j + 2 * BN);
        request(vr, V, (int)a.vs, j + BN);
        s0 = scores(buf ^ 1, 0);
        add_values(buf, 0, p0, r0);
        f = weights(s1, j + 32, masked, p1, r1, rose);
        rescale(f, rose, p1, r1);
    };
    const int open = kfull / BN < tiles ? kfull / BN : tiles;     // tiles without a mask
    for (int t = 0; t < open; ++t) tile(t, std::false_type());
    for (int t = open; t < tiles; ++t) tile(t, std::true_type());
    if (tiles > 0) {
        const int t = tiles - 1;
        add_values(t & 1, 1, p1, r1);
    }
    sum = across32(sum, added);
    const bool lost = !BF16W && lost_sums<D>(o, sum);
    if (lost || sm.hidden)
        give_back<D>(V, a.vs, lost ? 0 : open * BN, kend, seen, o, [](int) { return true; });

    if (q < b.lq && head < b.head_end) {
        // (a NaN sum is passed on; a row without keys gets zeros)
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        bf16 *const out = static_cast<bf16 *>(a.out) + (int64_t)(b.qrow + q) * a.os +
                          (int64_t)head * D + 4 * hf;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                float r[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) r[v] = o[i][e + v] * inv;
                store4<bf16>(out + 32 * i + 2 * e, r);
            }
        if (a.lse && hf == 0) {
            const float ref = m == -__builtin_inff() ? 0.0f : m;
            a.lse[(int64_t)(b.qrow + q) * a.H + head] = (ref + __builtin_amdgcn_logf(sum)) * kLn2;
        }
    }
}

// Few queries, or few heads: a block of NW waves takes one tile of queries (32 in
// bf16, 16 QT in float), and its waves the key tiles in turn, each with a running
// maximum and sum of its own; they are joined in LDS at the end. The chain of
// tiles that a wave walks is NW times shorter, and no matrix row is spent on
// queries that are not there; but every tile of keys is read for fewer queries.
// A wave's tiles are its own, staged in LDS of its own without barriers: rows read
// straight into the keys' operand would touch 32 lines with every load (2.1 us a
// round of 8 tiles of heads of 128, against 1.4; 1.6 since weights have two parts).
//
// join_waves: the waves' results (o scaled to the common maximum, in rows of
// D + 4 floats a query) and statistics, one thread per PER elements.
template <int D, int NQ, int NW> struct JoinSmem {
    __align__(16) float o[NW][NQ * (D + 4)];
};
template <typename T, int D, int NQ, int NW>
__device__ __forceinline__ void join_waves(const AttnArgs &a, const AttnBlock &b,
                                           const float (&o)[NW][NQ * (D + 4)],
                                           const float (&ml)[NW][2][NQ]) {
    constexpr int PER = NQ * D / (NW * 64), TPR = D / PER;
    static_assert(PER % 4 == 0, "whole vectors");
    const int row = (int)threadIdx.x / TPR, d0 = (int)threadIdx.x % TPR * PER, q = b.q0 + row;
    if (q >= b.lq) return;
    float top = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w][0][row]);
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    float sum = 0.0f, acc[PER] = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        sum += ml[w][1][row] * __builtin_amdgcn_exp2f(ml[w][0][row] - ref);
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] += o[w][row * (D + 4) + d0 + e];
    }
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    T *const out = static_cast<T *>(a.out) + (int64_t)(b.qrow + q) * a.os + (int64_t)b.head * D + d0;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= inv;
#pragma unroll
    for (int e = 0; e < PER; e += 4) store4<T>(out + e, acc + e);
    if (a.lse && d0 == 0)
        a.lse[(int64_t)(b.qrow + q) * a.H + b.head] = (ref + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <int D>
__global__ __launch_bounds__(512, 1) void attn_split_kernel(AttnArgs a)
{
    constexpr int NW = 8, BN = 32, KP = D + 8, VP = D + 32;
    constexpr int VL = BN * D / 512, LPV = D / 8, RV = 64 / LPV;   // value loads, lanes a row, rows a load
    typedef JoinSmem<D, 32, NW> JS;
    constexpr int TILES = NW * BN * (KP + VP) * 2;
    __shared__ __align__(16) char raw[sizeof(JS) > TILES ? sizeof(JS) : TILES];
    __shared__ float ml[NW][2][32];
    const AttnBlock b = attn_block(a, 32);
    if (b.seq < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), qi = lane & 31, hf = lane >> 5;
    const int q = b.q0 + qi, qc = q < b.lq ? q : b.lq - 1;
    const bf16 *const Q = static_cast<const bf16 *>(a.q) + (int64_t)(b.qrow + qc) * a.qs +
                          (int64_t)b.head * D + hf * 8;
    bf16x8 qf[D / 16];
#pragma unroll
    for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const bf16x8 *>(Q + 16 * s);
    const int seen = q < b.lq ? keys_seen(b, q) : 0;
    const int qlast = b.q0 + 31 < b.lq - 1 ? b.q0 + 31 : b.lq - 1;
    const int kend = keys_seen(b, qlast), kfull = b.q0 + 31 < b.lq ? keys_seen(b, b.q0) : 0;
    const int kopen = keys_seen(b, b.q0);          // keys that all queries there are see
    const bf16 *const K = static_cast<const bf16 *>(a.k) + (int64_t)b.krow * a.ks + (int64_t)b.kvh * D;
    const bf16 *const V = static_cast<const bf16 *>(a.v) + (int64_t)b.krow * a.vs + (int64_t)b.kvh * D;
    bf16 *const kw = reinterpret_cast<bf16 *>(raw) + wave * BN * (KP + VP), *const vw = kw + BN * KP;

    u32x4 kr[VL], vr[VL];
    auto request = [&](u32x4 (&r)[VL], const bf16 *base, int stride, int j0) __attribute__((always_inline)) {
        const int rows = b.lk - j0 < BN ? b.lk - j0 : BN;
        const rsrc_t rs = make_rsrc(base + (int64_t)j0 * stride,
                                    rows > 0 ? (uint32_t)((rows - 1) * stride + D) * 2 : 0u);
#pragma unroll
        for (int l = 0; l < VL; ++l)
            r[l] = __builtin_bit_cast(u32x4, buf_ld16(rs, (uint32_t)((l * RV + lane / LPV) * stride +
                                                                    lane % LPV * 8) * 2));
    };
    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float m = -__builtin_inff(), sum = 0.0f;
    bool odd = false;
    const int jl = lane & 15;
    const int vo = (4 * hf + (jl >> 2)) * VP + ((lane >> 4) & 1) * 16 + 4 * (jl & 3);
    if (wave * BN < kend) {
        request(kr, K, (int)a.ks, wave * BN);
        request(vr, V, (int)a.vs, wave * BN);
    }
    for (int j0 = wave * BN; j0 < kend; j0 += NW * BN) {
#pragma unroll
        for (int l = 0; l < VL; ++l)
            *reinterpret_cast<u32x4 *>(kw + (l * RV + lane / LPV) * KP + lane % LPV * 8) = kr[l];
        request(kr, K, (int)a.ks, j0 + NW * BN);
        wave_lds_sync();
        f32x16 s;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
        for (int st = 0; st < D / 16; ++st)
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                *reinterpret_cast<const bf16x8 *>(kw + qi * KP + 16 * st + 8 * hf), qf[st], s, 0, 0, 0);
        if (j0 + BN > kopen) {
#pragma unroll
            for (int l = 0; l < VL; ++l) odd |= take_out(vr[l], bf16());
        }
#pragma unroll
        for (int l = 0; l < VL; ++l)
            *reinterpret_cast<u32x4 *>(vw + (l * RV + lane / LPV) * VP + lane % LPV * 8) = vr[l];
        request(vr, V, (int)a.vs, j0 + NW * BN);
        if (j0 + BN > kfull) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (j0 + 8 * (e >> 2) + 4 * hf + (e & 3) >= seen) s[e] = -__builtin_inff();
        }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
        top = across32(top, larger) * a.scale2;
        const float was = m;
        m = fmaxf(m, top);
        const float ref = m == -__builtin_inff() ? 0.0f : m, f = __builtin_amdgcn_exp2f(was - ref);
        sum *= f;
        bf16x8 p[2], r[2];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float w = __builtin_amdgcn_exp2f(s[e] * a.scale2 - ref);
            sum += w;
            p[e >> 3][e & 7] = static_cast<bf16>(w);
            r[e >> 3][e & 7] = static_cast<bf16>(w - to_f32(p[e >> 3][e & 7]));
        }
        if (__any(top > was)) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] *= f;
        }
        wave_lds_sync();
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const v4i16 lo = lds_read_tr16(vw + vo + 16 * w * VP + 32 * i);
                const v4i16 hi = lds_read_tr16(vw + vo + (16 * w + 8) * VP + 32 * i);
                typedef short v8i16 __attribute__((ext_vector_type(8)));
                const v8i16 both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, both), p[w],
                                                               o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, both), r[w],
                                                               o[i], 0, 0, 0);
            }
        wave_lds_sync();
    }
    sum = across32(sum, added);
    const bool lost = lost_sums<D>(o, sum);
    if (lost || __any(odd))        // (from the wave that had the tile)
        give_back<D>(V, a.vs, lost ? 0 : kopen / BN * BN, kend, seen, o,
                     [&](int j) { return j / BN % NW == wave; });
    if (hf == 0) {
        ml[wave][0][qi] = m;
        ml[wave][1][qi] = sum;
    }
    __syncthreads();               // (also: the value tiles are done with)
    JS &js = *reinterpret_cast<JS *>(raw);
    float top = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w][0][qi]);
    const float f = __builtin_amdgcn_exp2f(m - (top == -__builtin_inff() ? 0.0f : top));
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            f32x4 v;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = o[i][e + k] * f;
            *reinterpret_cast<f32x4 *>(&js.o[wave][qi * (D + 4) + 32 * i + 2 * e + 4 * hf]) = v;
        }
    __syncthreads();
    join_waves<bf16, D, 32, NW>(a, b, js.o, ml);
}

// float heads of D, on the float32 matrix instructions (16 x 16 tiles, 4 dimensions
// or keys a step; their rate, an eighth of bf16's, is the bound): 16 QT queries a
// block, 4 waves that take tiles of 16 keys in turn. A lane holds the scores of
// query lane % 16 for keys 4 (lane / 16) + v; keys and values go straight from
// memory to the operands, 16 bytes a lane: the four dimensions that a lane gets
// of a value belong to four products, so row r of product 4 i + c is dimension
// 64 i + 4 r + c (with one element a load 199 us instead of 161: 19 prompts of 20,
// one of them on 8000 keys, 16 heads of 128).
template <int D, int QT>
__global__ __launch_bounds__(256, 1) void attn_f32_kernel(AttnArgs a)
{
    constexpr int NW = 4, BN = 16, NQ = 16 * QT;
    typedef JoinSmem<D, NQ, NW> JS;
    __shared__ JS js;
    __shared__ float ml[NW][2][NQ];
    const AttnBlock b = attn_block(a, NQ);
    if (b.seq < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6), qi = lane & 15, g = lane >> 4;
    f32x4 qf[QT][D / 16];
    int seen[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int q = b.q0 + 16 * t + qi, qc = q < b.lq ? q : b.lq - 1;
        const float *const Q = static_cast<const float *>(a.q) + (int64_t)(b.qrow + qc) * a.qs +
                               (int64_t)b.head * D + 4 * g;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[t][s] = *reinterpret_cast<const f32x4 *>(Q + 16 * s);
        seen[t] = q < b.lq ? keys_seen(b, q) : 0;
    }
    const int qlast = b.q0 + NQ - 1 < b.lq - 1 ? b.q0 + NQ - 1 : b.lq - 1;
    const int kend = keys_seen(b, qlast), kopen = keys_seen(b, b.q0);
    const float *const K = static_cast<const float *>(a.k) + (int64_t)b.krow * a.ks + (int64_t)b.kvh * D;
    const float *const V = static_cast<const float *>(a.v) + (int64_t)b.krow * a.vs + (int64_t)b.kvh * D;
    f32x4 kr[D / 16];
    f32x4 vr[4][D / 64];
    auto request_k = [&](int j0) __attribute__((always_inline)) {
        const int rows = b.lk - j0 < BN ? b.lk - j0 : BN;
        const rsrc_t rs = make_rsrc(K + (int64_t)j0 * a.ks,
                                    rows > 0 ? (uint32_t)((rows - 1) * (int)a.ks + D) * 4 : 0u);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
            kr[s] = __builtin_bit_cast(f32x4, buf_ld16(rs, (uint32_t)(qi * (int)a.ks + 16 * s + 4 * g) * 4));
    };
    auto request_v = [&](int j0) __attribute__((always_inline)) {
        const int rows = b.lk - j0 < BN ? b.lk - j0 : BN;
        const rsrc_t rs = make_rsrc(V + (int64_t)j0 * a.vs,
                                    rows > 0 ? (uint32_t)((rows - 1) * (int)a.vs + D) * 4 : 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                vr[e][i] = __builtin_bit_cast(f32x4, buf_ld16(rs, (uint32_t)((4 * g + e) * (int)a.vs +
                                                                            64 * i + 4 * qi) * 4));
    };
    f32x4 o[QT][D / 16];
    float m[QT], sum[QT];
    bool odd = false;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = -__builtin_inff();
        sum[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[t][i] = zero4();
    }
    if (wave * BN < kend) {
        request_k(wave * BN);
        request_v(wave * BN);
    }
    for (int j0 = wave * BN; j0 < kend; j0 += NW * BN) {
        f32x4 s[QT];
#pragma unroll
        for (int t = 0; t < QT; ++t) s[t] = zero4();
#pragma unroll
        for (int st = 0; st < D / 16; ++st)
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int t = 0; t < QT; ++t) s[t] = Mma<float>::run(kr[st][v], qf[t][st][v], s[t]);
        request_k(j0 + NW * BN);
        if (j0 + BN > kopen) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const bool bad = !(fabsf(vr[e][i / 4][i % 4]) < __builtin_inff());
                    odd |= bad;
                    vr[e][i / 4][i % 4] = bad ? 0.0f : vr[e][i / 4][i % 4];
                }
        }
        float p[QT][4];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float top = -__builtin_inff();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[t][e] = j0 + 4 * g + e < seen[t] ? s[t][e] * a.scale2 : -__builtin_inff();
                top = fmaxf(top, s[t][e]);
            }
            top = across32(across16(top, larger), larger);
            const float was = m[t];
            m[t] = fmaxf(was, top);
            const float ref = m[t] == -__builtin_inff() ? 0.0f : m[t];
            const float f = __builtin_amdgcn_exp2f(was - ref);
            sum[t] *= f;
            if (__any(top > was)) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[t][i] *= f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[t][e] = __builtin_amdgcn_exp2f(s[t][e] - ref);
                sum[t] += p[t][e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int t = 0; t < QT; ++t) o[t][i] = Mma<float>::run(vr[e][i / 4][i % 4], p[t][e], o[t][i]);
        request_v(j0 + NW * BN);
    }
    if (__any(odd)) {              // the values taken out, from the wave that had their tile
        for (int k = kopen / BN * BN; k < kend; ++k)
            if (k / BN % NW == wave)
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = V[(int64_t)k * a.vs + 64 * (i / 4) + 16 * g + 4 * e + i % 4];
#pragma unroll
                        for (int t = 0; t < QT; ++t)
                            if (k < seen[t] && !(fabsf(v) < __builtin_inff())) o[t][i][e] += v;
                    }
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        sum[t] = across32(across16(sum[t], added), added);
        if (g == 0) {
            ml[wave][0][16 * t + qi] = m[t];
            ml[wave][1][16 * t + qi] = sum[t];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float top = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w][0][16 * t + qi]);
        const float f = __builtin_amdgcn_exp2f(m[t] - (top == -__builtin_inff() ? 0.0f : top));
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 v = {o[t][4 * i][e] * f, o[t][4 * i + 1][e] * f, o[t][4 * i + 2][e] * f,
                                 o[t][4 * i + 3][e] * f};
                *reinterpret_cast<f32x4 *>(&js.o[wave][(16 * t + qi) * (D + 4) + 64 * i + 16 * g + 4 * e]) = v;
            }
    }
    __syncthreads();
    join_waves<float, D, NQ, NW>(a, b, js.o, ml);
}

// Which kernel a call runs.
struct AttnPlan {
    int hpb;      // bf16: heads of a group that a block takes
    bool split;   // bf16: attn_split_kernel instead
    bool two;     // float: two tiles of queries a block
};
static AttnPlan attn_plan(const AttnDims &d)
{
    AttnPlan p{1, false, false};
    if (d.S <= 0 || d.Tq <= 0) return p;
    const int64_t Tq = d.Tq, S = d.S, H = d.H, group = H / d.Hkv;
    // bf16: the waves of a block on 4 or 2 heads of a group where that divides it, or
    // where sequences are too short to fill 128 queries of one (32 sequences of 32
    // queries on 4224 cached keys: 32 heads of 128 on 8 key heads 409 us with one head
    // a block, 172 us with 4; 40 heads of 64, five to a key head, 295 and 151 us)
    p.hpb = group % 4 == 0 || (group > 2 && Tq <= 40 * S) ? 4 : (group % 2 == 0 ? 2 : 1);
    // ... or sharing the keys of 32 queries of one head, where there are no blocks for
    // most of the 256 CUs, or not for two rounds of them and the keys are long, the more
    // blocks the longer (heads of 128, without and with, us: 1523 tokens, 2 heads, 24
    // blocks: 51 and 19; 512 tokens, 32 heads on 8, 136 blocks: 23 and 19; 1500, 12
    // heads, 144: 53 and 35; 1100, 32 on 8, 280: 42 and 50; 3000, 12 heads, 288: 96 and
    // 84; 4096, 10 heads, 330: 126 and 115; 6144, 8 heads, 392: 185 and 175; 4000, 16 on
    // 4, 504: 136 and 167). With rounded weights, which the shared form does not take,
    // the other one takes a quarter less and the limit is lower (3000, 12 heads: 70 and 84). Of
    // several sequences one is taken to be twice the mean: the lengths are not known
    // here, and the cost of a long one missed is the greater (15 prompts of 4789 on 9321,
    // one of them on 8000, 4 heads, 208 blocks: 221 and 61; 11 prompts of 89 on 123, 8
    // heads on 2, 82 blocks: 14 and 16)
    const int64_t blocks = (Tq * p.hpb / 128 + S) * d.Hkv * ((group + p.hpb - 1) / p.hpb);
    const int64_t longest = S == 1 ? d.Tk : 2 * (int64_t)d.Tk / S;
    p.split = blocks <= 144 || (blocks <= (d.bf16w ? 272 : 400) && longest > 4 * blocks);
    // float: two tiles of queries share the keys once there are enough of them
    p.two = (Tq / 32 + S) * H >= 512;
    return p;
}

const char *attn_kernel_name(const AttnDims &d)
{
    const AttnPlan p = attn_plan(d);
    const int wide = d.D == 128;
    if (!d.bf16) {
        static const char *const f[2][2] = {{"attn_f32_kernel<64, 1>", "attn_f32_kernel<128, 1>"},
                                            {"attn_f32_kernel<64, 2>", "attn_f32_kernel<128, 2>"}};
        return f[p.two][wide];
    }
    if (p.split) return wide ? "attn_split_kernel<128>" : "attn_split_kernel<64>";
    static const char *const b[3][2] = {{"attn_kernel<64, 1>", "attn_kernel<128, 1>"},
                                        {"attn_kernel<64, 2>", "attn_kernel<128, 2>"},
                                        {"attn_kernel<64, 4>", "attn_kernel<128, 4>"}};
    return b[p.hpb / 2][wide];
}

void launch_attn(const AttnDims &d, const void *q, const void *k, const void *v,
                 const int32_t *cuq, const int32_t *cuk, void *out, float *lse, void *stream)
{
    if (d.S <= 0 || d.Tq <= 0) return;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const AttnArgs a{q, k, v, cuq, cuk, out, lse, d.qs, d.ks, d.vs, d.os, d.Tq, d.Tk, d.S, d.H,
                     d.Hkv, d.causal ? 1 : 0, d.scale * kLog2e};
    const int64_t Tq = d.Tq, S = d.S, H = d.H, group = H / d.Hkv;
    const AttnPlan p = attn_plan(d);
#define SSD_ATTN(KERNEL, BM, HEADS, THREADS) \
    hipLaunchKernelGGL((KERNEL), dim3((unsigned)((Tq / (BM) + S) * (HEADS))), dim3(THREADS), 0, st, a)
#define SSD_ATTN_W(DD, BF16W)                                                                 \
    do {                                                                                      \
        if (p.hpb == 4)                                                                         \
            SSD_ATTN((attn_kernel<DD, 4, BF16W>), 32, d.Hkv * ((group + 3) / 4), 256);        \
        else if (p.hpb == 2) SSD_ATTN((attn_kernel<DD, 2, BF16W>), 64, H / 2, 256);             \
        else SSD_ATTN((attn_kernel<DD, 1, BF16W>), 128, H, 256);                              \
    } while (0)
#define SSD_ATTN_D(DD)                                                                        \
    do {                                                                                      \
        if (d.bf16 && p.split) SSD_ATTN(attn_split_kernel<DD>, 32, H, 512);                     \
        else if (d.bf16 && d.bf16w) SSD_ATTN_W(DD, true);                                     \
        else if (d.bf16) SSD_ATTN_W(DD, false);                                               \
        else if (p.two) SSD_ATTN((attn_f32_kernel<DD, 2>), 32, H, 256);                         \
        else SSD_ATTN((attn_f32_kernel<DD, 1>), 16, H, 256);                                  \
    } while (0)
    if (d.D == 128) SSD_ATTN_D(128);
    else SSD_ATTN_D(64);
#undef SSD_ATTN_D
#undef SSD_ATTN_W
#undef SSD_ATTN
}

}  // namespace ssd
