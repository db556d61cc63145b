// Launchers of the operators around the scan (short convolution, channel-wise
// scan, attention, paged cache), and the device helpers they share. As in
// ssd_launch.h, every launcher only enqueues; arguments are validated by the
// caller.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ssd_launch.h"

namespace ssd {

struct ConvDims {
    int T, S, C, W, num_slots;
    bool in_bf16, state_bf16, silu;
    int64_t xs;            // row stride of x
    int yc[3];             // channels of each output
    int64_t ys[3];
};
// cu null: request s owns rows s T/S .. ; has null: no slot is read, unless
// `all_init` (the update: every slot is). write_state 0 leaves the cache.
void launch_conv(const ConvDims &d, const void *x, const float *w, const float *bias,
                 const int32_t *cu, void *cache, const int32_t *idx, const uint8_t *has,
                 bool all_init, void *const y[3], bool write_state, void *stream);
void launch_conv_commit(const ConvDims &d, const void *x, void *cache, const int32_t *idx,
                        const int32_t *accepted, void *stream);

struct ScanDims {
    int T, S, C, N, G, num_slots;
    bool in_bf16;
    int state_dtype;
    int64_t xs, dts, zs, bs, cs, ys;
    DtTf tf;
};
struct ScanArgs {
    const void *x, *dt, *B, *C, *z;
    const float *A, *D;
    const int32_t *cu, *idx;
    const uint8_t *has;
    void *cache, *y;
};
size_t scan_workspace(const ScanDims &d);
const char *scan_kernel_name(const ScanDims &d);
void launch_scan(const ScanDims &d, const ScanArgs &a, void *workspace, void *stream);
void launch_scan_update(const ScanDims &d, const ScanArgs &a, void *inter, void *stream);

struct AttnDims {
    int Tq, Tk, S, H, Hkv, D;
    bool bf16, causal, bf16w;
    float scale;
    int64_t qs, ks, vs, os;
};
const char *attn_kernel_name(const AttnDims &d);
void launch_attn(const AttnDims &d, const void *q, const void *k, const void *v,
                 const int32_t *cuq, const int32_t *cuk, void *out, float *lse, void *stream);

struct KvDims {
    int pages, page, Hkv, D;
    bool in_bf16, e4m3;
    int64_t ks, vs;
};
struct KvCache {
    void *k, *v;
    uint8_t *ksc, *vsc;
};
void launch_kv_store(const KvDims &d, int T, const void *k, const void *v, const int64_t *slots,
                     const KvCache &c, void *stream);
void launch_kv_load(const KvDims &d, int T, int S, int max_pages, const int32_t *cu,
                    const int32_t *table, const KvCache &c, void *k, void *v, void *stream);

struct DecodeAttnDims {
    KvDims kv;
    int R, T, H, max_pages;
    float scale;
    int64_t qs, os;
};
size_t decode_attn_workspace(const DecodeAttnDims &d);
void launch_decode_attn(const DecodeAttnDims &d, const void *q, const KvCache &c,
                        const int32_t *table, const int32_t *lens, void *out, float *lse,
                        void *workspace, void *stream);

}  // namespace ssd
