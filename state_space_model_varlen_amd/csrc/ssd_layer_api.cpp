// C ABI of the operators around the SSD scan: host-side validation and
// dispatch to the launchers (ssd_layer.h). As in ssd_api.cpp nothing here
// reads device memory or synchronises, and every check runs before the first
// launch of a call.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>

#include "ssd_layer.h"
#include "../../include/ssd_mi355x.h"

namespace {

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool float_ok(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }
size_t size_of(int32_t d) { return d == SSD_F32 ? 4 : 2; }

// A row stride: 0 means contiguous rows of n elements. False if rows overlap.
bool stride_of(int64_t given, int64_t n, int64_t *out)
{
    *out = given ? given : n;
    return *out >= n;
}

int launch_status()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

int conv_dims(const conv_problem *p, bool uniform, ssd::ConvDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->total_tokens < 0 || p->num_seqs < 0 || p->channels <= 0 || p->num_slots < 0)
        return SSD_ERR_SHAPE;
    if (p->num_seqs > 0 && p->num_slots <= 0) return SSD_ERR_SHAPE;
    if (p->num_seqs == 0 && p->total_tokens > 0) return SSD_ERR_SHAPE;
    if (uniform && p->num_seqs > 0 && p->total_tokens % p->num_seqs != 0) return SSD_ERR_SHAPE;
    if (!float_ok(p->in_dtype) || !float_ok(p->state_dtype)) return SSD_ERR_DTYPE;
    if (p->width < 2 || p->width > 4) return SSD_ERR_UNSUPPORTED;
    if (p->activation != SSD_ACT_NONE && p->activation != SSD_ACT_SILU) return SSD_ERR_UNSUPPORTED;
    if (!stride_of(p->x_stride, p->channels, &d->xs)) return SSD_ERR_SHAPE;
    int64_t sum = 0;
    for (int i = 0; i < 3; ++i) {
        if (p->y_channels[i] < 0) return SSD_ERR_SHAPE;
        sum += p->y_channels[i];
        d->yc[i] = p->y_channels[i];
    }
    if (sum == 0) d->yc[0] = p->channels;
    else if (sum != p->channels) return SSD_ERR_SHAPE;
    for (int i = 0; i < 3; ++i)
        if (!stride_of(p->y_stride[i], d->yc[i], &d->ys[i])) return SSD_ERR_SHAPE;
    // grid limit: token tiles of at least 4 tokens, and one for every sequence, times
    // blocks of at least 64 channels
    if (((int64_t)p->total_tokens / 4 + p->num_seqs) * (((int64_t)p->channels + 63) / 64) >
        0x7fffffffLL)
        return SSD_ERR_UNSUPPORTED;
    d->T = p->total_tokens;
    d->S = p->num_seqs;
    d->C = p->channels;
    d->W = p->width;
    d->num_slots = p->num_slots;
    d->in_bf16 = p->in_dtype == SSD_BF16;
    d->state_bf16 = p->state_dtype == SSD_BF16;
    d->silu = p->activation == SSD_ACT_SILU;
    return SSD_OK;
}

int conv_call(const conv_problem *p, bool uniform, const void *x, const float *weight,
              const float *bias, const int32_t *cu, void *cache, const int32_t *idx,
              const uint8_t *has, void *y0, void *y1, void *y2, bool write_state, void *stream)
{
    ssd::ConvDims d;
    const int rc = conv_dims(p, uniform, &d);
    if (rc) return rc;
    if (!x || !weight || !cache || !idx || (!uniform && !cu)) return SSD_ERR_NULL;
    void *const y[3] = {y0, y1, y2};
    const size_t e = size_of(p->in_dtype);
    for (int i = 0; i < 3; ++i) {
        if (d.yc[i] > 0 && !y[i]) return SSD_ERR_NULL;
        if (d.yc[i] > 0 && !aligned(y[i], e)) return SSD_ERR_ALIGN;
    }
    if (!aligned(x, e) || !aligned(cache, size_of(p->state_dtype)) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(cu, 4) || !aligned(idx, 4))
        return SSD_ERR_ALIGN;
    ssd::launch_conv(d, x, weight, bias, cu, cache, idx, has, uniform, y, write_state, stream);
    return launch_status();
}

int scan_dims(const scan_problem *p, bool uniform, const ssd_dt_transform *tf, ssd::ScanDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->total_tokens < 0 || p->num_seqs < 0 || p->channels <= 0 || p->d_state <= 0 ||
        p->ngroups <= 0 || p->num_slots < 0)
        return SSD_ERR_SHAPE;
    if (p->channels % p->ngroups != 0) return SSD_ERR_SHAPE;
    if (p->num_seqs > 0 && p->num_slots <= 0) return SSD_ERR_SHAPE;
    if (p->num_seqs == 0 && p->total_tokens > 0) return SSD_ERR_SHAPE;
    if (uniform && p->num_seqs > 0 && p->total_tokens % p->num_seqs != 0) return SSD_ERR_SHAPE;
    if (!float_ok(p->in_dtype) || !(float_ok(p->state_dtype) || p->state_dtype == SSD_F16))
        return SSD_ERR_DTYPE;
    if (p->d_state != 16 && p->d_state != 32 && p->d_state != 64) return SSD_ERR_UNSUPPORTED;
    const int64_t gn = (int64_t)p->ngroups * p->d_state;
    if (!stride_of(p->x_stride, p->channels, &d->xs) ||
        !stride_of(p->dt_stride, p->channels, &d->dts) ||
        !stride_of(p->z_stride, p->channels, &d->zs) || !stride_of(p->b_stride, gn, &d->bs) ||
        !stride_of(p->c_stride, gn, &d->cs) || !stride_of(p->y_stride, p->channels, &d->ys))
        return SSD_ERR_SHAPE;
    // a stage of up to 64 rows is addressed by 32-bit byte offsets
    for (int64_t v : {d->xs, d->dts, d->zs, d->bs, d->cs, d->ys})
        if (v > (1 << 21)) return SSD_ERR_UNSUPPORTED;
    d->tf = ssd::DtTf();
    if (tf) {
        if (!(tf->dt_min <= tf->dt_max)) return SSD_ERR_SHAPE;   // (NaN bounds fail too)
        d->tf.bias = tf->dt_bias;
        d->tf.lo = tf->dt_min;
        d->tf.hi = tf->dt_max;
        d->tf.on = 1;
    }
    // grid limits: channel blocks (at least 16 channels of one group each) times
    // sequences, and times the time segments of the prompt form
    const int64_t cb = ((int64_t)p->channels / p->ngroups + 15) / 16 * p->ngroups;
    if (cb * ((int64_t)p->num_seqs + p->total_tokens / 64 + 1) > 0x7fffffffLL)
        return SSD_ERR_UNSUPPORTED;
    d->T = p->total_tokens;
    d->S = p->num_seqs;
    d->C = p->channels;
    d->N = p->d_state;
    d->G = p->ngroups;
    d->num_slots = p->num_slots;
    d->in_bf16 = p->in_dtype == SSD_BF16;
    d->state_dtype = p->state_dtype;
    return SSD_OK;
}

int scan_pointers(const scan_problem *p, const ssd::ScanArgs &a)
{
    if (!a.x || !a.dt || !a.A || !a.B || !a.C || !a.cache || !a.idx || !a.y) return SSD_ERR_NULL;
    const size_t e = size_of(p->in_dtype);
    if (!aligned(a.x, e) || !aligned(a.dt, e) || !aligned(a.B, e) || !aligned(a.C, e) ||
        !aligned(a.z, e) || !aligned(a.y, e) || !aligned(a.A, 16) || !aligned(a.D, 4) ||
        !aligned(a.cache, 16) || !aligned(a.idx, 4) || !aligned(a.cu, 4))
        return SSD_ERR_ALIGN;
    return SSD_OK;
}

bool headdim_ok(int d) { return d == 64 || d == 128; }

// (the running maximum is taken before the scale is applied: it must be positive)
bool scale_of(float given, int headdim, float *out)
{
    *out = given == 0.0f ? 1.0f / std::sqrt((float)headdim) : given;
    return std::isfinite(*out) && *out > 0.0f;
}

int attn_dims(const attn_problem *p, ssd::AttnDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->total_q < 0 || p->total_k < 0 || p->num_seqs < 0 || p->nheads <= 0 ||
        p->nkv_heads <= 0 || p->headdim <= 0)
        return SSD_ERR_SHAPE;
    if (p->nheads % p->nkv_heads != 0) return SSD_ERR_SHAPE;
    if (p->num_seqs == 0 && (p->total_q > 0 || p->total_k > 0)) return SSD_ERR_SHAPE;
    if (!float_ok(p->dtype)) return SSD_ERR_DTYPE;
    if (!headdim_ok(p->headdim)) return SSD_ERR_UNSUPPORTED;
    if (p->bf16_weights != 0 && p->bf16_weights != 1) return SSD_ERR_UNSUPPORTED;
    // grid limit: query tiles of at least 16 rows, one more a sequence, times heads
    if (((int64_t)p->total_q / 16 + p->num_seqs) * p->nheads > 0x7fffffffLL)
        return SSD_ERR_UNSUPPORTED;
    const int64_t qr = (int64_t)p->nheads * p->headdim, kr = (int64_t)p->nkv_heads * p->headdim;
    if (!stride_of(p->q_stride, qr, &d->qs) || !stride_of(p->k_stride, kr, &d->ks) ||
        !stride_of(p->v_stride, kr, &d->vs) || !stride_of(p->o_stride, qr, &d->os))
        return SSD_ERR_SHAPE;
    // a tile of up to 256 rows is addressed by 32-bit byte offsets
    if (d->qs > (1 << 21) || d->ks > (1 << 21) || d->vs > (1 << 21)) return SSD_ERR_UNSUPPORTED;
    if (!scale_of(p->scale, p->headdim, &d->scale)) return SSD_ERR_SHAPE;
    d->Tq = p->total_q;
    d->Tk = p->total_k;
    d->S = p->num_seqs;
    d->H = p->nheads;
    d->Hkv = p->nkv_heads;
    d->D = p->headdim;
    d->bf16 = p->dtype == SSD_BF16;
    d->causal = p->causal != 0;
    d->bf16w = p->bf16_weights != 0;
    return SSD_OK;
}

int kv_dims(const kv_cache_problem *p, ssd::KvDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->num_pages <= 0 || p->page_size <= 0 || p->nkv_heads <= 0 || p->headdim <= 0)
        return SSD_ERR_SHAPE;
    if (!float_ok(p->in_dtype) || (p->cache_dtype != SSD_BF16 && p->cache_dtype != SSD_E4M3))
        return SSD_ERR_DTYPE;
    const int pg = p->page_size;
    if (!headdim_ok(p->headdim) || pg < 16 || pg > 256 || (pg & (pg - 1))) return SSD_ERR_UNSUPPORTED;
    if (p->nkv_heads > 65535) return SSD_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)p->nkv_heads * p->headdim;
    if (!stride_of(p->k_stride, row, &d->ks) || !stride_of(p->v_stride, row, &d->vs))
        return SSD_ERR_SHAPE;
    d->pages = p->num_pages;
    d->page = pg;
    d->Hkv = p->nkv_heads;
    d->D = p->headdim;
    d->in_bf16 = p->in_dtype == SSD_BF16;
    d->e4m3 = p->cache_dtype == SSD_E4M3;
    return SSD_OK;
}

int kv_pointers(const ssd::KvDims &d, const ssd::KvCache &c)
{
    if (!c.k || !c.v || (d.e4m3 && (!c.ksc || !c.vsc))) return SSD_ERR_NULL;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return SSD_ERR_ALIGN;
    return SSD_OK;
}

bool row_aligned(const void *p, int64_t stride, size_t e)
{
    return aligned(p, 16) && (uint64_t)stride * e % 16 == 0;
}

int decode_dims(const attn_decode_problem *p, ssd::DecodeAttnDims *d)
{
    if (!p) return SSD_ERR_NULL;
    const int rc = kv_dims(&p->kv, &d->kv);
    if (rc) return rc;
    if (p->num_reqs < 0 || p->tokens_per_req < 0 || p->nheads <= 0 || p->max_pages < 0)
        return SSD_ERR_SHAPE;
    if (p->nheads % p->kv.nkv_heads != 0) return SSD_ERR_SHAPE;
    if (p->kv.in_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->num_reqs > 65535 || (int64_t)p->tokens_per_req * p->nheads > 65535 ||
        (int64_t)p->max_pages * p->kv.page_size > 0x7fffff00LL)
        return SSD_ERR_UNSUPPORTED;
    if (!scale_of(p->scale, p->kv.headdim, &d->scale)) return SSD_ERR_SHAPE;
    const int64_t row = (int64_t)p->nheads * p->kv.headdim;
    if (!stride_of(p->q_stride, row, &d->qs) || !stride_of(p->o_stride, row, &d->os))
        return SSD_ERR_SHAPE;
    d->R = p->num_reqs;
    d->T = p->tokens_per_req;
    d->H = p->nheads;
    d->max_pages = p->max_pages;
    return SSD_OK;
}

}  // namespace

extern "C" {

int causal_conv1d_varlen(const conv_problem *p, const void *x, const float *weight,
                         const float *bias, const int32_t *cu_seqlens, void *conv_cache,
                         const int32_t *state_indices, const uint8_t *has_initial_state, void *y0,
                         void *y1, void *y2, void *stream)
{
    return conv_call(p, false, x, weight, bias, cu_seqlens, conv_cache, state_indices,
                     has_initial_state, y0, y1, y2, true, stream);
}

int causal_conv1d_update(const conv_problem *p, const void *x, const float *weight,
                         const float *bias, void *conv_cache, const int32_t *state_indices,
                         void *y0, void *y1, void *y2, int32_t update_cache, void *stream)
{
    return conv_call(p, true, x, weight, bias, nullptr, conv_cache, state_indices, nullptr, y0, y1,
                     y2, update_cache != 0, stream);
}

int causal_conv1d_commit(const conv_problem *p, const void *x, void *conv_cache,
                         const int32_t *state_indices, const int32_t *num_accepted, void *stream)
{
    ssd::ConvDims d;
    const int rc = conv_dims(p, true, &d);
    if (rc) return rc;
    if (!x || !conv_cache || !state_indices || !num_accepted) return SSD_ERR_NULL;
    if (!aligned(x, size_of(p->in_dtype)) || !aligned(conv_cache, size_of(p->state_dtype)) ||
        !aligned(state_indices, 4) || !aligned(num_accepted, 4))
        return SSD_ERR_ALIGN;
    ssd::launch_conv_commit(d, x, conv_cache, state_indices, num_accepted, stream);
    return launch_status();
}

size_t selective_scan_workspace_bytes(const scan_problem *p)
{
    ssd::ScanDims d;
    return scan_dims(p, false, nullptr, &d) ? 0 : ssd::scan_workspace(d);
}

const char *selective_scan_varlen_kernel(const scan_problem *p)
{
    ssd::ScanDims d;
    return scan_dims(p, false, nullptr, &d) ? "" : ssd::scan_kernel_name(d);
}

int selective_scan_varlen(const scan_problem *p, const void *x, const void *dt, const float *A,
                          const void *B, const void *C, const float *D, const void *z,
                          const ssd_dt_transform *dt_transform, const int32_t *cu_seqlens,
                          void *state_cache, const int32_t *state_indices,
                          const uint8_t *has_initial_state, void *y, void *workspace,
                          size_t workspace_bytes, void *stream)
{
    ssd::ScanDims d;
    int rc = scan_dims(p, false, dt_transform, &d);
    if (rc) return rc;
    const ssd::ScanArgs a{x, dt, B, C, z, A, D, cu_seqlens, state_indices, has_initial_state,
                          state_cache, y};
    if (!cu_seqlens) return SSD_ERR_NULL;
    rc = scan_pointers(p, a);
    if (rc) return rc;
    const size_t need = ssd::scan_workspace(d);
    if (need > 0) {
        if (!workspace) return SSD_ERR_NULL;
        if (!aligned(workspace, 16)) return SSD_ERR_ALIGN;
        if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    }
    ssd::launch_scan(d, a, workspace, stream);
    return launch_status();
}

int selective_scan_update(const scan_problem *p, const void *x, const void *dt, const float *A,
                          const void *B, const void *C, const float *D, const void *z,
                          const ssd_dt_transform *dt_transform, void *state_cache,
                          const int32_t *state_indices, void *y, void *intermediate_states,
                          void *stream)
{
    ssd::ScanDims d;
    int rc = scan_dims(p, true, dt_transform, &d);
    if (rc) return rc;
    const ssd::ScanArgs a{x, dt, B, C, z, A, D, nullptr, state_indices, nullptr, state_cache, y};
    rc = scan_pointers(p, a);
    if (rc) return rc;
    if (!aligned(intermediate_states, 16)) return SSD_ERR_ALIGN;
    ssd::launch_scan_update(d, a, intermediate_states, stream);
    return launch_status();
}

const char *attention_varlen_kernel(const attn_problem *p)
{
    ssd::AttnDims d;
    return attn_dims(p, &d) ? "" : ssd::attn_kernel_name(d);
}

int attention_varlen(const attn_problem *p, const void *q, const void *k, const void *v,
                     const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, void *out,
                     float *lse, void *stream)
{
    ssd::AttnDims d;
    const int rc = attn_dims(p, &d);
    if (rc) return rc;
    if (!q || !k || !v || !cu_seqlens_q || !cu_seqlens_k || !out) return SSD_ERR_NULL;
    const size_t e = size_of(p->dtype);
    if (!row_aligned(q, d.qs, e) || !row_aligned(k, d.ks, e) || !row_aligned(v, d.vs, e) ||
        !row_aligned(out, d.os, e) || !aligned(lse, 4) || !aligned(cu_seqlens_q, 4) ||
        !aligned(cu_seqlens_k, 4))
        return SSD_ERR_ALIGN;
    ssd::launch_attn(d, q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse, stream);
    return launch_status();
}

int kv_cache_store(const kv_cache_problem *p, int32_t num_tokens, const void *k, const void *v,
                   const int64_t *slot_mapping, void *k_cache, void *v_cache, uint8_t *k_scale,
                   uint8_t *v_scale, void *stream)
{
    ssd::KvDims d;
    int rc = kv_dims(p, &d);
    if (rc) return rc;
    if (num_tokens < 0) return SSD_ERR_SHAPE;
    if ((int64_t)num_tokens * d.Hkv > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
    const ssd::KvCache c{k_cache, v_cache, k_scale, v_scale};
    rc = kv_pointers(d, c);
    if (rc) return rc;
    if (!k || !v || !slot_mapping) return SSD_ERR_NULL;
    const size_t e = size_of(p->in_dtype);
    if (!row_aligned(k, d.ks, e) || !row_aligned(v, d.vs, e) || !aligned(slot_mapping, 8))
        return SSD_ERR_ALIGN;
    ssd::launch_kv_store(d, num_tokens, k, v, slot_mapping, c, stream);
    return launch_status();
}

int kv_cache_load(const kv_cache_problem *p, int32_t total_tokens, int32_t num_seqs,
                  int32_t max_pages, const int32_t *cu_seqlens, const int32_t *block_table,
                  const void *k_cache, const void *v_cache, const uint8_t *k_scale,
                  const uint8_t *v_scale, void *k, void *v, void *stream)
{
    ssd::KvDims d;
    int rc = kv_dims(p, &d);
    if (rc) return rc;
    if (total_tokens < 0 || num_seqs < 0 || max_pages < 0) return SSD_ERR_SHAPE;
    if (num_seqs == 0 && total_tokens > 0) return SSD_ERR_SHAPE;
    const ssd::KvCache c{const_cast<void *>(k_cache), const_cast<void *>(v_cache),
                         const_cast<uint8_t *>(k_scale), const_cast<uint8_t *>(v_scale)};
    rc = kv_pointers(d, c);
    if (rc) return rc;
    if (!cu_seqlens || !block_table || !k || !v) return SSD_ERR_NULL;
    const size_t e = size_of(p->in_dtype);
    if (!row_aligned(k, d.ks, e) || !row_aligned(v, d.vs, e) || !aligned(cu_seqlens, 4) ||
        !aligned(block_table, 4))
        return SSD_ERR_ALIGN;
    ssd::launch_kv_load(d, total_tokens, num_seqs, max_pages, cu_seqlens, block_table, c, k, v,
                        stream);
    return launch_status();
}

size_t attn_decode_workspace_bytes(const attn_decode_problem *p)
{
    ssd::DecodeAttnDims d;
    return decode_dims(p, &d) ? 0 : ssd::decode_attn_workspace(d);
}

int attention_decode(const attn_decode_problem *p, const void *q, const void *k_cache,
                     const void *v_cache, const uint8_t *k_scale, const uint8_t *v_scale,
                     const int32_t *block_table, const int32_t *context_lens, void *out,
                     float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    ssd::DecodeAttnDims d;
    int rc = decode_dims(p, &d);
    if (rc) return rc;
    const ssd::KvCache c{const_cast<void *>(k_cache), const_cast<void *>(v_cache),
                         const_cast<uint8_t *>(k_scale), const_cast<uint8_t *>(v_scale)};
    rc = kv_pointers(d.kv, c);
    if (rc) return rc;
    if (!q || !block_table || !context_lens || !out) return SSD_ERR_NULL;
    if (!row_aligned(q, d.qs, 2) || !row_aligned(out, d.os, 2) || !aligned(lse, 4) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4))
        return SSD_ERR_ALIGN;
    const size_t need = ssd::decode_attn_workspace(d);
    if (need > 0) {
        if (!workspace) return SSD_ERR_NULL;
        if (!aligned(workspace, 16)) return SSD_ERR_ALIGN;
        if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    }
    ssd::launch_decode_attn(d, q, c, block_table, context_lens, out, lse, workspace, stream);
    return launch_status();
}

}  // extern "C"
