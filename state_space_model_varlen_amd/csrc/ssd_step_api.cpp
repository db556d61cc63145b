// C ABI of the operators between and behind the layers: host-side validation
// and dispatch to the launchers (ssd_step.h). As in ssd_api.cpp nothing here
// reads device memory or synchronises, and every check runs before the first
// launch of a call.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>

#include "ssd_step.h"
#include "../../include/ssd_mi355x.h"

namespace {

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool float_ok(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }
size_t size_of(int32_t d) { return d == SSD_F32 ? 4 : d == SSD_BF16 ? 2 : 1; }
ssd::Elem elem(int32_t d)
{
    return d == SSD_F32 ? ssd::Elem::f32 : d == SSD_BF16 ? ssd::Elem::bf16 : ssd::Elem::e4m3;
}

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

// A launch has at most 2^32 - 1 threads in a direction.
bool launches(int64_t blocks, int64_t threads) { return blocks <= 0xffffffffLL / threads; }

int workspace_ok(const void *workspace, size_t given, size_t need)
{
    if (need == 0) return SSD_OK;
    if (!workspace) return SSD_ERR_NULL;
    if (!aligned(workspace, 16)) return SSD_ERR_ALIGN;
    return given < need ? SSD_ERR_WORKSPACE : SSD_OK;
}

int norm_dims(const norm_problem *p, ssd::NormDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->rows < 0 || p->hidden <= 0 || p->ngroups <= 0) return SSD_ERR_SHAPE;
    if (p->hidden % p->ngroups != 0) return SSD_ERR_SHAPE;
    if (!float_ok(p->in_dtype) || !float_ok(p->residual_dtype) ||
        !(float_ok(p->out_dtype) || p->out_dtype == SSD_E4M3))
        return SSD_ERR_DTYPE;
    if (!(p->eps >= 0.0f) || !std::isfinite(p->eps)) return SSD_ERR_SHAPE;
    if (p->out_dtype == SSD_E4M3 && p->hidden / p->ngroups % 32 != 0) return SSD_ERR_UNSUPPORTED;
    // (elements are counted in 32 bits, a block's threads ahead)
    if (p->hidden / p->ngroups > 1 << 30) return SSD_ERR_UNSUPPORTED;
    const int per = p->hidden / p->ngroups, lanes = per <= 128 ? 16 : per <= 512 ? 64 : per / 8 + 64;
    if (!launches((int64_t)p->rows * p->ngroups, lanes < 1024 ? lanes : 1024)) return SSD_ERR_UNSUPPORTED;
    const int64_t h = p->hidden;
    if (!stride_of(p->x_stride, h, &d->xs) || !stride_of(p->gate_stride, h, &d->gs) ||
        !stride_of(p->residual_stride, h, &d->rs) ||
        !stride_of(p->residual_out_stride, h, &d->ros) || !stride_of(p->out_stride, h, &d->os))
        return SSD_ERR_SHAPE;
    d->rows = p->rows;
    d->hidden = p->hidden;
    d->groups = p->ngroups;
    d->in = elem(p->in_dtype);
    d->residual = elem(p->residual_dtype);
    d->out = elem(p->out_dtype);
    d->eps = p->eps;
    return SSD_OK;
}

int linear_dims(const linear_problem *p, ssd::LinearDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->tokens < 0 || p->in_features <= 0 || p->out_features <= 0) return SSD_ERR_SHAPE;
    if ((p->x_dtype != SSD_BF16 && p->x_dtype != SSD_E4M3) || !float_ok(p->out_dtype))
        return SSD_ERR_DTYPE;
    if (p->cut_products != 0 && p->cut_products != 1) return SSD_ERR_UNSUPPORTED;
    if (p->in_features % 32 != 0) return SSD_ERR_UNSUPPORTED;
    if (!stride_of(p->x_stride, p->in_features, &d->xs) ||
        !stride_of(p->out_stride, p->out_features, &d->os))
        return SSD_ERR_SHAPE;
    // a tile of up to 256 rows of x or of the weights is addressed by 32-bit byte offsets
    if (d->xs > (1 << 21) || p->in_features > (1 << 21)) return SSD_ERR_UNSUPPORTED;
    // (the largest tile: 256 tokens by 256 outputs, 512 threads; a block of few tokens: 16 outputs)
    if (!launches(((int64_t)p->tokens / 256 + 1) * ((int64_t)p->out_features / 256 + 1), 512) ||
        !launches((int64_t)p->out_features / 16 + 1, 256))
        return SSD_ERR_UNSUPPORTED;
    d->T = p->tokens;
    d->K = p->in_features;
    d->N = p->out_features;
    d->e4m3 = p->x_dtype == SSD_E4M3;
    d->out_bf16 = p->out_dtype == SSD_BF16;
    d->cut = p->cut_products != 0;
    return SSD_OK;
}

int probs_dims(const probs_problem *p, ssd::ProbsDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->num_reqs < 0 || p->tokens_per_req < 0 || p->vocab <= 0) return SSD_ERR_SHAPE;
    if (!float_ok(p->in_dtype)) return SSD_ERR_DTYPE;
    if (!stride_of(p->logits_stride, p->vocab, &d->ls) ||
        !stride_of(p->probs_stride, p->vocab, &d->ps))
        return SSD_ERR_SHAPE;
    // (whole rows by up to 1024 threads, or parts of at least 4096 logits by 256)
    const int64_t rows = (int64_t)p->num_reqs * p->tokens_per_req;
    if (p->vocab > (1 << 27) || !launches(rows, 1024) || !launches(rows * (p->vocab / 4096 + 1), 256))
        return SSD_ERR_UNSUPPORTED;
    d->R = p->num_reqs;
    d->T = p->tokens_per_req;
    d->V = p->vocab;
    d->bf16 = p->in_dtype == SSD_BF16;
    return SSD_OK;
}

int verify_dims(const verify_problem *p, ssd::VerifyDims *d)
{
    if (!p) return SSD_ERR_NULL;
    if (p->num_reqs < 0 || p->tokens_per_req <= 0 || p->vocab <= 0) return SSD_ERR_SHAPE;
    if (!stride_of(p->target_stride, p->vocab, &d->ts) ||
        !stride_of(p->draft_stride, p->vocab, &d->ds))
        return SSD_ERR_SHAPE;
    // (the drafts of a request are tested by the lanes of one wave)
    if (p->tokens_per_req > 65 || p->num_reqs > 65535 || p->vocab > (1 << 27))
        return SSD_ERR_UNSUPPORTED;
    d->R = p->num_reqs;
    d->T = p->tokens_per_req;
    d->V = p->vocab;
    return SSD_OK;
}

bool row_aligned(const void *p, int64_t stride, size_t e)
{
    return aligned(p, 16) && (uint64_t)stride * e % 16 == 0;
}

}  // namespace

extern "C" {

int rms_norm(const norm_problem *p, const void *x, const void *gate, const void *residual,
             const float *weight, void *out, uint8_t *out_scale, void *residual_out,
             void *stream)
{
    ssd::NormDims d;
    const int rc = norm_dims(p, &d);
    if (rc) return rc;
    if (!x || !out || (d.out == ssd::Elem::e4m3 && !out_scale)) return SSD_ERR_NULL;
    if (residual_out && !residual) return SSD_ERR_NULL;
    if (gate && residual) return SSD_ERR_UNSUPPORTED;
    const size_t e = size_of(p->in_dtype), r = size_of(p->residual_dtype);
    if (!aligned(x, e) || !aligned(gate, e) || !aligned(residual, r) ||
        !aligned(residual_out, r) || !aligned(weight, 4) || !aligned(out, size_of(p->out_dtype)))
        return SSD_ERR_ALIGN;
    ssd::launch_rms_norm(d, x, gate, residual, weight, out, out_scale, residual_out, stream);
    return launch_status();
}

// (none is needed: sums that waves share are joined in LDS)
size_t linear_w4_workspace_bytes(const linear_problem *) { return 0; }

const char *linear_w4_kernel(const linear_problem *p)
{
    ssd::LinearDims d;
    return linear_dims(p, &d) ? "" : ssd::linear_kernel_name(d);
}

int linear_w4(const linear_problem *p, const void *x, const uint8_t *x_scale,
              const uint8_t *weight, const uint8_t *weight_scale, const float *bias, void *out,
              void *, size_t, void *stream)
{
    ssd::LinearDims d;
    const int rc = linear_dims(p, &d);
    if (rc) return rc;
    if (!x || !weight || !weight_scale || !out || (d.e4m3 && !x_scale)) return SSD_ERR_NULL;
    if (!row_aligned(x, d.xs, size_of(p->x_dtype)) || !aligned(weight, 16) || !aligned(bias, 4) ||
        !aligned(out, size_of(p->out_dtype)))
        return SSD_ERR_ALIGN;
    const ssd::LinearArgs a{x, x_scale, weight, weight_scale, bias, out};
    ssd::launch_linear(d, a, stream);
    return launch_status();
}

int linear_w4_encode(const linear_problem *p, int32_t dtype, const void *w, uint8_t *weight,
                     uint8_t *weight_scale, void *stream)
{
    if (!p) return SSD_ERR_NULL;
    if (p->in_features <= 0 || p->out_features <= 0) return SSD_ERR_SHAPE;
    if (!float_ok(dtype)) return SSD_ERR_DTYPE;
    if (p->in_features % 32 != 0 ||
        !launches((int64_t)p->in_features / 32 * p->out_features + 255, 1))
        return SSD_ERR_UNSUPPORTED;
    if (!w || !weight || !weight_scale) return SSD_ERR_NULL;
    if (!aligned(w, 16) || !aligned(weight, 16)) return SSD_ERR_ALIGN;
    ssd::launch_linear_encode(p->out_features, p->in_features, dtype == SSD_BF16, w, weight,
                              weight_scale, stream);
    return launch_status();
}

size_t token_probs_workspace_bytes(const probs_problem *p)
{
    ssd::ProbsDims d;
    return probs_dims(p, &d) ? 0 : ssd::probs_workspace(d);
}

int token_probs(const probs_problem *p, const void *logits, const float *temperature,
                float *probs, void *workspace, size_t workspace_bytes, void *stream)
{
    ssd::ProbsDims d;
    int rc = probs_dims(p, &d);
    if (rc) return rc;
    if (!logits || !probs) return SSD_ERR_NULL;
    if (!aligned(logits, size_of(p->in_dtype)) || !aligned(probs, 4) || !aligned(temperature, 4))
        return SSD_ERR_ALIGN;
    rc = workspace_ok(workspace, workspace_bytes, ssd::probs_workspace(d));
    if (rc) return rc;
    ssd::launch_probs(d, logits, temperature, probs, workspace, stream);
    return launch_status();
}

size_t verify_drafts_workspace_bytes(const verify_problem *p)
{
    ssd::VerifyDims d;
    return verify_dims(p, &d) ? 0 : ssd::verify_workspace(d);
}

int verify_drafts(const verify_problem *p, const float *target_probs, const float *draft_probs,
                  const int32_t *draft_tokens, const int32_t *num_drafts, const float *uniform,
                  int32_t *num_accepted, int32_t *tokens, void *workspace,
                  size_t workspace_bytes, void *stream)
{
    ssd::VerifyDims d;
    int rc = verify_dims(p, &d);
    if (rc) return rc;
    if (!target_probs || !uniform || !num_accepted || !tokens || (d.T > 1 && !draft_tokens))
        return SSD_ERR_NULL;
    if (!aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(draft_tokens, 4) ||
        !aligned(num_drafts, 4) || !aligned(uniform, 4) || !aligned(num_accepted, 4) ||
        !aligned(tokens, 4))
        return SSD_ERR_ALIGN;
    rc = workspace_ok(workspace, workspace_bytes, ssd::verify_workspace(d));
    if (rc) return rc;
    const ssd::VerifyArgs a{target_probs, draft_probs, draft_tokens, num_drafts, uniform,
                            num_accepted, tokens};
    ssd::launch_verify(d, a, workspace, stream);
    return launch_status();
}

}  // extern "C"
