// Launchers of the operators between and behind the layers (norm, products
// with 4-bit weights, token probabilities, verification of drafts). As in
// ssd_launch.h, every launcher only enqueues; arguments are validated by the
// caller.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ssd {

enum class Elem { f32, bf16, e4m3 };

struct NormDims {
    int64_t rows;
    int hidden, groups;
    Elem in, residual, out;
    float eps;
    int64_t xs, gs, rs, ros, os;
};
void launch_rms_norm(const NormDims &d, const void *x, const void *gate, const void *residual,
                     const float *weight, void *out, uint8_t *out_scale, void *residual_out,
                     void *stream);

struct LinearDims {
    int T, K, N;
    bool e4m3, out_bf16, cut;
    int64_t xs, os;
};
struct LinearArgs {
    const void *x;
    const uint8_t *x_scale, *w, *w_scale;
    const float *bias;
    void *out;
};
const char *linear_kernel_name(const LinearDims &d);
void launch_linear(const LinearDims &d, const LinearArgs &a, void *stream);
void launch_linear_encode(int N, int K, bool bf16, const void *w, uint8_t *codes, uint8_t *scale,
                          void *stream);

struct ProbsDims {
    int R, T, V;
    bool bf16;
    int64_t ls, ps;
};
size_t probs_workspace(const ProbsDims &d);
void launch_probs(const ProbsDims &d, const void *logits, const float *temperature, float *probs,
                  void *workspace, void *stream);

struct VerifyDims {
    int R, T, V;
    int64_t ts, ds;
};
struct VerifyArgs {
    const float *target, *draft;
    const int32_t *tokens, *count;
    const float *uniform;
    int32_t *accepted, *out;
};
size_t verify_workspace(const VerifyDims &d);
void launch_verify(const VerifyDims &d, const VerifyArgs &a, void *workspace, void *stream);

}  // namespace ssd
