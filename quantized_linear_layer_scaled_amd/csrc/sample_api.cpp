// C ABI of the sampler (declared in include/qll.h): argument validation and
// the launch.  Nothing here allocates, synchronizes or throws.
#include <hip/hip_runtime_api.h>

#include "../../include/qll.h"
#include "sample_internal.h"

using namespace qll;

namespace {

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

int validate(int64_t B, int64_t V)
{
    if (B < 0 || V < 1 || B >= (int64_t)1 << 22)
        return QLL_ERR_INVALID_ARG;
    return V > kSampleMaxVocab ? QLL_ERR_UNSUPPORTED : QLL_OK;
}

}  // namespace

extern "C" {

int64_t qll_sample_workspace_bytes(int64_t B, int64_t V)
{
    const int rc = validate(B, V);
    if (rc != QLL_OK)
        return -rc;
    const int parts = sample_parts(B, V);
    return parts > 1 ? B * parts * sample_part_bytes() : 0;
}

int sample_tokens(const void* logits, int logits_dtype, int64_t ld, const float* u,
                  const float* temperature, const int32_t* top_k, const float* top_p,
                  const float* min_p, int32_t* tokens, float* probs, int64_t B, int64_t V, void* ws,
                  size_t ws_bytes, void* stream)
{
    const int rc = validate(B, V);
    if (rc != QLL_OK)
        return rc;
    const bool bf16 = logits_dtype == QLL_OUT_BF16;
    if ((!bf16 && logits_dtype != QLL_OUT_FP32) || ld < V || ld > ((int64_t)1 << 40))
        return QLL_ERR_INVALID_ARG;
    if (B == 0)
        return QLL_OK;
    if (!logits || !u || !tokens)
        return QLL_ERR_INVALID_ARG;
    if (misaligned(logits, bf16 ? 2 : 4) || misaligned(u, 4) || misaligned(temperature, 4) ||
        misaligned(top_k, 4) || misaligned(top_p, 4) || misaligned(min_p, 4) ||
        misaligned(tokens, 4) || misaligned(probs, 4))
        return QLL_ERR_MISALIGNED;
    SampleArgs a = {};
    a.parts = sample_parts(B, V);
    if (a.parts > 1) {
        if (!ws || ws_bytes < (uint64_t)(B * a.parts * sample_part_bytes()))
            return QLL_ERR_WORKSPACE;
        if (misaligned(ws, 16))
            return QLL_ERR_MISALIGNED;
        a.ws = ws;
    }
    a.logits = logits;
    a.ld = ld;
    a.bf16 = bf16;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.probs = probs;
    a.B = (int)B;
    a.V = (int)V;
    int bits = 0;
    while ((V >> bits) != 0)
        ++bits;
    // a bin's sum holds V counts above V complements below 2^(ebits - 6)
    a.ebits = 70 - 2 * bits < 38 ? 70 - 2 * bits : 38;
    return launch_sample(a, (hipStream_t)stream) == hipSuccess ? QLL_OK : QLL_ERR_HIP;
}

}  // extern "C"
