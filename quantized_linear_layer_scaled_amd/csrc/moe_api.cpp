// C ABI of the expert operators (declared in include/qll.h): argument
// validation, workspace layout and launches.  Nothing here allocates,
// synchronizes or throws.
#include <hip/hip_runtime_api.h>

#include "../../include/qll.h"
#include "moe_internal.h"

namespace qll {
namespace {

constexpr int64_t kMaxDim = 0x3FFFFF00;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxRowBytes = (((int64_t)1 << 31) - 1) / 256;
constexpr int64_t kMaxChoices = (int64_t)1 << 26;  // (twice kLaunchWaves)

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? QLL_OK : QLL_ERR_HIP; }

int validate_choices(int64_t T, int64_t topk)
{
    if (T < 0 || topk < 1 || T > kMaxDim)
        return QLL_ERR_INVALID_ARG;
    if (topk > kMoeMaxTopk || T * topk > kMaxChoices)
        return QLL_ERR_UNSUPPORTED;
    return QLL_OK;
}

int validate_experts(int64_t T, int64_t E, int64_t topk, bool distinct)
{
    if (E < 1 || (distinct && topk > E))
        return QLL_ERR_INVALID_ARG;
    if (E > kMoeMaxExperts)
        return QLL_ERR_UNSUPPORTED;
    return validate_choices(T, topk);
}

SortArgs sort_args(const int32_t* ids, int32_t* offsets, int32_t* rows, int32_t* places, int64_t T,
                   int64_t E, int64_t topk, int64_t* need)
{
    SortArgs a = {};
    a.ids = ids;
    a.offsets = offsets;
    a.rows = rows;
    a.places = places;
    a.T = (int)T;
    a.E = (int)E;
    a.k = (int)topk;
    *need = moe_sort_plan(a);
    return a;
}

// The workspace of a sort, or why not.
int sort_workspace(SortArgs& a, int64_t need, void* ws, size_t ws_bytes)
{
    if (need == 0)
        return QLL_OK;
    if (!ws || ws_bytes < (uint64_t)need)
        return QLL_ERR_WORKSPACE;
    if (misaligned(ws, 16))
        return QLL_ERR_MISALIGNED;
    a.hist = (int*)ws;
    return QLL_OK;
}

int validate_combine(const void* y, bool need_y, const void* places, const void* weights, int dtype, int64_t T,
                     int64_t R, int64_t K, int64_t topk)
{
    if (R < 0 || K <= 0 || K % 8 || R > kMaxDim || K > kMaxDim || R * K > kMaxElems)
        return QLL_ERR_INVALID_ARG;
    const int rc = validate_choices(T, topk);
    if (rc != QLL_OK)
        return rc;
    if (T * K > kMaxElems || (dtype != QLL_OUT_BF16 && dtype != QLL_OUT_FP32))
        return QLL_ERR_INVALID_ARG;
    if (T == 0)
        return QLL_OK;
    if ((!y && need_y && R > 0) || !places)
        return QLL_ERR_INVALID_ARG;
    if (misaligned(y, 16) || misaligned(places, 4) || misaligned(weights, 4))
        return QLL_ERR_MISALIGNED;
    return QLL_OK;
}

CombineArgs combine_args(const void* y, const int32_t* places, const float* weights, int dtype,
                         int64_t T, int64_t R, int64_t K, int64_t topk)
{
    CombineArgs a = {};
    a.y = (const uint16_t*)y;
    a.places = places;
    a.weights = weights;
    a.fp32 = dtype == QLL_OUT_FP32;
    a.T = (int)T;
    a.R = (int)R;
    a.K = (int)K;
    a.k = (int)topk;
    return a;
}

}  // namespace
}  // namespace qll

using namespace qll;

extern "C" {

int64_t qll_moe_sort_workspace_bytes(int64_t T, int64_t E, int64_t topk)
{
    const int rc = validate_experts(T, E, topk, false);
    if (rc != QLL_OK)
        return -rc;
    int64_t need;
    sort_args(nullptr, nullptr, nullptr, nullptr, T, E, topk, &need);
    return need;
}

int moe_route(const void* logits, int logits_dtype, const float* bias, int score, int64_t groups,
              int64_t topk_groups, int group_best, int64_t topk, int renormalize, float scale,
              int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* places,
              int64_t T, int64_t E, void* ws, size_t ws_bytes, void* stream)
{
    int rc = validate_experts(T, E, topk, true);
    if (rc != QLL_OK)
        return rc;
    if (logits_dtype != QLL_OUT_BF16 && logits_dtype != QLL_OUT_FP32)
        return QLL_ERR_INVALID_ARG;
    if (score < 0 || score >= SCORE_COUNT || (group_best != 1 && group_best != 2))
        return QLL_ERR_INVALID_ARG;
    if (groups < 1 || groups > E || E % groups || topk_groups < 1 || topk_groups > groups ||
        topk > topk_groups * (E / groups))
        return QLL_ERR_INVALID_ARG;
    if (groups > 64)
        return QLL_ERR_UNSUPPORTED;
    // the sorted rows are wanted or not; without tokens the lists are empty,
    // and an empty tensor's address may be NULL
    if (T > 0 && ((offsets != nullptr) != (rows != nullptr) || (offsets != nullptr) != (places != nullptr)))
        return QLL_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !ids || !weights))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4) ||
        misaligned(offsets, 4) || misaligned(rows, 4) || misaligned(places, 4))
        return QLL_ERR_MISALIGNED;
    int64_t need = 0;
    RouteArgs a = {};
    a.sort = sort_args(ids, offsets, rows, places, T, E, topk, &need);
    if (offsets && (rc = sort_workspace(a.sort, need, ws, ws_bytes)) != QLL_OK)
        return rc;
    if (T == 0)
        return offsets ? hip_status(launch_moe_sort(a.sort, (hipStream_t)stream)) : QLL_OK;
    a.logits = logits;
    a.bf16 = logits_dtype == QLL_OUT_BF16;
    a.bias = bias;
    a.score = score;
    a.groups = (int)groups;
    a.keep = (int)topk_groups;
    a.group_best = group_best;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    return hip_status(launch_moe_route(a, (hipStream_t)stream));
}

int moe_route_backward(const void* logits, int logits_dtype, int score, int renormalize, float scale,
                       const int32_t* ids, const float* dweights, void* dlogits, int64_t T, int64_t E,
                       int64_t topk, void* stream)
{
    const int rc = validate_experts(T, E, topk, false);
    if (rc != QLL_OK)
        return rc;
    if ((logits_dtype != QLL_OUT_BF16 && logits_dtype != QLL_OUT_FP32) || score < 0 ||
        score >= SCORE_COUNT)
        return QLL_ERR_INVALID_ARG;
    if (T == 0)
        return QLL_OK;
    if (!logits || !ids || !dweights || !dlogits)
        return QLL_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(dlogits, 16) || misaligned(ids, 4) || misaligned(dweights, 4))
        return QLL_ERR_MISALIGNED;
    const RouteBackwardArgs a = {logits, logits_dtype == QLL_OUT_BF16, score, renormalize != 0, scale,
                                 ids, dweights, dlogits, (int)T, (int)E, (int)topk};
    return hip_status(launch_moe_route_backward(a, (hipStream_t)stream));
}

int moe_sort(const int32_t* ids, int32_t* offsets, int32_t* rows, int32_t* places, int64_t T,
             int64_t E, int64_t topk, void* ws, size_t ws_bytes, void* stream)
{
    int rc = validate_experts(T, E, topk, false);
    if (rc != QLL_OK)
        return rc;
    if (!offsets || (T > 0 && (!ids || !rows || !places)))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(ids, 4) || misaligned(offsets, 4) || misaligned(rows, 4) || misaligned(places, 4))
        return QLL_ERR_MISALIGNED;
    int64_t need;
    SortArgs a = sort_args(ids, offsets, rows, places, T, E, topk, &need);
    if ((rc = sort_workspace(a, need, ws, ws_bytes)) != QLL_OK)
        return rc;
    return hip_status(launch_moe_sort(a, (hipStream_t)stream));
}

int gated_fp8_grouped(const void* A, const void* Bg, const void* Bu, const float* sa, const float* sg,
                      const float* su, const int32_t* offsets, const int32_t* rows, int act, void* out,
                      int out_dtype, int64_t T, int64_t R, int64_t N, int64_t K, int64_t E,
                      void* stream)
{
    if (T < 0 || R < 0 || N <= 0 || K <= 0 || E < 1 || T > kMaxDim || R > kMaxDim || N > kMaxDim ||
        K > kMaxDim || E > 65536 || K % 16 || act < 0 || act >= ACT_COUNT)
        return QLL_ERR_INVALID_ARG;
    if (T * K > kMaxElems || R * N > kMaxElems || N * K > kMaxElems || E * (N * K) > 4 * kMaxElems)
        return QLL_ERR_INVALID_ARG;
    if ((out_dtype != QLL_OUT_BF16 && out_dtype != QLL_OUT_FP32) || (!rows && R != T))
        return QLL_ERR_INVALID_ARG;
    // a tile addresses up to 256 rows, or all tokens, with 31-bit byte offsets
    if (K > kMaxRowBytes || (rows && T * K > (((int64_t)1 << 31) - 1)))
        return QLL_ERR_UNSUPPORTED;
    if (R == 0)
        return QLL_OK;
    if (!Bg || !Bu || !sg || !su || !offsets || !out || (T > 0 && (!A || !sa)))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(A, 16) || misaligned(Bg, 16) || misaligned(Bu, 16) || misaligned(out, 16) ||
        misaligned(sa, 4) || misaligned(sg, 4) || misaligned(su, 4) || misaligned(offsets, 4) ||
        misaligned(rows, 4))
        return QLL_ERR_MISALIGNED;
    GroupedArgs a = {};
    a.f.P[0] = (const uint8_t*)Bg;
    a.f.P[1] = (const uint8_t*)Bu;
    a.f.Q[0] = a.f.Q[1] = (const uint8_t*)A;
    a.f.ldp = a.f.ldq = K;
    a.f.C = (int)N;
    a.f.R = (int)R;
    a.f.klen = (int)K;
    a.f.nseg = 1;
    a.f.nks = (int)((K + 127) / 128);
    a.f.splits = 1;
    a.f.out = out;
    a.f.row_split = 0x7FFFFFFF;
    a.f.ldo = N;
    a.f.out_fp32 = out_dtype == QLL_OUT_FP32;
    a.f.act = act;
    a.f.sq = sa;
    a.f.rows = rows;
    a.f.tokens = (int)T;
    a.f.sp[0] = sg;
    a.f.sp[1] = su;
    a.offsets = offsets;
    a.E = (int)E;
    if (!moe_gated_fits(a))
        return QLL_ERR_UNSUPPORTED;
    return hip_status(launch_moe_gated(a, (hipStream_t)stream));
}

int moe_combine(const void* y, const int32_t* places, const float* weights, const void* residual,
                void* out, int out_dtype, int64_t T, int64_t R, int64_t K, int64_t topk, void* stream)
{
    const int rc = validate_combine(y, true, places, weights, out_dtype, T, R, K, topk);
    if (rc != QLL_OK || T == 0)
        return rc;
    if (!out)
        return QLL_ERR_INVALID_ARG;
    if (misaligned(residual, 16) || misaligned(out, 16))
        return QLL_ERR_MISALIGNED;
    CombineArgs a = combine_args(y, places, weights, out_dtype, T, R, K, topk);
    a.residual = residual;
    a.out = out;
    return hip_status(launch_moe_combine(a, (hipStream_t)stream));
}

int moe_combine_backward(const void* y, const int32_t* places, const float* weights, const void* dout,
                         int dout_dtype, void* dy, float* dweights, int64_t T, int64_t R, int64_t K,
                         int64_t topk, void* stream)
{
    const int rc = validate_combine(y, dweights != nullptr, places, weights, dout_dtype, T, R, K, topk);
    if (rc != QLL_OK || T == 0)
        return rc;
    if (!dout || (!dy && !dweights && R > 0) || (dweights && !weights))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(dout, 16) || misaligned(dy, 16) || misaligned(dweights, 4))
        return QLL_ERR_MISALIGNED;
    CombineArgs a = combine_args(y, places, weights, dout_dtype, T, R, K, topk);
    a.dout = dout;
    a.dy = (uint16_t*)dy;
    a.dweights = dweights;
    return hip_status(launch_moe_combine_backward(a, (hipStream_t)stream));
}

}  // extern "C"
