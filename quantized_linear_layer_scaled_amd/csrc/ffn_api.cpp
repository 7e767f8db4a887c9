// C ABI of the feed-forward operators (declared in include/qll.h): argument
// validation, workspace layout and launches.  Nothing here allocates,
// synchronizes or throws.
#include <hip/hip_runtime_api.h>

#include "../../include/qll.h"
#include "ffn_internal.h"

namespace qll {
namespace {

// (64 rows per 256-thread workgroup of a column sum stay below 2^32 threads)
constexpr int64_t kMaxDim = 0x3FFFFF00;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
// a tile addresses up to 256 rows of an operand with 31-bit byte offsets
constexpr int64_t kMaxRowBytes = (((int64_t)1 << 31) - 1) / 256;

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

int validate_sizes(int64_t M, int64_t N, int64_t K, int64_t kmul, int64_t esz, int act)
{
    if (M < 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return QLL_ERR_INVALID_ARG;
    if (M * K > kMaxElems || N * K > kMaxElems || M * N > kMaxElems)
        return QLL_ERR_INVALID_ARG;
    if (K % kmul || act < 0 || act >= ACT_COUNT)
        return QLL_ERR_INVALID_ARG;
    if (K * esz > kMaxRowBytes)
        return QLL_ERR_UNSUPPORTED;
    return QLL_OK;
}

FfnArgs blank()
{
    FfnArgs a = {};
    a.nseg = 1;
    a.splits = 1;
    a.row_split = 0x7FFFFFFF;
    return a;
}

int stages(int64_t klen, int64_t esz) { return (int)((klen * esz + 127) / 128); }

int hip_status(hipError_t e) { return e == hipSuccess ? QLL_OK : QLL_ERR_HIP; }

// Forward product: out[m][n] over K-contiguous A [M][K] and B [N][K].
void set_forward(FfnArgs& a, const void* A, const void* B0, const void* B1, int64_t M, int64_t N,
                 int64_t K, int64_t esz)
{
    a.P[0] = (const uint8_t*)B0;
    a.P[1] = (const uint8_t*)B1;
    a.Q[0] = a.Q[1] = (const uint8_t*)A;
    a.ldp = a.ldq = K * esz;
    a.C = (int)N;
    a.R = (int)M;
    a.klen = (int)K;
    a.nks = stages(K, esz);
    a.ldo = N;
}

int forward_splits(int64_t M, int64_t N, int64_t K, int64_t esz)
{
    return ffn_skinny_fits(EPI_LINEAR, M, N, K * esz) ? 1 : ffn_splits(M, N, stages(K, esz));
}

int run_linear(int fp8, const void* A, const void* B, const float* sa, const float* sb,
               const void* bias, const void* residual, int act, void* out, int out_dtype, int64_t M,
               int64_t N, int64_t K, void* ws, size_t ws_bytes, void* stream)
{
    const int64_t esz = fp8 ? 1 : 2;
    int rc = validate_sizes(M, N, K, 16 / esz, esz, act);
    if (rc != QLL_OK)
        return rc;
    if (out_dtype != QLL_OUT_BF16 && out_dtype != QLL_OUT_FP32)
        return QLL_ERR_INVALID_ARG;
    if (M == 0)
        return QLL_OK;
    if (!A || !B || !out || (fp8 && (!sa || !sb)))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(A, 16) || misaligned(B, 16) || misaligned(out, 16) || misaligned(bias, 16) ||
        misaligned(residual, 16) || misaligned(sa, 4) || misaligned(sb, 4))
        return QLL_ERR_MISALIGNED;
    FfnArgs a = blank();
    set_forward(a, A, B, B, M, N, K, esz);
    a.out = out;
    a.out_fp32 = out_dtype == QLL_OUT_FP32;
    a.act = act;
    a.sq = sa;
    a.sp[0] = sb;
    a.bias = (const uint16_t*)bias;
    a.res = (const uint16_t*)residual;
    if (ffn_skinny_fits(EPI_LINEAR, M, N, K * esz))
        return hip_status(ffn_launch_skinny(fp8, EPI_LINEAR, a, (hipStream_t)stream));
    a.splits = forward_splits(M, N, K, esz);
    if (a.splits > 1) {
        if (!ws || ws_bytes < (uint64_t)a.splits * M * N * 4)
            return QLL_ERR_WORKSPACE;
        if (misaligned(ws, 16))
            return QLL_ERR_MISALIGNED;
        a.partial = (float*)ws;
    }
    return hip_status(ffn_launch(fp8, LAY_NT, EPI_LINEAR, a, (hipStream_t)stream));
}

int run_gated(int fp8, const void* A, const void* Bg, const void* Bu, const float* sa,
              const float* sg, const float* su, int act, void* out, int out_dtype, int64_t M,
              int64_t N, int64_t K, void* stream)
{
    const int64_t esz = fp8 ? 1 : 2;
    int rc = validate_sizes(M, N, K, 16 / esz, esz, act);
    if (rc != QLL_OK)
        return rc;
    if (out_dtype != QLL_OUT_BF16 && out_dtype != QLL_OUT_FP32)
        return QLL_ERR_INVALID_ARG;
    if (M == 0)
        return QLL_OK;
    if (!A || !Bg || !Bu || !out || (fp8 && (!sa || !sg || !su)))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(A, 16) || misaligned(Bg, 16) || misaligned(Bu, 16) || misaligned(out, 16) ||
        misaligned(sa, 4) || misaligned(sg, 4) || misaligned(su, 4))
        return QLL_ERR_MISALIGNED;
    FfnArgs a = blank();
    set_forward(a, A, Bg, Bu, M, N, K, esz);
    a.out = out;
    a.out_fp32 = out_dtype == QLL_OUT_FP32;
    a.act = act;
    a.sq = sa;
    a.sp[0] = sg;
    a.sp[1] = su;
    if (ffn_skinny_fits(EPI_GATED, M, N, K * esz))
        return hip_status(ffn_launch_skinny(fp8, EPI_GATED, a, (hipStream_t)stream));
    return hip_status(ffn_launch(fp8, LAY_NT, EPI_GATED, a, (hipStream_t)stream));
}

// Workspace of a backward pass: the pre-activation gradients, the bias
// gradient's strips, then Split-K pieces (used by one product at a time).
struct BackwardPlan {
    int64_t strips = 0, pieces = 0, total = 0;  // byte offsets behind the first part, and the end
    int64_t nstrips = 0;
    int splits_in = 1, splits_w = 1;
};

BackwardPlan backward_plan(int64_t M, int64_t N, int64_t K, int act, bool bias, bool gated)
{
    BackwardPlan p;
    const int64_t width = gated ? 2 * N : N;
    const bool own_dz = gated || act != ACT_NONE;
    p.strips = own_dz ? round256(M * width * 2) : 0;
    if (bias)
        p.nstrips = own_dz ? ffn_dz_strips(M, N) : (M + kColsumRows - 1) / kColsumRows;
    p.pieces = p.strips + round256(p.nstrips * N * 4);
    p.splits_in = ffn_splits(M, K, (gated ? 2 : 1) * stages(N, 2));
    p.splits_w = ffn_splits(width, K, stages(M, 2));
    const int64_t in = p.splits_in > 1 ? (int64_t)p.splits_in * M * K * 4 : 0;
    const int64_t w = p.splits_w > 1 ? (int64_t)p.splits_w * width * K * 4 : 0;
    p.total = p.pieces + (in > w ? in : w);
    return p;
}

// dA [M][K] = dz B, over one (dz, B) or two segments side by side in dz.
FfnArgs input_gradient(const void* dz, const void* B0, const void* B1, void* dA, int64_t M,
                       int64_t N, int64_t K, int splits, float* partial)
{
    FfnArgs a = blank();
    const int nseg = B1 ? 2 : 1;
    a.nseg = nseg;
    a.P[0] = (const uint8_t*)B0;
    a.P[1] = (const uint8_t*)(B1 ? B1 : B0);
    a.ldp = K * 2;
    a.ldq = nseg * N * 2;
    a.Q[0] = (const uint8_t*)dz;
    a.Q[1] = a.Q[0] + (nseg - 1) * N * 2;
    a.C = (int)K;
    a.R = (int)M;
    a.klen = (int)N;
    a.nks = stages(N, 2);
    a.splits = splits;
    a.partial = partial;
    a.out = dA;
    a.ldo = K;
    return a;
}

// dB [width][K] = dz^T A; rows from row_split on go to dB1.
FfnArgs weight_gradient(const void* dz, const void* A, void* dB0, void* dB1, int64_t row_split,
                        int64_t M, int64_t width, int64_t K, int splits, float* partial)
{
    FfnArgs a = blank();
    a.P[0] = a.P[1] = (const uint8_t*)A;
    a.ldp = K * 2;
    a.Q[0] = a.Q[1] = (const uint8_t*)dz;
    a.ldq = width * 2;
    a.C = (int)K;
    a.R = (int)width;
    a.klen = (int)M;
    a.nks = stages(M, 2);
    a.splits = splits;
    a.partial = partial;
    a.out = dB0;
    a.out2 = dB1;
    a.row_split = (int)row_split;
    a.ldo = K;
    return a;
}

// Either gradient, or both, in one launch where that pays.
hipError_t run_gradients(const FfnArgs* in, const FfnArgs* w, hipStream_t stream)
{
    if (in && w && ffn_pair_fits(*in, *w))
        return ffn_launch_pair(*in, *w, stream);
    hipError_t e = hipSuccess;
    if (in)
        e = ffn_launch(0, LAY_NN, EPI_PLAIN, *in, stream);
    if (w && e == hipSuccess)
        e = ffn_launch(0, LAY_TN, EPI_PLAIN, *w, stream);
    return e;
}

int validate_backward(int64_t M, int64_t N, int64_t K, int act)
{
    int rc = validate_sizes(M, N, K, 8, 2, act);
    if (rc != QLL_OK)
        return rc;
    if (N % 8)
        return QLL_ERR_INVALID_ARG;
    if (N * 4 > kMaxRowBytes)
        return QLL_ERR_UNSUPPORTED;
    return QLL_OK;
}

}  // namespace
}  // namespace qll

using namespace qll;

extern "C" {

int64_t qll_epilogue_workspace_bytes(int fp8, int64_t M, int64_t N, int64_t K)
{
    const int64_t esz = fp8 ? 1 : 2;
    const int rc = validate_sizes(M, N, K, 16 / esz, esz, ACT_NONE);
    if (rc != QLL_OK)
        return -rc;
    const int s = M ? forward_splits(M, N, K, esz) : 1;
    return s > 1 ? (int64_t)s * M * N * 4 : 0;
}

int gemm_bf16_epilogue(const void* A, const void* B, const void* bias, const void* residual,
                       int act, void* out, int out_dtype, int64_t M, int64_t N, int64_t K, void* ws,
                       size_t ws_bytes, void* stream)
{
    return run_linear(0, A, B, nullptr, nullptr, bias, residual, act, out, out_dtype, M, N, K, ws,
                      ws_bytes, stream);
}

int gemm_fp8_epilogue(const void* A, const void* B, const float* sa, const float* sb,
                      const void* bias, const void* residual, int act, void* out, int out_dtype,
                      int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes, void* stream)
{
    return run_linear(1, A, B, sa, sb, bias, residual, act, out, out_dtype, M, N, K, ws, ws_bytes,
                      stream);
}

int64_t qll_epilogue_backward_workspace_bytes(int act, int has_bias, int64_t M, int64_t N, int64_t K)
{
    const int rc = validate_backward(M, N, K, act);
    return rc != QLL_OK ? -rc : backward_plan(M, N, K, act, has_bias != 0, false).total;
}

int gemm_bf16_epilogue_backward(const void* A, const void* B, const void* dout, const void* bias,
                                int act, void* dA, void* dB, float* dbias, int64_t M, int64_t N,
                                int64_t K, void* ws, size_t ws_bytes, void* stream)
{
    int rc = validate_backward(M, N, K, act);
    if (rc != QLL_OK)
        return rc;
    // (without rows dA is empty, and an empty tensor's address may be NULL)
    if (!dB && !dbias && (!dA || M == 0))
        return M == 0 ? QLL_OK : QLL_ERR_INVALID_ARG;
    if (!B || (M > 0 && (!A || !dout)))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(A, 16) || misaligned(B, 16) || misaligned(dout, 16) || misaligned(bias, 16) ||
        misaligned(dA, 16) || misaligned(dB, 16) || misaligned(dbias, 4))
        return QLL_ERR_MISALIGNED;
    const BackwardPlan p = backward_plan(M, N, K, act, dbias != nullptr, false);
    if (p.total > 0) {
        if (!ws || ws_bytes < (uint64_t)p.total)
            return QLL_ERR_WORKSPACE;
        if (misaligned(ws, 16))
            return QLL_ERR_MISALIGNED;
    }
    hipStream_t s = (hipStream_t)stream;
    uint8_t* w = (uint8_t*)ws;
    float* strips = (float*)(w + p.strips);
    float* pieces = (float*)(w + p.pieces);
    const void* dz = dout;
    if (M > 0 && act != ACT_NONE) {
        FfnArgs a = blank();
        set_forward(a, A, B, B, M, N, K, 2);
        a.out = w;
        a.act = act;
        a.bias = (const uint16_t*)bias;
        a.dy = (const uint16_t*)dout;
        a.partial = dbias ? strips : nullptr;
        if (ffn_launch(0, LAY_NT, EPI_DZ, a, s) != hipSuccess)
            return QLL_ERR_HIP;
        dz = w;
    } else if (M > 0 && dbias) {
        if (launch_colsum_strips(dout, strips, M, N, s) != hipSuccess)
            return QLL_ERR_HIP;
    }
    if (dbias) {
        const ColsumArgs c = {strips, (int)p.nstrips, (int)N, {dbias, nullptr, nullptr}};
        if (launch_colsum_finish(c, 1, s) != hipSuccess)
            return QLL_ERR_HIP;
    }
    const FfnArgs in = input_gradient(dz, B, nullptr, dA, M, N, K, p.splits_in, pieces);
    const FfnArgs wt = weight_gradient(dz, A, dB, nullptr, 0x7FFFFFFF, M, N, K, p.splits_w, pieces);
    return hip_status(run_gradients(dA && M > 0 ? &in : nullptr, dB ? &wt : nullptr, s));
}

int gated_bf16(const void* A, const void* Bg, const void* Bu, int act, void* out, int out_dtype,
               int64_t M, int64_t N, int64_t K, void* stream)
{
    return run_gated(0, A, Bg, Bu, nullptr, nullptr, nullptr, act, out, out_dtype, M, N, K, stream);
}

int gated_fp8(const void* A, const void* Bg, const void* Bu, const float* sa, const float* sg,
              const float* su, int act, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
              void* stream)
{
    return run_gated(1, A, Bg, Bu, sa, sg, su, act, out, out_dtype, M, N, K, stream);
}

int64_t qll_gated_backward_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    const int rc = validate_backward(M, N, K, ACT_NONE);
    return rc != QLL_OK ? -rc : backward_plan(M, N, K, ACT_NONE, false, true).total;
}

int gated_bf16_backward(const void* A, const void* Bg, const void* Bu, const void* dout, int act,
                        void* dA, void* dBg, void* dBu, int64_t M, int64_t N, int64_t K, void* ws,
                        size_t ws_bytes, void* stream)
{
    int rc = validate_backward(M, N, K, act);
    if (rc != QLL_OK)
        return rc;
    if ((dBg == nullptr) != (dBu == nullptr))
        return QLL_ERR_INVALID_ARG;
    if (!dBg && (!dA || M == 0))
        return M == 0 ? QLL_OK : QLL_ERR_INVALID_ARG;
    if (!Bg || !Bu || (M > 0 && (!A || !dout)))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(A, 16) || misaligned(Bg, 16) || misaligned(Bu, 16) || misaligned(dout, 16) ||
        misaligned(dA, 16) || misaligned(dBg, 16) || misaligned(dBu, 16))
        return QLL_ERR_MISALIGNED;
    const BackwardPlan p = backward_plan(M, N, K, act, false, true);
    if (p.total > 0) {
        if (!ws || ws_bytes < (uint64_t)p.total)
            return QLL_ERR_WORKSPACE;
        if (misaligned(ws, 16))
            return QLL_ERR_MISALIGNED;
    }
    hipStream_t s = (hipStream_t)stream;
    uint8_t* w = (uint8_t*)ws;
    float* pieces = (float*)(w + p.pieces);
    if (M > 0) {
        FfnArgs a = blank();
        set_forward(a, A, Bg, Bu, M, N, K, 2);
        a.out = w;
        a.ldo = 2 * N;
        a.act = act;
        a.dy = (const uint16_t*)dout;
        if (ffn_launch(0, LAY_NT, EPI_DGATED, a, s) != hipSuccess)
            return QLL_ERR_HIP;
    }
    const FfnArgs in = input_gradient(w, Bg, Bu, dA, M, N, K, p.splits_in, pieces);
    const FfnArgs wt = weight_gradient(w, A, dBg, dBu, N, M, 2 * N, K, p.splits_w, pieces);
    return hip_status(run_gradients(dA && M > 0 ? &in : nullptr, dBg ? &wt : nullptr, s));
}

namespace {

int validate_norm(const void* y, const void* r, int r_dtype, const void* w_post, const void* gate,
                  const void* w_pre, float alpha, float eps, int64_t M, int64_t K)
{
    if (M < 0 || K <= 0 || K % 8 || M > kMaxDim || K > kMaxDim || M * K > kMaxElems)
        return QLL_ERR_INVALID_ARG;
    if (r_dtype != QLL_OUT_BF16 && r_dtype != QLL_OUT_FP32)
        return QLL_ERR_INVALID_ARG;
    if (!(eps >= 0.0f))
        return QLL_ERR_INVALID_ARG;
    if (K > kNormMaxK)
        return QLL_ERR_UNSUPPORTED;
    if (!w_pre || (M > 0 && !r))
        return QLL_ERR_INVALID_ARG;
    // without a block output there is nothing to norm, gate or scale
    if (!y && M > 0 && (w_post || gate || alpha != 1.0f))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(y, 16) || misaligned(r, 16) || misaligned(w_post, 16) || misaligned(gate, 16) ||
        misaligned(w_pre, 16))
        return QLL_ERR_MISALIGNED;
    return QLL_OK;
}

NormArgs norm_args(const void* y, const void* r, int r_dtype, const void* w_post, const void* gate,
                   const void* w_pre, float alpha, float beta, float eps, int64_t M, int64_t K)
{
    NormArgs a = {};
    a.y = (const uint16_t*)y;
    a.r = r;
    a.w_post = (const uint16_t*)w_post;
    a.gate = (const uint16_t*)gate;
    a.w_pre = (const uint16_t*)w_pre;
    a.alpha = alpha;
    a.beta = beta;
    a.eps = eps;
    a.M = (int)M;
    a.K = (int)K;
    a.r_fp32 = r_dtype == QLL_OUT_FP32;
    return a;
}

}  // namespace

int residual_norm(const void* y, const void* r, int r_dtype, const void* w_post, const void* gate,
                  const void* w_pre, float alpha, float beta, float eps, void* r_out, void* n_out,
                  float* n_scales, int64_t M, int64_t K, void* stream)
{
    const int rc = validate_norm(y, r, r_dtype, w_post, gate, w_pre, alpha, eps, M, K);
    if (rc != QLL_OK)
        return rc;
    if (n_scales && K % 16)
        return QLL_ERR_INVALID_ARG;
    if (M == 0)
        return QLL_OK;
    if (!n_out || (y != nullptr) != (r_out != nullptr))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(r_out, 16) || misaligned(n_out, 16) || misaligned(n_scales, 4))
        return QLL_ERR_MISALIGNED;
    NormArgs a = norm_args(y, r, r_dtype, w_post, gate, w_pre, alpha, beta, eps, M, K);
    a.r_out = r_out;
    a.n_out = n_out;
    a.n_scales = n_scales;
    a.quant = n_scales != nullptr;
    return hip_status(launch_residual_norm(a, (hipStream_t)stream));
}

int64_t qll_residual_norm_backward_workspace_bytes(int64_t M, int64_t K)
{
    if (M < 0 || K <= 0 || K % 8 || M > kMaxDim || K > kMaxDim || M * K > kMaxElems)
        return -QLL_ERR_INVALID_ARG;
    if (K > kNormMaxK)
        return -QLL_ERR_UNSUPPORTED;
    return ((int64_t)3 * norm_backward_blocks(M, K) * K + norm_backward_stats(M, K)) * 4;
}

int residual_norm_backward(const void* y, const void* r, int r_dtype, const void* w_post,
                           const void* gate, const void* w_pre, float alpha, float beta, float eps,
                           const void* dn, const void* dr_out, void* dy, void* dr, float* dw_post,
                           float* dgate, float* dw_pre, int64_t M, int64_t K, void* ws,
                           size_t ws_bytes, void* stream)
{
    const int rc = validate_norm(y, r, r_dtype, w_post, gate, w_pre, alpha, eps, M, K);
    if (rc != QLL_OK)
        return rc;
    if (!dw_pre || (w_post != nullptr) != (dw_post != nullptr) ||
        (gate != nullptr) != (dgate != nullptr))
        return QLL_ERR_INVALID_ARG;
    if (M > 0 && (!dn || !dr || (y != nullptr) != (dy != nullptr)))
        return QLL_ERR_INVALID_ARG;
    if (misaligned(dn, 16) || misaligned(dr_out, 16) || misaligned(dy, 16) || misaligned(dr, 16) ||
        misaligned(dw_post, 4) || misaligned(dgate, 4) || misaligned(dw_pre, 4))
        return QLL_ERR_MISALIGNED;
    const int blocks = norm_backward_blocks(M, K);
    if (M > 0) {
        if (!ws || ws_bytes < ((uint64_t)3 * blocks * K + norm_backward_stats(M, K)) * 4)
            return QLL_ERR_WORKSPACE;
        if (misaligned(ws, 16))
            return QLL_ERR_MISALIGNED;
    }
    NormArgs a = norm_args(y, r, r_dtype, w_post, gate, w_pre, alpha, beta, eps, M, K);
    a.dn = (const uint16_t*)dn;
    a.dr_out = dr_out;
    a.dy = (uint16_t*)dy;
    a.dr = dr;
    a.partial = (float*)ws;
    a.stats = a.partial + (size_t)3 * blocks * K;
    if (M > 0 && launch_residual_norm_backward(a, (hipStream_t)stream) != hipSuccess)
        return QLL_ERR_HIP;
    const ColsumArgs c = {a.partial, blocks, (int)K, {dw_pre, dw_post, dgate}};
    return hip_status(launch_colsum_finish(c, 3, (hipStream_t)stream));
}

}  // extern "C"
