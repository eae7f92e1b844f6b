// C ABI of the operators around the mixer (short convolution, state space scan, RMS norm):
// argument validation and dispatch. Nothing here allocates, frees or synchronises.
#include <math.h>

#include "kda_layer.h"

namespace {

using kda::set_error;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
template <typename... P> bool all_aligned16(P... p) { return (aligned(p, 16) && ...); }

bool is_dtype(int d) { return d == KDA_BF16 || d == KDA_F32; }

int launched(hipError_t err) {
    if (err == hipErrorInvalidConfiguration) return set_error(KDA_ERR_SHAPE, "grid too large");
    if (err != hipSuccess) return set_error(KDA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(err));
    return KDA_OK;
}

int check_sequences(const int32_t* cu, int N, int B, int T) {
    if (B < 0 || T < 0 || N < 0)
        return set_error(KDA_ERR_SHAPE, "sizes must be non-negative: B=%d T=%d N=%d", B, T, N);
    if (cu) {
        if (B != 1) return set_error(KDA_ERR_SHAPE, "packed sequences (cu_seqlens given) need B == 1, got B=%d", B);
    } else if (N != B) {
        return set_error(KDA_ERR_SHAPE, "without cu_seqlens N must equal B (N=%d, B=%d)", N, B);
    }
    if ((long long)B * T > 0x7fffffffLL)
        return set_error(KDA_ERR_SHAPE, "B*T=%lld exceeds 2^31-1 rows", (long long)B * T);
    return KDA_OK;
}

int check_stride(const char* name, long long stride, long long width, long long most = 1LL << 31) {
    if (stride < width)
        return set_error(KDA_ERR_SHAPE, "%s=%lld is less than a row's %lld elements", name, stride, width);
    if (stride > most)
        return set_error(KDA_ERR_SHAPE, "%s=%lld exceeds %lld", name, stride, most);
    return KDA_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need, uintptr_t align) {
    if (need == 0) return KDA_OK;
    if (!workspace) return set_error(KDA_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (bytes < need) return set_error(KDA_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", bytes, need);
    if (!aligned(workspace, align))
        return set_error(KDA_ERR_WORKSPACE, "workspace must be %d-byte aligned", (int)align);
    return KDA_OK;
}

int conv_args(kda::ConvArgs* a, const void* x, long long x_stride, const void* weight, const void* bias,
              const void* initial_state, const int32_t* cu_seqlens, int N, int B, int T, int D, int W, int dtype,
              int w_dtype, int activation, int32_t* dev_status, hipStream_t stream) {
    set_error(KDA_OK, "%s", "");
    if (!is_dtype(dtype) || !is_dtype(w_dtype))
        return set_error(KDA_ERR_DTYPE, "dtype and w_dtype must be KDA_BF16 (1) or KDA_F32 (0), got %d and %d", dtype, w_dtype);
    if (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU)
        return set_error(KDA_ERR_ARG, "activation must be KDA_ACT_NONE (0) or KDA_ACT_SILU (1), got %d", activation);
    if (int rc = check_sequences(cu_seqlens, N, B, T)) return rc;
    if (D <= 0 || D > (1 << 28)) return set_error(KDA_ERR_SHAPE, "D must be in 1 .. 2^28, got %d", D);
    if (W < 2 || W > 4) return set_error(KDA_ERR_UNSUPPORTED, "W must be 2, 3 or 4, got %d", W);
    if (int rc = check_stride("x_stride", x_stride, D)) return rc;
    if (N > 0 && !weight) return set_error(KDA_ERR_NULL, "weight must be non-NULL");
    if ((long long)B * T > 0 && !x) return set_error(KDA_ERR_NULL, "x must be non-NULL");
    a->x = x; a->x_stride = x_stride; a->weight = weight; a->bias = bias;
    a->initial_state = initial_state; a->cu_seqlens = cu_seqlens;
    a->y = nullptr; a->final_state = nullptr;
    a->N = N; a->B = B; a->T = T; a->D = D; a->W = W;
    a->dtype = dtype; a->w_dtype = w_dtype; a->silu = activation == KDA_ACT_SILU;
    a->wide = kda::rows_of_16_bytes(dtype, D, x_stride) && all_aligned16(x, initial_state, weight, bias);
    a->dev_status = dev_status; a->stream = stream;
    return KDA_OK;
}

size_t conv_bwd_need(int B, int T, int D, int W, int N, bool packed) {
    return (size_t)kda::conv_bwd_partials(B, T, D, N, packed) * (size_t)(W + 1) * (size_t)D * sizeof(float);
}

// positions are counted in int a chunk ahead (rows of 128 bytes and more for each of b and c: no
// card holds that many)
constexpr int SSM_MAX_ROWS = 0x7fffffff - 64;

int ssm_args(kda::SsmArgs* a, const void* x, long long x_stride, const void* dt, long long dt_stride,
             const float* A_log, const void* b, long long b_stride, const void* c, long long c_stride, const float* D,
             const float* dt_bias, const float* initial_state, const int32_t* cu_seqlens, int N, void* y,
             float* final_state, int B, int T, int H, int HV, int K, int V, int dtype, int dt_dtype, int dt_softplus,
             int32_t* dev_status, hipStream_t stream) {
    set_error(KDA_OK, "%s", "");
    if (!is_dtype(dtype) || !is_dtype(dt_dtype))
        return set_error(KDA_ERR_DTYPE, "dtype and dt_dtype must be KDA_BF16 (1) or KDA_F32 (0), got %d and %d", dtype, dt_dtype);
    if (int rc = check_sequences(cu_seqlens, N, B, T)) return rc;
    if ((long long)B * T > SSM_MAX_ROWS)
        return set_error(KDA_ERR_SHAPE, "B*T=%lld exceeds %d rows", (long long)B * T, SSM_MAX_ROWS);
    if (H <= 0 || HV <= 0) return set_error(KDA_ERR_SHAPE, "H and HV must be positive: H=%d HV=%d", H, HV);
    if (HV % H != 0) return set_error(KDA_ERR_SHAPE, "HV=%d must be a multiple of H=%d", HV, H);
    if (K != 64 && K != 128) return set_error(KDA_ERR_UNSUPPORTED, "K must be 64 or 128, got %d", K);
    if (V <= 0 || V % 64 != 0) return set_error(KDA_ERR_UNSUPPORTED, "V must be a multiple of 64, got %d", V);
    if ((long long)HV * V >= (1LL << 24) || (long long)HV * K >= (1LL << 24))
        return set_error(KDA_ERR_SHAPE, "a row of HV=%d heads of K=%d, V=%d is too wide", HV, K, V);
    if ((long long)N * HV > 0x7fffffffLL / (V / 32))
        return set_error(KDA_ERR_SHAPE, "N*HV=%lld too large", (long long)N * HV);
    if (int rc = check_stride("x_stride", x_stride, (long long)HV * V, (1 << 24) - 1)) return rc;
    if (int rc = check_stride("dt_stride", dt_stride, HV, (1 << 24) - 1)) return rc;
    if (int rc = check_stride("b_stride", b_stride, (long long)H * K, (1 << 24) - 1)) return rc;
    if (int rc = check_stride("c_stride", c_stride, (long long)H * K, (1 << 24) - 1)) return rc;
    const int vec = dtype == KDA_BF16 ? 8 : 4;
    if (x_stride % vec || b_stride % vec || c_stride % vec)
        return set_error(KDA_ERR_SHAPE, "x_stride, b_stride and c_stride must be multiples of %d (16 bytes)", vec);
    if ((long long)B * T > 0 && (!x || !dt || !b || !c || !y))
        return set_error(KDA_ERR_NULL, "x, dt, b, c and y must be non-NULL");
    if (N > 0 && !A_log) return set_error(KDA_ERR_NULL, "A_log must be non-NULL");
    if (!all_aligned16(x, b, c, y, initial_state, final_state))
        return set_error(KDA_ERR_SHAPE, "x, b, c, y and the states must be 16-byte aligned");
    a->x = x; a->dt = dt; a->A_log = A_log; a->b = b; a->c = c; a->D = D; a->dt_bias = dt_bias;
    a->initial_state = initial_state; a->cu_seqlens = cu_seqlens; a->y = y; a->final_state = final_state;
    a->N = N; a->B = B; a->T = T; a->H = H; a->HV = HV; a->K = K; a->V = V;
    a->x_stride = x_stride; a->dt_stride = dt_stride; a->b_stride = b_stride; a->c_stride = c_stride;
    a->dtype = dtype; a->dt_dtype = dt_dtype; a->softplus = dt_softplus != 0;
    a->workspace = nullptr; a->dev_status = dev_status; a->stream = stream;
    return KDA_OK;
}

int norm_fwd(const void* x, long long x_stride, const void* weight, const void* residual, void* y, float* scales,
             void* h, float* rstd, long long rows, int D, int group, float eps, int dtype, int w_dtype,
             hipStream_t stream) {
    set_error(KDA_OK, "%s", "");
    const bool quant = group != 0;
    if (!is_dtype(dtype) || !is_dtype(w_dtype))
        return set_error(KDA_ERR_DTYPE, "dtype and w_dtype must be KDA_BF16 (1) or KDA_F32 (0), got %d and %d", dtype, w_dtype);
    if (rows < 0 || rows > 0x7fffffffLL) return set_error(KDA_ERR_SHAPE, "rows must be in 0 .. 2^31-1, got %lld", rows);
    if (D <= 0) return set_error(KDA_ERR_SHAPE, "D must be positive, got %d", D);
    if (!(eps >= 0.0f) || !isfinite(eps)) return set_error(KDA_ERR_ARG, "eps must be finite and not negative, got %g", (double)eps);
    if (int rc = check_stride("x_stride", x_stride, D)) return rc;
    const bool wide = kda::rows_of_16_bytes(dtype, D, x_stride) && all_aligned16(x, weight, residual, y, h);
    if (D > kda::norm_max_width(wide, dtype))
        return set_error(KDA_ERR_UNSUPPORTED, "D must be at most %d%s, got %d", kda::norm_max_width(wide, dtype),
                         wide ? "" : " where rows are not whole aligned 16-byte pieces", D);
    if (quant && group != D && group != 128)
        return set_error(KDA_ERR_UNSUPPORTED, "group must be D=%d or 128, got %d", D, group);
    if (quant && group != D && (D % 128 != 0 || !wide))
        return set_error(KDA_ERR_UNSUPPORTED, "scales for 128 columns need D a multiple of 128 (got %d) and 16-byte aligned rows", D);
    if (rows == 0) return KDA_OK;
    if (!x || !weight || !y) return set_error(KDA_ERR_NULL, "x, weight and the output must be non-NULL");
    if (quant && !scales) return set_error(KDA_ERR_NULL, "scales must be non-NULL");
    kda::NormArgs a;
    a.x = x; a.x_stride = x_stride; a.weight = weight; a.residual = residual; a.y = y;
    a.scales = quant ? scales : nullptr; a.h = h; a.rstd = rstd; a.rows = rows; a.D = D; a.group = group;
    a.dtype = dtype; a.w_dtype = w_dtype; a.wide = wide; a.eps = eps; a.stream = stream;
    return launched(kda::launch_rmsnorm_fwd(a));
}

}  // namespace

extern "C" {

int kda_conv_fwd(const void* x, long long x_stride, const void* weight, const void* bias, const void* initial_state,
                 const int32_t* cu_seqlens, int N, void* y, void* final_state, int B, int T, int D, int W, int dtype,
                 int w_dtype, int activation, int32_t* dev_status, hipStream_t stream) {
    kda::ConvArgs a;
    if (int rc = conv_args(&a, x, x_stride, weight, bias, initial_state, cu_seqlens, N, B, T, D, W, dtype, w_dtype,
                           activation, dev_status, stream))
        return rc;
    if ((long long)B * T > 0 && !y) return set_error(KDA_ERR_NULL, "y must be non-NULL");
    if (N == 0) return KDA_OK;
    a.y = y; a.final_state = final_state;
    a.wide = a.wide && all_aligned16(y, final_state);
    return launched(kda::launch_conv_fwd(a));
}

size_t kda_conv_bwd_workspace_bytes(int B, int T, int D, int W, int N, int packed, int dtype) {
    if (B < 0 || T < 0 || N < 0 || D <= 0 || D > (1 << 28) || W < 2 || W > 4 || !is_dtype(dtype)) return 0;
    return conv_bwd_need(B, T, D, W, packed ? N : B, packed != 0);
}

int kda_conv_bwd(const void* dy, const void* x, long long x_stride, const void* weight, const void* bias,
                 const void* initial_state, const int32_t* cu_seqlens, int N, const void* dfinal, void* dx,
                 float* dweight, float* dbias, void* dinitial, int B, int T, int D, int W, int dtype, int w_dtype,
                 int activation, void* workspace, size_t workspace_bytes, int32_t* dev_status, hipStream_t stream) {
    kda::ConvBwdArgs b;
    if (int rc = conv_args(&b.f, x, x_stride, weight, bias, initial_state, cu_seqlens, N, B, T, D, W, dtype, w_dtype,
                           activation, dev_status, stream))
        return rc;
    if ((long long)B * T > 0 && (!dy || !dx)) return set_error(KDA_ERR_NULL, "dy and dx must be non-NULL");
    if (!dweight || !weight) return set_error(KDA_ERR_NULL, "weight and dweight must be non-NULL");
    if (int rc = check_workspace(workspace, workspace_bytes, conv_bwd_need(B, T, D, W, N, cu_seqlens != nullptr), 16))
        return rc;
    b.dy = dy; b.dfinal = dfinal; b.dx = dx; b.dweight = dweight; b.dbias = dbias; b.dinitial = dinitial;
    b.partial = static_cast<float*>(workspace);
    b.f.wide = b.f.wide && all_aligned16(dy, dfinal, dx, dinitial);
    return launched(kda::launch_conv_bwd(b));
}

size_t kda_ssm_chunk_fwd_workspace_bytes(int B, int T, int H, int HV, int K, int V, int N, int packed, int dtype) {
    if (B < 0 || T < 0 || H <= 0 || HV <= 0 || N < 0 || HV % H != 0 || (K != 64 && K != 128) || V <= 0 || V % 64 != 0 ||
        !is_dtype(dtype) || (long long)B * T > SSM_MAX_ROWS)
        return 0;
    return kda::ssm_chunk_workspace(B, T, H, HV, K, V, packed ? N : B, packed != 0, dtype);
}

int kda_ssm_chunk_fwd(const void* x, long long x_stride, const void* dt, long long dt_stride, const float* A_log,
                      const void* b, long long b_stride, const void* c, long long c_stride, const float* D,
                      const float* dt_bias, const float* initial_state, const int32_t* cu_seqlens, int N, void* y,
                      float* final_state, int B, int T, int H, int HV, int K, int V, int dtype, int dt_dtype,
                      int dt_softplus, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                      hipStream_t stream) {
    kda::SsmArgs a;
    if (int rc = ssm_args(&a, x, x_stride, dt, dt_stride, A_log, b, b_stride, c, c_stride, D, dt_bias, initial_state,
                          cu_seqlens, N, y, final_state, B, T, H, HV, K, V, dtype, dt_dtype, dt_softplus, dev_status,
                          stream))
        return rc;
    if (N == 0) return KDA_OK;
    const size_t need = kda::ssm_chunk_workspace(B, T, H, HV, K, V, N, cu_seqlens != nullptr, dtype);
    if (int rc = check_workspace(workspace, workspace_bytes, need, 256)) return rc;
    a.workspace = workspace;
    return launched(kda::launch_ssm_chunk(a));
}

int kda_ssm_recurrent_fwd(const void* x, long long x_stride, const void* dt, long long dt_stride, const float* A_log,
                          const void* b, long long b_stride, const void* c, long long c_stride, const float* D,
                          const float* dt_bias, const float* initial_state, const int32_t* cu_seqlens, int N, void* y,
                          float* final_state, int B, int T, int H, int HV, int K, int V, int dtype, int dt_dtype,
                          int dt_softplus, int32_t* dev_status, hipStream_t stream) {
    kda::SsmArgs a;
    if (int rc = ssm_args(&a, x, x_stride, dt, dt_stride, A_log, b, b_stride, c, c_stride, D, dt_bias, initial_state,
                          cu_seqlens, N, y, final_state, B, T, H, HV, K, V, dtype, dt_dtype, dt_softplus, dev_status,
                          stream))
        return rc;
    if (N == 0) return KDA_OK;
    return launched(kda::launch_ssm_recurrent(a));
}

int kda_rmsnorm_fwd(const void* x, long long x_stride, const void* weight, const void* residual, void* y, void* h,
                    float* rstd, long long rows, int D, float eps, int dtype, int w_dtype, hipStream_t stream) {
    return norm_fwd(x, x_stride, weight, residual, y, nullptr, h, rstd, rows, D, 0, eps, dtype, w_dtype, stream);
}

int kda_rmsnorm_quant_fwd(const void* x, long long x_stride, const void* weight, const void* residual, uint8_t* q,
                          float* scales, void* h, long long rows, int D, int group, float eps, int dtype, int w_dtype,
                          hipStream_t stream) {
    if (group == 0) return set_error(KDA_ERR_UNSUPPORTED, "group must be D=%d or 128, got 0", D);
    return norm_fwd(x, x_stride, weight, residual, q, scales, h, nullptr, rows, D, group, eps, dtype, w_dtype, stream);
}

size_t kda_rmsnorm_bwd_workspace_bytes(long long rows, int D, int dtype) {
    if (rows < 0 || rows > 0x7fffffffLL || D <= 0 || !is_dtype(dtype) || D > kda::norm_max_width(true, dtype)) return 0;
    return (size_t)kda::norm_bwd_partials(rows, D, dtype) * (size_t)D * sizeof(float);
}

int kda_rmsnorm_bwd(const void* dy, const void* h, const void* weight, const float* rstd, const void* dh, void* dx,
                    float* dweight, long long rows, int D, int dtype, int w_dtype, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
    set_error(KDA_OK, "%s", "");
    if (!is_dtype(dtype) || !is_dtype(w_dtype))
        return set_error(KDA_ERR_DTYPE, "dtype and w_dtype must be KDA_BF16 (1) or KDA_F32 (0), got %d and %d", dtype, w_dtype);
    if (rows < 0 || rows > 0x7fffffffLL) return set_error(KDA_ERR_SHAPE, "rows must be in 0 .. 2^31-1, got %lld", rows);
    if (D <= 0) return set_error(KDA_ERR_SHAPE, "D must be positive, got %d", D);
    const bool wide = kda::rows_of_16_bytes(dtype, D, D) && all_aligned16(dy, h, weight, dh, dx);
    if (D > kda::norm_max_width(wide, dtype))
        return set_error(KDA_ERR_UNSUPPORTED, "D must be at most %d%s, got %d", kda::norm_max_width(wide, dtype),
                         wide ? "" : " where rows are not whole aligned 16-byte pieces", D);
    if (!weight || !dweight) return set_error(KDA_ERR_NULL, "weight and dweight must be non-NULL");
    if (rows > 0 && (!dy || !h || !rstd || !dx)) return set_error(KDA_ERR_NULL, "dy, h, rstd and dx must be non-NULL");
    if (int rc = check_workspace(workspace, workspace_bytes,
                                 (size_t)kda::norm_bwd_partials(rows, D, dtype) * (size_t)D * sizeof(float), 16))
        return rc;
    kda::NormBwdArgs a;
    a.dy = dy; a.h = h; a.weight = weight; a.rstd = rstd; a.dh = dh; a.dx = dx; a.dweight = dweight;
    a.partial = static_cast<float*>(workspace); a.rows = rows; a.D = D; a.dtype = dtype; a.w_dtype = w_dtype;
    a.wide = wide; a.stream = stream;
    return launched(kda::launch_rmsnorm_bwd(a));
}

}  // extern "C"
