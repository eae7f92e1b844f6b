// Per-token selective state space recurrence (decode and token-by-token prefill) for
// gfx950. Per sequence and head, S fp32 [K, V]:
//     dt' = softplus(dt + dt_bias),  S <- e^(-exp(A_log) dt') S + b (dt' x)^T,
//     y = S^T c + D x
// -- the delta rule's recurrence with one decay per head and no erase. The state's layout,
// the work decomposition (one wave per sequence, head and BV-column slice, its state in
// registers) and the rule for BV are those of the delta rule's kernel: a step of one token
// is a pure stream of states, 2 x 4 K V bytes a head against 4 K V flops: 1024 sequences x 32
// heads, K = V = 128, 0.73 ms (5.9 TB/s).
#include "kda_layer.h"
#include "kda_state_rows.h"

namespace kda {

namespace {

template <int K, int BV, typename TIn>
__global__ __launch_bounds__(256) void ssm_recurrent_kernel(const SsmArgs a, int nvt, long long n_items) {
    constexpr int CG = BV / 4;   // column groups: lanes along the wave's BV columns
    constexpr int RG = 64 / CG;  // row groups: lanes along K
    constexpr int R = K / RG;    // rows per lane
    const int lane = threadIdx.x & 63;
    const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (item >= n_items) return;
    const int vt = (int)(item % nvt);
    const long long chain = item / nvt;
    const int hv = (int)(chain % a.HV);
    const int n = (int)(chain / a.HV);
    const int h = hv / (a.HV / a.H);
    const int cg = lane % CG;
    const int rg = lane / CG;
    const int c0 = vt * BV + 4 * cg;

    long long row0;
    int bos, eos;
    if (a.cu_seqlens) {
        bos = a.cu_seqlens[n];
        eos = a.cu_seqlens[n + 1];
        const bool ok = bos >= 0 && bos <= eos && eos <= a.T && (n != 0 || bos == 0);
        if (!ok) {
            if (lane == 0 && a.dev_status) atomicOr(a.dev_status, KDA_DEV_BAD_CU_SEQLENS);
            return;
        }
        row0 = 0;
    } else {
        bos = 0;
        eos = a.T;
        row0 = (long long)n * a.T;
    }

    const size_t sbase = ((size_t)n * a.HV + hv) * (size_t)K * a.V;
    f32x4 S[R];   // row i of the lane's block, columns c0 .. c0+3
    if (a.initial_state) {
        load_state<RG, R, false>(a.initial_state + sbase, K, a.V, rg, c0, S);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const double rate = ssm_rate(a.A_log[hv]);
    const float bias = a.dt_bias ? a.dt_bias[hv] : 0.f;
    const float skip = a.D ? a.D[hv] : 0.f;
    for (int t = bos; t < eos; ++t) {
        const long long r = row0 + t;
        float bb[R], cc[R], xx[4], out[4];
        load_rows<RG, R, false>(static_cast<const TIn*>(a.b) + r * a.b_stride + (size_t)h * K, rg, bb);
        load_rows<RG, R, false>(static_cast<const TIn*>(a.c) + r * a.c_stride + (size_t)h * K, rg, cc);
        load4(static_cast<const TIn*>(a.x) + r * a.x_stride + (size_t)hv * a.V + c0, xx);
        const float dt = ssm_step(load_scalar(a.dt, a.dt_dtype, r * a.dt_stride + hv), bias, a.softplus);
        const float keep = exp2_fast((float)ssm_log2_decay(dt, rate));
        float p[4] = {0.f, 0.f, 0.f, 0.f}, u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = dt * xx[j];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                S[i][j] = fmaf(bb[i], u[j], S[i][j] * keep);
                p[j] = fmaf(cc[i], S[i][j], p[j]);
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = fmaf(skip, xx[j], sum_row_groups<CG>(p[j]));
        if (rg == 0) store4(static_cast<TIn*>(a.y) + ((size_t)r * a.HV + hv) * a.V + c0, out);
    }
    if (a.final_state) store_state<RG, R, false>(a.final_state + sbase, K, a.V, rg, c0, S);
}

template <int K, int BV, typename TIn>
hipError_t launch_v(const SsmArgs& a) {
    const int nvt = a.V / BV;
    const long long n_items = (long long)a.N * a.HV * nvt;
    if (n_items == 0) return hipSuccess;
    if (!grid_fits((n_items + 3) / 4, 256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((ssm_recurrent_kernel<K, BV, TIn>), dim3((unsigned)((n_items + 3) / 4)), dim3(256), 0,
                       a.stream, a, nvt, n_items);
    return hipGetLastError();
}

template <int K, typename TIn>
hipError_t launch_t(const SsmArgs& a) {
    // about one token per sequence: longer row runs (1024 sequences x 32 heads, K = V = 128: 732
    // us, with 32 columns 793); else half the work a wave and token (4 x 64 tokens x 8 heads: 62
    // us, with 64 columns 82; 1 x 256 x 4 heads: 218 and 298)
    return 2LL * a.B * a.T <= 3LL * a.N ? launch_v<K, 64, TIn>(a) : launch_v<K, 32, TIn>(a);
}

}  // namespace

hipError_t launch_ssm_recurrent(const SsmArgs& a) {
    if (a.dtype == KDA_BF16) return a.K == 128 ? launch_t<128, __bf16>(a) : launch_t<64, __bf16>(a);
    return a.K == 128 ? launch_t<128, float>(a) : launch_t<64, float>(a);
}

}  // namespace kda
