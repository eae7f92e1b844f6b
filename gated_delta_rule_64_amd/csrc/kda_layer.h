// Launch descriptors and device helpers of the operators around the mixer: the short
// causal convolution, the selective state space scan and the RMS norm.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

struct ConvArgs {
    const void* x;
    long long x_stride;          // elements between consecutive rows (tokens) of x
    const void* weight;          // [D, W]
    const void* bias;            // [D] or NULL
    const void* initial_state;   // [N, W-1, D] or NULL (zeros), x's dtype
    const int32_t* cu_seqlens;
    void* y;                     // [B, T, D]
    void* final_state;           // [N, W-1, D] or NULL
    int N, B, T, D, W;
    int dtype, w_dtype, silu;
    bool wide;                   // rows and pointers allow 16-byte accesses
    int32_t* dev_status;
    hipStream_t stream;
};

struct ConvBwdArgs {
    ConvArgs f;                  // y, final_state unused
    const void* dy;              // [B, T, D]
    const void* dfinal;          // [N, W-1, D] or NULL
    void* dx;                    // [B, T, D]
    float* dweight;              // [D, W]
    float* dbias;                // [D] or NULL
    void* dinitial;              // [N, W-1, D] or NULL
    float* partial;              // conv_bwd_partials() x [W + 1][D]
};

struct NormArgs {
    const void* x;
    long long x_stride;
    const void* weight;
    const void* residual;        // [rows, D] or NULL
    void* y;                     // [rows, D] in x's dtype, or e4m3 codes when scales is set
    float* scales;               // [rows, D / group] or NULL (no quantisation)
    void* h;                     // [rows, D] or NULL
    float* rstd;                 // [rows] or NULL
    long long rows;
    int D, group;                // group: columns per scale (D or 128)
    int dtype, w_dtype;
    bool wide;
    float eps;
    hipStream_t stream;
};

struct NormBwdArgs {
    const void* dy;
    const void* h;
    const void* weight;
    const float* rstd;
    const void* dh;              // gradient arriving at h from the residual stream, or NULL
    void* dx;
    float* dweight;              // [D]
    float* partial;              // norm_bwd_partials() x [D]
    long long rows;
    int D, dtype, w_dtype;
    bool wide;
    hipStream_t stream;
};

struct SsmArgs {
    const void* x;               // [B, T, HV, V], rows x_stride apart
    const void* dt;              // [B, T, HV], rows dt_stride apart
    const float* A_log;          // [HV]
    const void* b;               // [B, T, H, K]
    const void* c;
    const float* D;              // [HV] or NULL
    const float* dt_bias;        // [HV] or NULL
    const float* initial_state;  // [N, HV, K, V] or NULL
    const int32_t* cu_seqlens;
    void* y;                     // [B, T, HV, V]
    float* final_state;
    int N, B, T, H, HV, K, V;
    long long x_stride, dt_stride, b_stride, c_stride;
    int dtype, dt_dtype, softplus;
    void* workspace;
    int32_t* dev_status;
    hipStream_t stream;
};

hipError_t launch_conv_fwd(const ConvArgs& a);
hipError_t launch_conv_bwd(const ConvBwdArgs& a);
long long conv_bwd_partials(int B, int T, int D, int N, bool packed);
// whether a row of D values can be moved 16 bytes at a time
inline bool rows_of_16_bytes(int dtype, int D, long long stride) {
    const int vec = dtype == KDA_BF16 ? 8 : 4;
    return D % vec == 0 && stride % vec == 0;
}
// a grid of at least `blocks` blocks (under 2^31), the further ones along y; see grid_fits
inline dim3 grid_of(long long blocks, int threads) {
    const long long most = (1LL << 31) / threads;
    return blocks <= most ? dim3((unsigned)blocks) : dim3((unsigned)most, (unsigned)((blocks + most - 1) / most));
}
// the block's number in it
__device__ __forceinline__ unsigned block_number() { return blockIdx.y * gridDim.x + blockIdx.x; }
// the widest row of the norms: rows held in registers, 1024 threads x 8 accesses
inline int norm_max_width(bool wide, int dtype) { return 8192 * (wide ? (dtype == KDA_BF16 ? 8 : 4) : 1); }
hipError_t launch_rmsnorm_fwd(const NormArgs& a);
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a);
int norm_bwd_partials(long long rows, int D, int dtype);
hipError_t launch_ssm_recurrent(const SsmArgs& a);
hipError_t launch_ssm_chunk(const SsmArgs& a);
size_t ssm_chunk_workspace(int B, int T, int H, int HV, int K, int V, int N, bool packed, int dtype);

// out[m] (or, transposed, out[(m % D) * (M / D) + m / D]) = sum over p of part[p * M + m],
// in the order of p
struct SumRows {
    const float* part;
    long long P, M;
    float* out;       // the first M - tail columns, as [D][taps] from [taps][D]
    float* out_tail;  // the last D columns, or NULL when there are none
    int D, taps;
};
hipError_t launch_sum_rows(const SumRows& s, hipStream_t stream);

// ---------------------------------------------------------------------------------
// VEC consecutive elements as fp32 (16-byte accesses for VEC = 8 bf16 / 4 fp32, 32-byte
// ones for 8 fp32; VEC = 1 has no alignment requirement)
// ---------------------------------------------------------------------------------
template <int VEC> __device__ __forceinline__ void load_vec(const __bf16* p, float (&o)[VEC]) {
    if constexpr (VEC == 8) {
        const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (float)v[e];
    } else if constexpr (VEC == 4) {
        const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (float)v[e];
    } else {
        static_assert(VEC == 1, "1, 4 or 8");
        o[0] = (float)p[0];
    }
}
template <int VEC> __device__ __forceinline__ void load_vec(const float* p, float (&o)[VEC]) {
    if constexpr (VEC == 1) {
        o[0] = p[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i + e] = v[e];
        }
    }
}
template <int VEC> __device__ __forceinline__ void store_vec(__bf16* p, const float (&o)[VEC]) {
    if constexpr (VEC == 1) p[0] = (__bf16)o[0];
    else store_run<__bf16, VEC>(p, o);
}
template <int VEC> __device__ __forceinline__ void store_vec(float* p, const float (&o)[VEC]) {
    if constexpr (VEC == 1) {
        p[0] = o[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
    }
}
// parameters in either type
template <int VEC> __device__ __forceinline__ void load_param(const void* p, int dtype, long long at, float (&o)[VEC]) {
    if (dtype == KDA_BF16) load_vec<VEC>(static_cast<const __bf16*>(p) + at, o);
    else load_vec<VEC>(static_cast<const float*>(p) + at, o);
}
__device__ __forceinline__ float load_scalar(const void* p, int dtype, long long at) {
    return dtype == KDA_BF16 ? (float)static_cast<const __bf16*>(p)[at] : static_cast<const float*>(p)[at];
}

// sigmoid in fp32: v_exp_f32 and v_rcp_f32 (about 1 ulp each); below -88 the exponential
// overflows to +inf and the result is 0
__device__ __forceinline__ float sigmoid_fast(float x) {
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(-LOG2E * x));
}

// ---------------------------------------------------------------------------------
// Tiles of a batch of sequences without a schedule: sequence n of a packed batch owns the
// tile indices from cu[n] / TT + n on. floor((a + len) / TT) - floor(a / TT) + 1 is at
// least ceil(len / TT) and at least 1, so the ranges hold every sequence's tiles (an empty
// one's single tile too), do not meet, and end below T / TT + N. Unused indices get
// len = -1. Offsets are checked here: a slot that breaks 0 = cu[0] <= cu[n] <= cu[n+1] <= T
// gets no tile and is flagged by whoever finds it.
// ---------------------------------------------------------------------------------
struct SeqTile {
    int n;            // sequence
    int pos;          // first position of the tile in its sequence
    int len;          // the sequence's length, or -1: nothing to do
    long long row0;   // row of position 0
};
__device__ __forceinline__ SeqTile seq_tile(long long tile, const int32_t* __restrict__ cu, int N, int T, int TT,
                                            int tiles_dense) {
    SeqTile s;
    s.len = -1;
    s.pos = 0;
    s.n = 0;
    s.row0 = 0;
    if (!cu) {
        s.n = (int)(tile / tiles_dense);
        if (s.n >= N) return s;
        s.pos = (int)(tile % tiles_dense) * TT;
        s.len = T;
        s.row0 = (long long)s.n * T;
        return s;
    }
    int lo = 0, hi = N;   // the last n with cu[n] / TT + n <= tile
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (cu[mid] / TT + (long long)mid <= tile) lo = mid;
        else hi = mid;
    }
    s.n = lo;
    const int bos = cu[lo], eos = cu[lo + 1];
    if (!(bos >= 0 && bos <= eos && eos <= T && (lo != 0 || bos == 0))) return s;
    const long long at = (tile - (bos / TT + (long long)lo)) * TT;
    if (at < 0 || (at >= eos - bos && at != 0)) return s;
    s.pos = (int)at;
    s.len = eos - bos;
    s.row0 = bos;
    return s;
}
// One block's threads check every slot's offsets and flag a broken one.
__device__ __forceinline__ void flag_bad_offsets(const int32_t* __restrict__ cu, int N, int T, int32_t* dev_status) {
    if (!cu || !dev_status) return;
    for (int n = threadIdx.x; n < N; n += blockDim.x) {
        const int bos = cu[n], eos = cu[n + 1];
        if (!(bos >= 0 && bos <= eos && eos <= T && (n != 0 || bos == 0))) atomicOr(dev_status, KDA_DEV_BAD_CU_SEQLENS);
    }
}

// log(1 + e^z) = max(z, 0) + log1p(e^-|z|), to about 9 half steps of fp32: with u = e^-|z| in
// (0, 1] (the exponent's rounding is carried into the result) log1p(u) = 2 atanh(t),
// t = u / (2 + u) <= 1/3, by its odd series to t^15 (the next term is under 2^-29 of it). z
// from 200 on and NaN are their own softplus. About 25 instructions, a quarter of what the
// general log1p and exp take.
__device__ __forceinline__ float softplus_f32(float z) {
    const float m = fminf(fabsf(z), 200.f);
    const float p = -m * LOG2E;
    const float e = fmaf(-m, LOG2E, -p) - m * 1.92596299112661746e-8f;   // m log2(e) beyond p
    float u = exp2_fast(p);
    u = fmaf(u, e * 0.693147180559945309f, u);
    const float d = 2.f + u;
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(fmaf(-d, r, 1.f), r, r);
    const float t = u * r, s = t * t;
    float q = fmaf(s, 1.f / 15, 1.f / 13);
    q = fmaf(s, q, 1.f / 11);
    q = fmaf(s, q, 1.f / 9);
    q = fmaf(s, q, 1.f / 7);
    q = fmaf(s, q, 1.f / 5);
    q = fmaf(s, q, 1.f / 3);
    q = fmaf(s, q, 1.f);
    return z < 200.f ? fmaf(2.f * t, q, fmaxf(z, 0.f)) : z;
}

// dt' of the scan: softplus(dt + bias), or dt + bias as it is
__device__ __forceinline__ float ssm_step(float raw, float bias, int softplus) {
    return softplus ? softplus_f32(raw + bias) : raw + bias;
}
// v, at least `least`; NaN stays NaN (fmax would drop it)
__device__ __forceinline__ double at_least(double v, double least) { return v < least ? least : v; }
// a head's log2 decay for dt' = 1 (finite, so that a step of 0 keeps the state whatever A_log),
// and the log2 decay of a step; that is bounded at -200, where its exponential is 0 all the
// same, so that sums of decays stay finite and their differences exact enough
__device__ __forceinline__ double ssm_rate(float A_log) {
    return at_least(-exp((double)A_log) * 1.4426950408889634, -1e300);
}
__device__ __forceinline__ double ssm_log2_decay(float dt, double rate) { return at_least((double)dt * rate, -200.0); }

}  // namespace kda
