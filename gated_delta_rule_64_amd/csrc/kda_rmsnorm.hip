// RMS norm with the residual's addition, optionally leaving 8-bit values with scales, and
// its gradient, for gfx950:
//     h = x + residual,  r = (mean_d h^2 + eps)^(-1/2),  y = h r w
//     8 bits: s = max(max |y|, 2^-110) / 448 over a row or over 128 columns of it, and the
//     codes e4m3(y / s) (448 is the largest e4m3 value)
//     backward: dx = dh + r (w dy - h r mean_d(w dy h r)),  dw = sum over rows of dy h r
//
// One pass over the data, bound by HBM: a row stays in the registers of its threads (16
// bytes an access, NV accesses a thread) between the sum of its squares and its scaled
// store, so x, the residual and h move once. h is kept in fp32 for the norm and rounded
// only where it is stored. Since r > 0, max |y| = r max |h w|: the 8-bit form needs no
// second look at the row. The parameters are read again for every row, from L1 or L2.
//
// 8192 x 4096 bf16 rows with a residual to 8 bits: 45 us (5.2 TB/s); their gradient with the
// residual stream's 53 us (5.0 TB/s) and 5 us for the sum over the blocks' partial sums.
//
// TPR threads share a row: 16, 32 or 64 within a wave (no barrier; a wave holds 64 / TPR
// rows) or 256 or 1024 (one row a block, its waves' sums joined in LDS).
#include "kda_layer.h"

namespace kda {

namespace {

constexpr float FP8_MAX = 448.f;
constexpr float FP8_TINY = 7.70371977754894341e-34f;   // 2^-110

// sum / maximum over WIDTH neighbouring lanes (a power of two, at most 64)
template <int WIDTH> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o /= 2) v += __shfl_xor(v, o, 64);
    return v;
}
template <int WIDTH> __device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o /= 2) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

// over the TPR threads of a row; `slot` is LDS of 2 * TPR / 64 floats, alternated by `turn`
// so that one barrier a call is enough
template <int TPR, bool MAX> __device__ __forceinline__ float row_reduce(float v, float* slot, int turn) {
    if constexpr (TPR <= 64) {
        return MAX ? lanes_max<TPR>(v) : lanes_sum<TPR>(v);
    } else {
        constexpr int NW = TPR / 64;
        v = MAX ? lanes_max<64>(v) : lanes_sum<64>(v);
        float* mine = slot + (turn & 1) * NW;
        if ((threadIdx.x & 63) == 0) mine[threadIdx.x >> 6] = v;
        __syncthreads();
        v = mine[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) v = MAX ? fmaxf(v, mine[i]) : v + mine[i];
        return v;
    }
}

// VEC e4m3 codes of v / s (v r already formed)
template <int VEC> __device__ __forceinline__ void store_fp8(uint8_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        p[0] = (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v[0], 0.f, 0, false) & 0xff);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            uint32_t u = 0;
            u = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], u, false);
            u = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], u, true);
            w[i] = u;
        }
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// v / s rounded once, for many v and one s: v times the rounded 1 / s, and one step of its
// remainder (v - q s, exact in an fma) back onto it. A value near a tie of two codes takes the
// neighbour's if the product alone stands for the quotient. An infinite s gives 0 (the remainder's
// factor is taken as 0), as the division does.
struct Divisor {
    float inv, back;
    __device__ __forceinline__ explicit Divisor(float s) : inv(1.f / s), back(s < __builtin_inff() ? -s : 0.f) {}
    __device__ __forceinline__ float quotient(float v) const {
        const float q = v * inv;
        return fmaf(fmaf(back, q, v), inv, q);
    }
};

template <typename T, int VEC, int TPR, int NV, bool QUANT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_fwd_kernel(const NormArgs a) {
    constexpr int THREADS = TPR < 256 ? 256 : TPR;
    constexpr int ROWS = THREADS / TPR;
    __shared__ float slot[TPR > 64 ? 2 * TPR / 64 : 1];
    const int tid = threadIdx.x % TPR;
    const long long row = (long long)block_number() * ROWS + threadIdx.x / TPR;
    if (row >= a.rows) return;   // TPR > 64 has one row a block: its threads leave together
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = static_cast<const T*>(a.residual);
    const long long at = row * (long long)a.D;
    float h[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (i * TPR + tid) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[i][e] = 0.f;
        if (d >= a.D) continue;
        load_vec<VEC>(x + d, h[i]);
        if (res) {
            float r[VEC];
            load_vec<VEC>(res + at + d, r);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i][e] += r[e];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(h[i][e], h[i][e], ss);
    if (a.h) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (i * TPR + tid) * VEC;
            if (d < a.D) store_vec<VEC>(static_cast<T*>(a.h) + at + d, h[i]);
        }
    }
    ss = row_reduce<TPR, false>(ss, slot, 0);
    const float rstd = 1.f / sqrtf(ss / (float)a.D + a.eps);
    if (a.rstd && tid == 0) a.rstd[row] = rstd;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (i * TPR + tid) * VEC;
        if (d >= a.D) continue;
        float w[VEC];
        load_param<VEC>(a.weight, a.w_dtype, d, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[i][e] = h[i][e] * rstd * w[e];
        if constexpr (!QUANT) {
            store_vec<VEC>(static_cast<T*>(a.y) + at + d, h[i]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) top = fmaxf(top, fabsf(h[i][e]));
        }
    }
    if constexpr (QUANT) {
        uint8_t* q = static_cast<uint8_t*>(a.y) + at;
        if (a.group == a.D) {
            top = row_reduce<TPR, true>(top, slot, 1);
            const float s = fmaxf(top, FP8_TINY) / FP8_MAX;
            if (tid == 0) a.scales[row] = s;
            const Divisor by(s);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int d = (i * TPR + tid) * VEC;
                if (d >= a.D) continue;
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[i][e] = by.quotient(h[i][e]);
                store_fp8<VEC>(q + d, h[i]);
            }
        } else if constexpr (VEC > 1 && TPR * VEC >= 128) {
            // 128 columns are 128 / VEC neighbouring lanes of one access
            constexpr int GL = 128 / VEC;
            const long long per_row = a.D / 128;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int d = (i * TPR + tid) * VEC;
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) m = fmaxf(m, fabsf(h[i][e]));
                m = lanes_max<GL>(m);
                if (d >= a.D) continue;
                const float s = fmaxf(m, FP8_TINY) / FP8_MAX;
                if ((tid & (GL - 1)) == 0) a.scales[row * per_row + d / 128] = s;
                const Divisor by(s);
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[i][e] = by.quotient(h[i][e]);
                store_fp8<VEC>(q + d, h[i]);
            }
        }
    }
}

template <typename T, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_bwd_kernel(const NormBwdArgs a) {
    constexpr int THREADS = TPR < 256 ? 256 : TPR;
    constexpr int ROWS = THREADS / TPR;
    extern __shared__ float smem[];   // ROWS > 1: [ROWS][D] partial sums; then the row sums' slot
    __shared__ float slot[TPR > 64 ? 2 * TPR / 64 : 1];
    const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
    const long long step = (long long)gridDim.x * ROWS;
    int turn = 0;
    for (long long row = (long long)blockIdx.x * ROWS + sub; row < a.rows; row += step, ++turn) {
        const long long at = row * (long long)a.D;
        const float r = a.rstd[row];
        float xh[NV][VEC], g[NV][VEC];
        float c = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (i * TPR + tid) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) xh[i][e] = g[i][e] = 0.f;
            if (d >= a.D) continue;
            load_vec<VEC>(static_cast<const T*>(a.h) + at + d, xh[i]);
            load_vec<VEC>(static_cast<const T*>(a.dy) + at + d, g[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (i * TPR + tid) * VEC;
            if (d >= a.D) continue;
            float w[VEC];
            load_param<VEC>(a.weight, a.w_dtype, d, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                xh[i][e] *= r;
                dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
                g[i][e] *= w[e];
                c = fmaf(g[i][e], xh[i][e], c);
            }
        }
        c = row_reduce<TPR, false>(c, slot, turn) / (float)a.D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (i * TPR + tid) * VEC;
            if (d >= a.D) continue;
            float o[VEC];
            if (a.dh) {
                load_vec<VEC>(static_cast<const T*>(a.dh) + at + d, o);
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = fmaf(r, g[i][e] - xh[i][e] * c, o[e]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = r * (g[i][e] - xh[i][e] * c);
            }
            store_vec<VEC>(static_cast<T*>(a.dx) + at + d, o);
        }
    }
    // one row of partial sums a block
    if constexpr (ROWS > 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int d = (i * TPR + tid) * VEC + e;
                if (d < a.D) smem[(size_t)sub * a.D + d] = dw[i][e];
            }
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += THREADS) {
            float acc = 0.f;
#pragma unroll
            for (int s = 0; s < ROWS; ++s) acc += smem[(size_t)s * a.D + d];
            a.partial[(long long)blockIdx.x * a.D + d] = acc;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (i * TPR + tid) * VEC;
            if (d < a.D) store_vec<VEC>(a.partial + (long long)blockIdx.x * a.D + d, dw[i]);
        }
    }
}

// Threads of a row and accesses of a thread for `n` accesses a row. Up to 128 both directions
// stay inside a wave. Beyond, the forward does best with four accesses a thread before it
// takes more threads (8192 x 2048 bf16: one wave of four 19 us, four waves of one 21; 4096 x
// 8192: four waves of four 36 us, sixteen of one 40; 8192 x 4096: one wave of eight 40 us, four
// of two 38), the backward, which holds three rows and the weight's sums, with as few as it
// can (the same sizes: 33 and 25 us, 59 and 44, 89 and 41). With D above 16384 the backward's
// rows do not fit its registers (scratch is used): 8192 x 8192 bf16 112 us (4.8 TB/s), 4096 x
// 16384 127 (4.2), 2048 x 32768 182 (2.9), 1024 x 65536 544 (1.0).
struct Shape { int tpr, nv; };
inline Shape shape_of(int n, int vec, bool bwd) {
    if (vec == 4 && n <= 32) return {32, 1};   // 128 fp32 columns are 32 lanes
    if (n <= 16) return {16, 1};
    if (n <= 32) return {16, 2};
    if (n <= 64) return {32, 2};
    if (n <= 128) return {64, 2};
    if (n <= 256) return bwd ? Shape{256, 1} : Shape{64, 4};
    if (n <= 512) return {256, 2};
    if (n <= 1024) return bwd ? Shape{1024, 1} : Shape{256, 4};
    if (n <= 2048 && bwd) return {1024, 2};
    if (n <= 4096) return {1024, 4};
    return {1024, 8};
}

// `go` is a struct with a call operator template <TPR, NV>
template <int VEC, bool BWD, typename F> hipError_t by_shape(const Shape& s, const F& go) {
    if (s.tpr == 16) {
        if constexpr (VEC != 4) return s.nv == 1 ? go.template operator()<16, 1>() : go.template operator()<16, 2>();
    }
    if (s.tpr == 32) {
        if constexpr (VEC == 4) { if (s.nv == 1) return go.template operator()<32, 1>(); }
        return go.template operator()<32, 2>();
    }
    if constexpr (BWD) {
        if (s.tpr == 64) return go.template operator()<64, 2>();
        if (s.tpr == 256) return s.nv == 1 ? go.template operator()<256, 1>() : go.template operator()<256, 2>();
        if (s.nv == 1) return go.template operator()<1024, 1>();
        if (s.nv == 2) return go.template operator()<1024, 2>();
    } else {
        if (s.tpr == 64) return s.nv == 2 ? go.template operator()<64, 2>() : go.template operator()<64, 4>();
        if (s.tpr == 256) return s.nv == 2 ? go.template operator()<256, 2>() : go.template operator()<256, 4>();
    }
    return s.nv == 4 ? go.template operator()<1024, 4>() : go.template operator()<1024, 8>();
}

template <typename T, int VEC, int TPR, int NV>
hipError_t fwd_n(const NormArgs& a) {
    constexpr int THREADS = TPR < 256 ? 256 : TPR, ROWS = THREADS / TPR;
    const long long blocks = (a.rows + ROWS - 1) / ROWS;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    if (a.scales) hipLaunchKernelGGL((rmsnorm_fwd_kernel<T, VEC, TPR, NV, true>), grid_of(blocks, THREADS), dim3(THREADS), 0, a.stream, a);
    else hipLaunchKernelGGL((rmsnorm_fwd_kernel<T, VEC, TPR, NV, false>), grid_of(blocks, THREADS), dim3(THREADS), 0, a.stream, a);
    return hipGetLastError();
}

template <typename T, int VEC> struct Fwd {
    const NormArgs& a;
    template <int TPR, int NV> hipError_t operator()() const { return fwd_n<T, VEC, TPR, NV>(a); }
};
template <typename T, int VEC> hipError_t fwd_v(const NormArgs& a) {
    return by_shape<VEC, false>(shape_of((a.D + VEC - 1) / VEC, VEC, false), Fwd<T, VEC>{a});
}

inline int bwd_rows_per_block(const Shape& s) { return s.tpr < 256 ? 256 / s.tpr : 1; }
inline int bwd_blocks(long long rows, const Shape& s) {
    const long long per = bwd_rows_per_block(s);
    const long long n = (rows + per - 1) / per;
    return (int)(n < 1 ? 1 : n > 1024 ? 1024 : n);
}

template <typename T, int VEC, int TPR, int NV>
hipError_t bwd_n(const NormBwdArgs& a, int blocks) {
    constexpr int THREADS = TPR < 256 ? 256 : TPR, ROWS = THREADS / TPR;
    const size_t lds = ROWS > 1 ? (size_t)ROWS * a.D * sizeof(float) : 0;
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, VEC, TPR, NV>), dim3((unsigned)blocks), dim3(THREADS), lds, a.stream, a);
    return hipGetLastError();
}

template <typename T, int VEC> struct Bwd {
    const NormBwdArgs& a;
    int blocks;
    template <int TPR, int NV> hipError_t operator()() const { return bwd_n<T, VEC, TPR, NV>(a, blocks); }
};
template <typename T, int VEC> hipError_t bwd_v(const NormBwdArgs& a) {
    const Shape s = shape_of((a.D + VEC - 1) / VEC, VEC, true);
    const int blocks = bwd_blocks(a.rows, s);
    const hipError_t err = by_shape<VEC, true>(s, Bwd<T, VEC>{a, blocks});
    if (err != hipSuccess) return err;
    SumRows r;
    r.part = a.partial; r.P = blocks; r.M = a.D; r.out = a.dweight; r.out_tail = nullptr; r.D = a.D; r.taps = 1;
    return launch_sum_rows(r, a.stream);
}

}  // namespace

int norm_bwd_partials(long long rows, int D, int dtype) {
    // the scalar and the 16-byte form differ in their blocks: room for either
    const int vec = dtype == KDA_BF16 ? 8 : 4;
    const int wide = bwd_blocks(rows, shape_of((D + vec - 1) / vec, vec, true)), narrow = bwd_blocks(rows, shape_of(D, 1, true));
    return wide > narrow ? wide : narrow;
}

hipError_t launch_rmsnorm_fwd(const NormArgs& a) {
    const bool wide = a.wide;
    if (a.dtype == KDA_BF16) return wide ? fwd_v<__bf16, 8>(a) : fwd_v<__bf16, 1>(a);
    return wide ? fwd_v<float, 4>(a) : fwd_v<float, 1>(a);
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a) {
    const bool wide = a.wide;
    if (a.dtype == KDA_BF16) return wide ? bwd_v<__bf16, 8>(a) : bwd_v<__bf16, 1>(a);
    return wide ? bwd_v<float, 4>(a) : bwd_v<float, 1>(a);
}

}  // namespace kda
