// Chunked selective state space scan (prompts) for gfx950. Per sequence and head, S fp32
// [K, V], dt' and the log2 decay a as in the per-token kernel; over a chunk of 64 tokens
// with cum the running sums of a inside it:
//     M_ij = (c_i . b_j) 2^(cum_i - cum_j) dt'_j  (j <= i, else 0)
//     y_i  = sum_j M_ij x_j + 2^(cum_i) S^T c_i + D x_i
//     S   <- 2^(cum_63) S + sum_j 2^(cum_63 - cum_j) dt'_j b_j x_j^T
// All exponents are <= 0 for dt' >= 0, so nothing overflows whatever the decay.
//
// One 256-thread block owns a (sequence, head, 64-column slab of V): wave w holds columns
// 16w .. 16w+15 of the state in matrix-core accumulators (rows 16t + 4(l/16) + r of tile t,
// column l % 16) and walks the chunks in order. An accumulator tile is its own operand:
// with the contraction index taken in the order the four registers hold it, the state
// feeds S^T c, and M (formed transposed, token j down the rows) feeds M x, without passing
// through LDS or lanes; the other operand is loaded in that same order.
#include "kda_layer.h"

namespace kda {

namespace {

constexpr int C = 64;       // tokens of a chunk
constexpr int SLAB = 64;    // columns of V of a block
constexpr int PAD = 4;

// Per-chunk scalars of one head in LDS
struct Steps {
    float dt[C];
    float hi[C], lo[C];   // running sums of the log2 decay, as hi + lo
    float grow[C];        // 2^(cum_63 - cum_j) dt'_j
    float fall[C];        // 2^(cum_i)
    float all;            // 2^(cum_63)
};

// One wave: lane j takes token j of `len`. The running sums are formed in fp64: the
// exponents are differences of them.
__device__ __forceinline__ void chunk_steps(const SsmArgs& a, long long row, int len, int hv, float A_log, float bias,
                                            Steps* s) {
    const int j = threadIdx.x & 63;
    float dt = 0.f;
    double cum = 0.0;
    if (j < len) {
        dt = ssm_step(load_scalar(a.dt, a.dt_dtype, (row + j) * a.dt_stride + hv), bias, a.softplus);
        cum = ssm_log2_decay(dt, A_log);
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const double up = __shfl_up(cum, o, 64);
        if (j >= o) cum += up;
    }
    const double end = __shfl(cum, 63, 64);
    s->dt[j] = dt;
    const float hi = (float)cum;
    s->hi[j] = hi;
    s->lo[j] = (float)(cum - (double)hi);
    s->grow[j] = exp2_fast((float)(end - cum)) * dt;
    s->fall[j] = exp2_fast(hi);
    if (j == 63) s->all = exp2_fast(hi);
}

template <int K, typename TIn>
__global__ __launch_bounds__(256) void ssm_chunk_kernel(const SsmArgs a, int slabs) {
    constexpr int KT = K / 16;
    constexpr int LDB = K + PAD, LDX = SLAB + PAD;
    __shared__ float Bs[C * LDB], Cs[C * LDB], Xs[C * LDX];
    __shared__ f32x4 Ms[10 * 64];   // M^T tiles (I, J <= I) in accumulator order
    __shared__ Steps st;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    const int slab = (int)(blockIdx.x % slabs);
    const long long chain = blockIdx.x / slabs;
    const int hv = (int)(chain % a.HV), n = (int)(chain / a.HV);
    const int h = hv / (a.HV / a.H);
    long long row0;
    int len;
    if (a.cu_seqlens) {
        const int bos = a.cu_seqlens[n], eos = a.cu_seqlens[n + 1];
        if (!(bos >= 0 && bos <= eos && eos <= a.T && (n != 0 || bos == 0))) {
            if (threadIdx.x == 0 && a.dev_status) atomicOr(a.dev_status, KDA_DEV_BAD_CU_SEQLENS);
            return;
        }
        row0 = bos;
        len = eos - bos;
    } else {
        row0 = (long long)n * a.T;
        len = a.T;
    }
    const int col = slab * SLAB + 16 * wave + l16;   // this lane's column of the state
    const size_t sbase = ((size_t)n * a.HV + hv) * (size_t)K * a.V;
    f32x4 S[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[t][r] = a.initial_state ? a.initial_state[sbase + (size_t)(16 * t + 4 * g + r) * a.V + col] : 0.f;
    const float A_log = a.A_log[hv];
    const float bias = a.dt_bias ? a.dt_bias[hv] : 0.f;
    const float skip = a.D ? a.D[hv] : 0.f;

    for (int p0 = 0; p0 < len; p0 += C) {
        const int cl = len - p0 < C ? len - p0 : C;
        const long long row = row0 + p0;
        __syncthreads();   // the last chunk's readers are done
        for (int i = threadIdx.x; i < C * K / 4; i += 256) {
            const int t = i / (K / 4), k = i % (K / 4) * 4;
            float u[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
            if (t < cl) {
                load_vec<4>(static_cast<const TIn*>(a.b) + (row + t) * a.b_stride + (size_t)h * K + k, u);
                load_vec<4>(static_cast<const TIn*>(a.c) + (row + t) * a.c_stride + (size_t)h * K + k, v);
            }
            store_vec<4>(Bs + t * LDB + k, u);
            store_vec<4>(Cs + t * LDB + k, v);
        }
        for (int i = threadIdx.x; i < C * SLAB / 4; i += 256) {
            const int t = i / (SLAB / 4), p = i % (SLAB / 4) * 4;
            float u[4] = {0.f, 0.f, 0.f, 0.f};
            if (t < cl) load_vec<4>(static_cast<const TIn*>(a.x) + (row + t) * a.x_stride + (size_t)hv * a.V + slab * SLAB + p, u);
            store_vec<4>(Xs + t * LDX + p, u);
        }
        if (wave == 0) chunk_steps(a, row, cl, hv, A_log, bias, &st);
        __syncthreads();
        // M^T: wave w forms rows J <= w of token column block w
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            if (J > wave) break;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const f32x4 u = *reinterpret_cast<const f32x4*>(Bs + (16 * J + l16) * LDB + 16 * t + 4 * g);
                const f32x4 v = *reinterpret_cast<const f32x4*>(Cs + (16 * wave + l16) * LDB + 16 * t + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc = Mma<float>::mma(u[r], v[r], acc);
            }
            const int i = 16 * wave + l16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * J + 4 * g + r;
                const float e = exp2_fast((st.hi[i] - st.hi[j]) + (st.lo[i] - st.lo[j])) * st.dt[j];
                acc[r] = j <= i ? acc[r] * e : 0.f;
            }
            Ms[(wave * (wave + 1) / 2 + J) * 64 + lane] = acc;
        }
        // this wave's columns of x, token 16 J + 4 g + r in register [J][r]
        f32x4 xt[4];
#pragma unroll
        for (int J = 0; J < 4; ++J)
#pragma unroll
            for (int r = 0; r < 4; ++r) xt[J][r] = Xs[(16 * J + 4 * g + r) * LDX + 16 * wave + l16];
        __syncthreads();
#pragma unroll
        for (int I = 0; I < 4; ++I) {
            if (16 * I >= cl) break;
            const int i = 16 * I + l16;
            // S^T c, then scaled by the token's decay, then the chunk's own tokens
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(Cs + i * LDB + 16 * t + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc = Mma<float>::mma(S[t][r], v[r], acc);
            }
            const float f = st.fall[i];
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] *= f;
#pragma unroll
            for (int J = 0; J < 4; ++J) {
                if (J > I) break;
                const f32x4 m = Ms[(I * (I + 1) / 2 + J) * 64 + lane];
#pragma unroll
                for (int r = 0; r < 4; ++r) acc = Mma<float>::mma(xt[J][r], m[r], acc);
            }
            if (i < cl) {   // columns 16 wave + 4 g .. +3 of token i
                const int p = 16 * wave + 4 * g;
                float out[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) out[r] = fmaf(skip, Xs[i * LDX + p + r], acc[r]);
                store_vec<4>(static_cast<TIn*>(a.y) + ((row + i) * a.HV + hv) * (long long)a.V + slab * SLAB + p, out);
            }
        }
        // the state at the chunk's end
        const float all = st.all;
#pragma unroll
        for (int J = 0; J < 4; ++J)
#pragma unroll
            for (int r = 0; r < 4; ++r) xt[J][r] *= st.grow[16 * J + 4 * g + r];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] *= all;
#pragma unroll
            for (int J = 0; J < 4; ++J)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[t] = Mma<float>::mma(Bs[(16 * J + 4 * g + r) * LDB + 16 * t + l16], xt[J][r], S[t]);
        }
    }
    if (a.final_state) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) a.final_state[sbase + (size_t)(16 * t + 4 * g + r) * a.V + col] = S[t][r];
    }
}

template <int K, typename TIn>
hipError_t launch_k(const SsmArgs& a) {
    const int slabs = a.V / SLAB;
    const long long blocks = (long long)a.N * a.HV * slabs;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((ssm_chunk_kernel<K, TIn>), dim3((unsigned)blocks), dim3(256), 0, a.stream, a, slabs);
    return hipGetLastError();
}

}  // namespace

size_t ssm_chunk_workspace(int, int, int, int, int, int, bool, int) { return 0; }

hipError_t launch_ssm_chunk(const SsmArgs& a) {
    if (a.dtype == KDA_BF16) return a.K == 128 ? launch_k<128, __bf16>(a) : launch_k<64, __bf16>(a);
    return a.K == 128 ? launch_k<128, float>(a) : launch_k<64, float>(a);
}

}  // namespace kda
