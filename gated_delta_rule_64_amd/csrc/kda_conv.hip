// Short causal depthwise convolution (W = 2..4 taps), with bias and SiLU, for gfx950:
//     pre[t, d] = bias[d] + sum_i w[d, i] x[t - (W-1) + i, d],   y = pre sigmoid(pre) or pre,
// rows before a sequence's first token coming from its state (the last W - 1 rows it saw),
// and the gradients of it. The layer's q, k and v (or x, b and c) go through it side by
// side as channels, ahead of the delta rule or the state space scan.
//
// Nothing is reused but the W - 1 neighbours, so both directions are bound by HBM: x in and
// y out, or x and dy in and dx out. A lane owns 16 bytes of a row (8 bf16 or 4 fp32
// channels; one channel where rows are not whole 16-byte pieces) and walks TT rows of one
// sequence with the window of the last W - 1 rows in registers, so a row is read once, and
// the W - 1 rows before the tile once more (from L2: the neighbouring tile's lanes read
// them). A wave is 64 such lanes side by side, one contiguous run of a row per access.
// 8192 rows of 8192 bf16 channels: 52 us (5.2 TB/s); gradients of 8192 x 6144: 98 us and 5 for
// the sum over the blocks' partial sums.
#include "kda_layer.h"

namespace kda {

namespace {

// Rows are taken R (backward: RB) at a time, the next ones in flight while these are worked
// on. Backward of 2 x 4096 rows x 6144 channels: RB 2 and tiles of 64 rows 99 us, 2 and 32
// 106, 4 and 32 121, 4 and 64 140 (more rows at once take registers the waves lack).
constexpr int TT_FWD = 32;
constexpr int TT_BWD = 64;
constexpr int R = 4;
constexpr int RB = 2;
constexpr long long BWD_BLOCKS = 512;

// lanes of a block along the channels (a power of two, at most 64); the block's other lanes
// take other tiles
inline int lanes_along(int D, int vec) {
    const int n = (D + vec - 1) / vec;
    int l = 1;
    while (l < n && l < 64) l *= 2;
    return l;
}

// VEC elements of a row as they are stored
template <typename T, int VEC> struct Raw { typedef __attribute__((ext_vector_type(VEC))) T type; };
template <typename T> struct Raw<T, 1> { typedef T type; };
template <typename T, int VEC> __device__ __forceinline__ typename Raw<T, VEC>::type load_raw(const T* p) {
    return *reinterpret_cast<const typename Raw<T, VEC>::type*>(p);
}
template <typename T, int VEC> __device__ __forceinline__ void widen(const typename Raw<T, VEC>::type& v, float (&o)[VEC]) {
    if constexpr (VEC == 1) {
        o[0] = (float)v;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = (float)v[e];
    }
}

// The taps and bias of channels d .. d + VEC - 1: VEC W contiguous weights.
template <int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int d, float (&w)[W][VEC], float (&bias)[VEC]) {
    float flat[W][VEC];   // piece by piece of the [VEC][W] block
#pragma unroll
    for (int i = 0; i < W; ++i) load_param<VEC>(a.weight, a.w_dtype, (long long)d * W + i * VEC, flat[i]);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int i = 0; i < W; ++i) w[i][e] = flat[(e * W + i) / VEC][(e * W + i) % VEC];
    if (a.bias) {
        load_param<VEC>(a.bias, a.w_dtype, d, bias);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) bias[e] = 0.f;
    }
}

// row `pos` (negative: rows of the state, or zeros) of a sequence
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_row(const ConvArgs& a, const SeqTile& s, int pos, int d, float (&o)[VEC]) {
    if (pos >= 0) {
        load_vec<VEC>(static_cast<const T*>(a.x) + (s.row0 + pos) * a.x_stride + d, o);
    } else if (a.initial_state) {
        load_vec<VEC>(static_cast<const T*>(a.initial_state) + ((long long)s.n * (W - 1) + (W - 1 + pos)) * a.D + d, o);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = 0.f;
    }
}

template <typename T, int VEC, int W>
__global__ __launch_bounds__(256) void conv_fwd_kernel(const ConvArgs a, int along, int dblocks, long long tiles,
                                                       int tiles_dense) {
    const unsigned block = block_number();
    if (block == 0) flag_bad_offsets(a.cu_seqlens, a.N, a.T, a.dev_status);
    const int dv = (int)(block % dblocks) * along + (threadIdx.x & (along - 1));
    const long long tile = (long long)(block / dblocks) * (256 / along) + threadIdx.x / along;
    const int d = dv * VEC;
    if (d >= a.D || tile >= tiles) return;
    const SeqTile s = seq_tile(tile, a.cu_seqlens, a.N, a.T, TT_FWD, tiles_dense);
    if (s.len < 0) return;
    const int end = s.len - s.pos < TT_FWD ? s.len - s.pos : TT_FWD;
    const T* xp = static_cast<const T*>(a.x) + (s.row0 + s.pos) * a.x_stride + d;
    T* yp = static_cast<T*>(a.y) + (s.row0 + s.pos) * (long long)a.D + d;

    // past the tile the last row stands in
    typename Raw<T, VEC>::type cur[R], next[R];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int k = 0; k < R; ++k) next[k] = load_raw<T, VEC>(xp + (long long)min(t0 + k, end - 1) * a.x_stride);
    };
    if (end > 0) fetch(0);
    float w[W][VEC], bias[VEC], win[W - 1 + R][VEC];
    load_taps<VEC, W>(a, d, w, bias);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) load_row<T, VEC, W>(a, s, s.pos - (W - 1) + i, d, win[i]);

    // the sequence's first tile hands on the last W - 1 rows it saw: before anything is
    // written, since final_state may be initial_state, which no other tile reads
    if (s.pos == 0 && a.final_state) {
        float last[W - 1][VEC];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_row<T, VEC, W>(a, s, s.len - (W - 1) + j, d, last[j]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_vec<VEC>(static_cast<T*>(a.final_state) + ((long long)s.n * (W - 1) + j) * a.D + d, last[j]);
    }
    for (int t0 = 0; t0 < end; t0 += R) {
#pragma unroll
        for (int k = 0; k < R; ++k) cur[k] = next[k];
        if (t0 + R < end) fetch(t0 + R);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            widen<T, VEC>(cur[k], win[W - 1 + k]);
            float out[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float acc = bias[e];
#pragma unroll
                for (int i = 0; i < W; ++i) acc = fmaf(w[i][e], win[k + i][e], acc);
                out[e] = a.silu ? acc * sigmoid_fast(acc) : acc;
            }
            if (t0 + k < end) store_vec<VEC>(yp + (long long)(t0 + k) * a.D, out);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) win[i][e] = win[R + i][e];
    }
}

// The gradients. A lane walks its tile's rows and the W - 1 after them (whose dpre it forms
// again), with windows of x and of dpre: dx[t] = sum_i w[i] dpre[t + W-1-i], and while
// t is one of its own rows, dw[i] += dpre[t] x[t - (W-1) + i] and db += dpre[t] in fp32.
// The sequence's first tile also has the state's rows (positions -(W-1) .. -1).
// The block adds its tiles' sums in LDS and leaves one row of partial sums; sum_rows adds
// those in order, so results do not depend on scheduling. A lane has four channels here (8
// bytes of bf16): with eight, the two windows and the sums take 250 registers.
template <typename T, int VEC, int W>
__global__ __launch_bounds__(256) void conv_bwd_kernel(const ConvBwdArgs b, int along, int dblocks, long long tiles,
                                                       int tiles_dense, long long P) {
    const ConvArgs& a = b.f;
    extern __shared__ float sums[];   // [256 / along][W + 1][along * VEC]
    if (blockIdx.x == 0) flag_bad_offsets(a.cu_seqlens, a.N, a.T, a.dev_status);
    const int ln = threadIdx.x & (along - 1), grp = threadIdx.x / along, groups = 256 / along;
    const int d = ((int)(blockIdx.x % dblocks) * along + ln) * VEC;
    const long long p = blockIdx.x / dblocks;
    const bool live = d < a.D;
    float w[W][VEC], bias[VEC], dw[W][VEC], db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) dw[i][e] = 0.f;
    }
    if (live) load_taps<VEC, W>(a, d, w, bias);
    for (long long tile = p * groups + grp; live && tile < tiles; tile += P * groups) {
        const SeqTile s = seq_tile(tile, a.cu_seqlens, a.N, a.T, TT_BWD, tiles_dense);
        if (s.len < 0) continue;
        // rows counted from the tile's first (a sequence may be 2^31 - 1 rows long): its own
        // are 0 .. end - 1, the sequence has `rest` of them
        const int rest = s.len - s.pos;
        const int end = min(rest, TT_BWD);
        const int first = s.pos == 0 ? -(W - 1) : 0;   // rows whose gradient is written
        const T* xp = static_cast<const T*>(a.x) + (s.row0 + s.pos) * a.x_stride + d;
        const T* yp = static_cast<const T*>(b.dy) + (s.row0 + s.pos) * (long long)a.D + d;
        T* dxp = static_cast<T*>(b.dx) + (s.row0 + s.pos) * (long long)a.D + d;
        // past the sequence the last row stands in, its dpre taken as 0
        typename Raw<T, VEC>::type cx[RB], cy[RB], nx[RB], ny[RB];
        auto fetch = [&](int t0) {
#pragma unroll
            for (int k = 0; k < RB; ++k) {
                const long long t = min(t0 + k, rest - 1);
                nx[k] = load_raw<T, VEC>(xp + t * a.x_stride);
                ny[k] = load_raw<T, VEC>(yp + t * a.D);
            }
        };
        if (rest > 0) fetch(0);
        float win[W - 1 + RB][VEC], dp[W - 1 + RB][VEC];   // x and dpre, the last rows and these
#pragma unroll
        for (int i = 0; i < W - 1; ++i) load_row<T, VEC, W>(a, s, s.pos - (W - 1) + i, d, win[i]);
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) dp[i][e] = 0.f;
        for (int t0 = 0; t0 < end + W - 1; t0 += RB) {
            if (rest > 0) {
#pragma unroll
                for (int k = 0; k < RB; ++k) {
                    cx[k] = nx[k];
                    cy[k] = ny[k];
                }
                if (t0 + RB < end + W - 1) fetch(t0 + RB);
            }
#pragma unroll
            for (int k = 0; k < RB; ++k) {
                const int t = t0 + k;
                if (rest > 0) {
                    widen<T, VEC>(cx[k], win[W - 1 + k]);
                    widen<T, VEC>(cy[k], dp[W - 1 + k]);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float g = dp[W - 1 + k][e];
                    if (a.silu) {
                        float acc = bias[e];
#pragma unroll
                        for (int i = 0; i < W; ++i) acc = fmaf(w[i][e], win[k + i][e], acc);
                        const float sg = sigmoid_fast(acc);
                        g *= sg * (1.f + acc * (1.f - sg));
                    }
                    g = t < rest ? g : 0.f;
                    dp[W - 1 + k][e] = g;
                    if (t < end) {
                        db[e] += g;
#pragma unroll
                        for (int i = 0; i < W; ++i) dw[i][e] = fmaf(g, win[k + i][e], dw[i][e]);
                    }
                }
                // row t - (W-1) has every term: dpre[t - (W-1) .. t] against w[W-1 .. 0]
                const int r = t - (W - 1);
                if (r >= first && r < end) {
                    float g[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        g[e] = 0.f;
#pragma unroll
                        for (int i = 0; i < W; ++i) g[e] = fmaf(w[W - 1 - i][e], dp[k + i][e], g[e]);
                    }
                    const int j = r - (rest - (W - 1));   // the row of the final state it is handed on as
                    if (b.dfinal && j >= 0) {
                        float f[VEC];
                        load_vec<VEC>(static_cast<const T*>(b.dfinal) + ((long long)s.n * (W - 1) + j) * a.D + d, f);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) g[e] += f[e];
                    }
                    if (r >= 0)
                        store_vec<VEC>(dxp + r * (long long)a.D, g);
                    else if (b.dinitial)
                        store_vec<VEC>(static_cast<T*>(b.dinitial) + ((long long)s.n * (W - 1) + W - 1 + r) * a.D + d, g);
                }
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    win[i][e] = win[RB + i][e];
                    dp[i][e] = dp[RB + i][e];
                }
        }
    }
    const int cols = along * VEC;
    float* mine = sums + (size_t)grp * (W + 1) * cols + ln * VEC;
#pragma unroll
    for (int i = 0; i <= W; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) mine[i * cols + e] = i < W ? dw[i < W ? i : 0][e] : db[e];
    __syncthreads();
    for (int k = threadIdx.x; k < (W + 1) * cols; k += 256) {
        float acc = 0.f;
        for (int g = 0; g < groups; ++g) acc += sums[(size_t)g * (W + 1) * cols + k];
        const int i = k / cols, dd = (int)(blockIdx.x % dblocks) * cols + k % cols;
        if (dd < a.D) b.partial[(p * (W + 1) + i) * a.D + dd] = acc;
    }
}

// Sums of P rows of M partial sums: a block takes 32 columns, 32 groups of the rows each,
// and adds the groups in order.
__global__ __launch_bounds__(1024) void sum_rows_kernel(const SumRows s) {
    __shared__ float part[32][33];
    const int ln = threadIdx.x & 31, q = threadIdx.x >> 5;
    const long long m = (long long)block_number() * 32 + ln;
    float acc = 0.f;
    if (m < s.M) {
        const long long each = (s.P + 31) / 32;
        const long long p0 = q * each, p1 = p0 + each < s.P ? p0 + each : s.P;
#pragma unroll 8
        for (long long p = p0; p < p1; ++p) acc += s.part[p * s.M + m];
    }
    part[q][ln] = acc;
    __syncthreads();
    if (q != 0 || m >= s.M) return;
#pragma unroll
    for (int k = 1; k < 32; ++k) acc += part[k][ln];
    const long long row = m / s.D;
    const int d = (int)(m % s.D);
    if (row < s.taps) s.out[(long long)d * s.taps + row] = acc;
    else if (s.out_tail) s.out_tail[d] = acc;
}

// tiles of a dense sequence, one at least
inline int tiles_dense_of(int T, int TT) { return T > 0 ? (T - 1) / TT + 1 : 1; }
inline long long tiles_of(int B, int T, int N, bool packed, int TT) {
    if (N == 0) return 0;
    return packed ? (long long)T / TT + N : (long long)B * tiles_dense_of(T, TT);
}

// blocks of the backward along the channels
inline int bwd_dblocks(int D, int vec) {
    const int cols = lanes_along(D, vec) * vec;
    return (D + cols - 1) / cols;
}
// Blocks along the rows, one row of partial sums each, then even rounds of them: BWD_BLOCKS over
// all channels (two a unit), and 128 at least. 262144 rows x 256 channels, one block wide: 128
// blocks 446 us (half the units idle, and a lane's sums four times as long), 512 154, 1024 167;
// 65536 x 1024 (four wide) 162, 163 and 173; 8192 x 6144 (24 wide) 103 for each.
inline long long bwd_rows_of_blocks(long long tiles, int D, int vec) {
    const int groups = 256 / lanes_along(D, vec);
    const long long most = (tiles + groups - 1) / groups;
    const long long cap = BWD_BLOCKS / bwd_dblocks(D, vec) > 128 ? BWD_BLOCKS / bwd_dblocks(D, vec) : 128;
    if (most <= cap) return most > 0 ? most : 1;
    const long long rounds = (most + cap - 1) / cap;
    return (most + rounds - 1) / rounds;
}

template <typename T, int VEC>
hipError_t fwd_v(const ConvArgs& a) {
    const int along = lanes_along(a.D, VEC);
    const int dblocks = (a.D + along * VEC - 1) / (along * VEC);
    const long long tiles = tiles_of(a.B, a.T, a.N, a.cu_seqlens != nullptr, TT_FWD);
    const int groups = 256 / along;
    const long long blocks = (tiles + groups - 1) / groups * dblocks;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    const int td = tiles_dense_of(a.T, TT_FWD);
    const dim3 grid = grid_of(blocks, 256), block(256);
    if (a.W == 4) hipLaunchKernelGGL((conv_fwd_kernel<T, VEC, 4>), grid, block, 0, a.stream, a, along, dblocks, tiles, td);
    else if (a.W == 3) hipLaunchKernelGGL((conv_fwd_kernel<T, VEC, 3>), grid, block, 0, a.stream, a, along, dblocks, tiles, td);
    else hipLaunchKernelGGL((conv_fwd_kernel<T, VEC, 2>), grid, block, 0, a.stream, a, along, dblocks, tiles, td);
    return hipGetLastError();
}

template <typename T, int VEC>
hipError_t bwd_v(const ConvBwdArgs& b) {
    const ConvArgs& a = b.f;
    const int along = lanes_along(a.D, VEC);
    const int dblocks = bwd_dblocks(a.D, VEC);
    const long long tiles = tiles_of(a.B, a.T, a.N, a.cu_seqlens != nullptr, TT_BWD);
    const long long P = bwd_rows_of_blocks(tiles, a.D, VEC);
    const long long blocks = P * dblocks;
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    const int td = tiles_dense_of(a.T, TT_BWD);
    const dim3 grid((unsigned)blocks), block(256);
    const size_t lds = (size_t)256 * VEC * (a.W + 1) * sizeof(float);
    if (a.W == 4) hipLaunchKernelGGL((conv_bwd_kernel<T, VEC, 4>), grid, block, lds, a.stream, b, along, dblocks, tiles, td, P);
    else if (a.W == 3) hipLaunchKernelGGL((conv_bwd_kernel<T, VEC, 3>), grid, block, lds, a.stream, b, along, dblocks, tiles, td, P);
    else hipLaunchKernelGGL((conv_bwd_kernel<T, VEC, 2>), grid, block, lds, a.stream, b, along, dblocks, tiles, td, P);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    SumRows s;
    s.part = b.partial; s.P = P; s.M = (long long)(a.W + 1) * a.D;
    s.out = b.dweight; s.out_tail = b.dbias; s.D = a.D; s.taps = a.W;
    return launch_sum_rows(s, a.stream);
}

}  // namespace

hipError_t launch_sum_rows(const SumRows& s, hipStream_t stream) {
    hipLaunchKernelGGL(sum_rows_kernel, grid_of((s.M + 31) / 32, 1024), dim3(1024), 0, stream, s);
    return hipGetLastError();
}

long long conv_bwd_partials(int B, int T, int D, int N, bool packed) {
    // the one-channel and the four-channel form differ in their blocks: room for either
    long long most = 0;
    for (int vec : {1, 4}) {
        const long long P = bwd_rows_of_blocks(tiles_of(B, T, N, packed, TT_BWD), D, vec);
        most = P > most ? P : most;
    }
    return most;
}

hipError_t launch_conv_fwd(const ConvArgs& a) {
    const bool wide = a.wide;
    if (a.dtype == KDA_BF16) return wide ? fwd_v<__bf16, 8>(a) : fwd_v<__bf16, 1>(a);
    return wide ? fwd_v<float, 4>(a) : fwd_v<float, 1>(a);
}

hipError_t launch_conv_bwd(const ConvBwdArgs& b) {
    const bool wide = b.f.wide;
    if (b.f.dtype == KDA_BF16) return wide ? bwd_v<__bf16, 4>(b) : bwd_v<__bf16, 1>(b);
    return wide ? bwd_v<float, 4>(b) : bwd_v<float, 1>(b);
}

}  // namespace kda
