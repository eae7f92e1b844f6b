// How a wave of the per-token kernels holds a state: its 64 lanes form CG = BV/4 column
// groups times RG = 64/CG row groups, each lane R rows x 4 columns in registers (see
// kda_recurrent.hip for the layouts and why).
#pragma once

#include "kda_device.h"

namespace kda {

__device__ __forceinline__ void load4(const __bf16* p, float* out) {
    bf16x4 x = *reinterpret_cast<const bf16x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = (float)x[j];
}

__device__ __forceinline__ void load4(const float* p, float* out) {
    f32x4 x = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = x[j];
}

__device__ __forceinline__ void store4(__bf16* p, const float* x) {
    bf16x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = (__bf16)x[j];
    *reinterpret_cast<bf16x4*>(p) = y;
}

__device__ __forceinline__ void store4(float* p, const float* x) {
    f32x4 y = {x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(p) = y;
}

// Sum over the row groups: lanes CG, 2 CG, ... apart hold the same columns.
template <int CG>
__device__ __forceinline__ float sum_row_groups(float x) {
#pragma unroll
    for (int off = CG; off < 64; off *= 2) x += __shfl_xor(x, off, 64);
    return x;
}

// Row i of a lane's block in row group rg of RG, R rows each: contiguous (rg R + i), or
// dealt four at a time (ILV) (see the work decomposition above). Rows i .. i+3, i a
// multiple of 4, are consecutive in both.
template <int RG, int R, bool ILV>
__device__ __forceinline__ int block_row(int rg, int i) {
    return ILV ? 4 * RG * (i >> 2) + 4 * rg + (i & 3) : rg * R + i;
}

// The lane's R entries of one K-vector (q, k, a gate row, dt_bias), in block-row order:
// 16-byte accesses of 8 (bf16) or 4 (fp32) elements where the rows are contiguous, else
// four consecutive elements at a time.
template <int RG, int R, bool ILV>
__device__ __forceinline__ void load_rows(const __bf16* p, int rg, float (&out)[R]) {
    if (!ILV) {
        p += rg * R;
#pragma unroll
        for (int i = 0; i < R; i += 8) {
            const bf16x8 x = *reinterpret_cast<const bf16x8*>(p + i);
#pragma unroll
            for (int e = 0; e < 8; ++e) out[i + e] = (float)x[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; i += 4) {
            const bf16x4 x = *reinterpret_cast<const bf16x4*>(p + block_row<RG, R, true>(rg, i));
#pragma unroll
            for (int e = 0; e < 4; ++e) out[i + e] = (float)x[e];
        }
    }
}

template <int RG, int R, bool ILV>
__device__ __forceinline__ void load_rows(const float* p, int rg, float (&out)[R]) {
#pragma unroll
    for (int i = 0; i < R; i += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p + block_row<RG, R, ILV>(rg, i));
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i + e] = x[e];
    }
}

// The lane's block of a state, columns c0 .. c0+3: [K][V] (row d at base + d V, rows
// contiguous per row group) or, with VK, [V][K] (column c at base + c K, rows dealt four
// at a time); 16-byte accesses in both.
template <int RG, int R, bool VK>
__device__ __forceinline__ void load_state(const float* base, int K, int V, int rg, int c0,
                                           f32x4 (&S)[R]) {
#pragma unroll
    for (int i = 0; i < R; i += 4) {
        const int d = block_row<RG, R, VK>(rg, i);
        if (!VK) {
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i + e] = *reinterpret_cast<const f32x4*>(base + (size_t)(d + e) * V + c0);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(base + (size_t)(c0 + j) * K + d);
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i + e][j] = x[e];
            }
        }
    }
}

template <int RG, int R, bool VK>
__device__ __forceinline__ void store_state(float* base, int K, int V, int rg, int c0,
                                            const f32x4 (&S)[R]) {
#pragma unroll
    for (int i = 0; i < R; i += 4) {
        const int d = block_row<RG, R, VK>(rg, i);
        if (!VK) {
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<f32x4*>(base + (size_t)(d + e) * V + c0) = S[i + e];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(base + (size_t)(c0 + j) * K + d) =
                    f32x4{S[i][j], S[i + 1][j], S[i + 2][j], S[i + 3][j]};
        }
    }
}

}  // namespace kda
