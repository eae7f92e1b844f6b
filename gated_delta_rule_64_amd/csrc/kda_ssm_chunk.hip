// Chunked selective state space scan (prompts) for gfx950. Per sequence and head, S fp32
// [K, V], dt' and the log2 decay a as in the per-token kernel; over a chunk of 64 tokens
// with cum the running sums of a inside it:
//     M_ij = (c_i . b_j) 2^(cum_i - cum_j) dt'_j  (j <= i, else 0)
//     y_i  = sum_j M_ij x_j + 2^(cum_i) S^T c_i + D x_i
//     S   <- 2^(cum_63) S + sum_j 2^(cum_63 - cum_j) dt'_j b_j x_j^T
// All exponents are <= 0 for dt' >= 0, so nothing overflows whatever the decay.
//
// One 256-thread block owns a segment of a sequence, a head and 64-column slabs of V: wave
// w holds columns 16w .. 16w+15 of the state in matrix-core accumulators (rows
// 16t + 4(l/16) + r of tile t, column l % 16) and walks the chunks in order. An accumulator
// tile is its own operand: with the contraction index taken in the order the four registers
// hold it, the state feeds S^T c, and M (formed transposed, token j down the rows) feeds
// M x, without passing through lanes; the other operand is loaded in that same order.
//
// Few sequences and heads would leave most of the chip idle, so sequences are cut into
// segments: a first pass forms each segment's own end state (the last one's apart), a small
// kernel joins them in order (H_(s+1) = L_s + 2^(decay of s) H_s), and the second pass walks
// every segment from its start state. Both passes read b and x and form the state's update:
// half as much matrix work again, for as many times more blocks as there are segments.
//
// 8192 tokens x 32 heads, K = V = 128, bf16: steps 5, first pass 34, join 11, second pass 85
// us (one pass over the bytes is 33 us at a plain stream's rate). A chunk of the second pass
// takes a unit about 4,000 cycles of vector, 3,200 of matrix and 2,300 of LDS work a SIMD, which
// overlap little (see the layout notes at the bf16 kernel).
#include "kda_layer.h"

namespace kda {

namespace {

constexpr int C = 64;       // tokens of a chunk
constexpr int SLAB = 64;    // columns of V of a wave set
constexpr int PAD = 4;

// How the work is cut. seg: tokens of a segment, a multiple of C. Sequence n's segments are
// tiles of seq_tile(.., TT = seg, ..); the end states of all but its last are kept in slots
// n (per - 1) + s (dense, `per` segments each) or cu[n] / seg + s (packed: the number kept,
// floor((len - 1) / seg), never exceeds floor((a + len) / seg) - floor(a / seg), so
// sequences' slots do not meet and end below T / seg).
struct Plan {
    int seg, per;
    int ns;               // slabs of a block
    int slabs, units;     // slabs of all heads; slabs / ns
    long long tiles;      // segments at most
    long long slots;      // kept end states
    float* ends;          // [slots][slabs][K * SLAB], in the accumulators' order
    float* starts;        // the same size: initial states of cut sequences, where final_state
                          // is initial_state and would be overwritten before it is read
    float* decay;         // [slots][slabs]
    const float* steps;   // [3][HV][rows], see ssm_steps_kernel
    const int* order;     // the second pass's segments, longest first, or NULL
    int* cuts;            // packed: whether any sequence is longer than a segment, or NULL
};

struct Work {
    int n, s, count;      // sequence, segment, segments of the sequence
    int len;              // tokens of the sequence, -1: no work
    long long row0;       // its first row
    long long slot0;      // its first slot
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ long long uniform(long long v) {
    return (long long)((unsigned long long)(unsigned)uniform((int)(v >> 32)) << 32 | (unsigned)uniform((int)v));
}
// the same for every lane, and known to be
__device__ __forceinline__ Work uniform(const Work& w) {
    return Work{uniform(w.n), uniform(w.s), uniform(w.count), uniform(w.len), uniform(w.row0), uniform(w.slot0)};
}

// A block's segment and unit. Blocks go to the chip's eight dies in turn, each with its own
// L2: the units of a segment, which read the same b and c, are kept on one.
__device__ __forceinline__ void place_of(long long block, long long tiles, int units, long long* tile, int* unit) {
    const long long whole = tiles / 8 * 8;
    if (block < whole * units) {
        const long long j = block / 8;
        *tile = j / units * 8 + block % 8;
        *unit = (int)(j % units);
    } else {
        *tile = block / units;
        *unit = (int)(block % units);
    }
}

__device__ __forceinline__ Work second_pass_work(long long tile, const SsmArgs& a, const Plan& p) {
    const SeqTile s = seq_tile(p.order ? p.order[tile] : tile, a.cu_seqlens, a.N, a.T, p.seg, p.per);
    Work w;
    w.n = s.n;
    w.len = s.len;
    w.s = s.pos / p.seg;
    w.row0 = s.row0;
    w.count = s.len > 0 ? (s.len - 1) / p.seg + 1 : 1;
    w.slot0 = a.cu_seqlens ? s.row0 / p.seg : (long long)s.n * (p.per - 1);
    return w;
}

// the segment whose end state slot `slot` keeps
__device__ __forceinline__ Work first_pass_work(long long slot, const SsmArgs& a, const Plan& p) {
    Work w;
    w.len = -1;
    w.n = 0;
    w.s = 0;
    w.count = 0;
    w.row0 = w.slot0 = 0;
    if (p.cuts && !*p.cuts) return w;
    if (!a.cu_seqlens) {
        w.n = (int)(slot / (p.per - 1));
        w.s = (int)(slot % (p.per - 1));
        w.len = a.T;
        w.row0 = (long long)w.n * a.T;
        w.slot0 = (long long)w.n * (p.per - 1);
        w.count = p.per;
        return w;
    }
    int lo = 0, hi = a.N;   // the last n with cu[n] / seg <= slot
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (a.cu_seqlens[mid] / p.seg <= slot) lo = mid;
        else hi = mid;
    }
    const int bos = a.cu_seqlens[lo], eos = a.cu_seqlens[lo + 1];
    if (!(bos >= 0 && bos <= eos && eos <= a.T && (lo != 0 || bos == 0))) return w;
    w.n = lo;
    w.slot0 = bos / p.seg;
    w.s = (int)(slot - w.slot0);
    w.count = eos > bos ? (eos - bos - 1) / p.seg + 1 : 1;
    if (w.s < 0 || w.s >= w.count - 1) return w;
    w.len = eos - bos;
    w.row0 = bos;
    return w;
}

// Per-chunk scalars of one head in LDS
struct alignas(16) Steps {
    float dt[C];
    float hi[C], lo[C];   // running sums of the log2 decay, as hi + lo
    float grow[C];        // 2^(cum_63 - cum_j) dt'_j
    float all;            // 2^(cum_63)
};

// dt' and the running sums of the log2 decay inside each chunk, for every row and head:
// steps[0], [1], [2] are dt', hi and lo as [HV][rows] (the sums are formed in fp64, since
// the exponents are differences of them) and kept as hi + lo. One block: a chunk of a
// sequence and 8 heads; a wave takes a head, its lane a token. Formed once instead of in
// every block that walks the chunk, where one wave's transcendentals and 64-bit prefix sums
// held up the others (first pass of 32768 tokens x 64 heads, when they were taken out: 157 us
// with, 129 without them).
constexpr int STEP_HEADS = 8;

// inclusive prefix sum over the wave: within the four rows of 16 lanes by lane shifts, then
// the sums of the rows before (no LDS)
template <int N> __device__ __forceinline__ double row_shr(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x110 + N, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), 0x110 + N, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_value(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), l) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((int)b, l));
}
__device__ __forceinline__ double wave_scan(double v) {
    v += row_shr<1>(v);
    v += row_shr<2>(v);
    v += row_shr<4>(v);
    v += row_shr<8>(v);
    const double a = lane_value(v, 15), b = a + lane_value(v, 31), c = b + lane_value(v, 47);
    const int row = (threadIdx.x & 63) >> 4;
    return v + (row == 0 ? 0.0 : row == 1 ? a : row == 2 ? b : c);
}

// The second pass's segments by length, longest first (their order changes no result): a
// packed batch of ragged prompts then ends with short ones. 64 slots of 1..1024 tokens x 16
// heads on 512 resident blocks: 16 chunks for the busiest instead of 24. One block; a
// counting sort over 256 lengths.
constexpr int ORDER_MAX = 4096;
__device__ void order_segments(const SsmArgs& a, const Plan& p, int* order) {
    __shared__ uint8_t bin[ORDER_MAX];
    __shared__ int count[256];
    const int tid = threadIdx.x;
    count[tid] = 0;
    __syncthreads();
    for (int i = tid; i < (int)p.tiles; i += 256) {
        const SeqTile s = seq_tile(i, a.cu_seqlens, a.N, a.T, p.seg, p.per);
        const int len = max(min(s.len - s.pos, p.seg), 0);
        bin[i] = (uint8_t)((long long)((len + C - 1) / C) * 255 / (p.seg / C));
        atomicAdd(&count[bin[i]], 1);
    }
    __syncthreads();
    // places of a length: after all longer ones (sums from the longest down, thread tid
    // holding length 255 - tid)
    __shared__ int wave_sum[4];
    const int mine = count[255 - tid];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const int v = __shfl_up(upto, o, 64);
        if ((tid & 63) >= o) upto += v;
    }
    if ((tid & 63) == 63) wave_sum[tid >> 6] = upto;
    __syncthreads();
    for (int k = 0; k < tid >> 6; ++k) upto += wave_sum[k];
    count[255 - tid] = upto - mine;
    __syncthreads();
    for (int i = tid; i < (int)p.tiles; i += 256) order[atomicAdd(&count[bin[i]], 1)] = i;
}

__global__ __launch_bounds__(256) void ssm_steps_kernel(const SsmArgs a, const Plan p, float* steps, int* order, int per, int hblocks) {
    __shared__ float raw[C][STEP_HEADS + 1];
    __shared__ double rate[STEP_HEADS];
    if (blockIdx.x == gridDim.x - 1) {   // the block behind the chunks'
        flag_bad_offsets(a.cu_seqlens, a.N, a.T, a.dev_status);
        if (p.cuts && threadIdx.x < 64) {   // does a sequence of this batch have to be cut at all
            int most = 0;
            for (int n = threadIdx.x; n < a.N; n += 64) most = max(most, a.cu_seqlens[n + 1] - a.cu_seqlens[n]);
#pragma unroll
            for (int o = 32; o > 0; o /= 2) most = max(most, __shfl_xor(most, o, 64));
            if (threadIdx.x == 0) *p.cuts = most > p.seg;
        }
        if (order) order_segments(a, p, order);
        return;
    }
    const int h0 = (int)(blockIdx.x % hblocks) * STEP_HEADS;
    const SeqTile s = seq_tile(blockIdx.x / hblocks, a.cu_seqlens, a.N, a.T, C, per);
    const int cl = min(s.len - s.pos, C);
    if (cl <= 0) return;
    const long long row = s.row0 + s.pos, rows = (long long)a.B * a.T;
    if (threadIdx.x < STEP_HEADS && h0 + threadIdx.x < a.HV) rate[threadIdx.x] = ssm_rate(a.A_log[h0 + threadIdx.x]);
    for (int i = threadIdx.x; i < C * STEP_HEADS; i += 256) {
        const int t = i / STEP_HEADS, hv = i % STEP_HEADS;
        if (t < cl && h0 + hv < a.HV) raw[t][hv] = load_scalar(a.dt, a.dt_dtype, (row + t) * a.dt_stride + h0 + hv);
    }
    __syncthreads();
    const int j = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < STEP_HEADS / 4; ++n) {
        const int k = (threadIdx.x >> 6) + 4 * n, hv = min(h0 + k, a.HV - 1);
        float dt = 0.f;
        double cum = 0.0;
        if (j < cl) {
            dt = ssm_step(raw[j][min(k, a.HV - 1 - h0)], a.dt_bias ? a.dt_bias[hv] : 0.f, a.softplus);
            cum = ssm_log2_decay(dt, rate[hv - h0]);
        }
        cum = wave_scan(cum);
        if (j < cl && h0 + k < a.HV) {
            const float hi = (float)cum;
            const long long at = (long long)hv * rows + row + j;
            steps[at] = dt;
            steps[at + a.HV * rows] = hi;
            steps[at + 2 * a.HV * rows] = (float)(cum - (double)hi);
        }
    }
}

// One wave's token of a chunk: what the steps kernel left for it, and from that the
// chunk's scalars. Tokens past the chunk's `cl` take its last one with a weight of 0.
struct Step { float dt, hi, lo; };
__device__ __forceinline__ Step load_step(const SsmArgs& a, const Plan& p, long long row, int cl, int hv) {
    const int j = threadIdx.x & 63;
    const long long rows = (long long)a.B * a.T, at = (long long)hv * rows + row + min(j, cl - 1);
    return Step{p.steps[at], p.steps[at + a.HV * rows], p.steps[at + 2 * a.HV * rows]};
}
__device__ __forceinline__ double place_steps(const Step& v, int cl, Steps* s) {
    const int j = threadIdx.x & 63;
    const float dt = j < cl ? v.dt : 0.f;
    const float eh = __shfl(v.hi, 63, 64), el = __shfl(v.lo, 63, 64);
    s->dt[j] = dt;
    s->hi[j] = v.hi;
    s->lo[j] = v.lo;
    s->grow[j] = exp2_fast((eh - v.hi) + (el - v.lo)) * dt;
    if (j == 63) s->all = exp2_fast(v.hi);
    return (double)eh + (double)el;
}

// The state a segment starts from, in accumulators, and where one goes: [K][V] with this
// lane's column `col` of the slab, or a slot in the accumulators' order (tile t of part
// `part` of the slab's SLAB / 16 parts).
template <int KT> __device__ __forceinline__ void load_start(f32x4 (&S)[KT], const SsmArgs& a, const Plan& p,
                                                             const Work& w, int slab, int col, int part, bool first_pass) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const size_t per_slab = (size_t)KT * 16 * SLAB;
    const float* kept = nullptr;
    if (w.s > 0) {
        if (!first_pass) kept = p.ends + ((size_t)(w.slot0 + w.s - 1) * p.slabs + slab) * per_slab;
    } else if (!first_pass && w.count > 1 && p.starts) {
        kept = p.starts + ((size_t)w.slot0 * p.slabs + slab) * per_slab;
    } else if (a.initial_state) {
        const int vs = a.V / SLAB, hv = slab / vs;
        const float* h0 = a.initial_state + ((size_t)w.n * a.HV + hv) * (size_t)(KT * 16) * a.V + (slab % vs) * SLAB + col;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] = h0[(size_t)(16 * t + 4 * g + r) * a.V];
        return;
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
        S[t] = kept ? *reinterpret_cast<const f32x4*>(kept + ((t * 4 + part) * 64 + lane) * 4) : f32x4{0.f, 0.f, 0.f, 0.f};
}
template <int KT> __device__ __forceinline__ void store_slot(const f32x4 (&S)[KT], float* base, const Plan& p, long long slot,
                                                             int slab, int part) {
    float* at = base + ((size_t)slot * p.slabs + slab) * (size_t)(KT * 16 * SLAB) + (part * 64 + (threadIdx.x & 63)) * 4;
#pragma unroll
    for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(at + t * 1024) = S[t];
}
template <int KT> __device__ __forceinline__ void store_final(const f32x4 (&S)[KT], const SsmArgs& a, int n, int slab, int col) {
    int g = (threadIdx.x & 63) >> 4;
    // the addresses are those load_start forms: keep the compiler from holding them in
    // registers (64 of them) all through the walk
    asm volatile("" : "+v"(g));
    const int vs = a.V / SLAB, hv = slab / vs;
    float* hT = a.final_state + ((size_t)n * a.HV + hv) * (size_t)(KT * 16) * a.V + (slab % vs) * SLAB + col;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) hT[(size_t)(16 * t + 4 * g + r) * a.V] = S[t][r];
}

__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) < __builtin_inff(); }

// ---------------------------------------------------------------------------------
// fp32 inputs: everything on the fp32 matrix cores, one slab a block. FIRST: the first
// pass, which only carries the state.
// ---------------------------------------------------------------------------------
template <int K, bool FIRST>
__global__ __launch_bounds__(256) void ssm_scan_f32_kernel(const SsmArgs a, const Plan p) {
    constexpr int KT = K / 16;
    constexpr int LDB = K + PAD, LDX = SLAB + PAD;
    constexpr int NB = C * K / 4 / 256, NX = C * SLAB / 4 / 256;   // 16-byte pieces a thread
    __shared__ __attribute__((aligned(16))) float Bs[C * LDB], Cs[FIRST ? 1 : C * LDB], Xs[C * LDX];
    __shared__ f32x4 Ms[FIRST ? 1 : 10 * 64];   // M^T tiles (I, J <= I) in accumulator order
    __shared__ Steps st;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    long long tile;
    int slab;
    place_of(blockIdx.x, FIRST ? p.slots : p.tiles, p.units, &tile, &slab);
    const Work w = FIRST ? first_pass_work(tile, a, p) : second_pass_work(tile, a, p);
    if (w.len < 0) return;
    const int vs = a.V / SLAB, hv = slab / vs, h = hv / (a.HV / a.H);
    f32x4 S[KT];
    load_start(S, a, p, w, slab, 16 * wave + l16, wave, FIRST);
    if (FIRST && w.s == 0 && p.starts) store_slot(S, p.starts, p, w.slot0, slab, wave);
    const float skip = a.D ? a.D[hv] : 0.f;
    double total = 0.0;

    const int stop = w.len - w.s * p.seg < p.seg ? w.len : (w.s + 1) * p.seg;
    for (int p0 = w.s * p.seg; p0 < stop; p0 += C) {
        const int cl = w.len - p0 < C ? w.len - p0 : C;
        const long long row = w.row0 + p0;
        __syncthreads();   // the last chunk's readers are done
        // all of the chunk's loads in flight before the first is stored
        f32x4 rb[NB], rc[FIRST ? 1 : NB], rx[NX];
        const f32x4 none = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int e = i * 256 + threadIdx.x, t = e / (K / 4), k = e % (K / 4) * 4;
            const float* at = static_cast<const float*>(a.b) + (row + min(t, cl - 1)) * a.b_stride + (size_t)h * K + k;
            rb[i] = *reinterpret_cast<const f32x4*>(at);
            if constexpr (!FIRST) {
                const float* ct = static_cast<const float*>(a.c) + (row + min(t, cl - 1)) * a.c_stride + (size_t)h * K + k;
                rc[i] = *reinterpret_cast<const f32x4*>(ct);
            }
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = i * 256 + threadIdx.x, t = e / (SLAB / 4), k = e % (SLAB / 4) * 4;
            rx[i] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.x) + (row + min(t, cl - 1)) * a.x_stride + (size_t)slab * SLAB + k);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int e = i * 256 + threadIdx.x, t = e / (K / 4), k = e % (K / 4) * 4;
            *reinterpret_cast<f32x4*>(Bs + t * LDB + k) = t < cl ? rb[i] : none;
            if constexpr (!FIRST) *reinterpret_cast<f32x4*>(Cs + t * LDB + k) = t < cl ? rc[i] : none;
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = i * 256 + threadIdx.x, t = e / (SLAB / 4), k = e % (SLAB / 4) * 4;
            *reinterpret_cast<f32x4*>(Xs + t * LDX + k) = t < cl ? rx[i] : none;
        }
        if (wave == 0) total += place_steps(load_step(a, p, row, cl, hv), cl, &st);
        __syncthreads();
        if constexpr (!FIRST) {
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
        }
        // this wave's columns of x, token 16 J + 4 g + r in register [J][r]
        f32x4 xt[4];
#pragma unroll
        for (int J = 0; J < 4; ++J)
#pragma unroll
            for (int r = 0; r < 4; ++r) xt[J][r] = Xs[(16 * J + 4 * g + r) * LDX + 16 * wave + l16];
        if constexpr (!FIRST) {
            // see `odd` of the bf16 kernel
            float zero = 0.f;
#pragma unroll
            for (int J = 0; J < 4; ++J)
#pragma unroll
                for (int r = 0; r < 4; ++r) zero = fmaf(xt[J][r], 0.f, zero);
            const bool odd = __any(zero != zero);
            if (odd) {
#pragma unroll
                for (int J = 0; J < 4; ++J)
#pragma unroll
                    for (int r = 0; r < 4; ++r) xt[J][r] = is_finite(xt[J][r]) ? xt[J][r] : 0.f;
            }
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
                const float f = exp2_fast(st.hi[i]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] *= f;
#pragma unroll
                for (int J = 0; J < 4; ++J) {
                    if (J > I) break;
                    const f32x4 m = Ms[(I * (I + 1) / 2 + J) * 64 + lane];
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc = Mma<float>::mma(xt[J][r], m[r], acc);
                }
                const int q = 16 * wave + 4 * g;
                if (odd) {
                    for (int j = 0; j <= i; ++j) {
                        const float m = Ms[(I * (I + 1) / 2 + (j >> 4)) * 64 + (j >> 2 & 3) * 16 + l16][j & 3];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float v = Xs[j * LDX + q + r];
                            if (!is_finite(v)) acc[r] = fmaf(m, v, acc[r]);
                        }
                    }
                }
                if (i < cl) {   // columns 16 wave + 4 g .. +3 of token i
                    float out[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) out[r] = fmaf(skip, Xs[i * LDX + q + r], acc[r]);
                    store_vec<4>(static_cast<float*>(a.y) + ((row + i) * p.slabs + slab) * (long long)SLAB + q, out);
                }
            }
            if (odd) {
#pragma unroll
                for (int J = 0; J < 4; ++J)
#pragma unroll
                    for (int r = 0; r < 4; ++r) xt[J][r] = Xs[(16 * J + 4 * g + r) * LDX + 16 * wave + l16];
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
    if (FIRST) {
        store_slot(S, p.ends, p, w.slot0 + w.s, slab, wave);
        if (threadIdx.x == 0) p.decay[(w.slot0 + w.s) * p.slabs + slab] = exp2_fast((float)at_least(total, -1000.0));
    } else if (a.final_state && w.s == w.count - 1) {
        store_final(S, a, w.n, slab, 16 * wave + l16);
    }
}

// ---------------------------------------------------------------------------------
// bf16 inputs: the bf16 matrix cores, NS slabs of one b / c group a block. Two slabs: a wave
// holds 32 columns of one of them (two column tiles), so that what it reads of b and c, the
// most of its LDS traffic, serves twice; one slab: 16 columns.
//   * c_i . b_j is exact bf16 products summed in fp32; M after its weights, and the state as
//     the operand of S^T c, are pairs of bf16 (a value rounded and the rest of it rounded: 2^-16
//     of every term), so that y is rounded once, where it is stored: its error against 64 bits is
//     that rounding's 1.7e-3, where one bf16 for each left up to 2.1e-3 (a packed batch of 64
//     prompts, in 161 us instead of 175; 8192 tokens x 32 heads 115 and 123).
//   * the state is kept to fp32: each weighted x is cut into three bf16 (24 bits), so its
//     update is three products.
//   * operands whose contraction runs over tokens (x and b down a column) are read from LDS
//     transposed (ds_read_b64_tr_b16: four consecutive rows of a column a lane).
//   * rows past the sequence's end are loaded as zeros and their stores dropped by the bounds
//     of the buffer descriptors (made for every chunk), without branches.
// Rows of b and x in LDS are 32 bytes longer than their data, and every eight rows begin 16
// bytes later: the transposed reads' half waves (8 rows x 32 bytes) and the row-wise 8-byte
// operand reads' (16 rows x 16 bytes) then both meet every bank once. c is read by rows only:
// 16 bytes of gap a row do for it.
// ---------------------------------------------------------------------------------
constexpr int GAP = 16;   // elements
template <int LD> __device__ __forceinline__ constexpr int row_at(int r) { return r * LD + 8 * (r >> 3); }
constexpr int GAP_C = 8;

typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

// four consecutive rows (tokens 16 J + 4 g ..) of one column: `t` points at this lane's part
// of the tile, row (lane / 4) of 16 and the four columns lane % 4 stands for
template <int LD> __device__ __forceinline__ bf16x4 read_col4(const __bf16* t, int J) {
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(t + row_at<LD>(16 * J))));
}
__device__ __forceinline__ bf16x8 join(bf16x4 u, bf16x4 v) { return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7); }
// a row's 32 elements of step s, in accumulator order: 4 g .. +3 of both halves. Volatile, so
// that the compiler does not pair the reads: a ds_read2_b64 on this layout takes 16 cycles of
// LDS, half of them conflicts, where two ds_read_b64 take 4 (scan of 32768 tokens x 64 heads
// 397 us with pairs, 391 without).
__device__ __forceinline__ bf16x8 read_row(const __bf16* row, int s) {
    typedef volatile __attribute__((address_space(3))) const bf16x4* lds;
    const bf16x4 u = *(lds)(row + 32 * s), v = *(lds)(row + 32 * s + 16);
    return join(u, v);
}
// elements e and e + 1 of x times their weights, each cut into three bf16 whose sum is the
// fp32 product exactly (8 + 8 + 8 bits, by truncation)
__device__ __forceinline__ void split3(bf16x8 x, int e, float w0, float w1, bf16x8 (&out)[3]) {
    const float v0 = (float)x[e] * w0, v1 = (float)x[e + 1] * w1;
    uint32_t b0 = __float_as_uint(v0), b1 = __float_as_uint(v1);
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const bf16x2 top = __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(b1, b0, 0x07060302u));
        out[u][e] = top[0];
        out[u][e + 1] = top[1];
        if (u < 2) {
            b0 = __float_as_uint(__uint_as_float(b0) - __uint_as_float(b0 & 0xffff0000u));
            b1 = __float_as_uint(__uint_as_float(b1) - __uint_as_float(b1 & 0xffff0000u));
        }
    }
}
__device__ __forceinline__ f32x4 mma32(bf16x8 a, bf16x8 b, f32x4 c) { return Mma<__bf16>::mma(a, b, c); }

// where M's tile of token blocks I and J <= I is kept: a lane's four values in accumulator
// order as bf16, and then what their rounding left
__device__ __forceinline__ constexpr int m_tile(int I, int J) { return I * (I + 1) / 2 + J; }
// v as hi + lo
__device__ __forceinline__ void split2(f32x4 v, bf16x4& hi, bf16x4& lo) {
#pragma unroll
    for (int r = 0; r < 4; ++r) hi[r] = (__bf16)v[r];
#pragma unroll
    for (int r = 0; r < 4; ++r) lo[r] = (__bf16)(v[r] - (float)hi[r]);
}

// a descriptor of `bytes` bytes at p: loads past them give 0, stores there are dropped
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, unsigned bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
__device__ __forceinline__ bf16x8 buffer_piece(__amdgpu_buffer_rsrc_t r, unsigned at) {
    return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}

template <int K, int NS, int WAVES, bool FIRST>
__global__ __launch_bounds__(64 * WAVES, WAVES == 8 ? 4 : 2) void ssm_scan_bf16_kernel(const SsmArgs a, const Plan p) {
    constexpr int KT = K / 16, KS = K / 32;
    constexpr int THREADS = 64 * WAVES;
    constexpr int CT = 4 * NS / WAVES;                                          // column tiles of a wave
    constexpr int LDK = K + GAP, LDC = K + GAP_C, LDX = SLAB + GAP;
    constexpr int NB = C * K / 8 / THREADS, NX = C * SLAB / 8 / THREADS;   // 16-byte pieces a thread
    constexpr int RB = THREADS / (K / 8), RX = THREADS / (SLAB / 8);       // rows between them
    __shared__ __attribute__((aligned(16))) __bf16 Bs[row_at<LDK>(C)], Cs[FIRST ? 8 : LDC * C], Xs[NS][row_at<LDX>(C)];
    __shared__ __attribute__((aligned(16))) __bf16 Ms[FIRST ? 1 : NS][FIRST ? 8 : 10 * 64 * 8];
    __shared__ Steps steps[2][NS];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    long long tile;
    int slab0;
    place_of(blockIdx.x, FIRST ? p.slots : p.tiles, p.units, &tile, &slab0);
    slab0 *= NS;
    const Work w = uniform(FIRST ? first_pass_work(tile, a, p) : second_pass_work(tile, a, p));
    if (w.len < 0) return;
    const int vs = a.V / SLAB, h = slab0 / vs / (a.HV / a.H);
    const int begin = w.s * p.seg;
    const int stop = w.len - begin < p.seg ? w.len : begin + p.seg;
    // this wave's columns. Two slabs a block: tile u of a half slab (32 columns from base on)
    // has column base + 8 (m / 4) + 4 u + m % 4 at m (an accumulator's lane % 16, its operand's
    // row), so that a lane's four rows of a half's two tiles are 16 contiguous bytes of y; a
    // wave holds both (four waves) or one (eight). One slab: base + m.
    const int q = CT == 2 ? wave >> 1 : wave >> 2;
    const int base = CT == 2 ? 32 * (wave & 1) : NS == 2 ? 32 * (wave >> 1 & 1) + 4 * (wave & 1) : 16 * wave;
    const int slab = slab0 + q;
    auto column = [&](int u) { return NS == 2 ? base + 8 * (l16 >> 2) + 4 * u + (l16 & 3) : base + l16; };
    auto part = [&](int u) { return CT == 2 ? 2 * (wave & 1) + u : wave & 3; };

    // this thread's pieces of a chunk, as byte offsets from the chunk's row (a stride is
    // under 2^24), and where they go in LDS (rows 16 i, RB i and RX i are whole groups of
    // eight, so their offsets there add)
    const int tb = tid / (K / 8), tx = tid / (SLAB / 8);
    const unsigned kb = tid % (K / 8) * 8, kx = tid % (SLAB / 8) * 8;
    const __bf16* bp = static_cast<const __bf16*>(a.b) + w.row0 * a.b_stride + (size_t)h * K;
    const __bf16* cp = static_cast<const __bf16*>(a.c) + w.row0 * a.c_stride + (size_t)h * K;
    const __bf16* xp = static_cast<const __bf16*>(a.x) + w.row0 * a.x_stride + (size_t)slab0 * SLAB;
    const unsigned bs2 = (unsigned)a.b_stride * 2, cs2 = (unsigned)a.c_stride * 2, xs2 = (unsigned)a.x_stride * 2;
    const unsigned b_at = tb * bs2 + kb * 2, c_at = tb * cs2 + kb * 2, x_at = tx * xs2 + kx * 2;
    const int putk = row_at<LDK>(tb) + kb, putc = LDC * tb + kb, putx = row_at<LDX>(tx) + kx;
    // this lane's place in a row-wise operand of b and of c, in a transposed one of b, and of x
    const int rowk = row_at<LDK>(l16) + 4 * g, rowc = LDC * l16 + 4 * g;
    const int colb = row_at<LDK>(lane >> 2) + 4 * (lane & 3);
    const int colx = row_at<LDX>(lane >> 2) + base + 4 * NS * (lane & 3);
    bf16x8 rb[NB], rc[FIRST ? 1 : NB], rx[NS][NX];
    auto fetch = [&](int p0) {
        const unsigned last = min(w.len - p0, C) - 1;
        const auto bd = buffer_of(bp + p0 * a.b_stride, last * bs2 + K * 2);
        const auto cd = buffer_of(cp + p0 * a.c_stride, last * cs2 + K * 2);
        const auto xd = buffer_of(xp + p0 * a.x_stride, last * xs2 + NS * SLAB * 2);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            rb[i] = buffer_piece(bd, b_at + i * RB * bs2);
            if constexpr (!FIRST) rc[i] = buffer_piece(cd, c_at + i * RB * cs2);
        }
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int v = 0; v < NS; ++v) rx[v][i] = buffer_piece(xd, x_at + i * RX * xs2 + v * SLAB * 2);
    };
    // wave 3 - v (the ones with the fewest of M's tiles) places slab v's steps, a chunk ahead,
    // from what it loads two chunks ahead
    const int mine = WAVES - 1 - wave;
    const int my_hv = (slab0 + (mine < NS ? mine : 0)) / vs;
    Step ahead{0.f, 0.f, 0.f};
    double total = 0.0;
    auto fetch_steps = [&](int p0) {
        if (mine < NS) ahead = load_step(a, p, w.row0 + p0, min(w.len - p0, C), my_hv);
    };
    auto form_steps = [&](int p0) {
        if (mine < NS) total += place_steps(ahead, min(w.len - p0, C), &steps[(p0 / C) & 1][mine]);
    };
    if (begin < stop) {
        fetch_steps(begin);
        fetch(begin);
    }

    f32x4 S[CT][KT];
#pragma unroll
    for (int u = 0; u < CT; ++u) load_start(S[u], a, p, w, slab, column(u), part(u), FIRST);
    if (FIRST && w.s == 0 && p.starts)
#pragma unroll
        for (int u = 0; u < CT; ++u) store_slot(S[u], p.starts, p, w.slot0, slab, part(u));
    const float skip = a.D ? a.D[slab / vs] : 0.f;
    if (begin < stop) {
        form_steps(begin);
        if (begin + C < stop) fetch_steps(begin + C);
    }
    const unsigned y_row = p.slabs * SLAB * 2;
    const unsigned y_at = l16 * y_row + (base + 4 * CT * g) * 2;
    const __bf16* yp = static_cast<const __bf16*>(a.y) + (w.row0 + begin) * (long long)(p.slabs * SLAB) + slab * SLAB;

    for (int p0 = begin; p0 < stop; p0 += C, yp += C * (long long)(p.slabs * SLAB)) {
        const Steps* st = steps[(p0 / C) & 1];
        lds_barrier();   // the last chunk's readers are done
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            *reinterpret_cast<bf16x8*>(Bs + putk + row_at<LDK>(i * RB)) = rb[i];
            if constexpr (!FIRST) *reinterpret_cast<bf16x8*>(Cs + putc + LDC * i * RB) = rc[i];
        }
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int v = 0; v < NS; ++v) *reinterpret_cast<bf16x8*>(Xs[v] + putx + row_at<LDX>(i * RX)) = rx[v][i];
        lds_barrier();
        if (p0 + C < stop) {   // in flight while this chunk is worked on
            fetch(p0 + C);
            form_steps(p0 + C);
            if (p0 + 2 * C < stop) fetch_steps(p0 + 2 * C);
        }
        // this wave's columns of x down the tokens
        auto column_of_x = [&](int u, int s) {
            return join(read_col4<LDX>(Xs[q] + colx + 4 * u, 2 * s), read_col4<LDX>(Xs[q] + colx + 4 * u, 2 * s + 1));
        };
        bf16x8 xf[CT][2];
#pragma unroll
        for (int u = 0; u < CT; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                xf[u][s] = column_of_x(u, s);
        f32x4 acc[FIRST ? 1 : CT][FIRST ? 1 : 4];
        if constexpr (!FIRST) {
            // A NaN or infinity among this wave's x: M's zeros above the diagonal times it would
            // reach the tokens before it. Such values are left out of M x and come in one by one,
            // for the tokens from their own on (and are back for the state's update). Found by a
            // product with 0 on the matrix cores (1% of the pass).
            f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < CT; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s) zero = mma32(bf16x8{}, xf[u][s], zero);
            const bool odd = __any(zero[0] != zero[0]);
            if (odd) {
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (!is_finite((float)xf[u][s][e])) xf[u][s][e] = (__bf16)0.f;
            }
            // M^T's ten tiles (token rows J, columns I >= J), three or two a wave: 4 bits of
            // I and J each, the first tile lowest
            static_assert(WAVES == 4, "M's tiles are dealt to four waves");
            const unsigned tiles = wave == 0 ? 0x323130u : wave == 1 ? 0x212033u : wave == 2 ? 0x1022u : 0x0011u;
            const int count = wave < 2 ? 3 : 2;
            for (int n = 0; n < count; ++n) {
                const int I = tiles >> (8 * n + 4) & 15, J = tiles >> (8 * n) & 15;
                const int i = 16 * I + l16, j0 = 16 * J + 4 * g;
                f32x4 cb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    cb = mma32(read_row(Bs + rowk + row_at<LDK>(16) * J, s), read_row(Cs + rowc + LDC * 16 * I, s), cb);
#pragma unroll
                for (int v = 0; v < NS; ++v) {
                    const f32x4 hj = *reinterpret_cast<const f32x4*>(st[v].hi + j0), lj = *reinterpret_cast<const f32x4*>(st[v].lo + j0);
                    const f32x4 dj = *reinterpret_cast<const f32x4*>(st[v].dt + j0);
                    const float hi = st[v].hi[i], lo = st[v].lo[i];
                    f32x4 m;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float e = exp2_fast((hi - hj[r]) + (lo - lj[r])) * dj[r];
                        m[r] = j0 + r <= i ? cb[r] * e : 0.f;
                    }
                    bf16x4 mh, ml;
                    split2(m, mh, ml);
                    *reinterpret_cast<bf16x8*>(Ms[v] + (m_tile(I, J) * 64 + lane) * 8) = join(mh, ml);
                }
            }
            // S^T c of the chunk's four token blocks, scaled by the tokens' decays
#pragma unroll
            for (int I = 0; I < 4; ++I)
#pragma unroll
                for (int u = 0; u < CT; ++u) acc[u][I] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                bf16x8 sh[CT], sl[CT];
#pragma unroll
                for (int u = 0; u < CT; ++u) {
                    bf16x4 h0, l0, h1, l1;
                    split2(S[u][2 * s], h0, l0);
                    split2(S[u][2 * s + 1], h1, l1);
                    sh[u] = join(h0, h1);
                    sl[u] = join(l0, l1);
                }
#pragma unroll
                for (int I = 0; I < 4; ++I) {
                    const bf16x8 cf = read_row(Cs + rowc + LDC * 16 * I, s);
#pragma unroll
                    for (int u = 0; u < CT; ++u) acc[u][I] = mma32(sl[u], cf, acc[u][I]);
#pragma unroll
                    for (int u = 0; u < CT; ++u) acc[u][I] = mma32(sh[u], cf, acc[u][I]);
                }
            }
#pragma unroll
            for (int I = 0; I < 4; ++I) {
                const float f = exp2_fast(st[q].hi[16 * I + l16]);
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[u][I][r] *= f;
            }
            lds_barrier();   // M is there
            const auto yd = buffer_of(yp, (min(w.len - p0, C) - 1) * y_row + SLAB * 2);
#pragma unroll
            for (int I = 0; I < 4; ++I) {
#pragma unroll
                for (int s = 0; s <= (I >> 1); ++s) {
                    // token blocks 2 s and 2 s + 1, the second above the diagonal where I = 2 s
                    const bf16x8 m0 = *reinterpret_cast<const bf16x8*>(Ms[q] + (m_tile(I, 2 * s) * 64 + lane) * 8);
                    bf16x8 m1{};
                    if (2 * s + 1 <= I) m1 = *reinterpret_cast<const bf16x8*>(Ms[q] + (m_tile(I, 2 * s + 1) * 64 + lane) * 8);
                    const bf16x8 mh = __builtin_shufflevector(m0, m1, 0, 1, 2, 3, 8, 9, 10, 11);
                    const bf16x8 ml = __builtin_shufflevector(m0, m1, 4, 5, 6, 7, 12, 13, 14, 15);
#pragma unroll
                    for (int u = 0; u < CT; ++u) acc[u][I] = mma32(xf[u][s], ml, acc[u][I]);
#pragma unroll
                    for (int u = 0; u < CT; ++u) acc[u][I] = mma32(xf[u][s], mh, acc[u][I]);
                }
                if (odd) {
                    const int i = 16 * I + l16;
                    for (int j = 0; j <= i; ++j) {
                        const __bf16* mj = Ms[q] + (m_tile(I, j >> 4) * 64 + (j >> 2 & 3) * 16 + l16) * 8 + (j & 3);
                        const float m = (float)mj[0] + (float)mj[4];
                        const __bf16* xj = Xs[q] + row_at<LDX>(j) + base + 4 * CT * g;
#pragma unroll
                        for (int e = 0; e < 4 * CT; ++e) {
                            const float v = (float)xj[e];
                            if (!is_finite(v)) acc[e >> 2][I][e & 3] = fmaf(m, v, acc[e >> 2][I][e & 3]);
                        }
                    }
                }
                // columns base + 4 NS g .. of token 16 I + l % 16
                const __bf16* xi = Xs[q] + row_at<LDX>(l16) + base + 4 * CT * g + row_at<LDX>(16 * I);
                if constexpr (CT == 2) {
                    const bf16x8 x8 = *reinterpret_cast<const bf16x8*>(xi);
                    bf16x8 out;
#pragma unroll
                    for (int e = 0; e < 8; ++e) out[e] = (__bf16)fmaf(skip, (float)x8[e], acc[e >> 2][I][e & 3]);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, out), yd, y_at + I * 16 * y_row, 0, 0);
                } else {
                    const bf16x4 x4 = *reinterpret_cast<const bf16x4*>(xi);
                    bf16x4 out;
#pragma unroll
                    for (int e = 0; e < 4; ++e) out[e] = (__bf16)fmaf(skip, (float)x4[e], acc[0][I][e]);
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, out), yd, y_at + I * 16 * y_row, 0, 0);
                }
            }
            if (odd) {
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int s = 0; s < 2; ++s) xf[u][s] = column_of_x(u, s);
            }
        }
        // the state at the chunk's end
        const float all = st[q].all;
#pragma unroll
        for (int u = 0; u < CT; ++u)
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[u][t][r] *= all;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 xw[CT][3];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const f32x4 grow = *reinterpret_cast<const f32x4*>(st[q].grow + 32 * s + 16 * hf + 4 * g);
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int r = 0; r < 4; r += 2) split3(xf[u][s], 4 * hf + r, grow[r], grow[r + 1], xw[u]);
            }
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const bf16x8 bt = join(read_col4<LDK>(Bs + colb + 16 * t, 2 * s), read_col4<LDK>(Bs + colb + 16 * t, 2 * s + 1));
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int u = 0; u < CT; ++u) S[u][t] = mma32(bt, xw[u][k], S[u][t]);
            }
        }
    }
    if constexpr (FIRST) {
#pragma unroll
        for (int u = 0; u < CT; ++u) store_slot(S[u], p.ends, p, w.slot0 + w.s, slab, part(u));
        if (mine < NS && lane == 0)
            p.decay[(w.slot0 + w.s) * p.slabs + slab0 + mine] = exp2_fast((float)at_least(total, -1000.0));
    } else if (a.final_state && w.s == w.count - 1) {
#pragma unroll
        for (int u = 0; u < CT; ++u) store_final(S[u], a, w.n, slab, column(u));
    }
}

// Joins the kept end states of a sequence in order: slot s becomes the state its segment
// s + 1 starts from. One thread: four values of one slab; one block: K SLAB / JOIN_PARTS.
constexpr int JOIN_PARTS = 4;
constexpr int BATCH = 8;
template <int K>
__global__ __launch_bounds__(K * SLAB / 4 / JOIN_PARTS) void ssm_join_kernel(const SsmArgs a, const Plan p) {
    const int part = (int)(blockIdx.x % JOIN_PARTS);
    const int slab = (int)(blockIdx.x / JOIN_PARTS % p.slabs);
    const long long seq = blockIdx.x / JOIN_PARTS / p.slabs;   // dense: the sequence; packed: a slot
    const Work w = first_pass_work(a.cu_seqlens ? seq : seq * (p.per - 1), a, p);
    if (w.len < 0 || w.s != 0 || w.count <= 2) return;
    const size_t step = (size_t)p.slabs * K * SLAB;
    float* at = p.ends + ((size_t)w.slot0 * p.slabs + slab) * (size_t)(K * SLAB) + (part * blockDim.x + threadIdx.x) * 4;
    f32x4 H = *reinterpret_cast<const f32x4*>(at);
    // loads of eight slots at a time are in flight before the first is stored over
    for (int s = 1; s < w.count - 1; s += BATCH) {
        const int m = min(BATCH, w.count - 1 - s);
        f32x4 L[BATCH];
        float d[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int k = i < m ? i : 0;
            L[i] = *reinterpret_cast<const f32x4*>(at + (k + 1) * step);
            d[i] = p.decay[(w.slot0 + s + k) * p.slabs + slab];
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (i >= m) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) H[r] = fmaf(d[i], H[r], L[i][r]);
            *reinterpret_cast<f32x4*>(at + (i + 1) * step) = H;
        }
        at += BATCH * step;
    }
}

// Dense sequences are cut only where their blocks would leave half the chip's 256 units idle
// (N x units <= 128), into pieces of at least SEG_MIN chunks, for about BLOCKS_WANTED blocks,
// two a unit: 32768 tokens x 64 heads 419 us (256 blocks 458, 768 450, 1024 436), 8192 x 32 heads
// 138 (147, 154, 157). N x 4096 tokens x 32 heads, K = V = 128, cut and whole: N x units = 64
// 132 and 333 us, 128 224 and 340, 192 325 and 346, 256 371 and 352 (the first pass then costs
// what the second gains).
constexpr int SEG_MIN = 4;
constexpr long long BLOCKS_WANTED = 512;

Plan plan_of(int B, int T, int H, int HV, int K, int V, int N, bool packed, int dtype) {
    Plan p;
    p.slabs = HV * (V / SLAB);
    // two slabs a block share b, c and their products where a group has an even number of slabs
    // (32768 tokens x 64 heads: 419 us, one slab a block 471; 8192 x 32 heads 138 and 147)
    p.ns = dtype == KDA_BF16 && (p.slabs / H) % 2 == 0 ? 2 : 1;
    p.units = p.slabs / p.ns;
    const long long chunks = ((long long)T + C - 1) / C;
    long long seg = chunks > 0 ? chunks : 1;   // chunks of a segment
    if (packed) {
        // lengths are on the device: cut what is longer than twice an even share of the rows
        // (64 slots of 1..1024 tokens x 16 heads: 182 us, with once a share 242: the first pass
        // then works on a few sequences only, in order; one prompt of 8192 x 32 heads takes 138 us
        // either way, and as a dense one)
        const long long share = 2 * chunks * p.units / BLOCKS_WANTED;
        const long long piece = share > SEG_MIN ? share : SEG_MIN;
        if (piece < seg) seg = piece;
    } else if ((long long)N * p.units <= 128) {
        const long long pieces = BLOCKS_WANTED / ((long long)N * p.units > 0 ? (long long)N * p.units : 1);
        long long piece = (chunks + pieces - 1) / pieces;
        if (piece < SEG_MIN) piece = SEG_MIN;
        if (piece < seg) seg = piece;
    }
    p.seg = (int)(seg * C);
    p.per = (int)((chunks + seg - 1) / seg);
    if (p.per < 1) p.per = 1;
    p.tiles = packed ? (long long)T / p.seg + N : (long long)N * p.per;
    p.slots = packed ? (T > p.seg ? (long long)T / p.seg : 0) : (long long)N * (p.per - 1);
    p.ends = p.starts = p.decay = nullptr;
    p.steps = nullptr;
    p.order = nullptr;
    p.cuts = nullptr;
    return p;
}

inline size_t slots_bytes(const Plan& p, int K) { return (size_t)p.slots * p.slabs * K * SLAB * sizeof(float); }

// waves of a two-slab block: the second pass shares its operand reads between two column
// tiles a wave; the first has half the registers to hold and gains more from eight waves
template <int K, bool FIRST> void launch_pass(const SsmArgs& a, const Plan& p, unsigned blocks) {
    if (a.dtype == KDA_F32)
        hipLaunchKernelGGL((ssm_scan_f32_kernel<K, FIRST>), dim3(blocks), dim3(256), 0, a.stream, a, p);
    else if (p.ns == 2)
        hipLaunchKernelGGL((ssm_scan_bf16_kernel<K, 2, FIRST ? 8 : 4, FIRST>), dim3(blocks), dim3(FIRST ? 512 : 256), 0, a.stream, a, p);
    else
        hipLaunchKernelGGL((ssm_scan_bf16_kernel<K, 1, 4, FIRST>), dim3(blocks), dim3(256), 0, a.stream, a, p);
}

// The workspace: [ends][starts][steps][decay][cuts][order]
inline size_t steps_bytes(int B, int T, int HV) { return (size_t)3 * HV * B * T * sizeof(float); }
inline size_t decay_bytes(const Plan& p) { return (size_t)p.slots * p.slabs * sizeof(float); }
inline size_t order_bytes(const Plan& p, bool packed) { return packed && p.tiles <= ORDER_MAX ? (size_t)p.tiles * sizeof(int) : 0; }
inline size_t cuts_bytes(const Plan& p, bool packed) { return packed && p.slots > 0 ? sizeof(int) : 0; }

template <int K> hipError_t launch_k(const SsmArgs& a) {
    Plan p = plan_of(a.B, a.T, a.H, a.HV, K, a.V, a.N, a.cu_seqlens != nullptr, a.dtype);
    const long long first = p.slots * p.units, second = p.tiles * p.units;
    const long long join = p.slots > 0 ? (a.cu_seqlens ? p.slots : (long long)a.N) * p.slabs * JOIN_PARTS : 0;
    const int per = (a.T + C - 1) / C, hblocks = (a.HV + STEP_HEADS - 1) / STEP_HEADS;
    const bool packed = a.cu_seqlens != nullptr;
    const long long chunks = (packed ? (long long)a.T / C + a.N : (long long)a.N * per) * hblocks + 1;
    if (!grid_fits(first, 512) || !grid_fits(second, 256) || !grid_fits(join, K * SLAB / 4 / JOIN_PARTS) || !grid_fits(chunks, 256))
        return hipErrorInvalidConfiguration;
    char* ws = static_cast<char*>(a.workspace);
    p.ends = reinterpret_cast<float*>(ws);
    if (a.final_state && a.final_state == a.initial_state) p.starts = reinterpret_cast<float*>(ws + slots_bytes(p, K));
    float* steps = reinterpret_cast<float*>(ws + 2 * slots_bytes(p, K));
    p.steps = steps;
    p.decay = reinterpret_cast<float*>(ws + 2 * slots_bytes(p, K) + steps_bytes(a.B, a.T, a.HV));
    int* tail = reinterpret_cast<int*>(p.decay + p.slots * p.slabs);
    if (cuts_bytes(p, packed)) p.cuts = tail++;
    int* order = order_bytes(p, packed) ? tail : nullptr;
    p.order = order;
    hipLaunchKernelGGL(ssm_steps_kernel, dim3((unsigned)chunks), dim3(256), 0, a.stream, a, p, steps, order, per, hblocks);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (p.slots > 0) {
        launch_pass<K, true>(a, p, (unsigned)first);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL((ssm_join_kernel<K>), dim3((unsigned)join), dim3(K * SLAB / 4 / JOIN_PARTS), 0, a.stream, a, p);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (second > 0) launch_pass<K, false>(a, p, (unsigned)second);
    return hipGetLastError();
}

}  // namespace

size_t ssm_chunk_workspace(int B, int T, int H, int HV, int K, int V, int N, bool packed, int dtype) {
    const Plan p = plan_of(B, T, H, HV, K, V, N, packed, dtype);
    return 2 * slots_bytes(p, K) + steps_bytes(B, T, HV) + decay_bytes(p) + cuts_bytes(p, packed) + order_bytes(p, packed);
}

hipError_t launch_ssm_chunk(const SsmArgs& a) { return a.K == 128 ? launch_k<128>(a) : launch_k<64>(a); }

}  // namespace kda
