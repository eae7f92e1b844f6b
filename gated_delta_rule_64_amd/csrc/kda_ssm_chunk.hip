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
// every segment from its start state. Both passes read b and x and form the state's update,
// which is a third more matrix work for as many times more blocks as there are segments.
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
};

struct Work {
    int n, s, count;      // sequence, segment, segments of the sequence
    int len;              // tokens of the sequence, -1: no work
    long long row0;       // its first row
    long long slot0;      // its first slot
};

__device__ __forceinline__ Work second_pass_work(long long tile, const SsmArgs& a, const Plan& p) {
    const SeqTile s = seq_tile(tile, a.cu_seqlens, a.N, a.T, p.seg, p.per);
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
struct Steps {
    float dt[C];
    float hi[C], lo[C];   // running sums of the log2 decay, as hi + lo
    float grow[C];        // 2^(cum_63 - cum_j) dt'_j
    float fall[C];        // 2^(cum_i)
    double end;           // cum_63
    float all;            // 2^(cum_63)
};

// The bits of token `row`'s dt of head hv: widened only where they are used, so that the load
// is not waited for before.
__device__ __forceinline__ uint32_t load_dt_bits(const SsmArgs& a, long long row, int hv) {
    const long long at = row * a.dt_stride + hv;
    return a.dt_dtype == KDA_BF16 ? (uint32_t) static_cast<const uint16_t*>(a.dt)[at] : static_cast<const uint32_t*>(a.dt)[at];
}
__device__ __forceinline__ float dt_of_bits(const SsmArgs& a, uint32_t bits) {
    return __uint_as_float(a.dt_dtype == KDA_BF16 ? bits << 16 : bits);
}

// One wave: lane j takes token j of `len`, whose raw dt it brings. The running sums are
// formed in fp64: the exponents are differences of them.
__device__ __forceinline__ void chunk_steps(float raw, int len, float A_log, float bias, int softplus, Steps* s) {
    const int j = threadIdx.x & 63;
    float dt = 0.f;
    double cum = 0.0;
    if (j < len) {
        dt = ssm_step(raw, bias, softplus);
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
    if (j == 63) {
        s->end = cum;
        s->all = exp2_fast(hi);
    }
}

// The state a segment starts from, in accumulators, and where one goes: [K][V] with this
// lane's column `col`, or a slot in the accumulators' order.
template <int KT> __device__ __forceinline__ void load_start(f32x4 (&S)[KT], const SsmArgs& a, const Plan& p,
                                                             const Work& w, int slab, bool first_pass) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
    const size_t per_slab = (size_t)KT * 16 * SLAB;
    const float* kept = nullptr;
    if (w.s > 0) {
        if (!first_pass) kept = p.ends + ((size_t)(w.slot0 + w.s - 1) * p.slabs + slab) * per_slab;
    } else if (!first_pass && w.count > 1 && p.starts) {
        kept = p.starts + ((size_t)w.slot0 * p.slabs + slab) * per_slab;
    } else if (a.initial_state) {
        const int vs = a.V / SLAB, hv = slab / vs;
        const float* h0 = a.initial_state + ((size_t)w.n * a.HV + hv) * (size_t)(KT * 16) * a.V + (slab % vs) * SLAB + 16 * wave + l16;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] = h0[(size_t)(16 * t + 4 * g + r) * a.V];
        return;
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
        S[t] = kept ? *reinterpret_cast<const f32x4*>(kept + ((t * 4 + wave) * 64 + lane) * 4) : f32x4{0.f, 0.f, 0.f, 0.f};
}
template <int KT> __device__ __forceinline__ void store_slot(const f32x4 (&S)[KT], float* base, const Plan& p, long long slot,
                                                             int slab) {
    float* at = base + ((size_t)slot * p.slabs + slab) * (size_t)(KT * 16 * SLAB) + threadIdx.x * 4;
#pragma unroll
    for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(at + t * 1024) = S[t];
}
template <int KT> __device__ __forceinline__ void store_final(const f32x4 (&S)[KT], const SsmArgs& a, int n, int slab) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
    const int vs = a.V / SLAB, hv = slab / vs;
    float* hT = a.final_state + ((size_t)n * a.HV + hv) * (size_t)(KT * 16) * a.V + (slab % vs) * SLAB + 16 * wave + l16;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) hT[(size_t)(16 * t + 4 * g + r) * a.V] = S[t][r];
}

// ---------------------------------------------------------------------------------
// fp32 inputs: everything on the fp32 matrix cores, one slab a block. FIRST: the first
// pass, which only carries the state.
// ---------------------------------------------------------------------------------
template <int K, bool FIRST>
__global__ __launch_bounds__(256) void ssm_scan_f32_kernel(const SsmArgs a, const Plan p) {
    constexpr int KT = K / 16;
    constexpr int LDB = K + PAD, LDX = SLAB + PAD;
    __shared__ float Bs[C * LDB], Cs[FIRST ? 1 : C * LDB], Xs[C * LDX];
    __shared__ f32x4 Ms[FIRST ? 1 : 10 * 64];   // M^T tiles (I, J <= I) in accumulator order
    __shared__ Steps st;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    if (!FIRST && blockIdx.x == 0) flag_bad_offsets(a.cu_seqlens, a.N, a.T, a.dev_status);
    const int slab = (int)(blockIdx.x % p.slabs);
    const long long tile = blockIdx.x / p.slabs;
    const Work w = FIRST ? first_pass_work(tile, a, p) : second_pass_work(tile, a, p);
    if (w.len < 0) return;
    const int vs = a.V / SLAB, hv = slab / vs, h = hv / (a.HV / a.H);
    f32x4 S[KT];
    load_start(S, a, p, w, slab, FIRST);
    if (FIRST && w.s == 0 && p.starts) store_slot(S, p.starts, p, w.slot0, slab);
    const float A_log = a.A_log[hv];
    const float bias = a.dt_bias ? a.dt_bias[hv] : 0.f;
    const float skip = a.D ? a.D[hv] : 0.f;
    double total = 0.0;

    const int stop = w.len - w.s * p.seg < p.seg ? w.len : (w.s + 1) * p.seg;
    for (int p0 = w.s * p.seg; p0 < stop; p0 += C) {
        const int cl = w.len - p0 < C ? w.len - p0 : C;
        const long long row = w.row0 + p0;
        __syncthreads();   // the last chunk's readers are done
        for (int i = threadIdx.x; i < C * K / 4; i += 256) {
            const int t = i / (K / 4), k = i % (K / 4) * 4;
            float u[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
            if (t < cl) {
                load_vec<4>(static_cast<const float*>(a.b) + (row + t) * a.b_stride + (size_t)h * K + k, u);
                if (!FIRST) load_vec<4>(static_cast<const float*>(a.c) + (row + t) * a.c_stride + (size_t)h * K + k, v);
            }
            store_vec<4>(Bs + t * LDB + k, u);
            if (!FIRST) store_vec<4>(Cs + t * LDB + k, v);
        }
        for (int i = threadIdx.x; i < C * SLAB / 4; i += 256) {
            const int t = i / (SLAB / 4), q = i % (SLAB / 4) * 4;
            float u[4] = {0.f, 0.f, 0.f, 0.f};
            if (t < cl) load_vec<4>(static_cast<const float*>(a.x) + (row + t) * a.x_stride + (size_t)slab * SLAB + q, u);
            store_vec<4>(Xs + t * LDX + q, u);
        }
        if (wave == 0) {
            chunk_steps(dt_of_bits(a, load_dt_bits(a, row + min(lane, cl - 1), hv)), cl, A_log, bias, a.softplus, &st);
        }
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
                    const int q = 16 * wave + 4 * g;
                    float out[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) out[r] = fmaf(skip, Xs[i * LDX + q + r], acc[r]);
                    store_vec<4>(static_cast<float*>(a.y) + ((row + i) * p.slabs + slab) * (long long)SLAB + q, out);
                }
            }
        }
        // the state at the chunk's end
        const float all = st.all;
        if (FIRST) total += st.end;
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
        store_slot(S, p.ends, p, w.slot0 + w.s, slab);
        if (threadIdx.x == 0) p.decay[(w.slot0 + w.s) * p.slabs + slab] = exp2_fast((float)fmax(total, -1000.0));
    } else if (a.final_state && w.s == w.count - 1) {
        store_final(S, a, w.n, slab);
    }
}

// ---------------------------------------------------------------------------------
// bf16 inputs: the bf16 matrix cores, NS slabs of one b / c group a block.
//   * c_i . b_j is exact bf16 products summed in fp32; M is rounded to bf16 once after its
//     weights, and the state once as the operand of S^T c: half a bf16 step of every term,
//     which is what y's own storage costs.
//   * the state is kept to fp32: each weighted x is split into three bf16 (24 bits), so its
//     update is three products.
//   * operands whose contraction runs over tokens (x and b down a column) are read from LDS
//     transposed (ds_read_b64_tr_b16: four consecutive rows of a column a lane).
// Rows in LDS are 32 bytes longer than their data, so that both the row-wise 8-byte operand
// reads and the transposed ones (16 rows x 32 bytes a wave) spread over all banks.
// ---------------------------------------------------------------------------------
constexpr int GAP = 16;   // elements

typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// four consecutive rows (tokens 16 J + 4 g ..) of column c0 + l % 16 of a [C][LD] tile
template <int LD> __device__ __forceinline__ bf16x4 read_col4(const __bf16* t, int J, int c0) {
    const int lane = threadIdx.x & 63;
    const __bf16* at = t + (16 * J + (lane >> 2)) * LD + c0 + 4 * (lane & 3);
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at)));
}
__device__ __forceinline__ bf16x8 join(bf16x4 u, bf16x4 v) { return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7); }
// a row's 32 elements of step s, in accumulator order: 4 g .. +3 of both halves
__device__ __forceinline__ bf16x8 read_row(const __bf16* row, int s, int g) {
    return join(*reinterpret_cast<const bf16x4*>(row + 32 * s + 4 * g), *reinterpret_cast<const bf16x4*>(row + 32 * s + 16 + 4 * g));
}
__device__ __forceinline__ f32x4 mma32(bf16x8 a, bf16x8 b, f32x4 c) { return Mma<__bf16>::mma(a, b, c); }

// where M's operand fragment of token block I, step s (token blocks 2s and 2s+1) is kept
__device__ __forceinline__ constexpr int m_frag(int I, int s) { return I < 2 ? I : 2 * I - 2 + s; }

template <int K, int NS, bool FIRST>
__global__ __launch_bounds__(256, 2) void ssm_scan_bf16_kernel(const SsmArgs a, const Plan p) {
    constexpr int KT = K / 16, KS = K / 32;
    constexpr int LDK = K + GAP, LDX = SLAB + GAP;
    constexpr int NB = C * K / 8 / 256, NX = C * SLAB / 8 / 256;   // 16-byte pieces a thread
    constexpr int RB = 256 / (K / 8), RX = 256 / (SLAB / 8);       // rows between them
    __shared__ __attribute__((aligned(16))) __bf16 Bs[C * LDK], Cs[FIRST ? 8 : C * LDK], Xs[NS][C * LDX];
    __shared__ __attribute__((aligned(16))) __bf16 Ms[FIRST ? 1 : NS][FIRST ? 8 : 6 * 64 * 8];
    __shared__ Steps steps[2][NS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    if (!FIRST && blockIdx.x == 0) flag_bad_offsets(a.cu_seqlens, a.N, a.T, a.dev_status);
    const int slab0 = (int)(blockIdx.x % p.units) * NS;
    const long long tile = blockIdx.x / p.units;
    const Work w = FIRST ? first_pass_work(tile, a, p) : second_pass_work(tile, a, p);
    if (w.len < 0) return;
    const int vs = a.V / SLAB, h = slab0 / vs / (a.HV / a.H);
    const int begin = w.s * p.seg;
    const int stop = w.len - begin < p.seg ? w.len : begin + p.seg;

    // this thread's pieces of a chunk; past the sequence's end the last row stands in (its
    // weights are 0 there)
    const int tb = tid / (K / 8), tx = tid / (SLAB / 8);
    const __bf16* bp = static_cast<const __bf16*>(a.b) + w.row0 * a.b_stride + (size_t)h * K + tid % (K / 8) * 8;
    const __bf16* cp = static_cast<const __bf16*>(a.c) + w.row0 * a.c_stride + (size_t)h * K + tid % (K / 8) * 8;
    const __bf16* xp = static_cast<const __bf16*>(a.x) + w.row0 * a.x_stride + (size_t)slab0 * SLAB + tid % (SLAB / 8) * 8;
    bf16x8 rb[NB], rc[FIRST ? 1 : NB], rx[NS][NX];
    auto fetch = [&](int p0) {
        const int last = w.len - 1;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const long long t = min(p0 + tb + i * RB, last);
            rb[i] = *reinterpret_cast<const bf16x8*>(bp + t * a.b_stride);
            if constexpr (!FIRST) rc[i] = *reinterpret_cast<const bf16x8*>(cp + t * a.c_stride);
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const __bf16* at = xp + (long long)min(p0 + tx + i * RX, last) * a.x_stride;
#pragma unroll
            for (int q = 0; q < NS; ++q) rx[q][i] = *reinterpret_cast<const bf16x8*>(at + q * SLAB);
        }
    };
    // wave q < NS forms slab q's steps, a chunk ahead, from dt it loads two chunks ahead
    const int my_hv = (slab0 + (wave < NS ? wave : 0)) / vs;
    const float my_A = a.A_log[my_hv], my_bias = a.dt_bias ? a.dt_bias[my_hv] : 0.f;
    uint32_t bits = 0;
    auto fetch_dt = [&](int p0) {
        if (wave < NS) bits = load_dt_bits(a, w.row0 + min(p0 + lane, w.len - 1), my_hv);
    };
    auto form_steps = [&](int p0) {
        if (wave < NS) chunk_steps(dt_of_bits(a, bits), w.len - p0, my_A, my_bias, a.softplus, &steps[(p0 / C) & 1][wave]);
    };
    if (begin < stop) {
        fetch_dt(begin);
        fetch(begin);
    }

    f32x4 S[NS][KT];
#pragma unroll
    for (int q = 0; q < NS; ++q) load_start(S[q], a, p, w, slab0 + q, FIRST);
    if (FIRST && w.s == 0 && p.starts)
#pragma unroll
        for (int q = 0; q < NS; ++q) store_slot(S[q], p.starts, p, w.slot0, slab0 + q);
    float skip[NS];
#pragma unroll
    for (int q = 0; q < NS; ++q) skip[q] = a.D ? a.D[(slab0 + q) / vs] : 0.f;
    double total = 0.0;
    if constexpr (!FIRST) {
        // the halves of M's fragments above the diagonal: token blocks 1 of I = 0, 3 of I = 2
        if (wave == 0)
#pragma unroll
            for (int q = 0; q < NS; ++q) {
                *reinterpret_cast<bf16x4*>(Ms[q] + (m_frag(0, 0) * 64 + lane) * 8 + 4) = bf16x4{};
                *reinterpret_cast<bf16x4*>(Ms[q] + (m_frag(2, 1) * 64 + lane) * 8 + 4) = bf16x4{};
            }
    }
    if (begin < stop) {
        form_steps(begin);
        if (begin + C < stop) fetch_dt(begin + C);
    }
    const long long y_row = (long long)p.slabs * SLAB;
    __bf16* yp = static_cast<__bf16*>(a.y) + (w.row0 + begin + l16) * y_row + slab0 * SLAB + 16 * wave + 4 * g;

    for (int p0 = begin; p0 < stop; p0 += C, yp += C * y_row) {
        const int cl = w.len - p0 < C ? w.len - p0 : C;
        const Steps* st = steps[(p0 / C) & 1];
        lds_barrier();   // the last chunk's readers are done
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            *reinterpret_cast<bf16x8*>(Bs + (tb + i * RB) * LDK + tid % (K / 8) * 8) = rb[i];
            if constexpr (!FIRST) *reinterpret_cast<bf16x8*>(Cs + (tb + i * RB) * LDK + tid % (K / 8) * 8) = rc[i];
        }
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int q = 0; q < NS; ++q) *reinterpret_cast<bf16x8*>(Xs[q] + (tx + i * RX) * LDX + tid % (SLAB / 8) * 8) = rx[q][i];
        lds_barrier();
        if (p0 + C < stop) {   // in flight while this chunk is worked on
            fetch(p0 + C);
            form_steps(p0 + C);
            if (p0 + 2 * C < stop) fetch_dt(p0 + 2 * C);
        }

        if constexpr (!FIRST) {
            // M^T: wave w forms token rows J <= w of token columns 16 w ..
            bf16x8 cf[KS];
            const int i = 16 * wave + l16;
#pragma unroll
            for (int s = 0; s < KS; ++s) cf[s] = read_row(Cs + i * LDK, s, g);
#pragma unroll
            for (int J = 0; J < 4; ++J) {
                if (J > wave) break;
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < KS; ++s) acc = mma32(read_row(Bs + (16 * J + l16) * LDK, s, g), cf[s], acc);
                const int j0 = 16 * J + 4 * g;
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    const f32x4 hj = *reinterpret_cast<const f32x4*>(st[q].hi + j0), lj = *reinterpret_cast<const f32x4*>(st[q].lo + j0);
                    const f32x4 dj = *reinterpret_cast<const f32x4*>(st[q].dt + j0);
                    const float hi = st[q].hi[i], lo = st[q].lo[i];
                    bf16x4 m;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float e = exp2_fast((hi - hj[r]) + (lo - lj[r])) * dj[r];
                        m[r] = (__bf16)(J < wave || j0 + r <= i ? acc[r] * e : 0.f);
                    }
                    *reinterpret_cast<bf16x4*>(Ms[q] + (m_frag(wave, J >> 1) * 64 + lane) * 8 + 4 * (J & 1)) = m;
                }
            }
        }
        // this wave's columns of x down the tokens
        bf16x8 xf[NS][2];
#pragma unroll
        for (int q = 0; q < NS; ++q)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                xf[q][s] = join(read_col4<LDX>(Xs[q], 2 * s, 16 * wave), read_col4<LDX>(Xs[q], 2 * s + 1, 16 * wave));
        if constexpr (!FIRST) {
            bf16x8 sf[NS][KS];
#pragma unroll
            for (int q = 0; q < NS; ++q)
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        sf[q][s][r] = (__bf16)S[q][2 * s][r];
                        sf[q][s][4 + r] = (__bf16)S[q][2 * s + 1][r];
                    }
            lds_barrier();
#pragma unroll
            for (int I = 0; I < 4; ++I) {
                if (16 * I >= cl) break;
                const int i = 16 * I + l16;
                bf16x8 cf[KS];
#pragma unroll
                for (int s = 0; s < KS; ++s) cf[s] = read_row(Cs + i * LDK, s, g);
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < KS; ++s) acc = mma32(sf[q][s], cf[s], acc);
                    const float f = st[q].fall[i];
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r] *= f;
#pragma unroll
                    for (int s = 0; s <= (I >> 1); ++s)
                        acc = mma32(xf[q][s], *reinterpret_cast<const bf16x8*>(Ms[q] + (m_frag(I, s) * 64 + lane) * 8), acc);
                    // columns 16 wave + 4 g .. +3 of token i
                    const bf16x4 xi = *reinterpret_cast<const bf16x4*>(Xs[q] + i * LDX + 16 * wave + 4 * g);
                    bf16x4 out;
#pragma unroll
                    for (int r = 0; r < 4; ++r) out[r] = (__bf16)fmaf(skip[q], (float)xi[r], acc[r]);
                    if (i < cl) *reinterpret_cast<bf16x4*>(yp + 16 * I * y_row + q * SLAB) = out;
                }
                __builtin_amdgcn_sched_barrier(0);   // keeps the four blocks' operands from being live at once
            }
        }
        // the state at the chunk's end
        if (FIRST && wave < NS) total += st[wave].end;
#pragma unroll
        for (int q = 0; q < NS; ++q) {
            const float all = st[q].all;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[q][t][r] *= all;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 xw[NS][3];
#pragma unroll
            for (int q = 0; q < NS; ++q)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const f32x4 grow = *reinterpret_cast<const f32x4*>(st[q].grow + 32 * s + 16 * hf + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int e = 4 * hf + r;
                        const float v = (float)xf[q][s][e] * grow[r];
                        const __bf16 v0 = (__bf16)v;
                        const float r1 = v - (float)v0;
                        const __bf16 v1 = (__bf16)r1;
                        xw[q][0][e] = v0;
                        xw[q][1][e] = v1;
                        xw[q][2][e] = (__bf16)(r1 - (float)v1);
                    }
                }
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const bf16x8 bt = join(read_col4<LDK>(Bs, 2 * s, 16 * t), read_col4<LDK>(Bs, 2 * s + 1, 16 * t));
#pragma unroll
                for (int q = 0; q < NS; ++q)
#pragma unroll
                    for (int u = 2; u >= 0; --u) S[q][t] = mma32(bt, xw[q][u], S[q][t]);
            }
        }
    }
    if constexpr (FIRST) {
#pragma unroll
        for (int q = 0; q < NS; ++q) store_slot(S[q], p.ends, p, w.slot0 + w.s, slab0 + q);
        if (wave < NS && lane == 0)
            p.decay[(w.slot0 + w.s) * p.slabs + slab0 + wave] = exp2_fast((float)fmax(total, -1000.0));
    } else if (a.final_state && w.s == w.count - 1) {
#pragma unroll
        for (int q = 0; q < NS; ++q) store_final(S[q], a, w.n, slab0 + q);
    }
}

// Joins the kept end states of a sequence in order: slot s becomes the state its segment
// s + 1 starts from. One thread: four values of one slab.
template <int K>
__global__ __launch_bounds__(256) void ssm_join_kernel(const SsmArgs a, const Plan p) {
    constexpr int BLOCKS = K * SLAB / 1024;   // blocks a slab
    const int part = (int)(blockIdx.x % BLOCKS);
    const int slab = (int)(blockIdx.x / BLOCKS % p.slabs);
    const long long seq = blockIdx.x / BLOCKS / p.slabs;   // dense: the sequence; packed: a slot
    const Work w = first_pass_work(a.cu_seqlens ? seq : seq * (p.per - 1), a, p);
    if (w.len < 0 || w.s != 0 || w.count <= 2) return;
    const size_t step = (size_t)p.slabs * K * SLAB;
    float* at = p.ends + ((size_t)w.slot0 * p.slabs + slab) * (size_t)(K * SLAB) + part * 1024 + threadIdx.x * 4;
    f32x4 H = *reinterpret_cast<const f32x4*>(at);
#pragma unroll 4
    for (int s = 1; s < w.count - 1; ++s) {
        at += step;
        const float d = p.decay[(w.slot0 + s) * p.slabs + slab];
        const f32x4 L = *reinterpret_cast<const f32x4*>(at);
#pragma unroll
        for (int r = 0; r < 4; ++r) H[r] = fmaf(d, H[r], L[r]);
        *reinterpret_cast<f32x4*>(at) = H;
    }
}

// A sequence is cut only where its blocks would leave half the chip's 256 units idle, into
// pieces of at least SEG_MIN chunks, for about BLOCKS_WANTED blocks.
constexpr int SEG_MIN = 4;
constexpr long long BLOCKS_WANTED = 512;

Plan plan_of(int B, int T, int H, int HV, int K, int V, int N, bool packed, int dtype) {
    Plan p;
    p.slabs = HV * (V / SLAB);
    p.ns = dtype == KDA_BF16 && (p.slabs / H) % 2 == 0 ? 2 : 1;
    p.units = p.slabs / p.ns;
    const long long chunks = (T + C - 1) / C;
    long long seg = chunks > 0 ? chunks : 1;   // chunks of a segment
    if (packed) {
        // lengths are on the device: bound a long sequence's piece by an even share of the rows
        const long long share = chunks * p.units / BLOCKS_WANTED;
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
    return p;
}

inline size_t slots_bytes(const Plan& p, int K) { return (size_t)p.slots * p.slabs * K * SLAB * sizeof(float); }

template <int K, bool FIRST> void launch_pass(const SsmArgs& a, const Plan& p, unsigned blocks) {
    if (a.dtype == KDA_F32)
        hipLaunchKernelGGL((ssm_scan_f32_kernel<K, FIRST>), dim3(blocks), dim3(256), 0, a.stream, a, p);
    else if (p.ns == 2)
        hipLaunchKernelGGL((ssm_scan_bf16_kernel<K, 2, FIRST>), dim3(blocks), dim3(256), 0, a.stream, a, p);
    else
        hipLaunchKernelGGL((ssm_scan_bf16_kernel<K, 1, FIRST>), dim3(blocks), dim3(256), 0, a.stream, a, p);
}

template <int K> hipError_t launch_k(const SsmArgs& a) {
    Plan p = plan_of(a.B, a.T, a.H, a.HV, K, a.V, a.N, a.cu_seqlens != nullptr, a.dtype);
    const long long first = p.slots * p.units, second = p.tiles * p.units;
    const long long join = p.slots > 0 ? (a.cu_seqlens ? p.slots : (long long)a.N) * p.slabs * (K * SLAB / 1024) : 0;
    if (first > 0x7fffffffLL || second > 0x7fffffffLL || join > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    if (p.slots > 0) {
        char* ws = static_cast<char*>(a.workspace);
        p.ends = reinterpret_cast<float*>(ws);
        if (a.final_state && a.final_state == a.initial_state) p.starts = reinterpret_cast<float*>(ws + slots_bytes(p, K));
        p.decay = reinterpret_cast<float*>(ws + 2 * slots_bytes(p, K));
        launch_pass<K, true>(a, p, (unsigned)first);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL((ssm_join_kernel<K>), dim3((unsigned)join), dim3(256), 0, a.stream, a, p);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (second > 0) launch_pass<K, false>(a, p, (unsigned)second);
    return hipGetLastError();
}

}  // namespace

size_t ssm_chunk_workspace(int B, int T, int H, int HV, int K, int V, int N, bool packed, int dtype) {
    const Plan p = plan_of(B, T, H, HV, K, V, N, packed, dtype);
    return 2 * slots_bytes(p, K) + (size_t)p.slots * p.slabs * sizeof(float);
}

hipError_t launch_ssm_chunk(const SsmArgs& a) { return a.K == 128 ? launch_k<128>(a) : launch_k<64>(a); }

}  // namespace kda
