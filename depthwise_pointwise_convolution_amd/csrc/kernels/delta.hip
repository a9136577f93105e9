// delta.hip -- gated delta rule: a head's state S, [Dk][Dv], is decayed by alpha, and what it answers for the
// key k is moved towards the value v by the rate beta:
//   S <- alpha S;  S <- S + beta k (v - k^T S)^T;  o = S^T q.
//
// Single tokens: one workgroup per sequence and head holds the whole state in registers, so it is read and
// written once.  With ks = k^T S and qs = q^T S of the old state, both sums over rows at once,
//   u = beta (v - alpha ks),  S <- alpha S + k u^T,  o = alpha qs + (q.k) u.
//
// Prompts: chunks of 64 tokens.  With G_i the product of alpha from the chunk's first token to its i-th,
//   (I + L) U = diag(beta) (V - diag(G) K S0),   L_ij = beta_i (k_i.k_j) G_i / G_j  for j < i
//   o_i = G_i S0^T q_i + sum_{j <= i} (G_i / G_j) (q_i.k_j) u_j
//   S   = G_last S0 + sum_j (G_last / G_j) k_j u_j^T.
// A first kernel finds, for all chunks at the same time, (I + L)^-1 diag(beta) and the weights of the u_j in o;
// a second one goes through each sequence's chunks in order with a slice of 16 NT columns of S in registers.
//
// Products run on the bf16 matrix instructions.  The state and all that is computed stay 32-bit values: one is
// fed as three bf16 pieces, each the nearest to what the ones before leave (2^-8 and 2^-16 of the value), 16-bit inputs
// as they are (fp16: two pieces, exactly).  Of three pieces by three, the products of a second with a third are left out,
// 2^-24 of the factors' product each and of either sign.  What only goes into 16-bit outputs (not into the state) has two
// pieces, and the product of both seconds is left out: with the missing thirds 3 * 2^-16 of the sum of the products'
// magnitudes at most, a tenth of what rounding the output to fp16 may take; with three, 4096 tokens of 16 heads took
// 160 us instead of 150, 8192 of 32 401 instead of 394.  (Cut pieces, which round towards zero, cost the same and left
// sums of positive products 1.4e-5 too small on average.)  Quotients G_i / G_j are exponentials of differences of sums
// held in 64 bits: in 32 the difference of two sums of a few hundred would be off by 2^-16.
#include <float.h>
#include <limits.h>

#include "mm_common.h"
#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

constexpr int kChunk = 64;  // tokens of a chunk
constexpr float kLog2e = 1.44269504f;

// bf16 pieces of an input, and of a computed value where it only goes into an output.
template <typename T>
struct Pieces {
    static constexpr int IN = sizeof(T) == 4 ? 3 : std::is_same<T, _Float16>::value ? 2 : 1;
    static constexpr int OUT = sizeof(T) == 4 ? 3 : 2;
};

// Eight values as N operands of eight bf16 pieces each: the nearest, that of the rest, and so on.  (From 2^128 - 2^119
// on a value's nearest is infinite.)
template <int N>
__device__ __forceinline__ void split8(const float* v, u32x4* out) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
    for (int p = 0; p < N; ++p) {
        typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf2 h = {(__bf16)r[2 * i], (__bf16)r[2 * i + 1]};
            const uint32_t u = __builtin_bit_cast(uint32_t, h);
            out[p][i] = u;
            if (p + 1 < N) {
                r[2 * i] -= __builtin_bit_cast(float, u << 16);
                r[2 * i + 1] -= __builtin_bit_cast(float, u & 0xffff0000u);
            }
        }
    }
}

// acc += A B over pieces: a[p] b[q] with p + q < KEEP.
template <int NA, int NB, int KEEP>
__device__ __forceinline__ f32x4 mm_pieces(const u32x4* a, const u32x4* b, f32x4 acc) {
#pragma unroll
    for (int s = KEEP - 1; s >= 0; --s)  // small ones first
#pragma unroll
        for (int p = 0; p < NA; ++p)
            if (s - p >= 0 && s - p < NB) acc = mfma<__bf16>(a[p], b[s - p], acc);
    return acc;
}

// The same from zero in two chains of half the length: a product that adds to the one before waits for it.
template <int NA, int NB, int KEEP>
__device__ __forceinline__ f32x4 mm_pieces2(const u32x4* a, const u32x4* b) {
    f32x4 acc[2] = {};
    int n = 0;
#pragma unroll
    for (int s = KEEP - 1; s >= 0; --s)
#pragma unroll
        for (int p = 0; p < NA; ++p)
            if (s - p >= 0 && s - p < NB) {
                acc[n & 1] = mfma<__bf16>(a[p], b[s - p], acc[n & 1]);
                ++n;
            }
    return acc[0] + acc[1];
}

// What the first kernel leaves for the second: for each chunk and key head the operands of K, Q (tokens x
// channels) and of K transposed, for each chunk and value head those of (I + L)^-1 diag(beta) and of the
// output's weights (their six lower pieces of 16 x 32), and the rows' factors.
constexpr int kFrag = 1024;  // bytes of an operand: 16 of each lane
struct Layout {
    long long kf, qf, kt, key_bytes;  // of a key head
    long long tf, pf, rows, head_bytes;
};
__host__ __device__ inline Layout layout(int pieces, int out, int nkb) {
    Layout l;
    const long long one = (long long)pieces * 4 * nkb * kFrag;
    l.kf = 0;
    l.qf = one;
    l.kt = 2 * one;
    l.key_bytes = 3 * one;
    l.tf = 0;
    l.pf = 3 * 6 * kFrag;
    l.rows = l.pf + out * 6 * kFrag;
    l.head_bytes = l.rows + 4 * kChunk * 4;  // (the fourth row holds G_last)
    return l;
}
// Operand of rows mt of four and columns kb of two, of those that are not all above the diagonal.
__host__ __device__ constexpr int lower(int mt, int kb) { return mt < 2 ? mt : 2 * mt - 2 + kb; }
// Token of row r of tile mt: chosen so that what two tiles' accumulators hold in a lane, four rows each, are
// the eight tokens of an operand over tokens.
__device__ __forceinline__ int tile_token(int mt, int r) {
    return 32 * (mt >> 1) + 8 * (r >> 2) + 4 * (mt & 1) + (r & 3);
}
// (channels of a tile of the state likewise)

// Chunks of sequence b start at this place: they fit, as ceil(n / 64) is at most one more than what n adds to
// the quotient.
__device__ __forceinline__ int first_chunk(const int32_t* cu, int b, int tokens) {
    return seq_offset(cu, b, tokens) / kChunk + b;
}

template <typename T>
__device__ __forceinline__ float rate_of(T b) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f((float)b * -kLog2e));
}

// log2 of a step's decay.  A step of zero keeps the state whatever the rate; beyond 2^-16384 and 2^16384 every
// power is zero or infinite, and the bound keeps differences of sums from being NaN.
template <typename T>
__device__ __forceinline__ double log_decay(T a, float dt_bias, float A, int soft) {
    float d = (float)a + dt_bias;
    if (soft) d = softplus(d);
    const double p = d == 0.0f ? 0.0 : (double)d * (double)A * 1.4426950408889634;
    return p < -16384.0 ? -16384.0 : p > 16384.0 ? 16384.0 : p;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {  // 16-byte aligned
    if constexpr (sizeof(T) == 4) {
        unpack16<T>(ld16(p), v);
        unpack16<T>(ld16(p + 4), v + 4);
    } else {
        unpack16<T>(ld16(p), v);
    }
}
// Operand pieces of eight inputs.
template <typename T>
__device__ __forceinline__ void input_pieces(const T* p, u32x4* out) {
    if constexpr (Pieces<T>::IN == 1) {
        out[0] = ld16(p);
    } else {
        float v[8];
        load8<T>(p, v);
        split8<Pieces<T>::IN>(v, out);
    }
}

// An operand's store, whose registers an LDS read right behind it may not yet overwrite.
__device__ __forceinline__ void st_operand(char* p, u32x4 v) {
    st16(p, v);
    asm volatile("s_nop 0" ::: "memory");
}

// One workgroup per chunk and key head.  What is written bounds it: for 8192 tokens of 16 key heads and 32 value heads of
// 128 channels 225 MB (and 100 MB read) in 85 us, 3.8 TB/s; where there are few workgroups it is the latency of one, 26 us.
// The value heads' decays are summed four heads at a time, a wave each, while the rows are under way.
template <typename T, int NKB>
__global__ __launch_bounds__(256, 4) void delta_prep_kernel(DeltaArgs a) {
    constexpr int PI = Pieces<T>::IN, PQ = Pieces<T>::OUT, DK = 32 * NKB, LD = DK + 8, LM = 68;
    constexpr int kIn = 2 * kChunk * LD * (int)sizeof(T), kMat = 2 * kChunk * LM * 4;
    __shared__ __attribute__((aligned(16))) char smem[kIn > kMat ? kIn : kMat];
    __shared__ double alongs[4][kChunk];  // of four value heads, a wave each
    __shared__ float betas[4][kChunk], rq[kChunk], rk[kChunk];
    T* in = (T*)smem;             // q rows, then k rows
    float* m1 = (float*)smem;     // (after their last use) output weights, then L
    float* m2 = m1 + kChunk * LM; // its inverse
    const int hk = blockIdx.x % a.Hk, id = blockIdx.x / a.Hk;
    // the sequence whose chunks begin last at or before this place
    int b = 0;
    for (int span = a.seqs; span > 1;) {
        const int half = span / 2;
        if (first_chunk(a.cu, b + half, a.tokens) <= id) b += half;
        span -= half;
    }
    const int t0 = seq_offset(a.cu, b, a.tokens) + (id - first_chunk(a.cu, b, a.tokens)) * kChunk;
    const int end = seq_offset(a.cu, b + 1, a.tokens);
    if (id < first_chunk(a.cu, b, a.tokens) || t0 >= end) return;
    if (end - seq_offset(a.cu, b, a.tokens) <= a.shortest) return;
    const int n = end - t0 < kChunk ? end - t0 : kChunk;
    const int tid = threadIdx.x, lane = tid & 63, sub = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Layout lay = layout(PI, PQ, NKB);
    const long long place = id;
    char* key = (char*)a.ws + (place * a.Hk + hk) * lay.key_bytes;
    char* heads = (char*)a.ws + a.places * a.Hk * lay.key_bytes;

    // decays from the chunk's start and rates of head h0 + wave
    const int share = a.Hv / a.Hk;
    T ga, gb;
    auto load_steps = [&](int h0) {
        const bool in = h0 + wave < (hk + 1) * share && lane < n;
        ga = in ? ((const T*)a.a)[(t0 + lane) * a.lda + h0 + wave] : (T)0.0f;
        gb = in ? ((const T*)a.b)[(t0 + lane) * a.ldb + h0 + wave] : (T)0.0f;
    };
    auto add_steps = [&](int h0) {
        const int h = h0 + wave;
        if (h >= (hk + 1) * share) return;
        double p = lane < n ? log_decay(ga, a.dt_bias ? a.dt_bias[h] : 0.0f, a.A[h], a.softplus) : 0.0;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double v = __shfl_up(p, o);
            if (lane >= o) p += v;
        }
        alongs[wave][lane] = p;
        betas[wave][lane] = lane < n ? rate_of(gb) : 0.0f;
    };
    load_steps(hk * share);

    // rows into LDS, zero behind the sequence and behind the last channel
    constexpr int VE = Vec<T>::N;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        const T* src = (const T*)(part ? a.k : a.q) + (long long)hk * a.Dk;
        const long long ld = part ? a.ldk : a.ldq;
        T* dst = in + part * kChunk * LD;
        const bool wide = part ? a.wide_k : a.wide_q;
        if (wide) {
            for (int i = tid; i < kChunk * (DK / VE); i += 256) {
                const int t = i / (DK / VE), c = i % (DK / VE) * VE;
                u32x4 v = {};
                if (t < n && c < a.Dk) v = ld16(src + (t0 + t) * ld + c);
                st16(dst + t * LD + c, v);
            }
        } else {
            for (int i = tid; i < kChunk * DK; i += 256) {
                const int t = i / DK, c = i % DK;
                dst[t * LD + c] = t < n && c < a.Dk ? src[(t0 + t) * ld + c] : (T)0.0f;
            }
        }
    }
    add_steps(hk * share);
    __syncthreads();
    // the rows' norms: four lanes a row
    {
        float s[2] = {0.0f, 0.0f};
        const int t = tid >> 2;
        for (int c = (tid & 3) * 8; c < DK; c += 32)
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                float v[8];
                load8<T>(in + (part * kChunk + t) * LD + c, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[part] = __builtin_fmaf(v[i], v[i], s[part]);
            }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            s[part] += __shfl_xor(s[part], 1);
            s[part] += __shfl_xor(s[part], 2);
        }
        if ((tid & 3) == 0) {
            rq[t] = a.scale * (a.qk_norm ? 1.0f / __builtin_sqrtf(s[0] + a.eps) : 1.0f);
            rk[t] = a.qk_norm ? 1.0f / __builtin_sqrtf(s[1] + a.eps) : 1.0f;
        }
    }
    // operands of q and k as they are
    const T* qs = in;
    const T* ks = in + kChunk * LD;
    for (int kb = 0; kb < NKB; ++kb) {
        const int at = tile_token(wave, sub) * LD + 32 * kb + 8 * grp;
        u32x4 f[PI];
        input_pieces<T>(ks + at, f);
#pragma unroll
        for (int p = 0; p < PI; ++p)
            st_operand(key + lay.kf + ((p * 4 + wave) * NKB + kb) * kFrag + lane * 16, f[p]);
        input_pieces<T>(qs + at, f);
#pragma unroll
        for (int p = 0; p < PI; ++p)
            st_operand(key + lay.qf + ((p * 4 + wave) * NKB + kb) * kFrag + lane * 16, f[p]);
    }
    // and of k transposed: tile s of channels, tokens 32 * kb ..
    for (int s = wave; s < 2 * NKB; s += 4)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int c = 32 * (s >> 1) + 8 * (sub >> 2) + 4 * (s & 1) + (sub & 3);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)ks[(32 * kb + 8 * grp + e) * LD + c];
            u32x4 f[PI];
            split8<PI>(v, f);
#pragma unroll
            for (int p = 0; p < PI; ++p)
                st_operand(key + lay.kt + ((p * 2 * NKB + s) * 2 + kb) * kFrag + lane * 16, f[p]);
        }
    // k.k and q.k of the tiles on and below the diagonal: wave w has rows 16 w ..
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{};
    for (int kb = 0; kb < NKB; ++kb) {
        const int c = 32 * kb + 8 * grp;
        u32x4 fq[PI], fk[PI];
        input_pieces<T>(qs + (16 * wave + sub) * LD + c, fq);
        input_pieces<T>(ks + (16 * wave + sub) * LD + c, fk);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wave) {
                u32x4 fb[PI];
                input_pieces<T>(ks + (16 * j + sub) * LD + c, fb);
                kk[j] = mm_pieces<PI, PI, 3>(fk, fb, kk[j]);
                qk[j] = mm_pieces<PI, PI, PQ>(fq, fb, qk[j]);
            }
    }
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        char* head = heads + (place * a.Hv + h) * lay.head_bytes;
        const int hi = (h - hk * share) & 3;
        __syncthreads();  // (the rows in LDS, or the last head's matrices, are done with)
        if (hi == 0 && h > hk * share) {
            load_steps(h);
            add_steps(h);
            __syncthreads();
        }
        const double* along = alongs[hi];
        const float* beta = betas[hi];
        if (wave == 1) {
            const double p = along[lane], last = along[kChunk - 1];
            const float grown = __builtin_amdgcn_exp2f((float)p);
            float* rows = (float*)(head + lay.rows);
            rows[lane] = grown * rk[lane];
            rows[kChunk + lane] = grown * rq[lane];
            rows[2 * kChunk + lane] = __builtin_amdgcn_exp2f((float)(last - p)) * rk[lane];
            if (lane == 0) rows[3 * kChunk] = __builtin_amdgcn_exp2f((float)last);
        }
        f32x4 low[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wave) {
                const int col = 16 * j + sub;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * wave + 4 * grp + i;
                    const float d = __builtin_amdgcn_exp2f((float)(along[row] - along[col]));
                    low[j][i] = col < row ? kk[j][i] * (beta[row] * rk[row] * rk[col]) * d : 0.0f;
                    m1[row * LM + col] = col <= row ? qk[j][i] * (rq[row] * rk[col]) * d : 0.0f;
                }
            }
        __syncthreads();
        // operand pieces of a lower matrix: rows of tile `wave`, with a factor for each column
        auto emit = [&](const float* m, const float* by, char* to, auto pieces) {
            constexpr int N = decltype(pieces)::value;
            const int row = tile_token(wave, sub);
            for (int kb = 0; kb <= (wave >> 1); ++kb) {
                const int col = 32 * kb + 8 * grp;
                float v[8];
                unpack16<float>(ld16(m + row * LM + col), v);
                unpack16<float>(ld16(m + row * LM + col + 4), v + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = col + e <= row ? v[e] * (by ? by[col + e] : 1.0f) : 0.0f;
                u32x4 f[N];
                split8<N>(v, f);
#pragma unroll
                for (int p = 0; p < N; ++p)
                    st_operand(to + (p * 6 + lower(wave, kb)) * kFrag + lane * 16, f[p]);
            }
        };
        emit(m1, nullptr, head + lay.pf, std::integral_constant<int, PQ>());
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wave)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    m1[(16 * wave + 4 * grp + i) * LM + 16 * j + sub] = low[j][i];
        __builtin_amdgcn_wave_barrier();
        // The inverse of I + L.  Blocks of 16 on the diagonal by substitution, a column in each of 16 lanes;
        // below them  T_ij = -T_ii sum_m L_im T_mj, column by column, one wave each, in 32-bit products.
        {
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float v = r == sub ? 1.0f : 0.0f;
#pragma unroll
                for (int m = 0; m < r; ++m)
                    v = __builtin_fmaf(-m1[(16 * wave + r) * LM + 16 * wave + m], x[m], v);
                x[r] = v;
            }
            if (lane < 16)
#pragma unroll
                for (int r = 0; r < 16; ++r) m2[(16 * wave + r) * LM + 16 * wave + sub] = x[r];
        }
        __syncthreads();
        for (int i = wave + 1; i < 4; ++i) {
            f32x4 x = {};
            for (int m = wave; m < i; ++m)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    x = __builtin_amdgcn_mfma_f32_16x16x4f32(
                        m1[(16 * i + sub) * LM + 16 * m + 4 * s + grp],
                        m2[(16 * m + 4 * s + grp) * LM + 16 * wave + sub], x, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) m2[(16 * i + 4 * grp + e) * LM + 16 * wave + sub] = x[e];
            __builtin_amdgcn_wave_barrier();
            f32x4 y = {};
#pragma unroll
            for (int s = 0; s < 4; ++s)
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(
                    m2[(16 * i + sub) * LM + 16 * i + 4 * s + grp],
                    m2[(16 * i + 4 * s + grp) * LM + 16 * wave + sub], y, 0, 0, 0);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int e = 0; e < 4; ++e) m2[(16 * i + 4 * grp + e) * LM + 16 * wave + sub] = -y[e];
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();
        emit(m2, beta, head + lay.tf, std::integral_constant<int, 3>());
    }
}

// N neighbouring columns of a state's row, from `c` on; behind the last any (what is computed with them is not stored).
template <int N>
__device__ __forceinline__ void load_state(const float* row, int c, int most, bool wide, float* out) {
    if (N == 2 && wide) {  // (an even number of columns)
        const float2 v = *(const float2*)(row + (c < most ? c : most - 2));
        out[0] = v.x;
        out[N - 1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = row[c + i < most ? c + i : most - 1];
    }
}
template <int N>
__device__ __forceinline__ void store_state(float* row, int c, int most, bool wide, const float* in) {
    if (N == 2 && wide) {
        if (c < most) *(float2*)(row + c) = float2{in[0], in[N - 1]};
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < most) row[c + i] = in[i];
    }
}

// A lane's four rows of a chunk and N neighbouring columns of a tensor of tokens.  The chunk's rows are a range of
// their own: what is behind the last row reads as zero and is not stored, and a column behind the last has no place.
template <typename T, int N>
struct ChunkRows {
    uint32_t at[N], step;
    uint32_t row;  // bytes from the head's first row
    const char* base;
    long long ld;
    bool wide;
    __device__ __forceinline__ ChunkRows(const void* p, long long ld_, long long column, int col, int most, int tok, bool wide_) {
        base = (const char*)p + column * (long long)sizeof(T);
        ld = ld_ * (long long)sizeof(T);
        step = (uint32_t)ld;
        wide = wide_;
#pragma unroll
        for (int i = 0; i < N; ++i)
            at[i] = col + i < most ? (uint32_t)tok * step + (uint32_t)(col + i) * (uint32_t)sizeof(T) : mm::kOob;
        row = (uint32_t)most * (uint32_t)sizeof(T);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t range(int t0, int end) const {
        const int n = end - t0 < kChunk ? end - t0 : kChunk;
        return mm::rsrc(base + t0 * ld, (uint32_t)(n - 1) * step + row);
    }
    __device__ __forceinline__ void load(int t0, int end, T (&v)[4][N]) const {
        const __amdgpu_buffer_rsrc_t r = range(t0, end);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (N == 2 && wide) {
                if constexpr (sizeof(T) == 4) {
                    const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(r, at[0], i * step, 0);
                    // (a bit cast of a vector's element takes the first one)
                    const uint32_t low = x[0], high = x[1];
                    v[i][0] = __builtin_bit_cast(T, low), v[i][N - 1] = __builtin_bit_cast(T, high);
                } else {
                    const uint32_t x = __builtin_amdgcn_raw_buffer_load_b32(r, at[0], i * step, 0);
                    v[i][0] = __builtin_bit_cast(T, (uint16_t)x), v[i][N - 1] = __builtin_bit_cast(T, (uint16_t)(x >> 16));
                }
            } else {
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    if constexpr (sizeof(T) == 4)
                        v[i][t] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, at[t], i * step, 0));
                    else
                        v[i][t] = __builtin_bit_cast(T, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at[t], i * step, 0));
                }
            }
        }
    }
    __device__ __forceinline__ void store(int t0, int end, const f32x4 (&o)[N]) const {
        const __amdgpu_buffer_rsrc_t r = range(t0, end);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (N == 2 && wide) {
                const T x = (T)o[0][i], y = (T)o[N - 1][i];
                if constexpr (sizeof(T) == 4)
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)}, r, at[0], i * step, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16, r, at[0], i * step, 0);
            } else {
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    const T x = (T)o[t][i];
                    if constexpr (sizeof(T) == 4)
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), r, at[t], i * step, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, x), r, at[t], i * step, 0);
                }
            }
        }
    }
};

// The sum of a row of 16 lanes, in each of them.
__device__ __forceinline__ float sum16(float v) {
#define FCM_DPP_ADD(ctrl)                                                                         \
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, 0xf, 0xf, true))
    FCM_DPP_ADD(0xb1);   // neighbours of a pair, of a quad, the halves of eight, of sixteen
    FCM_DPP_ADD(0x4e);
    FCM_DPP_ADD(0x141);
    FCM_DPP_ADD(0x140);
#undef FCM_DPP_ADD
    return v;
}

// The i-th sequence of more than `shortest` tokens, or -1.
__device__ __forceinline__ int long_sequence(const int32_t* cu, int seqs, int tokens, int shortest, int i) {
    if (shortest < 0) return i;
    const int lane = threadIdx.x & 63;
    for (int b = 0; b < seqs; b += 64) {
        const bool in = b + lane < seqs &&
                        seq_offset(cu, b + lane + 1, tokens) - seq_offset(cu, b + lane, tokens) > shortest;
        uint64_t who = __ballot(in);
        const int n = __popcll(who);
        if (i < n) {
            for (; i > 0; --i) who &= who - 1;
            return b + __ffsll((unsigned long long)who) - 1;
        }
        i -= n;
    }
    return -1;
}
// More tokens than `shortest` have at most so many sequences.
int long_sequences(int seqs, int tokens, int shortest) {
    return shortest < 0 || seqs < tokens / (shortest + 1) ? seqs : tokens / (shortest + 1);
}

// One workgroup per sequence, value head and slice of 16 NT columns, NT neighbouring ones a lane.
//
// A chunk is a chain: the state as an operand, what the values differ by, U, the new state, each through LDS.  Four
// waves do only that: wave w has the tokens of tile w of each chunk and the state's channels of k-blocks w, w + 4.
// Four more have the same tokens' outputs, from the same state and U, beside it.  What a wave reads of the next
// chunk is loaded as soon as this one is done with the registers.
//
// The chain's latency bounds it: 16 heads of one sequence take 1.6 us a chunk (2.9 with all of it on four waves), 8192
// tokens of 32 heads of 128 channels 250 us, 3.8 us a chunk of one workgroup a CU, where its products are 0.75 us: the
// matrix units are busy in 21% of its cycles, LDS in 24%, and its waves wait for results in 46% of theirs.
template <typename T, int NKB, int NT>
__global__ __launch_bounds__(512) void delta_chunks_kernel(DeltaArgs a, int slices) {
    constexpr int PI = Pieces<T>::IN, PQ = Pieces<T>::OUT, KW = (NKB + 3) / 4;
    __shared__ u32x4 sb[NKB][NT][PQ][64];  // the state as an operand over channels
    __shared__ f32x4 parts[4][4][NT][64];  // k S of each wave's channels, by tiles of tokens
    __shared__ u32x4 rb[2][NT][3][64];    // what the values differ by, over tokens
    __shared__ u32x4 ub[2][NT][PQ][64];   // U
    __shared__ u32x4 ud[2][NT][3][64];    // U with the decay to the chunk's end
    const int tid = threadIdx.x, lane = tid & 63, sub = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
    const bool outputs = __builtin_amdgcn_readfirstlane(tid >> 6) >= 4;
    // the slices of a head, which read the same operands, go to one XCD
    const int xcd = blockIdx.x & 7, rest = blockIdx.x >> 3;
    const int slice = rest % slices, bh = (rest / slices) * 8 + xcd;
    const int b = bh < a.seqs * a.Hv ? long_sequence(a.cu, a.seqs, a.tokens, a.shortest, bh / a.Hv) : -1;
    if (b < 0) return;
    const int h = bh % a.Hv, hk = h / (a.Hv / a.Hk);
    const int start = seq_offset(a.cu, b, a.tokens), end = seq_offset(a.cu, b + 1, a.tokens);
    const Layout lay = layout(PI, PQ, NKB);
    const int col = (slice * 16 + sub) * NT;
    const long long hv = (long long)h * a.Dv;
    const int tok = 32 * (wave >> 1) + 8 * grp + 4 * (wave & 1);  // this lane's tokens of a chunk: .. + i
    const long long key_step = a.Hk * lay.key_bytes, head_step = a.Hv * lay.head_bytes;
    const int first = first_chunk(a.cu, b, a.tokens);
    const char* key = (const char*)a.ws + first * key_step + hk * lay.key_bytes;
    const char* head = (const char*)a.ws + a.places * key_step + first * head_step + h * lay.head_bytes;
    // the lower operands of tile `wave`: columns that lie above the first tiles' rows read as zero
    auto lower_operand = [&](const __amdgpu_buffer_rsrc_t& r, long long from, int p, int kb) {
        return __builtin_amdgcn_raw_buffer_load_b128(
            r, kb <= (wave >> 1) ? (int)(from + (p * 6 + lower(wave, kb)) * kFrag + lane * 16) : (int)mm::kOob, 0, 0);
    };

    if (outputs) {
        const bool gate = !a.norm && a.z;
        const ChunkRows<T, NT> ys(a.y, a.ldy, hv, col, a.Dv, tok, a.wide_y), zs(a.z, a.ldz, hv, col, a.Dv, tok, a.wide_z);
        const ChunkRows<float, NT> os(a.outs, (long long)a.Hv * a.Dv, hv, col, a.Dv, tok, a.Dv % 2 == 0);
        u32x4 q[NKB][PI], pw[2][PQ];
        f32x4 seen;
        T z[4][NT];
        auto load_q = [&]() {
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                for (int p = 0; p < PI; ++p) q[kb][p] = ld16(key + lay.qf + ((p * 4 + wave) * NKB + kb) * kFrag + lane * 16);
            seen = *(const f32x4*)((const float*)(head + lay.rows) + kChunk + tok);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto load_weights = [&](int t0) {
            const __amdgpu_buffer_rsrc_t rh = mm::rsrc(head, (uint32_t)lay.head_bytes);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int p = 0; p < PQ; ++p) pw[kb][p] = lower_operand(rh, lay.pf, p, kb);
            if (gate) zs.load(t0, end, z);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (start < end) {
            load_q();
            load_weights(start);
        }
        for (int t0 = start; t0 < end; t0 += kChunk) {
            // (behind the last chunk it is loaded once more)
            const bool more = t0 + kChunk < end;
            key += more ? key_step : 0;
            head += more ? head_step : 0;
            __syncthreads();
            __syncthreads();
            f32x4 o[NT];
            // (in the chain's second part: in the first it reads more of LDS itself)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                u32x4 f[NKB][PQ];
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                    for (int p = 0; p < PQ; ++p) f[kb][p] = sb[kb][t][p][lane];
                __builtin_amdgcn_sched_barrier(0);
                o[t] = f32x4{};
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) o[t] = mm_pieces<PI, PQ, PQ>(q[kb], f[kb], o[t]);
                o[t] *= seen;
            }
            load_q();
            __syncthreads();
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                u32x4 f[2][PQ];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int p = 0; p < PQ; ++p) f[kb][p] = ub[kb][t][p][lane];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) o[t] = mm_pieces<PQ, PQ, PQ>(pw[kb], f[kb], o[t]);
            }
            if (gate)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][i] *= silu((float)z[i][t]);
            load_weights(more ? t0 + kChunk : t0);
            if (a.norm) {
                float squares[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = 0.0f;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (col + t < a.Dv) v = __builtin_fmaf(o[t][i], o[t][i], v);
                    squares[i] = sum16(v);
                }
                float* to = a.squares + ((long long)(t0 + tok) * a.Hv + h) * slices + slice;
                if (sub == 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + tok + i < end) to[(long long)i * a.Hv * slices] = squares[i];
            }
            if (a.norm && sizeof(T) < 4)
                os.store(t0, end, o);
            else
                ys.store(t0, end, o);
        }
        return;
    }

    const int slot = a.state ? seq_slot(a.slots, b, a.nslots) : -1;
    float* state = slot >= 0 ? a.state + ((long long)slot * a.Hv + h) * a.Dk * a.Dv : nullptr;
    const bool carried = state && a.carry && a.carry[b] != 0;
    // channel of row r = 4 grp + i of tile half hf of k-block kb: 32 kb + 8 grp + 4 hf + i
    f32x4 S[KW][2][NT];
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 32 * (wave + 4 * k) + 8 * grp + 4 * hf + i;
                float v[NT] = {};
                if (carried && c < a.Dk) load_state<NT>(state + (long long)c * a.Dv, col, a.Dv, a.wide_state, v);
#pragma unroll
                for (int t = 0; t < NT; ++t) S[k][hf][t][i] = v[t];
            }
        }
    // (here, or the loop would wait for its own loads too)
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(S[k][hf][t]));
    const ChunkRows<T, NT> vs(a.v, a.ldv, hv, col, a.Dv, tok, a.wide_v);
    u32x4 kf[4][KW][PI], kt[KW][2][2][PI], tw[2][3];
    f32x4 known, left;  // the rows' factors
    float last;
    T v[4][NT];
    // (the compiler would move the loads to their use)
    auto load_k = [&](int t0) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int k = 0; k < KW; ++k)
#pragma unroll
                for (int p = 0; p < PI; ++p) {
                    // (a wave without channels has nothing to do with these: any will do)
                    const int kb = wave + 4 * k < NKB ? wave + 4 * k : 0;
                    kf[m][k][p] = ld16(key + lay.kf + ((p * 4 + m) * NKB + kb) * kFrag + lane * 16);
                }
        known = *(const f32x4*)((const float*)(head + lay.rows) + tok);
        vs.load(t0, end, v);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto load_inverse = [&]() {
        const __amdgpu_buffer_rsrc_t rh = mm::rsrc(head, (uint32_t)lay.head_bytes);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int p = 0; p < 3; ++p) tw[kb][p] = lower_operand(rh, lay.tf, p, kb);
        left = *(const f32x4*)((const float*)(head + lay.rows) + 2 * kChunk + tok);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto load_kt = [&]() {
#pragma unroll
        for (int k = 0; k < KW; ++k)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int p = 0; p < PI; ++p) {
                        // (a wave without channels has nothing to do with these: any will do)
                        const int s = wave + 4 * k < NKB ? 2 * (wave + 4 * k) + hf : 0;
                        kt[k][hf][kb][p] = ld16(key + lay.kt + ((p * 2 * NKB + s) * 2 + kb) * kFrag + lane * 16);
                    }
        last = ((const float*)(head + lay.rows))[3 * kChunk];
        __builtin_amdgcn_sched_barrier(0);
    };
    if (start < end) {
        load_k(start);
        load_inverse();
        load_kt();
    }
    for (int t0 = start; t0 < end; t0 += kChunk) {
        const bool more = t0 + kChunk < end;
        key += more ? key_step : 0;
        head += more ? head_step : 0;
        // (the column tiles beside each other: their products wait for none of each other's)
        {
            u32x4 f[NT][KW][3];
            f32x4 ks[NT][4] = {};
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = S[k][i >> 2][t][i & 3];
                    split8<3>(x, f[t][k]);
                }
#pragma unroll
            for (int s = 2; s >= 0; --s)
#pragma unroll
                for (int k = 0; k < KW; ++k)
#pragma unroll
                    for (int p = 0; p < PI; ++p)
                        if (s - p >= 0)
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int m = 0; m < 4; ++m) ks[t][m] = mfma<__bf16>(kf[m][k][p], f[t][k][s - p], ks[t][m]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int m = 0; m < 4; ++m) parts[wave][m][t][lane] = ks[t][m];
#pragma unroll
                for (int k = 0; k < KW; ++k)
                    if (NKB % 4 == 0 || wave + 4 * k < NKB)
#pragma unroll
                        for (int p = 0; p < PQ; ++p) sb[wave + 4 * k][t][p][lane] = f[t][k][p];
            }
        }
        __syncthreads();
        // (all reads, then what follows: the compiler would wait for each)
        f32x4 ks[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int w = 0; w < 4 && w < NKB; ++w) ks[t][w] = parts[w][wave][t][lane];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float r[8] = {};
#pragma unroll
            for (int w = 1; w < 4 && w < NKB; ++w) ks[t][0] += ks[t][w];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __builtin_fmaf(-known[i], ks[t][0][i], (float)v[i][t]);
            u32x4 g[3];
            split8<3>(r, g);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *(u32x2*)((char*)&rb[wave >> 1][t][p][lane] + 8 * (wave & 1)) = u32x2{g[p][0], g[p][1]};
        }
        load_k(more ? t0 + kChunk : t0);
        __syncthreads();
        f32x4 us[NT];
        {
            u32x4 f[NT][2][3];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int p = 0; p < 3; ++p) f[t][kb][p] = rb[kb][t][p][lane];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                us[t] = mm_pieces2<3, 3, 3>(tw[0], f[t][0]) + mm_pieces2<3, 3, 3>(tw[1], f[t][1]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 u = us[t];
            float x[8] = {}, w[8] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = u[i];
                w[i] = u[i] * left[i];
            }
            u32x4 g[3];
            split8<3>(w, g);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *(u32x2*)((char*)&ud[wave >> 1][t][p][lane] + 8 * (wave & 1)) = u32x2{g[p][0], g[p][1]};
            split8<PQ>(x, g);
#pragma unroll
            for (int p = 0; p < PQ; ++p)
                *(u32x2*)((char*)&ub[wave >> 1][t][p][lane] + 8 * (wave & 1)) = u32x2{g[p][0], g[p][1]};
        }
        load_inverse();
        __syncthreads();
        {
            u32x4 f[NT][2][3];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int p = 0; p < 3; ++p) f[t][kb][p] = ud[kb][t][p][lane];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < KW; ++k)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        S[k][hf][t] = mm_pieces<PI, 3, 3>(kt[k][hf][0], f[t][0], S[k][hf][t] * last) +
                                      mm_pieces<PI, 3, 3>(kt[k][hf][1], f[t][1], f32x4{});
        }
        load_kt();
    }
    if (!state) return;
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 32 * (wave + 4 * k) + 8 * grp + 4 * hf + i;
                float x[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t] = S[k][hf][t][i];
                if (c < a.Dk) store_state<NT>(state + (long long)c * a.Dv, col, a.Dv, a.wide_state, x);
            }
}

// The output's norm and gate: the second kernel left the outputs in 32 bits (in the workspace, or in y where that has
// them) and its slices their sums of squares, a negative one the short sequences' kernel, which has done it all.  A group
// of `width` lanes has kNormRows rows of heads, one after the other in memory, whose loads are all under way before the
// first is used.  HBM bounds it: 8192 tokens of 32 heads of 128 channels in bf16, 268 MB, in 55 us, 4.9 TB/s.  z is read and
// y written without a place in the caches, which leaves it to the outputs (with one: 61 us).  Outputs in the storage type would
// be 67 MB less to read, but a second rounding, and infinite above fp16's largest number though the norm brings them to 1.
constexpr int kNormRows = 4;
template <typename T, bool WIDE, bool ASK>
__global__ __launch_bounds__(256) void delta_norm_kernel(DeltaArgs a, int slices, int width) {
    constexpr int VE = Vec<T>::N;
    const int x = threadIdx.x & (width - 1), groups = 256 / width;
    // (tokens * Hv is below 2^26, or the launch would not be)
    const uint32_t first = (uint32_t)blockIdx.x * (groups * kNormRows) + threadIdx.x / width;
    const int from = seq_offset(a.cu, 0, a.tokens), to = seq_offset(a.cu, a.seqs, a.tokens);
    T* y[kNormRows];
    const float* o[kNormRows];
    u32x4 vo[kNormRows][VE / 4], vz[kNormRows];
    float s[kNormRows], norm[VE];
    bool live[kNormRows];
    const int c = x * VE;  // (WIDE: a row has no more vectors than lanes)
#pragma unroll
    for (int r = 0; r < kNormRows; ++r) {
        const uint32_t id = first + r * groups;
        const long long t = id / (uint32_t)a.Hv;
        const int h = id - (uint32_t)t * a.Hv;
        live[r] = t >= from && t < to;
        if (ASK) live[r] = live[r] && !(a.squares[(long long)id * slices] < 0.0f);
        if (!live[r]) continue;
        y[r] = (T*)a.y + t * a.ldy + (long long)h * a.Dv;
        o[r] = sizeof(T) < 4 ? a.outs + (long long)id * a.Dv : (const float*)y[r];
        if (WIDE && c < a.Dv) {
#pragma unroll
            for (int i = 0; i < VE / 4; ++i) vo[r][i] = ld16(o[r] + c + 4 * i);
            if (a.z) vz[r] = __builtin_nontemporal_load((const u32x4*)((const T*)a.z + t * a.ldz + (long long)h * a.Dv + c));
        }
        s[r] = a.squares[(long long)id * slices];
        if (s[r] < 0.0f) live[r] = false;
        for (int i = 1; i < slices; ++i) s[r] += a.squares[(long long)id * slices + i];
    }
    if (WIDE && c < a.Dv)
#pragma unroll
        for (int i = 0; i < VE; ++i) norm[i] = a.norm[c + i];
#pragma unroll
    for (int r = 0; r < kNormRows; ++r) {
        if (!live[r]) continue;
        const float f = 1.0f / __builtin_sqrtf(s[r] / (float)a.Dv + a.eps);
        if constexpr (WIDE) {
            if (c >= a.Dv) continue;
            float v[VE], g[VE];
#pragma unroll
            for (int i = 0; i < VE / 4; ++i) unpack16<float>(vo[r][i], v + 4 * i);
            if (a.z) unpack16<T>(vz[r], g);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                v[i] *= f * norm[i];
                if (a.z) v[i] *= silu(g[i]);
            }
            __builtin_nontemporal_store(pack16<T>(v), (u32x4*)(y[r] + c));
        } else {
            const uint32_t id = first + r * groups;
            const long long t = id / (uint32_t)a.Hv;
            const int h = id - (uint32_t)t * a.Hv;
            const T* z = a.z ? (const T*)a.z + t * a.ldz + (long long)h * a.Dv : nullptr;
            for (int i = x; i < a.Dv; i += width) {
                float v = o[r][i] * f * a.norm[i];
                if (z) v *= silu((float)z[i]);
                y[r][i] = (T)v;
            }
        }
    }
}

// Tokens one after the other, with the state in registers: the single-token call, and sequences of up to kShort tokens
// (drafted ones, a prompt's last few) among prompts, for which chunks would read and write 100 KB of operands a head.
//
// A workgroup has a sequence and a head, a wave 16 columns of its state: lane l has rows RPL * (l % 16) .. of four columns
// from 4 * (l / 16) on, so that sums over rows stay within 16 lanes and no wave waits for another.  (With rows over the
// waves and their sums through LDS, 32 sequences of 5 tokens took 62 us.)  Outputs wait in LDS for the norm, which is over all
// columns.  HBM bounds single tokens: 256 of them with 32 states of 128 x 128, 1.1 GB, take 221 us, 4.9 TB/s; behind a few
// tokens the vector units do, 1100 cycles a token and wave.  RPL is what a head's rows need, so that none of a small
// head's lanes is idle; 16 rows take twice the registers, so their workgroups have at most eight waves.
//
// 32 sequences of 32 heads, us, here / as chunks: of 5 tokens 57 / 169, of 16 105 / 170, of 24 144 / 140, of 32 184 / 139;
// 8 of 8 heads in 32 bits: of 5 tokens 24 / 39, of 16 39 / 39, of 32 66 / 40.
constexpr int kShort = 16;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
// N elements of a row from c on, zero behind the last; they stay in the storage type until they are used.  (A vector
// access from any element's address is one instruction.)
template <typename T, int N>
__device__ __forceinline__ vec_t<T, N> load_some(const T* p, int c, int most) {
    constexpr int VN = N * sizeof(T) < 16 ? N : 16 / sizeof(T);
    typedef vec_t<T, VN> V __attribute__((aligned(sizeof(T))));
    vec_t<T, N> out = {};
#pragma unroll
    for (int i = 0; i < N; i += VN) {
        if (c + i + VN <= most) {
            const V v = *(const V*)(p + c + i);
#pragma unroll
            for (int j = 0; j < VN; ++j) out[i + j] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < VN; ++j)
                if (c + i + j < most) out[i + j] = p[c + i + j];
        }
    }
    return out;
}

template <typename T, int RPL>
__global__ __launch_bounds__(RPL == 16 ? 512 : 1024) void delta_tokens_kernel(DeltaArgs a, int slices) {
    __shared__ float outs[kShort][256], squares[kShort][16];
    const int tid = threadIdx.x, lane = tid & 63, rg = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
    const int b = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, hk = h / (a.Hv / a.Hk);
    const int start = a.cu ? seq_offset(a.cu, b, a.tokens) : b;
    const int n = a.cu ? seq_offset(a.cu, b + 1, a.tokens) - start : 1;
    if (n > kShort) return;
    const long long hv = (long long)h * a.Dv;
    const int slot = a.state ? seq_slot(a.slots, b, a.nslots) : -1;
    if (!a.cu && slot < 0) {  // an idle row
        for (int c = tid; c < a.Dv; c += blockDim.x) ((T*)a.y)[(long long)b * a.ldy + hv + c] = (T)0.0f;
        return;
    }
    float* state = slot >= 0 ? a.state + ((long long)slot * a.Hv + h) * a.Dk * a.Dv : nullptr;
    const bool carried = state && (!a.cu || (a.carry && a.carry[b] != 0));
    const int r0 = RPL * rg, columns = (a.Dv + 15) / 16;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f, A = a.A[h];
    for (int block = wave; block < columns; block += waves) {
        const int c0 = 16 * block + 4 * (lane >> 4);
        f32x4 S[RPL];
#pragma unroll
        for (int j = 0; j < RPL; ++j) {
            S[j] = f32x4{};
            if (carried && r0 + j < a.Dk) S[j] = load_some<float, 4>(state + (long long)(r0 + j) * a.Dv, c0, a.Dv);
        }
        vec_t<T, RPL> q, k;
        vec_t<T, 4> v;
        T ga, gb;
        auto load = [&](int t) {
            const long long row = start + t;
            q = load_some<T, RPL>((const T*)a.q + row * a.ldq + (long long)hk * a.Dk, r0, a.Dk);
            k = load_some<T, RPL>((const T*)a.k + row * a.ldk + (long long)hk * a.Dk, r0, a.Dk);
            v = load_some<T, 4>((const T*)a.v + row * a.ldv + hv, c0, a.Dv);
            ga = ((const T*)a.a)[row * a.lda + h];
            gb = ((const T*)a.b)[row * a.ldb + h];
        };
        if (n > 0) load(0);
        for (int t = 0; t < n; ++t) {
            float fq[RPL], fk[RPL], fv[4];
#pragma unroll
            for (int j = 0; j < RPL; ++j) fq[j] = (float)q[j], fk[j] = (float)k[j];
#pragma unroll
            for (int i = 0; i < 4; ++i) fv[i] = (float)v[i];
            const float alpha = __builtin_amdgcn_exp2f((float)log_decay(ga, bias, A, a.softplus));
            const float beta = rate_of(gb);
            if (t + 1 < n) load(t + 1);
            float qq = 0.0f, kk = 0.0f, qk = 0.0f;
            f32x4 ks = {}, qs = {};
#pragma unroll
            for (int j = 0; j < RPL; ++j) {
                qq = __builtin_fmaf(fq[j], fq[j], qq);
                kk = __builtin_fmaf(fk[j], fk[j], kk);
                qk = __builtin_fmaf(fq[j], fk[j], qk);
                ks += fk[j] * S[j];
                qs += fq[j] * S[j];
            }
            qk = sum16(qk);
            float rq = a.scale, rk = 1.0f;
            if (a.qk_norm) {
                rq /= __builtin_sqrtf(sum16(qq) + a.eps);
                rk /= __builtin_sqrtf(sum16(kk) + a.eps);
            }
            f32x4 u;
            float o[4], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = beta * (fv[i] - alpha * (rk * sum16(ks[i])));
                o[i] = rq * (alpha * sum16(qs[i]) + qk * rk * u[i]);
                if (c0 + i < a.Dv) sum = __builtin_fmaf(o[i], o[i], sum);
            }
            const f32x4 w = rk * u;
#pragma unroll
            for (int j = 0; j < RPL; ++j) S[j] = alpha * S[j] + fk[j] * w;
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (rg == 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) outs[t][c0 + i] = o[i];
            if (lane == 0) squares[t][block] = sum;
        }
        if (state)
#pragma unroll
            for (int j = 0; j < RPL; ++j) {
                if (r0 + j >= a.Dk) continue;
                float* p = state + (long long)(r0 + j) * a.Dv + c0;
                if (c0 + 4 <= a.Dv) {
                    *(f32x4_any*)p = S[j];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c0 + i < a.Dv) p[i] = S[j][i];
                }
            }
    }
    __syncthreads();
    for (int t = wave; t < n; t += waves) {
        const long long row = start + t;
        float f = 1.0f;
        if (a.norm) {
            float sum = 0.0f;
            for (int i = 0; i < columns; ++i) sum += squares[t][i];
            f = 1.0f / __builtin_sqrtf(sum / (float)a.Dv + a.eps);
            // (the chunks' norm leaves the row alone)
            if (slices > 0 && lane == 0) a.squares[(row * a.Hv + h) * slices] = -1.0f;
        }
        for (int c = lane; c < a.Dv; c += 64) {
            float y = outs[t][c];
            if (a.norm) y *= f * a.norm[c];
            if (a.z) y *= silu((float)((const T*)a.z)[row * a.ldz + hv + c]);
            ((T*)a.y)[row * a.ldy + hv + c] = (T)y;
        }
    }
}

int k_blocks(int Dk) { return Dk <= 32 ? 1 : Dk <= 64 ? 2 : Dk <= 128 ? 4 : 8; }
int pieces_in(int dtype) { return dtype == FCM_F32 ? 3 : dtype == FCM_F16 ? 2 : 1; }
int pieces_out(int dtype) { return dtype == FCM_F32 ? 3 : 2; }
long long chunk_places(int tokens, int seqs) { return (long long)tokens / kChunk + seqs + 1; }
// Tiles of 16 columns of a workgroup: two share what is read of the keys where they fill the card, one is the shorter
// chain where they do not.  4096 tokens, Dv = 128, us, one / two: 16 heads of one sequence 130 / 200, 32 heads of three 191 / 206,
// of four 172 / 159; 8192 tokens, 32 heads of eight 397 / 334.
int slice_tiles(int seqs, int Hv, int Dv) { return (long long)seqs * Hv * ((Dv + 31) / 32) >= 512 ? 2 : 1; }
int column_slices(int Dv, int nt) { return (Dv + 16 * nt - 1) / (16 * nt); }
// 32-bit outputs before the norm (y holds those of 32-bit types)
long long outs_bytes(int tokens, int Hv, int Dv, int dtype) {
    return dtype == FCM_F32 ? 0 : ((long long)tokens * Hv * Dv * 4 + 15) / 16 * 16;
}

template <typename T, int NKB, int NT>
int chunks(const DeltaArgs& a, int slices, hipStream_t s) {
    const int seqs = long_sequences(a.seqs, a.tokens, a.shortest);
    delta_chunks_kernel<T, NKB, NT><<<(seqs * a.Hv + 7) / 8 * 8 * slices, 512, 0, s>>>(a, slices);
    return (int)hipGetLastError();
}

template <typename T>
int by_tokens(const DeltaArgs& a, int slices, hipStream_t s) {
    const int waves = (a.Dv + 15) / 16;
    if (a.Dk <= 64)
        delta_tokens_kernel<T, 4><<<a.seqs * a.Hv, 64 * waves, 0, s>>>(a, slices);
    else if (a.Dk <= 128)
        delta_tokens_kernel<T, 8><<<a.seqs * a.Hv, 64 * waves, 0, s>>>(a, slices);
    else
        delta_tokens_kernel<T, 16><<<a.seqs * a.Hv, 64 * (waves < 8 ? waves : 8), 0, s>>>(a, slices);
    return (int)hipGetLastError();
}

// Which sequences are short only the device knows, unless there is one or few tokens.
template <typename T, int NKB>
int run(DeltaArgs a, hipStream_t s) {
    const int nt = slice_tiles(a.seqs, a.Hv, a.Dv), slices = column_slices(a.Dv, nt);
    int rc = 0;
    a.shortest = a.seqs > 1 || a.tokens <= kShort ? kShort : -1;
    if (a.shortest > 0) {
        rc = by_tokens<T>(a, a.tokens <= kShort ? 0 : slices, s);
        if (rc != 0 || a.tokens <= kShort) return rc;
    }
    delta_prep_kernel<T, NKB><<<(int)a.places * a.Hk, 256, 0, s>>>(a);
    rc = (int)hipGetLastError();
    if (rc != 0) return rc;
    rc = nt == 2 ? chunks<T, NKB, 2>(a, slices, s) : chunks<T, NKB, 1>(a, slices, s);
    if (rc != 0 || !a.norm || a.tokens == 0) return rc;
    // as many lanes as a row has vectors, a power of two of them
    constexpr int VE = Vec<T>::N;
    int width = 1;
    while (width < 64 && width * VE < a.Dv) width *= 2;
    const int rows = 256 / width * kNormRows;
    const int grid = (int)(((long long)a.tokens * a.Hv + rows - 1) / rows);
    const bool wide = a.Dv % VE == 0 && rows16(a.y, a.ldy, sizeof(T)) && (!a.z || rows16(a.z, a.ldz, sizeof(T)));
    // Where most sequences are likely short it first asks whose the rows are: 32 sequences of 5 tokens take 57 us with the kernels
    // before it instead of 60, as rows that are done take no place in the caches; of 8192 tokens of 11 sequences it would
    // take 57 us instead of 55, of one of 4096 17 instead of 16.
    if (!wide)
        delta_norm_kernel<T, false, false><<<grid, 256, 0, s>>>(a, slices, width);
    else if (a.shortest > 0 && a.tokens < 2ll * kShort * a.seqs)
        delta_norm_kernel<T, true, true><<<grid, 256, 0, s>>>(a, slices, width);
    else
        delta_norm_kernel<T, true, false><<<grid, 256, 0, s>>>(a, slices, width);
    return (int)hipGetLastError();
}

template <typename T>
int pick_channels(const DeltaArgs& a, hipStream_t s) {
    switch (k_blocks(a.Dk)) {
        case 1: return run<T, 1>(a, s);
        case 2: return run<T, 2>(a, s);
        case 4: return run<T, 4>(a, s);
        default: return run<T, 8>(a, s);
    }
}

}  // namespace

long long delta_workspace_bytes(const fcm_delta_problem& p) {
    const Layout l = layout(pieces_in(p.dtype), pieces_out(p.dtype), k_blocks(p.Dk));
    const long long places = chunk_places(p.tokens, p.seqs);
    return places * (p.Hk * l.key_bytes + p.Hv * l.head_bytes) + outs_bytes(p.tokens, p.Hv, p.Dv, p.dtype) +
           (long long)p.tokens * p.Hv * column_slices(p.Dv, 1) * 4;
}

long long delta_threads(const fcm_delta_problem& p) {
    const long long prep = chunk_places(p.tokens, p.seqs) * p.Hk * 256;
    const long long chunks = ((long long)p.seqs * p.Hv + 7) / 8 * 8 * column_slices(p.Dv, 1) * 512;
    const long long norm = (long long)p.tokens * p.Hv * 64 + 255;
    const long long token = (long long)p.seqs * p.Hv * 1024;
    long long most = prep > chunks ? prep : chunks;
    most = most > norm ? most : norm;
    return most > token ? most : token;
}

int launch_delta_fwd(DeltaArgs a, int dtype, void* stream) {
    const Layout l = layout(pieces_in(dtype), pieces_out(dtype), k_blocks(a.Dk));
    a.places = chunk_places(a.tokens, a.seqs);
    a.outs = (float*)((char*)a.ws + a.places * (a.Hk * l.key_bytes + a.Hv * l.head_bytes));
    a.squares = (float*)((char*)a.outs + outs_bytes(a.tokens, a.Hv, a.Dv, dtype));
    const int e = dtype == FCM_F32 ? 4 : 2;
    a.wide_q = a.Dk % (16 / e) == 0 && rows16(a.q, a.ldq, e);
    a.wide_k = a.Dk % (16 / e) == 0 && rows16(a.k, a.ldk, e);
    auto pairs = [](const void* p, long long ld, int Dv, int size) {
        return Dv % 2 == 0 && ld % 2 == 0 && ((uintptr_t)p & (2 * size - 1)) == 0;
    };
    a.wide_v = pairs(a.v, a.ldv, a.Dv, e);
    a.wide_z = pairs(a.z, a.ldz, a.Dv, e);
    a.wide_y = pairs(a.y, a.ldy, a.Dv, e);
    a.wide_state = pairs(a.state, 0, a.Dv, 4);
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return pick_channels<float>(a, s);
    if (dtype == FCM_F16) return pick_channels<_Float16>(a, s);
    return pick_channels<__bf16>(a, s);
}

int launch_delta_step(const DeltaArgs& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return by_tokens<float>(a, 0, s);
    if (dtype == FCM_F16) return by_tokens<_Float16>(a, 0, s);
    return by_tokens<__bf16>(a, 0, s);
}

}  // namespace fcm
