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
// fed as three bf16 pieces (its 24 bits, cut into eight at a time), 16-bit inputs as they are (fp16: two
// pieces), and the products of pieces that together are below 2^-24 of the result are left out.  16-bit outputs
// (not the state) leave out those below 2^-16.  Quotients G_i / G_j are exponentials of differences of sums
// held in 64 bits: in 32 the difference of two sums of a few hundred would be off by 2^-16.
#include <float.h>

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

// Eight values as N operands of eight bf16 pieces each: the upper 16 bits, those of the rest, and so on.
template <int N>
__device__ __forceinline__ void split8(const float* v, u32x4* out) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
    for (int p = 0; p < N; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[p][i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, r[2 * i + 1]),
                                              __builtin_bit_cast(uint32_t, r[2 * i]), 0x07060302u);
        if (p + 1 < N)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, r[i]) & 0xffff0000u);
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

// One workgroup per chunk and key head.
template <typename T, int NKB>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a) {
    constexpr int PI = Pieces<T>::IN, PQ = Pieces<T>::OUT, DK = 32 * NKB, LD = DK + 8, LM = 68;
    constexpr int kIn = 2 * kChunk * LD * (int)sizeof(T), kMat = 2 * kChunk * LM * 4;
    __shared__ __attribute__((aligned(16))) char smem[kIn > kMat ? kIn : kMat];
    __shared__ double along[kChunk];
    __shared__ float beta[kChunk], rq[kChunk], rk[kChunk];
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
    const int n = end - t0 < kChunk ? end - t0 : kChunk;
    const int tid = threadIdx.x, lane = tid & 63, sub = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Layout lay = layout(PI, PQ, NKB);
    const long long place = id;
    char* key = (char*)a.ws + (place * a.Hk + hk) * lay.key_bytes;
    char* heads = (char*)a.ws + a.places * a.Hk * lay.key_bytes;

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
    const int share = a.Hv / a.Hk;
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        char* head = heads + (place * a.Hv + h) * lay.head_bytes;
        __syncthreads();  // (the rows in LDS, or the last head's matrices, are done with)
        if (wave == 0) {
            double p = 0.0;
            float r = 0.0f;
            if (lane < n) {
                const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
                p = log_decay(((const T*)a.a)[(t0 + lane) * a.lda + h], bias, A, a.softplus);
                r = rate_of(((const T*)a.b)[(t0 + lane) * a.ldb + h]);
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double v = __shfl_up(p, o);
                if (lane >= o) p += v;
            }
            along[lane] = p;
            beta[lane] = r;
            const double last = __shfl(p, 63);
            const float grown = __builtin_amdgcn_exp2f((float)p);
            float* rows = (float*)(head + lay.rows);
            rows[lane] = grown * rk[lane];
            rows[kChunk + lane] = grown * rq[lane];
            rows[2 * kChunk + lane] = __builtin_amdgcn_exp2f((float)(last - p)) * rk[lane];
            if (lane == 0) rows[3 * kChunk] = __builtin_amdgcn_exp2f((float)last);
        }
        __syncthreads();
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

// One workgroup per sequence, value head and slice of 16 NT columns; wave w has the tokens of tile w of each
// chunk and the state's channels of k-blocks w, w + 4.
template <typename T, int NKB, int NT>
__global__ __launch_bounds__(256) void delta_chunks_kernel(DeltaArgs a, int slices) {
    constexpr int PI = Pieces<T>::IN, PQ = Pieces<T>::OUT, KW = (NKB + 3) / 4;
    __shared__ u32x4 sb[NKB][NT][3][64];  // the state as an operand over channels
    __shared__ u32x4 rb[2][NT][3][64];    // what the values differ by, over tokens
    __shared__ u32x4 ub[2][NT][PQ][64];   // U
    __shared__ u32x4 ud[2][NT][3][64];    // U with the decay to the chunk's end
    const int tid = threadIdx.x, lane = tid & 63, sub = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the slices of a head, which read the same operands, go to one XCD
    const int xcd = blockIdx.x & 7, rest = blockIdx.x >> 3;
    const int slice = rest % slices, bh = (rest / slices) * 8 + xcd;
    if (bh >= a.seqs * a.Hv) return;
    const int b = bh / a.Hv, h = bh % a.Hv, hk = h / (a.Hv / a.Hk);
    const int start = seq_offset(a.cu, b, a.tokens), end = seq_offset(a.cu, b + 1, a.tokens);
    const int slot = a.state ? seq_slot(a.slots, b, a.nslots) : -1;
    const Layout lay = layout(PI, PQ, NKB);
    float* state = slot >= 0 ? a.state + ((long long)slot * a.Hv + h) * a.Dk * a.Dv : nullptr;
    const bool carried = state && a.carry && a.carry[b] != 0;
    int col[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) col[t] = (slice * NT + t) * 16 + sub;

    // channel of row r = 4 grp + i of tile half hf of k-block kb: 32 kb + 8 grp + 4 hf + i
    f32x4 S[KW][2][NT];
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 32 * (wave + 4 * k) + 8 * grp + 4 * hf + i;
                    S[k][hf][t][i] = carried && c < a.Dk && col[t] < a.Dv ? state[(long long)c * a.Dv + col[t]] : 0.0f;
                }
    int place = first_chunk(a.cu, b, a.tokens);
    for (int t0 = start; t0 < end; t0 += kChunk, ++place) {
        const char* key = (const char*)a.ws + ((long long)place * a.Hk + hk) * lay.key_bytes;
        const char* head = (const char*)a.ws + a.places * a.Hk * lay.key_bytes +
                           ((long long)place * a.Hv + h) * lay.head_bytes;
        const float* rows = (const float*)(head + lay.rows);
        const int tok = 32 * (wave >> 1) + 8 * grp + 4 * (wave & 1);  // .. + i
#pragma unroll
        for (int k = 0; k < KW; ++k)
            if (wave + 4 * k < NKB)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = S[k][i >> 2][t][i & 3];
                    u32x4 f[3];
                    split8<3>(v, f);
#pragma unroll
                    for (int p = 0; p < 3; ++p) sb[wave + 4 * k][t][p][lane] = f[p];
                }
        __syncthreads();
        f32x4 ks[NT], o[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) ks[t] = o[t] = f32x4{};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            u32x4 fk[PI], fq[PI];
#pragma unroll
            for (int p = 0; p < PI; ++p) {
                fk[p] = ld16(key + lay.kf + ((p * 4 + wave) * NKB + kb) * kFrag + lane * 16);
                fq[p] = ld16(key + lay.qf + ((p * 4 + wave) * NKB + kb) * kFrag + lane * 16);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                u32x4 f[3];
#pragma unroll
                for (int p = 0; p < 3; ++p) f[p] = sb[kb][t][p][lane];
                ks[t] = mm_pieces<PI, 3, 3>(fk, f, ks[t]);
                o[t] = mm_pieces<PI, 3, PQ>(fq, f, o[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float r[8] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = tok + i;
                float v = 0.0f;
                if (t0 + m < end && col[t] < a.Dv)
                    v = (float)((const T*)a.v)[(t0 + m) * a.ldv + (long long)h * a.Dv + col[t]];
                r[i] = __builtin_fmaf(-rows[m], ks[t][i], v);
                o[t][i] *= rows[kChunk + m];
            }
            u32x4 f[3];
            split8<3>(r, f);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *(uint2*)((char*)&rb[wave >> 1][t][p][lane] + 8 * (wave & 1)) = uint2{f[p][0], f[p][1]};
        }
        __syncthreads();
        f32x4 u[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) u[t] = f32x4{};
        for (int kb = 0; kb <= (wave >> 1); ++kb) {
            u32x4 ft[3];
#pragma unroll
            for (int p = 0; p < 3; ++p) ft[p] = ld16(head + lay.tf + (p * 6 + lower(wave, kb)) * kFrag + lane * 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                u32x4 f[3];
#pragma unroll
                for (int p = 0; p < 3; ++p) f[p] = rb[kb][t][p][lane];
                u[t] = mm_pieces<3, 3, 3>(ft, f, u[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float v[8] = {}, w[8] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = u[t][i];
                w[i] = u[t][i] * rows[2 * kChunk + tok + i];
            }
            u32x4 f[3];
            split8<PQ>(v, f);
#pragma unroll
            for (int p = 0; p < PQ; ++p)
                *(uint2*)((char*)&ub[wave >> 1][t][p][lane] + 8 * (wave & 1)) = uint2{f[p][0], f[p][1]};
            split8<3>(w, f);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *(uint2*)((char*)&ud[wave >> 1][t][p][lane] + 8 * (wave & 1)) = uint2{f[p][0], f[p][1]};
        }
        __syncthreads();
        const float last = rows[3 * kChunk];
#pragma unroll
        for (int k = 0; k < KW; ++k)
            if (wave + 4 * k < NKB)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) S[k][hf][t] *= last;
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb) {
                        u32x4 fk[PI];
#pragma unroll
                        for (int p = 0; p < PI; ++p)
                            fk[p] = ld16(key + lay.kt + ((p * 2 * NKB + 2 * (wave + 4 * k) + hf) * 2 + kb) * kFrag + lane * 16);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            u32x4 f[3];
#pragma unroll
                            for (int p = 0; p < 3; ++p) f[p] = ud[kb][t][p][lane];
                            S[k][hf][t] = mm_pieces<PI, 3, 3>(fk, f, S[k][hf][t]);
                        }
                    }
                }
        for (int kb = 0; kb <= (wave >> 1); ++kb) {
            u32x4 fp[PQ];
#pragma unroll
            for (int p = 0; p < PQ; ++p) fp[p] = ld16(head + lay.pf + (p * 6 + lower(wave, kb)) * kFrag + lane * 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                u32x4 f[PQ];
#pragma unroll
                for (int p = 0; p < PQ; ++p) f[p] = ub[kb][t][p][lane];
                o[t] = mm_pieces<PQ, PQ, PQ>(fp, f, o[t]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = t0 + tok + i;
            if (m >= end) continue;
            float squares = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (col[t] >= a.Dv) continue;
                float v = o[t][i];
                squares = __builtin_fmaf(v, v, squares);
                const long long at = (long long)h * a.Dv + col[t];
                if (!a.norm && a.z) v *= silu((float)((const T*)a.z)[m * a.ldz + at]);
                ((T*)a.y)[m * a.ldy + at] = (T)v;
            }
            if (a.norm) {
#pragma unroll
                for (int s = 1; s < 16; s <<= 1) squares += __shfl_xor(squares, s);
                if (sub == 0) a.squares[((long long)m * a.Hv + h) * slices + slice] = squares;
            }
        }
    }
    if (!state) return;
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 32 * (wave + 4 * k) + 8 * grp + 4 * hf + i;
                    if (c < a.Dk && col[t] < a.Dv) state[(long long)c * a.Dv + col[t]] = S[k][hf][t][i];
                }
}

// The output's norm and gate, in place: the second kernel's slices left their sums of squares.  A wave per row
// and head.
template <typename T>
__global__ __launch_bounds__(256) void delta_norm_kernel(DeltaArgs a, int slices) {
    const int lane = threadIdx.x & 63;
    const long long id = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long t = id / a.Hv, h = id % a.Hv;
    if (t < seq_offset(a.cu, 0, a.tokens) || t >= seq_offset(a.cu, a.seqs, a.tokens)) return;
    float s = 0.0f;
    for (int i = 0; i < slices; ++i) s += a.squares[id * slices + i];
    const float f = 1.0f / __builtin_sqrtf(s / (float)a.Dv + a.eps);
    T* y = (T*)a.y + t * a.ldy + h * a.Dv;
    const T* z = a.z ? (const T*)a.z + t * a.ldz + h * a.Dv : nullptr;
    for (int c = lane; c < a.Dv; c += 64) {
        float v = (float)y[c] * f * a.norm[c];
        if (z) v *= silu((float)z[c]);
        y[c] = (T)v;
    }
}

// Single tokens.  A workgroup has a sequence and a head: lanes along the columns, four each, tx of them, and
// a.Dk rows over the groups of tx threads, 16 rows each.
template <typename T, bool WIDE>
__global__ __launch_bounds__(1024) void delta_step_kernel(DeltaArgs a, int tx, int groups) {
    __shared__ float vec[2][256];           // q and k with their factors
    __shared__ float part[2][16][256 + 4];  // the groups' sums over their rows
    const int tid = threadIdx.x, lane = tid & 63;
    const int b = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, hk = h / (a.Hv / a.Hk);
    const int slot = seq_slot(a.slots, b, a.nslots);
    T* y = (T*)a.y + b * a.ldy + (long long)h * a.Dv;
    if (slot < 0) {
        for (int c = tid; c < a.Dv; c += blockDim.x) y[c] = (T)0.0f;
        return;
    }
    float* state = a.state + ((long long)slot * a.Hv + h) * a.Dk * a.Dv;
    const int x = tid % tx, rg = tid / tx, c0 = 4 * x;
    const bool mine = rg < groups;  // (the last wave may be larger)
    f32x4 S[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int r = rg + groups * j;
        S[j] = f32x4{};
        if (mine && r < a.Dk) {
            const float* p = state + (long long)r * a.Dv + c0;
            if constexpr (WIDE) {
                S[j] = *(const f32x4*)p;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 + i < a.Dv) S[j][i] = p[i];
            }
        }
    }
    // q, k: every wave finds their norms and product for itself, the first one keeps them
    float qq = 0.0f, kk = 0.0f, qk = 0.0f, qv[4], kv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane + 64 * i;
        qv[i] = c < a.Dk ? (float)((const T*)a.q)[b * a.ldq + (long long)hk * a.Dk + c] : 0.0f;
        kv[i] = c < a.Dk ? (float)((const T*)a.k)[b * a.ldk + (long long)hk * a.Dk + c] : 0.0f;
        qq = __builtin_fmaf(qv[i], qv[i], qq);
        kk = __builtin_fmaf(kv[i], kv[i], kk);
        qk = __builtin_fmaf(qv[i], kv[i], qk);
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        qq += __shfl_xor(qq, s);
        kk += __shfl_xor(kk, s);
        qk += __shfl_xor(qk, s);
    }
    const float rq = a.scale * (a.qk_norm ? 1.0f / __builtin_sqrtf(qq + a.eps) : 1.0f);
    const float rk = a.qk_norm ? 1.0f / __builtin_sqrtf(kk + a.eps) : 1.0f;
    qk *= rq * rk;
    if (tid < 64)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            vec[0][lane + 64 * i] = qv[i] * rq;
            vec[1][lane + 64 * i] = kv[i] * rk;
        }
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    const float alpha = __builtin_amdgcn_exp2f(
        (float)log_decay(((const T*)a.a)[b * a.lda + h], bias, a.A[h], a.softplus));
    const float beta = rate_of(((const T*)a.b)[b * a.ldb + h]);
    __syncthreads();
    f32x4 ks = {}, qs = {};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int r = rg + groups * j;
        if (r < a.Dk) {
            ks += vec[1][r] * S[j];
            qs += vec[0][r] * S[j];
        }
    }
    if (mine)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            part[0][rg][c0 + i] = ks[i];
            part[1][rg][c0 + i] = qs[i];
        }
    __syncthreads();
    ks = qs = f32x4{};
    for (int g = 0; g < groups; ++g) {
        ks += *(const f32x4*)&part[0][g][c0];
        qs += *(const f32x4*)&part[1][g][c0];
    }
    f32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = c0 + i < a.Dv ? (float)((const T*)a.v)[b * a.ldv + (long long)h * a.Dv + c0 + i] : 0.0f;
        u[i] = beta * (v - alpha * ks[i]);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int r = rg + groups * j;
        if (mine && r < a.Dk) {
            const f32x4 now = alpha * S[j] + vec[1][r] * u;
            float* p = state + (long long)r * a.Dv + c0;
            if constexpr (WIDE) {
                *(f32x4*)p = now;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 + i < a.Dv) p[i] = now[i];
            }
        }
    }
    if (tid >= 64) return;
    // the first wave has the output's columns (tx is at most 64)
    float o[4], squares = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = alpha * qs[i] + qk * u[i];
        if (rg == 0 && c0 + i < a.Dv) squares = __builtin_fmaf(o[i], o[i], squares);
    }
    float f = 1.0f;
    if (a.norm) {
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) squares += __shfl_xor(squares, s);
        f = 1.0f / __builtin_sqrtf(squares / (float)a.Dv + a.eps);
    }
    if (rg == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + i;
            if (c >= a.Dv) continue;
            float v = o[i];
            if (a.norm) v *= f * a.norm[c];
            if (a.z) v *= silu((float)((const T*)a.z)[b * a.ldz + (long long)h * a.Dv + c]);
            y[c] = (T)v;
        }
}

int k_blocks(int Dk) { return Dk <= 32 ? 1 : Dk <= 64 ? 2 : Dk <= 128 ? 4 : 8; }
int pieces_in(int dtype) { return dtype == FCM_F32 ? 3 : dtype == FCM_F16 ? 2 : 1; }
int pieces_out(int dtype) { return dtype == FCM_F32 ? 3 : 2; }
long long chunk_places(int tokens, int seqs) { return (long long)tokens / kChunk + seqs + 1; }
int column_slices(int Dv, int nt) { return (Dv + 16 * nt - 1) / (16 * nt); }

template <typename T, int NKB>
int run(DeltaArgs a, hipStream_t s) {
    delta_prep_kernel<T, NKB><<<(int)a.places * a.Hk, 256, 0, s>>>(a);
    int rc = (int)hipGetLastError();
    if (rc != 0) return rc;
    const int slices = column_slices(a.Dv, 1);
    delta_chunks_kernel<T, NKB, 1><<<(a.seqs * a.Hv + 7) / 8 * 8 * slices, 256, 0, s>>>(a, slices);
    rc = (int)hipGetLastError();
    if (rc != 0 || !a.norm || a.tokens == 0) return rc;
    delta_norm_kernel<T><<<(int)(((long long)a.tokens * a.Hv + 3) / 4), 256, 0, s>>>(a, slices);
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

template <typename T>
int step(const DeltaArgs& a, hipStream_t s) {
    const int tx = (a.Dv + 3) / 4, groups = (a.Dk + 15) / 16;
    const int threads = (tx * groups + 63) / 64 * 64;
    const bool wide = a.Dv % 4 == 0 && ((uintptr_t)a.state & 15) == 0;
    if (wide)
        delta_step_kernel<T, true><<<a.seqs * a.Hv, threads, 0, s>>>(a, tx, groups);
    else
        delta_step_kernel<T, false><<<a.seqs * a.Hv, threads, 0, s>>>(a, tx, groups);
    return (int)hipGetLastError();
}

}  // namespace

long long delta_workspace_bytes(const fcm_delta_problem& p) {
    const Layout l = layout(pieces_in(p.dtype), pieces_out(p.dtype), k_blocks(p.Dk));
    const long long places = chunk_places(p.tokens, p.seqs);
    return places * (p.Hk * l.key_bytes + p.Hv * l.head_bytes) +
           (long long)p.tokens * p.Hv * column_slices(p.Dv, 1) * 4;
}

long long delta_threads(const fcm_delta_problem& p) {
    const long long prep = chunk_places(p.tokens, p.seqs) * p.Hk * 256;
    const long long chunks = ((long long)p.seqs * p.Hv + 7) / 8 * 8 * column_slices(p.Dv, 1) * 256;
    const long long norm = ((long long)p.tokens * p.Hv + 3) / 4 * 256;
    const long long token = (long long)p.seqs * p.Hv * 1024;
    long long most = prep > chunks ? prep : chunks;
    most = most > norm ? most : norm;
    return most > token ? most : token;
}

int launch_delta_fwd(DeltaArgs a, int dtype, void* stream) {
    const Layout l = layout(pieces_in(dtype), pieces_out(dtype), k_blocks(a.Dk));
    a.places = chunk_places(a.tokens, a.seqs);
    a.squares = (float*)((char*)a.ws + a.places * (a.Hk * l.key_bytes + a.Hv * l.head_bytes));
    const int e = dtype == FCM_F32 ? 4 : 2;
    a.wide_q = a.Dk % (16 / e) == 0 && rows16(a.q, a.ldq, e);
    a.wide_k = a.Dk % (16 / e) == 0 && rows16(a.k, a.ldk, e);
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return pick_channels<float>(a, s);
    if (dtype == FCM_F16) return pick_channels<_Float16>(a, s);
    return pick_channels<__bf16>(a, s);
}

int launch_delta_step(const DeltaArgs& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return step<float>(a, s);
    if (dtype == FCM_F16) return step<_Float16>(a, s);
    return step<__bf16>(a, s);
}

}  // namespace fcm
