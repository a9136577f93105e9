// mx4.hip -- microscaled 4-bit floating point: blocks of 32 channels share a power of two, a channel is a sign,
// two bits of exponent and one of mantissa.  Quantisation and its inverse, and pointwise layers
//   y[m][k] = act(bias[k] + sum_c W[k][c] x[m][c])
// with such weights for 16-bit tokens (a few) and for tokens that are quantised as well (any number).
#include "mm_common.h"
#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// The activation as a clamp that lets NaN through (a median of three would not).
__device__ __forceinline__ float clamp_act(float v, Act act) {
    return v < act.lo ? act.lo : v > act.hi ? act.hi : v;
}

// The conversions take a block's power of two as a float, by its exponent bits alone: those are the stored
// scale (0 stands for 2^-127, 255 for NaN).
__device__ __forceinline__ float scale_float(uint32_t code) { return __builtin_bit_cast(float, code << 23); }

// ------------------------------------------------------------------------------------------
// quantisation: eight channels a lane, four lanes a block.  HBM bounds it: 8192 x 4096 bf16, 85 MB, in 19 us, 4.5 TB/s
// ------------------------------------------------------------------------------------------
constexpr int kPer = 4;  // pieces of eight channels of a thread

// Row and channel of piece i of eight channels; dense rows are one long row.
__device__ __forceinline__ long long piece_at(long long i, int C, long long ld) {
    if (ld == C) return i * 8;
    const long long row = i / (C / 8);
    return row * ld + (i - row * (C / 8)) * 8;
}

template <typename T, bool WIDE>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(Mx4Args a, long long pieces) {
    const T* x = (const T*)a.x;
    uint8_t* q = (uint8_t*)a.q;
    uint8_t* scales = (uint8_t*)a.scales;
    const long long first = (long long)blockIdx.x * (256 * kPer) + threadIdx.x;
    float v[kPer][8];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const long long i = first + 256 * j;
        const T* p = x + piece_at(i < pieces ? i : 0, a.C, a.ldx);
        if constexpr (WIDE) {
#pragma unroll
            for (int e = 0; e < 8 / Vec<T>::N; ++e) unpack16<T>(ld16(p + e * Vec<T>::N), v[j] + e * Vec<T>::N);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = (float)p[e];
        }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const long long i = first + 256 * j;
        // magnitudes order as integers, infinities and NaN above all
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = __builtin_bit_cast(uint32_t, v[j][e]) & 0x7fffffffu;
            top = m > top ? m : top;
        }
        uint32_t o = __shfl_xor(top, 1);
        top = o > top ? o : top;
        o = __shfl_xor(top, 2);
        top = o > top ? o : top;
        const uint32_t exponent = top >> 23;
        const uint32_t scale = exponent == 255 ? 255 : exponent > 2 ? exponent - 2 : 0;
        const float by = scale_float(scale);
        uint32_t codes = 0;
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[j][0], v[j][1], by, 0);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[j][2], v[j][3], by, 1);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[j][4], v[j][5], by, 2);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[j][6], v[j][7], by, 3);
        if (i < pieces) {
            *(uint32_t*)(q + i * 4) = codes;
            if ((i & 3) == 0) scales[i >> 2] = (uint8_t)scale;
        }
    }
}

template <typename T, bool WIDE>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(Mx4Args a, long long pieces) {
    T* y = (T*)a.y;
    const long long first = (long long)blockIdx.x * (256 * kPer) + threadIdx.x;
    uint32_t codes[kPer], scale[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const long long i = first + 256 * j < pieces ? first + 256 * j : 0;
        codes[j] = *(const uint32_t*)(a.q + i * 4);
        scale[j] = a.scales[i >> 2];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const long long i = first + 256 * j;
        if (i >= pieces) return;
        const float by = scale_float(scale[j]);
        const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], by, 0);
        const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], by, 1);
        const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], by, 2);
        const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], by, 3);
        const float v[8] = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
        T* p = y + piece_at(i, a.C, a.ldy);
        if constexpr (WIDE) {
#pragma unroll
            for (int e = 0; e < 8 / Vec<T>::N; ++e) st16(p + e * Vec<T>::N, pack16<T>(v + e * Vec<T>::N));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = (T)v[e];
        }
    }
}

// ------------------------------------------------------------------------------------------
// 16-bit tokens
// ------------------------------------------------------------------------------------------
// bf16 pieces of eight 16-bit inputs: fp16's 11 bits are two of them, exactly.  The first of an infinity is infinite;
// what is left of it, inf - inf, is a NaN, on this card a negative one, and with it all its outputs would be NaN.  As a 16-bit
// integer that lies above -256, and so becomes it (the second pieces are smaller): one instruction for two of them.
template <typename T>
struct XPieces {
    static constexpr int N = std::is_same<T, _Float16>::value ? 2 : 1;
};
template <typename T>
__device__ __forceinline__ void x_pieces(u32x4 raw, u32x4* out) {
    if constexpr (XPieces<T>::N == 1) {
        out[0] = raw;
    } else {
        float v[8];
        unpack16<T>(raw, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __builtin_bit_cast(uint32_t, v[2 * i]), hi = __builtin_bit_cast(uint32_t, v[2 * i + 1]);
            out[0][i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
            const float rl = v[2 * i] - __builtin_bit_cast(float, lo & 0xffff0000u);
            const float rh = v[2 * i + 1] - __builtin_bit_cast(float, hi & 0xffff0000u);
            const uint32_t rest = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, rh), __builtin_bit_cast(uint32_t, rl), 0x07060302u);
            out[1][i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, rest), u16x2{0xc380, 0xc380}));
        }
    }
}

constexpr int kStep = 128;  // channels a wave takes at a time: 64 bytes of an output channel
// Byte offset in x of the channels behind the last, which read as zero: beyond every range of a
// tile's tokens (31 row strides below 2^26 elements and 2^20 channels, 0xf8200000 bytes), and with a
// step's own offset of up to 2^21 still below 2^32.
constexpr uint32_t kBehind = 0xfc000000u;

typedef u32x2 __attribute__((aligned(1))) u32x2_any;

// The scales of TILES tiles of 16 rows, kSteps steps of four blocks at a time, in the wave's own LDS: four lanes load 32
// bytes of a row (a byte a step for itself would bring in the whole cache line each time).  Where a row has fewer than eight
// left they are its last eight, moved down; a row of fewer than eight in all is loaded by bytes.
constexpr int kSteps = 8;
template <int TILES>
struct StepScales {
    const uint8_t* row[TILES];  // this lane's row of each tile, from the lane's eight blocks on
    int blocks, part;
    u32x2 raw[TILES];
    __device__ __forceinline__ void fetch(int s0) {
        const int want = 4 * s0 + part, at = want + 8 <= blocks ? want : blocks - 8;
        if (blocks >= 8) {
#pragma unroll
            for (int r = 0; r < TILES; ++r) raw[r] = *(const u32x2_any*)(row[r] + at);
        } else {
#pragma unroll
            for (int r = 0; r < TILES; ++r) {
                raw[r] = u32x2{0, 0};
                for (int b = want; b < blocks; ++b) raw[r][(b - want) >> 2] |= (uint32_t)row[r][b] << (8 * (b & 3));
            }
        }
    }
    __device__ __forceinline__ void stage(int s0, u32x2 (*to)[64]) const {
        const int want = 4 * s0 + part;
        int gone = blocks < 8 || want + 8 <= blocks ? 0 : want - (blocks - 8);
        gone = gone < 8 ? gone : 8;
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
            const uint64_t u = (__builtin_bit_cast(uint64_t, raw[r]) >> (4 * gone)) >> (4 * gone);
            to[r][threadIdx.x & 63] = __builtin_bit_cast(u32x2, u);
        }
    }
    // of row l % 16, block l / 16 of step j
    __device__ __forceinline__ static uint32_t read(const u32x2* from, int j) {
        const int lane = threadIdx.x & 63;
        return ((const uint8_t*)from)[32 * (lane & 15) + 4 * j + (lane >> 4)];
    }
};

// A workgroup has 16 * RT output channels and 16 * MT tokens (or 4, 8: NI = 1, 2); its waves share
// the steps of 128 channels and add their sums through LDS.
//
// Four neighbouring lanes load 64 bytes of an output channel (16 lanes 256 bytes of a token), and the wave passes
// them through its own piece of LDS, in 16-byte chunks whose place is turned by the row so that a column of them
// has no bank twice: matrix operands want neighbouring lanes on different rows, 64 separate accesses a load.
// Lane l then holds one whole block, l / 16 of the step's four, of output channel l % 16; the conversion to bf16
// multiplies with the block's power of two (exact), and the four products of a step take eight channels of each
// block, in the same order from both sides.
//
// HBM bounds few tokens, and the conversions in turns with it more of them: 4096 channels -> 65536, 143 MB of codes,
// with 1 token 32 us (4.5 TB/s), 4 tokens 34, 8 tokens 38 (3.8 TB/s), 16 tokens 40, 32 tokens 55; in fp16, whose tokens are
// two pieces, 34, 36, 39, 40 and 77; 2048 -> 8192 with one token 4.1, the launch.  Prompts it reads the weights for again and
// again: 4096 -> 8192 takes 1024 tokens 156 us and 8192 tokens 1153, with the tokens quantised for the kernels below 42 and
// 207.
template <typename T, int NI, int MT, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void mx4_kernel(Mx4Args a) {
    constexpr int XI = MT * NI, TOKENS = 4 * XI, XP = XPieces<T>::N;
    static_assert(TOKENS <= 32, "kBehind lies behind a tile's tokens");
    __shared__ u32x4 stage[NW][RT + XP * XI][64];
    __shared__ u32x2 scales[NW][RT][64];
    auto part = [&](int w, int r, int i) { return (float*)stage[w] + (r * XI + i) * 64; };
    static_assert(RT * XI <= 4 * (RT + XP * XI), "the sums fit");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane & 15, grp = lane >> 4;
    const int steps = (a.C + kStep - 1) / kStep, blocks = a.C / 32;
    const int k0 = blockIdx.x * (16 * RT);
    const int m0 = blockIdx.y * TOKENS;
    const int lrow = lane >> 2, lchunk = (lane & 3) ^ (lrow >> 2);
    const int krows = a.K - k0 < 16 * RT ? a.K - k0 : 16 * RT;
    const int trows = a.M - m0 < TOKENS ? a.M - m0 : TOKENS;
    const __amdgpu_buffer_rsrc_t rq =
        mm::rsrc(a.q + (long long)k0 * (a.C / 2), (uint32_t)krows * (a.C / 2));
    const __amdgpu_buffer_rsrc_t rx = mm::rsrc((const T*)a.x + (long long)m0 * a.ldx,
                                               ((uint32_t)(trows - 1) * (uint32_t)a.ldx + a.C) * 2);
    uint32_t xat[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int t = 4 * i + grp;  // of the tile's tokens
        xat[i] = (t * (uint32_t)a.ldx + 8 * (sub ^ (t & 15))) * 2;
    }
    struct Step {
        u32x4 w[RT], x[XI];
    };
    auto fetch = [&](int s, Step& v) {
        // (channels behind the last: codes and tokens read as zero)
        const bool in = s * 4 + lchunk < blocks;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const uint32_t at = (16 * r + lrow) * (uint32_t)(a.C / 2) + 16 * lchunk;
            v.w[r] = __builtin_amdgcn_raw_buffer_load_b128(rq, in ? at : mm::kOob, s * (kStep / 2), 0);
        }
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            uint32_t at = xat[i];
            if (s * kStep + 8 * (sub ^ ((4 * i + grp) & 15)) >= a.C) at = kBehind;
            v.x[i] = __builtin_amdgcn_raw_buffer_load_b128(rx, at, s * kStep * 2, 0);
        }
    };
    f32x4 total[RT][MT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) total[r][m] = f32x4{};
    // token of accumulator row `sub` (of 16 tokens)
    const int tok = (sub >> 2) * NI + ((sub & 3) < NI ? sub & 3 : 0);
    const int wplace = sub * 4 + (grp ^ (sub >> 2));
    auto use = [&](Step& v, int j, int then) {
        uint32_t scale[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            stage[wave][r][lane] = v.w[r];
            scale[r] = StepScales<RT>::read(scales[wave][r], j);
        }
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            u32x4 f[XP];
            x_pieces<T>(v.x[i], f);
#pragma unroll
            for (int p = 0; p < XP; ++p) stage[wave][RT + p * XI + i][lane] = f[p];
        }
        fetch(then, v);
        __builtin_amdgcn_wave_barrier();
        u32x4 w[RT], x[MT][4][XP];
#pragma unroll
        for (int r = 0; r < RT; ++r) w[r] = stage[wave][r][wplace];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int p = 0; p < XP; ++p)
                    x[m][j][p] = stage[wave][RT + p * XI + NI * m + tok / 4][(tok & 3) * 16 + ((4 * grp + j) ^ (tok + 4 * NI * m & 15))];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float by = scale_float(scale[r]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
                u32x4 u;
                u[0] = __builtin_bit_cast(uint32_t, (bf2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[r][j], by, 0));
                u[1] = __builtin_bit_cast(uint32_t, (bf2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[r][j], by, 1));
                u[2] = __builtin_bit_cast(uint32_t, (bf2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[r][j], by, 2));
                u[3] = __builtin_bit_cast(uint32_t, (bf2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[r][j], by, 3));
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int p = XP - 1; p >= 0; --p) total[r][m] = mfma<__bf16>(x[m][j][p], u, total[r][m]);
            }
        }
    };
    // each wave has neighbouring steps
    const int share = (steps + NW - 1) / NW, first = wave * share, end = first + share < steps ? first + share : steps;
    if (first < end) {
        StepScales<RT> ss;
        ss.blocks = blocks;
        ss.part = 8 * (lane & 3);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            // (a row behind the last takes the last one's: it is not stored)
            const int row = 16 * r + lrow < krows ? 16 * r + lrow : krows - 1;
            ss.row[r] = a.scales + (long long)(k0 + row) * blocks;
        }
        Step v;
        ss.fetch(first);
        fetch(first, v);
        for (int s0 = first; s0 < end; s0 += kSteps) {
            ss.stage(s0, scales[wave]);
            ss.fetch(s0 + kSteps < end ? s0 + kSteps : s0);
            __builtin_amdgcn_wave_barrier();
            const int n = end - s0 < kSteps ? end - s0 : kSteps;
            for (int j = 0; j < n; ++j) use(v, j, s0 + j + 1 < end ? s0 + j + 1 : end - 1);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < XI; ++i) part(wave, r, i)[lane] = total[r][i / NI][i % NI];
    __syncthreads();
    const Act act = act_bounds(a.act);
    // lane l of sum i: token 16 * (i / NI) + (l / 16) * NI + i % NI (of MT tiles), output channel l % 16
    for (int j = threadIdx.x; j < RT * XI * 64; j += 64 * NW) {
        const int l = j & 63, i = (j >> 6) % XI, r = (j >> 6) / XI;
        const int m = m0 + i / NI * (4 * NI) + (l >> 4) * NI + i % NI, k = k0 + 16 * r + (l & 15);
        if (m >= a.M || k >= a.K) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < NW; ++q) v += part(q, r, i)[l];
        if (a.bias) v += a.bias[k];
        ((T*)a.y)[(long long)m * a.ldy + k] = (T)clamp_act(v, act);
    }
}

template <typename T, int NI, int MT>
int run(const Mx4Args& a, hipStream_t s) {
    const int tiles = (a.M + 4 * NI * MT - 1) / (4 * NI * MT);
    auto go = [&](auto rt, auto nw) {
        constexpr int RT = decltype(rt)::value, NW = decltype(nw)::value;
        const dim3 grid((a.K + 16 * RT - 1) / (16 * RT), tiles);
        mx4_kernel<T, NI, MT, RT, NW><<<grid, 64 * NW, 0, s>>>(a);
        return (int)hipGetLastError();
    };
    using std::integral_constant;
    // Wide layers: more output channels a workgroup, which share the tokens' operands, on fewer waves, which join
    // fewer sums; narrow ones need every wave there is.  At 4096 channels, us: 1 token, one tile on 8 waves / two on
    // 4: 12288 outputs 6.9 / 7.1, 16384 10.4 / 8.9, 32768 18.6 / 16.3; 16 tokens, one on 8 / two / four on 4: 8192 7.3 / - / 7.8,
    // 12288 11.6 / - / 8.6, 32768 30.7 / 22.1 / 18.8, 65536 58 / 52 / 40; 32 tokens, one on 8 / two on 4: 4096 6.3 / 7.7,
    // 8192 10.2 / 8.4, 65536 85 / 53.
    const long long rows = (long long)((a.K + 15) / 16) * tiles;
    if constexpr (NI == 4 && MT == 1) {
        if (rows >= 768) return go(integral_constant<int, 4>(), integral_constant<int, 4>());
    } else {
        if (rows >= (MT == 2 ? 512 : 1024)) return go(integral_constant<int, 2>(), integral_constant<int, 4>());
    }
    return go(integral_constant<int, 1>(), integral_constant<int, 8>());
}

template <typename T>
int pick_tokens(const Mx4Args& a, hipStream_t s) {
    if (a.M <= 4) return run<T, 1, 1>(a, s);
    if (a.M <= 8) return run<T, 2, 1>(a, s);
    if (a.M <= 16) return run<T, 4, 1>(a, s);
    return run<T, 4, 2>(a, s);
}

// ------------------------------------------------------------------------------------------
// tokens in 4 bits too
// ------------------------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x8 fp4_operand(u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// The bias of a tile's output channels k0 .. in LDS, once all waves are done with what was there.
__device__ __forceinline__ void stage_bias(const Mx4Args& a, float* to, int n, int k0) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = a.bias && k0 + i < a.K ? a.bias[k0 + i] : 0.0f;
    __syncthreads();
}

// A wave's RK x RM accumulators, of output channels k0 .. and tokens m0 .., through its own LDS, a tile of tokens at a
// time.  Row e of a lane's accumulator is output channel 8 * (e / 4) + 4 * half + e % 4, of token `sub`.
template <typename T, int RK, int RM>
__device__ __forceinline__ void store_tiles(const Mx4Args& a, const f32x16 (&acc)[RK][RM], T* out, const float* bias, int m0, int k0) {
    constexpr int PW = 32 * RK + 8;  // elements of a token in LDS
    const int lane = threadIdx.x & 63, sub = lane & 31, half = lane >> 5;
    const Act act = act_bounds(a.act);
    const bool whole = a.ldy % 8 == 0 && ((uintptr_t)a.y & 15) == 0 && m0 + 32 * RM <= a.M && k0 + 32 * RK <= a.K;
#pragma unroll
    for (int j = 0; j < RM; ++j) {
#pragma unroll
        for (int i = 0; i < RK; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int c = 32 * i + 8 * (e / 4) + 4 * half;
                const f32x4 b = *(const f32x4*)(bias + c);
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = clamp_act(acc[i][j][e + q] + b[q], act);
                *(uint2*)(out + sub * PW + c) = pack8<T>(v);
            }
        __builtin_amdgcn_wave_barrier();
        constexpr int CH = 4 * RK, N = 32 * CH / 64;  // 16-byte pieces of a token, and of a lane
        const int t = lane / CH, c = lane % CH * 8;
        u32x4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = ld16(out + (t + 64 / CH * i) * PW + c);
        T* y = (T*)a.y + (long long)(m0 + 32 * j + t) * a.ldy + k0 + c;
        if (whole) {
#pragma unroll
            for (int i = 0; i < N; ++i) st16(y + 64 / CH * i * a.ldy, v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const vec_t<T, 8> w = __builtin_bit_cast(vec_t<T, 8>, v[i]);
                if (m0 + 32 * j + t + 64 / CH * i < a.M)
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (k0 + c + q < a.K) y[64 / CH * i * a.ldy + q] = w[q];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

constexpr int kSpan = 8;  // steps whose scales are loaded at a time: 32 bytes of a row

// Workgroups of WK x WM waves; a wave has RK x RM tiles of 32 output channels x 32 tokens.  A step's 64 bytes of
// every row are in registers while the one before is multiplied, then go to the other of two LDS buffers, in
// 16-byte blocks whose place is turned by the row so that a column of them has no bank twice.
//
// A 32 x 32 x 64 product takes a block of each half of the wave, and any two blocks will do as long as both sides
// take the same: in product j half g has block 2 g + j.  Output channels are the rows of the product: a lane has four
// neighbouring ones of a token, which pass through LDS and are stored as 16 bytes.
template <typename T, int WK, int WM, int RK, int RM>
__global__ __launch_bounds__(64 * WK * WM, 2) void mx4x4_kernel(Mx4Args a, int mtiles, int ktiles) {
    constexpr int NW = WK * WM, TK = 32 * WK * RK, TM = 32 * WM * RM, ROWS = TK + TM;
    constexpr int KL = TK / (16 * NW), LOADS = ROWS / (16 * NW);  // of a thread: 16 rows for each wave
    constexpr int SROWS = 16 * NW;                                // rows whose scales a step loads
    static_assert(TK % SROWS == 0 && TM % SROWS == 0 && ROWS / SROWS <= kSpan, "a step's rows are of one side");
    __shared__ u32x4 data[2][ROWS][4];
    __shared__ u32x2 scale[2][kSpan / 2][ROWS];  // of two steps each
    const int tid = threadIdx.x, lane = tid & 63, sub = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK * (32 * RK), wm = wave / WK * (32 * RM);
    // tiles in columns of 8 token tiles, an XCD's next to each other: they share rows in its L2
    const int id = xcd_logical_id(blockIdx.x, gridDim.x);
    const int band = id / (8 * ktiles), height = mtiles - 8 * band < 8 ? mtiles - 8 * band : 8;
    const int m0 = (8 * band + id % (8 * ktiles) % height) * TM, k0 = id % (8 * ktiles) / height * TK;
    const int blocks = a.C / 32, steps = (blocks + 3) / 4;
    const int krows = a.K - k0 < TK ? a.K - k0 : TK, mrows = a.M - m0 < TM ? a.M - m0 : TM;
    const uint32_t pitch = a.C / 2;
    // (rows behind the last read as zero; a tile's rows are below 2^28 bytes)
    const __amdgpu_buffer_rsrc_t rq = mm::rsrc(a.q + (long long)k0 * pitch, krows * pitch);
    const __amdgpu_buffer_rsrc_t rx = mm::rsrc((const uint8_t*)a.x + (long long)m0 * pitch, mrows * pitch);
    const int lrow = tid >> 2, chunk = tid & 3;
    const uint32_t lat = lrow * pitch + 16 * chunk;
    u32x4 raw[LOADS];
    auto fetch = [&](int s) {
        const bool in = 4 * s + chunk < blocks;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const bool tok = i >= KL;
            const int r = 16 * NW * (tok ? i - KL : i);
            raw[i] = __builtin_amdgcn_raw_buffer_load_b128(tok ? rx : rq, in && lrow + r < (tok ? mrows : krows) ? lat : mm::kOob,
                                                           s * (kStep / 2) + r * pitch, 0);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) data[buf][lrow + 16 * NW * i][chunk ^ (lrow >> 2 & 3)] = raw[i];
    };
    // Scales of kSpan steps at a time: a step loads some of the rows, 32 bytes of four lanes each, for the steps after the
    // present eight.  Where two steps have fewer than eight they are the last eight of the row, moved down on
    // their way to LDS.  (A row behind the last takes the last one's: its outputs are not stored.  Rows of fewer than
    // eight are loaded before the first step, and here any eight bytes, which no step uses: of the side's own codes,
    // 16 bytes for each scale, so that they end before the last row of that side does.)
    constexpr int PARTS = ROWS / SROWS;
    u32x2 sraw;
    const int spart = tid & 3;
    const bool some = blocks >= 8;
    const uint8_t* kscales = some ? a.scales + (long long)k0 * blocks : a.q;
    const uint8_t* mscales = some ? a.xscales + (long long)m0 * blocks : (const uint8_t*)a.x;
    auto scale_at = [&](int group) {
        const int b = 4 * kSpan * group + 8 * spart;
        return b < blocks ? b : blocks & ~7;
    };
    auto fetch_scales = [&](int group, int part) {
        const int want = scale_at(group), at = want + 8 <= blocks ? want : some ? blocks - 8 : 0;
        const bool tok = SROWS * part >= TK;
        const int r = SROWS * part + (tid >> 2) - (tok ? TK : 0), most = (tok ? mrows : krows) - 1;
        return *(const u32x2_any*)((tok ? mscales : kscales) + (uint32_t)(r < most ? r : most) * (uint32_t)blocks + at);
    };
    auto stage_scales = [&](int group, int part, u32x2 v) {
        const int want = scale_at(group), gone = want + 8 <= blocks ? 0 : want - (blocks - 8);  // (8: none left)
        const uint64_t u = (__builtin_bit_cast(uint64_t, v) >> (4 * gone)) >> (4 * gone);
        scale[group & 1][spart][SROWS * part + (tid >> 2)] = __builtin_bit_cast(u32x2, u);
    };
    f32x16 acc[RK][RM];
#pragma unroll
    for (int i = 0; i < RK; ++i)
#pragma unroll
        for (int j = 0; j < RM; ++j) acc[i][j] = f32x16{};
    fetch(0);
    if (some) {
        u32x2 v[PARTS];
#pragma unroll
        for (int q = 0; q < PARTS; ++q) v[q] = fetch_scales(0, q);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) stage_scales(0, q, v[q]);
    } else {
        for (int row = tid; row < ROWS; row += 64 * NW) {
            const bool tok = row >= TK;
            const int r = tok ? row - TK : row, most = (tok ? mrows : krows) - 1;
            const uint8_t* p = (tok ? a.xscales + (long long)m0 * blocks : a.scales + (long long)k0 * blocks) + (r < most ? r : most) * blocks;
            u32x2 v = {0, 0};
            for (int b = 0; b < blocks; ++b) v[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
            scale[0][0][row] = v;
        }
    }
    stage(0);
    fetch(steps > 1 ? 1 : 0);
    sraw = fetch_scales(1, 0);
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        // (without branches, which would pull loads and products apart: the last steps load and store once more, and
        // the last parts' scales of a group are loaded again)
        const int buf = s & 1;
        auto part_of = [](int t) { return t % kSpan < PARTS ? t % kSpan : PARTS - 1; };
        stage(buf ^ 1);
        stage_scales(s / kSpan + 1, part_of(s), sraw);
        fetch(s + 2 < steps ? s + 2 : steps - 1);
        sraw = fetch_scales((s + 1) / kSpan + 1, part_of(s + 1));
        // (the compiler would move the loads behind the products, where their registers are free sooner)
        __builtin_amdgcn_sched_barrier(0);
        const u32x2* sp = scale[s / kSpan & 1][s % kSpan / 2];
        int sk[RK], sm[RM];
#pragma unroll
        for (int i = 0; i < RK; ++i) sk[i] = sp[wk + 32 * i + sub][s & 1] >> (16 * half);
#pragma unroll
        for (int i = 0; i < RM; ++i) sm[i] = sp[TK + wm + 32 * i + sub][s & 1] >> (16 * half);
        auto block = [&](auto which) {
            constexpr int J = decltype(which)::value;
            i32x8 fk[RK], fm[RM];
            const int place = (2 * half + J) ^ (sub >> 2 & 3);
#pragma unroll
            for (int i = 0; i < RK; ++i) fk[i] = fp4_operand(data[buf][wk + 32 * i + sub][place]);
#pragma unroll
            for (int i = 0; i < RM; ++i) fm[i] = fp4_operand(data[buf][TK + wm + 32 * i + sub][place]);
#pragma unroll
            for (int i = 0; i < RK; ++i)
#pragma unroll
                for (int j = 0; j < RM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fk[i], fm[j], acc[i][j], 4, 4, J, sk[i], J, sm[j]);
        };
        block(std::integral_constant<int, 0>());
        block(std::integral_constant<int, 1>());
        __syncthreads();
    }
    float* bias = (float*)&scale[0][0][0];
    stage_bias(a, bias, TK, k0);
    store_tiles<T, RK, RM>(a, acc, (T*)&data[0][0][0] + wave * 32 * (32 * RK + 8), bias + wk, m0 + wm, k0 + wk);
    static_assert(NW * 32 * (32 * RK + 8) * (int)sizeof(T) <= (int)sizeof(data), "the outputs' LDS");
}

// The order of a block of 16 products: one of the first kind behind each of the first eight, one of the second behind the
// others.
constexpr int kProduct = 0x008, kLoad = 0x020, kLdsRead = 0x100, kLdsWrite = 0x200;
template <int FIRST, int SECOND>
__device__ __forceinline__ void order() {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
        if (i < 8)
            __builtin_amdgcn_sched_group_barrier(FIRST, 1, 0);
        else
            __builtin_amdgcn_sched_group_barrier(SECOND, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// The same for products that fill the card: 256 x 256 outputs by four waves, 128 x 128 each in half of a SIMD's
// registers, steps of 256 channels.  A wave reads operands at half the rate per product, so LDS no longer takes
// longer than the matrix units; but there is one wave a SIMD, so its own instructions have to follow each other without a
// pause.  A step is four blocks of 16 products; in each the next block's operands are read, and in turn the next
// step goes to LDS and the one after is loaded.  The barrier between the third and the fourth says that all waves have
// read this step and stored the next, whose first operands are read in the fourth.
//
// 8192 tokens, 4096 -> 8192 channels, take 185 us (3.0 PFLOP/s; 4.4 inside a tile, the rest are the starts and ends of the
// four tiles that each CU has).  No unit is full: at the 1.9 GHz that the card holds here the matrix units, whose
// instruction alone makes 8.1 PFLOP/s, are busy in 37% of the cycles (55% inside a tile), LDS in 39% and 15% more for banks
// asked twice, and the one wave of a SIMD waits for results in 22%.  What bounds it is that one wave, which has to issue all of
// it one after the other.  With eight waves and a 128-channel step it was 230, with two workgroups of 128 x 256 a CU 224.
template <typename T>
__global__ __launch_bounds__(256, 1) void mx4x4_large_kernel(Mx4Args a, int mtiles, int ktiles) {
    constexpr int TILE = 256, ROWS = 2 * TILE, R = 4, LOADS = 16, SPAN = 4;
    __shared__ u32x4 data[2][ROWS][8];
    __shared__ u32x2 scale[2][SPAN][ROWS];
    const int tid = threadIdx.x, lane = tid & 63, sub = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % 2 * 128, wm = wave / 2 * 128;
    const int id = xcd_logical_id(blockIdx.x, gridDim.x);
    const int band = id / (8 * ktiles), height = mtiles - 8 * band < 8 ? mtiles - 8 * band : 8;
    const int m0 = (8 * band + id % (8 * ktiles) % height) * TILE, k0 = id % (8 * ktiles) / height * TILE;
    const int blocks = a.C / 32, steps = (blocks + 7) / 8;
    const int krows = a.K - k0 < TILE ? a.K - k0 : TILE, mrows = a.M - m0 < TILE ? a.M - m0 : TILE;
    const uint32_t pitch = a.C / 2;
    const __amdgpu_buffer_rsrc_t rq = mm::rsrc(a.q + (long long)k0 * pitch, krows * pitch);
    const __amdgpu_buffer_rsrc_t rx = mm::rsrc((const uint8_t*)a.x + (long long)m0 * pitch, mrows * pitch);
    const int lrow = tid >> 3, chunk = tid & 7;
    const uint32_t lat = lrow * pitch + 16 * chunk;
    u32x4 raw[LOADS];
    auto fetch = [&](int s, auto from) {  // eight of them
        constexpr int F = decltype(from)::value;
        const bool in = 8 * s + chunk < blocks;
#pragma unroll
        for (int i = F; i < F + 8; ++i) {
            const int r = 32 * (i - F);
            raw[i] = __builtin_amdgcn_raw_buffer_load_b128(F ? rx : rq, in && lrow + r < (F ? mrows : krows) ? lat : mm::kOob,
                                                           s * 128 + r * pitch, 0);
        }
    };
    auto stage = [&](int buf, auto from) {
        constexpr int F = decltype(from)::value;
#pragma unroll
        for (int i = F; i < F + 8; ++i) data[buf][lrow + 32 * i][chunk ^ (lrow & 7)] = raw[i];
    };
    // scales as in the kernel above: of SPAN steps at a time, a quarter of the rows each step, here two rows a lane
    u32x2 sraw[2];
    const int spart = tid & 3;
    auto scale_at = [&](int group) {
        const int b = 8 * (SPAN * group + spart);
        return b < blocks ? b : blocks & ~7;
    };
    auto fetch_scales = [&](int group, int part, u32x2 (&sraw)[2]) {
        const int want = scale_at(group), at = want + 8 <= blocks ? want : blocks - 8;
        const uint8_t* p = part >= 2 ? a.xscales + (long long)m0 * blocks : a.scales + (long long)k0 * blocks;
        const int most = (part >= 2 ? mrows : krows) - 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 128 * (part & 1) + 64 * i + (tid >> 2);
            sraw[i] = *(const u32x2_any*)(p + (uint32_t)(r < most ? r : most) * (uint32_t)blocks + at);
        }
    };
    auto stage_scales = [&](int group, int part, const u32x2 (&sraw)[2]) {
        const int want = scale_at(group), gone = want + 8 <= blocks ? 0 : want - (blocks - 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t u = (__builtin_bit_cast(uint64_t, sraw[i]) >> (4 * gone)) >> (4 * gone);
            scale[group & 1][spart][128 * part + 64 * i + (tid >> 2)] = __builtin_bit_cast(u32x2, u);
        }
    };
    f32x16 acc[R][R];
    const std::integral_constant<int, 0> zero;
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 3> three;
    const std::integral_constant<int, 8> eight;
    struct Operands {
        u32x4 k[R], m[R];
    };
    auto read = [&](int buf, int j, Operands& f) {
        const int place = (4 * half + j) ^ (sub & 7);
#pragma unroll
        for (int i = 0; i < R; ++i) f.k[i] = data[buf][wk + 32 * i + sub][place];
#pragma unroll
        for (int i = 0; i < R; ++i) f.m[i] = data[buf][TILE + wm + 32 * i + sub][place];
    };
    uint32_t sk[R], sm[R];
    auto read_scales = [&](int s, uint32_t (&k)[R], uint32_t (&m)[R]) {
        const u32x2* sp = scale[s / SPAN & 1][s % SPAN];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            k[i] = sp[wk + 32 * i + sub][half];
            m[i] = sp[TILE + wm + 32 * i + sub][half];
        }
    };
    auto multiply = [&](const Operands& f, auto which) {
        constexpr int J = decltype(which)::value;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < R; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(f.k[i]), fp4_operand(f.m[j]), acc[i][j], 4, 4, J, sk[i], J, sm[j]);
    };
    fetch(0, zero);
    fetch(0, eight);
    u32x2 all[SPAN][2];
#pragma unroll
    for (int q = 0; q < SPAN; ++q) fetch_scales(0, q, all[q]);
    stage(0, zero);
    stage(0, eight);
    // (in the loop's order, by which the compiler counts what it waits for)
    fetch_scales(1, 0, sraw);
    fetch(steps > 1 ? 1 : 0, zero);
    fetch(steps > 1 ? 1 : 0, eight);
#pragma unroll
    for (int q = 0; q < SPAN; ++q) stage_scales(0, q, all[q]);
    __syncthreads();
    Operands f, g;
    read(0, 0, f);
    read_scales(0, sk, sm);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) acc[i][j] = f32x16{};
    for (int s = 0; s < steps; ++s) {
        // (without branches: the last steps load and store once more)
        const int buf = s & 1, then = s + 2 < steps ? s + 2 : steps - 1;
        read(buf, 1, g);
        stage(buf ^ 1, zero);
        multiply(f, zero);
        order<kLdsRead, kLdsWrite>();
        read(buf, 2, f);
        stage(buf ^ 1, eight);
        stage_scales(s / SPAN + 1, s % SPAN, sraw);
        multiply(g, one);
        order<kLdsRead, kLdsWrite>();
        read(buf, 3, g);
        fetch_scales((s + 1) / SPAN + 1, (s + 1) % SPAN, sraw);
        fetch(then, zero);
        multiply(f, two);
        order<kLdsRead, kLoad>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        read(buf ^ 1, 0, f);
        uint32_t nk[R], nm[R];
        read_scales(s + 1, nk, nm);
        fetch(then, eight);
        multiply(g, three);
        order<kLdsRead, kLoad>();
#pragma unroll
        for (int i = 0; i < R; ++i) sk[i] = nk[i], sm[i] = nm[i];
    }
    float* bias = (float*)&data[1][0][0];
    stage_bias(a, bias, TILE, k0);
    store_tiles<T, R, R>(a, acc, (T*)&data[0][0][0] + wave * 32 * (32 * R + 8), bias + wk, m0 + wm, k0 + wk);
    static_assert(4 * 32 * (32 * R + 8) * (int)sizeof(T) <= (int)sizeof(data[0]), "the outputs' LDS");
}

// A few tokens (16 MT): the waves share the channels as in mx4_kernel, tokens are loaded as output channels are.
// HBM bounds it: 4096 channels -> 65536 with 1 token 32 us, 16 tokens 38, 32 tokens 43.
template <typename T, int MT, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void mx4x4_few_kernel(Mx4Args a) {
    constexpr int TILES = RT + MT;
    __shared__ u32x4 stage[NW][TILES > RT * MT ? TILES : RT * MT][64];
    __shared__ u32x2 scales[NW][TILES][64];
    auto part = [&](int w, int r, int m) { return (f32x4*)stage[w] + (r * MT + m) * 64; };
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane & 15, grp = lane >> 4;
    const int blocks = a.C / 32, steps = (blocks + 3) / 4;
    const int k0 = blockIdx.x * (16 * RT), m0 = blockIdx.y * (16 * MT);
    const int lrow = lane >> 2, lchunk = (lane & 3) ^ (lrow >> 2);
    const int krows = a.K - k0 < 16 * RT ? a.K - k0 : 16 * RT;
    const int mrows = a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT;
    const uint32_t pitch = a.C / 2;
    const __amdgpu_buffer_rsrc_t rq = mm::rsrc(a.q + (long long)k0 * pitch, krows * pitch);
    const __amdgpu_buffer_rsrc_t rx = mm::rsrc((const uint8_t*)a.x + (long long)m0 * pitch, mrows * pitch);
    struct Step {
        u32x4 w[TILES];
    };
    auto fetch = [&](int s, Step& v) {
        const bool in = s * 4 + lchunk < blocks;
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
            const int row = 16 * (r < RT ? r : r - RT);
            const uint32_t at = (row + lrow) * pitch + 16 * lchunk;
            v.w[r] = __builtin_amdgcn_raw_buffer_load_b128(r < RT ? rq : rx, in ? at : mm::kOob, s * (kStep / 2), 0);
        }
    };
    f32x4 total[RT][MT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) total[r][m] = f32x4{};
    const int place = sub * 4 + (grp ^ (sub >> 2));
    const int share = (steps + NW - 1) / NW, first = wave * share, end = first + share < steps ? first + share : steps;
    if (first < end) {
        StepScales<TILES> ss;
        ss.blocks = blocks;
        ss.part = 8 * (lane & 3);
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
            const int at = 16 * (r < RT ? r : r - RT) + lrow, most = (r < RT ? krows : mrows) - 1, row = at < most ? at : most;
            ss.row[r] = r < RT ? a.scales + (long long)(k0 + row) * blocks : a.xscales + (long long)(m0 + row) * blocks;
        }
        Step v;
        ss.fetch(first);
        fetch(first, v);
        for (int s0 = first; s0 < end; s0 += kSteps) {
            ss.stage(s0, scales[wave]);
            ss.fetch(s0 + kSteps < end ? s0 + kSteps : s0);
            __builtin_amdgcn_wave_barrier();
            const int n = end - s0 < kSteps ? end - s0 : kSteps;
            for (int j = 0; j < n; ++j) {
                uint32_t scale[TILES];
#pragma unroll
                for (int r = 0; r < TILES; ++r) {
                    stage[wave][r][lane] = v.w[r];
                    scale[r] = StepScales<TILES>::read(scales[wave][r], j);
                }
                fetch(s0 + j + 1 < end ? s0 + j + 1 : end - 1, v);
                __builtin_amdgcn_wave_barrier();
                i32x8 f[TILES];
#pragma unroll
                for (int r = 0; r < TILES; ++r) f[r] = fp4_operand(stage[wave][r][place]);
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        total[r][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f[RT + m], f[r], total[r][m], 4, 4, 0, scale[RT + m], 0, scale[r]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) part(wave, r, m)[lane] = total[r][m];
    __syncthreads();
    const Act act = act_bounds(a.act);
    for (int j = threadIdx.x; j < RT * MT * 64; j += 64 * NW) {
        const int l = j & 63, m = (j >> 6) % MT, r = (j >> 6) / MT;
        const int k = k0 + 16 * r + (l & 15);
        if (k >= a.K) continue;
        f32x4 v = part(0, r, m)[l];
#pragma unroll
        for (int q = 1; q < NW; ++q) v += part(q, r, m)[l];
        const float bias = a.bias ? a.bias[k] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = m0 + 16 * m + 4 * (l >> 4) + i;
            if (t < a.M) ((T*)a.y)[(long long)t * a.ldy + k] = (T)clamp_act(v[i] + bias, act);
        }
    }
}

template <typename T>
int quantize(const Mx4Args& a, hipStream_t s) {
    const long long pieces = (long long)a.M * a.C / 8;
    const int grid = (int)((pieces + 256 * kPer - 1) / (256 * kPer));
    if (rows16(a.x, a.ldx, sizeof(T)))
        mx4_quantize_kernel<T, true><<<grid, 256, 0, s>>>(a, pieces);
    else
        mx4_quantize_kernel<T, false><<<grid, 256, 0, s>>>(a, pieces);
    return (int)hipGetLastError();
}
template <typename T>
int dequantize(const Mx4Args& a, hipStream_t s) {
    const long long pieces = (long long)a.M * a.C / 8;
    const int grid = (int)((pieces + 256 * kPer - 1) / (256 * kPer));
    if (rows16(a.y, a.ldy, sizeof(T)))
        mx4_dequantize_kernel<T, true><<<grid, 256, 0, s>>>(a, pieces);
    else
        mx4_dequantize_kernel<T, false><<<grid, 256, 0, s>>>(a, pieces);
    return (int)hipGetLastError();
}
template <typename T>
int product(const Mx4Args& a, hipStream_t s) {
    using std::integral_constant;
    auto few = [&](auto mt, auto rt, auto nw) {
        constexpr int MT = decltype(mt)::value, RT = decltype(rt)::value, NW = decltype(nw)::value;
        const dim3 grid((a.K + 16 * RT - 1) / (16 * RT), (a.M + 16 * MT - 1) / (16 * MT));
        mx4x4_few_kernel<T, MT, RT, NW><<<grid, 64 * NW, 0, s>>>(a);
        return (int)hipGetLastError();
    };
    auto tiles = [&](auto wk, auto wm, auto rk, auto rm) {
        constexpr int WK = decltype(wk)::value, WM = decltype(wm)::value, RK = decltype(rk)::value, RM = decltype(rm)::value;
        const int ktiles = (a.K + 32 * WK * RK - 1) / (32 * WK * RK), mtiles = (a.M + 32 * WM * RM - 1) / (32 * WM * RM);
        mx4x4_kernel<T, WK, WM, RK, RM><<<ktiles * mtiles, 64 * WK * WM, 0, s>>>(a, mtiles, ktiles);
        return (int)hipGetLastError();
    };
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const integral_constant<int, 4> four;
    const integral_constant<int, 8> eight;
    // Few outputs leave tiles of 128 x 128 on few CUs, each with a long way over the channels to itself; many tokens have
    // the waves that share the channels read the weights again for every 64 of them.  At 4096 channels, us, shared / tiles:
    // 16 x 4096 outputs 4.5 / 22, 128 x 8192 11 / 22, 32 x 32768 22 / 28, 256 x 4096 11 / 22, 48 x 32768 31 / 29, 256 x 8192
    // 23 / 22, 256 x 32768 84 / 38.  (Two output tiles on 4 waves or one on 8: 16 x 4096 5.4 / 4.5, 32 x 8192 6.4 / 7.5,
    // 64 x 8192 8.1 / 11.)
    if (a.M <= 32 || (long long)a.M * a.K <= 1 << 20) {
        const int tokens = a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64;
        const bool wide = (long long)((a.K + 15) / 16) * ((a.M + tokens - 1) / tokens) >= 512;
        if (tokens == 16) return wide ? few(one, two, four) : few(one, one, eight);
        if (tokens == 32) return wide ? few(two, two, four) : few(two, one, eight);
        return wide ? few(four, two, four) : few(four, one, eight);
    }
    // Tiles of 256 x 256 take one CU each, and 41 us for 4096 channels whether they fill the card or not: 2048 x 4096
    // outputs (128 tiles) take 33 us in those of 128 x 128, 2560 x 4096 43, 3328 x 4096 60 / 41, 8192 x 4096 115 / 86.
    // Their longer start and end want channels to pay for them: 4096 x 4096 outputs of 256 channels 17 / 16 us, of 1024
    // 22 / 22, of 4096 45 / 61.
    const int ktiles = (a.K + 255) / 256, mtiles = (a.M + 255) / 256;
    if ((long long)ktiles * mtiles >= 160 && a.C >= 1024) {
        mx4x4_large_kernel<T><<<ktiles * mtiles, 256, 0, s>>>(a, mtiles, ktiles);
        return (int)hipGetLastError();
    }
    return tiles(two, two, two, two);
}

}  // namespace

long long mx4x4_threads(const fcm_mx4_problem& p) {
    return ((long long)p.M + 127) / 128 * ((p.K + 127) / 128) * 256;
}

int launch_mx4_quantize(const Mx4Args& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return quantize<float>(a, s);
    if (dtype == FCM_F16) return quantize<_Float16>(a, s);
    return quantize<__bf16>(a, s);
}
int launch_mx4_dequantize(const Mx4Args& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return dequantize<float>(a, s);
    if (dtype == FCM_F16) return dequantize<_Float16>(a, s);
    return dequantize<__bf16>(a, s);
}
int launch_mx4(const Mx4Args& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    return dtype == FCM_F16 ? pick_tokens<_Float16>(a, s) : pick_tokens<__bf16>(a, s);
}
int launch_mx4x4(const Mx4Args& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    return dtype == FCM_F16 ? product<_Float16>(a, s) : product<__bf16>(a, s);
}

}  // namespace fcm
