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

// The activation as a clamp that lets NaN through (a median of three would not).
__device__ __forceinline__ float clamp_act(float v, Act act) {
    return v < act.lo ? act.lo : v > act.hi ? act.hi : v;
}

// The conversions take a block's power of two as a float, by its exponent bits alone: those are the stored
// scale (0 stands for 2^-127, 255 for NaN).
__device__ __forceinline__ float scale_float(uint32_t code) { return __builtin_bit_cast(float, code << 23); }

// ------------------------------------------------------------------------------------------
// quantisation: eight channels a lane, four lanes a block
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
// bf16 pieces of eight 16-bit inputs: fp16's 11 bits are two of them, exactly.
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
            out[1][i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, rh), __builtin_bit_cast(uint32_t, rl), 0x07060302u);
        }
    }
}

constexpr int kStep = 128;  // channels a wave takes at a time: 64 bytes of an output channel
// Byte offset in x of the channels behind the last, which read as zero: beyond every range of a
// tile's tokens (31 row strides below 2^26 elements and 2^20 channels, 0xf8200000 bytes), and with a
// step's own offset of up to 2^21 still below 2^32.
constexpr uint32_t kBehind = 0xfc000000u;

// A workgroup has 16 * RT output channels and 16 * MT tokens (or 4, 8: NI = 1, 2); its waves take
// every NW-th step of 128 channels and add their sums through LDS.
//
// Four neighbouring lanes load 64 bytes of an output channel (16 lanes 256 bytes of a token), and the wave passes
// them through its own piece of LDS, in 16-byte chunks whose place is turned by the row so that a column of them
// has no bank twice: matrix operands want neighbouring lanes on different rows, 64 separate accesses a load.
// Lane l then holds one whole block, l / 16 of the step's four, of output channel l % 16; the conversion to bf16
// multiplies with the block's power of two (exact), and the four products of a step take eight channels of each
// block, in the same order from both sides.
template <typename T, int NI, int MT, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void mx4_kernel(Mx4Args a) {
    constexpr int XI = MT * NI, TOKENS = 4 * XI, XP = XPieces<T>::N;
    static_assert(TOKENS <= 32, "kBehind lies behind a tile's tokens");
    __shared__ u32x4 stage[NW][RT + XP * XI][64];
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
    const __amdgpu_buffer_rsrc_t rs = mm::rsrc(a.scales + (long long)k0 * blocks, (uint32_t)krows * blocks);
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
        uint32_t scale[RT];
    };
    auto fetch = [&](int s, Step& v) {
        // (channels behind the last: codes and tokens read as zero)
        const bool in = s * 4 + lchunk < blocks, mine = s * 4 + grp < blocks;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const uint32_t at = (16 * r + lrow) * (uint32_t)(a.C / 2) + 16 * lchunk;
            v.w[r] = __builtin_amdgcn_raw_buffer_load_b128(rq, in ? at : mm::kOob, s * (kStep / 2), 0);
            const uint32_t sat = (16 * r + sub) * (uint32_t)blocks + grp;
            v.scale[r] = __builtin_amdgcn_raw_buffer_load_b8(rs, mine ? sat : mm::kOob, s * 4, 0);
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
    auto use = [&](Step& v, int then) {
        uint32_t scale[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            stage[wave][r][lane] = v.w[r];
            scale[r] = v.scale[r];
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
    const int last = steps - 1;
    auto at_most = [&](int s) { return s < last ? s : last; };
    Step v;
    fetch(at_most(wave), v);
    for (int s = wave; s < steps; s += NW) use(v, at_most(s + NW));
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
    const long long rows = (long long)((a.K + 15) / 16) * tiles;
    if (rows >= 1024) return go(integral_constant<int, 2>(), integral_constant<int, 4>());
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
// A workgroup of four waves has 128 x 128 outputs, a wave 64 x 64.
template <typename T>
__global__ __launch_bounds__(256) void mx4x4_kernel(Mx4Args a, int ktiles) {
    const int lane = threadIdx.x & 63, sub = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = blockIdx.x / ktiles * 128 + (wave >> 1) * 64, k0 = blockIdx.x % ktiles * 128 + (wave & 1) * 64;
    const int blocks = a.C / 32;
    const uint8_t* x = (const uint8_t*)a.x;
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
    for (int b = 0; b < blocks; b += 4) {
        i32x8 fx[4], fw[4];
        int sx[4], sw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (rows behind the last repeat it, and are not stored)
            const int m = m0 + 16 * i + sub < a.M ? m0 + 16 * i + sub : a.M - 1;
            const int k = k0 + 16 * i + sub < a.K ? k0 + 16 * i + sub : a.K - 1;
            u32x4 vx = {}, vw = {};
            sx[i] = sw[i] = 0;
            if (b + grp < blocks) {
                vx = ld16(x + ((long long)m * blocks + b + grp) * 16);
                vw = ld16(a.q + ((long long)k * blocks + b + grp) * 16);
                sx[i] = a.xscales[(long long)m * blocks + b + grp];
                sw[i] = a.scales[(long long)k * blocks + b + grp];
            }
            fx[i] = i32x8{(int)vx[0], (int)vx[1], (int)vx[2], (int)vx[3], 0, 0, 0, 0};
            fw[i] = i32x8{(int)vw[0], (int)vw[1], (int)vw[2], (int)vw[3], 0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fx[i], fw[j], acc[i][j], 4, 4, 0, sx[i], 0, sw[j]);
    }
    const Act act = act_bounds(a.act);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = k0 + 16 * j + sub;
        if (k >= a.K) continue;
        const float bias = a.bias ? a.bias[k] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int m = m0 + 16 * i + 4 * grp + e;
                if (m < a.M) ((T*)a.y)[(long long)m * a.ldy + k] = (T)clamp_act(acc[i][j][e] + bias, act);
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
    const int ktiles = (a.K + 127) / 128;
    mx4x4_kernel<T><<<(a.M + 127) / 128 * ktiles, 256, 0, s>>>(a, ktiles);
    return (int)hipGetLastError();
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
