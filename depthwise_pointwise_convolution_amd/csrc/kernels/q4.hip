// q4.hip -- pointwise layer with 4-bit weights and group scales for a few tokens:
//   y[m][k] = act(bias[k] + sum_groups scale[k][g] * sum_{c in g} (q[k][c] - zero[k][g]) x[m][c]).
//
// A tile of tokens, 32 at most, reads the weights once, and the bytes of q are its floor; the products
// run on the matrix cores, where the spare tokens of a 16-row tile cost nothing.  On MI355X, 65536 x
// 4096: one token 28 us (4.9 TB/s of codes and scales), 16 tokens with groups of 64 39 us (3.7
// TB/s; vector units busy 42% of the time with unpacking and scales, the loads take turns with
// them), 32 tokens 64 us (the products' and scales' work for each 16); 8192 x 2048 for one token 4.2 us,
// most of it launch and one memory latency.  More tokens than 32 read and unpack the weights again.
#include "mm_common.h"
#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

// The activation as a clamp that lets NaN through (a median of three would not).
__device__ __forceinline__ float clamp_act(float v, Act act) {
    return v < act.lo ? act.lo : v > act.hi ? act.hi : v;
}

// A word of 8 codes as 8 storage values 16 + q, exact in both types: q goes into the mantissa of a
// number in [16, 32).  Pair i is (code i, code i + 4): the other operand has its channels in the
// same order.  Eight operations for eight codes, with no conversion: a shift and an and-or each
// (with the constants in registers; as literals they make an and and an or of it).
template <typename T>
struct Codes {
    static constexpr bool F16 = std::is_same<T, _Float16>::value;
    // 16.0 = 0x4c00 in fp16, where 1 is 1 << 6, and 0x4180 in bf16, where 1 is 1 << 3
    uint32_t mask, base;
    __device__ __forceinline__ Codes() : mask(F16 ? 0x03c003c0u : 0x00780078u),
                                         base(F16 ? 0x4c004c00u : 0x41804180u) {
        asm("" : "+s"(mask), "+v"(base));
    }
    __device__ __forceinline__ uint32_t pick(uint32_t w) const { return (w & mask) | base; }
    __device__ __forceinline__ u32x4 unpack(uint32_t w) const {
        if constexpr (F16) return u32x4{pick(w << 6), pick(w << 2), pick(w >> 2), pick(w >> 6)};
        else return u32x4{pick(w << 3), pick(w >> 1), pick(w >> 5), pick(w >> 9)};
    }
};

// Eight channels of x in that order: (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ u32x4 order_codes(u32x4 v) {
    u32x4 r;
    r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
    r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
    r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
    r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
    return r;
}

// Words w[j] of lane group i  <->  words w[i] of lane group j (groups of 16 lanes): a lane's 32
// consecutive channels become its 8 channels of each of four 32-channel blocks.
__device__ __forceinline__ void transpose_groups(uint32_t* w) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    u2 p;
    p = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false), w[0] = p[0], w[2] = p[1];
    p = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false), w[1] = p[0], w[3] = p[1];
    p = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false), w[0] = p[0], w[1] = p[1];
    p = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false), w[2] = p[0], w[3] = p[1];
}

constexpr int kStep = 128;   // channels a wave takes at a time: 64 bytes of an output channel
constexpr int kSpan = 8;      // steps whose scales a workgroup holds in LDS at a time

// Byte offset in x of the channels behind the last, which read as zero: beyond every range of a
// tile's tokens (31 row strides below 2^26 elements and 2^20 channels, 0xf8200000 bytes), and with a
// step's own offset of up to 2^21 still below 2^32.
constexpr uint32_t kBehind = 0xfc000000u;

// A workgroup has 16 * RT output channels and 16 * MT tokens (or 4, 8: NI = 1, 2); its waves take
// every NW-th step of 128 channels and add their sums through LDS.
//
// The matrix instructions want neighbouring lanes to hold different output channels, but such a
// load is 64 separate 16-byte accesses.  So four neighbouring lanes load 64 bytes of one channel
// (16 lanes 256 bytes of a token), and the wave passes them through its own piece of LDS, in 16-byte
// chunks whose place is turned by the row so that a column of them has no bank twice.  The next
// step's loads are in flight meanwhile.
//
// In a step lane l then holds chunk l / 16, 32 channels, of output channel l % 16.  With a group of
// 128 the four matrix products of a step may take its channels in any order, so the words are used
// as they lie; smaller groups need each product within one 32-channel block, so the words are
// exchanged between lane groups first.
//
// The matrix products sum (16 + q) x in fp32 within a group; a product with ones gives the group's
// sum of x, and then  total += scale * sum - scale * (16 + zero) * sum_x,  both factors exact in
// fp32.  The offset 16 costs the exact sum at most a factor of 31 / |q - zero| in rounding, far
// below the rounding of y.
//
// Tokens sit in the accumulator's rows 4 * (l / 16) + i: with at most 4 (8) tokens they are put
// into rows with i = 0 (i < 2), and the other rows' scaling is not done.
template <typename T, int GROUP, int NI, int MT, int RT, int NW, bool WIDE>
__global__ __launch_bounds__(64 * NW, (MT == 2 && RT == 2) || (GROUP == 32 && RT == 4) ? 3 : 4) void q4_kernel(Q4Args a) {
    constexpr int GS = kStep / GROUP;      // groups of a step
    constexpr int SG = kSpan * GS;
    static_assert(kSpan % NW == 0, "a wave's steps are the same ones of every span");
    constexpr int XI = MT * NI;            // loads of 4 tokens
    constexpr int TOKENS = 4 * XI;
    static_assert(TOKENS <= 32, "kBehind lies behind a tile's tokens");
    // a wave's steps pass through `stage`; its sums lie there at the end
    __shared__ u32x4 stage[NW][RT + XI][64];
    __shared__ float2 sz[SG][16 * RT];
    auto part = [&](int w, int r, int i) { return (float*)stage[w] + (r * XI + i) * 64; };
    static_assert(RT * XI <= 4 * (RT + XI), "the sums fit");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane & 15, grp = lane >> 4;
    const int groups = (a.C + GROUP - 1) / GROUP;
    const int steps = (a.C + kStep - 1) / kStep;
    const int k0 = blockIdx.x * (16 * RT);
    const int m0 = blockIdx.y * TOKENS;
    // Loading: this lane's output channel and chunk of it, as range-checked offsets from the tile's
    // first channel and token (channels and tokens behind the last read as zero), which a step
    // moves by a scalar.
    const int lrow = lane >> 2, lchunk = (lane & 3) ^ (lrow >> 2);
    const int krows = a.K - k0 < 16 * RT ? a.K - k0 : 16 * RT;
    const int trows = a.M - m0 < TOKENS ? a.M - m0 : TOKENS;
    const __amdgpu_buffer_rsrc_t rq =
        mm::rsrc(a.q + (long long)k0 * (a.C / 2), (uint32_t)krows * (a.C / 2));
    const __amdgpu_buffer_rsrc_t rx = mm::rsrc((const T*)a.x + (long long)m0 * a.ldx,
                                               ((uint32_t)(trows - 1) * (uint32_t)a.ldx + a.C) * 2);
    const T* scale0 = (const T*)a.scales + (long long)k0 * groups;
    const uint8_t* zero0 = a.zeros ? a.zeros + (long long)k0 * groups : nullptr;
    uint32_t qat[RT], xat[XI];
#pragma unroll
    for (int r = 0; r < RT; ++r) qat[r] = (16 * r + lrow) * (a.C / 2) + 16 * lchunk;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int t = 4 * i + grp;  // of the tile's tokens
        xat[i] = (t * (uint32_t)a.ldx + 8 * (sub ^ (t & 15))) * 2;
    }
    struct Step {
        u32x4 w[RT], x[XI];
    };
    auto fetch = [&](int s, Step& v) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if constexpr (WIDE) {
                v.w[r] = __builtin_amdgcn_raw_buffer_load_b128(rq, qat[r], s * (kStep / 2), 0);
            } else {
                const int c = s * kStep + 32 * lchunk;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v.w[r][j] = __builtin_amdgcn_raw_buffer_load_b32(
                        rq, c + 8 * j < a.C ? qat[r] + 4 * j : mm::kOob, s * (kStep / 2), 0);
            }
        }
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            uint32_t at = xat[i];
            if (!WIDE && s * kStep + 8 * (sub ^ ((4 * i + grp) & 15)) >= a.C) at = kBehind;
            v.x[i] = __builtin_amdgcn_raw_buffer_load_b128(rx, at, s * kStep * 2, 0);
        }
    };
    const u32x4 ones = std::is_same<T, _Float16>::value
                           ? u32x4{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u}
                           : u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const Codes<T> codes;
    float total[RT][XI];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < XI; ++i) total[r][i] = 0.0f;
    // token of accumulator row `sub` (of 16 tokens)
    const int tok = (sub >> 2) * NI + ((sub & 3) < NI ? sub & 3 : 0);
    const int wplace = sub * 4 + (grp ^ (sub >> 2));

    // a step out of its loads, which are replaced by those of step `then`; g0: its first group of
    // the span
    auto use = [&](Step& v, int g0, int then) {
#pragma unroll
        for (int r = 0; r < RT; ++r) stage[wave][r][lane] = v.w[r];
#pragma unroll
        for (int i = 0; i < XI; ++i) stage[wave][RT + i][lane] = order_codes(v.x[i]);
        fetch(then, v);
        __builtin_amdgcn_wave_barrier();
        uint32_t w[RT][4];
        u32x4 x[MT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const u32x4 u = stage[wave][r][wplace];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[r][j] = u[j];
            if constexpr (GROUP != 128) transpose_groups(w[r]);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // product j's channels of this lane: as the words lie, or of the j-th block
                const int c = GROUP == 128 ? 4 * grp + j : 4 * j + grp;
                x[m][j] = stage[wave][RT + 4 * m + tok / 4][(tok & 3) * 16 + (c ^ tok)];
            }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int g = 0; g < GS; ++g) {
            constexpr int PG = 4 / GS;  // products of a group
            f32x4 sx[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                sx[m] = f32x4{};
#pragma unroll
                for (int j = g * PG; j < (g + 1) * PG; ++j) sx[m] = mfma<T>(x[m][j], ones, sx[m]);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float2 f = sz[g0 + g][16 * r + sub];
                u32x4 u[PG];
#pragma unroll
                for (int j = 0; j < PG; ++j) u[j] = codes.unpack(w[r][g * PG + j]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    f32x4 acc;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = i < NI ? f.y * sx[m][i] : 0.0f;
#pragma unroll
                    for (int j = 0; j < PG; ++j) acc = mfma<T>(x[m][g * PG + j], u[j], acc);
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        total[r][m * NI + i] = __builtin_fmaf(f.x, acc[i], total[r][m * NI + i]);
                }
            }
        }
    };
    const int last = steps - 1;
    auto at_most = [&](int s) { return s < last ? s : last; };
    Step v;
    fetch(at_most(wave), v);
    for (int s0 = 0; s0 < steps; s0 += kSpan) {
        if (s0) __syncthreads();
        for (int j = threadIdx.x; j < 16 * RT * SG; j += 64 * NW) {
            const int row = j / SG, g = s0 * GS + j % SG;
            // (a step has places for groups behind the last: zero, or a scale that is not finite
            // would meet their zero sums)
            const bool in = row < krows && g < groups;
            const uint32_t at = in ? row * groups + g : 0;
            const float z = a.zeros ? (float)(zero0[at] & 15) : 8.0f;
            const float scale = (float)scale0[at];
            sz[j % SG][row] = in ? float2{scale, -16.0f - z} : float2{};
        }
        __syncthreads();
        const int end = s0 + kSpan < steps ? s0 + kSpan : steps;
        for (int s = s0 + wave; s < end; s += NW) use(v, (s - s0) * GS, at_most(s + NW));
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < XI; ++i) part(wave, r, i)[lane] = total[r][i];
    __syncthreads();
    const Act act = act_bounds(a.act);
    // lane l of sum i: token 16 * (i / NI) + (l / 16) * NI + i % NI, output channel l % 16
    for (int j = threadIdx.x; j < RT * XI * 64; j += 64 * NW) {
        const int l = j & 63, i = (j >> 6) % XI, r = (j >> 6) / XI;
        const int m = m0 + i / NI * 16 + (l >> 4) * NI + i % NI, k = k0 + 16 * r + (l & 15);
        if (m >= a.M || k >= a.K) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < NW; ++q) v += part(q, r, i)[l];
        if (a.bias) v += a.bias[k];
        ((T*)a.y)[(long long)m * a.ldy + k] = (T)clamp_act(v, act);
    }
}

// Output channels of a workgroup.  More of them share the reading of x but leave fewer workgroups
// and registers.  C = 4096, times in us with RT = 1 / 2 / 4, groups of 128 (one token) and 64:
//   1 token, K = 4096: 5.1 / 6.8 / 10.9, 16384: 11.1 / 9.5 / 14.3, 65536: 37 / 30 / 40;
//   16 tokens, K = 4096: 7.0 / 9.2 / 14, 16384: 16.9 / 14.3 / 15.4, 65536: 66 / 45 / 38;
//   32 tokens (two tiles of 16), K = 4096: 9.4 / 13.9, 16384: 25 / 21, 65536: 96 / 66.
// So two 16-channel tiles from 1024 tiles on, four where x is a whole tile of 16 tokens and there
// are 3072; below, eight waves share the channels' sum.
template <typename T, int GROUP, int NI, int MT, bool WIDE>
int run(const Q4Args& a, hipStream_t s) {
    const int tiles = (a.M + 4 * NI * MT - 1) / (4 * NI * MT);
    auto go = [&](auto rt, auto nw) {
        constexpr int RT = decltype(rt)::value, NW = decltype(nw)::value;
        const dim3 grid((a.K + 16 * RT - 1) / (16 * RT), tiles);
        q4_kernel<T, GROUP, NI, MT, RT, NW, WIDE><<<grid, 64 * NW, 0, s>>>(a);
        return (int)hipGetLastError();
    };
    using std::integral_constant;
    const long long rows = (long long)((a.K + 15) / 16) * tiles;
    if constexpr (NI == 4 && MT == 1 && WIDE)
        if (rows >= 3072) return go(integral_constant<int, 4>(), integral_constant<int, 4>());
    if (rows >= 1024) return go(integral_constant<int, 2>(), integral_constant<int, 4>());
    return go(integral_constant<int, 1>(), integral_constant<int, 8>());
}

template <typename T, int GROUP, bool WIDE>
int pick_tokens(const Q4Args& a, hipStream_t s) {
    if (a.M <= 4) return run<T, GROUP, 1, 1, WIDE>(a, s);
    if (a.M <= 8) return run<T, GROUP, 2, 1, WIDE>(a, s);
    if (a.M <= 16) return run<T, GROUP, 4, 1, WIDE>(a, s);
    return run<T, GROUP, 4, 2, WIDE>(a, s);
}

template <typename T, int GROUP>
int pick_rows(const Q4Args& a, hipStream_t s) {
    const bool wide = a.C % kStep == 0 && ((uintptr_t)a.q & 15) == 0;
    return wide ? pick_tokens<T, GROUP, true>(a, s) : pick_tokens<T, GROUP, false>(a, s);
}

template <typename T>
int pick_group(const Q4Args& a, hipStream_t s) {
    if (a.group == 32) return pick_rows<T, 32>(a, s);
    if (a.group == 64) return pick_rows<T, 64>(a, s);
    return pick_rows<T, 128>(a, s);
}

}  // namespace

int launch_q4(const Q4Args& a, int dtype, void* stream) {
    if (dtype == FCM_F16) return pick_group<_Float16>(a, (hipStream_t)stream);
    return pick_group<__bf16>(a, (hipStream_t)stream);
}

}  // namespace fcm
