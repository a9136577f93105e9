// draft.hip -- verification of drafted tokens against the target's probabilities.
//
// Three launches: the logits' rows are read once for their largest value and the sum of exponentials above it;
// then every workgroup of a request finds from these how many tokens stand, and sums its part of the weights of
// the one row that the next token is drawn from; at last one workgroup a request finds the part, and in it the
// token, at which the running sum passes the given number's share of the total.
//
// Sums and exponentials are 64-bit: whether a token is the one asked for goes by sums over the whole vocabulary, whose
// 32-bit errors of 2^-24 would move the border past one of 65536 tokens once in a few hundred draws.
#include <float.h>
#include <limits.h>

#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

// 16 bytes from any address: one access like an aligned one.
typedef u32x4 __attribute__((aligned(1))) u32x4_any;

constexpr int kLane = 8;
constexpr int kBlock = 64 * kLane;   // tokens a wave looks at at a time
constexpr int kPart = 256 * kLane;   // tokens of a workgroup's part of the weights

struct Split {   // of a row: its largest logit and sum of exponentials above it, or (temperature 0) its token
    double sum;
    float top;
    int32_t token;
};
struct Row {     // of a request, as the second launch leaves it
    double ptop, psum, qtop, qsum;  // the row drawn from and the draft's
    int32_t place, cut;             // its place; the token whose weight is left out, or -1
    int32_t residual;               // the draft's probabilities are taken off
    int32_t pad;
};
struct Sums {
    double weight, p;
};

__host__ __device__ inline int split_blocks(int vocab) { return ((vocab + kBlock - 1) / kBlock + 63) / 64; }
__host__ __device__ inline int row_splits(int vocab) {
    const int per = split_blocks(vocab) * kBlock;
    return (vocab + per - 1) / per;
}
__host__ __device__ inline int row_parts(int vocab) { return (vocab + kPart - 1) / kPart; }

// exp(x) for x <= 0 in 64 bits: Cody and Waite's reduction, x = n log(2) + r with log(2) in two parts, and 2^n times the
// Taylor series of e^r to r^12, |r| <= log(2)/2, whose rest is below 2^-52.  The first part is log(2) cut to 40 bits behind the
// point, so that its product with n, of up to 11 bits, is exact; the second is the rest, rounded.  (At -750 the value is zero,
// as far below.)  The coefficients are in scalar registers: as literals each of them
// would be moved to vector registers for each use, as many instructions again as the series has.
struct Series {
    double c[11], log2e, high, low;
    static __device__ __forceinline__ double held(double v) {
        uint64_t u = __builtin_bit_cast(uint64_t, v);
        asm("" : "+s"(u));
        return __builtin_bit_cast(double, u);
    }
    __device__ __forceinline__ Series() {
        const double f[11] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0,
                              1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5};
#pragma unroll
        for (int i = 0; i < 11; ++i) c[i] = held(f[i]);
        log2e = held(1.4426950408889634);
        high = held(-0x1.62e42fefa2p-1);
        low = held(-0x1.9ef35793c7673p-41);
    }
    __device__ __forceinline__ double exp_neg(double x) const {
        x = __builtin_fmax(x, -750.0);
        const double n = __builtin_rint(x * log2e);
        double r = __builtin_fma(n, high, x);
        r = __builtin_fma(n, low, r);
        double s = __builtin_fma(c[0], r, c[1]);
#pragma unroll
        for (int i = 2; i < 11; ++i) s = __builtin_fma(s, r, c[i]);
        s = __builtin_fma(s, r, 1.0);
        s = __builtin_fma(s, r, 1.0);
        return __builtin_ldexp(s, (int)n);
    }
    // exp((v - top) / temperature) with a finite top: zero for a masked token.
    __device__ __forceinline__ double weight(float v, double top, double inv) const {
        return exp_neg(((double)v - top) * inv);
    }
};

// Logits as they count: NaN as -inf, +inf as the largest float.
__device__ __forceinline__ float counted(float v) {
    return v > -__builtin_inff() ? __builtin_fminf(v, FLT_MAX) : -__builtin_inff();
}
// kLane tokens of the row `l` in this lane, from base + its place: VE at a time, `stride` lanes apart.
template <typename T>
__device__ __forceinline__ int token_at(int base, int lane, int lanes, int e) {
    constexpr int VE = Vec<T>::N;
    return base + ((e / VE) * lanes + lane) * VE + e % VE;
}
template <typename T>
__device__ __forceinline__ void load_tokens(const T* l, int base, int lane, int lanes, int vocab, float* v) {
    constexpr int VE = Vec<T>::N;
#pragma unroll
    for (int j = 0; j < kLane / VE; ++j) {
        const int t = base + (j * lanes + lane) * VE;
        if (t <= vocab - VE) {
            unpack16<T>(*(const u32x4_any*)(l + t), v + j * VE);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) v[j * VE + i] = t < vocab - i ? (float)l[t + i] : -__builtin_inff();
        }
    }
}

// kLane neighbouring tokens from `first` on.
template <typename T>
__device__ __forceinline__ void load_run(const T* l, int first, int vocab, float* v) {
    constexpr int VE = Vec<T>::N;
#pragma unroll
    for (int j = 0; j < kLane; j += VE) {
        if (first + j <= vocab - VE) {
            unpack16<T>(*(const u32x4_any*)(l + first + j), v + j);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) v[j + i] = first + j < vocab - i ? (float)l[first + j + i] : -__builtin_inff();
        }
    }
}

// Over the wave's 64 lanes by shifts within rows of 16 lanes, then from row to row: a step takes a few cycles,
// where one through LDS takes a hundred.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t shifted(uint32_t v, uint32_t old) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double v) {  // zero from outside
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = shifted<CTRL, ROWS>((uint32_t)u, 0u), hi = shifted<CTRL, ROWS>((uint32_t)(u >> 32), 0u);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The sum of this lane's value and those of the lanes before it.
__device__ __forceinline__ double wave_scan(double v) {
    v += shifted<0x111, 0xf>(v);  // by 1, 2, 4, 8 lanes of a row
    v += shifted<0x112, 0xf>(v);
    v += shifted<0x114, 0xf>(v);
    v += shifted<0x118, 0xf>(v);
    v += shifted<0x142, 0xa>(v);  // last lane of a row to the next row
    v += shifted<0x143, 0xc>(v);  // last lane of the lower half to the upper
    return v;
}
__device__ __forceinline__ double wave_sum(double v) { return lane_of(wave_scan(v), 63); }
__device__ __forceinline__ float wave_maxf(float v) {
#define FCM_DPP_MAX(ctrl, rows)                                                                  \
    v = __builtin_fmaxf(v, __builtin_bit_cast(float, shifted<ctrl, rows>(__builtin_bit_cast(uint32_t, v), 0xff800000u)))
    FCM_DPP_MAX(0x111, 0xf);
    FCM_DPP_MAX(0x112, 0xf);
    FCM_DPP_MAX(0x114, 0xf);
    FCM_DPP_MAX(0x118, 0xf);
    FCM_DPP_MAX(0x142, 0xa);
    FCM_DPP_MAX(0x143, 0xc);
#undef FCM_DPP_MAX
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// One wave per (row, split).  Rows: a request's drafts + 1 of the target, then those of the draft.  Its 64-bit
// exponentials bound it: 32 requests of 5 drafts, all in use, over 65537 fp32 logits, 92 MB, in 32 us, 2.9 TB/s, with vector
// instructions in 85% of its CUs' cycles; with temperature 0, which has none, 50 MB in 12 us, 4.1 TB/s.  (With 16 tokens of a lane at a time instead of 8, the whole call took 53 us instead of 48.)
template <typename T>
__global__ __launch_bounds__(256) void draft_rows_kernel(DraftArgs a, int splits, int blocks, int per) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // (there are fewer than 2^26 waves, or the launch would not be)
    const uint32_t id = blockIdx.x * 4 + wave, row = id / (uint32_t)splits;
    const int split = id - row * splits;
    if (row >= (uint32_t)a.requests * (uint32_t)per) return;
    const int r = row / (uint32_t)per, i = row - r * per;
    int count = a.counts ? a.counts[r] : a.drafts;
    count = count < 0 ? 0 : count > a.drafts ? a.drafts : count;
    const bool target = i <= a.drafts;
    if ((target ? i : i - a.drafts) > count) return;  // (not looked at)
    const T* l = target ? (const T*)a.target + ((long long)r * (a.drafts + 1) + i) * a.ldt
                        : (const T*)a.draft + ((long long)r * a.drafts + i - a.drafts - 1) * a.ldd;
    const double inv = 1.0 / (double)a.temperature;
    const bool greedy = a.temperature == 0.0f;
    const Series series;
    // a lane keeps its own tokens' largest logit and sum (or token); the wave's lanes are joined once, at the end
    float top = -__builtin_inff();
    double sum = 0.0;
    int token = INT_MAX;
    const int first = split * blocks * kBlock;
    float v[kLane], ahead[kLane];
    load_tokens<T>(l, first, lane, 64, a.vocab, ahead);
    for (int b = 0; b < blocks; ++b) {
        const int base = first + b * kBlock;
        if (base >= a.vocab) break;
        float m = -__builtin_inff();
#pragma unroll
        for (int e = 0; e < kLane; ++e) v[e] = ahead[e];
        if (b + 1 < blocks && base + kBlock < a.vocab) load_tokens<T>(l, base + kBlock, lane, 64, a.vocab, ahead);
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            v[e] = counted(v[e]);
            m = __builtin_fmaxf(m, v[e]);
        }
        if (greedy) {
            if (m > top) {  // (later blocks have higher tokens)
                int t = INT_MAX;
#pragma unroll
                for (int e = 0; e < kLane; ++e) {
                    const int at = token_at<T>(base, lane, 64, e);
                    if (v[e] == m && at < t) t = at;
                }
                token = t;
                top = m;
            }
            continue;
        }
        const float now = __builtin_fmaxf(top, m);
        if (!(now > -__builtin_inff())) continue;
        double s = sum * series.weight(top, now, inv);
#pragma unroll
        for (int e = 0; e < kLane; ++e) s += series.weight(v[e], now, inv);
        sum = s;
        top = now;
    }
    const float all = wave_maxf(top);
    if (greedy) {
        if (top != all) token = INT_MAX;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const int other = __shfl_xor(token, o);
            token = other < token ? other : token;
        }
    } else {
        sum = wave_sum(all > -__builtin_inff() ? sum * series.weight(top, all, inv) : 0.0);
    }
    top = all;
    if (lane == 0) ((Split*)a.ws)[id] = Split{sum, top, token};
}

__device__ __forceinline__ Row* request_rows(const DraftArgs& a, int per, int splits) {
    return (Row*)((Split*)a.ws + (long long)a.requests * per * splits);
}

// Temperature 0: one wave a request.
__global__ __launch_bounds__(64) void draft_best_kernel(DraftArgs a, int splits, int per) {
    const int r = blockIdx.x, lane = threadIdx.x;
    int count = a.counts ? a.counts[r] : a.drafts;
    count = count < 0 ? 0 : count > a.drafts ? a.drafts : count;
    int i = 0, best = -1;
    for (;; ++i) {
        Split s{0.0, -__builtin_inff(), INT_MAX};
        if (lane < splits) s = ((const Split*)a.ws)[((long long)r * per + i) * splits + lane];
        const float top = wave_maxf(s.top);
        const uint64_t who = __ballot(s.top == top);  // splits are in the tokens' order
        best = __shfl(s.token, __ffsll((unsigned long long)who) - 1);
        if (!(top > -__builtin_inff())) best = -1;
        if (i == count || best < 0 || a.tokens[(long long)r * a.drafts + i] != best) break;
    }
    if (lane == 0) {
        a.accepted[r] = i;
        a.next[r] = best;
    }
}

// Largest logit and sum of a row from its splits.
__device__ __forceinline__ void join_splits(const Series& series, const Split* in, int splits, double inv, int lane,
                                            double* top, double* sum) {
    Split s{0.0, -__builtin_inff(), 0};
    if (lane < splits) s = in[lane];
    const float m = wave_maxf(s.top);
    *sum = wave_sum(m > -__builtin_inff() ? s.sum * series.weight(s.top, m, inv) : 0.0);
    *top = m;
}

// What a token counts for in the row that is drawn from, and its probability there.  Where the draft's row is the
// target's the difference has to be zero, or the token would be drawn from what roundings leave: the product is
// rounded before it is taken off, not fused with the subtraction.
__device__ __forceinline__ Sums draw_weight(const Series& series, const Row& row, float l, float d, int token, double inv, double ip, double iq) {
#pragma clang fp contract(off)
    const double p = row.psum > 0.0 ? series.weight(l, row.ptop, inv) * ip : 0.0;
    double w = p;
    if (row.residual) {
        w -= row.qsum > 0.0 ? series.weight(d, row.qtop, inv) * iq : 0.0;
        w = w > 0.0 ? w : 0.0;
    }
    if (token == row.cut) w = 0.0;
    return Sums{w, p};
}

// This lane's kLane tokens of a part, from `first` on: their weights.
template <typename T>
__device__ __forceinline__ void part_weights(const Series& series, const DraftArgs& a, const Row& row, int r, int first, Sums* w) {
    const double inv = 1.0 / (double)a.temperature;
    float l[kLane], d[kLane];
    load_run<T>((const T*)a.target + ((long long)r * (a.drafts + 1) + row.place) * a.ldt, first, a.vocab, l);
    if (row.residual) load_run<T>((const T*)a.draft + ((long long)r * a.drafts + row.place) * a.ldd, first, a.vocab, d);
    const double ip = 1.0 / row.psum, iq = 1.0 / row.qsum;
#pragma unroll
    for (int e = 0; e < kLane; ++e)
        w[e] = draw_weight(series, row, counted(l[e]), row.residual ? counted(d[e]) : 0.0f, first + e, inv, ip, iq);
}

// Workgroups (request, part).  Two rows of every request are read again and weighed: 12 us of the same call.
template <typename T>
__global__ __launch_bounds__(256) void draft_weights_kernel(DraftArgs a, int splits, int per, int parts) {
    __shared__ double tops[129], sums[129];
    __shared__ Row row;
    __shared__ Sums halves[4];
    const int r = blockIdx.x / parts, part = blockIdx.x % parts;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int count = a.counts ? a.counts[r] : a.drafts;
    count = count < 0 ? 0 : count > a.drafts ? a.drafts : count;
    const double inv = 1.0 / (double)a.temperature;
    const Series series;
    for (int i = wave; i < per; i += 4) {
        if ((i <= a.drafts ? i : i - a.drafts) > count) continue;
        double top, sum;
        join_splits(series, (const Split*)a.ws + ((long long)r * per + i) * splits, splits, inv, lane, &top, &sum);
        if (lane == 0) tops[i] = top, sums[i] = sum;
    }
    __syncthreads();
    if (wave == 0) {
        // a lane for each drafted token
        bool fails = false;
        if (lane < count) {
            const int x = a.tokens[(long long)r * a.drafts + lane];
            fails = true;
            if (x >= 0 && x < a.vocab && sums[lane] > 0.0) {
                const float l = counted((float)((const T*)a.target)[((long long)r * (a.drafts + 1) + lane) * a.ldt + x]);
                const double p = series.weight(l, tops[lane], inv) / sums[lane];
                double q = 1.0;
                if (a.draft) {
                    const int j = a.drafts + 1 + lane;
                    const float d = counted((float)((const T*)a.draft)[((long long)r * a.drafts + lane) * a.ldd + x]);
                    q = sums[j] > 0.0 ? series.weight(d, tops[j], inv) / sums[j] : 0.0;
                }
                fails = !((double)a.uniform[(long long)r * (a.drafts + 1) + lane] * q < p);
            }
        }
        const uint64_t who = __ballot(fails);
        const int place = who ? __ffsll((unsigned long long)who) - 1 : count;
        if (lane == 0) {
            Row o;
            o.place = place;
            o.residual = place < count && a.draft;
            o.cut = place < count && !a.draft ? a.tokens[(long long)r * a.drafts + place] : -1;
            o.ptop = tops[place];
            o.psum = sums[place];
            o.qtop = o.residual ? tops[a.drafts + 1 + place] : 0.0;
            o.qsum = o.residual ? sums[a.drafts + 1 + place] : 0.0;
            o.pad = 0;
            row = o;
            if (part == 0) request_rows(a, per, splits)[r] = o;
        }
    }
    __syncthreads();
    Sums w[kLane], s{0.0, 0.0};
    part_weights<T>(series, a, row, r, part * kPart + (int)threadIdx.x * kLane, w);
#pragma unroll
    for (int e = 0; e < kLane; ++e) s.weight += w[e].weight, s.p += w[e].p;
    s.weight = wave_sum(s.weight);
    s.p = wave_sum(s.p);
    if (lane == 0) halves[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 4; ++i) s.weight += halves[i].weight, s.p += halves[i].p;
        ((Sums*)(request_rows(a, per, splits) + a.requests))[(long long)r * parts + part] = s;
    }
}

// One workgroup a request: a chain of latencies, 5 us.
template <typename T>
__global__ __launch_bounds__(256) void draft_pick_kernel(DraftArgs a, int splits, int per, int parts) {
    __shared__ double ends[4];
    __shared__ int found[4], last[4];
    const int r = blockIdx.x, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Series series;
    const Row row = request_rows(a, per, splits)[r];
    const Sums* in = (const Sums*)(request_rows(a, per, splits) + a.requests) + (long long)r * parts;
    if (threadIdx.x == 0) a.accepted[r] = row.place;
    // every wave goes over the parts: all of them, then up to the one where the sum passes its share
    Sums total{0.0, 0.0};
    for (int i = lane; i < parts; i += 64) total.weight += in[i].weight, total.p += in[i].p;
    total.weight = wave_sum(total.weight);
    total.p = wave_sum(total.p);
    const bool plain = !(total.weight > 0.0);  // the draft never differs
    const double all = plain ? total.p : total.weight;
    if (!(all > 0.0)) {  // no token at all
        if (threadIdx.x == 0) a.next[r] = -1;
        return;
    }
    const double share = (double)a.uniform[(long long)r * (a.drafts + 1) + a.drafts] * all;
    double before = 0.0;  // the sum of what is before `at`
    int part = -1, some = -1;
    double some_before = 0.0;  // the last part with any weight
    for (int i = 0; i < parts && part < 0; i += 64) {
        double v = 0.0;
        if (i + lane < parts) v = plain ? in[i + lane].p : in[i + lane].weight;
        const double s = wave_scan(v);
        const uint64_t passed = __ballot(v > 0.0 && before + s > share), any = __ballot(v > 0.0);
        if (any) {
            const int j = 63 - __clzll((long long)any);
            some = i + j;
            some_before = before + (lane_of(s, j) - lane_of(v, j));
        }
        if (passed) {
            const int j = __ffsll((unsigned long long)passed) - 1;
            part = i + j;
            before += lane_of(s, j) - lane_of(v, j);
        } else {
            before += lane_of(s, 63);
        }
    }
    if (part < 0) {  // (rounding, or a number of 1 and above)
        part = some;
        before = some_before;
    }
    // Within the part a lane has kLane neighbouring tokens: the one at which the sum passes is found by the lane that
    // holds it, and where none does (rounding again) it is the last with any weight.
    Sums w[kLane];
    const int first = part * kPart + (int)threadIdx.x * kLane;
    part_weights<T>(series, a, row, r, first, w);
    double sum = 0.0;
    int high = -1;
#pragma unroll
    for (int e = 0; e < kLane; ++e) {
        const double v = plain ? w[e].p : w[e].weight;
        sum += v;
        if (v > 0.0) high = first + e;
    }
    const double upto = wave_scan(sum);
    const uint64_t any = __ballot(high >= 0);
    const int top = any ? __builtin_amdgcn_readlane(high, 63 - __clzll((long long)any)) : -1;
    if (lane == 63) ends[wave] = upto, last[wave] = top;
    __syncthreads();
    double at = before + (upto - sum);
    for (int q = 0; q < wave; ++q) at += ends[q];
    int mine = INT_MAX;
#pragma unroll
    for (int e = 0; e < kLane; ++e) {
        const double v = plain ? w[e].p : w[e].weight;
        at += v;
        if (v > 0.0 && at > share && mine == INT_MAX) mine = first + e;
    }
    const uint64_t hit = __ballot(mine != INT_MAX);
    if (lane == 0) found[wave] = hit ? __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)hit) - 1) : INT_MAX;
    __syncthreads();
    if (threadIdx.x != 0) return;
    int best = INT_MAX, tail = -1;
    for (int q = 0; q < 4; ++q) {
        best = found[q] < best ? found[q] : best;
        tail = last[q] > tail ? last[q] : tail;
    }
    a.next[r] = best != INT_MAX ? best : tail;
}

template <typename T>
int run(const DraftArgs& a, hipStream_t s) {
    const bool greedy = a.temperature == 0.0f;
    const int splits = row_splits(a.vocab), blocks = split_blocks(a.vocab), parts = row_parts(a.vocab);
    const int per = a.drafts + 1 + (a.draft && !greedy ? a.drafts : 0);
    const long long waves = (long long)a.requests * per * splits;
    draft_rows_kernel<T><<<(int)((waves + 3) / 4), 256, 0, s>>>(a, splits, blocks, per);
    int rc = (int)hipGetLastError();
    if (rc != 0) return rc;
    if (greedy) {
        draft_best_kernel<<<a.requests, 64, 0, s>>>(a, splits, per);
        return (int)hipGetLastError();
    }
    draft_weights_kernel<T><<<a.requests * parts, 256, 0, s>>>(a, splits, per, parts);
    rc = (int)hipGetLastError();
    if (rc != 0) return rc;
    draft_pick_kernel<T><<<a.requests, 256, 0, s>>>(a, splits, per, parts);
    return (int)hipGetLastError();
}

}  // namespace

long long draft_workspace_bytes(const fcm_draft_problem& p) {
    const long long rows = (long long)p.requests * (2 * p.drafts + 1);
    return rows * row_splits(p.vocab) * (long long)sizeof(Split) + p.requests * (long long)sizeof(Row) +
           p.requests * (long long)row_parts(p.vocab) * (long long)sizeof(Sums);
}

long long draft_threads(const fcm_draft_problem& p) {
    const long long rows = ((long long)p.requests * (2 * p.drafts + 1) * row_splits(p.vocab) + 3) / 4 * 256;
    const long long weights = (long long)p.requests * row_parts(p.vocab) * 256;
    return rows > weights ? rows : weights;
}

int launch_draft_verify(const DraftArgs& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return run<float>(a, s);
    if (dtype == FCM_F16) return run<_Float16>(a, s);
    return run<__bf16>(a, s);
}

}  // namespace fcm
