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

constexpr int kLane = 16;
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

// exp(x) for x <= 0 in 64 bits: 2^n times the Taylor series of e^r to r^12, |r| <= log(2)/2, whose rest is below
// 2^-52.  (At -750 it is zero, as far below.)
__device__ __forceinline__ double exp_neg(double x) {
    x = x < -750.0 ? -750.0 : x;
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(n, -0.693147180369123816490, x);
    r = __builtin_fma(n, -1.90821492927058770002e-10, r);
    double s = 1.0 / 479001600.0;
    s = __builtin_fma(s, r, 1.0 / 39916800.0);
    s = __builtin_fma(s, r, 1.0 / 3628800.0);
    s = __builtin_fma(s, r, 1.0 / 362880.0);
    s = __builtin_fma(s, r, 1.0 / 40320.0);
    s = __builtin_fma(s, r, 1.0 / 5040.0);
    s = __builtin_fma(s, r, 1.0 / 720.0);
    s = __builtin_fma(s, r, 1.0 / 120.0);
    s = __builtin_fma(s, r, 1.0 / 24.0);
    s = __builtin_fma(s, r, 1.0 / 6.0);
    s = __builtin_fma(s, r, 0.5);
    s = __builtin_fma(s, r, 1.0);
    s = __builtin_fma(s, r, 1.0);
    return __builtin_ldexp(s, (int)n);
}

// Logits as they count: NaN as -inf, +inf as the largest float.
__device__ __forceinline__ float counted(float v) {
    return v > -__builtin_inff() ? __builtin_fminf(v, FLT_MAX) : -__builtin_inff();
}
// exp((v - top) / temperature), zero for a masked token or a row without any.
__device__ __forceinline__ double weight(float v, double top, double inv) {
    return v > -__builtin_inff() ? exp_neg(((double)v - top) * inv) : 0.0;
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
#pragma unroll
    for (int e = 0; e < kLane; ++e) v[e] = counted(v[e]);
}

__device__ __forceinline__ float wave_maxf(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// One wave per (row, split).  Rows: a request's drafts + 1 of the target, then those of the draft.
template <typename T>
__global__ __launch_bounds__(256) void draft_rows_kernel(DraftArgs a, int splits, int blocks, int per) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long id = (long long)blockIdx.x * 4 + wave;
    const long long row = id / splits;
    const int split = id % splits;
    if (row >= (long long)a.requests * per) return;
    const int r = row / per, i = row % per;
    int count = a.counts ? a.counts[r] : a.drafts;
    count = count < 0 ? 0 : count > a.drafts ? a.drafts : count;
    const bool target = i <= a.drafts;
    if ((target ? i : i - a.drafts) > count) return;  // (not looked at)
    const T* l = target ? (const T*)a.target + ((long long)r * (a.drafts + 1) + i) * a.ldt
                        : (const T*)a.draft + ((long long)r * a.drafts + i - a.drafts - 1) * a.ldd;
    const double inv = 1.0 / (double)a.temperature;
    const bool greedy = a.temperature == 0.0f;
    float top = -__builtin_inff();
    double sum = 0.0;
    int token = INT_MAX;
    for (int b = 0; b < blocks; ++b) {
        const int base = (split * blocks + b) * kBlock;
        if (base >= a.vocab) break;
        float v[kLane], m = -__builtin_inff();
        load_tokens<T>(l, base, lane, 64, a.vocab, v);
#pragma unroll
        for (int e = 0; e < kLane; ++e) m = __builtin_fmaxf(m, v[e]);
        m = wave_maxf(m);
        if (!(m > -__builtin_inff())) continue;
        if (greedy) {
            if (m > top) {  // (later blocks have higher tokens)
                int t = INT_MAX;
#pragma unroll
                for (int e = kLane - 1; e >= 0; --e)
                    if (v[e] == m) {
                        const int at = token_at<T>(base, lane, 64, e);
                        t = at < t ? at : t;
                    }
#pragma unroll
                for (int o = 32; o > 0; o >>= 1) {
                    const int other = __shfl_xor(t, o);
                    t = other < t ? other : t;
                }
                token = t;
                top = m;
            }
            continue;
        }
        double s = 0.0;
#pragma unroll
        for (int e = 0; e < kLane; ++e) s += weight(v[e], m, inv);
        s = wave_sum(s);
        const float now = __builtin_fmaxf(top, m);
        sum = sum * weight(top, now, inv) + s * weight(m, now, inv);
        top = now;
    }
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
__device__ __forceinline__ void join_splits(const Split* in, int splits, double inv, int lane, double* top,
                                            double* sum) {
    Split s{0.0, -__builtin_inff(), 0};
    if (lane < splits) s = in[lane];
    const float m = wave_maxf(s.top);
    *sum = wave_sum(m > -__builtin_inff() ? s.sum * weight(s.top, m, inv) : 0.0);
    *top = m;
}

// What a token counts for in the row that is drawn from, and its probability there.
__device__ __forceinline__ Sums draw_weight(const Row& row, float l, float d, int token, double inv, double ip, double iq) {
    const double p = row.psum > 0.0 ? weight(l, row.ptop, inv) * ip : 0.0;
    double w = p;
    if (row.residual) {
        w -= row.qsum > 0.0 ? weight(d, row.qtop, inv) * iq : 0.0;
        w = w > 0.0 ? w : 0.0;
    }
    if (token == row.cut) w = 0.0;
    return Sums{w, p};
}

// This lane's kLane tokens of a part: their weights.
template <typename T>
__device__ __forceinline__ void part_weights(const DraftArgs& a, const Row& row, int r, int part, Sums* w) {
    const double inv = 1.0 / (double)a.temperature;
    float l[kLane], d[kLane];
    load_tokens<T>((const T*)a.target + ((long long)r * (a.drafts + 1) + row.place) * a.ldt, part * kPart,
                   threadIdx.x, 256, a.vocab, l);
    if (row.residual)
        load_tokens<T>((const T*)a.draft + ((long long)r * a.drafts + row.place) * a.ldd, part * kPart,
                       threadIdx.x, 256, a.vocab, d);
    const double ip = 1.0 / row.psum, iq = 1.0 / row.qsum;
#pragma unroll
    for (int e = 0; e < kLane; ++e)
        w[e] = draw_weight(row, l[e], row.residual ? d[e] : 0.0f,
                           token_at<T>(part * kPart, threadIdx.x, 256, e), inv, ip, iq);
}

// Workgroups (request, part).
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
    for (int i = wave; i < per; i += 4) {
        if ((i <= a.drafts ? i : i - a.drafts) > count) continue;
        double top, sum;
        join_splits((const Split*)a.ws + ((long long)r * per + i) * splits, splits, inv, lane, &top, &sum);
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
                const double p = weight(l, tops[lane], inv) / sums[lane];
                double q = 1.0;
                if (a.draft) {
                    const int j = a.drafts + 1 + lane;
                    const float d = counted((float)((const T*)a.draft)[((long long)r * a.drafts + lane) * a.ldd + x]);
                    q = sums[j] > 0.0 ? weight(d, tops[j], inv) / sums[j] : 0.0;
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
    part_weights<T>(a, row, r, part, w);
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

// One workgroup a request.
template <typename T>
__global__ __launch_bounds__(256) void draft_pick_kernel(DraftArgs a, int splits, int per, int parts) {
    __shared__ double ends[4];
    __shared__ int found[4], last[4];
    const int r = blockIdx.x, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Row row = request_rows(a, per, splits)[r];
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
        double s = v;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double x = __shfl_up(s, o);
            if (lane >= o) s += x;
        }
        const uint64_t passed = __ballot(v > 0.0 && before + s > share), any = __ballot(v > 0.0);
        if (any) {
            const int j = 63 - __clzll((long long)any);
            some = i + j;
            some_before = before + (__shfl(s, j) - __shfl(v, j));
        }
        if (passed) {
            const int j = __ffsll((unsigned long long)passed) - 1;
            part = i + j;
            before += __shfl(s, j) - __shfl(v, j);
        } else {
            before += __shfl(s, 63);
        }
    }
    if (part < 0) {  // (rounding, or a number of 1 and above)
        part = some;
        before = some_before;
    }
    // Within the part, tokens in order: pieces of VE tokens, 256 lanes after one another, kLane / VE times.
    constexpr int VE = Vec<T>::N;
    Sums w[kLane];
    part_weights<T>(a, row, r, part, w);
    int tail = -1;
    for (int j = 0; j < kLane / VE; ++j) {
        double v[VE], s = 0.0;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            v[i] = 0.0;
#pragma unroll
            for (int e = 0; e < kLane; ++e)
                if (e == j * VE + i) v[i] = plain ? w[e].p : w[e].weight;
            s += v[i];
        }
        double upto = s;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double x = __shfl_up(upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 63) ends[wave] = upto;
        __syncthreads();
        double at = before + (upto - s);
        for (int q = 0; q < wave; ++q) at += ends[q];
        int mine = INT_MAX, high = -1;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            at += v[i];
            const int t = part * kPart + (j * 256 + (int)threadIdx.x) * VE + i;
            if (v[i] > 0.0) {
                high = t;
                if (at > share && mine == INT_MAX) mine = t;
            }
        }
        const uint64_t hit = __ballot(mine != INT_MAX), some_here = __ballot(high >= 0);
        const int first = hit ? __shfl(mine, __ffsll((unsigned long long)hit) - 1) : INT_MAX;
        const int top = some_here ? __shfl(high, 63 - __clzll((long long)some_here)) : -1;
        if (lane == 0) found[wave] = first, last[wave] = top;
        __syncthreads();
        int best = INT_MAX;
        for (int q = 0; q < 4; ++q) {
            best = found[q] < best ? found[q] : best;
            tail = last[q] > tail ? last[q] : tail;
            before += ends[q];
        }
        if (best != INT_MAX) {
            if (threadIdx.x == 0) a.next[r] = best;
            return;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) a.next[r] = tail;
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
