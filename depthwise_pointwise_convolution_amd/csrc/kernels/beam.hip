// beam.hip -- beam search: the best continuations of each request over beams and vocabulary,
// and the reordering of the beams' states.
//
// Both are readings of memory.  On MI355X, 32 requests of 8 beams over 65537 fp32 logits: the rows
// 25 us (67 MB, 2.7 TB/s.  Neither the bytes nor issue bounds them, the vector units are busy 45% of the
// time: a wave loads a block, takes W maxima one after the other, and only then loads the next; half of
// its life it waits for such results, a third for its turn to issue.  16 or 32 tokens a lane, one block
// or several a wave take 25 to 29 us),
// the merge 8.5 us (a chain of latencies), the copies of 158 states of 1.1 MB 52 us (7 TB/s, part of
// it from the Infinity Cache).  One request of 4 beams over 32000 fp16 logits: 4.6, 5 and 4 us.
#include <float.h>
#include <limits.h>

#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

// 16 bytes from any address: one access like an aligned one.
typedef u32x4 __attribute__((aligned(1))) u32x4_any;

// Selection works on keys that order as integers: a float's bits turned so that they ascend, and
// below them the complement of the token, so that among equal logits the lowest token is largest.
// 0 is below every key.
typedef uint64_t Key;
__device__ __forceinline__ uint32_t ascending(float f) {
    const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);  // (-0 is 0)
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ascending(uint32_t u) {
    return __builtin_bit_cast(float, u ^ (u >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ Key make_key(float f, int token) {
    return (Key)ascending(f) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ int key_token(Key k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_logit(Key k) { return from_ascending((uint32_t)(k >> 32)); }

// Largest of the wave's 64 values: shifts within rows of 16 lanes, then from row to row.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define FCM_DPP_MAX(ctrl, rows)                                                            \
    {                                                                                      \
        const uint32_t o = __builtin_amdgcn_update_dpp(0u, v, ctrl, rows, 0xf, false);     \
        v = v > o ? v : o;                                                                 \
    }
    FCM_DPP_MAX(0x111, 0xf)  // row_shr 1, 2, 4, 8
    FCM_DPP_MAX(0x112, 0xf)
    FCM_DPP_MAX(0x114, 0xf)
    FCM_DPP_MAX(0x118, 0xf)
    FCM_DPP_MAX(0x142, 0xa)  // last lane of a row to the next row
    FCM_DPP_MAX(0x143, 0xc)  // last lane of the lower half to the upper
#undef FCM_DPP_MAX
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ Key wave_max(Key k) {
    const uint32_t hi = wave_max((uint32_t)(k >> 32));
    const uint32_t lo = wave_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (Key)hi << 32 | lo;
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// A wave looks at kBlock tokens of a row at a time, kLane of them in a lane's registers; one
// wave's tokens are a split, of which a row has at most 64.
constexpr int kLane = 16;
constexpr int kBlock = 64 * kLane;
// What selection keeps of a split: its largest logit, the sum of exp(logit - largest), and its
// best tokens as keys, best first.
struct SplitHead {
    float top, sum;
};
__host__ __device__ inline long long split_bytes(int beams) {
    return (long long)sizeof(SplitHead) + (long long)beams * sizeof(Key);
}
__host__ __device__ inline int split_blocks(int vocab) {
    const int blocks = (vocab + kBlock - 1) / kBlock;
    return (blocks + 63) / 64;
}
__host__ __device__ inline int row_splits(int vocab) {
    const int per = split_blocks(vocab) * kBlock;
    return (vocab + per - 1) / per;
}

// One wave per (row, split): one reading of the logits.  The W-th largest of the 64 lanes' own
// maxima is a bound that W tokens reach, so only tokens that reach it can be among the best W: a
// dozen or so, gathered through LDS and ranked against each other.  Where many tokens are equal
// (a masked row, coarse logits) more than 64 may reach it; then the best are taken one by one.
template <typename T>
__global__ __launch_bounds__(256, 8) void beam_rows_kernel(BeamArgs a, int splits, int blocks) {
    __shared__ Key pool[4][64], best[4][32];
    constexpr int VE = Vec<T>::N;
    const float inf = __builtin_inff();
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int id = blockIdx.x * 4 + wave;
    const int row = id / splits, split = id % splits, W = a.beams;
    if (row >= a.requests * W) return;
    const T* l = (const T*)a.logits + row * a.ldl;
    Key mine = 0;  // lane r: the r-th best so far
    int have = 0;
    float top = -inf, sum = 0.0f;
    for (int b = 0; b < blocks; ++b) {
        const int base = (split * blocks + b) * kBlock;
        if (base >= a.vocab) break;
        float v[kLane];
#pragma unroll
        for (int j = 0; j < kLane / VE; ++j) {
            const int t = base + (j * 64 + lane) * VE;
            if (t + VE <= a.vocab) {
                // (rows may start at any element)
                unpack16<T>(*(const u32x4_any*)(l + t), v + j * VE);
            } else {
#pragma unroll
                for (int i = 0; i < VE; ++i) v[j * VE + i] = t + i < a.vocab ? (float)l[t + i] : -inf;
            }
        }
        float m = -inf;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            v[e] = v[e] > -inf ? __builtin_fminf(v[e], FLT_MAX) : -inf;  // (NaN becomes -inf)
            m = __builtin_fmaxf(m, v[e]);
        }
        // the bound: the have-th best so far where there are W, and the W-th largest lane maximum
        uint32_t bound = 0;
        float block_top = -inf;
        {
            uint32_t rest = ascending(m);
            for (int i = 0; i < W; ++i) {
                bound = wave_max(rest);
                if (i == 0) block_top = from_ascending(bound);
                const uint64_t at = __ballot(rest == bound);
                if (lane == __ffsll((unsigned long long)at) - 1) rest = 0;
            }
            if (have == W) {
                const uint32_t old = __builtin_amdgcn_readlane((int)(mine >> 32), W - 1);
                bound = old > bound ? old : bound;
            }
        }
        if (block_top > -inf) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < kLane; ++e)
                s += __builtin_amdgcn_exp2f((v[e] - block_top) * 1.44269504f);
            s = wave_sum(s);
            const float now = __builtin_fmaxf(top, block_top);
            sum = sum * __builtin_amdgcn_exp2f((top - now) * 1.44269504f) +
                  s * __builtin_amdgcn_exp2f((block_top - now) * 1.44269504f);
            top = now;
        }
        const float reach = from_ascending(bound);
        auto token = [&](int e) { return base + ((e / VE) * 64 + lane) * VE + e % VE; };
        if (lane < have) pool[wave][lane] = mine;
        int n = have;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            const bool in = v[e] >= reach;
            const uint64_t who = __ballot(in);
            if (who) {
                const int at = n + __builtin_amdgcn_mbcnt_hi(
                                       (uint32_t)(who >> 32),
                                       __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
                if (in && at < 64) pool[wave][at] = make_key(v[e], token(e));
                n += __popcll(who);
            }
        }
        __builtin_amdgcn_wave_barrier();
        if (n <= 64) {
            const Key k = lane < n ? pool[wave][lane] : 0;
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += pool[wave][j] > k;
            have = n < W ? n : W;
            if (lane < n && rank < W) best[wave][rank] = k;
            __builtin_amdgcn_wave_barrier();
            mine = lane < have ? best[wave][lane] : 0;
        } else {
            Key last = ~(Key)0, next = 0;
            for (int r = 0; r < W; ++r) {
                Key k = mine < last ? mine : 0;
#pragma unroll
                for (int e = 0; e < kLane; ++e) {
                    const Key c = make_key(v[e], token(e));
                    if (c < last && c > k) k = c;
                }
                last = wave_max(k);
                if (lane == r) next = last;
            }
            mine = next;
            have = W;
        }
        __builtin_amdgcn_wave_barrier();
    }
    char* out = (char*)a.ws + id * split_bytes(W);
    if (lane == 0) *(SplitHead*)out = SplitHead{top, sum};
    // (tokens behind the vocabulary are no tokens)
    if (lane < W) ((Key*)(out + sizeof(SplitHead)))[lane] =
        lane < have && key_token(mine) < a.vocab ? mine : 0;
}

// (Rows and merge in one launch, sixteen waves a request, saves a launch but reads a row's blocks
// one after the other, 3 us each: 31 against 9.7 us for 4 rows of 32000.)
//
// One workgroup per request.  A wave per beam (in turn): the splits' sums give the row's
// log-sum-exp, kept as its largest logit and the log of the sum above that (beside 3e38, a mask of the
// type's lowest value or an infinite logit, the log would be lost also in 64 bits), and lane s walks split s's best tokens while the best head of all lanes is taken
// W times.  Then the first wave does the same over the beams, on scores in 64 bits.
__global__ __launch_bounds__(512) void beam_merge_kernel(BeamArgs a, int splits) {
    __shared__ Key rowbest[32][32];
    __shared__ double rowtop[32], rowlog[32];
    constexpr int AHEAD = 4;  // of a split's tokens, loaded at once
    const int r = blockIdx.x, lane = threadIdx.x & 63, W = a.beams;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float inf = __builtin_inff();
    const long long size = split_bytes(W);
    const int row = r * W + (lane < W ? lane : 0);  // of the first wave, at the end
    const float score = a.scores[row];
    const int ended = a.done ? a.done[row] : 0;
    for (int w = wave; w < W; w += blockDim.x / 64) {
        const char* in = (const char*)a.ws + ((long long)(r * W + w) * splits + lane) * size;
        const Key* keys = (const Key*)(in + sizeof(SplitHead));
        const bool live = lane < splits;
        SplitHead head = {-inf, 0.0f};
        Key ahead[AHEAD];
        if (live) head = *(const SplitHead*)in;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) ahead[i] = live && i < W ? keys[i] : 0;
        const float top = from_ascending(wave_max(ascending(head.top)));
        double part = 0.0;
        if (head.top > -inf) part = (double)head.sum * exp((double)head.top - (double)top);
        part = wave_sum(part);
        if (lane == 0) {
            rowtop[w] = top;
            rowlog[w] = top > -inf ? log(part) : 0.0;
        }
        int at = 0;
        Key cur = ahead[0];
        for (int i = 0; i < W; ++i) {
            const Key k = wave_max(cur);
            if (lane == 0) rowbest[w][i] = k;
            if (cur == k && k != 0) {
                ++at;
                Key next = 0;
                if (at < W) {
                    next = at >= AHEAD ? keys[at] : ahead[AHEAD - 1];
#pragma unroll
                    for (int q = 1; q < AHEAD - 1; ++q)
                        if (at == q) next = ahead[q];
                }
                cur = next;
            }
        }
    }
    __syncthreads();
    if (wave != 0) return;
    const bool live = lane < W;
    const double rtop = rowtop[live ? lane : 0], rlog = rowlog[live ? lane : 0];
    const bool dead = !(score > -inf) || !(rtop > -(double)inf);
    int at = 0;  // tokens of this beam taken so far
    for (int k = 0; k < W; ++k) {
        double total = -(double)inf;
        int tok = -1;
        if (live && at < W) {
            if (ended != 0 && score > -inf) {
                // eos, then the other tokens in order
                if (at == 0) {
                    tok = a.eos;
                    total = score;
                } else {
                    tok = at - 1 < a.eos ? at - 1 : at;
                    if (tok >= a.vocab) tok = -1;
                }
            } else if (dead) {
                tok = at < a.vocab ? at : -1;
            } else {
                const Key c = rowbest[lane][at];
                tok = c != 0 ? key_token(c) : -1;
                const float l = key_logit(c);
                if (tok >= 0 && l > -inf) total = (double)score + (((double)l - rtop) - rlog);
            }
        }
        // the largest total, then the lowest place in beams x vocabulary
        const uint32_t low = ~(uint32_t)(lane * a.vocab + tok);
        uint64_t u = __builtin_bit_cast(uint64_t, total + 0.0);
        u ^= u >> 63 ? ~(uint64_t)0 : (uint64_t)1 << 63;
        if (tok < 0) u = 0;
        const Key first = wave_max((Key)u);
        const uint32_t place = wave_max(u == first && tok >= 0 ? low : 0u);
        if (tok >= 0 && u == first && low == place) {
            const int i = r * W + k;
            a.next_scores[i] = (float)total;
            a.parent[i] = lane;
            a.token[i] = tok;
            if (a.next_done) a.next_done[i] = ended != 0 || tok == a.eos;
            ++at;
        }
    }
}

// (8 / 16 / 32 / 64 KB: 65 / 52 / 56 / 56 us for 158 states of 1.1 MB)
constexpr long long kChunk = 16384;  // bytes of a pool one workgroup copies

// Workgroups (beam, chunk): the beam's place among its parent's children says whether it keeps
// the parent's slot (nothing to copy) or takes a freed one.  Slots that are read from belong to
// beams with children and slots that are written to belong to beams without, so the copies of a
// request can run in any order.
__global__ __launch_bounds__(256) void beam_reorder_kernel(ReorderArgs a, int chunks) {
    const int lane = threadIdx.x & 63;
    const int beam = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int r = beam / a.beams, w = beam % a.beams;
    const int base = r * a.beams;
    int p = lane < a.beams ? a.parent[base + lane] : -1;
    if (lane < a.beams && (unsigned)p >= (unsigned)a.beams) p = 0;
    uint64_t firsts = 0;  // children that keep their parent's slot
    uint64_t freed = 0;   // beams without a child
    for (int b = 0; b < a.beams; ++b) {
        const uint64_t kids = __ballot(p == b);
        if (kids)
            firsts |= kids & (0 - kids);
        else
            freed |= 1ull << b;
    }
    const int mine = __shfl(p, w);
    const int src = a.slots[base + mine];
    if (firsts >> w & 1) {
        if (chunk == 0 && threadIdx.x == 0) a.next_slots[beam] = src;
        return;
    }
    // as many beams are without a child as children find their parent's slot taken
    int rank = __popcll(~firsts & ((1ull << w) - 1));
    for (; rank > 0; --rank) freed &= freed - 1;
    const int dst = a.slots[base + __ffsll((unsigned long long)freed) - 1];
    if (chunk == 0 && threadIdx.x == 0) a.next_slots[beam] = dst;
    long long at = chunk * kChunk;  // along the pools laid end to end, each rounded up to chunks
    for (int q = 0; q < a.npools; ++q) {
        const long long room = (a.bytes[q] + kChunk - 1) / kChunk * kChunk;
        if (at >= room) {
            at -= room;
            continue;
        }
        if (src < 0 || src >= a.nslots[q] || dst < 0 || dst >= a.nslots[q]) return;
        const char* from = a.pool[q] + src * a.bytes[q];
        char* to = a.pool[q] + dst * a.bytes[q];
        const long long end = at + kChunk < a.bytes[q] ? at + kChunk : a.bytes[q];
        // (slots may start at any byte: such 16-byte accesses are still one instruction)
        if (end - at == kChunk) {
            // a whole chunk: all of its loads in flight before the first store
            constexpr int N = kChunk / (256 * 16);
            u32x4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = *(const u32x4_any*)(from + at + (i * 256 + threadIdx.x) * 16);
#pragma unroll
            for (int i = 0; i < N; ++i)
                *(u32x4_any*)(to + at + (i * 256 + threadIdx.x) * 16) = v[i];
        } else {
            const long long whole = at + (end - at) / 16 * 16;
            for (long long i = at + threadIdx.x * 16; i < whole; i += 256 * 16)
                *(u32x4_any*)(to + i) = *(const u32x4_any*)(from + i);
            if (whole + threadIdx.x < end) to[whole + threadIdx.x] = from[whole + threadIdx.x];
        }
        return;
    }
}

}  // namespace

long long beam_workspace_bytes(const fcm_beam_problem& p) {
    return (long long)p.requests * p.beams * row_splits(p.vocab) * split_bytes(p.beams);
}

long long beam_rows_threads(const fcm_beam_problem& p) {
    return ((long long)p.requests * p.beams * row_splits(p.vocab) + 3) / 4 * 256;
}

int launch_beam_select(const BeamArgs& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    const int splits = row_splits(a.vocab), blocks = split_blocks(a.vocab);
    const long long waves = (long long)a.requests * a.beams * splits;
    const int grid = (int)((waves + 3) / 4);
    if (dtype == FCM_F32)
        beam_rows_kernel<float><<<grid, 256, 0, s>>>(a, splits, blocks);
    else if (dtype == FCM_F16)
        beam_rows_kernel<_Float16><<<grid, 256, 0, s>>>(a, splits, blocks);
    else
        beam_rows_kernel<__bf16><<<grid, 256, 0, s>>>(a, splits, blocks);
    const int rc = (int)hipGetLastError();
    if (rc != 0) return rc;
    beam_merge_kernel<<<a.requests, 64 * (a.beams < 8 ? a.beams : 8), 0, s>>>(a, splits);
    return (int)hipGetLastError();
}

namespace {
long long reorder_chunks(const ReorderArgs& a) {
    long long chunks = 0;
    for (int q = 0; q < a.npools; ++q) chunks += (a.bytes[q] + kChunk - 1) / kChunk;
    return chunks > 0 ? chunks : 1;
}
}  // namespace

long long beam_reorder_threads(const ReorderArgs& a) {
    return reorder_chunks(a) * a.requests * a.beams * 256;
}

int launch_beam_reorder(const ReorderArgs& a, void* stream) {
    const int chunks = (int)reorder_chunks(a);
    beam_reorder_kernel<<<chunks * a.requests * a.beams, 256, 0, (hipStream_t)stream>>>(a, chunks);
    return (int)hipGetLastError();
}

}  // namespace fcm
