// beam.hip -- beam search: the best continuations of each request over beams and vocabulary,
// and the reordering of the beams' states.
#include <float.h>
#include <limits.h>

#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

// What selection keeps of a logits row: its log-sum-exp, and its best tokens, best first.
struct RowHead {
    double lse;
    double pad;
};
struct Cand {
    float logit;
    int token;  // -1: the vocabulary has no more
};

__host__ __device__ inline long long row_bytes(int beams) {
    return (long long)sizeof(RowHead) + ((long long)beams * sizeof(Cand) + 15) / 16 * 16;
}

__device__ __forceinline__ bool before(float v, int i, float w, int j) {
    return v > w || (v == w && i < j);
}

template <typename T>
__device__ __forceinline__ float clean(T v) {
    const float f = (float)v;
    return f != f ? -__builtin_inff() : __builtin_fminf(f, FLT_MAX);
}

// One workgroup per row: a pass for the log-sum-exp, then one pass for each kept token.
template <typename T>
__global__ __launch_bounds__(256) void beam_rows_kernel(BeamArgs a) {
    __shared__ float sv[4];
    __shared__ int si[4];
    __shared__ double sd[4];
    const int row = blockIdx.x, tid = threadIdx.x, wave = tid >> 6;
    const T* l = (const T*)a.logits + row * a.ldl;
    char* out = (char*)a.ws + row * row_bytes(a.beams);
    Cand* cand = (Cand*)(out + sizeof(RowHead));
    float top = 0.0f;
    float pv = __builtin_inff();
    int pi = -1;
    for (int k = 0; k < a.beams; ++k) {
        // the best candidate behind (pv, pi)
        float bv = -__builtin_inff();
        int bi = INT_MAX;
        for (int v = tid; v < a.vocab; v += 256) {
            const float f = clean(l[v]);
            if (before(pv, pi, f, v) && before(f, v, bv, bi)) bv = f, bi = v;
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const float v = __shfl_xor(bv, o);
            const int i = __shfl_xor(bi, o);
            if (before(v, i, bv, bi)) bv = v, bi = i;
        }
        if ((tid & 63) == 0) sv[wave] = bv, si[wave] = bi;
        __syncthreads();
        for (int w = 0; w < 4; ++w)
            if (before(sv[w], si[w], bv, bi)) bv = sv[w], bi = si[w];
        __syncthreads();
        if (k == 0) top = bv;
        pv = bv;
        pi = bi;
        if (tid == 0) {
            cand[k].logit = bv;
            cand[k].token = bi == INT_MAX ? -1 : bi;
        }
    }
    double sum = 0.0;
    if (top > -__builtin_inff())
        for (int v = tid; v < a.vocab; v += 256)
            sum += (double)__builtin_amdgcn_exp2f((clean(l[v]) - top) * 1.44269504f);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if ((tid & 63) == 0) sd[wave] = sum;
    __syncthreads();
    if (tid == 0) ((RowHead*)out)->lse = (double)top + log(sd[0] + sd[1] + sd[2] + sd[3]);
}

// One wave per request: lane w walks beam w's best tokens, and the best head of all lanes is
// taken `beams` times.
__global__ __launch_bounds__(64) void beam_merge_kernel(BeamArgs a) {
    const int r = blockIdx.x, w = threadIdx.x;
    const bool live = w < a.beams;
    const int row = r * a.beams + (live ? w : 0);
    const char* in = (const char*)a.ws + row * row_bytes(a.beams);
    const Cand* cand = (const Cand*)(in + sizeof(RowHead));
    const double lse = ((const RowHead*)in)->lse;
    const float score = a.scores[row];
    const int ended = a.done ? a.done[row] : 0;
    const float inf = __builtin_inff();
    const bool dead = !(score > -inf) || !(lse > -(double)inf);
    int at = 0;  // tokens of this beam taken so far
    for (int k = 0; k < a.beams; ++k) {
        double total = -(double)inf;
        int flat = INT_MAX;
        if (live) {
            int tok = -1;
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
                tok = cand[at].token;
                const float l = cand[at].logit;
                if (tok >= 0 && l > -inf) total = (double)score + ((double)l - lse);
            }
            if (tok >= 0) flat = w * a.vocab + tok;
        }
        double bt = total;
        int bf = flat;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const double t = __shfl_xor(bt, o);
            const int f = __shfl_xor(bf, o);
            if (t > bt || (t == bt && f < bf)) bt = t, bf = f;
        }
        if (live && flat == bf) {
            const int i = r * a.beams + k;
            a.next_scores[i] = (float)bt;
            a.parent[i] = w;
            a.token[i] = bf - w * a.vocab;
            if (a.next_done) a.next_done[i] = ended != 0 || bf - w * a.vocab == a.eos;
            ++at;
        }
    }
}

constexpr long long kChunk = 32768;  // bytes of a pool one workgroup copies

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
        const long long whole = (a.bytes[q] + kChunk - 1) / kChunk * kChunk;
        if (at >= whole) {
            at -= whole;
            continue;
        }
        if (src < 0 || src >= a.nslots[q] || dst < 0 || dst >= a.nslots[q]) return;
        const char* from = a.pool[q] + src * a.bytes[q];
        char* to = a.pool[q] + dst * a.bytes[q];
        const long long end = at + kChunk < a.bytes[q] ? at + kChunk : a.bytes[q];
        if ((a.bytes[q] & 15) == 0 && ((uintptr_t)a.pool[q] & 15) == 0) {
            for (long long i = at + threadIdx.x * 16; i < end; i += 256 * 16)
                st16(to + i, ld16(from + i));
        } else {
            for (long long i = at + threadIdx.x * 4; i < end; i += 256 * 4)
                *(uint32_t*)(to + i) = *(const uint32_t*)(from + i);
        }
        return;
    }
}

}  // namespace

long long beam_workspace_bytes(const fcm_beam_problem& p) {
    return (long long)p.requests * p.beams * row_bytes(p.beams);
}

int launch_beam_select(const BeamArgs& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    const int rows = a.requests * a.beams;
    if (dtype == FCM_F32)
        beam_rows_kernel<float><<<rows, 256, 0, s>>>(a);
    else if (dtype == FCM_F16)
        beam_rows_kernel<_Float16><<<rows, 256, 0, s>>>(a);
    else
        beam_rows_kernel<__bf16><<<rows, 256, 0, s>>>(a);
    const int rc = (int)hipGetLastError();
    if (rc != 0) return rc;
    beam_merge_kernel<<<a.requests, 64, 0, s>>>(a);
    return (int)hipGetLastError();
}

int launch_beam_reorder(const ReorderArgs& a, void* stream) {
    long long chunks = 0;
    for (int q = 0; q < a.npools; ++q) chunks += (a.bytes[q] + kChunk - 1) / kChunk;
    if (chunks == 0) chunks = 1;
    const long long grid = chunks * a.requests * a.beams;
    if (grid > INT_MAX) return (int)hipErrorInvalidConfiguration;
    beam_reorder_kernel<<<(int)grid, 256, 0, (hipStream_t)stream>>>(a, (int)chunks);
    return (int)hipGetLastError();
}

}  // namespace fcm
