// scan.hip -- selective state-space scan, for packed prompts and for one token of each
// sequence.  Per channel d and state n:
//   h = exp(delta * A) * h + delta * B * x,   y = (sum_n C * h + skip * x) * silu(z).
//
// Prompts: an element of x takes N exponentials (two issue slots each) and 4 N multiplies and
// multiply-adds, about 130 slots with N = 16 against 8 bytes: the vector units bound it.  The
// recurrence leaves D * seqs independent chains, too few for 1024 SIMDs, so long sequences are cut
// into chunks and scanned twice, 11/6 of the work.  On MI355X: eleven prompts, 8192 tokens x 4096
// fp16 channels in all, N = 16: 238 us (in a kernel trace, where kernels do not overlap and each is a
// little slower, first pass 99, join 17, second pass 135; a pass without the cut would take 110 at the
// vector units' peak, the bytes 53); one prompt of 2048 x 2048 bf16: 51 us (20, 9 and 23).  For the
// eleven prompts the vector units are busy 86% of the first and 85% of the second pass (counters).
//
// One token: the fp32 state is read and written, 8 N bytes a channel: HBM bounds it.  256 tokens x
// 4096 channels: 26 us, 5.5 TB/s.
#include <float.h>

#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

// A in base 2.  A decay rate of -infinity is taken as the largest float: a step of zero then still
// leaves the state alone (0 * infinity would be NaN).  A rate that is NaN stays so (a maximum would
// make it -FLT_MAX).
__device__ __forceinline__ float rate2(float A) {
    const float r = A * 1.44269504f;
    return r < -FLT_MAX ? -FLT_MAX : r;
}

// A channel's N <= NP values: in 16-byte pieces (`wide`: N is a multiple of 4 and the array 16-byte
// aligned), or one by one.
template <int NP>
__device__ __forceinline__ void load_states(const float* p, int N, bool wide, float* v) {
    if (wide) {
#pragma unroll
        for (int q = 0; q < NP / 4; ++q) {
            const f32x4 w = 4 * q < N ? *(const f32x4*)(p + 4 * q) : f32x4{};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * q + j] = w[j];
        }
    } else {
#pragma unroll
        for (int n = 0; n < NP; ++n) v[n] = n < N ? p[n] : 0.0f;
    }
}
template <int NP>
__device__ __forceinline__ void store_states(float* p, int N, bool wide, const float* v) {
    if (wide) {
#pragma unroll
        for (int q = 0; q < NP / 4; ++q)
            if (4 * q < N) *(f32x4*)(p + 4 * q) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    } else {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            if (n < N) p[n] = v[n];
    }
}

// A chunk of a sequence, the work of one wave for 64 channels.
struct Chunk {
    int seq, first, end;  // rows [first, end)
    int index, count;     // of the sequence's chunks
};

// Chunk c of the batch: sequence b has max(1, ceil(length / len)) chunks, numbered one sequence
// after the other.  False behind the last.
__device__ __forceinline__ bool find_chunk(const ScanArgs& a, int len, int c, Chunk* out) {
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 64) {
        const int b = b0 + lane;
        int n = 0, start = 0, end = 0;
        if (b < a.seqs) {
            start = seq_offset(a.cu, b, a.tokens);
            end = seq_offset(a.cu, b + 1, a.tokens);
            n = end - start > len ? (end - start + len - 1) / len : 1;
        }
        int upto = n;  // chunks of sequences b0 .. b
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o);
            if (lane >= o) upto += v;
        }
        const int k = __popcll(__ballot(base + upto <= c));
        if (k < 64 && b0 + k < a.seqs) {
            const int before = base + __builtin_amdgcn_readlane(upto - n, k);
            out->seq = b0 + k;
            out->count = __builtin_amdgcn_readlane(n, k);
            out->index = c - before;
            out->first = __builtin_amdgcn_readlane(start, k) + out->index * len;
            const int last = __builtin_amdgcn_readlane(end, k);
            out->end = out->first + len < last ? out->first + len : last;
            return true;
        }
        base += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// Tokens of one turn of the scan's loop: the next ones are being loaded meanwhile.
constexpr int kTurn = 4;
constexpr int kScanWaves = 4;  // waves of a workgroup, 64 channels each

// Tokens whose B and C a workgroup holds in LDS at a time: 16 KB of fp32 for NS states.
template <int NS>
constexpr int scan_tile() {
    return 16384 / (2 * NS * 4) / kTurn * kTurn;
}

// Sum over the Q neighbouring lanes of a channel.
template <int Q>
__device__ __forceinline__ float quad_sum(float v) {
    if constexpr (Q > 1)  // lanes 1 0 3 2
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, true));
    if constexpr (Q > 2)  // lanes 2 3 0 1
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, v), 0x4e, 0xf, 0xf, true));
    return v;
}

// The scan of one chunk, in one of two passes.  Q neighbouring lanes have one channel, NP of its
// N states each, in registers.  A sequence longer than a chunk is scanned twice, so that its chunks
// run at the same time: LAST = false finds what a chunk adds to a state (from zero; the first chunk
// from the sequence's own) and the sum of its steps, whose exponential is the chunk's whole decay;
// scan_join_kernel adds up where every chunk starts; LAST = true starts there and gives outputs and
// the sequence's final state.  Workspace: starts [chunks][N][D], then sums [chunks][D].
//
// B and C are the same for all channels of a group: the workgroup converts them to fp32 in LDS
// once a tile, and its lanes read them by broadcast, four states an instruction.
template <typename T, int NP, int Q, bool LAST, bool GATE>
__global__ __launch_bounds__(64 * kScanWaves, 4) void scan_fwd_kernel(ScanArgs a, int len, int chunks,
                                                                   int gblocks, bool wide) {
    constexpr int NS = NP * Q, TILE = scan_tile<NS>();
    __shared__ f32x4 bc[TILE][(LAST ? 2 : 1) * NS / 4];
    const int per = a.D / a.groups;
    const int cblocks = gblocks * a.groups;
    float* starts = (float*)a.ws;
    float* sums = starts + (long long)chunks * a.N * a.D;
    const int c = blockIdx.x / cblocks;
    const int cb = blockIdx.x % cblocks;
    Chunk k;
    if (!find_chunk(a, len, c, &k)) return;
    if (!LAST && k.index == k.count - 1) return;
    // channel blocks of one group: B and C are the same for the whole workgroup
    const int g = cb / gblocks;
    const int dg = ((cb % gblocks) * blockDim.x + threadIdx.x) / Q;
    const bool live = dg < per;
    const int d = g * per + (live ? dg : 0);
    // this lane's states: [n0, n0 + left) of the channel's
    const int n0 = threadIdx.x % Q * NP;
    const int left = a.N - n0 < NP ? a.N - n0 : NP;
    // Row pointers, the same for the whole wave; they stay on the last row once they are there.
    const T* px = (const T*)a.x + k.first * a.ldx;
    const T* pd = (const T*)a.dt + k.first * a.lddt;
    const T* pz = (const T*)a.z + (GATE ? k.first * a.ldz : 0);
    T* py = (T*)a.y + k.first * a.ldy;
    T xs[kTurn], ds[kTurn], zs[kTurn];
    auto fetch = [&](int t, T* xv, T* dv, T* zv) {
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            xv[i] = px[d];
            dv[i] = pd[d];
            if (GATE) zv[i] = pz[d];
            const bool more = t + i + 1 < k.end;
            px += more ? a.ldx : 0;
            pd += more ? a.lddt : 0;
            if (GATE) pz += more ? a.ldz : 0;
        }
    };
    if (k.first < k.end) fetch(k.first, xs, ds, zs);
    const int slot = a.state ? seq_slot(a.slots, k.seq, a.nslots) : -1;
    float* st = slot >= 0 ? a.state + ((long long)slot * a.D + d) * a.N + n0 : nullptr;
    const bool carried = st && a.carry && a.carry[k.seq] != 0;
    float h[NP], A[NP];
    load_states<NP>(a.A + (long long)d * a.N + n0, left, wide, A);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        A[n] = rate2(A[n]);
        h[n] = 0.0f;
    }
    // (with several chunks the last one may already be writing the state)
    if (LAST && k.count > 1) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            if (n < left) h[n] = starts[((long long)c * a.N + n0 + n) * a.D + d];
    } else if (k.index == 0 && carried) {
        load_states<NP>(st, left, wide, h);
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f;
    const float skip = LAST && a.skip ? a.skip[d] : 0.0f;
    if (!LAST && k.index == 0 && live) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            if (n < left) starts[((long long)c * a.N + n0 + n) * a.D + d] = h[n];
    }
    float sum = 0.0f;
    for (int tile = k.first; tile < k.end; tile += TILE) {
        const int rows = tile + TILE < k.end ? TILE : k.end - tile;
        __syncthreads();
        // (up to whole turns, with zeros for the tokens behind the end)
        const int filled = (rows + kTurn - 1) / kTurn * kTurn * NS;
        for (int i = threadIdx.x; i < filled; i += blockDim.x) {
            const int t = i / NS, n = i % NS;
            const long long r = tile + t;
            const bool in = n < a.N && t < rows;
            const T* b = (const T*)a.Bm + r * a.ldb + (long long)g * a.N + n;
            const T* cc = (const T*)a.Cm + r * a.ldc + (long long)g * a.N + n;
            float* to = (float*)bc[t];
            to[n] = in ? (float)*b : 0.0f;
            if (LAST) to[NS + n] = in ? (float)*cc : 0.0f;
        }
        __syncthreads();
        for (int t0 = 0; t0 < rows; t0 += kTurn) {
            T xn[kTurn], dn[kTurn], zn[kTurn];
            fetch(tile + t0 + kTurn, xn, dn, zn);
            float outs[kTurn];
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                // Tokens behind the end take a step of zero on a B of zero, which leaves the state as
                // it is.
                const bool here = t0 + i < rows;
                const f32x4* row = bc[t0 + i] + n0 / 4;
                const float xv = (float)xs[i];
                const float v = (float)ds[i] + bias;
                const float sp = softplus(v);
                const float delta = here ? (a.softplus ? sp : v) : 0.0f;
                const float dx = here ? delta * xv : 0.0f;
                float out = 0.0f;
#pragma unroll
                for (int q = 0; q < NP / 4; ++q) {
                    const f32x4 B = row[q];
                    f32x4 C;
                    if (LAST) C = row[NS / 4 + q];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int n = 4 * q + j;
                        const float e = __builtin_amdgcn_exp2f(delta * A[n]);
                        h[n] = __builtin_fmaf(e, h[n], dx * B[j]);
                        if (LAST) out = __builtin_fmaf(C[j], h[n], out);
                    }
                }
                if (LAST) {
                    out = __builtin_fmaf(skip, xv, quad_sum<Q>(out));
                    outs[i] = GATE ? out * silu((float)zs[i]) : out;
                    // Few states a lane: the turn's tokens are one block of straight code, whose
                    // chains overlap, and are stored behind it.  With many states their operands
                    // would not fit in the registers: the store ends each token's block.
                    if (NP >= 8 && here && live && n0 == 0) (py + i * a.ldy)[d] = (T)outs[i];
                } else {
                    sum += delta;
                }
            }
            if (LAST) {
                if (NP < 8) {
#pragma unroll
                    for (int i = 0; i < kTurn; ++i)
                        if (t0 + i < rows && live && n0 == 0) (py + i * a.ldy)[d] = (T)outs[i];
                }
                py += kTurn * a.ldy;
            }
#pragma unroll
            for (int i = 0; i < kTurn; ++i) xs[i] = xn[i], ds[i] = dn[i], zs[i] = zn[i];
        }
    }
    if (!live) return;
    if (LAST) {
        if (st && k.index == k.count - 1) store_states<NP>(st, left, wide, h);
    } else if (c + 1 < chunks) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            if (n < left) starts[((long long)(c + 1) * a.N + n0 + n) * a.D + d] = h[n];
        if (n0 == 0) sums[(long long)c * a.D + d] = sum;
    }
}

// Where a sequence's chunks start: start[j] = (what chunk j-1 added) + decay(j-1) * start[j-1].
// The first pass left the starts of chunks 0 and 1 whole.  One thread per (sequence, state,
// channel) goes along the chunks, kJoin of them at a time while the next are being loaded.
constexpr int kJoin = 16;
__global__ __launch_bounds__(256) void scan_join_kernel(ScanArgs a, int len, int chunks,
                                                        int blocks, long long units) {
    float* starts = (float*)a.ws;
    const float* sums = starts + (long long)chunks * a.N * a.D;
    const long long plane = (long long)a.N * a.D;
    const int lane = threadIdx.x & 63;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int seq = (int)(u / blocks);
        int before = 0, count = 0;  // chunks of the sequences before it, and its own
        for (int b0 = 0; b0 <= seq; b0 += 64) {
            const int b = b0 + lane;
            int n = 0;
            if (b <= seq) {
                const int rows = seq_offset(a.cu, b + 1, a.tokens) - seq_offset(a.cu, b, a.tokens);
                n = rows > len ? (rows + len - 1) / len : 1;
            }
            if (b == seq) count = n;
            int all = b < seq ? n : 0;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o);
            before += all;
        }
        count = __shfl(count, seq & 63);
        if (before + count > chunks) count = chunks - before;
        const uint32_t i = (uint32_t)(u % blocks) * 256 + threadIdx.x;  // (N * D is at most 2^30)
        if (count <= 2 || i >= plane) continue;
        const uint32_t d = i % (uint32_t)a.D;
        const float A = rate2(a.A[(long long)d * a.N + i / (uint32_t)a.D]);
        float* s = starts + (long long)before * plane + i;
        const float* w = sums + (long long)before * a.D + d;
        float add[kJoin], sum[kJoin];
        auto fetch = [&](int j) {
#pragma unroll
            for (int q = 0; q < kJoin; ++q) {
                const int c = j + q < count ? j + q : count - 1;
                add[q] = s[c * plane];
                sum[q] = w[(long long)(c - 1) * a.D];
            }
        };
        float h = s[plane];
        fetch(2);
        for (int j = 2; j < count; j += kJoin) {
            float start[kJoin];
#pragma unroll
            for (int q = 0; q < kJoin; ++q) {
                h = __builtin_fmaf(__builtin_amdgcn_exp2f(sum[q] * A), h, add[q]);
                start[q] = h;
            }
            if (j + kJoin < count) fetch(j + kJoin);
#pragma unroll
            for (int q = 0; q < kJoin; ++q)
                if (j + q < count) s[(j + q) * plane] = start[q];
        }
    }
}

// One thread per (row, channel).
template <typename T, int NP>
__global__ __launch_bounds__(64) void scan_step_kernel(ScanArgs a, int cblocks, long long units) {
    const T *x = (const T*)a.x, *dt = (const T*)a.dt, *z = (const T*)a.z;
    const T *Bm = (const T*)a.Bm, *Cm = (const T*)a.Cm;
    T* y = (T*)a.y;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int row = (int)(u / cblocks);
        const int d = (int)(u % cblocks) * 64 + threadIdx.x;
        if (d >= a.D) continue;
        const int g = d / (a.D / a.groups);
        const int slot = seq_slot(a.slots, row, a.nslots);
        float out = 0.0f;
        if (slot >= 0) {
            float* st = a.state + ((long long)slot * a.D + d) * a.N;
            const float xv = (float)x[row * a.ldx + d];
            float delta = (float)dt[row * a.lddt + d] + (a.dt_bias ? a.dt_bias[d] : 0.0f);
            if (a.softplus) delta = softplus(delta);
            const float dx = delta * xv;
            const T* b = Bm + row * a.ldb + (long long)g * a.N;
            const T* c = Cm + row * a.ldc + (long long)g * a.N;
            if (a.skip) out = a.skip[d] * xv;
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                if (n < a.N) {
                    const float A = rate2(a.A[(long long)d * a.N + n]);
                    const float h = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A), st[n],
                                                   dx * (float)b[n]);
                    st[n] = h;
                    out = __builtin_fmaf((float)c[n], h, out);
                }
            }
            if (z) out *= silu((float)z[row * a.ldz + d]);
        }
        y[row * a.ldy + d] = (T)out;
    }
}

// The same with Q neighbouring lanes a channel, four states a lane, so that a wave's state is one
// run of 16-byte pieces; the lanes' parts of the output are added among them.  A thread takes ROWS
// rows of the batch, all their loads in flight at once, and reads A once for them.  The state's
// bytes, read and written, bound it.
template <typename T, int Q, int ROWS>
__global__ __launch_bounds__(256) void scan_step4_kernel(ScanArgs a, int cblocks) {
    constexpr int CH = 256 / Q;  // channels of a workgroup
    const T *x = (const T*)a.x, *dt = (const T*)a.dt, *z = (const T*)a.z;
    T* y = (T*)a.y;
    const int row0 = blockIdx.x / cblocks * ROWS;
    const int d0 = blockIdx.x % cblocks * CH + threadIdx.x / Q;
    const int n = threadIdx.x % Q * 4;
    const bool live = d0 < a.D;
    const bool mine = live && n < a.N;  // (N need not fill the Q lanes)
    const int d = live ? d0 : 0, nn = mine ? n : 0;
    const long long bc = (long long)(d / (a.D / a.groups)) * a.N + nn;
    float* st[ROWS];
    f32x4 h[ROWS];
    T xs[ROWS], ds[ROWS], zs[ROWS], B[ROWS][4], C[ROWS][4];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const long long row = row0 + i < a.seqs ? row0 + i : a.seqs - 1;
        const int slot = seq_slot(a.slots, (int)row, a.nslots);
        st[i] = slot >= 0 && row0 + i < a.seqs
                    ? a.state + ((long long)slot * a.D + d) * a.N + nn : nullptr;
        if (st[i]) h[i] = *(const f32x4*)st[i];
        xs[i] = x[row * a.ldx + d];
        ds[i] = dt[row * a.lddt + d];
        if (z) zs[i] = z[row * a.ldz + d];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            B[i][j] = ((const T*)a.Bm)[row * a.ldb + bc + j];
            C[i][j] = ((const T*)a.Cm)[row * a.ldc + bc + j];
        }
    }
    f32x4 A = *(const f32x4*)(a.A + (long long)d * a.N + nn);
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] = rate2(A[j]);
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f;
    const float skip = a.skip ? a.skip[d] : 0.0f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (row0 + i >= a.seqs) break;
        float out = 0.0f;
        if (st[i]) {
            const float xv = (float)xs[i];
            float delta = (float)ds[i] + bias;
            if (a.softplus) delta = softplus(delta);
            const float dx = delta * xv;
            if (mine) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[i][j] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A[j]), h[i][j],
                                             dx * (float)B[i][j]);
                    out = __builtin_fmaf((float)C[i][j], h[i][j], out);
                }
                *(f32x4*)st[i] = h[i];
            }
#pragma unroll
            for (int o = 1; o < Q; o <<= 1) out += __shfl_xor(out, o);
            out = __builtin_fmaf(skip, xv, out);
            if (z) out *= silu((float)zs[i]);
        }
        if (live && n == 0) y[(row0 + i) * a.ldy + d] = (T)out;
    }
}

// Waves of one chunk at 64 channels each.
long long chunk_waves(int D, int groups) { return (long long)((D / groups + 63) / 64) * groups; }
// Waves the scan would have if each took 64 channels of one token, in 4096ths.
long long token_waves(int tokens, int D, int groups) {
    return tokens * chunk_waves(D, groups) / 4096;
}

// Tokens of a chunk: short ones bring waves for a small batch, long ones hand on fewer states.
// us with 8 / 16 / 32 / 64 / 128 tokens, 16 states, bf16:
//   512 x 1024: 27 / 29 / 38 / 59 / 102, 512 x 4096: 40 / 35 / 40 / 60 / 102,
//   2048 x 2048: 76 / 59 / 54 / 65 / 107, 8192 x 4096: 425 / 291 / 237 / 221 / 232.
// One thread goes along a sequence's chunks to join them, so there are no more than 256 a sequence:
// 16000 x 256 takes 87 us with 32 tokens and 80 with 64.  That is of all sequences together (the host
// does not know their lengths): 8000 x 64 takes 43 us as one sequence and as four equal ones, but 109
// us as one of 7997 tokens beside three short ones, whose thousand chunks one thread joins.
int chunk_len(int tokens, int seqs, int D, int groups) {
    const long long w = token_waves(tokens, D, groups);
    int len = w < 2 ? 8 : w < 12 ? 16 : w < 48 ? 32 : 64;
    // Nor more than 2^23 waves for them (four times that where a channel has four lanes; the one chunk at
    // least of every sequence adds up to 2^25): a launch has fewer than 2^32 threads.
    while (len < (1 << 30) && (tokens / len > 256ll * (seqs > 0 ? seqs : 1) ||
                               tokens / len * chunk_waves(D, groups) > (1 << 23)))
        len *= 2;
    return len;
}

int grid_of(long long units) { return (int)(units < (1 << 22) ? units : (1 << 22)); }

template <typename T, int NP, int Q>
int run_fwd(const ScanArgs& a, hipStream_t s) {
    const int len = chunk_len(a.tokens, a.seqs, a.D, a.groups);
    const int chunks = a.tokens / len + a.seqs;
    const int waves = (a.D / a.groups * Q + 63) / 64;
    const int block = 64 * (waves < kScanWaves ? waves : kScanWaves);
    const int gblocks = (a.D / a.groups + block / Q - 1) / (block / Q);
    const int grid = chunks * gblocks * a.groups;
    const bool wide = a.N % 4 == 0 && (((uintptr_t)a.A | (uintptr_t)a.state) & 15) == 0;
    if (a.tokens > len) {
        scan_fwd_kernel<T, NP, Q, false, false><<<grid, block, 0, s>>>(a, len, chunks, gblocks, wide);
        if (a.tokens > 2 * len) {
            const int blocks = (int)(((long long)a.N * a.D + 255) / 256);
            const long long joins = (long long)a.seqs * blocks;
            scan_join_kernel<<<grid_of(joins), 256, 0, s>>>(a, len, chunks, blocks, joins);
        }
    }
    if (a.z)
        scan_fwd_kernel<T, NP, Q, true, true><<<grid, block, 0, s>>>(a, len, chunks, gblocks, wide);
    else
        scan_fwd_kernel<T, NP, Q, true, false><<<grid, block, 0, s>>>(a, len, chunks, gblocks, wide);
    return (int)hipGetLastError();
}

// Lanes of a channel.  16 states a lane leave the least to do twice; more states than that are
// spread over lanes, and so are those of a batch too small to give every SIMD a wave, whose time
// is the chain of one wave: 300 x 64 channels of 16 states take 23 us on one lane, 18 on four.
template <typename T>
int fwd_states(const ScanArgs& a, hipStream_t s) {
    const bool few = token_waves(a.tokens, a.D, a.groups) < 3;
    if (a.N <= 8) return few ? run_fwd<T, 4, 2>(a, s) : run_fwd<T, 8, 1>(a, s);
    if (a.N <= 16) return few ? run_fwd<T, 4, 4>(a, s) : run_fwd<T, 16, 1>(a, s);
    if (a.N <= 24) return run_fwd<T, 12, 2>(a, s);
    if (a.N <= 32) return run_fwd<T, 16, 2>(a, s);
    if (a.N <= 48) return run_fwd<T, 12, 4>(a, s);
    return run_fwd<T, 16, 4>(a, s);
}

template <typename T, int Q>
int run_step4(const ScanArgs& a, hipStream_t s) {
    const int cblocks = (a.D + 256 / Q - 1) / (256 / Q);
    // Rows of a thread: 256 x 4096 channels of 16 states take 29.5 / 27.4 / 30 us with 1 / 2 / 4;
    // one while the batch does not fill the card.
    if ((long long)a.seqs * cblocks >= 4096) {
        scan_step4_kernel<T, Q, 2><<<(a.seqs + 1) / 2 * cblocks, 256, 0, s>>>(a, cblocks);
    } else {
        scan_step4_kernel<T, Q, 1><<<a.seqs * cblocks, 256, 0, s>>>(a, cblocks);
    }
    return (int)hipGetLastError();
}

template <typename T, int NP>
int run_step1(const ScanArgs& a, hipStream_t s) {
    const int cblocks = (a.D + 63) / 64;
    const long long units = (long long)a.seqs * cblocks;
    scan_step_kernel<T, NP><<<grid_of(units), 64, 0, s>>>(a, cblocks, units);
    return (int)hipGetLastError();
}

template <typename T>
int step_states(const ScanArgs& a, hipStream_t s) {
    if (a.N % 4 == 0 && (((uintptr_t)a.A | (uintptr_t)a.state) & 15) == 0) {
        if (a.N <= 4) return run_step4<T, 1>(a, s);
        if (a.N <= 8) return run_step4<T, 2>(a, s);
        if (a.N <= 16) return run_step4<T, 4>(a, s);
        if (a.N <= 32) return run_step4<T, 8>(a, s);
        return run_step4<T, 16>(a, s);
    }
    if (a.N <= 8) return run_step1<T, 8>(a, s);
    if (a.N <= 16) return run_step1<T, 16>(a, s);
    if (a.N <= 32) return run_step1<T, 32>(a, s);
    return run_step1<T, 64>(a, s);
}

}  // namespace

int launch_scan_fwd(const ScanArgs& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return fwd_states<float>(a, s);
    if (dtype == FCM_F16) return fwd_states<_Float16>(a, s);
    return fwd_states<__bf16>(a, s);
}
int launch_scan_step(const ScanArgs& a, int dtype, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F32) return step_states<float>(a, s);
    if (dtype == FCM_F16) return step_states<_Float16>(a, s);
    return step_states<__bf16>(a, s);
}
long long scan_workspace_bytes(const fcm_scan_problem& p) {
    const int groups = p.groups > 0 ? p.groups : 1;
    const int len = chunk_len(p.tokens, p.seqs, p.D, groups);
    if (p.tokens <= len) return 0;
    return (long long)(p.tokens / len + p.seqs) * p.D * (p.N + 1) * 4;
}

}  // namespace fcm
