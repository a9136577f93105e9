// dw1d.hip -- causal depthwise layer along the token axis, for packed prompts and for one
// token of each sequence:  y[t] = act(bias + sum_k w[k] * x[t - (W-1) + k])  per channel.
//
// W multiply-adds an element: HBM bounds it.  On MI355X, 8192 tokens x 4096 bf16 channels, W = 4:
// 30 us, 4.5 TB/s of the 134 MB that have to move (a large copy reaches 5.2); one token of 96
// sequences: 3.8 us on the device, most of it launch and one memory latency.
#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

// Tokens of one workgroup: with 4 / 8 / 12 / 16 an 8192 x 4096 bf16 layer takes 36 / 30 / 31 / 31 us
// (fewer re-read more rows at their start; more than four waves a SIMD would spill them).
constexpr int kRun = 8;

template <typename T, int W, int V>
struct Taps {
    float w[V][W], b[V];
    __device__ __forceinline__ void load(const Dw1dArgs& a, int c) {
        // a channel's taps are consecutive, so V channels of them are V * W elements
        const T* p = (const T*)a.w + (long long)c * W;
        float flat[V * W];
        if constexpr (V == Vec<T>::N) {
#pragma unroll
            for (int i = 0; i < W; ++i) unpack16<T>(ld16(p + i * V), flat + i * V);
        } else {
#pragma unroll
            for (int i = 0; i < V * W; ++i) flat[i] = (float)p[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b[i] = a.bias ? a.bias[c + i] : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[i][k] = flat[i * W + k];
        }
    }
    // win[k]: the inputs of tap k
    __device__ __forceinline__ void apply(const float (*win)[V], int silu_on, float* out) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s = b[i];
#pragma unroll
            for (int k = 0; k < W; ++k) s = __builtin_fmaf(w[i][k], win[k][i], s);
            out[i] = silu_on ? silu(s) : s;
        }
    }
};

// V consecutive elements as they were loaded.
template <typename T, int V>
struct Raw {
    static constexpr bool WIDE = V == Vec<T>::N;
    typename std::conditional<WIDE, u32x4, vec_t<T, V>>::type v;
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (WIDE) {
            v = ld16(p);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = p[i];
        }
    }
    __device__ __forceinline__ void get(float* out) const {
        if constexpr (WIDE) {
            unpack16<T>(v, out);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = (float)v[i];
        }
    }
};

// One workgroup per (run of kRun tokens, block of channels), and one per (sequence, block of
// channels).  A run's workgroup writes the tokens whose whole window lies in the sequence's
// own rows; a sequence's workgroup writes its first W-1 tokens, which see the carried window,
// and then the new window.  So one workgroup alone touches a slot and reads it before writing.
template <typename T, int W, int V>
__global__ __launch_bounds__(256) void dw1d_fwd_kernel(Dw1dArgs a, int cblocks, long long units) {
    const T* x = (const T*)a.x;
    T* y = (T*)a.y;
    T* state = (T*)a.state;
    const int runs = (a.tokens + kRun - 1) / kRun;
    // An output larger than the L2s together (32 MB) is stored past them.  Alone that gains (64 MB:
    // 37.5 -> 33 us, 128 MB: 65 -> 59), and with the projection that reads it next too from 128 MB on
    // (129 -> 123 us, 64 MB: 81 both ways); below 32 MB that reader finds it in the L2s (32 MB: 48
    // against 49 us, 2 MB: 18 against 19).
    const bool past_l2 = (long long)a.tokens * a.D * (int)sizeof(T) > (32ll << 20);
    // Neighbouring runs, which read the same rows at their seam, on one XCD and its L2: 93 -> 68 MB
    // of reads for the layer above, at the same time.
    for (long long u = xcd_logical_id(blockIdx.x, gridDim.x); u < units; u += gridDim.x) {
        const int row = (int)(u / cblocks);
        const int c = (int)((u % cblocks) * blockDim.x + threadIdx.x) * V;
        const bool live = c < a.D;
        Taps<T, W, V> taps;
        if (row < runs) {
            const int t0 = row * kRun;
            // the loads first: which sequence the run is in is found meanwhile
            Raw<T, V> win[kRun + W - 1];
            const int cc = live ? c : 0;
#pragma unroll
            for (int i = 0; i < kRun + W - 1; ++i) {
                const int t = t0 + i - (W - 1);
                win[i].load(x + (t < 0 ? 0 : t < a.tokens ? t : a.tokens - 1) * a.ldx + cc);
            }
            taps.load(a, cc);
            int seq = seq_of_row(a.cu, a.seqs, t0);
            if (!live) continue;
            int start = seq_offset(a.cu, seq < a.seqs ? seq : a.seqs, a.tokens);
            int end = seq < a.seqs ? seq_offset(a.cu, seq + 1, a.tokens) : a.tokens;
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const int t = t0 + i;
                if (t >= a.tokens) break;
                while (seq < a.seqs && t >= end) {
                    ++seq;
                    start = end;
                    end = seq < a.seqs ? seq_offset(a.cu, seq + 1, a.tokens) : a.tokens;
                }
                if (seq >= a.seqs) break;
                if (t - start < W - 1) continue;
                float in[W][V], out[V];
#pragma unroll
                for (int k = 0; k < W; ++k) win[i + k].get(in[k]);
                taps.apply(in, a.silu, out);
                T* to = y + t * a.ldy + c;
                if (V == Vec<T>::N && past_l2) {
                    asm volatile("");  // (or both stores become one, which does not stream)
                    __builtin_nontemporal_store(pack16<T>(out), (u32x4*)to);
                    asm volatile("");
                } else {
                    store_row<T, V>(to, out);
                }
            }
        } else {
            const int seq = row - runs;
            if (!live) continue;
            const int start = seq_offset(a.cu, seq, a.tokens);
            const int end = seq_offset(a.cu, seq + 1, a.tokens);
            const int slot = a.state ? seq_slot(a.slots, seq, a.nslots) : -1;
            T* st = slot >= 0 ? state + (long long)slot * (W - 1) * a.D + c : nullptr;
            const bool carried = st && a.carry && a.carry[seq] != 0;
            const int len = end > start ? end - start : 0;
            // rows -(W-1) .. W-2 around the start: the carried window, then the first rows
            float line[2 * (W - 1)][V];
#pragma unroll
            for (int i = 0; i < 2 * (W - 1); ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) line[i][j] = 0.0f;
                if (i < W - 1) {
                    if (carried) load_row<T, V>(st + (long long)i * a.D, line[i]);
                } else if (i - (W - 1) < len) {
                    load_row<T, V>(x + (start + i - (W - 1)) * a.ldx + c, line[i]);
                }
            }
            taps.load(a, c);
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                if (i >= len) break;
                float out[V];
                taps.apply(line + i, a.silu, out);
                store_row<T, V>(y + (start + i) * a.ldy + c, out);
            }
            if (st) {
                // the new window: rows len-(W-1) .. len-1
#pragma unroll
                for (int i = 0; i < W - 1; ++i) {
                    float v[V];
                    if (len >= W - 1) {
                        load_row<T, V>(x + (long long)(end - (W - 1) + i) * a.ldx + c, v);
                    } else {
#pragma unroll
                        for (int k = 0; k < W - 1; ++k)  // (a select: registers have no index)
                            if (k == len)
#pragma unroll
                                for (int j = 0; j < V; ++j) v[j] = line[i + k][j];
                    }
                    store_row<T, V>(st + (long long)i * a.D, v);
                }
            }
        }
    }
}

template <typename T, int W, int V>
__global__ __launch_bounds__(256) void dw1d_step_kernel(Dw1dArgs a, int cblocks, long long units) {
    const T* x = (const T*)a.x;
    T* y = (T*)a.y;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int row = (int)(u / cblocks);
        const int c = (int)((u % cblocks) * blockDim.x + threadIdx.x) * V;
        if (c >= a.D) continue;
        const int slot = seq_slot(a.slots, row, a.nslots);
        float out[V];
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = 0.0f;
        if (slot >= 0) {
            T* st = (T*)a.state + (long long)slot * (W - 1) * a.D + c;
            Taps<T, W, V> taps;
            float win[W][V];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) load_row<T, V>(st + (long long)i * a.D, win[i]);
            load_row<T, V>(x + (long long)row * a.ldx + c, win[W - 1]);
            taps.load(a, c);
#pragma unroll
            for (int i = 0; i < W - 1; ++i) store_row<T, V>(st + (long long)i * a.D, win[i + 1]);
            taps.apply(win, a.silu, out);
        }
        store_row<T, V>(y + (long long)row * a.ldy + c, out);
    }
}

template <typename T, int W, int V>
int launch(const Dw1dArgs& a, bool step, void* stream) {
    const int vecs = (a.D + V - 1) / V;
    const int block = vecs >= 256 ? 256 : (vecs + 63) / 64 * 64;
    const int cblocks = (vecs + block - 1) / block;
    const long long rows = step ? a.seqs : (a.tokens + kRun - 1) / kRun + (long long)a.seqs;
    const long long units = rows * cblocks;
    const int grid = (int)(units < (1 << 22) ? (units + 7) / 8 * 8 : (1 << 22));
    if (step)
        dw1d_step_kernel<T, W, V><<<grid, block, 0, (hipStream_t)stream>>>(a, cblocks, units);
    else
        dw1d_fwd_kernel<T, W, V><<<grid, block, 0, (hipStream_t)stream>>>(a, cblocks, units);
    return (int)hipGetLastError();
}

// 16-byte vectors where every row of every tensor is a whole number of them; else one channel
// of a thread.
template <typename T, int W>
int pick_vec(const Dw1dArgs& a, bool step, void* stream) {
    constexpr int N = Vec<T>::N;
    const bool wide = a.D % N == 0 && rows16(a.x, a.ldx, sizeof(T)) &&
                      rows16(a.y, a.ldy, sizeof(T)) && rows16(a.w, 0, sizeof(T)) &&
                      rows16(a.state, a.D, sizeof(T));
    return wide ? launch<T, W, N>(a, step, stream) : launch<T, W, 1>(a, step, stream);
}

template <typename T>
int pick_taps(const Dw1dArgs& a, int W, bool step, void* stream) {
    switch (W) {
        case 2: return pick_vec<T, 2>(a, step, stream);
        case 3: return pick_vec<T, 3>(a, step, stream);
        case 4: return pick_vec<T, 4>(a, step, stream);
        case 5: return pick_vec<T, 5>(a, step, stream);
        case 6: return pick_vec<T, 6>(a, step, stream);
        case 7: return pick_vec<T, 7>(a, step, stream);
        case 8: return pick_vec<T, 8>(a, step, stream);
    }
    return (int)hipErrorInvalidValue;
}

int pick(const Dw1dArgs& a, int dtype, int W, bool step, void* stream) {
    if (dtype == FCM_F32) return pick_taps<float>(a, W, step, stream);
    if (dtype == FCM_F16) return pick_taps<_Float16>(a, W, step, stream);
    return pick_taps<__bf16>(a, W, step, stream);
}

}  // namespace

int launch_dw1d_fwd(const Dw1dArgs& a, int dtype, int W, void* stream) {
    return pick(a, dtype, W, false, stream);
}
int launch_dw1d_step(const Dw1dArgs& a, int dtype, int W, void* stream) {
    return pick(a, dtype, W, true, stream);
}

}  // namespace fcm
