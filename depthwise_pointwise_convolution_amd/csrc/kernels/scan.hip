// scan.hip -- selective state-space scan, for packed prompts and for one token of each
// sequence.  Per channel d and state n:
//   h = exp(delta * A) * h + delta * B * x,   y = (sum_n C * h + skip * x) * silu(z).
#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

constexpr float kLog2e = 1.44269504f;

// One thread per (sequence, channel): the channel's N states in registers, token after token.
template <typename T, int NP>
__global__ __launch_bounds__(64) void scan_fwd_kernel(ScanArgs a, int cblocks, long long units) {
    const T *x = (const T*)a.x, *dt = (const T*)a.dt, *z = (const T*)a.z;
    const T *Bm = (const T*)a.Bm, *Cm = (const T*)a.Cm;
    T* y = (T*)a.y;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int seq = (int)(u / cblocks);
        const int d = (int)(u % cblocks) * 64 + threadIdx.x;
        if (d >= a.D) continue;
        const int g = d / (a.D / a.groups);
        const int start = seq_offset(a.cu, seq, a.tokens);
        const int end = seq_offset(a.cu, seq + 1, a.tokens);
        const int slot = a.state ? seq_slot(a.slots, seq, a.nslots) : -1;
        float* st = slot >= 0 ? a.state + ((long long)slot * a.D + d) * a.N : nullptr;
        const bool carried = st && a.carry && a.carry[seq] != 0;
        float h[NP], A[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            A[n] = n < a.N ? a.A[(long long)d * a.N + n] * kLog2e : 0.0f;
            h[n] = carried && n < a.N ? st[n] : 0.0f;
        }
        const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f;
        const float skip = a.skip ? a.skip[d] : 0.0f;
        for (int t = start; t < end; ++t) {
            const float xv = (float)x[t * a.ldx + d];
            float delta = (float)dt[t * a.lddt + d] + bias;
            if (a.softplus) delta = softplus(delta);
            const float dx = delta * xv;
            const T* b = Bm + t * a.ldb + (long long)g * a.N;
            const T* c = Cm + t * a.ldc + (long long)g * a.N;
            float out = skip * xv;
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                if (n < a.N) {
                    h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A[n]), h[n],
                                          dx * (float)b[n]);
                    out = __builtin_fmaf((float)c[n], h[n], out);
                }
            }
            if (z) out *= silu((float)z[t * a.ldz + d]);
            y[t * a.ldy + d] = (T)out;
        }
        if (st) {
#pragma unroll
            for (int n = 0; n < NP; ++n)
                if (n < a.N) st[n] = h[n];
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
                    const float A = a.A[(long long)d * a.N + n] * kLog2e;
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

template <typename T>
int pick_states(const ScanArgs& a, bool step, void* stream) {
    const int cblocks = (a.D + 63) / 64;
    const long long units = (long long)a.seqs * cblocks;
    const int grid = (int)(units < (1 << 22) ? units : (1 << 22));
    hipStream_t s = (hipStream_t)stream;
    auto go = [&](auto np) {
        constexpr int NP = decltype(np)::value;
        if (step)
            scan_step_kernel<T, NP><<<grid, 64, 0, s>>>(a, cblocks, units);
        else
            scan_fwd_kernel<T, NP><<<grid, 64, 0, s>>>(a, cblocks, units);
        return (int)hipGetLastError();
    };
    if (a.N <= 8) return go(std::integral_constant<int, 8>());
    if (a.N <= 16) return go(std::integral_constant<int, 16>());
    if (a.N <= 32) return go(std::integral_constant<int, 32>());
    return go(std::integral_constant<int, 64>());
}

int pick(const ScanArgs& a, int dtype, bool step, void* stream) {
    if (dtype == FCM_F32) return pick_states<float>(a, step, stream);
    if (dtype == FCM_F16) return pick_states<_Float16>(a, step, stream);
    return pick_states<__bf16>(a, step, stream);
}

}  // namespace

int launch_scan_fwd(const ScanArgs& a, int dtype, void* stream) {
    return pick(a, dtype, false, stream);
}
int launch_scan_step(const ScanArgs& a, int dtype, void* stream) {
    return pick(a, dtype, true, stream);
}
long long scan_workspace_bytes(const fcm_scan_problem&) { return 0; }

}  // namespace fcm
