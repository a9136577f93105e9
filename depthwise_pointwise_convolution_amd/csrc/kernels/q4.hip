// q4.hip -- pointwise layer with 4-bit weights and group scales for a few tokens:
//   y[m][k] = act(bias[k] + sum_groups scale[k][g] * sum_{c in g} (q[k][c] - zero[k][g]) x[m][c]).
#include "seq_common.h"
#include "../seq.h"

namespace fcm {
namespace {

// The activation as a clamp that lets NaN through (a median of three would not).
__device__ __forceinline__ float clamp_act(float v, Act act) {
    return v < act.lo ? act.lo : v > act.hi ? act.hi : v;
}

// One wave per (output channel, token), lanes over words of 8 channels; the 64 partial sums
// are added across the wave.
template <typename T>
__global__ __launch_bounds__(256) void q4_kernel(Q4Args a, long long units) {
    const int lane = threadIdx.x & 63;
    const T* x = (const T*)a.x;
    const T* scales = (const T*)a.scales;
    T* y = (T*)a.y;
    const int groups = (a.C + a.group - 1) / a.group;
    for (long long u = blockIdx.x * 4ll + (threadIdx.x >> 6); u < units; u += gridDim.x * 4ll) {
        const int m = (int)(u % a.M);
        const int k = (int)(u / a.M);
        float sum = 0.0f;
        for (int c = lane * 8; c < a.C; c += 512) {
            const uint32_t w = *(const uint32_t*)(a.q + (long long)k * (a.C / 2) + c / 2);
            float xv[8];
            load_row<T, 8>(x + m * a.ldx + c, xv);
            const int g = c / a.group;
            const float s = (float)scales[(long long)k * groups + g];
            const float z = a.zeros ? (float)(a.zeros[(long long)k * groups + g] & 15) : 8.0f;
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part = __builtin_fmaf((float)((w >> (4 * i)) & 15) - z, xv[i], part);
            sum = __builtin_fmaf(s, part, sum);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
        if (lane == 0) {
            y[m * a.ldy + k] = (T)clamp_act(sum + (a.bias ? a.bias[k] : 0.0f), act_bounds(a.act));
        }
    }
}

}  // namespace

int launch_q4(const Q4Args& a, int dtype, void* stream) {
    const long long units = (long long)a.K * a.M;
    const long long blocks = (units + 3) / 4;
    const int grid = (int)(blocks < (1 << 22) ? blocks : (1 << 22));
    hipStream_t s = (hipStream_t)stream;
    if (dtype == FCM_F16)
        q4_kernel<_Float16><<<grid, 256, 0, s>>>(a, units);
    else
        q4_kernel<__bf16><<<grid, 256, 0, s>>>(a, units);
    return (int)hipGetLastError();
}

}  // namespace fcm
