// seq_common.h -- device-side pieces the sequence operators share: the batch's offsets and
// slots, element loads in fp32, and the gate and step-size functions.
#pragma once

#include "common.h"

namespace fcm {

// Offset i of a batch, inside the tensors whatever the array holds.
__device__ __forceinline__ int seq_offset(const int32_t* cu, int i, int tokens) {
    const int v = cu[i];
    return v < 0 ? 0 : v > tokens ? tokens : v;
}

// The sequence that owns row t: the number of sequences that end at or before it (empty
// ones own no row).  t is the same for the whole wave, whose lanes look at 64 offsets a step.
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int seqs, int t) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int b = 0; b < seqs; b += 64)
        n += __popcll(__ballot(b + lane < seqs && cu[b + lane + 1] <= t));
    return n;
}

// Slot of sequence b, or -1 if it has none.
__device__ __forceinline__ int seq_slot(const int32_t* slots, int b, int nslots) {
    const int s = slots ? slots[b] : b;
    return (unsigned)s < (unsigned)nslots ? s : -1;
}

// V consecutive elements in fp32: one 16-byte load where V fills it, else element by element.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, float* out) {
    if constexpr (V == Vec<T>::N) {
        unpack16<T>(ld16(p), out);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = (float)p[i];
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float* v) {
    if constexpr (V == Vec<T>::N) {
        st16(p, pack16<T>(v));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = (T)v[i];
    }
}

// v * sigmoid(v) with the hardware's base-2 exponential and reciprocal (both within 1 ulp).
// exp(-v) overflows to infinity for v below -88, where the value is 0 to within 1e-36.
__device__ __forceinline__ float silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) <= 1.  u = 1 + e loses the low bits of
// a small e; what it lost, e - (u - 1), is exact and is added back to log(u), whose slope there
// is 1 to within e.  The exponential's argument is rounded: far below zero, where the result is e, its
// relative error is about (3 + 1.5 |v|) 2^-24, and below -87.3, where e would be subnormal, it is zero.
__device__ __forceinline__ float softplus(float v) {
    const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(v) * -1.44269504f);
    const float u = 1.0f + e;
    const float lost = e - (u - 1.0f);
    const float l = __builtin_fmaf(__builtin_amdgcn_logf(u), 0.69314718f, lost);
    return __builtin_fmaxf(v, 0.0f) + l;
}

inline bool rows16(const void* p, long long ld, int elem) {
    return ((uintptr_t)p & 15) == 0 && (ld * elem) % 16 == 0;
}

}  // namespace fcm
