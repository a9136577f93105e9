// seq.h -- argument blocks and launchers of the sequence operators (causal depthwise
// layer, selective scan, gated delta rule, 4-bit pointwise products, beam selection,
// verification of drafted tokens), shared by the API layer and the kernel translation units.  A launcher enqueues on `stream` and returns
// the hipError_t of the launch as an int.
#pragma once

#include <stdint.h>

#include "../../include/fcm.h"

namespace fcm {

// Records the calling thread's error text (NULL: clears it) and returns the status.
fcm_status set_error(fcm_status s, const char* text) noexcept;

struct Dw1dArgs {
    const void* x;
    const void* w;
    const float* bias;
    const int32_t* cu;     // NULL in the single-token call
    const int32_t* slots;
    const int32_t* carry;
    void* state;
    void* y;
    long long ldx, ldy;
    int D, tokens, seqs, nslots, silu;
};
int launch_dw1d_fwd(const Dw1dArgs& a, int dtype, int W, void* stream);
int launch_dw1d_step(const Dw1dArgs& a, int dtype, int W, void* stream);

struct ScanArgs {
    const void* x;
    const void* dt;
    const float* A;
    const void* Bm;
    const void* Cm;
    const float* skip;
    const float* dt_bias;
    const void* z;
    const int32_t* cu;
    const int32_t* slots;
    const int32_t* carry;
    float* state;
    void* ws;
    void* y;
    long long ldx, lddt, ldb, ldc, ldz, ldy;
    int D, N, groups, tokens, seqs, nslots, softplus;
};
int launch_scan_fwd(const ScanArgs& a, int dtype, void* stream);
int launch_scan_step(const ScanArgs& a, int dtype, void* stream);
long long scan_workspace_bytes(const fcm_scan_problem& p);

struct DeltaArgs {
    const void* q;
    const void* k;
    const void* v;
    const void* a;
    const void* b;
    const float* A;
    const float* dt_bias;
    const float* norm;
    const void* z;
    const int32_t* cu;     // NULL in the single-token call
    const int32_t* slots;
    const int32_t* carry;
    float* state;
    void* ws;
    void* y;
    long long ldq, ldk, ldv, lda, ldb, ldz, ldy;
    float scale, eps;
    int Hk, Hv, Dk, Dv, tokens, seqs, nslots, qk_norm, softplus;
    // set by the launcher
    long long places;  // for chunks, in the workspace
    float* squares;
    int wide_q, wide_k, wide_v, wide_z, wide_y, wide_state;  // alignment for vectors
    int shortest;  // sequences of up to so many tokens are another kernel's
    float* outs;   // before the norm, of 16-bit types
};
int launch_delta_fwd(DeltaArgs a, int dtype, void* stream);
int launch_delta_step(const DeltaArgs& a, int dtype, void* stream);
long long delta_workspace_bytes(const fcm_delta_problem& p);
long long delta_threads(const fcm_delta_problem& p);

struct Q4Args {
    const void* x;
    const uint8_t* q;
    const void* scales;
    const uint8_t* zeros;
    const float* bias;
    void* y;
    long long ldx, ldy;
    int M, C, K, group, act;
};
int launch_q4(const Q4Args& a, int dtype, void* stream);

struct Mx4Args {
    const void* x;          // 16-bit values, or codes
    const uint8_t* xscales; // of codes
    const uint8_t* q;
    const uint8_t* scales;
    const float* bias;
    void* y;
    long long ldx, ldy;
    int M, C, K, act;
};
int launch_mx4_quantize(const Mx4Args& a, int dtype, void* stream);
int launch_mx4_dequantize(const Mx4Args& a, int dtype, void* stream);
int launch_mx4(const Mx4Args& a, int dtype, void* stream);
int launch_mx4x4(const Mx4Args& a, int dtype, void* stream);
long long mx4x4_threads(const fcm_mx4_problem& p);

struct BeamArgs {
    const void* logits;
    const float* scores;
    const int32_t* done;
    void* ws;
    float* next_scores;
    int32_t* parent;
    int32_t* token;
    int32_t* next_done;
    long long ldl;
    int requests, beams, vocab, eos;
};
int launch_beam_select(const BeamArgs& a, int dtype, void* stream);
long long beam_workspace_bytes(const fcm_beam_problem& p);
long long beam_rows_threads(const fcm_beam_problem& p);

struct ReorderArgs {
    const int32_t* parent;
    const int32_t* slots;
    int32_t* next_slots;
    char* pool[FCM_BEAM_POOLS];
    long long bytes[FCM_BEAM_POOLS];
    long long nslots[FCM_BEAM_POOLS];
    int npools, requests, beams;
};
int launch_beam_reorder(const ReorderArgs& a, void* stream);
long long beam_reorder_threads(const ReorderArgs& a);

struct DraftArgs {
    const void* target;
    const void* draft;
    const int32_t* tokens;
    const int32_t* counts;
    const float* uniform;
    void* ws;
    int32_t* accepted;
    int32_t* next;
    long long ldt, ldd;
    float temperature;
    int requests, drafts, vocab;
};
int launch_draft_verify(const DraftArgs& a, int dtype, void* stream);
long long draft_workspace_bytes(const fcm_draft_problem& p);
long long draft_threads(const fcm_draft_problem& p);

}  // namespace fcm
