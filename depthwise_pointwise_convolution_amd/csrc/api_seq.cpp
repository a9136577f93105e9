// api_seq.cpp -- the C ABI of the sequence operators: argument checks and dispatch.
// Every check happens on the host before anything is enqueued.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include "../../include/fcm.h"
#include "seq.h"

namespace fcm {
namespace {

fcm_status invalid(const char* text) { return set_error(FCM_ERR_INVALID_ARG, text); }
fcm_status unsupported(const char* text) { return set_error(FCM_ERR_UNSUPPORTED, text); }
fcm_status done(int rc) {
    return rc == 0 ? set_error(FCM_OK, nullptr)
                   : set_error(FCM_ERR_HIP, hipGetErrorString((hipError_t)rc));
}

#define SEQ_TRY(expr)                  \
    do {                               \
        fcm_status _s = (expr);        \
        if (_s != FCM_OK) return _s;   \
    } while (0)

constexpr long long kThreads = 1ll << 32;  // a launch has fewer

int elem(int dtype) { return dtype == FCM_F32 ? 4 : 2; }
bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

fcm_status float_type(int dtype) {
    if (dtype == FCM_F32 || dtype == FCM_F16 || dtype == FCM_BF16) return FCM_OK;
    if (dtype == FCM_I8) return unsupported("int8 storage has no sequence operators");
    return invalid("dtype is not an fcm_dtype");
}

// A required tensor with its element's alignment.
fcm_status tensor(const void* p, int align, const char* what_null, const char* what_align) {
    if (!p) return invalid(what_null);
    if (misaligned(p, align)) return invalid(what_align);
    return FCM_OK;
}
#define NEED(p, align) SEQ_TRY(tensor(p, align, #p " is NULL", #p " is misaligned for its type"))
#define MAYBE(p, align)                                                              \
    do {                                                                             \
        if ((p) && misaligned(p, align)) return invalid(#p " is misaligned for its type"); \
    } while (0)

// Row stride: 0 means dense; a smaller one than the row overlaps rows.
fcm_status stride(long long* ld, long long row) {
    if (*ld == 0) *ld = row;
    if (*ld < row) return invalid("a row stride is below its row's length");
    if (*ld > (1ll << 40)) return invalid("a row stride is above 2^40 elements");
    return FCM_OK;
}

fcm_status sequences(int tokens, int seqs, int slots, const int32_t* cu, const int32_t* slot_of,
                     const int32_t* carry, const void* state) {
    NEED(cu, 4);
    MAYBE(slot_of, 4);
    MAYBE(carry, 4);
    if (!state && (slot_of || carry))
        return invalid("slots and carry need a state array");
    if (state && !slot_of && slots < seqs)
        return invalid("slots == NULL needs at least seqs slots");
    if ((long long)tokens + seqs > (1 << 30)) return invalid("tokens + seqs is above 2^30");
    return FCM_OK;
}

fcm_status check_dw1d(const fcm_dw1d_problem* p) {
    if (!p) return invalid("problem is NULL");
    SEQ_TRY(float_type(p->dtype));
    if (p->D < 1 || p->W < 1 || p->tokens < 0 || p->seqs < 0 || p->slots < 0)
        return invalid("D and W must be positive, tokens, seqs and slots not negative");
    if (p->D > (1 << 24)) return unsupported("D above 2^24");
    if (p->W < 2 || p->W > 8) return unsupported("causal depthwise filters have 2 to 8 taps");
    if (p->silu != 0 && p->silu != 1) return invalid("silu must be 0 or 1");
    return FCM_OK;
}

fcm_status dw1d_args(const fcm_dw1d_problem* p, const void* x, const void* w, const float* bias,
                     const int32_t* slots, void* state, void* y, Dw1dArgs* a) {
    const int e = elem(p->dtype);
    NEED(w, e);
    if (p->tokens > 0) {
        NEED(x, e);
        NEED(y, e);
    }
    MAYBE(bias, 4);
    MAYBE(state, e);
    memset(a, 0, sizeof(*a));
    a->x = x;
    a->w = w;
    a->bias = bias;
    a->slots = slots;
    a->state = state;
    a->y = y;
    a->ldx = p->ldx;
    a->ldy = p->ldy;
    SEQ_TRY(stride(&a->ldx, p->D));
    SEQ_TRY(stride(&a->ldy, p->D));
    a->D = p->D;
    a->tokens = p->tokens;
    a->seqs = p->seqs;
    a->nslots = p->slots;
    a->silu = p->silu;
    return FCM_OK;
}

fcm_status check_scan(const fcm_scan_problem* p) {
    if (!p) return invalid("problem is NULL");
    SEQ_TRY(float_type(p->dtype));
    if (p->D < 1 || p->N < 1 || p->groups < 0 || p->tokens < 0 || p->seqs < 0 || p->slots < 0)
        return invalid("D and N must be positive, groups, tokens, seqs and slots not negative");
    if (p->D > (1 << 24)) return unsupported("D above 2^24");
    if (p->N > 64) return unsupported("more than 64 states of a channel");
    if ((long long)p->seqs * p->D > (1 << 25)) return unsupported("seqs * D above 2^25");
    if (p->groups > 0 && p->D % p->groups != 0) return invalid("groups must divide D");
    if (p->softplus != 0 && p->softplus != 1) return invalid("softplus must be 0 or 1");
    if ((long long)p->tokens + p->seqs > (1 << 30)) return invalid("tokens + seqs is above 2^30");
    return FCM_OK;
}

fcm_status scan_args(const fcm_scan_problem* p, const void* x, const void* dt, const float* A,
                     const void* Bm, const void* Cm, const float* skip, const float* dt_bias,
                     const void* z, const int32_t* slots, float* state, void* y, ScanArgs* a) {
    const int e = elem(p->dtype);
    NEED(A, 4);
    if (p->tokens > 0) {
        NEED(x, e);
        NEED(dt, e);
        NEED(Bm, e);
        NEED(Cm, e);
        NEED(y, e);
    }
    MAYBE(skip, 4);
    MAYBE(dt_bias, 4);
    MAYBE(z, e);
    MAYBE(state, 4);
    memset(a, 0, sizeof(*a));
    a->x = x;
    a->dt = dt;
    a->A = A;
    a->Bm = Bm;
    a->Cm = Cm;
    a->skip = skip;
    a->dt_bias = dt_bias;
    a->z = z;
    a->slots = slots;
    a->state = state;
    a->y = y;
    a->groups = p->groups > 0 ? p->groups : 1;
    const long long bc = (long long)a->groups * p->N;
    a->ldx = p->ldx;
    a->lddt = p->lddt;
    a->ldb = p->ldb;
    a->ldc = p->ldc;
    a->ldz = p->ldz;
    a->ldy = p->ldy;
    SEQ_TRY(stride(&a->ldx, p->D));
    SEQ_TRY(stride(&a->lddt, p->D));
    SEQ_TRY(stride(&a->ldz, p->D));
    SEQ_TRY(stride(&a->ldy, p->D));
    SEQ_TRY(stride(&a->ldb, bc));
    SEQ_TRY(stride(&a->ldc, bc));
    a->D = p->D;
    a->N = p->N;
    a->tokens = p->tokens;
    a->seqs = p->seqs;
    a->nslots = p->slots;
    a->softplus = p->softplus;
    return FCM_OK;
}

fcm_status check_beam(const fcm_beam_problem* p) {
    if (!p) return invalid("problem is NULL");
    SEQ_TRY(float_type(p->dtype));
    if (p->requests < 0 || p->beams < 1 || p->vocab < 1)
        return invalid("beams and vocab must be positive, requests not negative");
    if (p->beams > 32) return unsupported("more than 32 beams of a request");
    if (p->eos < -1 || p->eos >= p->vocab) return invalid("eos must be -1 or a token");
    // (the selection's places reach up to a split, vocab / 64, behind the vocabulary)
    if (p->vocab > INT_MAX - (1 << 25) + 1) return unsupported("vocab above 2^31 - 2^25");
    if ((long long)p->beams * p->vocab > INT_MAX) return unsupported("beams * vocab above 2^31-1");
    if ((long long)p->requests * p->beams > (1 << 24)) return unsupported("requests * beams above 2^24");
    return FCM_OK;
}

}  // namespace
}  // namespace fcm

using namespace fcm;

extern "C" {

fcm_status fcm_dw1d_fwd(const fcm_dw1d_problem* prob, const void* x, const void* w,
                        const float* bias, const int32_t* cu, const int32_t* slots,
                        const int32_t* carry, void* state, void* y, void* stream) {
    SEQ_TRY(check_dw1d(prob));
    SEQ_TRY(sequences(prob->tokens, prob->seqs, prob->slots, cu, slots, carry, state));
    Dw1dArgs a;
    SEQ_TRY(dw1d_args(prob, x, w, bias, slots, state, y, &a));
    a.cu = cu;
    a.carry = carry;
    if (prob->seqs == 0) return done(0);
    return done(launch_dw1d_fwd(a, prob->dtype, prob->W, stream));
}

fcm_status fcm_dw1d_step(const fcm_dw1d_problem* prob, const void* x, const void* w,
                         const float* bias, const int32_t* slots, void* state, void* y,
                         void* stream) {
    SEQ_TRY(check_dw1d(prob));
    if (prob->tokens != prob->seqs) return invalid("the single-token call needs tokens == seqs");
    NEED(state, 1);
    MAYBE(slots, 4);
    if (!slots && prob->slots < prob->seqs) return invalid("slots == NULL needs at least seqs slots");
    Dw1dArgs a;
    SEQ_TRY(dw1d_args(prob, x, w, bias, slots, state, y, &a));
    if (prob->seqs == 0) return done(0);
    return done(launch_dw1d_step(a, prob->dtype, prob->W, stream));
}

int64_t fcm_scan_workspace(const fcm_scan_problem* prob) {
    if (check_scan(prob) != FCM_OK) return -1;
    set_error(FCM_OK, nullptr);
    return scan_workspace_bytes(*prob);
}

fcm_status fcm_scan_fwd(const fcm_scan_problem* prob, const void* x, const void* dt,
                        const float* A, const void* Bm, const void* Cm, const float* skip,
                        const float* dt_bias, const void* z, const int32_t* cu,
                        const int32_t* slots, const int32_t* carry, float* state,
                        void* workspace, void* y, void* stream) {
    SEQ_TRY(check_scan(prob));
    SEQ_TRY(sequences(prob->tokens, prob->seqs, prob->slots, cu, slots, carry, state));
    ScanArgs a;
    SEQ_TRY(scan_args(prob, x, dt, A, Bm, Cm, skip, dt_bias, z, slots, state, y, &a));
    if (scan_workspace_bytes(*prob) > 0) NEED(workspace, 16);
    a.cu = cu;
    a.carry = carry;
    a.ws = workspace;
    if (prob->seqs == 0) return done(0);
    return done(launch_scan_fwd(a, prob->dtype, stream));
}

fcm_status fcm_scan_step(const fcm_scan_problem* prob, const void* x, const void* dt,
                         const float* A, const void* Bm, const void* Cm, const float* skip,
                         const float* dt_bias, const void* z, const int32_t* slots,
                         float* state, void* y, void* stream) {
    SEQ_TRY(check_scan(prob));
    if (prob->tokens != prob->seqs) return invalid("the single-token call needs tokens == seqs");
    NEED(state, 4);
    MAYBE(slots, 4);
    if (!slots && prob->slots < prob->seqs) return invalid("slots == NULL needs at least seqs slots");
    ScanArgs a;
    SEQ_TRY(scan_args(prob, x, dt, A, Bm, Cm, skip, dt_bias, z, slots, state, y, &a));
    if (prob->seqs == 0) return done(0);
    return done(launch_scan_step(a, prob->dtype, stream));
}

fcm_status fcm_q4_fwd(const fcm_q4_problem* prob, const void* x, const void* q,
                      const void* scales, const uint8_t* zeros, const float* bias, void* y,
                      void* stream) {
    if (!prob) return invalid("problem is NULL");
    const fcm_q4_problem& p = *prob;
    SEQ_TRY(float_type(p.dtype));
    if (p.dtype == FCM_F32) return unsupported("4-bit weights need 16-bit activations");
    if (p.M < 0 || p.C < 1 || p.K < 1) return invalid("C and K must be positive, M not negative");
    if (p.C % 8 != 0) return unsupported("C must be a multiple of 8");
    if (p.group != 32 && p.group != 64 && p.group != 128)
        return unsupported("groups have 32, 64 or 128 channels");
    if (p.act < FCM_ACT_NONE || p.act > FCM_ACT_RELU6) return invalid("act is not an fcm_act");
    if (p.C > (1 << 20) || p.M > (1 << 20) || p.K > (1 << 24))
        return unsupported("C or M above 2^20, K above 2^24");
    Q4Args a;
    memset(&a, 0, sizeof(a));
    a.ldx = p.ldx;
    a.ldy = p.ldy;
    SEQ_TRY(stride(&a.ldx, p.C));
    SEQ_TRY(stride(&a.ldy, p.K));
    if (a.ldx % 8 != 0) return invalid("ldx must be a multiple of 8");
    if (a.ldx >= (1ll << 26)) return unsupported("ldx of 2^26 or more");
    NEED(q, 4);
    NEED(scales, 2);
    MAYBE(bias, 4);
    if (p.M == 0) return done(0);
    NEED(x, 16);
    NEED(y, 2);
    a.x = x;
    a.q = (const uint8_t*)q;
    a.scales = scales;
    a.zeros = zeros;
    a.bias = bias;
    a.y = y;
    a.M = p.M;
    a.C = p.C;
    a.K = p.K;
    a.group = p.group;
    a.act = p.act;
    return done(launch_q4(a, p.dtype, stream));
}

int64_t fcm_beam_workspace(const fcm_beam_problem* prob) {
    if (check_beam(prob) != FCM_OK) return -1;
    set_error(FCM_OK, nullptr);
    return beam_workspace_bytes(*prob);
}

fcm_status fcm_beam_select(const fcm_beam_problem* prob, const void* logits,
                           const float* scores, const int32_t* done_flags, void* workspace,
                           float* next_scores, int32_t* parent, int32_t* token,
                           int32_t* next_done, void* stream) {
    SEQ_TRY(check_beam(prob));
    BeamArgs a;
    memset(&a, 0, sizeof(a));
    a.ldl = prob->ldl;
    SEQ_TRY(stride(&a.ldl, prob->vocab));
    if (prob->requests == 0) return done(0);
    NEED(logits, elem(prob->dtype));
    NEED(scores, 4);
    MAYBE(done_flags, 4);
    if (done_flags && prob->eos < 0) return invalid("done flags need an eos token");
    if (beam_workspace_bytes(*prob) > 0) NEED(workspace, 16);
    NEED(next_scores, 4);
    NEED(parent, 4);
    NEED(token, 4);
    MAYBE(next_done, 4);
    a.logits = logits;
    a.scores = scores;
    a.done = done_flags;
    a.ws = workspace;
    a.next_scores = next_scores;
    a.parent = parent;
    a.token = token;
    a.next_done = next_done;
    a.requests = prob->requests;
    a.beams = prob->beams;
    a.vocab = prob->vocab;
    a.eos = prob->eos;
    if (beam_rows_threads(*prob) >= kThreads)
        return unsupported("too large requests * beams * vocab for one launch");
    return done(launch_beam_select(a, prob->dtype, stream));
}

fcm_status fcm_beam_reorder(const fcm_beam_problem* prob, const int32_t* parent,
                            const int32_t* slots, int32_t* next_slots, int32_t npools,
                            void* const* pools, const int64_t* pool_bytes,
                            const int64_t* pool_slots, void* stream) {
    SEQ_TRY(check_beam(prob));
    if (npools < 0 || npools > FCM_BEAM_POOLS) return invalid("npools must be 0 to FCM_BEAM_POOLS");
    if (npools > 0 && (!pools || !pool_bytes || !pool_slots))
        return invalid("pools, pool_bytes or pool_slots is NULL");
    ReorderArgs a;
    memset(&a, 0, sizeof(a));
    for (int p = 0; p < npools; ++p) {
        if (!pools[p]) return invalid("a pool is NULL");
        if (pool_bytes[p] < 1 || pool_bytes[p] > (1ll << 40))
            return invalid("a slot's bytes must be 1 to 2^40");
        if (pool_slots[p] < 0) return invalid("pool_slots must not be negative");
        a.pool[p] = (char*)pools[p];
        a.bytes[p] = pool_bytes[p];
        a.nslots[p] = pool_slots[p];
    }
    if (prob->requests == 0) return done(0);
    NEED(parent, 4);
    NEED(slots, 4);
    NEED(next_slots, 4);
    if (slots == next_slots) return invalid("slots and next_slots must be distinct arrays");
    a.parent = parent;
    a.slots = slots;
    a.next_slots = next_slots;
    a.npools = npools;
    a.requests = prob->requests;
    a.beams = prob->beams;
    if (beam_reorder_threads(a) >= kThreads)
        return unsupported("more than 2^24 pieces of 16 KB in all beams' states");
    return done(launch_beam_reorder(a, stream));
}

}  // extern "C"
