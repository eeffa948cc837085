// Internal declarations of the logits operators around a round, shared by
// their C ABI (specv_logits_api.hip) and kernels (specv_adjust.hip,
// specv_record.hip, specv_distill.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specv.h"

namespace specv {

// What an entry point needs of a handle that it uses no workspace of.
int handle_device(specv_handle h);
int handle_max_vocab(specv_handle h);
// The event pair of the next profiled call, or nullptr (profiling off, the
// stream being captured, or an event that could not be read).
hipEvent_t* handle_events(specv_handle h, hipStream_t stream);

struct AdjustArgs {
    const void* in;
    long long i_sb, i_sp;         // element strides
    void* out;
    long long o_sb, o_sp;
    int B, n, V, C;               // C: chunks per row
    int pos0;
    int pp, PG;                   // positions per workgroup, position groups
    const specv_penalties* pen;   // nullptr: no penalties
    const int* counts;
    const unsigned* seen;
    int n_slots;
    const int* tokens;            // nullptr: no drafts
    long long tok_sb;
    const int* bias_off;          // nullptr: no biases
    const int* bias_tok;
    const float* bias_val;
    int n_bias;
    const unsigned* mask;         // nullptr: no mask
    long long m_sb, m_sp;         // word strides
};
hipError_t launch_adjust(AdjustArgs& a, bool bf16, hipStream_t stream, hipEvent_t* ev);

struct HistoryArgs {
    const int* slots;
    const int* tokens;            // nullptr: reset
    long long tok_sb;
    const int* lengths;
    int B, n, V, prompt;
    int* counts;
    unsigned* seen;
    int n_slots;
};
hipError_t launch_history_add(const HistoryArgs& a, hipStream_t stream, hipEvent_t* ev);
hipError_t launch_history_reset(const HistoryArgs& a, hipStream_t stream, hipEvent_t* ev);

struct RecordArgs {
    const void* in;
    long long sb, sp;
    int B, n, V, K;
    float scale, inv_t;           // log2(e) / T, 1 / T
    int* tok;
    float* val;
    float* lse;
    int blocks, reps;             // blocks per thread, loads of four groups per block (set by the launch)
};
hipError_t launch_top_logits(const RecordArgs& a, bool bf16, hipStream_t stream, hipEvent_t* ev);

enum DistillOp { kDistillLoss = 0, kDistillGrad = 1, kDistillLossGrad = 2 };

struct DistillArgs {
    const void* in;
    long long sb, sp;
    int B, n, V, K;
    const int* tok;
    const float* val;
    const float* tlse;
    long long rec_sb;
    const float* w;               // nullptr: 1
    float scale, inv_t;           // log2(e) / T, 1 / T
    int bucket;
    const float* slse;            // the student's log-sum-exps (gradient alone)
    float2* part;                 // workspace (nullptr: none): [row][parts] (max, sum) of the rest
    float* zs;                    // [row][2][K]: the student's logits of S; 1 where an entry stands for
                                  // its token
    int parts;
    float* loss;
    float* lse;
    int* flags;
    void* grad;
    long long g_sb, g_sp;
};
// Bytes of workspace that make the rows' parts separate workgroups; 0 where
// one workgroup per row is as fast.
size_t distill_workspace(DistillOp op, bool bf16, long long rows, int V, int K);
hipError_t launch_distill(const DistillArgs& a, DistillOp op, bool bf16, hipStream_t stream, hipEvent_t* ev);

}  // namespace specv
