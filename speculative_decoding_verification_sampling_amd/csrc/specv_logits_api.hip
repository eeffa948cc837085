// libspecv C ABI, the logits operators around a round: argument validation
// and launches.  They use nothing of a handle's workspace; every argument
// error is returned before anything is enqueued.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "specv.h"
#include "specv_logits.hpp"

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;   // keeps every offset far inside 64 bits
constexpr double kLog2eD = 1.4426950408889634;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Makes the handle's device current for one call.
class DeviceScope {
public:
    explicit DeviceScope(int device) {
        ok_ = hipGetDevice(&prev_) == hipSuccess && (prev_ == device || hipSetDevice(device) == hipSuccess);
        changed_ = ok_ && prev_ != device;
    }
    ~DeviceScope() {
        if (changed_) (void)hipSetDevice(prev_);
    }
    bool ok() const { return ok_; }

private:
    int prev_ = 0;
    bool ok_ = false, changed_ = false;
};

// Rows [B, n, V] at element strides: sizes and types every call checks.
specv_status check_rows(specv_handle h, specv_dtype dtype, int B, int n, int V, int64_t sb, int64_t sp) {
    if (!h) return SPECV_E_NULL;
    if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_E_DTYPE;
    if (B < 0 || n < 0 || V < 1) return SPECV_E_SHAPE;
    if (sb < 0 || sp < 0 || sb > kMaxStride || sp > kMaxStride) return SPECV_E_SHAPE;
    if (V > specv::handle_max_vocab(h)) return SPECV_E_CAPACITY;
    if ((int64_t)B * n > 0x7fffffffLL) return SPECV_E_SHAPE;
    return SPECV_OK;
}

// No element of one output row belongs to another.
bool rows_disjoint(int B, int n, int V, int64_t sb, int64_t sp) {
    const bool pos_inner = (n == 1 || sp >= V) && (B == 1 || sb >= (n - 1) * sp + V);
    const bool row_inner = (B == 1 || sb >= V) && (n == 1 || sp >= (B - 1) * sb + V);
    return pos_inner || row_inner;
}

// An output may be its input, or must lie apart from it.
bool same_or_apart(const void* in, int64_t isb, int64_t isp, const void* out, int64_t osb, int64_t osp, int B,
                   int n, int V, size_t es) {
    if (in == out && (B == 1 || isb == osb) && (n == 1 || isp == osp)) return true;
    const uintptr_t i0 = reinterpret_cast<uintptr_t>(in), o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t i1 = i0 + ((B - 1) * isb + (n - 1) * isp + V) * es;
    const uintptr_t o1 = o0 + ((B - 1) * osb + (n - 1) * osp + V) * es;
    return i1 <= o0 || o1 <= i0;
}

specv_status done(hipError_t e) {
    if (e == hipSuccess) return SPECV_OK;
    return e == hipErrorInvalidValue ? SPECV_E_SHAPE : SPECV_E_HIP;
}

specv_status check_history(specv_handle h, const int32_t* slots, int B, int V, const int32_t* counts,
                           const uint32_t* seen, int n_slots) {
    if (!h) return SPECV_E_NULL;
    if (B < 0 || V < 1 || n_slots < 0) return SPECV_E_SHAPE;
    if (V > specv::handle_max_vocab(h)) return SPECV_E_CAPACITY;
    if (B == 0 || n_slots == 0) return SPECV_OK;
    if (!slots || !counts || !seen) return SPECV_E_NULL;
    if (!aligned(slots, 4) || !aligned(counts, 4) || !aligned(seen, 4)) return SPECV_E_ALIGN;
    return SPECV_OK;
}

// The arguments every specv_distill_* call shares; B * n == 0 leaves with SPECV_OK.
specv_status distill_args(specv_handle h, const void* student, int64_t sb, int64_t sp, specv_dtype dtype, int B,
                          int n, int V, const specv_teacher* rec, const float* weights, float temperature,
                          specv_tail tail, specv::DistillArgs* a) {
    const specv_status st = check_rows(h, dtype, B, n, V, sb, sp);
    if (st != SPECV_OK) return st;
    if (tail != SPECV_TAIL_RENORM && tail != SPECV_TAIL_BUCKET) return SPECV_E_PARAM;
    if (!(temperature > 0.f) || !isfinite(temperature) || !isfinite((float)(kLog2eD / temperature)))
        return SPECV_E_PARAM;
    if (!rec) return SPECV_E_NULL;
    if (rec->K < 1 || rec->K > SPECV_MAX_RECORD_K) return SPECV_E_PARAM;
    if (B == 0 || n == 0) return SPECV_OK;
    if (rec->stride_b < n || rec->stride_b > kMaxStride) return SPECV_E_SHAPE;
    if (!student || !rec->tokens || !rec->logits || (tail == SPECV_TAIL_BUCKET && !rec->lse)) return SPECV_E_NULL;
    if (!aligned(student, dtype == SPECV_BF16 ? 2 : 4) || !aligned(rec->tokens, 4) || !aligned(rec->logits, 4) ||
        (rec->lse && !aligned(rec->lse, 8)) || (weights && !aligned(weights, 4)))
        return SPECV_E_ALIGN;
    a->in = student;
    a->sb = sb;
    a->sp = sp;
    a->B = B;
    a->n = n;
    a->V = V;
    a->K = rec->K;
    a->tok = rec->tokens;
    a->val = rec->logits;
    a->tlse = rec->lse;
    a->rec_sb = rec->stride_b;
    a->w = weights;
    a->scale = (float)(kLog2eD / temperature);
    a->inv_t = (float)(1.0 / temperature);
    a->bucket = tail == SPECV_TAIL_BUCKET;
    return SPECV_OK;
}

specv_status grad_args(const specv::DistillArgs& a, specv_dtype dtype, void* grad, int64_t gsb, int64_t gsp) {
    if (gsb < 0 || gsp < 0 || gsb > kMaxStride || gsp > kMaxStride) return SPECV_E_SHAPE;
    const size_t es = dtype == SPECV_BF16 ? 2 : 4;
    if (!grad) return SPECV_E_NULL;
    if (!aligned(grad, es)) return SPECV_E_ALIGN;
    if (!rows_disjoint(a.B, a.n, a.V, gsb, gsp) ||
        !same_or_apart(a.in, a.sb, a.sp, grad, gsb, gsp, a.B, a.n, a.V, es))
        return SPECV_E_SHAPE;
    return SPECV_OK;
}

// Takes a given workspace, when it is large enough and parts are worth it.
specv_status use_workspace(specv::DistillArgs& a, specv::DistillOp op, specv_dtype dtype, void* workspace,
                           int64_t bytes) {
    if (!workspace) return SPECV_OK;
    if (!aligned(workspace, 16)) return SPECV_E_ALIGN;
    const size_t need = specv::distill_workspace(op, dtype == SPECV_BF16, (long long)a.B * a.n, a.V, a.K);
    if (bytes < 0 || (size_t)bytes < need) return SPECV_E_CAPACITY;
    if (need == 0) return SPECV_OK;
    const size_t z = (size_t)a.B * a.n * 2 * a.K * sizeof(float);
    a.part = static_cast<float2*>(workspace);
    a.zs = reinterpret_cast<float*>(static_cast<char*>(workspace) + (need - z));
    return SPECV_OK;
}

specv_status launch_distill_op(specv_handle h, void* stream, const specv::DistillArgs& a, specv::DistillOp op,
                               specv_dtype dtype) {
    DeviceScope dev(specv::handle_device(h));
    if (!dev.ok()) return SPECV_E_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return done(specv::launch_distill(a, op, dtype == SPECV_BF16, s, specv::handle_events(h, s)));
}

}  // namespace

extern "C" {

specv_status specv_adjust_logits(specv_handle h, void* stream, const void* logits, int64_t stride_b,
                                 int64_t stride_pos, void* out, int64_t out_stride_b, int64_t out_stride_pos,
                                 specv_dtype dtype, int B, int n_pos, int V, int pos0,
                                 const specv_adjustments* adj) {
    const specv_status st = check_rows(h, dtype, B, n_pos, V, stride_b, stride_pos);
    if (st != SPECV_OK) return st;
    if (n_pos > SPECV_MAX_GAMMA + 1 || pos0 < 0 || pos0 > SPECV_MAX_GAMMA) return SPECV_E_SHAPE;
    if (out_stride_b < 0 || out_stride_pos < 0 || out_stride_b > kMaxStride || out_stride_pos > kMaxStride)
        return SPECV_E_SHAPE;
    if (!adj) return SPECV_E_NULL;
    if (B == 0 || n_pos == 0) return SPECV_OK;
    if (!logits || !out) return SPECV_E_NULL;
    const size_t es = dtype == SPECV_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(out, es)) return SPECV_E_ALIGN;
    specv::AdjustArgs a{};
    if (adj->penalties) {
        if (!aligned(adj->penalties, 16)) return SPECV_E_ALIGN;
        if (adj->n_slots < 0) return SPECV_E_SHAPE;
        if (adj->n_slots > 0 && (!adj->counts || !adj->seen)) return SPECV_E_NULL;
        if (adj->n_slots > 0 && (!aligned(adj->counts, 4) || !aligned(adj->seen, 4))) return SPECV_E_ALIGN;
        a.pen = adj->penalties;
        a.counts = adj->counts;
        a.seen = adj->seen;
        a.n_slots = adj->n_slots;
        const int before = pos0 + n_pos - 1;        // drafts that stand before a row of this call
        if (adj->draft_tokens && before > 0) {
            if (adj->token_stride < before || adj->token_stride > kMaxStride) return SPECV_E_SHAPE;
            if (!aligned(adj->draft_tokens, 4)) return SPECV_E_ALIGN;
            a.tokens = adj->draft_tokens;
            a.tok_sb = adj->token_stride;
        }
    }
    if (adj->bias_offsets) {
        if (adj->n_bias < 0) return SPECV_E_SHAPE;
        if (adj->n_bias > 0) {
            if (!adj->bias_tokens || !adj->bias_values) return SPECV_E_NULL;
            if (!aligned(adj->bias_offsets, 4) || !aligned(adj->bias_tokens, 4) || !aligned(adj->bias_values, 4))
                return SPECV_E_ALIGN;
            a.bias_off = adj->bias_offsets;
            a.bias_tok = adj->bias_tokens;
            a.bias_val = adj->bias_values;
            a.n_bias = adj->n_bias;
        }
    }
    if (adj->mask) {
        if (adj->mask_stride_b < 0 || adj->mask_stride_pos < 0 || adj->mask_stride_b > kMaxStride ||
            adj->mask_stride_pos > kMaxStride)
            return SPECV_E_SHAPE;
        if (!aligned(adj->mask, 4)) return SPECV_E_ALIGN;
        a.mask = adj->mask;
        a.m_sb = adj->mask_stride_b;
        a.m_sp = adj->mask_stride_pos;
    }
    if (!rows_disjoint(B, n_pos, V, out_stride_b, out_stride_pos) ||
        !same_or_apart(logits, stride_b, stride_pos, out, out_stride_b, out_stride_pos, B, n_pos, V, es))
        return SPECV_E_SHAPE;
    a.in = logits;
    a.i_sb = stride_b;
    a.i_sp = stride_pos;
    a.out = out;
    a.o_sb = out_stride_b;
    a.o_sp = out_stride_pos;
    a.B = B;
    a.n = n_pos;
    a.V = V;
    a.pos0 = pos0;
    DeviceScope dev(specv::handle_device(h));
    if (!dev.ok()) return SPECV_E_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return done(specv::launch_adjust(a, dtype == SPECV_BF16, s, specv::handle_events(h, s)));
}

specv_status specv_history_add(specv_handle h, void* stream, const int32_t* slots, const int32_t* tokens,
                               int64_t token_stride, const int32_t* lengths, int B, int n_tokens, int V,
                               int prompt, int32_t* counts, uint32_t* seen, int n_slots) {
    const specv_status st = check_history(h, slots, B, V, counts, seen, n_slots);
    if (st != SPECV_OK) return st;
    if (n_tokens < 0 || token_stride > kMaxStride) return SPECV_E_SHAPE;
    if (B == 0 || n_tokens == 0 || n_slots == 0) return SPECV_OK;
    if (!tokens) return SPECV_E_NULL;
    if (B > 1 && token_stride < 0) return SPECV_E_SHAPE;
    if (!aligned(tokens, 4) || (lengths && !aligned(lengths, 4))) return SPECV_E_ALIGN;
    specv::HistoryArgs a{};
    a.slots = slots;
    a.tokens = tokens;
    a.tok_sb = token_stride;
    a.lengths = lengths;
    a.B = B;
    a.n = n_tokens;
    a.V = V;
    a.prompt = prompt != 0;
    a.counts = counts;
    a.seen = seen;
    a.n_slots = n_slots;
    DeviceScope dev(specv::handle_device(h));
    if (!dev.ok()) return SPECV_E_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return done(specv::launch_history_add(a, s, specv::handle_events(h, s)));
}

specv_status specv_history_reset(specv_handle h, void* stream, const int32_t* slots, int n, int V,
                                 int32_t* counts, uint32_t* seen, int n_slots) {
    const specv_status st = check_history(h, slots, n, V, counts, seen, n_slots);
    if (st != SPECV_OK || n == 0 || n_slots == 0) return st;
    specv::HistoryArgs a{};
    a.slots = slots;
    a.B = n;
    a.V = V;
    a.counts = counts;
    a.seen = seen;
    a.n_slots = n_slots;
    DeviceScope dev(specv::handle_device(h));
    if (!dev.ok()) return SPECV_E_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return done(specv::launch_history_reset(a, s, specv::handle_events(h, s)));
}

specv_status specv_top_logits(specv_handle h, void* stream, const void* logits, int64_t stride_b,
                              int64_t stride_pos, specv_dtype dtype, int B, int n_pos, int V, int K,
                              float temperature, int32_t* out_tokens, float* out_logits, float* out_lse) {
    const specv_status st = check_rows(h, dtype, B, n_pos, V, stride_b, stride_pos);
    if (st != SPECV_OK) return st;
    if (K < 1 || K > SPECV_MAX_RECORD_K) return SPECV_E_PARAM;
    if (!(temperature > 0.f) || !isfinite(temperature) || !isfinite((float)(kLog2eD / temperature)))
        return SPECV_E_PARAM;
    if (B == 0 || n_pos == 0) return SPECV_OK;
    if (!logits || !out_tokens || !out_logits || !out_lse) return SPECV_E_NULL;
    if (!aligned(logits, dtype == SPECV_BF16 ? 2 : 4) || !aligned(out_tokens, 4) || !aligned(out_logits, 4) ||
        !aligned(out_lse, 8))
        return SPECV_E_ALIGN;
    specv::RecordArgs a{};
    a.in = logits;
    a.sb = stride_b;
    a.sp = stride_pos;
    a.B = B;
    a.n = n_pos;
    a.V = V;
    a.K = K;
    a.scale = (float)(kLog2eD / temperature);
    a.inv_t = (float)(1.0 / temperature);
    a.tok = out_tokens;
    a.val = out_logits;
    a.lse = out_lse;
    DeviceScope dev(specv::handle_device(h));
    if (!dev.ok()) return SPECV_E_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return done(specv::launch_top_logits(a, dtype == SPECV_BF16, s, specv::handle_events(h, s)));
}

int64_t specv_distill_workspace(specv_dtype dtype, int B, int n_pos, int V, int K) {
    if ((dtype != SPECV_F32 && dtype != SPECV_BF16) || B < 0 || n_pos < 0 || V < 1 || V > SPECV_MAX_VOCAB || K < 1 ||
        K > SPECV_MAX_RECORD_K)
        return 0;
    return (int64_t)specv::distill_workspace(specv::kDistillLossGrad, dtype == SPECV_BF16, (long long)B * n_pos, V, K);
}

specv_status specv_distill_loss(specv_handle h, void* stream, const void* student, int64_t stride_b,
                                int64_t stride_pos, specv_dtype dtype, int B, int n_pos, int V,
                                const specv_teacher* teacher, const float* weights, float temperature,
                                specv_tail tail, float* out_loss, float* out_lse, int32_t* out_flags,
                                void* workspace, int64_t workspace_bytes) {
    specv::DistillArgs a{};
    specv_status st = distill_args(h, student, stride_b, stride_pos, dtype, B, n_pos, V, teacher, weights,
                                         temperature, tail, &a);
    if (st != SPECV_OK || B == 0 || n_pos == 0) return st;
    if (!out_loss || !out_lse) return SPECV_E_NULL;
    if (!aligned(out_loss, 4) || !aligned(out_lse, 8) || (out_flags && !aligned(out_flags, 4))) return SPECV_E_ALIGN;
    a.loss = out_loss;
    a.lse = out_lse;
    a.flags = out_flags;
    st = use_workspace(a, specv::kDistillLoss, dtype, workspace, workspace_bytes);
    if (st != SPECV_OK) return st;
    return launch_distill_op(h, stream, a, specv::kDistillLoss, dtype);
}

specv_status specv_distill_grad(specv_handle h, void* stream, const void* student, int64_t stride_b,
                                int64_t stride_pos, specv_dtype dtype, int B, int n_pos, int V,
                                const specv_teacher* teacher, const float* weights, float temperature,
                                specv_tail tail, const float* student_lse, void* grad, int64_t grad_stride_b,
                                int64_t grad_stride_pos) {
    specv::DistillArgs a{};
    specv_status st = distill_args(h, student, stride_b, stride_pos, dtype, B, n_pos, V, teacher, weights,
                                   temperature, tail, &a);
    if (st != SPECV_OK || B == 0 || n_pos == 0) return st;
    if (!student_lse) return SPECV_E_NULL;
    if (!aligned(student_lse, 8)) return SPECV_E_ALIGN;
    st = grad_args(a, dtype, grad, grad_stride_b, grad_stride_pos);
    if (st != SPECV_OK) return st;
    a.slse = student_lse;
    a.grad = grad;
    a.g_sb = grad_stride_b;
    a.g_sp = grad_stride_pos;
    return launch_distill_op(h, stream, a, specv::kDistillGrad, dtype);
}

specv_status specv_distill_loss_grad(specv_handle h, void* stream, const void* student, int64_t stride_b,
                                     int64_t stride_pos, specv_dtype dtype, int B, int n_pos, int V,
                                     const specv_teacher* teacher, const float* weights, float temperature,
                                     specv_tail tail, float* out_loss, int32_t* out_flags, void* grad,
                                     int64_t grad_stride_b, int64_t grad_stride_pos, void* workspace,
                                     int64_t workspace_bytes) {
    specv::DistillArgs a{};
    specv_status st = distill_args(h, student, stride_b, stride_pos, dtype, B, n_pos, V, teacher, weights,
                                   temperature, tail, &a);
    if (st != SPECV_OK || B == 0 || n_pos == 0) return st;
    if (!out_loss) return SPECV_E_NULL;
    if (!aligned(out_loss, 4) || (out_flags && !aligned(out_flags, 4))) return SPECV_E_ALIGN;
    st = grad_args(a, dtype, grad, grad_stride_b, grad_stride_pos);
    if (st != SPECV_OK) return st;
    a.loss = out_loss;
    a.flags = out_flags;
    a.grad = grad;
    a.g_sb = grad_stride_b;
    a.g_sp = grad_stride_pos;
    st = use_workspace(a, specv::kDistillLossGrad, dtype, workspace, workspace_bytes);
    if (st != SPECV_OK) return st;
    return launch_distill_op(h, stream, a, specv::kDistillLossGrad, dtype);
}

}  // extern "C"
