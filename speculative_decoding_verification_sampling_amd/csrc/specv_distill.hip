// specv_distill_loss / _grad / _loss_grad: the distillation loss of student
// rows against a teacher's record, and its gradient.
//
// With x_v = z_v / T, S the record's tokens, and L, L_o the log-sum-exps of x
// over the whole row and over the tokens outside S:
//   log q_v = x_v - L,  log q_o = L_o - L
//   d loss / d z_v = w / T * (P q_v - p_v)                          v in S
//                    w / T * (P exp(x_v - L) - p_o exp(x_v - L_o))  otherwise
// One workgroup per row.  The tokens of S are marked in a bit row in LDS, so
// that the sum over the rest is a sum of its own (as a difference of sums it
// would lose what is left of a student that has learned S); S itself is
// summed from its K gathered logits.

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specv_device.hpp"

namespace specv {
namespace {

constexpr int kDisBlock = 1024;
constexpr int kDisWaves = kDisBlock / kWave;
constexpr int kMaxK = SPECV_MAX_RECORD_K;

struct DistillScratch {
    int tok[kMaxK];              // the record's tokens; -1: ignored
    float p[kMaxK];              // the teacher's probability (0 where ignored)
    float red[kDisWaves], red2[kDisWaves];
};

struct BlockMax {
    __device__ static inline float wave(float x) { return wave_max(x); }
    __device__ static inline float join(float a, float b) { return fmaxf(a, b); }
};
struct BlockSum {
    __device__ static inline float wave(float x) { return wave_sum(x); }
    __device__ static inline float join(float a, float b) { return a + b; }
};
template <typename Op>
__device__ inline float block_reduce(float x, float* red) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    x = Op::wave(x);
    __syncthreads();
    if (lane == 0) red[wave] = x;
    __syncthreads();
    x = red[0];
    for (int w = 1; w < kDisWaves; ++w) x = Op::join(x, red[w]);
    return x;
}

__device__ inline bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

template <bool BF16>
__device__ inline void store_elem(void* row, long long v, float x) {
    if constexpr (BF16) static_cast<__bf16*>(row)[v] = static_cast<__bf16>(x);
    else static_cast<float*>(row)[v] = x;
}

// What a workgroup knows of its row's record: this thread's entry (threads
// below K) and the sums over all.
struct Record {
    int tok;                     // -1: none
    float p, logp;               // the entry's probability
    float p_rest, logp_rest;     // the rest's (0 without a bucket)
    float P;                     // sum of all of them
    bool ok;                     // there is a probability
};

__device__ inline Record load_record(const DistillArgs& a, long long rec, DistillScratch& sc) {
    const int tid = threadIdx.x;
    Record r;
    r.tok = -1;
    float t = -kInf;
    bool bad = false;
    if (tid < a.K) {
        const int v = a.tok[rec * a.K + tid];
        if (v >= 0 && v < a.V) {
            r.tok = v;
            t = a.val[rec * a.K + tid] * a.inv_t;
            bad = !(t <= 3.402823466e38f);
        }
    }
    float lse = 0.f;
    r.p_rest = 0.f;
    r.logp_rest = -kInf;
    if (a.bucket) {
        lse = a.tlse[rec * 2];
        r.logp_rest = a.tlse[rec * 2 + 1] - lse;
        r.p_rest = expf(r.logp_rest);
        bad = bad || !finite(lse) || !finite(r.p_rest);
    } else {
        const float m = block_reduce<BlockMax>(t, sc.red);
        const float e = t == -kInf ? 0.f : expf(t - m);
        lse = m + logf(block_reduce<BlockSum>(e, sc.red2));
    }
    r.logp = t - lse;
    r.p = t == -kInf ? 0.f : expf(r.logp);
    const float sum = block_reduce<BlockSum>(r.p, sc.red);
    r.P = sum + r.p_rest;
    r.ok = !__syncthreads_or(bad) && r.P > 0.f && finite(r.P);
    if (tid < a.K) {
        sc.tok[tid] = r.tok;
        sc.p[tid] = r.p;
    }
    __syncthreads();
    return r;
}

// This thread's entry is the first of its token; ``p`` then gets the sum of
// all its entries.
__device__ inline bool first_entry(const DistillArgs& a, const Record& r, const DistillScratch& sc, float& p) {
    if (r.tok < 0) return false;
    p = 0.f;
    bool first = true;
    for (int k = 0; k < a.K; ++k)
        if (sc.tok[k] == r.tok) {
            if (k < (int)threadIdx.x) first = false;
            p += sc.p[k];
        }
    return first;
}

template <bool BF16, int OP>
__global__ __launch_bounds__(kDisBlock) void k_distill(DistillArgs a) {
    __shared__ DistillScratch sc;
    extern __shared__ unsigned inside[];          // one bit per token: in S
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.n, i = blockIdx.x % a.n;
    const void* row = row_ptr<BF16>(a.in, a.sb, a.sp, b, i);
    void* grow = OP == kDistillLoss ? nullptr : const_cast<void*>(row_ptr<BF16>(a.grad, a.g_sb, a.g_sp, b, i));
    const float w = a.w ? a.w[blockIdx.x] : 1.f;
    const Record r = load_record(a, (long long)b * a.rec_sb + i, sc);

    if (OP != kDistillLoss && (w == 0.f || !r.ok)) {
        for (int v = tid; v < a.V; v += kDisBlock) store_elem<BF16>(grow, v, 0.f);
        if (OP == kDistillLossGrad && tid == 0) {
            a.loss[blockIdx.x] = 0.f;
            if (a.flags) a.flags[blockIdx.x] = w == 0.f ? 0 : SPECV_FLAG_NONFINITE_ROW;
        }
        return;
    }
    float p_tok = 0.f;
    const bool first = first_entry(a, r, sc, p_tok);
    const float z_tok = r.tok >= 0 ? load_elem<BF16>(row, r.tok) : -kInf;

    float lse, lse_rest;
    if (OP == kDistillGrad) {
        lse = a.slse[(long long)blockIdx.x * 2];
        lse_rest = a.slse[(long long)blockIdx.x * 2 + 1];
    } else {
        const int words = (a.V + 31) / 32;
        for (int k = tid; k < words; k += kDisBlock) inside[k] = 0;
        __syncthreads();
        if (first) atomicOr(&inside[r.tok / 32], 1u << (r.tok % 32));
        __syncthreads();
        // the rest: running maximum and sum
        float m = -kInf, s = 0.f;
        unsigned bad = 0;
        for (int v = tid; v < a.V; v += kDisBlock) {
            const float x = load_elem<BF16>(row, v);
            bad |= !(x <= 3.402823466e38f);
            if ((inside[v / 32] >> (v % 32)) & 1) continue;
            if (x > m) {
                s *= fast_exp2((m - x) * a.scale);
                m = x;
            }
            if (x > -kInf) s += fast_exp2((x - m) * a.scale);
        }
        const float M = block_reduce<BlockMax>(m, sc.red);
        s = block_reduce<BlockSum>(m == -kInf ? 0.f : s * fast_exp2((m - M) * a.scale), sc.red2);
        lse_rest = M == -kInf ? -kInf : fmaf(M, a.inv_t, logf(s));
        // S
        const float MS = block_reduce<BlockMax>(z_tok, sc.red);
        const float MA = fmaxf(M, MS);
        float sa = block_reduce<BlockSum>(first && z_tok > -kInf ? fast_exp2((z_tok - MA) * a.scale) : 0.f, sc.red2);
        if (M > -kInf) sa += s * fast_exp2((M - MA) * a.scale);
        lse = fmaf(MA, a.inv_t, logf(sa));
        if (__syncthreads_or(bad) || MA == -kInf) lse = lse_rest = __builtin_nanf("");
        const float term = r.p > 0.f ? r.p * (r.logp - (z_tok * a.inv_t - lse)) : 0.f;
        float kl = block_reduce<BlockSum>(term, sc.red);
        if (r.p_rest > 0.f) kl += r.p_rest * (r.logp_rest - (lse_rest - lse));
        if (tid == 0) {
            a.loss[blockIdx.x] = w == 0.f || !r.ok ? 0.f : w * kl;
            if (OP == kDistillLoss) {
                a.lse[(long long)blockIdx.x * 2] = lse;
                a.lse[(long long)blockIdx.x * 2 + 1] = lse_rest;
            }
            if (a.flags) a.flags[blockIdx.x] = r.ok && lse == lse ? 0 : SPECV_FLAG_NONFINITE_ROW;
        }
    }
    if (OP == kDistillLoss) return;

    // gradient: the whole row by the rest's formula, then S over it
    __syncthreads();                              // (in place) every logit of S has been read
    const float g = w * a.inv_t;
    for (int v = tid; v < a.V; v += kDisBlock) {
        const float x = load_elem<BF16>(row, v) * a.inv_t;
        float d = r.P * expf(x - lse);
        if (r.p_rest > 0.f && lse_rest != -kInf) d -= r.p_rest * expf(x - lse_rest);
        store_elem<BF16>(grow, v, g * d);
    }
    __syncthreads();
    if (first) store_elem<BF16>(grow, r.tok, g * (r.P * expf(z_tok * a.inv_t - lse) - p_tok));
}

template <bool BF16>
void (*pick(DistillOp op))(DistillArgs) {
    if (op == kDistillLoss) return k_distill<BF16, kDistillLoss>;
    if (op == kDistillGrad) return k_distill<BF16, kDistillGrad>;
    return k_distill<BF16, kDistillLossGrad>;
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, DistillOp op, bool bf16, hipStream_t stream, hipEvent_t* ev) {
    const long long rows = (long long)a.B * a.n;
    auto fn = bf16 ? pick<true>(op) : pick<false>(op);
    const size_t lds = op == kDistillGrad ? 0 : (size_t)((a.V + 31) / 32) * 4;    // at most 64 KB
    if (ev)
        hipExtLaunchKernelGGL(fn, dim3((unsigned)rows), dim3(kDisBlock), lds, stream, ev[0], ev[1], 0, a);
    else
        hipLaunchKernelGGL(fn, dim3((unsigned)rows), dim3(kDisBlock), lds, stream, a);
    return hipGetLastError();
}

}  // namespace specv
