// specv_distill_loss / _grad / _loss_grad: the distillation loss of student
// rows against a teacher's record, and its gradient.
//
// With x_v = z_v / T, S the record's tokens, and L, L_o the log-sum-exps of x
// over the whole row and over the tokens outside S:
//   log q_v = x_v - L,  log q_o = L_o - L
//   d loss / d z_v = w / T * (P q_v - p_v)                          v in S
//                    w / T * (P exp(x_v - L) - p_o exp(x_v - L_o))  otherwise
//                  = c exp(x_v - L_o),  c = w / T * (P exp(L_o - L) - p_o)
// so outside S a row takes one exponential per logit and one factor.  The
// tokens of S are marked in a bit row in LDS, so that the sum over the rest
// is a sum of its own (as a difference of sums it would lose what is left of
// a student that has learned S); S itself is summed from its K gathered
// logits, by one wave, which also takes the teacher's side.

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specv_device.hpp"

namespace specv {
namespace {

constexpr int kMaxK = SPECV_MAX_RECORD_K;
constexpr int kE = kMaxK / kWave;                // record entries per lane of the wave that takes them
constexpr int kMaxWaves = 16;

struct DistillScratch {
    int tok[kMaxK];              // the record's tokens; -1: ignored
    float t[kMaxK];              // the teacher's logits / T
    float p[kMaxK];              // the teacher's probabilities (0 where ignored)
    float z[kMaxK];              // the student's logits
    int rep[kMaxK];              // the entry stands for its token (others of the same do not)
    float red[kMaxWaves], red2[kMaxWaves];
    float P, p_rest;             // the teacher's sum and rest
    float m_s, s_s;              // the student's maximum and sum over S
    int twice;                   // a token comes more than once
    int ok, bad;                 // there is a probability; a logit of S is NaN or +inf
};

__device__ inline bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// (m, s) statistics joined across the wave.
__device__ inline void wave_join_ms(float& m, float& s, float scale) {
    const float M = wave_max(m);
    s = wave_sum(m == -kInf ? 0.f : s * fast_exp2((m - M) * scale));
    m = M;
}

// The record's entries, lane l of one wave taking l, l + 64, ..
struct Entries {
    int tok[kE];
    float t[kE];
};

__device__ inline void issue_entries(const DistillArgs& a, long long rec, Entries& r) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        r.tok[u] = -1;
        r.t[u] = -kInf;
        const int k = lane + u * kWave;
        if (k < a.K) {
            r.tok[u] = a.tok[rec * a.K + k];
            r.t[u] = a.val[rec * a.K + k];
        }
    }
}
__device__ inline void finish_entries(const DistillArgs& a, Entries& r) {
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        if (r.tok[u] < 0 || r.tok[u] >= a.V) {
            r.tok[u] = -1;
            r.t[u] = -kInf;
        }
        r.t[u] *= a.inv_t;
    }
}

// The teacher's side, in one wave: the probabilities of the entries (sc.p)
// and of the rest.
struct Teacher {
    float P, p_rest, logp_rest;
    bool ok;
    float m, lse;                // log p_j = (t_j - m) - lse
};

__device__ inline Teacher take_teacher(const DistillArgs& a, long long rec, DistillScratch& sc) {
    const int lane = threadIdx.x % kWave;
    Teacher r;
    bool bad = false;
    float m = -kInf;
    for (int k = lane; k < a.K; k += kWave) {
        const float t = sc.t[k];
        bad |= !(t <= 3.402823466e38f);
        m = fmaxf(m, t);
    }
    r.lse = 0.f;
    r.p_rest = 0.f;
    r.logp_rest = -kInf;
    if (a.bucket) {
        r.m = a.tlse[rec * 2];
        r.logp_rest = a.tlse[rec * 2 + 1] - r.m;
        r.p_rest = expf(r.logp_rest);
        bad |= !finite(r.m) || !finite(r.p_rest);
    } else {
        r.m = wave_max(m);
        float e = 0.f;
        for (int k = lane; k < a.K; k += kWave) e += sc.t[k] == -kInf ? 0.f : expf(sc.t[k] - r.m);
        r.lse = logf(wave_sum(e));               // relative to m, as the logits
    }
    float sum = 0.f;
    for (int k = lane; k < a.K; k += kWave) {
        const float p = sc.t[k] == -kInf ? 0.f : expf((sc.t[k] - r.m) - r.lse);
        sc.p[k] = p;
        sum += p;
    }
    r.P = wave_sum(sum) + r.p_rest;
    r.ok = __ballot(bad) == 0 && r.P > 0.f && finite(r.P);
    return r;
}

// The sum of the probabilities of all entries of token t.
__device__ inline float token_p(const DistillArgs& a, const DistillScratch& sc, int t) {
    float p = 0.f;
    for (int k = 0; k < a.K; ++k) p += sc.tok[k] == t ? sc.p[k] : 0.f;
    return p;
}

// Statistics of G entries, those of S (bits of ``in``) left out.
template <bool BF16>
__device__ __forceinline__ void leave_out(RowGroup<BF16>& r, unsigned in) {
    constexpr int G = RowGroup<BF16>::G;
#pragma unroll
    for (int e = 0; e < G; ++e) {
        if (!((in >> e) & 1)) continue;
        if constexpr (BF16) r.q[e / 2] = (e & 1) ? ((r.q[e / 2] & 0xFFFFu) | 0xFF800000u) : ((r.q[e / 2] & 0xFFFF0000u) | 0xFF80u);
        else r.q[e] = 0xFF800000u;
    }
}

// A group's gradient outside S: c exp2((x - ref) scale), or 0 for a row left
// out (whose logits may be anything).
template <typename Group>
__device__ __forceinline__ Group grad_group(Group& x, const ExpRef& er, float c, bool on) {
    float y[Group::G];
    const float cf = c * er.fix;
    x.pin();
#pragma unroll
    for (int e = 0; e < Group::G; ++e) y[e] = er.fast(x.elem(e)) * cf;
    if (__builtin_expect(er.step || !on, 0)) {
        x.pin();
#pragma unroll
        for (int e = 0; e < Group::G; ++e) y[e] = on ? er.at_step(x.elem(e)) * c : 0.f;
    }
    Group o;
    o.pack(y);
    return o;
}

// The bits of group g's tokens.
template <bool BF16>
__device__ inline unsigned group_bits(const unsigned* inside, int g) {
    if constexpr (BF16) return reinterpret_cast<const unsigned char*>(inside)[g];
    else return (reinterpret_cast<const unsigned char*>(inside)[g / 2] >> (4 * (g & 1))) & 0xF;
}

// One row by one workgroup of NT threads.  The first NG groups of a thread
// stay in registers between the sums and the gradient; a longer row's others
// are read again (the loss alone holds none).
// Streamed groups are loaded LD at a time.
template <bool BF16, int NT, int NG, int LD, int MW, int OP>
__global__ __launch_bounds__(NT, MW) void k_distill(DistillArgs a) {
    constexpr int G = RowGroup<BF16>::G, NW = NT / kWave;
    __shared__ DistillScratch sc;
    extern __shared__ unsigned inside[];          // one bit per token: in S
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int b = blockIdx.x / a.n, i = blockIdx.x % a.n;
    const void* row = row_ptr<BF16>(a.in, a.sb, a.sp, b, i);
    void* grow = OP == kDistillLoss ? nullptr : const_cast<void*>(row_ptr<BF16>(a.grad, a.g_sb, a.g_sp, b, i));
    const long long rec = (long long)b * a.rec_sb + i;
    const float w = a.w ? a.w[blockIdx.x] : 1.f;
    const int full = a.V / G;

    if (OP == kDistillLossGrad && w == 0.f) {
        RowGroup<BF16> zero;
        zero.q = u32x4{0, 0, 0, 0};
        for (int g = tid; g < full; g += NT) zero.store(grow, g);
        for (int v = full * G + tid; v < a.V; v += NT) store_elem<BF16>(grow, v, 0.f);
        if (tid == 0) {
            a.loss[blockIdx.x] = 0.f;
            if (a.flags) a.flags[blockIdx.x] = 0;
        }
        return;
    }

    Entries r;
    if (wave == 0) issue_entries(a, rec, r);
    RowGroup<BF16> h[NG > 0 ? NG : 1];
    if constexpr (NG > 0) {
#pragma unroll
        for (int j = 0; j < NG; ++j) h[j].issue(row, j * NT + tid, full);
    }
    for (int k = tid; k < (a.V + 31) / 32; k += NT) inside[k] = 0;
    if (tid == 0) sc.twice = 0;
    __syncthreads();
    if (wave == 0) {
        finish_entries(a, r);
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int k = lane + u * kWave;
            if (k >= a.K) continue;
            int rep = 0;
            float z = -kInf;
            if (r.tok[u] >= 0) {
                const unsigned bit = 1u << (r.tok[u] % 32);
                rep = !(atomicOr(&inside[r.tok[u] / 32], bit) & bit);
                if (!rep) sc.twice = 1;
                z = load_elem<BF16>(row, r.tok[u]);
            }
            sc.tok[k] = r.tok[u];
            sc.t[k] = r.t[u];
            sc.rep[k] = rep;
            sc.z[k] = z;
        }
    }
    __syncthreads();

    // the rest's maximum and sum
    float m = -kInf, s = 0.f;
    if constexpr (NG > 0) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int g = j * NT + tid;
            if ((j + 1) * NT > full) h[j].clear(g, full);
            const unsigned in = g < full ? group_bits<BF16>(inside, g) : 0;
            if (__ballot(in != 0)) leave_out<BF16>(h[j], in);    // for good: S is written over the rest at the end
#pragma unroll
            for (int e = 0; e < G; ++e) m = fmaxf(m, h[j].elem(e));
        }
        s = sum_exp<NG>(h, ExpRef(m, a.scale));
    }
    if (NG * NT < full) {
        RowGroup<BF16> nx[LD], x[LD];
#pragma unroll
        for (int l = 0; l < LD; ++l) nx[l].issue(row, (NG + l) * NT + tid, full);
        for (int j = NG; j * NT < full; j += LD) {
#pragma unroll
            for (int l = 0; l < LD; ++l) x[l] = nx[l];
            if ((j + LD) * NT < full) {
#pragma unroll
                for (int l = 0; l < LD; ++l) nx[l].issue(row, (j + LD + l) * NT + tid, full);
            }
            float gm = -kInf;
#pragma unroll
            for (int l = 0; l < LD; ++l) {
                const int g = (j + l) * NT + tid;
                x[l].clear(g, full);
                const unsigned in = g < full ? group_bits<BF16>(inside, g) : 0;
                if (__ballot(in != 0)) leave_out<BF16>(x[l], in);
#pragma unroll
                for (int e = 0; e < G; ++e) gm = fmaxf(gm, x[l].elem(e));
            }
            const float gs = sum_exp<LD>(x, ExpRef(gm, a.scale));
            merge_ms(m, s, gm, gs, a.scale);
        }
    }
    bool bad = s != s;                             // NaN or +inf among them
    if (tid == 0) {
        for (int v = full * G; v < a.V; ++v) {     // the row's last, partial group
            if ((inside[v / 32] >> (v % 32)) & 1) continue;
            const float x = load_elem<BF16>(row, v);
            bad |= !(x <= 3.402823466e38f);
            merge_ms(m, s, x, x == -kInf ? 0.f : 1.f, a.scale);
        }
    }
    if (bad) s = __builtin_nanf("");
    wave_join_ms(m, s, a.scale);
    if (__ballot(bad)) s = __builtin_nanf("");
    if (lane == 0) {
        sc.red[wave] = m;
        sc.red2[wave] = s;
    }
    Teacher t{};
    if (wave == 0) {
        t = take_teacher(a, rec, sc);
        float ms = -kInf, ss = 0.f;
        bool bad_s = false;
        for (int k = lane; k < a.K; k += kWave) {
            ms = fmaxf(ms, sc.z[k]);
            bad_s |= !(sc.z[k] <= 3.402823466e38f);
        }
        ms = wave_max(ms);
        for (int k = lane; k < a.K; k += kWave)
            if (sc.rep[k] && sc.z[k] > -kInf) ss += fast_exp2((sc.z[k] - ms) * a.scale);
        ss = wave_sum(ss);
        bad_s = __ballot(bad_s) != 0;
        if (lane == 0) {
            sc.P = t.P;
            sc.p_rest = t.p_rest;
            sc.m_s = ms;
            sc.s_s = ss;
            sc.ok = t.ok;
            sc.bad = bad_s;
        }
    }
    __syncthreads();
    m = lane < NW ? sc.red[lane] : -kInf;
    s = lane < NW ? sc.red2[lane] : 0.f;
    bad = __ballot(s != s) != 0 || sc.bad;
    wave_join_ms(m, s, a.scale);
    const float m_all = fmaxf(m, sc.m_s);
    bad |= m_all == -kInf;
    float s_all = sc.s_s > 0.f ? sc.s_s * fast_exp2((sc.m_s - m_all) * a.scale) : 0.f;
    const float share = m == -kInf ? 0.f : fast_exp2((m - m_all) * a.scale);
    s_all += s * share;

    if (OP != kDistillLoss) {
        // the gradient: the whole row by the rest's formula, then S over it
        float c = 0.f;
        const ExpRef er(m, a.scale);
        const float gw = w * a.inv_t;
        if (sc.ok) {
            if (m > -kInf) c = gw * (sc.P * share / s_all - sc.p_rest / s);
            if (bad) c = __builtin_nanf("");
        }
        if constexpr (NG > 0) {
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int g = j * NT + tid;
                const RowGroup<BF16> o = grad_group(h[j], er, c, sc.ok != 0);
                if (g < full) o.store(grow, g);
            }
        }
        for (int g = NG * NT + tid; g < full; g += NT) {
            RowGroup<BF16> x;
            x.issue(row, g, full);
            grad_group(x, er, c, sc.ok != 0).store(grow, g);
        }
        if (tid == 0) {
            for (int v = full * G; v < a.V; ++v) {
                const float y = sc.ok ? er.any(load_elem<BF16>(row, v)) * c : 0.f;
                store_elem<BF16>(grow, v, y);
            }
        }
        __syncthreads();
        if (wave == 0 && sc.ok) {
            for (int k = lane; k < a.K; k += kWave) {
                if (!sc.rep[k]) continue;
                const float p = sc.twice ? token_p(a, sc, sc.tok[k]) : sc.p[k];
                float y = gw * (sc.P * fast_exp2((sc.z[k] - m_all) * a.scale) / s_all - p);
                if (bad) y = __builtin_nanf("");
                store_elem<BF16>(grow, sc.tok[k], y);
            }
        }
    }
    if (wave == 0) {
        const float log_all = logf(s_all);
        float kl = 0.f;
        for (int k = lane; k < a.K; k += kWave)
            if (sc.p[k] > 0.f)
                kl += sc.p[k] * (((sc.t[k] - t.m) - t.lse) - ((sc.z[k] - m_all) * a.inv_t - log_all));
        kl = wave_sum(kl);
        if (t.p_rest > 0.f) {
            const float logq = m == -kInf ? -kInf : (m - m_all) * a.inv_t + (logf(s) - log_all);
            kl += t.p_rest * (t.logp_rest - logq);
        }
        if (lane == 0) {
            const float nan = __builtin_nanf("");
            a.loss[blockIdx.x] = w == 0.f || !t.ok ? 0.f : bad ? nan : w * kl;
            if (OP == kDistillLoss) {
                a.lse[(long long)blockIdx.x * 2] = bad ? nan : fmaf(m_all, a.inv_t, log_all);
                a.lse[(long long)blockIdx.x * 2 + 1] =
                    bad ? nan : m == -kInf ? -kInf : fmaf(m, a.inv_t, logf(s));
            }
            if (a.flags) a.flags[blockIdx.x] = t.ok && !bad ? 0 : SPECV_FLAG_NONFINITE_ROW;
        }
    }
}

// The gradient from given log-sum-exps: a part of a row, kGradLoads groups a
// thread, per workgroup.  Its logits are on their way while one wave takes
// the record; the tokens of S inside the part are written over it at the end.
constexpr int kGradLoads = 4;

template <bool BF16>
__global__ __launch_bounds__(kBlock) void k_distill_grad(DistillArgs a, int parts) {
    constexpr int G = RowGroup<BF16>::G;
    constexpr int kPart = kBlock * kGradLoads * G; // tokens of a part
    __shared__ DistillScratch sc;
    __shared__ unsigned mark[kPart / 32];          // tokens of S seen so far
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const long long ri = blockIdx.x / parts;
    const int part = blockIdx.x % parts;
    const int b = (int)(ri / a.n), i = (int)(ri % a.n);
    const void* row = row_ptr<BF16>(a.in, a.sb, a.sp, b, i);
    void* grow = const_cast<void*>(row_ptr<BF16>(a.grad, a.g_sb, a.g_sp, b, i));
    const float w = a.w ? a.w[ri] : 1.f;
    const int full = a.V / G, g0 = part * kBlock * kGradLoads;
    const int v0 = part * kPart, v1 = min(v0 + kPart, a.V);

    const long long rec = (long long)b * a.rec_sb + i;
    const float lse = a.slse[ri * 2], lse_rest = a.slse[ri * 2 + 1];
    Entries r;
    RowGroup<BF16> h[kGradLoads];
    if (w != 0.f) {
        if (wave == 0) issue_entries(a, rec, r);
#pragma unroll
        for (int l = 0; l < kGradLoads; ++l) h[l].issue(row, g0 + l * kBlock + tid, full);
    }
    for (int k = tid; k < kPart / 32; k += kBlock) mark[k] = 0;
    if (tid == 0) sc.twice = 0;
    __syncthreads();
    if (wave == 0 && w != 0.f) {
        finish_entries(a, r);
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int k = lane + u * kWave;
            if (k >= a.K) continue;
            const int t = r.tok[u];
            sc.tok[k] = t;
            sc.t[k] = r.t[u];
            if (t >= v0 && t < v1) {
                const unsigned bit = 1u << (t % 32);
                if (atomicOr(&mark[(t - v0) / 32], bit) & bit) sc.twice = 1;
                sc.z[k] = load_elem<BF16>(row, t);
            }
        }
        const Teacher t = take_teacher(a, rec, sc);
        if (lane == 0) {
            sc.P = t.P;
            sc.p_rest = t.p_rest;
            sc.ok = t.ok;
        }
    }
    __syncthreads();                                // (in place) this part's logits of S have been read
    const bool on = w != 0.f && sc.ok;
    const float gw = w * a.inv_t;
    float c = 0.f, ref = 0.f;
    if (on && lse_rest != -kInf) {
        c = gw * (sc.P * expf(lse_rest - lse) - sc.p_rest);
        ref = lse_rest / a.inv_t;
    }
    if (on && lse != lse) c = __builtin_nanf("");
    const ExpRef er(ref, a.scale);
#pragma unroll
    for (int l = 0; l < kGradLoads; ++l) {
        const int g = g0 + l * kBlock + tid;
        if (g < full) grad_group(h[l], er, c, on).store(grow, g);
    }
    for (int v = max(full * G, v0) + tid; v < v1; v += kBlock)               // the row's last, partial group
        store_elem<BF16>(grow, v, on ? er.any(load_elem<BF16>(row, v)) * c : 0.f);
    __syncthreads();
    if (wave == 0 && on) {
        for (int k = lane; k < a.K; k += kWave) {
            if (sc.tok[k] < v0 || sc.tok[k] >= v1) continue;
            const float p = sc.twice ? token_p(a, sc, sc.tok[k]) : sc.p[k];     // (entries of one token write the same)
            store_elem<BF16>(grow, sc.tok[k], gw * (sc.P * expf(sc.z[k] * a.inv_t - lse) - p));
        }
    }
}

template <typename... A>
hipError_t launch(void (*fn)(A...), long long blocks, int threads, size_t lds, hipStream_t stream, hipEvent_t* ev,
                  A... args) {
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    if (ev)
        hipExtLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), lds, stream, ev[0], ev[1], 0, args...);
    else
        hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), lds, stream, args...);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_rows(const DistillArgs& a, DistillOp op, hipStream_t stream, hipEvent_t* ev) {
    constexpr int G = RowGroup<BF16>::G;
    const long long rows = (long long)a.B * a.n;
    if (op == kDistillGrad) {
        const int per = kBlock * kGradLoads * G, parts = (a.V + per - 1) / per;
        return launch(k_distill_grad<BF16>, rows * parts, kBlock, 0, stream, ev, a, parts);
    }
    const size_t lds = (size_t)((a.V + 31) / 32) * 4;    // at most 64 KB
    if (op == kDistillLoss) return launch(k_distill<BF16, 512, 0, 4, 4, kDistillLoss>, rows, 512, lds, stream, ev, a);
    const int full = a.V / G;
#define SPECV_ROWS(NG, LD, MW) launch(k_distill<BF16, 1024, NG, LD, MW, kDistillLossGrad>, rows, 1024, lds, stream, ev, a)
    if (full <= 4 * 1024) return SPECV_ROWS(4, 2, 8);
    if constexpr (BF16) return SPECV_ROWS(6, 2, 8);
    else return full <= 16 * 1024 ? SPECV_ROWS(16, 4, 4) : SPECV_ROWS(20, 4, 4);
#undef SPECV_ROWS
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, DistillOp op, bool bf16, hipStream_t stream, hipEvent_t* ev) {
    return bf16 ? launch_rows<true>(a, op, stream, ev) : launch_rows<false>(a, op, stream, ev);
}

}  // namespace specv
