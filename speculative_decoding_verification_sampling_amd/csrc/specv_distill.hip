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
// logits.
//
// Bound by memory for many rows: loss and gradient of 2048 rows of 128256
// bfloat16 logits take 198 us for 1.05 GB read and written (5.3 TB/s; with the
// part that is read twice the device moves 1.2 GB); the gradient alone 171 us
// (6.1 TB/s), the loss alone 97 us for 525 MB (5.4 TB/s).  320 rows: 41 us and
// 25 us; a fifth of the CUs then hold two rows and the others wait.

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specv_logits_device.hpp"

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

// Of entries with one token the first alone stands for it, whichever of them an
// atomic has picked: sums over S then run in one order.  (Records rarely hold
// a token twice; one wave.)
__device__ inline void first_stands(const DistillArgs& a, const Entries& r, int (&rep)[kE]) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int u = 0; u < kE; ++u) rep[u] = r.tok[u] >= 0;
#pragma unroll
    for (int q = 0; q < kE; ++q) {
        const int left = min(kWave, a.K - q * kWave);
        for (int l = 0; l < left; ++l) {
            const int t = __builtin_amdgcn_readlane(r.tok[q], l);
#pragma unroll
            for (int u = 0; u < kE; ++u)
                if (r.tok[u] == t && u * kWave + lane > q * kWave + l) rep[u] = 0;
        }
    }
}

// The student's logits of the entries whose token lies in [v0, v1), -inf for
// the others: all loads first, so that they wait once.
template <bool BF16>
__device__ inline void load_logits(const void* row, const Entries& r, int v0, int v1, float (&z)[kE]) {
    unsigned raw[kE];
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        raw[u] = BF16 ? 0xFF80u : 0xFF800000u;
        if (r.tok[u] >= v0 && r.tok[u] < v1) {
            if constexpr (BF16) raw[u] = static_cast<const unsigned short*>(row)[r.tok[u]];
            else raw[u] = static_cast<const unsigned*>(row)[r.tok[u]];
        }
    }
#pragma unroll
    for (int u = 0; u < kE; ++u) z[u] = __uint_as_float(BF16 ? raw[u] << 16 : raw[u]);
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

// The student's maximum and sum over S (sc.z, sc.rep), in one wave; returns
// whether one of them is NaN or +inf.
__device__ inline bool take_student(const DistillArgs& a, const DistillScratch& sc, float& m, float& s) {
    const int lane = threadIdx.x % kWave;
    m = -kInf;
    s = 0.f;
    bool bad = false;
    for (int k = lane; k < a.K; k += kWave) {
        m = fmaxf(m, sc.z[k]);
        bad |= !(sc.z[k] <= 3.402823466e38f);
    }
    m = wave_max(m);
    for (int k = lane; k < a.K; k += kWave)
        if (sc.rep[k] && sc.z[k] > -kInf) s += fast_exp2((sc.z[k] - m) * a.scale);
    s = wave_sum(s);
    return __ballot(bad) != 0;
}

// The row's loss, log-sum-exps and flags, by one wave; (m, s) of the rest and
// (m_all, s_all) of the row.
template <int OP>
__device__ inline void write_row(const DistillArgs& a, const DistillScratch& sc, const Teacher& t, long long ri,
                                 float w, float m, float s, float m_all, float s_all, bool bad) {
    const int lane = threadIdx.x % kWave;
    const float log_all = logf(s_all);
    float kl = 0.f;
    for (int k = lane; k < a.K; k += kWave)
        if (sc.p[k] > 0.f) kl += sc.p[k] * (((sc.t[k] - t.m) - t.lse) - ((sc.z[k] - m_all) * a.inv_t - log_all));
    kl = wave_sum(kl);
    if (t.p_rest > 0.f) {
        const float logq = m == -kInf ? -kInf : (m - m_all) * a.inv_t + (logf(s) - log_all);
        kl += t.p_rest * (t.logp_rest - logq);
    }
    if (lane == 0) {
        const float nan = __builtin_nanf("");
        a.loss[ri] = w == 0.f || !t.ok ? 0.f : bad ? nan : w * kl;
        if (OP == kDistillLoss) {
            a.lse[ri * 2] = bad ? nan : fmaf(m_all, a.inv_t, log_all);
            a.lse[ri * 2 + 1] = bad ? nan : m == -kInf ? -kInf : fmaf(m, a.inv_t, logf(s));
        }
        if (a.flags) a.flags[ri] = t.ok && !bad ? 0 : SPECV_FLAG_NONFINITE_ROW;
    }
}

// The sum of the probabilities of all entries of token t.
__device__ inline float token_p(const DistillArgs& a, const DistillScratch& sc, int t) {
    float p = 0.f;
    for (int k = 0; k < a.K; ++k) p += sc.tok[k] == t ? sc.p[k] : 0.f;
    return p;
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
// are read again (the loss alone holds none).  Bfloat16 rows longer than
// 32768 hold 6 of (V / 8192) groups a thread in 64 registers, two workgroups
// per CU, one reading while the other computes: 2048 rows of 128256 took
// 234 us so, 248 with all groups held (128 registers, one workgroup), 251
// with none; float32 rows, twice the bytes, 142 / 120 / 144 us (512 rows), so
// they hold what fits.
// Streamed groups are loaded LD at a time; PAST: loads that are a row's last
// go past the caches.
template <bool BF16, int NT, int NG, int LD, int MW, int OP, bool PAST>
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
        for (int j = 0; j < NG; ++j) h[j].template issue<PAST>(row, j * NT + tid, full);
    }
    for (int k = tid; k < (a.V + 31) / 32; k += NT) inside[k] = 0;
    if (tid == 0) sc.twice = 0;
    __syncthreads();
    float z[kE];
    if (wave == 0) {
        finish_entries(a, r);
        int rep[kE];
        bool twice = false;
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            rep[u] = 0;
            if (r.tok[u] >= 0) {
                const unsigned bit = 1u << (r.tok[u] % 32);
                rep[u] = !(atomicOr(&inside[r.tok[u] / 32], bit) & bit);
                twice |= !rep[u];
            }
        }
        if (__ballot(twice)) {
            first_stands(a, r, rep);
            if (lane == 0) sc.twice = 1;
        }
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int k = lane + u * kWave;
            if (k >= a.K) continue;
            sc.tok[k] = r.tok[u];
            sc.t[k] = r.t[u];
            sc.rep[k] = rep[u];
        }
        load_logits<BF16>(row, r, 0, a.V, z);
#pragma unroll
        for (int u = 0; u < kE; ++u)
            if (lane + u * kWave < a.K) sc.z[lane + u * kWave] = z[u];
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
            if (__ballot(in != 0)) leave_out(h[j], in);    // for good: S is written over the rest at the end
#pragma unroll
            for (int e = 0; e < G; ++e) m = fmaxf(m, h[j].elem(e));
        }
        s = sum_exp<NG>(h, ExpRef(m, a.scale));
    }
    if (NG * NT < full) {
        RowGroup<BF16> nx[LD], x[LD];
#pragma unroll
        for (int l = 0; l < LD; ++l) nx[l].template issue<PAST && OP == kDistillLoss>(row, (NG + l) * NT + tid, full);
        for (int j = NG; j * NT < full; j += LD) {
#pragma unroll
            for (int l = 0; l < LD; ++l) x[l] = nx[l];
            if ((j + LD) * NT < full) {
#pragma unroll
                for (int l = 0; l < LD; ++l) nx[l].template issue<PAST && OP == kDistillLoss>(row, (j + LD + l) * NT + tid, full);
            }
            float gm = -kInf;
#pragma unroll
            for (int l = 0; l < LD; ++l) {
                const int g = (j + l) * NT + tid;
                x[l].clear(g, full);
                const unsigned in = g < full ? group_bits<BF16>(inside, g) : 0;
                if (__ballot(in != 0)) leave_out(x[l], in);
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
        if (lane == 0) {
            sc.P = t.P;
            sc.p_rest = t.p_rest;
            sc.ok = t.ok;
        }
    } else if (wave == 1) {
        float ms, ss;
        const bool bad_s = take_student(a, sc, ms, ss);
        if (lane == 0) {
            sc.m_s = ms;
            sc.s_s = ss;
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
            x.template issue<PAST>(row, g, full);
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
        write_row<OP>(a, sc, t, blockIdx.x, w, m, s, m_all, s_all, bad);
    }
}

// Rows in parts, kPartLoads groups a thread of kBlock threads each.  Where a
// call's rows are few, a workgroup per row leaves most CUs idle; parts do
// not, for a second read of the row and a second launch:
//   k_part_stats    the maximum and sum over each part's rest, and the
//                   student's logits of S, into the workspace;
//   k_part_loss     joins a row's parts (one wave): loss, log-sum-exps;
//   k_part_grad     the gradient of a part; every part joins the row's sums.
// k_part_grad without a workspace takes given log-sum-exps (the gradient
// alone).
constexpr int kPartLoads = 4;

template <bool BF16>
constexpr int kPart = kBlock * kPartLoads * RowGroup<BF16>::G;     // tokens of a part

template <bool BF16>
__global__ __launch_bounds__(kBlock) void k_part_stats(DistillArgs a, bool skip) {
    __shared__ unsigned mark[kPart<BF16> / 32];
    __shared__ float red[kWaves], red2[kWaves];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    constexpr int G = RowGroup<BF16>::G;
    const long long ri = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts;
    const int b = (int)(ri / a.n), i = (int)(ri % a.n);
    if (skip && a.w && a.w[ri] == 0.f) return;                      // nothing of this row is needed
    const void* row = row_ptr<BF16>(a.in, a.sb, a.sp, b, i);
    const int full = a.V / G, g0 = part * kBlock * kPartLoads;
    const int v0 = part * kPart<BF16>, v1 = min(v0 + kPart<BF16>, a.V);
    Entries r;
    if (wave == 0) issue_entries(a, (long long)b * a.rec_sb + i, r);
    RowGroup<BF16> h[kPartLoads];
#pragma unroll
    for (int l = 0; l < kPartLoads; ++l) h[l].issue(row, g0 + l * kBlock + tid, full);
    for (int k = tid; k < kPart<BF16> / 32; k += kBlock) mark[k] = 0;
    __syncthreads();
    float* z = a.zs + ri * 2 * a.K;
    if (wave == 0) {
        finish_entries(a, r);
        float x[kE];
        load_logits<BF16>(row, r, v0, v1, x);
        int rep[kE];
        bool twice = false;
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int t = r.tok[u];
            rep[u] = 0;
            if (t >= v0 && t < v1) {
                const unsigned bit = 1u << (t % 32);
                rep[u] = !(atomicOr(&mark[(t - v0) / 32], bit) & bit);
                twice |= !rep[u];
            }
        }
        if (__ballot(twice)) first_stands(a, r, rep);
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int k = lane + u * kWave, t = r.tok[u];
            if (k >= a.K) continue;
            if (t >= v0 && t < v1) {
                z[k] = x[u];
                z[a.K + k] = rep[u] ? 1.f : 0.f;
            } else if (t < 0 && part == 0) {
                z[k] = -kInf;
                z[a.K + k] = 0.f;
            }
        }
    }
    __syncthreads();
    float m = -kInf;
#pragma unroll
    for (int l = 0; l < kPartLoads; ++l) {
        const int g = g0 + l * kBlock + tid;
        h[l].clear(g, full);
        const unsigned in = g < full ? group_bits<BF16>(mark, g - g0) : 0;
        if (__ballot(in != 0)) leave_out(h[l], in);
#pragma unroll
        for (int e = 0; e < G; ++e) m = fmaxf(m, h[l].elem(e));
    }
    float s = sum_exp<kPartLoads>(h, ExpRef(m, a.scale));
    bool bad = s != s;
    if (tid == 0) {
        for (int v = max(full * G, v0); v < v1; ++v) {              // the row's last, partial group
            if ((mark[(v - v0) / 32] >> (v % 32)) & 1) continue;
            const float x = load_elem<BF16>(row, v);
            bad |= !(x <= 3.402823466e38f);
            merge_ms(m, s, x, x == -kInf ? 0.f : 1.f, a.scale);
        }
    }
    if (bad) s = 0.f;
    wave_join_ms(m, s, a.scale);
    if (__ballot(bad)) s = __builtin_nanf("");
    if (lane == 0) {
        red[wave] = m;
        red2[wave] = s;
    }
    __syncthreads();
    if (wave == 0) {
        m = lane < kWaves ? red[lane] : -kInf;
        s = lane < kWaves ? red2[lane] : 0.f;
        bad = __ballot(s != s) != 0;
        wave_join_ms(m, s, a.scale);
        if (lane == 0) a.part[ri * a.parts + part] = make_float2(m, bad ? __builtin_nanf("") : s);
    }
}

// The row's entries and parts, joined by one wave: sc, (m, s) of the rest and
// (m_all, s_all) of the row; returns whether the row has NaN, +inf or no
// finite logit.
__device__ inline bool join_parts(const DistillArgs& a, long long ri, long long rec, DistillScratch& sc, Teacher& t,
                                  float& m, float& s, float& m_all, float& s_all) {
    const int lane = threadIdx.x % kWave;
    Entries r;
    issue_entries(a, rec, r);
    const float* z = a.zs + ri * 2 * a.K;
    m = -kInf;
    s = 0.f;
    bool bad = false;
    for (int q = lane; q < a.parts; q += kWave) {
        const float2 p = a.part[ri * a.parts + q];
        bad |= p.y != p.y;
        merge_ms(m, s, p.x, p.y, a.scale);
    }
    finish_entries(a, r);
    bool twice = false;
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        const int k = lane + u * kWave;
        if (k >= a.K) continue;
        const bool rep = z[a.K + k] != 0.f;
        sc.tok[k] = r.tok[u];
        sc.t[k] = r.t[u];
        sc.z[k] = z[k];
        sc.rep[k] = rep;
        twice |= r.tok[u] >= 0 && !rep;
    }
    t = take_teacher(a, rec, sc);
    float ms, ss;
    bad |= take_student(a, sc, ms, ss);
    bad = __ballot(bad) != 0;
    if (bad) s = 0.f;
    wave_join_ms(m, s, a.scale);
    m_all = fmaxf(m, ms);
    s_all = ss > 0.f ? ss * fast_exp2((ms - m_all) * a.scale) : 0.f;
    if (m > -kInf) s_all += s * fast_exp2((m - m_all) * a.scale);
    if (__ballot(twice) && lane == 0) sc.twice = 1;
    return bad || m_all == -kInf;
}

__global__ __launch_bounds__(kWave) void k_part_loss(DistillArgs a) {
    __shared__ DistillScratch sc;
    const long long ri = blockIdx.x;
    const long long rec = (ri / a.n) * a.rec_sb + ri % a.n;
    const float w = a.w ? a.w[ri] : 1.f;
    Teacher t;
    float m, s, m_all, s_all;
    const bool bad = join_parts(a, ri, rec, sc, t, m, s, m_all, s_all);
    write_row<kDistillLoss>(a, sc, t, ri, w, m, s, m_all, s_all, bad);
}

template <bool BF16, bool JOIN, bool PAST>
__global__ __launch_bounds__(kBlock) void k_part_grad(DistillArgs a) {
    constexpr int G = RowGroup<BF16>::G;
    __shared__ DistillScratch sc;
    __shared__ unsigned mark[JOIN ? 1 : kPart<BF16> / 32];           // tokens of S seen so far
    __shared__ float coef[4];                                       // c, ref; factors of S: P / sum, reference
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const long long ri = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts;
    const int b = (int)(ri / a.n), i = (int)(ri % a.n);
    const void* row = row_ptr<BF16>(a.in, a.sb, a.sp, b, i);
    void* grow = const_cast<void*>(row_ptr<BF16>(a.grad, a.g_sb, a.g_sp, b, i));
    const float w = a.w ? a.w[ri] : 1.f, gw = w * a.inv_t;
    const int full = a.V / G, g0 = part * kBlock * kPartLoads;
    const int v0 = part * kPart<BF16>, v1 = min(v0 + kPart<BF16>, a.V);
    const long long rec = (long long)b * a.rec_sb + i;

    Entries r;
    RowGroup<BF16> h[kPartLoads];
    if (w != 0.f) {
        if (!JOIN && wave == 0) issue_entries(a, rec, r);
#pragma unroll
        for (int l = 0; l < kPartLoads; ++l) h[l].template issue<PAST>(row, g0 + l * kBlock + tid, full);
    }
    if (!JOIN)
        for (int k = tid; k < kPart<BF16> / 32; k += kBlock) mark[k] = 0;
    if (tid == 0) {
        sc.twice = 0;
        sc.ok = 0;
    }
    __syncthreads();
    if (wave == 0 && w != 0.f) {
        Teacher t;
        float c = 0.f, ref = 0.f, fs, rs;
        bool bad;
        if constexpr (JOIN) {
            float m, s, m_all, s_all;
            bad = join_parts(a, ri, rec, sc, t, m, s, m_all, s_all);
            if (part == 0) write_row<kDistillLossGrad>(a, sc, t, ri, w, m, s, m_all, s_all, bad);
            if (m > -kInf) {
                c = gw * (t.P * fast_exp2((m - m_all) * a.scale) / s_all - t.p_rest / s);
                ref = m;
            }
            fs = t.P / s_all;
            rs = m_all;
        } else {
            finish_entries(a, r);
            float z[kE];
            load_logits<BF16>(row, r, v0, v1, z);
#pragma unroll
            for (int u = 0; u < kE; ++u) {
                const int k = lane + u * kWave, tk = r.tok[u];
                if (k >= a.K) continue;
                sc.tok[k] = tk;
                sc.t[k] = r.t[u];
                if (tk >= v0 && tk < v1) {
                    const unsigned bit = 1u << (tk % 32);
                    if (atomicOr(&mark[(tk - v0) / 32], bit) & bit) sc.twice = 1;
                    sc.z[k] = z[u];
                }
            }
            t = take_teacher(a, rec, sc);
            const float lse = a.slse[ri * 2], lse_rest = a.slse[ri * 2 + 1];
            if (lse_rest != -kInf) {
                c = gw * (t.P * expf(lse_rest - lse) - t.p_rest);
                ref = lse_rest / a.inv_t;
            }
            bad = lse != lse;
            fs = t.P;
            rs = lse / a.inv_t;
        }
        if (lane == 0) {
            sc.ok = t.ok;
            coef[0] = bad ? __builtin_nanf("") : c;
            coef[1] = ref;
            coef[2] = bad ? __builtin_nanf("") : fs;
            coef[3] = rs;
        }
    } else if (JOIN && wave == 0 && part == 0 && lane == 0) {
        a.loss[ri] = 0.f;
        if (a.flags) a.flags[ri] = 0;
    }
    __syncthreads();                                // (in place) this part's logits of S have been read
    const bool on = w != 0.f && sc.ok;
    const float c = on ? coef[0] : 0.f;
    const ExpRef er(on ? coef[1] : 0.f, a.scale);
#pragma unroll
    for (int l = 0; l < kPartLoads; ++l) {
        const int g = g0 + l * kBlock + tid;
        if (g < full) grad_group(h[l], er, c, on).store(grow, g);
    }
    for (int v = max(full * G, v0) + tid; v < v1; v += kBlock)      // the row's last, partial group
        store_elem<BF16>(grow, v, on ? er.any(load_elem<BF16>(row, v)) * c : 0.f);
    __syncthreads();
    if (wave == 0 && on) {
        for (int k = lane; k < a.K; k += kWave) {
            const int t = sc.tok[k];
            if (t < v0 || t >= v1) continue;
            const float p = sc.twice ? token_p(a, sc, t) : sc.p[k];   // (entries of one token write the same)
            store_elem<BF16>(grow, t, gw * (coef[2] * fast_exp2((sc.z[k] - coef[3]) * a.scale) - p));
        }
    }
}

// One launch, with the events of a profiled call (each may be nullptr).
template <typename... A>
hipError_t launch_with(void (*fn)(A...), long long blocks, int threads, size_t lds, hipStream_t stream,
                       hipEvent_t start, hipEvent_t stop, A... args) {
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    if (start || stop)
        hipExtLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), lds, stream, start, stop, 0, args...);
    else
        hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), lds, stream, args...);
    return hipGetLastError();
}
template <typename... A>
hipError_t launch(void (*fn)(A...), long long blocks, int threads, size_t lds, hipStream_t stream, hipEvent_t* ev,
                  A... args) {
    return launch_with(fn, blocks, threads, lds, stream, ev ? ev[0] : nullptr, ev ? ev[1] : nullptr, args...);
}

// Rows go in parts, when the caller gives a workspace, from this many parts a
// row on and up to this many rows.  distill_loss_grad / distill_loss, bfloat16,
// whole rows against parts, us:
//   V 128256 (16 parts):   1 row 20.0 / 13.5, 10.9 / 9.1;   16 rows 20.6 / 14.2, 11.4 / 10.0;
//                          64 rows 21.3 / 14.8, 16.1 / 13.0; 128 rows 22.6 / 15.6, 22.8 / 17.6
//   V 33000 (5 parts):     1 row 9.4 / 7.1, 10.7 / 8.9;     64 rows 10.3 / 7.9, 12.8 / 10.6
constexpr int kMinParts = 12;
constexpr long long kPartRows = 64;

// From this many bytes of logits on, loads that are a row's last go past the
// caches: the 256 MB last-level cache cannot hold the rows until anything
// reads them again.  distill_loss_grad of 2048 rows of 128256 bfloat16 logits
// (525 MB): 212 -> 198 us; distill_grad of 1024 rows of 32000 (66 MB), read
// back to back: 24.4 us, 27.8 with it.
constexpr long long kPastBytes = 256ll << 20;

// Threads by a row's 16-byte groups: four a thread or so, or the joins of idle
// waves cost more than the row (2048 rows, bfloat16, us with 256 / 512 / 1024
// threads: loss and gradient of 1000 groups 18.4 / 23.6 / 38.9, of 1500
// 23.5 / 26.0 / 40.2 and for 16 rows 7.2 / 6.1 / 7.9, of 3000 40.2 / 37.6 /
// 45.4, of 4000 55.6 / 54.2 / 54.7 and for 16 rows 12.9 / 9.2 / 8.4; the loss
// of 1000 groups 12.3 / 18.1, of 2000 19.3 / 21.0 and for 16 rows 5.9 / 5.0).
// Float32 rows of up to 16 groups a thread are held whole, longer ones by 18.
template <bool BF16, int OP, bool PAST>
hipError_t launch_rows(const DistillArgs& a, hipStream_t stream, hipEvent_t* ev) {
    constexpr int G = RowGroup<BF16>::G;
    const long long rows = (long long)a.B * a.n;
    const size_t lds = (size_t)((a.V + 31) / 32) * 4;    // at most 64 KB
    const int full = a.V / G;
    (void)full;
    if constexpr (OP == kDistillGrad) return launch(k_part_grad<BF16, false, PAST>, rows * a.parts, kBlock, 0, stream, ev, a);
    else if constexpr (OP == kDistillLoss)
        return full <= 1024 ? launch(k_distill<BF16, 256, 0, 4, 4, OP, PAST>, rows, 256, lds, stream, ev, a)
                            : launch(k_distill<BF16, 512, 0, 4, 4, OP, PAST>, rows, 512, lds, stream, ev, a);
    else {
#define SPECV_ROWS(NT, NG, LD, MW) launch(k_distill<BF16, NT, NG, LD, MW, OP, PAST>, rows, NT, lds, stream, ev, a)
        if (full <= 4 * 256) return SPECV_ROWS(256, 4, 2, 8);
        if (full <= 6 * 512) return SPECV_ROWS(512, 4, 2, 8);
        if (full <= 4 * 1024) return SPECV_ROWS(1024, 4, 2, 8);
        if constexpr (BF16) return SPECV_ROWS(1024, 6, 2, 8);
        else return full <= 16 * 1024 ? SPECV_ROWS(1024, 16, 4, 4) : SPECV_ROWS(1024, 18, 4, 4);
#undef SPECV_ROWS
    }
}

template <bool BF16>
hipError_t launch_parts(const DistillArgs& a, DistillOp op, hipStream_t stream, hipEvent_t* ev) {
    const long long rows = (long long)a.B * a.n;
    const hipError_t e = launch_with(k_part_stats<BF16>, rows * a.parts, kBlock, 0, stream, ev ? ev[0] : nullptr, nullptr, a,
                               op == kDistillLossGrad);
    if (e != hipSuccess) return e;
    if (op == kDistillLoss) return launch_with(k_part_loss, rows, kWave, 0, stream, nullptr, ev ? ev[1] : nullptr, a);
    return launch_with(k_part_grad<BF16, true, false>, rows * a.parts, kBlock, 0, stream, nullptr,
                       ev ? ev[1] : nullptr, a);
}

template <bool BF16>
hipError_t launch_op(DistillArgs& a, DistillOp op, hipStream_t stream, hipEvent_t* ev) {
    a.parts = (a.V + kPart<BF16> - 1) / kPart<BF16>;
    if (a.part) return launch_parts<BF16>(a, op, stream, ev);
    const bool past = (long long)a.B * a.n * a.V * (BF16 ? 2 : 4) > kPastBytes;
    if (op == kDistillLoss)
        return past ? launch_rows<BF16, kDistillLoss, true>(a, stream, ev)
                    : launch_rows<BF16, kDistillLoss, false>(a, stream, ev);
    if (op == kDistillGrad)
        return past ? launch_rows<BF16, kDistillGrad, true>(a, stream, ev)
                    : launch_rows<BF16, kDistillGrad, false>(a, stream, ev);
    return past ? launch_rows<BF16, kDistillLossGrad, true>(a, stream, ev)
                : launch_rows<BF16, kDistillLossGrad, false>(a, stream, ev);
}

}  // namespace

size_t distill_workspace(DistillOp op, bool bf16, long long rows, int V, int K) {
    if (op == kDistillGrad || rows <= 0 || rows > kPartRows) return 0;
    const int part = bf16 ? kPart<true> : kPart<false>, parts = (V + part - 1) / part;
    if (parts < kMinParts) return 0;
    return (size_t)rows * (parts * sizeof(float2) + 2 * (size_t)K * sizeof(float));
}

hipError_t launch_distill(const DistillArgs& a, DistillOp op, bool bf16, hipStream_t stream, hipEvent_t* ev) {
    DistillArgs r = a;
    return bf16 ? launch_op<true>(r, op, stream, ev) : launch_op<false>(r, op, stream, ev);
}

}  // namespace specv
