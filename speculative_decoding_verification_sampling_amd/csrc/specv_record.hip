// specv_top_logits: a teacher's record of logits rows, the K largest logits
// with their tokens and the log-sum-exps of the row and of the rest.
//
// One workgroup per row.  The K-th largest value comes from a radix select
// on order keys (32-bit, larger key = larger logit), digit by digit over the
// row; then one pass sums the exponentials below it and collects what lies
// above, equal values are taken in token order, and the K entries are ranked
// by counting.

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specv_device.hpp"

namespace specv {
namespace {

constexpr int kRecBlock = 1024;
constexpr int kRecWaves = kRecBlock / kWave;
constexpr int kBins = 2048;                     // 11-bit digits (the last one 10 bits)

// Order key of a logit: larger key, larger value; -0 counts as +0.
__device__ inline unsigned order_key(float x) {
    const unsigned u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ inline float key_value(unsigned k) {
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

struct RecordScratch {
    unsigned hist[kBins];
    unsigned long long ent[SPECV_MAX_RECORD_K];     // (key << 32) | ~token
    float top[SPECV_MAX_RECORD_K];                  // exponentials of the record, by rank
    float red[kRecWaves];
    float red2[kRecWaves];
    unsigned cnt[kRecWaves];
    unsigned digit, need, n_above;
};

// Sum over the workgroup, in a fixed order.
__device__ inline float block_sum(float x, float* red) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    x = wave_sum(x);
    __syncthreads();
    if (lane == 0) red[wave] = x;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < kRecWaves; ++w) s += red[w];
    return s;
}

__device__ inline float block_max(float x, float* red) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    x = wave_max(x);
    __syncthreads();
    if (lane == 0) red[wave] = x;
    __syncthreads();
    for (int w = 0; w < kRecWaves; ++w) x = fmaxf(x, red[w]);
    return x;
}

template <bool BF16>
__global__ __launch_bounds__(kRecBlock) void k_top_logits(RecordArgs a) {
    __shared__ RecordScratch sc;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int b = blockIdx.x / a.n, i = blockIdx.x % a.n;
    const void* row = row_ptr<BF16>(a.in, a.sb, a.sp, b, i);
    int* otok = a.tok + (long long)blockIdx.x * a.K;
    float* oval = a.val + (long long)blockIdx.x * a.K;
    float* olse = a.lse + (long long)blockIdx.x * 2;
    const int K = min(a.K, a.V);

    // row maximum and finiteness
    float mx = -kInf;
    unsigned bad = 0;
    for (int v = tid; v < a.V; v += kRecBlock) {
        const float x = load_elem<BF16>(row, v);
        bad |= !(x <= 3.402823466e38f);
        mx = fmaxf(mx, x);
    }
    mx = wave_max(mx);
    bad = wave_or(bad);
    if (lane == 0) {
        sc.red[wave] = mx;
        sc.cnt[wave] = bad;
    }
    __syncthreads();
    for (int w = 0; w < kRecWaves; ++w) {
        mx = fmaxf(mx, sc.red[w]);
        bad |= sc.cnt[w];
    }
    if (bad || mx == -kInf) {
        for (int k = tid; k < a.K; k += kRecBlock) {
            otok[k] = -1;
            oval[k] = -kInf;
        }
        if (tid < 2) olse[tid] = __builtin_nanf("");
        return;
    }

    // radix select of the K-th largest key
    unsigned prefix = 0, mask = 0;
    unsigned need = (unsigned)K;                   // its rank among the keys that match the prefix
    for (int d = 0; d < 3; ++d) {
        const int bits = d < 2 ? 11 : 10, shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        __syncthreads();
        for (int k = tid; k < kBins; k += kRecBlock) sc.hist[k] = 0;
        __syncthreads();
        for (int v = tid; v < a.V; v += kRecBlock) {
            const unsigned key = order_key(load_elem<BF16>(row, v));
            if ((key & mask) == prefix) atomicAdd(&sc.hist[(key >> shift) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            unsigned left = need;
            int k = (1 << bits) - 1;
            while (sc.hist[k] < left) left -= sc.hist[k--];
            sc.digit = (unsigned)k;
            sc.need = left;
        }
        __syncthreads();
        prefix |= sc.digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        need = sc.need;
    }
    const unsigned kth = prefix;                   // ``need`` of the values equal to it are in the record
    const float zk = key_value(kth);

    // the rest's sum (relative to the K-th value) and the entries above
    __syncthreads();
    if (tid == 0) sc.n_above = 0;
    __syncthreads();
    float s = 0.f, below = -kInf;
    unsigned ties = 0;
    for (int v = tid; v < a.V; v += kRecBlock) {
        const float x = load_elem<BF16>(row, v);
        const unsigned key = order_key(x);
        if (key > kth) {
            sc.ent[atomicAdd(&sc.n_above, 1u)] = ((unsigned long long)key << 32) | ~(unsigned)v;
        } else if (key == kth) {
            ++ties;
        } else {
            s += fast_exp2((x - zk) * a.scale);
            below = fmaxf(below, x);
        }
    }
    float rest = block_sum(s, sc.red) + (block_sum((float)ties, sc.red2) - (float)need);
    float ref = zk;
    if (rest == 0.f) {
        // nothing left, or all of it too far below: sum again from the largest of the rest
        below = block_max(below, sc.red);
        if (below > -kInf) {
            ref = below;
            s = 0.f;
            for (int v = tid; v < a.V; v += kRecBlock) {
                const float x = load_elem<BF16>(row, v);
                if (order_key(x) < kth) s += fast_exp2((x - ref) * a.scale);
            }
            rest = block_sum(s, sc.red);
        }
    }
    // ties in token order
    const unsigned above = (unsigned)K - need;
    unsigned taken = 0;
    for (int v0 = 0; v0 < a.V && taken < need; v0 += kRecBlock) {
        const int v = v0 + tid;
        const bool tie = v < a.V && order_key(load_elem<BF16>(row, v)) == kth;
        const unsigned long long m = __ballot(tie);
        __syncthreads();
        if (lane == 0) sc.cnt[wave] = __popcll(m);
        __syncthreads();
        unsigned before = taken;
        for (int w = 0; w < kRecWaves; ++w) {
            if (w < wave) before += sc.cnt[w];
            taken += sc.cnt[w];
        }
        const unsigned my = before + __popcll(m & ((1ull << lane) - 1));
        if (tie && my < need) sc.ent[above + my] = ((unsigned long long)kth << 32) | ~(unsigned)v;
    }
    __syncthreads();
    // rank by counting; entries are distinct
    if (tid < K) {
        const unsigned long long e = sc.ent[tid];
        int rank = 0;
        for (int k = 0; k < K; ++k) rank += sc.ent[k] > e;
        const float x = key_value((unsigned)(e >> 32));
        otok[rank] = (int)~(unsigned)e;
        oval[rank] = x;
        sc.top[rank] = fast_exp2((x - mx) * a.scale);
    }
    for (int k = K + tid; k < a.K; k += kRecBlock) {
        otok[k] = -1;
        oval[k] = -kInf;
    }
    __syncthreads();
    const float top = block_sum(tid < K ? sc.top[tid] : 0.f, sc.red);    // in rank order: the same every time
    if (tid == 0) {
        const bool none = zk == -kInf || !(rest > 0.f);
        const float all = top + (none ? 0.f : rest * fast_exp2((ref - mx) * a.scale));
        olse[0] = fmaf(mx, a.inv_t, logf(all));
        olse[1] = none ? -kInf : fmaf(ref, a.inv_t, logf(rest));
    }
}

}  // namespace

hipError_t launch_top_logits(const RecordArgs& a, bool bf16, hipStream_t stream, hipEvent_t* ev) {
    const long long rows = (long long)a.B * a.n;
    auto fn = bf16 ? k_top_logits<true> : k_top_logits<false>;
    if (ev)
        hipExtLaunchKernelGGL(fn, dim3((unsigned)rows), dim3(kRecBlock), 0, stream, ev[0], ev[1], 0, a);
    else
        hipLaunchKernelGGL(fn, dim3((unsigned)rows), dim3(kRecBlock), 0, stream, a);
    return hipGetLastError();
}

}  // namespace specv
