// Device helpers of the logits operators: rows in 16-byte groups at any
// address, and exponentials relative to a reference.
#pragma once

#include "specv_device.hpp"
#include "specv_logits.hpp"

namespace specv {
namespace {

// 16 bytes at any element-aligned address (one global_load / store_dwordx4:
// gfx950 takes them unaligned).
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

// Group g (16 bytes: 8 bfloat16 or 4 float32 entries) of a row of V entries
// at any address, entries past the end as -inf.  ``issue`` starts the load of
// a whole group (others load group 0, or nothing when the row has none) and
// ``finish`` puts the last, partial group and the ones past it right.
template <bool BF16>
struct RowGroup {
    static constexpr int G = BF16 ? 8 : 4;
    u32x4 q;
    // PAST: past the caches, for rows too many to be found there later.
    template <bool PAST = false>
    __device__ inline void issue(const void* row, long long g, int full) {
        if (full <= 0) return;
        const u32x4_a2* p = static_cast<const u32x4_a2*>(row) + (g < full ? g : 0);
        if constexpr (PAST) q = __builtin_nontemporal_load(p);
        else q = *p;
    }
    __device__ inline void finish(const void* row, long long g, int full, int V) {
        if (g < full) return;
        const unsigned ninf = BF16 ? 0xFF80FF80u : 0xFF800000u;
        unsigned w[4] = {ninf, ninf, ninf, ninf};
        if (g == full) {
            const int rem = V - full * G;
#pragma unroll
            for (int e = 0; e < G - 1; ++e) {
                if (e < rem) {
                    if constexpr (BF16) {
                        const unsigned h = static_cast<const unsigned short*>(row)[(long long)full * G + e];
                        w[e / 2] = (e & 1) ? ((w[e / 2] & 0xFFFFu) | (h << 16)) : ((w[e / 2] & 0xFFFF0000u) | h);
                    } else {
                        w[e] = static_cast<const unsigned*>(row)[(long long)full * G + e];
                    }
                }
            }
        }
        q = u32x4{w[0], w[1], w[2], w[3]};
    }
    // A group that ``issue`` did not load becomes -inf.
    __device__ inline void clear(long long g, int full) {
        const unsigned ninf = BF16 ? 0xFF80FF80u : 0xFF800000u;
        if (g >= full) q = u32x4{ninf, ninf, ninf, ninf};
    }
    __device__ inline float elem(int e) const {
        if constexpr (BF16) return (e & 1) ? bf16_hi(q[e / 2]) : bf16_lo(q[e / 2]);
        else return __uint_as_float(q[e]);
    }
    // Entry e for a per-lane e.
    __device__ inline float elem_dyn(int e) const {
        constexpr int P = G / 4;                  // entries of a word
        const unsigned lo = e < P ? q[0] : q[1], hi = e < 3 * P ? q[2] : q[3];
        const unsigned w = e < 2 * P ? lo : hi;
        if constexpr (BF16) return __uint_as_float((e & 1) ? w & 0xFFFF0000u : w << 16);
        else return __uint_as_float(w);
    }
    // Keeps the group packed between two passes over it: the compiler would
    // otherwise unpack it once and hold the floats, twice the registers.
    __device__ inline void pin() { asm volatile("" : "+v"(q)); }
    // G values rounded to the row's type (bfloat16: to nearest even).
    __device__ inline void pack(const float (&x)[G]) {
        if constexpr (BF16) {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const bf16x2 h = {static_cast<__bf16>(x[2 * w]), static_cast<__bf16>(x[2 * w + 1])};
                q[w] = __builtin_bit_cast(unsigned, h);
            }
        } else {
#pragma unroll
            for (int e = 0; e < G; ++e) q[e] = __float_as_uint(x[e]);
        }
    }
    // For rows that a kernel writes once and does not read again: past the
    // caches, which keep what is read (distill_loss_grad, 2048 rows of 128256
    // bfloat16 logits: 234 -> 213 us).
    __device__ inline void store(void* row, long long g) const {
        __builtin_nontemporal_store(q, static_cast<u32x4_a2*>(row) + g);
    }
};

// The entries named by the bits of ``in`` become -inf.
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

// exp2((x - ref) * scale) for many x and one ref, as one fused multiply-add
// each: 2^(x scale - R) with R = ref scale rounded, and the factor
// ``fix`` = 2^(R - ref scale) that makes up for the rounding, applied to the
// sum.  ``step`` where R overflows (ref near the type's lowest or largest
// value): neighbouring floats are then far more than 128 apart in exponent,
// and the exponential is 1 at ref and 0 below it.
struct ExpRef {
    float ref, nr, fix, scale;
    bool step;
    __device__ inline ExpRef(float r, float sc) : ref(r == -kInf ? 0.f : r), scale(sc) {
        nr = -(ref * scale);
        step = !(fabsf(nr) <= 3.402823466e38f);
        fix = step ? 1.f : fast_exp2(-fmaf(ref, scale, nr));
    }
    __device__ inline float fast(float x) const { return fast_exp2(fmaf(x, scale, nr)); }
    __device__ inline float at_step(float x) const {     // NaN for NaN and +inf, as ``fast``
        return x < ref ? 0.f : x == ref && x <= 3.402823466e38f ? 1.f : __builtin_nanf("");
    }
    __device__ inline float any(float x) const { return step ? at_step(x) : fast(x) * fix; }
};

// Sum of exp2((x - ref) * scale) over N groups; ``ref`` is their maximum or
// above it.
template <int N, typename Group>
__device__ __forceinline__ float sum_exp(Group (&r)[N], const ExpRef& x) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        r[j].pin();
#pragma unroll
        for (int e = 0; e < Group::G; ++e) s += x.fast(r[j].elem(e));
    }
    s *= x.fix;
    if (__builtin_expect(__ballot(x.step) != 0, 0)) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            r[j].pin();
#pragma unroll
            for (int e = 0; e < Group::G; ++e) t += x.at_step(r[j].elem(e));
        }
        s = x.step ? t : s;
    }
    return s;
}

template <bool BF16>
__device__ inline void store_elem(void* row, long long v, float x) {
    if constexpr (BF16) static_cast<__bf16*>(row)[v] = static_cast<__bf16>(x);
    else static_cast<float*>(row)[v] = x;
}

}  // namespace
}  // namespace specv
