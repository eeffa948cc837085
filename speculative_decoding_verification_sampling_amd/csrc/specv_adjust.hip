// specv_adjust_logits: penalties for repeated tokens, sparse biases and
// grammar masks on logits rows; specv_history_add / specv_history_reset: the
// token histories behind the penalties.
//
// A thread owns 8 consecutive tokens of a chunk (one byte of a bit row) and
// walks the positions of a batch row over them: the seen bits, the counts
// (loaded where a bit is set) and the row's biases serve every position, the
// drafts of the round are added to the counts as the positions pass them, and
// each position costs one 16-byte load and store per 8 bfloat16 logits plus
// one byte of its mask.
//
// Bound by memory: 64 x 6 rows of 128256 bfloat16 logits (205 MB with masks)
// take 44 us (4.7 TB/s) with penalties, biases and masks, 39.5 us with
// penalties alone, 37.5 us with masks alone, which is the rate of a copy; the
// difference is the chain of loads before the first logit can be written
// (penalties, seen bits, counts) and the arithmetic of used tokens.  Masks in
// place on 32 x 6 rows of 152064 (58 MB written): 12 us.  One row of 32000:
// 4 us, a launch.

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "specv_logits_device.hpp"

namespace specv {
namespace {

constexpr int kTok = 8;                        // tokens per thread: one byte of a bit row
constexpr long long kFill = 1024;              // workgroups below which positions are split
constexpr int kAdjChunk = kBlock * kTok;       // tokens per workgroup

constexpr int kHistBlock = 512;                // threads of a workgroup that gathers bits, and its tokens
constexpr int kHistSpan = 16384, kHistSpanCounted = 1024;
constexpr int kHistFrom = 512;                 // row length from which it does (below, both take a launch)

// 8 logits as they are stored.
template <bool BF16>
struct Group;

template <>
struct Group<true> {
    u32x4 q;
    __device__ inline void load(const void* row, long long v) {
        q = *reinterpret_cast<const u32x4_a2*>(static_cast<const unsigned short*>(row) + v);
    }
    __device__ inline void store(void* row, long long v) const {
        __builtin_nontemporal_store(q, reinterpret_cast<u32x4_a2*>(static_cast<unsigned short*>(row) + v));
    }
    __device__ inline void load_part(const void* row, long long v, int m) {
        const unsigned short* p = static_cast<const unsigned short*>(row) + v;
        unsigned w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kTok - 1; ++e)
            if (e < m) w[e / 2] |= (unsigned)p[e] << (16 * (e & 1));
        q = u32x4{w[0], w[1], w[2], w[3]};
    }
    __device__ inline void store_part(void* row, long long v, int m) const {
        unsigned short* p = static_cast<unsigned short*>(row) + v;
#pragma unroll
        for (int e = 0; e < kTok - 1; ++e)
            if (e < m) p[e] = (unsigned short)(q[e / 2] >> (16 * (e & 1)));
    }
    __device__ inline float get(int e) const { return (e & 1) ? bf16_hi(q[e / 2]) : bf16_lo(q[e / 2]); }
    __device__ inline void put(int e, float x) {
        const unsigned h = __builtin_bit_cast(unsigned short, static_cast<__bf16>(x));
        q[e / 2] = (e & 1) ? ((q[e / 2] & 0xFFFFu) | (h << 16)) : ((q[e / 2] & 0xFFFF0000u) | h);
    }
    __device__ inline void mask(unsigned allowed) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const unsigned lo = (allowed >> (2 * w)) & 1, hi = (allowed >> (2 * w + 1)) & 1;
            q[w] = (lo ? q[w] & 0xFFFFu : 0xFF80u) | (hi ? q[w] & 0xFFFF0000u : 0xFF800000u);
        }
    }
};

template <>
struct Group<false> {
    u32x4 q[2];
    __device__ inline void load(const void* row, long long v) {
        const float* p = static_cast<const float*>(row) + v;
        q[0] = *reinterpret_cast<const u32x4_a2*>(p);
        q[1] = *reinterpret_cast<const u32x4_a2*>(p + 4);
    }
    __device__ inline void store(void* row, long long v) const {
        float* p = static_cast<float*>(row) + v;
        __builtin_nontemporal_store(q[0], reinterpret_cast<u32x4_a2*>(p));
        __builtin_nontemporal_store(q[1], reinterpret_cast<u32x4_a2*>(p + 4));
    }
    __device__ inline void load_part(const void* row, long long v, int m) {
        const unsigned* p = static_cast<const unsigned*>(row) + v;
        q[0] = q[1] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kTok - 1; ++e)
            if (e < m) q[e / 4][e % 4] = p[e];
    }
    __device__ inline void store_part(void* row, long long v, int m) const {
        unsigned* p = static_cast<unsigned*>(row) + v;
#pragma unroll
        for (int e = 0; e < kTok - 1; ++e)
            if (e < m) p[e] = q[e / 4][e % 4];
    }
    __device__ inline float get(int e) const { return __uint_as_float(q[e / 4][e % 4]); }
    __device__ inline void put(int e, float x) { q[e / 4][e % 4] = __float_as_uint(x); }
    __device__ inline void mask(unsigned allowed) {
#pragma unroll
        for (int e = 0; e < kTok; ++e)
            if (!((allowed >> e) & 1)) q[e / 4][e % 4] = 0xFF800000u;
    }
};

// The biases of a batch row on this thread's tokens v .. v + 7 (added in list
// order into sum[]); returns their bits.  Every wave walks the row's entries
// 64 at a time and stops only at those among its own tokens, so the workgroup
// needs no LDS and no barrier for them.  ``issue`` loads the first 64, to be
// on their way with other loads.
struct BiasEntries {
    int lo, hi, tok;
    float val;
    __device__ __forceinline__ void load(const AdjustArgs& a, int base) {
        const int i = min(base + (int)threadIdx.x % kWave, hi - 1);
        tok = a.bias_tok[i];
        val = a.bias_val[i];
    }
    __device__ __forceinline__ void issue(const AdjustArgs& a, int b) {
        lo = min(max(a.bias_off[b], 0), a.n_bias);
        hi = min(max(a.bias_off[b + 1], 0), a.n_bias);
        if (lo < hi) load(a, lo);
    }
    __device__ __forceinline__ unsigned gather(const AdjustArgs& a, int v0, float (&sum)[kTok]) {
        const int lane = threadIdx.x % kWave;
        const int first = v0 + ((int)threadIdx.x - lane) * kTok;             // the wave's tokens
        const int len = min(kWave * kTok, a.V - first);
        unsigned bits = 0;
        for (int base = lo; base < hi; base += kWave) {
            if (base > lo) load(a, base);
            unsigned long long m = __ballot(base + lane < hi && tok >= first && tok - first < len);
            while (m) {
                const int k = __builtin_ctzll(m);
                m &= m - 1;
                const int rel = __builtin_amdgcn_readlane(tok, k) - first - lane * kTok;
                const float x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(val), k));
#pragma unroll
                for (int e = 0; e < kTok; ++e)
                    if (rel == e) {
                        sum[e] += x;
                        bits |= 1u << e;
                    }
            }
        }
        return bits;
    }
};

// x / d, correctly rounded, from inv = 1 / d correctly rounded: the quotient's
// remainder corrects it once.  An infinite or NaN quotient stays.
__device__ inline float divide(float x, float d, float inv) {
    const float q = x * inv;
    const float r = fmaf(-q, d, x);
    return fabsf(q) <= 3.402823466e38f ? fmaf(r, inv, q) : q;
}

// kAhead positions are loaded at once (mask bytes first: a group of which the
// mask leaves nothing is not read); four at once take 65 registers, a
// workgroup per CU less, and 8 % more time.  In place only the groups
// that change are read and written.  Stores go past the caches (64 x 6 rows:
// 6 % more time without).  Eight workgroups per CU in bfloat16; the float32 copy of
// the kernel would spill at that and is given one less.
template <bool BF16, bool INPLACE>
__global__ __launch_bounds__(kBlock, BF16 ? 8 : 7) void k_adjust(AdjustArgs a) {
    constexpr int kAhead = 2;
    const int tid = threadIdx.x;
    const unsigned per_row = (unsigned)a.C * a.PG;
    const int b = blockIdx.x / per_row;
    const int rem = blockIdx.x % per_row;
    const int pg = rem / a.C, c = rem % a.C;
    const int v0 = c * kAdjChunk;
    const int len = min(kAdjChunk, a.V - v0);
    const int i0 = pg * a.pp, i1 = min(i0 + a.pp, a.n);
    const int m = min(max(len - tid * kTok, 0), kTok);        // this thread's tokens
    const unsigned live = (1u << m) - 1;
    const long long v = (long long)v0 + tid * kTok;

    Group<BF16> g[kAhead];
    unsigned allowed[kAhead];
    const auto load_masks = [&](int i) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            allowed[k] = live;
            if (a.mask && i + k < i1 && m > 0)
                allowed[k] &= reinterpret_cast<const unsigned char*>(a.mask + (long long)b * a.m_sb +
                                                                     (long long)(i + k) * a.m_sp)[v / 8];
        }
    };
    const auto load_rows = [&](int i, unsigned special) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const bool read = allowed[k] != 0 && (!INPLACE || (special & allowed[k]) || allowed[k] != live);
            if (i + k < i1 && read) {
                const void* in = row_ptr<BF16>(a.in, a.i_sb, a.i_sp, b, i + k);
                if (m == kTok) g[k].load(in, v);
                else g[k].load_part(in, v, m);
            }
        }
    };
    load_masks(i0);
    if (!INPLACE) load_rows(i0, 0);                             // on their way during the preparations

    BiasEntries be;
    if (a.bias_off) be.issue(a, b);

    float rep = 1.f, pres = 0.f, freq = 0.f;
    unsigned used = 0;
    float cnt[kTok], bias[kTok];
#pragma unroll
    for (int e = 0; e < kTok; ++e) cnt[e] = bias[e] = 0.f;
    const int* tok = nullptr;
    if (a.pen) {
        const specv_penalties p = a.pen[b];
        rep = p.repetition;
        pres = p.presence;
        freq = p.frequency;
        if (p.slot >= 0 && p.slot < a.n_slots && m > 0) {
            const long long words = (a.V + 31) / 32;
            used = reinterpret_cast<const unsigned char*>(a.seen + p.slot * words)[v / 8] & live;
            const int* cr = a.counts + (long long)p.slot * a.V + v;
            if (used) {
                // all of them at once: one load each, converted where it lands, would wait eight times
                int ci[kTok];
                if (m == kTok) {
                    const u32x4 lo = *reinterpret_cast<const u32x4_a2*>(cr), hi = *reinterpret_cast<const u32x4_a2*>(cr + 4);
#pragma unroll
                    for (int e = 0; e < kTok; ++e) ci[e] = (int)(e < 4 ? lo[e] : hi[e - 4]);
                } else {
#pragma unroll
                    for (int e = 0; e < kTok; ++e) ci[e] = cr[min(e, m - 1)];
                }
#pragma unroll
                for (int e = 0; e < kTok; ++e) cnt[e] = (used >> e) & 1 ? (float)ci[e] : 0.f;
            }
        }
        if (a.tokens) tok = a.tokens + (long long)b * a.tok_sb;
    }
    const unsigned biased = a.bias_off ? be.gather(a, v0, bias) : 0;
    const float inv = 1.f / rep;

    int p = 0;                                                  // drafts taken into the counts so far
    for (int ib = i0; ib < i1; ib += kAhead) {
        if (ib > i0) load_masks(ib);
        if (INPLACE) {
            // the drafts of these positions may still mark tokens
            unsigned special = used | biased;
            if (tok) {
                for (int q = p; q < a.pos0 + min(ib + kAhead, i1) - 1; ++q) {
                    const long long rel = (long long)tok[q] - v;
                    if (rel >= 0 && rel < m) special |= 1u << rel;
                }
            }
            load_rows(ib, special);
        } else if (ib > i0) {
            load_rows(ib, 0);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = ib + k;
            if (i >= i1) break;
            if (tok) {
                for (const int before = a.pos0 + i; p < before; ++p) {
                    const long long t = tok[p];
                    if (t < v0 || t >= (long long)v0 + len) continue;   // uniform
                    const int rel = (int)(t - v0) - tid * kTok;
#pragma unroll
                    for (int e = 0; e < kTok; ++e)
                        if (rel == e) {
                            cnt[e] += 1.f;
                            used |= 1u << e;
                        }
                }
            }
            const unsigned special = (used | biased) & allowed[k];
            if (m == 0 || (INPLACE && !special && allowed[k] == live)) continue;
            if (special) {
#pragma unroll
                for (int e = 0; e < kTok; ++e) {
                    if (!((special >> e) & 1)) continue;
                    const float z = g[k].get(e);            // no branches in here: selects are cheaper
                    const float q = divide(z, rep, inv);
                    float x = z > 0.f ? q : z * rep;
                    x = (used >> e) & 1 ? x : z;
                    const float y = (x - freq * cnt[e]) - pres;
                    x = cnt[e] > 0.f ? y : x;
                    const float w = x + bias[e];
                    x = (biased >> e) & 1 ? w : x;
                    g[k].put(e, x);
                }
            }
            if (allowed[k] != live) g[k].mask(allowed[k]);
            void* out = const_cast<void*>(row_ptr<BF16>(a.out, a.o_sb, a.o_sp, b, i));
            if (m == kTok) g[k].store(out, v);
            else g[k].store_part(out, v, m);
        }
    }
}

// One thread per (batch row, token).
__global__ __launch_bounds__(kBlock) void k_history_add(HistoryArgs a, int blocks_per_row) {
    const int b = blockIdx.x / blocks_per_row;
    const int t = (blockIdx.x % blocks_per_row) * kBlock + threadIdx.x;
    const int slot = a.slots[b];
    if (slot < 0 || slot >= a.n_slots) return;
    const int len = a.lengths ? min(a.lengths[b], a.n) : a.n;
    if (t >= len) return;
    const int v = a.tokens[(long long)b * a.tok_sb + t];
    if (v < 0 || v >= a.V) return;
    const long long words = (a.V + 31) / 32;
    unsigned* w = a.seen + slot * words + v / 32;
    atomicOr(w, 1u << (v % 32));
    if (!a.prompt) atomicAdd(a.counts + (long long)slot * a.V + v, 1);
}

// Long rows of tokens: text repeats its tokens, and atomics on one address
// queue up.  A workgroup gathers the bits of ``span`` tokens in a bit row in
// LDS first, so that a word of the seen bits gets one atomic of it.  Skewed
// tokens, V 128256, against a thread per token with its own atomics: 64
// prompts of 4000 / 8000 / 40000 tokens 9.3 / 17 / 85 -> 4.6 / 7.0 / 12 us;
// 64 rows of 2000 / 8000 generated ones 8.9 / 33 -> 7.1 / 21.  Counted tokens
// take short spans: their atomics need many workgroups (one row of 8000: 4.1 us
// in spans of 1024, 8.8 of 4096).  A table of counts in LDS gained nothing.
__global__ __launch_bounds__(kHistBlock) void k_history_add_span(HistoryArgs a, int spans, int span) {
    extern __shared__ unsigned bits[];
    const int b = blockIdx.x / spans;
    const int t0 = (blockIdx.x % spans) * span;
    const int slot = a.slots[b];
    const int len = a.lengths ? min(a.lengths[b], a.n) : a.n;
    if (slot < 0 || slot >= a.n_slots || t0 >= len) return;          // uniform
    const int words = (a.V + 31) / 32, t1 = min(len - t0, span) + t0;
    for (int w = threadIdx.x; w < words; w += kHistBlock) bits[w] = 0;
    __syncthreads();
    const int* tok = a.tokens + (long long)b * a.tok_sb;
    int* counts = a.counts + (long long)slot * a.V;
    for (int t = t0 + (int)threadIdx.x; t < t1; t += kHistBlock) {
        const int v = tok[t];
        if (v < 0 || v >= a.V) continue;
        atomicOr(&bits[v / 32], 1u << (v % 32));
        if (!a.prompt) atomicAdd(counts + v, 1);
    }
    __syncthreads();
    unsigned* seen = a.seen + (long long)slot * words;
    for (int w = threadIdx.x; w < words; w += kHistBlock)
        if (bits[w]) atomicOr(seen + w, bits[w]);
}

// One thread per word of seen bits; counts are cleared where a bit is set.
// A slot listed twice is cleared by whichever thread sees the word first or
// by both.
__global__ __launch_bounds__(kBlock) void k_history_reset(HistoryArgs a, int blocks_per_row) {
    const int b = blockIdx.x / blocks_per_row;
    const int i = (blockIdx.x % blocks_per_row) * kBlock + threadIdx.x;
    const int slot = a.slots[b];
    const int words = (a.V + 31) / 32;
    if (slot < 0 || slot >= a.n_slots || i >= words) return;
    unsigned* w = a.seen + (long long)slot * words + i;
    unsigned bits = *w;
    if (!bits) return;
    int* cr = a.counts + (long long)slot * a.V + i * 32;
    *w = 0;
    if (i * 32 + 32 > a.V) bits &= (1u << (a.V - i * 32)) - 1;
    while (bits) {
        const int e = __builtin_ctz(bits);
        bits &= bits - 1;
        cr[e] = 0;
    }
}

template <typename... A>
hipError_t launch(void (*fn)(A...), long long blocks, int threads, hipStream_t stream, hipEvent_t* ev, size_t lds,
                  A... args) {
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    if (ev)
        hipExtLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), lds, stream, ev[0], ev[1], 0, args...);
    else
        hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), lds, stream, args...);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adjust(AdjustArgs& a, bool bf16, hipStream_t stream, hipEvent_t* ev) {
    a.C = (a.V + kAdjChunk - 1) / kAdjChunk;
    // a workgroup takes all positions of its tokens (64 x 6 rows of 128256: 61 us, one
    // position each 100) unless there are too few to fill the device
    const long long wgs = (long long)a.B * a.C;
    const int groups = (int)std::min<long long>(a.n, (kFill + wgs - 1) / wgs);
    a.pp = (a.n + groups - 1) / groups;
    a.PG = (a.n + a.pp - 1) / a.pp;
    const bool inplace = a.in == a.out;
    auto fn = bf16 ? (inplace ? k_adjust<true, true> : k_adjust<true, false>)
                   : (inplace ? k_adjust<false, true> : k_adjust<false, false>);
    return launch(fn, (long long)a.B * a.PG * a.C, kBlock, stream, ev, 0, a);
}

hipError_t launch_history_add(const HistoryArgs& a, hipStream_t stream, hipEvent_t* ev) {
    if (a.n >= kHistFrom) {
        const int span = a.prompt ? kHistSpan : kHistSpanCounted, spans = (a.n - 1) / span + 1;
        return launch(k_history_add_span, (long long)a.B * spans, kHistBlock, stream, ev, (size_t)((a.V + 31) / 32) * 4,
                      a, spans, span);
    }
    const int per_row = (a.n - 1) / kBlock + 1;
    return launch(k_history_add, (long long)a.B * per_row, kBlock, stream, ev, 0, a, per_row);
}

hipError_t launch_history_reset(const HistoryArgs& a, hipStream_t stream, hipEvent_t* ev) {
    const int words = (a.V + 31) / 32;
    const int per_row = (words + kBlock - 1) / kBlock;
    return launch(k_history_reset, (long long)a.B * per_row, kBlock, stream, ev, 0, a, per_row);
}

}  // namespace specv
