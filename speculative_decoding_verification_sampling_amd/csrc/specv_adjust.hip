// specv_adjust_logits: penalties for repeated tokens, sparse biases and
// grammar masks on logits rows; specv_history_add / specv_history_reset: the
// token histories behind the penalties.
//
// A thread owns 8 consecutive tokens of a chunk and walks the positions of a
// batch row over them: the seen bits (one byte), the counts (loaded where a
// bit is set) and the row's biases (gathered once into LDS) serve every
// position, the drafts of the round are added to the counts as the positions
// pass them, and each position costs one 16-byte load and store per 8
// bfloat16 logits plus one byte of its mask.

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specv_device.hpp"

namespace specv {
namespace {

constexpr int kTok = 8;                        // tokens per thread: one byte of a bit row
constexpr int kAdjChunk = kBlock * kTok;       // tokens per workgroup

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
        *reinterpret_cast<u32x4_a2*>(static_cast<unsigned short*>(row) + v) = q;
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
        *reinterpret_cast<u32x4_a2*>(p) = q[0];
        *reinterpret_cast<u32x4_a2*>(p + 4) = q[1];
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

struct BiasScratch {
    float sum[kAdjChunk];        // the row's bias per token of the chunk
    unsigned bits[kBlock / 4];   // one byte per thread: its tokens with a bias
    int tok[kBlock];             // one batch of entries inside the chunk, in list order
    float val[kBlock];
    int wave_n[kWaves];
};

// The biases of batch row b inside the chunk at v0, added in list order:
// entries are taken kBlock at a time and compacted in order; the first entry
// of each token adds the later ones of its batch up.  Returns whether there
// are any; sc.sum and sc.bits are then complete.  Whole workgroup.
__device__ __forceinline__ bool gather_bias(const AdjustArgs& a, int b, int v0, int len, BiasScratch& sc) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int lo = min(max(a.bias_off[b], 0), a.n_bias), hi = min(max(a.bias_off[b + 1], 0), a.n_bias);
    if (lo >= hi) return false;
    bool any = false;
    for (int base = lo; base < hi; base += kBlock) {
        const int i = min(base + tid, hi - 1);
        const long long t = a.bias_tok[i];
        const float val = a.bias_val[i];
        const bool in = base + tid < hi && t >= v0 && t < (long long)v0 + len;
        const unsigned long long m = __ballot(in);
        if (lane == 0) sc.wave_n[wave] = __popcll(m);
        __syncthreads();
        int before = 0, total = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) before += sc.wave_n[w];
            total += sc.wave_n[w];
        }
        if (total && !any) {
#pragma unroll
            for (int e = 0; e < kTok; ++e) sc.sum[tid + e * kBlock] = 0.f;
            if (tid < kBlock / 4) sc.bits[tid] = 0;
            any = true;
        }
        const int my = before + __popcll(m & ((1ull << lane) - 1));
        if (in) {
            sc.tok[my] = (int)(t - v0);
            sc.val[my] = val;
        }
        __syncthreads();
        if (tid < total) {
            const int rel = sc.tok[tid];
            bool first = true;
            for (int q = 0; q < tid; ++q) first = first && sc.tok[q] != rel;
            if (first) {
                float s = sc.sum[rel];
                for (int q = tid; q < total; ++q)
                    if (sc.tok[q] == rel) s += sc.val[q];
                sc.sum[rel] = s;
                atomicOr(&sc.bits[rel / 32], 1u << (rel % 32));
            }
        }
        __syncthreads();
    }
    return any;
}

template <bool BF16>
__global__ __launch_bounds__(kBlock) void k_adjust(AdjustArgs a) {
    __shared__ BiasScratch sc;
    const int tid = threadIdx.x;
    const unsigned per_row = (unsigned)a.C * a.PG;
    const int b = blockIdx.x / per_row;
    const int rem = blockIdx.x % per_row;
    const int pg = rem / a.C, c = rem % a.C;
    const int v0 = c * kAdjChunk;
    const int len = min(kAdjChunk, a.V - v0);
    const int i0 = pg * a.pp, i1 = min(i0 + a.pp, a.n);
    const int m = min(max(len - tid * kTok, 0), kTok);        // this thread's tokens
    const long long v = (long long)v0 + tid * kTok;

    float rep = 1.f, pres = 0.f, freq = 0.f;
    unsigned used = 0;
    int cnt[kTok];
#pragma unroll
    for (int e = 0; e < kTok; ++e) cnt[e] = 0;
    const int* tok = nullptr;
    if (a.pen) {
        const specv_penalties p = a.pen[b];
        rep = p.repetition;
        pres = p.presence;
        freq = p.frequency;
        if (p.slot >= 0 && p.slot < a.n_slots && m > 0) {
            const long long words = (a.V + 31) / 32;
            used = reinterpret_cast<const unsigned char*>(a.seen + p.slot * words)[v / 8];
            used &= (1u << m) - 1;
            const int* cr = a.counts + (long long)p.slot * a.V + v;
#pragma unroll
            for (int e = 0; e < kTok; ++e)
                if ((used >> e) & 1) cnt[e] = cr[e];
        }
        if (a.tokens) tok = a.tokens + (long long)b * a.tok_sb;
    }
    unsigned biased = 0;
    if (a.bias_off && gather_bias(a, b, v0, len, sc)) biased = (sc.bits[tid / 4] >> (8 * (tid % 4))) & 0xFF;

    const bool inplace = a.in == a.out;
    int p = 0;                                                  // drafts taken into the counts so far
    for (int i = i0; i < i1; ++i) {
        if (tok) {
            for (const int before = a.pos0 + i; p < before; ++p) {
                const long long t = tok[p];
                if (t < v0 || t >= (long long)v0 + len) continue;   // uniform
                const int rel = (int)(t - v0) - tid * kTok;
#pragma unroll
                for (int e = 0; e < kTok; ++e)
                    if (rel == e) {
                        cnt[e]++;
                        used |= 1u << e;
                    }
            }
        }
        if (m == 0) continue;
        unsigned allowed = 0xFF;
        if (a.mask)
            allowed = reinterpret_cast<const unsigned char*>(a.mask + (long long)b * a.m_sb +
                                                             (long long)i * a.m_sp)[v / 8];
        allowed |= 0xFFu << m;
        const unsigned special = (used | biased) & allowed;
        const bool masked = (allowed & ((1u << m) - 1)) != ((1u << m) - 1);
        if (inplace && !special && !masked) continue;
        const void* in = row_ptr<BF16>(a.in, a.i_sb, a.i_sp, b, i);
        void* out = const_cast<void*>(row_ptr<BF16>(a.out, a.o_sb, a.o_sp, b, i));
        Group<BF16> g{};
        if ((allowed & ((1u << m) - 1)) != 0) {
            if (m == kTok) g.load(in, v);
            else g.load_part(in, v, m);
        }
        if (special) {
#pragma unroll
            for (int e = 0; e < kTok; ++e) {
                if (!((special >> e) & 1)) continue;
                float x = g.get(e);
                if ((used >> e) & 1) {
                    x = x > 0.f ? x / rep : x * rep;
                    if (cnt[e] > 0) x = (x - freq * (float)cnt[e]) - pres;
                }
                if ((biased >> e) & 1) x += sc.sum[tid * kTok + e];
                g.put(e, x);
            }
        }
        if (masked) g.mask(allowed);
        if (m == kTok) g.store(out, v);
        else g.store_part(out, v, m);
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
hipError_t launch(void (*fn)(A...), long long blocks, int threads, hipStream_t stream, hipEvent_t* ev, A... args) {
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    if (ev)
        hipExtLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), 0, stream, ev[0], ev[1], 0, args...);
    else
        hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), 0, stream, args...);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adjust(AdjustArgs& a, bool bf16, hipStream_t stream, hipEvent_t* ev) {
    a.C = (a.V + kAdjChunk - 1) / kAdjChunk;
    a.pp = a.n;
    a.PG = (a.n + a.pp - 1) / a.pp;
    return launch(bf16 ? k_adjust<true> : k_adjust<false>, (long long)a.B * a.PG * a.C, kBlock, stream, ev, a);
}

hipError_t launch_history_add(const HistoryArgs& a, hipStream_t stream, hipEvent_t* ev) {
    const int per_row = (a.n - 1) / kBlock + 1;
    return launch(k_history_add, (long long)a.B * per_row, kBlock, stream, ev, a, per_row);
}

hipError_t launch_history_reset(const HistoryArgs& a, hipStream_t stream, hipEvent_t* ev) {
    const int words = (a.V + 31) / 32;
    const int per_row = (words + kBlock - 1) / kBlock;
    return launch(k_history_reset, (long long)a.B * per_row, kBlock, stream, ev, a, per_row);
}

}  // namespace specv
