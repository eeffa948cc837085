// specv_top_logits: a teacher's record of logits rows, the K largest logits
// with their tokens and the log-sum-exps of the row and of the rest.
//
// Bound by memory for many rows: 4096 rows of 128256 bfloat16 logits, K 64,
// take 200 us (5.3 TB/s).  384 such rows take 29 us: all of them are resident
// at once and read in 15 us (6.5 TB/s), and the select behind the read, 7 us
// of dependent steps, has nothing left to hide behind.  5 rows of 32000
// float32 logits: 8 us.

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specv_logits_device.hpp"

namespace specv {
namespace {

// Threads per row.  384 rows of 128256 bfloat16 logits, K 64 / 256: 28.5 / 35.7
// us; with 1024 threads 32.0 / 38.6 (longer joins), with 256 28.1 / 414 (too
// few maxima to bound 256 candidates by).
constexpr int NT = 512;
constexpr int NW = NT / kWave;
constexpr int kBins = 2048;                     // 11-bit digits of the radix select (the last one 10 bits)
constexpr int kLoads = 4;                       // 16-byte groups a thread loads at once
constexpr int kMaxBlocks = 8;                   // blocks per thread (their statistics stand in LDS)
constexpr int kWaveBlk = 128;                   // blocks a wave reads again
constexpr int kCandCap = 1024;                  // candidates ranked
constexpr int kSortFrom = 192;                  // by sorted lists when there are more than this: by counting
                                                // 336 take 6.2 us a row, by lists 280 take 3.2
constexpr unsigned kLowestFinite = 0x00800000u; // the order key of -FLT_MAX; -inf lies below

// Order key of a logit: larger key, larger value; -0 counts as +0.
__device__ inline unsigned order_key(float x) {
    const unsigned u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ inline float key_value(unsigned k) {
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

struct RecordScratch {
    union {
        unsigned hist[kBins];
        struct {
            unsigned short blk[NW][kWaveBlk];        // per wave: blocks with a candidate, block * NT + thread
            float sorted[kCandCap];                  // candidates by rank
        } c;
    } u;
    unsigned long long ent[kCandCap];                // (key << 32) | ~token
    float red[NW], red2[NW];
    unsigned cnt[NW];
    unsigned digit, need, n;
};

__device__ inline float wave_min(float x) { return -wave_max(-x); }

// (m, s) statistics joined across the wave.
__device__ inline void wave_join_ms(float& m, float& s, float scale) {
    const float M = wave_max(m);
    s = wave_sum(m == -kInf ? 0.f : s * fast_exp2((m - M) * scale));
    m = M;
}

// Reductions over the workgroup, in a fixed order.
template <typename Join>
__device__ inline float block_join(float x, float* red, Join join) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    __syncthreads();
    if (lane == 0) red[wave] = x;
    __syncthreads();
    x = red[0];
    for (int w = 1; w < NW; ++w) x = join(x, red[w]);
    return x;
}
__device__ inline float block_sum(float x, float* red) {
    return block_join(wave_sum(x), red, [](float a, float b) { return a + b; });
}
__device__ inline float block_max(float x, float* red) {
    return block_join(wave_max(x), red, [](float a, float b) { return fmaxf(a, b); });
}

// The log-sum-exps from the record's sum (relative to the row's maximum) and
// the rest's (m, s).
__device__ inline void write_lse(const RecordArgs& a, float* olse, float mx, float top, float m, float s) {
    const bool none = m == -kInf || !(s > 0.f);
    const float all = top + (none ? 0.f : s * fast_exp2((m - mx) * a.scale));
    olse[0] = fmaf(mx, a.inv_t, logf(all));
    olse[1] = none ? -kInf : fmaf(m, a.inv_t, logf(s));
}

// Ranks the n distinct entries by counting, writes the first ``keep`` out and
// leaves the values by rank; places behind the V-th get token -1.
__device__ inline void rank_entries(const RecordArgs& a, int n, int keep, int* otok, float* oval,
                                    RecordScratch& sc) {
    if (n > kSortFrom) {
        // many: every wave sorts 64 entries in registers, largest first, and an entry's rank is
        // its place in its own list plus, by binary search, its places in the others
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, lists = (n + kWave - 1) / kWave;
        constexpr int kOwn = kCandCap / NT;                           // lists of a wave
        unsigned long long own[kOwn];
#pragma unroll
        for (int u = 0; u < kOwn; ++u) {
            const int l = wave + u * NW, t = l * kWave + lane;
            if (l >= lists) break;
            unsigned long long e = t < n ? sc.ent[t] : 0;
#pragma unroll 1
            for (int k = 2; k <= kWave; k *= 2)
#pragma unroll 1
                for (int d = k / 2; d > 0; d /= 2) {
                    const unsigned long long o = __shfl_xor(e, d);
                    const bool larger = ((lane & d) == 0) == ((lane & k) == 0);    // which of the two stays here
                    e = (e > o) == larger ? e : o;
                }
            own[u] = e;
            sc.ent[t] = e;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kOwn; ++u) {
            const int l = wave + u * NW;
            if (l >= lists || own[u] == 0) break;
            int rank = lane;
#pragma unroll 4
            for (int q = 0; q < lists; ++q) {
                const unsigned long long* o = sc.ent + q * kWave;
                int at = 0;                                           // entries of the list that are larger
#pragma unroll
                for (int d = kWave / 2; d > 0; d /= 2) at += o[at + d - 1] > own[u] ? d : 0;
                at += o[at] > own[u];
                rank += q == l ? 0 : at;
            }
            const float x = key_value((unsigned)(own[u] >> 32));
            if (rank < keep) {
                otok[rank] = (int)~(unsigned)own[u];
                oval[rank] = x;
            }
            sc.u.c.sorted[rank] = x;
        }
        n = 0;                                                        // done
    }
    // an entry is compared by ``parts`` neighbouring lanes, as many as there are threads for
    int parts = 1;
    while (parts < 16 && n * parts * 2 <= NT) parts *= 2;
    for (int x0 = 0; x0 < n * parts; x0 += NT) {
        const int t = (x0 + (int)threadIdx.x) / parts;
        const unsigned long long e = t < n ? sc.ent[t] : 0;
        int rank = 0;
        if (t < n) {
            int k = (int)threadIdx.x % parts;
            for (; k + 7 * parts < n; k += 8 * parts) {
                unsigned long long o[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) o[u] = sc.ent[k + u * parts];
#pragma unroll
                for (int u = 0; u < 8; ++u) rank += o[u] > e;
            }
            for (; k < n; k += parts) rank += sc.ent[k] > e;
        }
        for (int d = 1; d < parts; d *= 2) rank += __shfl_xor(rank, d);
        if (t < n && threadIdx.x % parts == 0) {
            const float x = key_value((unsigned)(e >> 32));
            if (rank < keep) {
                otok[rank] = (int)~(unsigned)e;
                oval[rank] = x;
            }
            sc.u.c.sorted[rank] = x;
        }
    }
    for (int k = min(a.K, a.V) + (int)threadIdx.x; k < a.K; k += NT) {
        otok[k] = -1;
        oval[k] = -kInf;
    }
    __syncthreads();
}

// f(token, logit, whether there is one) for every entry of a row, by the whole
// workgroup; all lanes of a wave call f together.
template <bool BF16, typename F>
__device__ __forceinline__ void each_entry(const RecordArgs& a, const void* row, F f) {
    constexpr int G = RowGroup<BF16>::G;
    const int full = a.V / G, groups = (a.V + G - 1) / G;
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += NT) {
        const int g = g0 + (int)threadIdx.x;
        RowGroup<BF16> x;
        x.issue(row, g, full);
        x.finish(row, g, full, a.V);
#pragma unroll
        for (int e = 0; e < G; ++e) f(g * G + e, x.elem(e), g * G + e < a.V);
    }
}

// The record of a row whose candidates are too many (values equal or nearly
// so, or unevenly spread): the K-th largest value by a radix select on order
// keys, digit by digit over the row, then the entries above it and the first
// of those equal to it.  Whole workgroup; mx is the row's maximum.
template <bool BF16>
__device__ __forceinline__ void record_by_digits(const RecordArgs& a, const void* row, int K, float mx, int* otok,
                                              float* oval, float* olse, RecordScratch& sc) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    // radix select of the K-th largest key
    unsigned prefix = 0, mask = 0;
    unsigned need = (unsigned)K;                   // its rank among the keys that match the prefix
    for (int d = 0; d < 3; ++d) {
        const int bits = d < 2 ? 11 : 10, shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        __syncthreads();
        for (int k = tid; k < kBins; k += NT) sc.u.hist[k] = 0;
        __syncthreads();
        each_entry<BF16>(a, row, [&](int, float x, bool in) {
            const unsigned key = order_key(x);
            in = in && (key & mask) == prefix;
            const unsigned digit = (key >> shift) & ((1u << bits) - 1);
            // the first lane's digit in one addition: rows of few values would queue up at one bin
            const unsigned long long on = __ballot(in);
            if (!on) return;
            const unsigned d0 = __builtin_amdgcn_readlane(digit, __builtin_ctzll(on));
            const unsigned long long same = __ballot(in && digit == d0);
            if (lane == 0) atomicAdd(&sc.u.hist[d0], (unsigned)__popcll(same));
            if (in && digit != d0) atomicAdd(&sc.u.hist[digit], 1u);
        });
        __syncthreads();
        // the bin that holds the need-th key from the top: four bins a thread, the highest first
        int c[kBins / NT], mine = 0;
#pragma unroll
        for (int u = 0; u < kBins / NT; ++u) {
            c[u] = (int)sc.u.hist[kBins - 1 - (tid * (kBins / NT) + u)];
            mine += c[u];
        }
        const int incl = wave_scan_incl(mine);
        if (lane == kWave - 1) sc.cnt[wave] = (unsigned)incl;
        __syncthreads();
        int before = incl - mine;
        for (int w = 0; w < wave; ++w) before += (int)sc.cnt[w];
        if (before < (int)need && before + mine >= (int)need) {
            int left = (int)need - before, u = 0;
#pragma unroll
            for (int k = 0; k < kBins / NT - 1; ++k)
                if (u == k && c[k] < left) {
                    left -= c[k];
                    ++u;
                }
            sc.digit = (unsigned)(kBins - 1 - (tid * (kBins / NT) + u));
            sc.need = (unsigned)left;
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
    if (tid == 0) sc.n = 0;
    __syncthreads();
    float s = 0.f, below = -kInf;
    unsigned ties = 0;
    each_entry<BF16>(a, row, [&](int v, float x, bool in) {
        if (!in) return;
        const unsigned key = order_key(x);
        if (key > kth) {
            sc.ent[atomicAdd(&sc.n, 1u)] = ((unsigned long long)key << 32) | ~(unsigned)v;
        } else if (key == kth) {
            ++ties;
        } else {
            s += fast_exp2((x - zk) * a.scale);
            below = fmaxf(below, x);
        }
    });
    float rest = block_sum(s, sc.red) + (block_sum((float)ties, sc.red2) - (float)need);
    float ref = zk;
    if (rest == 0.f) {
        // nothing left, or all of it too far below: sum again from the largest of the rest
        below = block_max(below, sc.red);
        if (below > -kInf) {
            ref = below;
            s = 0.f;
            for (int v = tid; v < a.V; v += NT) {
                const float x = load_elem<BF16>(row, v);
                if (order_key(x) < kth) s += fast_exp2((x - ref) * a.scale);
            }
            rest = block_sum(s, sc.red);
        }
    }
    // ties in token order
    const unsigned above = (unsigned)K - need;
    unsigned taken = 0;
    for (int v0 = 0; v0 < a.V && taken < need; v0 += NT) {
        const int v = v0 + tid;
        const bool tie = v < a.V && order_key(load_elem<BF16>(row, v)) == kth;
        const unsigned long long m = __ballot(tie);
        __syncthreads();
        if (lane == 0) sc.cnt[wave] = __popcll(m);
        __syncthreads();
        unsigned before = taken;
        for (int w = 0; w < NW; ++w) {
            if (w < wave) before += sc.cnt[w];
            taken += sc.cnt[w];
        }
        const unsigned my = before + __popcll(m & ((1ull << lane) - 1));
        if (tie && my < need) sc.ent[above + my] = ((unsigned long long)kth << 32) | ~(unsigned)v;
    }
    __syncthreads();
    rank_entries(a, K, K, otok, oval, sc);
    const float top = block_sum(tid < K ? fast_exp2((sc.u.c.sorted[tid] - mx) * a.scale) : 0.f, sc.red);
    if (tid == 0) write_lse(a, olse, mx, top, zk == -kInf ? -kInf : ref, rest);
}

// A record by one workgroup per row, one pass over the row.
//
// Thread t takes blocks of ``a.reps`` times four 16-byte groups (neighbouring
// threads neighbouring groups) and leaves of each block its maximum and the
// sum of its exponentials relative to it.  With k a wave's share of K (by the
// groups it holds, rounded up), the k-th largest of its lanes' maxima (two a
// lane) bounds k entries from below, so the smallest of the waves' bounds is
// one for the K-th largest entry, L.  Only blocks whose maximum reaches L are read again
// (from cache; 1.2 to 1.6 K of them on ordinary rows): their entries from L
// on are the candidates, ranked by counting, and the sums of the other
// blocks, the smaller entries and the candidates behind the K-th make the
// rest.  Loops are kept rolled: a row is one short run through this code, and
// straight-line code costs an instruction fetch from L2 every 64 bytes.
template <bool BF16>
__global__ __launch_bounds__(NT) void k_top_logits(RecordArgs a) {
    constexpr int G = RowGroup<BF16>::G;
    __shared__ RecordScratch sc;
    extern __shared__ float2 stat[];                // [block][thread]: maximum, sum
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int b = blockIdx.x / a.n, i = blockIdx.x % a.n;
    const void* row = row_ptr<BF16>(a.in, a.sb, a.sp, b, i);
    int* otok = a.tok + (long long)blockIdx.x * a.K;
    float* oval = a.val + (long long)blockIdx.x * a.K;
    float* olse = a.lse + (long long)blockIdx.x * 2;
    const int K = min(a.K, a.V), full = a.V / G, groups = (a.V + G - 1) / G;
    const int steps = a.blocks * a.reps;            // of kLoads * NT groups
    const int whole = full / (kLoads * NT);         // steps that every thread has groups for
    if (tid == 0) sc.n = 0;

    // the blocks' statistics
    float key0 = -kInf, key1 = -kInf;               // the lane's maxima over even and odd blocks
    bool bad = false;
    float bm = -kInf, bs = 0.f;
    int rep = 0, blk = 0;
    RowGroup<BF16> r[kLoads], nx[kLoads];
    const auto issue = [&](int t) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) nx[l].issue(row, (t * kLoads + l) * NT + tid, full);
    };
    issue(0);
    for (int t = 0; t < steps; ++t) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) r[l] = nx[l];
        if (t + 1 < steps) issue(t + 1);            // the next step's loads over this one's sums
        if (t >= whole) {
#pragma unroll
            for (int l = 0; l < kLoads; ++l) r[l].clear((t * kLoads + l) * NT + tid, full);
        }
        float m = -kInf;
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
#pragma unroll
            for (int e = 0; e < G; ++e) m = fmaxf(m, r[l].elem(e));
        float s = sum_exp<kLoads>(r, ExpRef(m, a.scale));
        if (t >= whole && full * G < a.V && full >= t * kLoads * NT && (full - t * kLoads * NT) % NT == tid) {
            // the row's last, partial group: its place was cleared above
#pragma unroll 1
            for (int v = full * G; v < a.V; ++v) {
                const float x = load_elem<BF16>(row, v);
                bad |= x != x || x == kInf;
                merge_ms(m, s, x, x == -kInf ? 0.f : 1.f, a.scale);
            }
        }
        if (rep == 0) {
            bm = m;
            bs = s;
        } else {
            merge_ms(bm, bs, m, s, a.scale);
        }
        if (++rep == a.reps) {
            stat[blk * NT + tid] = make_float2(bm, bs);
            bad |= bs != bs;                        // NaN or +inf in the block
            if (blk & 1) key1 = fmaxf(key1, bm);
            else key0 = fmaxf(key0, bm);
            rep = 0;
            ++blk;
        }
    }

    // the bound: 16 bits of the wave's k-th largest lane maximum, k its share
    // of K by the groups it holds (rounded up), then the smallest of the waves'
    const int held = groups / NT * kWave + min(max(groups % NT - wave * kWave, 0), kWave);
    const int k_wave = (int)(((long long)K * held + groups - 1) / groups);
    const unsigned u0 = order_key(key0) >> 16, u1 = order_key(key1) >> 16;
    // (bits that all lanes share need no count)
    float mx = wave_max(fmaxf(key0, key1));
    const unsigned hi = order_key(mx) >> 16;
    const unsigned lo = order_key(wave_min(a.blocks > 1 ? fminf(key0, key1) : key0)) >> 16;
    unsigned bit = 0x8000u, bound = 0;
    if (k_wave <= (a.blocks > 1 ? 2 * kWave : kWave)) {
        bit = hi == lo ? 0u : 0x80000000u >> __builtin_clz(hi ^ lo);
        bound = hi & ~(2 * bit - 1);
        if (hi == lo) bound = hi;
    }
#pragma unroll 1
    for (; bit; bit >>= 1) {
        const unsigned c = bound | bit;
        if (__popcll(__ballot(u0 >= c)) + __popcll(__ballot(u1 >= c)) >= k_wave) bound = c;
    }
    if (k_wave == 0) bound = 0xFFFFu;
    const bool wave_bad = __ballot(bad) != 0;
    if (lane == 0) {
        sc.red[wave] = mx;
        sc.cnt[wave] = wave_bad ? 0xFFFFFFFFu : bound;
    }
    __syncthreads();
    mx = wave_max(lane < NW ? sc.red[lane] : -kInf);
    const unsigned wb = lane < NW ? sc.cnt[lane] : 0xFFFFu;
    bad = __ballot(wb == 0xFFFFFFFFu) != 0;
    bound = (unsigned)wave_min_int((int)(wb & 0x7FFFFFFFu));
    if (bad || mx == -kInf) {
        for (int k = tid; k < a.K; k += NT) {
            otok[k] = -1;
            oval[k] = -kInf;
        }
        if (tid < 2) olse[tid] = __builtin_nanf("");
        return;
    }
    const float L = key_value(max(bound << 16, kLowestFinite));      // -inf entries are no candidates

    // the wave's blocks with candidates, and the sums of the others
    float2 st[kMaxBlocks];
    float m = -kInf, s = 0.f;
    int n_blk = 0;
#pragma unroll
    for (int q = 0; q < kMaxBlocks; ++q) st[q] = q < a.blocks ? stat[q * NT + tid] : make_float2(-kInf, 0.f);
#pragma unroll
    for (int q = 0; q < kMaxBlocks; ++q) {
        const bool in = st[q].x >= L;
        const unsigned long long set = __ballot(in);
        if (in) {
            const int at = n_blk + __popcll(set & ((1ull << lane) - 1));
            if (at < kWaveBlk) sc.u.c.blk[wave][at] = (unsigned short)(q * NT + tid);
            st[q] = make_float2(-kInf, 0.f);
        }
        m = fmaxf(m, st[q].x);
        n_blk += __popcll(set);
    }
    const float ref = m == -kInf ? 0.f : m;
#pragma unroll
    for (int q = 0; q < kMaxBlocks; ++q) s += st[q].y * fast_exp2((st[q].x - ref) * a.scale);
    const int per_blk = kLoads * a.reps;
    if (n_blk > kWaveBlk) {
        if (lane == 0) atomicAdd(&sc.n, kCandCap + 1u);              // too many: the other way, below
    } else {
        const int reads = n_blk * per_blk;
        const auto group = [&](int k) {                              // the k-th group to read, past the end: none
            if (k >= reads) return groups;
            const int q = a.reps == 1 ? k / kLoads : k / per_blk;
            const int id = sc.u.c.blk[wave][q];
            return ((id / NT) * per_blk + k - q * per_blk) * NT + id % NT;
        };
        int next = group(lane);
        RowGroup<BF16> nx;
        nx.issue(row, next, full);
#pragma unroll 1
        for (int k0 = 0; k0 < reads; k0 += kWave) {
            const int g = next;
            RowGroup<BF16> x = nx;
            if (k0 + kWave < reads) {
                next = group(k0 + kWave + lane);
                nx.issue(row, next, full);
            }
            x.finish(row, g, full, a.V);                             // past the end: -inf
            unsigned in = 0;
#pragma unroll
            for (int e = 0; e < G; ++e) in |= x.elem(e) >= L ? 1u << e : 0u;
            const int mine = __popc(in), incl = wave_scan_incl(mine);
            unsigned base = 0;
            if (lane == kWave - 1 && incl) base = atomicAdd(&sc.n, (unsigned)incl);
            unsigned slot = __builtin_amdgcn_readlane(base, kWave - 1) + (unsigned)(incl - mine);
            for (unsigned left = in; left; left &= left - 1) {       // mostly one
                const int e = __builtin_ctz(left);
                if (slot < kCandCap)
                    sc.ent[slot] = ((unsigned long long)order_key(x.elem_dyn(e)) << 32) | ~(unsigned)(g * G + e);
                ++slot;
            }
            RowGroup<BF16> y[1] = {x};
            leave_out(y[0], in);
            float gm = -kInf;
#pragma unroll
            for (int e = 0; e < G; ++e) gm = fmaxf(gm, y[0].elem(e));
            const float gs = sum_exp<1>(y, ExpRef(gm, a.scale));
            merge_ms(m, s, gm, gs, a.scale);
        }
    }
    wave_join_ms(m, s, a.scale);
    __syncthreads();                                                 // sc.red and sc.cnt have been read
    if (lane == 0) {
        sc.red[wave] = m;
        sc.red2[wave] = s;
    }
    const int n = (int)sc.n;
    if (n > kCandCap) {
        record_by_digits<BF16>(a, row, K, mx, otok, oval, olse, sc);
        return;
    }
    rank_entries(a, n, min(n, K), otok, oval, sc);                   // ends with a barrier
    if (wave == 0) {
        if (n < K) {
            // fewer finite logits than K: the first tokens at -inf, all within the first K
            int taken = n;
            for (int v0 = 0; v0 < K; v0 += kWave) {
                const bool empty = v0 + lane < K && load_elem<BF16>(row, v0 + lane) == -kInf;
                const unsigned long long set = __ballot(empty);
                const int my = taken + __popcll(set & ((1ull << lane) - 1));
                if (empty && my < K) {
                    otok[my] = v0 + lane;
                    oval[my] = -kInf;
                }
                taken += __popcll(set);
            }
        }
        // the record's sum; candidates behind the K-th belong to the rest
        float top = 0.f;
        m = lane < NW ? sc.red[lane] : -kInf;
        s = lane < NW ? sc.red2[lane] : 0.f;
#pragma unroll 1
        for (int k = lane; k < n; k += kWave) {
            const float x = sc.u.c.sorted[k];
            if (k < K) top += fast_exp2((x - mx) * a.scale);
            else merge_ms(m, s, x, 1.f, a.scale);
        }
        top = wave_sum(top);
        wave_join_ms(m, s, a.scale);
        if (lane == 0) write_lse(a, olse, mx, top, m, s);
    }
}

}  // namespace

hipError_t launch_top_logits(const RecordArgs& a, bool bf16, hipStream_t stream, hipEvent_t* ev) {
    const long long rows = (long long)a.B * a.n;
    RecordArgs r = a;
    const int step = NT * kLoads * (bf16 ? 8 : 4), steps = (a.V - 1) / step + 1;
    r.reps = (steps - 1) / kMaxBlocks + 1;
    r.blocks = (steps - 1) / r.reps + 1;
    const size_t lds = (size_t)r.blocks * NT * sizeof(float2);       // at most 32 KB
    auto fn = bf16 ? k_top_logits<true> : k_top_logits<false>;
    if (ev)
        hipExtLaunchKernelGGL(fn, dim3((unsigned)rows), dim3(NT), lds, stream, ev[0], ev[1], 0, r);
    else
        hipLaunchKernelGGL(fn, dim3((unsigned)rows), dim3(NT), lds, stream, r);
    return hipGetLastError();
}

}  // namespace specv
