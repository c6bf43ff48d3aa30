// moe_sample.cu -- a token for each row of logits, by given random numbers (moe_sample).
//
//   w_i = exp((l_i - max) / t);  tokens in order: larger logit first, then smaller index
//   k-th token, then the first at which sum w >= top_p * (sum up to there), then the
//   first at which sum w > u * (sum up to there)
//
// All three are one question: the first token, in order, at which a sum over the order
// reaches a target, so no sort is needed.  Tokens are dealt into bins that keep the
// order (2048 equal parts of the logits' range), a bin's tokens are counted and their
// weights added up, a scan over the bins finds the target's, and only that bin's
// tokens (or all up to it, where those are few) are looked at one by one.
//
// Weights are whole numbers, in units of 2^-45 (the largest token weighs 2^45, 2^18 of
// them fit 64 bits): sums do not depend on the order of additions, so atomics give
// the same bits every run, and borders are compared exactly.  A weight is
// 2^-x, x = (max - l) log2(e) / t in two floats: 2^-(j / 64) from a table, the rest, below
// 1/128, by its series; off by 2^-36 of itself.  (fp32 would be off by 2^-24, and one
// row in a thousand would get another token than the formula says.)
//
// A row belongs to a cluster of blocks, each with a part of the row in shared
// memory, so that logits are read once; the blocks add up their bins through
// distributed shared memory and the first one decides.
#include "moe_internal.h"
#include "moe_layer_internal.h"

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

namespace moe {
namespace {
#include "moe_device.cuh"
#include "moe_layer_device.cuh"

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048, kPer = kBins / kThreads;  // bins of a pass over a row; of a thread
constexpr int kList = 2048;                           // tokens that are looked at one by one
constexpr int kFew = 32;                              // tokens that one warp orders
constexpr int kMaxCluster = 8;
constexpr int kOne = 45;                              // a weight of 1 is 2^45
constexpr float kGreedy = 1e-6f;

// A token's place in the order: its bin, its logit as an integer (larger logits
// smaller), its index.  Unique, so ties need no case of their own.
constexpr int kIdxBits = 18, kBinShift = kIdxBits + 32;
static_assert(1 << kIdxBits == MOE_SAMPLE_MAX_VOCAB, "an index fits its bits");

// 2^(-j / 64) in units of 2^-61, by exp's series.
struct Powers {
    u64 v[64];
};
constexpr Powers make_powers()
{
    Powers t{};
    for (int j = 0; j < 64; ++j) {
        const double x = -0.69314718055994530942 * j / 64;
        double term = 1, sum = 1;
        for (int i = 1; i < 30; ++i) {
            term *= x / i;
            sum += term;
        }
        t.v[j] = static_cast<u64>(sum * 2305843009213693952.0 + 0.5);
    }
    return t;
}
__device__ const Powers kPowers = make_powers();

struct Control {
    u64 klo, khi;                  // what the cluster is asked to look at
    int op, shift;
    u64 mn, mx;                    // smallest and largest place in range (first: best order and index, last order)
    int n;                         // tokens in the list
    u64 powers[64];
    u64 scan_w[kWarps];
    uint32_t scan_n[kWarps];
    u64 red[2 * kWarps];
    // a target's bin, or its token
    int bin;
    u64 base_w, key_found, w_found;
    uint32_t base_n, bin_n;
    int few;
    int small[kFew];
};
enum Op { kDone, kRange, kHist, kGather };

// ---- cluster
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster, and what they wrote to any block's shared memory.
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of p (in this block's shared memory) in block r's.
__device__ __forceinline__ uint32_t map_rank(const void *p, uint32_t r)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(r));
    return a;
}
__device__ __forceinline__ uint32_t remote32(const void *p, uint32_t r)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(p, r)) : "memory");
    return v;
}
__device__ __forceinline__ u64 remote64(const void *p, uint32_t r)
{
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_rank(p, r)) : "memory");
    return v;
}

// ---- a row's settings and what its tokens weigh
struct Row {
    float max, ch, cl, bins;  // 1 / t in units of log2(e), two floats; bins for a unit of x
    bool infinite;            // the largest logit is +infinity
    u64 least;                // min-p's least weight (1: any)
};

// A logit as it counts: NaN as -infinity, -0 as 0.
__device__ __forceinline__ float clean(float l) { return l == l ? l + 0.f : -INFINITY; }
__device__ __forceinline__ float counted(const Row &r, float l)
{
    return r.infinite ? (l == INFINITY ? 0.f : -INFINITY) : l;
}
__device__ __forceinline__ uint32_t order_of(float l)
{
    const uint32_t u = __float_as_uint(l);
    return ~(u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u));
}
__device__ __forceinline__ float logit_of(uint32_t order)
{
    const uint32_t u = ~order;
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// x = (max - l) log2(e) / t as p + e.  p falls as l grows (every step of it rounds).
__device__ __forceinline__ void exponent(const Row &r, float l, float &p, float &e)
{
    const float d = r.max - l, bb = d - r.max;
    const float dl = (r.max - (d - bb)) + (-l - bb);  // d + dl = max - l
    p = d * r.ch;
    e = fmaf(d, r.ch, -p) + fmaf(d, r.cl, dl * r.ch);
}
constexpr float kNone = 46.5f;  // 2^-46.5 rounds to nothing

// 2^-(p + e) in units of 2^-45.
__device__ __forceinline__ u64 weight(const u64 *powers, float p, float e)
{
    if (!(p < kNone)) return 0ull;
    const float kf = fmaf(p, 64.f, 12582912.f);  // the nearest whole number, in the low bits
    const int j = __float_as_int(kf) - 0x4B400000;
    const float r = fmaf(kf - 12582912.f, -1.f / 64.f, p);
    // 2^-(r + e) - 1 = s - y - ye
    const float y = r * 0.693147182f, ye = fmaf(r, 0.693147182f, -y) + fmaf(r, -1.90465421e-9f, e * 0.693147182f);
    const float z = y + ye, s = z * z * (0.5f - z * (1.f / 6.f - z * (1.f / 24.f)));
    const int dq = __float2int_rn(y * -274877906944.f) + __float2int_rn((s - ye) * 274877906944.f);  // in units of 2^-38
    const u64 t = powers[j & 63];
    const u64 w = t + static_cast<u64>((static_cast<long long>(static_cast<int>(t >> 31)) * dq) >> 7);
    const int n = (61 - kOne) + (j >> 6);
    return (w + (1ull << (n - 1))) >> n;
}

__device__ __forceinline__ u64 place(const Row &r, float p, float l, int idx)
{
    const int bin = min(kBins - 1, static_cast<int>(p * r.bins));
    return static_cast<u64>(bin) << kBinShift | static_cast<u64>(order_of(l)) << kIdxBits | static_cast<u64>(idx);
}

// floor(f * z), and whether that is all of it; f in [0, 1).
__device__ __forceinline__ u64 part_of(float f, u64 z, bool &exact)
{
    const uint32_t u = __float_as_uint(f), ex = u >> 23;
    const u64 m = ex ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;
    const int s = ex ? 150 - static_cast<int>(ex) : 149;  // f = m 2^-s, s >= 24
    const u64 lo = m * z, hi = __umul64hi(m, z);
    if (s >= 128) {
        exact = (lo | hi) == 0;
        return 0;
    }
    if (s >= 64) {
        exact = lo == 0 && (hi & ((1ull << (s - 64)) - 1)) == 0;
        return hi >> (s - 64);
    }
    exact = (lo & ((1ull << s) - 1)) == 0;
    return lo >> s | hi << (64 - s);
}

// ---- the block
__device__ __forceinline__ u64 warp_min(u64 v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// The smallest a and the largest b of the block (all threads get them).
__device__ __forceinline__ void block_range(Control *ct, u64 &a, u64 &b)
{
    const int w = threadIdx.x >> 5;
    a = warp_min(a);
    b = ~warp_min(~b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        ct->red[2 * w] = a;
        ct->red[2 * w + 1] = b;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        a = min(a, ct->red[2 * i]);
        b = max(b, ct->red[2 * i + 1]);
    }
}
// Sums over the threads before this one; the block's sums in total.
__device__ __forceinline__ void block_scan(Control *ct, u64 w, uint32_t n, u64 &before_w, uint32_t &before_n, u64 &all_w,
                                           uint32_t &all_n)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    u64 sw = w;
    uint32_t sn = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 a = __shfl_up_sync(0xffffffffu, sw, o);
        const uint32_t c = __shfl_up_sync(0xffffffffu, sn, o);
        if (lane >= o) sw += a, sn += c;
    }
    __syncthreads();
    if (lane == 31) {
        ct->scan_w[wid] = sw;
        ct->scan_n[wid] = sn;
    }
    __syncthreads();
    before_w = sw - w, before_n = sn - n;
    all_w = 0, all_n = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i == wid) before_w += all_w, before_n += all_n;
        all_w += ct->scan_w[i];
        all_n += ct->scan_n[i];
    }
}

// A part of a row, and the bins and the list beside it.
template <typename IN>
struct Part {
    const IN *l;  // the part's logits, in shared memory
    int n, first; // how many; the first one's index in the row
    uint32_t *lo, *hi, *cnt;  // [kBins] weights in two words, tokens
    u64 *list, *list_w;       // [kList] places; weights (of the first block)
    __device__ __forceinline__ float logit(int i) const;
};
template <>
__device__ __forceinline__ float Part<float>::logit(int i) const { return clean(l[i]); }
template <>
__device__ __forceinline__ float Part<uint16_t>::logit(int i) const { return clean(__uint_as_float(static_cast<uint32_t>(l[i]) << 16)); }

__device__ __forceinline__ void add_weight(uint32_t *lo, uint32_t *hi, uint32_t *cnt, int bin, u64 w)
{
    const uint32_t a = static_cast<uint32_t>(w), old = atomicAdd(lo + bin, a);
    const uint32_t b = static_cast<uint32_t>(w >> 32) + (old + a < old ? 1u : 0u);
    if (b) atomicAdd(hi + bin, b);
    atomicAdd(cnt + bin, 1u);
}

// f(place, p, e) for each token of the part that is not masked and whose place is in [klo, khi].
template <typename IN, typename F>
__device__ __forceinline__ void each(const Part<IN> &pt, const Row &r, u64 klo, u64 khi, F f)
{
    for (int i = threadIdx.x; i < pt.n; i += kThreads) {
        const float l = counted(r, pt.logit(i));
        if (l == -INFINITY) continue;
        float p, e;
        exponent(r, l, p, e);
        if (!(p < kNone)) continue;
        const u64 k = place(r, p, l, pt.first + i);
        if (k >= klo && k <= khi) f(k, p, e);
    }
}

// Tokens of places in [klo, khi] into bins of 2^shift places from klo on; the cluster's
// sums end in the first block's bins.
template <typename IN>
__device__ __forceinline__ void histogram(const Part<IN> &pt, const Row &r, Control *ct, u64 klo, u64 khi, int shift, int rank,
                                          int blocks)
{
    const int tid = threadIdx.x;
    for (int i = tid; i < kBins; i += kThreads) pt.lo[i] = pt.hi[i] = pt.cnt[i] = 0u;
    __syncthreads();
    each(pt, r, klo, khi, [&](u64 k, float p, float e) {
        const u64 w = weight(ct->powers, p, e);
        if (w != 0 && w >= r.least) add_weight(pt.lo, pt.hi, pt.cnt, static_cast<int>((k - klo) >> shift), w);
    });
    cluster_sync();
    if (blocks == 1) return;
    // each block adds up a share of the bins, in its own place for them (which no other reads)
    const int share = kBins / blocks;
    for (int i = rank * share + tid; i < (rank + 1) * share; i += kThreads) {
        u64 w = 0;
        uint32_t n = 0;
        for (int x = 0; x < blocks; ++x) {
            w += static_cast<u64>(remote32(pt.hi + i, x)) << 32;
            w += remote32(pt.lo + i, x);
            n += remote32(pt.cnt + i, x);
        }
        pt.lo[i] = static_cast<uint32_t>(w);
        pt.hi[i] = static_cast<uint32_t>(w >> 32);
        pt.cnt[i] = n;
    }
    cluster_sync();
    if (rank != 0) return;
    for (int i = share + tid; i < kBins; i += kThreads) {
        const int x = i / share;
        pt.lo[i] = remote32(pt.lo + i, x);
        pt.hi[i] = remote32(pt.hi + i, x);
        pt.cnt[i] = remote32(pt.cnt + i, x);
    }
    __syncthreads();
}

// What the cluster does for the first block's question (all of its threads, after it was put).
template <typename IN>
__device__ __forceinline__ void answer(const Part<IN> &pt, const Row &r, Control *ct, int op, u64 klo, u64 khi, int shift, int rank,
                                       int blocks)
{
    const int tid = threadIdx.x;
    if (op == kRange) {
        u64 a = ~0ull, b = 0ull;
        each(pt, r, klo, khi, [&](u64 k, float p, float e) {
            const u64 w = weight(ct->powers, p, e);
            if (w != 0 && w >= r.least) a = min(a, k), b = max(b, k);
        });
        block_range(ct, a, b);
        if (tid == 0) ct->mn = a, ct->mx = b;
        cluster_sync();
        if (rank == 0) {
            for (int x = 1; x < blocks; ++x) a = min(a, remote64(&ct->mn, x)), b = max(b, remote64(&ct->mx, x));
            __syncthreads();
            if (tid == 0) ct->mn = a, ct->mx = b;
            __syncthreads();
        }
    } else if (op == kHist) {
        histogram(pt, r, ct, klo, khi, shift, rank, blocks);
    } else {
        if (tid == 0) ct->n = 0;
        __syncthreads();
        each(pt, r, klo, khi, [&](u64 k, float p, float e) {
            const u64 w = weight(ct->powers, p, e);
            if (w != 0 && w >= r.least) {
                const int at = atomicAdd(&ct->n, 1);
                if (at < kList) pt.list[at] = k;
            }
        });
        cluster_sync();
        if (rank == 0) {
            int n = min(ct->n, kList);
            for (int x = 1; x < blocks; ++x) {
                const int m = min(static_cast<int>(remote32(&ct->n, x)), kList - n);
                for (int i = tid; i < m; i += kThreads) pt.list[n + i] = remote64(pt.list + i, x);
                n += m;
            }
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                float p, e;
                exponent(r, logit_of(static_cast<uint32_t>(pt.list[i] >> kIdxBits)), p, e);
                pt.list_w[i] = weight(ct->powers, p, e);
            }
            if (tid == 0) ct->n = n;
            __syncthreads();
        }
    }
}

// ---- the first block's decisions
struct Found {
    u64 key, w, upto;  // the token's place and weight, the weights up to it (it included)
};

template <typename IN>
struct Chooser {
    const Part<IN> &pt;
    const Row &r;
    Control *ct;
    int blocks;
    u64 w[kPer], before_w, all_w;  // the thread's bins of the first pass
    uint32_t n[kPer], before_n, all_n;
    u64 glo = 1, ghi = 0;          // places that the list covers (none)

    __device__ __forceinline__ void ask(int op, u64 klo, u64 khi, int shift)
    {
        if (threadIdx.x == 0) ct->op = op, ct->klo = klo, ct->khi = khi, ct->shift = shift;
        cluster_sync();
        answer(pt, r, ct, op, klo, khi, shift, 0, blocks);
    }

    // Bins of the last pass, four a thread.
    __device__ __forceinline__ void load_bins(u64 (&bw)[kPer], uint32_t (&bn)[kPer], u64 &bef_w, uint32_t &bef_n, u64 &tot_w,
                                              uint32_t &tot_n)
    {
        u64 sw = 0;
        uint32_t sn = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const int i = kPer * threadIdx.x + q;
            bw[q] = static_cast<u64>(pt.hi[i]) << 32 | pt.lo[i];
            bn[q] = pt.cnt[i];
            sw += bw[q];
            sn += bn[q];
        }
        block_scan(ct, sw, sn, bef_w, bef_n, tot_w, tot_n);
    }

    // The bin at which the sums before it (base) and in order reach t.
    template <int Q>
    __device__ __forceinline__ void find_bin(const u64 (&bw)[Q], const uint32_t (&bn)[Q], u64 bef_w, uint32_t bef_n, u64 base_w,
                                             uint32_t base_n, u64 t, bool count)
    {
        u64 cw = base_w + bef_w;
        uint32_t cn = base_n + bef_n;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const u64 a = count ? cn : cw, b = count ? cn + bn[q] : cw + bw[q];
            if (a < t && t <= b) {
                ct->bin = Q * threadIdx.x + q;
                ct->base_w = cw;
                ct->base_n = cn;
                ct->bin_n = bn[q];
            }
            cw += bw[q];
            cn += bn[q];
        }
        __syncthreads();
    }

    // The first token at which the count (or the weights) reaches t, 1 <= t <= all of them.
    __device__ Found find(u64 t, bool count)
    {
        find_bin(w, n, before_w, before_n, 0, 0, t, count);
        u64 klo = static_cast<u64>(ct->bin) << kBinShift, khi = klo + ((1ull << kBinShift) - 1), bw = ct->base_w;
        uint32_t bn = ct->base_n, m = ct->bin_n;
        __syncthreads();
        if (klo < glo || khi > ghi) {
            if (bn + m <= kList) {
                glo = 0;
            } else {
                // many tokens in a bin: parts of its range, until few are left (each round leaves
                // 11 bits less of a place's 64)
                for (int round = 0; m > kList && round < 6; ++round) {
                    ask(kRange, klo, khi, 0);
                    klo = ct->mn;
                    const u64 span = ct->mx - klo;
                    const int shift = max(0, 64 - __clzll(span) - 11);
                    ask(kHist, klo, ct->mx, shift);
                    u64 xw[kPer], xbw, xall;
                    uint32_t xn[kPer], xbn, xalln;
                    load_bins(xw, xn, xbw, xbn, xall, xalln);
                    find_bin(xw, xn, xbw, xbn, bw, bn, t, count);
                    klo += static_cast<u64>(ct->bin) << shift;
                    khi = klo + ((1ull << shift) - 1);
                    bw = ct->base_w, bn = ct->base_n, m = ct->bin_n;
                    __syncthreads();
                }
                glo = klo;
            }
            ghi = khi;
            ask(kGather, glo, ghi, 0);
        }
        return look(klo, khi, bw, bn, t, count);
    }

    // The same among the listed tokens in [klo, khi], with the sums before klo.
    __device__ Found look(u64 klo, u64 khi, u64 bw, uint32_t bn, u64 t, bool count)
    {
        const int tid = threadIdx.x, lane = tid & 31, len = ct->n;
        for (int round = 0;; ++round) {  // (each leaves 9 bits less)
            u64 a = ~0ull, b = 0ull;
            if (tid == 0) ct->few = 0;
            __syncthreads();
            for (int i = tid; i < len; i += kThreads) {
                const u64 k = pt.list[i];
                if (k < klo || k > khi) continue;
                a = min(a, k), b = max(b, k);
                const int at = atomicAdd(&ct->few, 1);
                if (at < kFew) ct->small[at] = i;
            }
            block_range(ct, a, b);
            if (ct->few <= kFew || round == 8) break;
            klo = a;
            const int shift = max(0, 64 - __clzll(b - a) - 9);  // (b - a) >> shift < kThreads
            pt.lo[tid] = pt.hi[tid] = pt.cnt[tid] = 0u;
            __syncthreads();
            for (int i = tid; i < len; i += kThreads) {
                const u64 k = pt.list[i];
                if (k >= klo && k <= khi) add_weight(pt.lo, pt.hi, pt.cnt, static_cast<int>((k - klo) >> shift), pt.list_w[i]);
            }
            __syncthreads();
            const u64 xw[1] = {static_cast<u64>(pt.hi[tid]) << 32 | pt.lo[tid]};
            const uint32_t xn[1] = {pt.cnt[tid]};
            u64 xbw, xall;
            uint32_t xbn, xalln;
            block_scan(ct, xw[0], xn[0], xbw, xbn, xall, xalln);
            find_bin(xw, xn, xbw, xbn, bw, bn, t, count);
            klo += static_cast<u64>(ct->bin) << shift;
            khi = min(khi, klo + ((1ull << shift) - 1));
            bw = ct->base_w, bn = ct->base_n;
            __syncthreads();
        }
        if (tid < 32) {  // a token a lane: the sums up to it, from all that come before
            const int few = min(ct->few, kFew);
            const u64 k = lane < few ? pt.list[ct->small[lane]] : ~0ull, mine = lane < few ? pt.list_w[ct->small[lane]] : 0ull;
            u64 cw = bw;
            uint32_t cn = bn;
            for (int i = 0; i < few; ++i) {
                const u64 ok = __shfl_sync(0xffffffffu, k, i), ow = __shfl_sync(0xffffffffu, mine, i);
                if (ok < k) cw += ow, ++cn;
            }
            const u64 c0 = count ? cn : cw, c1 = count ? cn + 1 : cw + mine;
            if (lane < few && c0 < t && t <= c1) ct->key_found = k, ct->w_found = mine, ct->base_w = cw + mine;
        }
        __syncthreads();
        const Found f{ct->key_found, ct->w_found, ct->base_w};
        __syncthreads();
        return f;
    }
};

struct Params {
    moe_sample_desc d;
    int part;  // logits of a block
};

__device__ __forceinline__ float setting(const float *a, float one, int t) { return a ? a[t] : one; }

template <typename IN>
__global__ void __launch_bounds__(kThreads, 2) moe_sample_kernel(const __grid_constant__ Params p, int blocks)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Control *ct = reinterpret_cast<Control *>(smem);
    u64 *list = reinterpret_cast<u64 *>(smem + (sizeof(Control) + 15) / 16 * 16);
    uint32_t *bins = reinterpret_cast<uint32_t *>(list + 2 * kList);
    IN *buf = reinterpret_cast<IN *>(bins + 3 * kBins);
    const moe_sample_desc &d = p.d;
    const int tid = threadIdx.x, rank = cluster_rank(), t = blockIdx.x / blocks;
    const int first = min(rank * p.part, d.V), n = min(p.part, d.V - first);
    const Part<IN> pt{buf, n, first, bins, bins + kBins, bins + 2 * kBins, list, list + kList};
    if (tid < 64) ct->powers[tid] = kPowers.v[tid];
    grid_wait();
    grid_release();

    // ---- the part's logits; the first in order, the smallest that is not masked
    const IN *src = static_cast<const IN *>(d.logits_dev) + static_cast<long long>(t) * d.stride + first;
    u64 best = ~0ull;
    float low = INFINITY;
    for (int i0 = tid; i0 < n; i0 += 8 * kThreads) {
        IN v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (i0 + x * kThreads < n) v[x] = src[i0 + x * kThreads];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (i0 + x * kThreads < n) {
                const int i = i0 + x * kThreads;
                buf[i] = v[x];
                const float l = pt.logit(i);
                best = min(best, static_cast<u64>(order_of(l)) << kIdxBits | static_cast<u64>(first + i));
                if (l > -INFINITY) low = fminf(low, l);
            }
    }
    u64 last = low == INFINITY ? 0ull : order_of(low);
    block_range(ct, best, last);
    if (tid == 0) ct->mn = best, ct->mx = last;
    cluster_sync();
    for (int x = 0; x < blocks; ++x) {
        best = min(best, remote64(&ct->mn, x));
        last = max(last, remote64(&ct->mx, x));
    }
    Row r;
    r.max = logit_of(static_cast<uint32_t>(best >> kIdxBits));
    const int top = static_cast<int>(best & (MOE_SAMPLE_MAX_VOCAB - 1));
    const float temperature = setting(d.temperature_dev, d.temperature, t);
    const int top_k = d.top_k_dev ? d.top_k_dev[t] : d.top_k;
    const bool nothing = r.max == -INFINITY;
    if (nothing || !(temperature > kGreedy) || top_k == 1) {
        if (rank == 0 && tid == 0) {
            d.token_dev[t] = nothing ? -1 : top;
            if (d.prob_dev) d.prob_dev[t] = nothing ? 0.f : 1.f;
        }
        cluster_sync();  // nobody's shared memory is read any more
        return;
    }
    const double c = 1.4426950408889634074 / static_cast<double>(temperature);
    r.ch = static_cast<float>(c);
    r.cl = static_cast<float>(c - static_cast<double>(r.ch));
    r.infinite = r.max == INFINITY;
    if (r.infinite) r.max = 0.f;
    const float least = setting(d.min_p_dev, d.min_p, t);
    r.least = least > 0.f ? static_cast<u64>(ceil(static_cast<double>(fminf(least, 1.f)) * 35184372088832.0)) : 1ull;
    const float range = r.infinite ? 0.f : fminf((r.max - logit_of(static_cast<uint32_t>(last))) * r.ch, kNone);
    r.bins = range > 0.f ? kBins / range : 0.f;

    histogram(pt, r, ct, 0ull, ~0ull, kBinShift, rank, blocks);
    if (rank != 0) {
        for (;;) {
            cluster_sync();  // a question
            const int op = remote32(&ct->op, 0);
            if (op == kDone) break;
            answer(pt, r, ct, op, remote64(&ct->klo, 0), remote64(&ct->khi, 0), remote32(&ct->shift, 0), rank, blocks);
        }
        cluster_sync();
        return;
    }
    Chooser<IN> ch{pt, r, ct, blocks};
    ch.load_bins(ch.w, ch.n, ch.before_w, ch.before_n, ch.all_w, ch.all_n);
    u64 z = ch.all_w;
    if (top_k > 0 && static_cast<uint32_t>(top_k) < ch.all_n) z = ch.find(top_k, true).upto;
    const float top_p = setting(d.top_p_dev, d.top_p, t);
    if (top_p < 1.f) {
        bool exact = true;
        const u64 f = top_p > 0.f ? part_of(top_p, z, exact) : 0ull;
        z = ch.find(max(1ull, f + (exact ? 0 : 1)), false).upto;
    }
    const float u = d.u_dev[t];
    bool exact;
    const Found f = ch.find(u >= 1.f ? z : (u > 0.f ? min(z, part_of(u, z, exact) + 1) : 1ull), false);
    if (tid == 0) {
        d.token_dev[t] = static_cast<int32_t>(f.key & (MOE_SAMPLE_MAX_VOCAB - 1));
        if (d.prob_dev) d.prob_dev[t] = static_cast<float>(static_cast<double>(f.w) / static_cast<double>(z));
    }
    if (tid == 0) ct->op = kDone;
    cluster_sync();
    cluster_sync();
}

template <typename IN>
cudaError_t launch_in(const moe_sample_desc &d, cudaStream_t st)
{
    int blocks = 1;
    while (blocks < kMaxCluster && d.V > 4096 * blocks) blocks *= 2;
    Params p{d, (d.V + blocks - 1) / blocks};
    const int smem = static_cast<int>((sizeof(Control) + 15) / 16 * 16 + 2 * kList * 8 + 3 * kBins * 4) + (p.part * static_cast<int>(sizeof(IN)) + 15) / 16 * 16;
    auto *fn = moe_sample_kernel<IN>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(d.T * blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, p, blocks);
}

}  // namespace

cudaError_t launch_sample(const moe_sample_desc &d, cudaStream_t st)
{
    return d.bf16 ? launch_in<uint16_t>(d, st) : launch_in<float>(d, st);
}

}  // namespace moe
