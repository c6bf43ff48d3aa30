// moe_sample.cu -- a token for each row of logits, by given random numbers (moe_sample).
//
//   w_i = exp((l_i - max) / t);  tokens in order: larger logit first, then smaller index
//   k-th token, then the first at which sum w >= top_p * (sum up to there), then the
//   first at which sum w > u * (sum up to there)
//
// All three are one question: the first token, in order, at which a sum over the order
// reaches a target, so no sort is needed.  Tokens are dealt into bins that keep the
// order (1024 equal parts of the logits' range), a bin's tokens are counted and their
// weights added up, a scan over the bins finds the target's, and only that bin's
// tokens (or all up to it, where those are few) are looked at one by one.
//
// Weights are whole numbers, in units of 2^-45 (the largest token weighs 2^45, 2^18 of
// them fit 64 bits): sums do not depend on the order of additions, so atomics give
// the same bits every run, and borders are compared exactly.  A weight is
// 2^-x, x = (max - l) log2(e) / t in two floats: 2^-(j / 64) from a table, the rest, below
// 1/128, by its series; off by half a unit and 2^-36 of itself, and from 2^-16 down, where
// most tokens are and 32 bits hold it, by half a unit and 2^-29 of itself: a unit at most.  (fp32 would
// be off by 2^-24, and one row in a thousand would get another token than the formula says.)
//
// A row belongs to a cluster of blocks, each with a part of it; the blocks add up their
// bins through distributed shared memory and the first one decides: it puts questions
// (a range's places, finer bins of it, its tokens), which all answer.  16-bit logits are
// counted by their value first, of which there are few, where a block has many: each
// value is weighed once.
//
// Few rows are bound by latency: one of 65543 fp32 logits takes 21 us with top-k and top-p, of which
// the weights take 5, adding up the bins 3, the list 4, each further target 1.5 (a barrier of the
// cluster takes 0.5); 24 such rows of settings of their own 37 us.  Many rows are bound by the integer
// units (80 operations a weight, 45 a small one), 16-bit ones by the shared memory's atomics (6
// cycles for a warp's): 256 rows of 131075 take 239 us in fp32, 87 us in bf16 (239 us with
// every token weighed), which are two turns of a row an SM: 152 rows take 48 us.  Code that is there
// once matters: with the passes unrolled into each other, 2.5 MB of objects, one
// row took 26 to 30 us, the instruction cache's misses.
#include "moe_internal.h"
#include "moe_layer_internal.h"

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace moe {
namespace {
#include "moe_device.cuh"
#include "moe_layer_device.cuh"

using u64 = unsigned long long;

constexpr int kMaxWarps = 32;
constexpr int kBinBits = 10, kBins = 1 << kBinBits;  // bins of a pass over a row
constexpr int kList = 2048;       // tokens that are looked at one by one
constexpr int kFew = 32;          // tokens that one warp orders
constexpr int kMaxCluster = 8;
constexpr int kOne = 45;          // a weight of 1 is 2^45
constexpr int kCounters = 65536;  // of 16-bit logits by their bits, two to a word
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

// What the first block asks of all: the smallest and largest place in [klo, khi]; bins of
// 2^shift places from klo on; a list of the tokens in [klo, khi]; the sum of the tail.
enum Op { kDone, kRange, kHist, kGather, kTail };

struct Control {
    u64 best[kMaxCluster], last[kMaxCluster];  // of each block: smallest and largest place (first: order) in range
    int ns[kMaxCluster];           // of each block: tokens in its list
    u64 klo, khi;                  // the question, and kRange's answer
    int op, shift;
    int n, all;                    // tokens in the list, tokens that were meant to be
    uint32_t tail[2];              // of each block: what tokens of less than half a unit weigh, in units of 2^-63, low word first
    uint32_t most_tail;            // units that they all together weigh at most; 0: there are none, or it is settled
    float min_p;
    u64 powers[64];                // 2^(-j / 64) in units of 2^-61
    int powers32[64];              // and of 2^-30
    u64 scan_w[kMaxWarps], red[2 * kMaxWarps];
    uint32_t scan_n[kMaxWarps];
    int bin;                       // where a target lies: the bin, its tokens, the sums before it
    uint32_t base_n, bin_n;
    u64 base_w, key_found, w_found;
    int few, small[kFew];
};

// ---- cluster
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// In two halves around a kernel's start: no block's shared memory is touched from
// another before that one runs.
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// All threads of the cluster, and what they wrote to any block's shared memory.
__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
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

__device__ __forceinline__ void put32(const void *p, uint32_t r, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(p, r)), "r"(v) : "memory");
}
__device__ __forceinline__ void put64(const void *p, uint32_t r, u64 v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_rank(p, r)), "l"(v) : "memory");
}

// ---- a row's settings and what its tokens weigh
struct Row {
    float max, ch, cl, bins;  // 1 / t in units of log2(e), two floats; bins for a unit of x
    bool infinite;            // the largest logit is +infinity
    u64 least;                // min-p's least weight (1: any)
};

// A logit as it counts in a row whose largest is +infinity.
__device__ __forceinline__ float as_infinite(float l) { return l == INFINITY ? 0.f : -INFINITY; }
__device__ __forceinline__ uint32_t order_of(float l)
{
    const uint32_t u = __float_as_uint(l + 0.f);  // (-0 is 0)
    return ~(u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u));
}
__device__ __forceinline__ float logit_of(uint32_t order)
{
    const uint32_t u = ~order;
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// The functions of a token's weight and place are worked out in several places and
// have to give the same everywhere: every operation says how it rounds.

// x = (max - l) log2(e) / t as p + e.  p falls as l grows (every step of it rounds).
__device__ __forceinline__ void exponent(const Row &r, float l, float &p, float &e)
{
    const float d = __fsub_rn(r.max, l), bb = __fsub_rn(d, r.max);
    const float dl = __fsub_rn(__fsub_rn(r.max, __fsub_rn(d, bb)), __fadd_rn(l, bb));  // d + dl = max - l
    p = __fmul_rn(d, r.ch);
    e = __fadd_rn(__fmaf_rn(d, r.ch, -p), __fmaf_rn(d, r.cl, __fmul_rn(dl, r.ch)));
}
constexpr float kNone = 46.5f;   // 2^-46.5 rounds to nothing
constexpr float kSmall = 16.f;   // from here on 32 bits are enough
constexpr float kMagic = 12582912.f;        // 1.5 * 2^23: adding it leaves the nearest whole number in the low bits,
constexpr int kMagicBits = 0x4B400000;      // above these

// 2^-(p + e) in units of 2^-ONE, ONE - 29 <= p < ONE + 1.5.
template <int ONE>
__device__ __forceinline__ uint32_t weight32(const Control *ct, float p, float e)
{
    const float kf = __fmaf_rn(p, 64.f, kMagic);
    const int j = __float_as_int(kf) - kMagicBits;
    const float r = __fmaf_rn(__fsub_rn(kf, kMagic), -1.f / 64.f, p);
    const float z = __fmul_rn(__fadd_rn(r, e), 0.693147182f);
    // 2^-(r + e) - 1 = z^2 (1 / 2 - z / 6) - z
    const float s = __fmaf_rn(__fmul_rn(z, z), __fmaf_rn(z, -1.f / 6.f, 0.5f), -z);
    const int dq = __float2int_rn(__fmul_rn(s, 4294967296.f));
    const int t = ct->powers32[j & 63];
    const uint32_t w = static_cast<uint32_t>(t + __mulhi(t, dq));
    const int n = (j >> 6) - (ONE - 30);
    return ((w >> (n - 1)) + 1u) >> 1;
}

// 2^-(p + e) in units of 2^-45, kSmall <= p < kNone (0 for another p).
__device__ __forceinline__ uint32_t small_weight(const Control *ct, float p, float e)
{
    const bool in = p >= kSmall && p < kNone;
    if (!in) p = kSmall, e = 0.f;
    const uint32_t w = weight32<kOne>(ct, p, e);
    return in ? w : 0u;
}

// The same for any p.
__device__ __forceinline__ u64 weight(const Control *ct, float p, float e)
{
    if (p >= kSmall) return small_weight(ct, p, e);
    if (!(p < kSmall)) return 0ull;
    const float kf = __fmaf_rn(p, 64.f, kMagic);
    const int j = __float_as_int(kf) - kMagicBits;
    const float r = __fmaf_rn(__fsub_rn(kf, kMagic), -1.f / 64.f, p);
    // 2^-(r + e) - 1 = s - y - ye
    const float y = __fmul_rn(r, 0.693147182f);
    const float ye = __fadd_rn(__fmaf_rn(r, 0.693147182f, -y), __fmaf_rn(r, -1.90465421e-9f, __fmul_rn(e, 0.693147182f)));
    const float z = __fadd_rn(y, ye);
    const float s = __fmul_rn(__fmul_rn(z, z), __fmaf_rn(z, -__fmaf_rn(z, -1.f / 24.f, 1.f / 6.f), 0.5f));
    const int dq = __float2int_rn(__fmul_rn(y, -274877906944.f)) + __float2int_rn(__fmul_rn(__fsub_rn(s, ye), 274877906944.f));  // in units of 2^-38
    const u64 t = ct->powers[j & 63];
    const u64 w = t + static_cast<u64>((static_cast<long long>(static_cast<int>(t >> 31)) * dq) >> 7);
    return ((w >> (j >> 6)) + (1ull << (60 - kOne))) >> (61 - kOne);
}

// The bin of p (0 .. kBins - 1: p is at most the range that r.bins was made for), as the float that holds it.
__device__ __forceinline__ float bin_float(const Row &r, float p) { return __fmaf_rn(p, r.bins, kMagic); }
__device__ __forceinline__ int bin_of(const Row &r, float p) { return __float_as_int(bin_float(r, p)) - kMagicBits; }

__device__ __forceinline__ u64 place(const Row &r, float p, float l, int idx)
{
    return static_cast<u64>(bin_of(r, p)) << kBinShift | static_cast<u64>(order_of(l)) << kIdxBits | static_cast<u64>(idx);
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
// The smallest a and the largest b of the block (all threads get them).
template <int NT>
__device__ __forceinline__ void block_range(Control *ct, u64 &a, u64 &b)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    auto over = [&](int lanes) {
        for (int o = lanes / 2; o > 0; o >>= 1) {
            a = min(a, __shfl_xor_sync(0xffffffffu, a, o));
            b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
    };
    over(32);
    __syncthreads();
    if (lane == 0) {
        ct->red[2 * w] = a;
        ct->red[2 * w + 1] = b;
    }
    __syncthreads();
    a = ct->red[2 * (lane % (NT / 32))];
    b = ct->red[2 * (lane % (NT / 32)) + 1];
    over(NT / 32);
}
// Sums over the threads before this one; the block's sums in total.
template <int NT>
__device__ __forceinline__ void block_scan(Control *ct, u64 w, uint32_t n, u64 &before_w, uint32_t &before_n, u64 &all_w,
                                           uint32_t &all_n)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    auto scan = [&](u64 &sw, uint32_t &sn) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 a = __shfl_up_sync(0xffffffffu, sw, o);
            const uint32_t c = __shfl_up_sync(0xffffffffu, sn, o);
            if (lane >= o) sw += a, sn += c;
        }
    };
    u64 sw = w;
    uint32_t sn = n;
    scan(sw, sn);
    __syncthreads();
    if (lane == 31) {
        ct->scan_w[wid] = sw;
        ct->scan_n[wid] = sn;
    }
    __syncthreads();
    u64 tw = lane < NT / 32 ? ct->scan_w[lane] : 0;
    uint32_t tn = lane < NT / 32 ? ct->scan_n[lane] : 0;
    scan(tw, tn);
    all_w = __shfl_sync(0xffffffffu, tw, 31);
    all_n = __shfl_sync(0xffffffffu, tn, 31);
    const u64 ow = __shfl_sync(0xffffffffu, tw, (wid + 31) & 31);
    const uint32_t on = __shfl_sync(0xffffffffu, tn, (wid + 31) & 31);
    before_w = sw - w + (wid ? ow : 0);
    before_n = sn - n + (wid ? on : 0);
}

// A part of a row, and the bins and the list beside it.
template <typename IN>
struct Part {
    const IN *l;              // the part's logits
    int n, first;             // how many; the first one's index in the row
    uint32_t *lo, *hi, *cnt;  // [kBins] weights in two words, tokens
    u64 *list, *list_w;       // [kList] places; weights
};

// A part's logits by groups of 16 bytes, as they lie in memory; what is outside the part
// counts as NaN.
template <typename IN>
struct Groups {
    static constexpr int VEC = 16 / sizeof(IN);
    const IN *l;
    int n, from, count;  // from: the first group's first logit (negative: it begins before the part)
    __device__ __forceinline__ explicit Groups(const Part<IN> &pt) : l(pt.l), n(pt.n)
    {
        const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(pt.l) & 15)) & 15) / static_cast<int>(sizeof(IN));
        from = head == 0 ? 0 : head - VEC;
        count = (n - from + VEC - 1) / VEC;
    }
    __device__ __forceinline__ uint4 load(int g) const
    {
        const uint32_t none = sizeof(IN) == 4 ? 0x7FC00000u : 0x7FC07FC0u;
        const int at = from + g * VEC;
        uint4 x = make_uint4(none, none, none, none);
        if (at >= 0 && at + VEC <= n) {
            x = *reinterpret_cast<const uint4 *>(l + at);
        } else if (g < count) {
            x = edge(at);
        }
        return x;
    }
    // A group that is partly outside.
    __device__ __noinline__ uint4 edge(int at) const
    {
        const uint32_t none = sizeof(IN) == 4 ? 0x7FC00000u : 0x7FC07FC0u;
        uint32_t w[4] = {none, none, none, none};
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (at + i >= 0 && at + i < n) {
                if (sizeof(IN) == 4)
                    w[i & 3] = reinterpret_cast<const uint32_t *>(l)[at + i];
                else
                    w[i / 2] = __byte_perm(w[i / 2], reinterpret_cast<const uint16_t *>(l)[at + i], i & 1 ? 0x5410 : 0x3254);
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Logits h .. h + 3 of a group.
    __device__ __forceinline__ static void four(const uint4 &x, int h, float (&v)[4])
    {
        if (sizeof(IN) == 4) {
            v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
        } else {
            const uint32_t a = h ? x.z : x.x, b = h ? x.w : x.y;
            v[0] = bf16_lo(a), v[1] = bf16_hi(a), v[2] = bf16_lo(b), v[3] = bf16_hi(b);
        }
    }
};

// f(four logits, their number in the turn) for all of the part, little work each: eight groups a
// thread at a time (g, g + NT, ...), their loads in flight together; end(groups, g) after each turn.
template <int NT, typename IN, typename F, typename E>
__device__ __forceinline__ void each_light(const Part<IN> &pt, F f, E end)
{
    const Groups<IN> gr(pt);
#pragma unroll 1
    for (int g = threadIdx.x; (g & ~31) < gr.count; g += 8 * NT) {
        uint4 x[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) x[y] = gr.load(g + y * NT);
#pragma unroll
        for (int y = 0; y < 8; ++y)
#pragma unroll
            for (int h = 0; h < gr.VEC; h += 4) {
                float v[4];
                gr.four(x[y], h, v);
                f(v, y * (gr.VEC / 4) + h / 4);
            }
        end(gr, g);
    }
}

// f(four logits) for all of the part, much work each: loads are four ahead, and the code of f is
// there once (copies side by side ran out of the instruction cache).  Warps stay together.
template <int NT, typename IN, typename F>
__device__ __forceinline__ void each_four(const Part<IN> &pt, F f)
{
    const Groups<IN> gr(pt);
    int g = threadIdx.x;
    uint4 x[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) x[y] = gr.load(g + y * NT);
#pragma unroll 1
    for (; (g & ~31) < gr.count; g += NT) {
        const uint4 next = gr.load(g + 4 * NT);
#pragma unroll 1
        for (int h = 0; h < gr.VEC; h += 4) {
            float v[4];
            gr.four(x[0], h, v);
            f(v);
        }
        x[0] = x[1], x[1] = x[2], x[2] = x[3], x[3] = next;
    }
}

__device__ __forceinline__ float select4(const float (&v)[4], int i) { return i & 2 ? (i & 1 ? v[3] : v[2]) : (i & 1 ? v[1] : v[0]); }

__device__ __forceinline__ void add_weight(uint32_t *lo, uint32_t *hi, int bin, u64 w)
{
    const uint32_t a = static_cast<uint32_t>(w), old = atomicAdd(lo + bin, a);
    const uint32_t b = static_cast<uint32_t>(w >> 32) + (old + a < old ? 1u : 0u);
    if (b) atomicAdd(hi + bin, b);
}

// A token whose weight rounds to no unit is in no bin and is never given.  A long tail of such
// tokens still adds up, 2^18 of them to 2^-28, and decides where equal logits meet a border exactly.  So
// where a target lies nearer to the end of the token found than a tail can be, the tail is added up, in units
// of 2^-63 (from 2^-63.5 down a weight is none), and the target is looked for again.  (Added up in every row
// that can have one, in the first pass, it cost 2 to 4 % of all calls; so only a row that needs it
// pays: one of 65543 logits 26.5 us instead of 19.)
constexpr int kTailOne = 63;
constexpr float kTailFrom = 45.5f, kTailEnd = 63.5f;
template <int NT, typename IN>
__device__ __noinline__ void add_tail(Control *ct, const IN *l, int n, float max, float ch, float cl)
{
    const Part<IN> pt{l, n, 0, nullptr, nullptr, nullptr, nullptr, nullptr};
    Row r;
    r.max = max, r.ch = ch, r.cl = cl;
    bool exact = true;
    const float min_p = ct->min_p;
    uint32_t least = min_p > 0.f ? static_cast<uint32_t>(part_of(min_p, 1ull << kTailOne, exact)) : 1u;
    if (!exact || least == 0) ++least;
    each_four<NT>(pt, [&](const float(&v)[4]) {
        uint32_t sum = 0;  // (at most 2^17 a token)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x, e;
            exponent(r, v[i], x, e);
            const bool in = x >= kTailFrom && x < kTailEnd && small_weight(ct, x, e) == 0;
            const uint32_t w = weight32<kTailOne>(ct, in ? x : kTailFrom, in ? e : 0.f);
            if (in && w >= least) sum += w;
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (sum != 0 && (threadIdx.x & 31) == 0) add_weight(ct->tail, ct->tail + 1, 0, sum);
    });
}

template <int NT, typename IN>
__device__ __forceinline__ void clear_bins(const Part<IN> &pt)
{
    for (int i = threadIdx.x; i < kBins; i += NT) pt.lo[i] = pt.hi[i] = pt.cnt[i] = 0u;
    __syncthreads();
}

// The bins of all blocks added up in the first block's (each block's are complete).
template <int NT, typename IN>
__device__ __forceinline__ void reduce_bins(const Part<IN> &pt, int rank, int blocks)
{
    const int tid = threadIdx.x;
    if (blocks == 1) {
        __syncthreads();
        return;
    }
    cluster_sync();
    // each block adds up a share of the bins, in its own place for them (which no other reads)
    const int share = kBins / blocks;
    for (int i = rank * share + tid; i < (rank + 1) * share; i += NT) {
        uint32_t h[kMaxCluster], l[kMaxCluster], n[kMaxCluster];
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
            const int y = min(x, blocks - 1);
            h[x] = remote32(pt.hi + i, y);
            l[x] = remote32(pt.lo + i, y);
            n[x] = remote32(pt.cnt + i, y);
        }
        u64 w = 0;
        uint32_t m = 0;
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x)
            if (x < blocks) w += static_cast<u64>(h[x]) << 32 | l[x], m += n[x];
        pt.lo[i] = static_cast<uint32_t>(w);
        pt.hi[i] = static_cast<uint32_t>(w >> 32);
        pt.cnt[i] = m;
    }
    cluster_sync();
    if (rank != 0) return;
    constexpr int IT = kBins / NT;
    uint32_t h[IT], l[IT], n[IT];
#pragma unroll
    for (int y = 0; y < IT; ++y) {
        const int i = tid + y * NT, x = i / share;
        h[y] = remote32(pt.hi + i, x);
        l[y] = remote32(pt.lo + i, x);
        n[y] = remote32(pt.cnt + i, x);
    }
#pragma unroll
    for (int y = 0; y < IT; ++y) {
        const int i = tid + y * NT;
        pt.hi[i] = h[y], pt.lo[i] = l[y], pt.cnt[i] = n[y];
    }
    __syncthreads();
}

// The smallest a and the largest b of the cluster (all threads get them).
template <int NT>
__device__ __forceinline__ void gather_range(Control *ct, u64 &a, u64 &b, int rank, int blocks)
{
    const int tid = threadIdx.x;
    block_range<NT>(ct, a, b);
    if (blocks == 1) return;
    if (tid < blocks) {
        put64(&ct->best[rank], tid, a);
        put64(&ct->last[rank], tid, b);
    }
    cluster_sync();
    for (int x = 0; x < blocks; ++x) a = min(a, ct->best[x]), b = max(b, ct->last[x]);
}

// What the cluster does for the first block's question.
template <int NT, typename IN>
__device__ __forceinline__ void answer(const Part<IN> &pt, const Row &r, Control *ct, int rank, int blocks)
{
    const int tid = threadIdx.x, op = ct->op, shift = ct->shift;
    const u64 klo = ct->klo, khi = ct->khi;
    if (op == kTail) {
        add_tail<NT>(ct, pt.l, pt.n, r.max, r.ch, r.cl);
        if (blocks > 1)
            cluster_sync();
        else
            __syncthreads();
        return;
    }
    if (op == kHist) clear_bins<NT>(pt);
    if (tid == 0) ct->n = 0;
    __syncthreads();
    // whole bins: what a token weighs is left for when they are side by side
    const u64 inside = (1ull << kBinShift) - 1;
    const bool whole = op == kGather && (klo & inside) == 0 && (khi & inside) == inside;
    const int lo = static_cast<int>(klo >> kBinShift), hi = static_cast<int>(khi >> kBinShift);
    const float blo = static_cast<float>(lo) + kMagic, bhi = static_cast<float>(hi) + kMagic;
    // most tokens are told from their logits alone: outside the bins' bounds, a bin and some roundings wider
    float most = r.max - (lo - 1) / r.bins / r.ch, least = r.max - (hi + 1) / r.bins / r.ch;
    most += (fabsf(r.max) + fabsf(most)) * 0x1p-20f;
    least -= (fabsf(r.max) + fabsf(least)) * 0x1p-20f;
    if (!(r.bins > 0.f && r.ch > 0.f)) most = INFINITY, least = -INFINITY;
    least = fmaxf(least, -3.402823466e38f);
    if (r.infinite) least = INFINITY, most = INFINITY;
    u64 a = ~0ull, b = 0ull;
    u64 hits = 0;
    each_light<NT>(
        pt,
        [&](const float(&v)[4], int q) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v[i] >= least && v[i] <= most) m |= 1u << i;
            hits |= static_cast<u64>(m) << (4 * q);
        },
        [&](const Groups<IN> &gr, int g) {
#pragma unroll 1
            for (; hits; hits &= hits - 1) {
                const int x = __ffsll(static_cast<long long>(hits)) - 1, at = gr.from + (g + x / gr.VEC * NT) * gr.VEC + x % gr.VEC;
                const int idx = pt.first + at;
                float l = sizeof(IN) == 4 ? __uint_as_float(reinterpret_cast<const uint32_t *>(pt.l)[at])
                                          : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(pt.l)[at]) << 16);
                float p, e;
                if (r.infinite) l = as_infinite(l);
                exponent(r, l, p, e);
                const float bin = bin_float(r, p);
                if (!(p < kNone && bin >= blo && bin <= bhi)) continue;
                if (!whole) {
                    const u64 k = place(r, p, l, idx), w = weight(ct, p, e);
                    if (k < klo || k > khi || w == 0 || w < r.least) continue;
                    if (op == kRange) {
                        a = min(a, k), b = max(b, k);
                        continue;
                    }
                    if (op == kHist) {
                        const int y = static_cast<int>((k - klo) >> shift);
                        add_weight(pt.lo, pt.hi, y, w);
                        atomicAdd(pt.cnt + y, 1u);
                        continue;
                    }
                }
                const int to = atomicAdd(&ct->n, 1);
                if (to < kList) pt.list[to] = static_cast<u64>(__float_as_uint(l)) << 32 | static_cast<u64>(idx);
            }
            __syncwarp();
        });
    if (op == kRange) {
        gather_range<NT>(ct, a, b, rank, blocks);
        if (rank != 0) return;  // (the next question may be here already)
        __syncthreads();        // (all have read this one)
        if (tid == 0) ct->klo = a, ct->khi = b;
        __syncthreads();
        return;
    }
    if (op == kHist) {
        reduce_bins<NT>(pt, rank, blocks);
        return;
    }
    __syncthreads();
    for (int i = tid, n = min(ct->n, kList); i < n; i += NT) {
        const u64 v = pt.list[i];
        const float l = __uint_as_float(static_cast<uint32_t>(v >> 32));
        float p, e;
        exponent(r, l, p, e);
        const u64 w = weight(ct, p, e);
        const bool in = w != 0 && w >= r.least;  // (a place behind all others if not)
        pt.list[i] = in ? place(r, p, l, static_cast<int>(v & 0xFFFFFFFFu)) : ~0ull;
        pt.list_w[i] = in ? w : 0ull;
    }
    if (blocks == 1) {
        __syncthreads();
        if (tid == 0) ct->all = ct->n, ct->n = min(ct->n, kList);
        __syncthreads();
        return;
    }
    if (tid == 0) put32(&ct->ns[rank], 0, ct->n);
    cluster_sync();
    if (rank != 0) return;
    // the others' tokens behind its own: the i-th is the block's whose tokens cover i
    int upto[kMaxCluster], all = 0;
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
        if (x < blocks) all += ct->ns[x];
        upto[x] = all;
    }
    const int n = min(all, kList);
    for (int i = min(upto[0], kList) + tid; i < n; i += NT) {
        int x = 0, before = 0;
#pragma unroll
        for (int y = 0; y < kMaxCluster - 1; ++y)
            if (i >= upto[y]) x = y + 1, before = upto[y];
        const u64 k = remote64(pt.list + (i - before), x), w = remote64(pt.list_w + (i - before), x);
        pt.list[i] = k;
        pt.list_w[i] = w;
    }
    __syncthreads();
    if (tid == 0) ct->n = n, ct->all = all;
    __syncthreads();
}

// ---- the first block's decisions
template <int NT, typename IN>
struct Chooser {
    static constexpr int kPer = kBins / NT;
    const Part<IN> &pt;
    Control *ct;
    int blocks;
    bool counts;                   // the bins of the first pass have their tokens counted
    int top_k;
    float top_p, u;
    u64 w[kPer], before_w, z;      // the thread's bins of the first pass; the weights that are left
    uint32_t n[kPer], before_n, all_n;
    u64 glo = 1, ghi = 0;          // places that the list covers (none)
    // the target that is looked for: the first place at which the count (or the weights) reaches t, known to
    // be in [klo, khi], with the sums before klo
    int stage = 0, phase = 0, rounds = 0;
    u64 t, klo, khi, bw;
    uint32_t bn;
    bool count;
    u64 key, key_w;                // what was found last

    __device__ __forceinline__ void ask(int op, int shift)
    {
        if (threadIdx.x < blocks) {  // to every block, so that none has to read it here
            put32(&ct->op, threadIdx.x, op);
            put32(&ct->shift, threadIdx.x, shift);
            put64(&ct->klo, threadIdx.x, op == kGather ? glo : klo);
            put64(&ct->khi, threadIdx.x, op == kGather ? ghi : khi);
        }
    }

    // Bins of the last pass, a few a thread.
    __device__ __forceinline__ void load_bins(u64 (&xw)[kPer], uint32_t (&xn)[kPer], u64 &bef_w, uint32_t &bef_n, u64 &tot_w,
                                              uint32_t &tot_n)
    {
        u64 sw = 0;
        uint32_t sn = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const int i = kPer * threadIdx.x + q;
            xw[q] = static_cast<u64>(pt.hi[i]) << 32 | pt.lo[i];
            xn[q] = pt.cnt[i];
            sw += xw[q];
            sn += xn[q];
        }
        block_scan<NT>(ct, sw, sn, bef_w, bef_n, tot_w, tot_n);
    }

    // The bin at which the sums before it (base) and in order reach t.
    template <int Q>
    __device__ __forceinline__ void find_bin(const u64 (&xw)[Q], const uint32_t (&xn)[Q], u64 bef_w, uint32_t bef_n, u64 base_w,
                                             uint32_t base_n)
    {
        u64 cw = base_w + bef_w;
        uint32_t cn = base_n + bef_n;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const u64 a = count ? cn : cw, b = count ? cn + xn[q] : cw + xw[q];
            if (a < t && t <= b) {
                ct->bin = Q * threadIdx.x + q;
                ct->base_w = cw;
                ct->base_n = cn;
                ct->bin_n = xn[q];
            }
            cw += xw[q];
            cn += xn[q];
        }
        __syncthreads();
    }

    // The next target; whether there is one.
    __device__ __forceinline__ bool next_target()
    {
        bool exact = true;
        if (stage == 0) {
            ++stage;
            if (top_k > 0 && static_cast<uint32_t>(top_k) < all_n) {
                t = top_k, count = true;
                return true;
            }
        }
        count = false;
        if (stage == 1) {
            ++stage;
            if (top_p < 1.f) {
                t = top_p > 0.f ? part_of(top_p, z, exact) : 0ull;
                t = max(1ull, t + (exact ? 0 : 1));
                return true;
            }
        }
        t = u >= 1.f ? z : (u > 0.f ? min(z, part_of(u, z, exact) + 1) : 1ull);
        return ++stage == 3;
    }

    // Goes on until something has to be asked of the cluster (true) or the token is found.
    __device__ __forceinline__ bool go_on()
    {
        for (;;) {
            if (phase == 0 || phase == 5) {  // a new target, the last one once more
                if (phase == 5)
                    target_with_tail();
                else if (!next_target())
                    return false;
                find_bin(w, n, before_w, before_n, 0, 0);
                klo = static_cast<u64>(ct->bin) << kBinShift, khi = klo + ((1ull << kBinShift) - 1);
                bw = ct->base_w, bn = ct->base_n;
                const uint32_t m = ct->bin_n;
                __syncthreads();
                phase = 4;
                if (klo < glo || khi > ghi) {
                    if (counts && m > kList) {
                        ask(kRange, 0);
                        phase = 2;
                    } else {
                        // all tokens up to the bin's, where they are few (what is asked next lies among them)
                        glo = counts && bn + m <= kList ? 0 : klo, ghi = khi;
                        ask(kGather, 0);
                        phase = 1;
                    }
                    return true;
                }
            } else if (phase == 1) {  // after a list
                phase = 4;
                if (ct->all > kList && rounds < 6) {
                    ask(kRange, 0);
                    phase = 2;
                    return true;
                }
            } else if (phase == 2) {
                // many tokens in a bin: parts of its range, until few are left (each round
                // leaves kBinBits less of a place's bits)
                klo = ct->klo, khi = ct->khi;
                __syncthreads();
                ask(kHist, max(0, 64 - __clzll(khi - klo) - kBinBits));  // (khi - klo) >> shift < kBins
                phase = 3;
                return true;
            } else if (phase == 3) {
                const int shift = ct->shift;
                u64 xw[kPer], xbw, xall;
                uint32_t xn[kPer], xbn, xalln;
                load_bins(xw, xn, xbw, xbn, xall, xalln);
                find_bin(xw, xn, xbw, xbn, bw, bn);
                klo += static_cast<u64>(ct->bin) << shift;
                khi = klo + ((1ull << shift) - 1);
                bw = ct->base_w, bn = ct->base_n;
                const uint32_t m = ct->bin_n;
                __syncthreads();
                if (m > kList && ++rounds < 6) {
                    ask(kRange, 0);
                    phase = 2;
                } else {
                    glo = klo, ghi = khi;
                    ask(kGather, 0);
                    phase = 1;
                }
                return true;
            } else {
                look();
                phase = rounds = 0;
                const u64 upto = ct->base_w;  // the weights up to the token, its own included
                const bool near = !count && t + ct->most_tail > upto && tail_counts();
                __syncthreads();
                if (near) {
                    ask(kTail, 0);
                    phase = 5;
                    return true;
                }
                if (stage < 3) z = upto;
            }
        }
    }

    // Whether the target is a part of a sum that the tokens in no bin belong to and that can be told from others
    // (top-k takes them all away, or leaves some, of which more is not known than their sum).
    __device__ __forceinline__ bool tail_counts() const
    {
        if (ct->most_tail == 0 || (top_k > 0 && static_cast<uint32_t>(top_k) <= all_n)) return false;
        return stage < 3 ? top_p > 0.f : !(top_p < 1.f) && u > 0.f && u < 1.f;
    }

    // The same target as a part of a sum that has the tail.  (Below the bins' own: top_p and u are 2^-24
    // below 1, and the tail is 2^-28 of z at most.)
    __device__ __forceinline__ void target_with_tail()
    {
        u64 f = 0;
        for (int x = 0; x < blocks; ++x) f += static_cast<u64>(remote32(ct->tail + 1, x)) << 32 | remote32(ct->tail, x);
        constexpr int kShift = kTailOne - kOne;
        z += f >> kShift;
        bool exact = true;
        t = part_of(stage < 3 ? top_p : u, z, exact);
        if (stage == 3 || !exact || (f & ((1ull << kShift) - 1)) != 0) ++t;
        if (threadIdx.x == 0) ct->most_tail = 0;
    }

    // The target's place among the listed tokens in [klo, khi].
    __device__ __forceinline__ void look()
    {
        const int tid = threadIdx.x, lane = tid & 31, len = ct->n;
#pragma unroll 1
        for (int round = 0;; ++round) {  // (each leaves 9 bits less)
            u64 a = ~0ull, b = 0ull;
            if (tid == 0) ct->few = 0;
            __syncthreads();
            for (int i = tid; i < len; i += NT) {
                const u64 k = pt.list[i];
                if (k < klo || k > khi) continue;
                a = min(a, k), b = max(b, k);
                const int at = atomicAdd(&ct->few, 1);
                if (at < kFew) ct->small[at] = i;
            }
            __syncthreads();
            if (ct->few <= kFew || round == 8) break;
            block_range<NT>(ct, a, b);
            klo = a;
            const int shift = max(0, 64 - __clzll(b - a) - (NT == 1024 ? 10 : 9));  // (b - a) >> shift < NT
            pt.lo[tid] = pt.hi[tid] = pt.cnt[tid] = 0u;
            __syncthreads();
            for (int i = tid; i < len; i += NT) {
                const u64 k = pt.list[i];
                if (k < klo || k > khi) continue;
                const int y = static_cast<int>((k - klo) >> shift);
                add_weight(pt.lo, pt.hi, y, pt.list_w[i]);
                atomicAdd(pt.cnt + y, 1u);
            }
            __syncthreads();
            const u64 xw[1] = {static_cast<u64>(pt.hi[tid]) << 32 | pt.lo[tid]};
            const uint32_t xn[1] = {pt.cnt[tid]};
            u64 xbw, xall;
            uint32_t xbn, xalln;
            block_scan<NT>(ct, xw[0], xn[0], xbw, xbn, xall, xalln);
            find_bin(xw, xn, xbw, xbn, bw, bn);
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
#pragma unroll 1
            for (int i = 0; i < few; ++i) {
                const u64 ok = __shfl_sync(0xffffffffu, k, i), ow = __shfl_sync(0xffffffffu, mine, i);
                if (ok < k) cw += ow, ++cn;
            }
            const u64 c0 = count ? cn : cw, c1 = count ? cn + 1 : cw + mine;
            if (lane < few && c0 < t && t <= c1) ct->key_found = k, ct->w_found = mine, ct->base_w = cw + mine;
        }
        __syncthreads();
        key = ct->key_found, key_w = ct->w_found;
    }
};

struct Params {
    moe_sample_desc d;
    int part;    // logits of a block
    int blocks;  // of a row: a cluster
};

__device__ __forceinline__ float setting(const float *a, float one, int t) { return a ? a[t] : one; }

// NT threads; COUNT: 16-bit logits are counted by value first.
template <typename IN, int NT, bool COUNT>
__global__ void __launch_bounds__(NT, 1024 / NT) moe_sample_kernel(const __grid_constant__ Params p)
{
    const int blocks = p.blocks;
    extern __shared__ __align__(16) uint8_t smem[];
    Control *ct = reinterpret_cast<Control *>(smem);
    u64 *list = reinterpret_cast<u64 *>(smem + (sizeof(Control) + 15) / 16 * 16);
    uint32_t *bins = reinterpret_cast<uint32_t *>(list + 2 * kList);
    uint32_t *counters = bins + 3 * kBins;  // COUNT: [kCounters / 2]
    const moe_sample_desc &d = p.d;
    const int tid = threadIdx.x, lane = tid & 31, rank = cluster_rank(), t = blockIdx.x / blocks;
    const int first = min(rank * p.part, d.V), n = min(p.part, d.V - first);
    const Part<IN> pt{static_cast<const IN *>(d.logits_dev) + static_cast<long long>(t) * d.stride + first, n, first,
                      bins, bins + kBins, bins + 2 * kBins, list, list + kList};
    if (tid < 64) {
        const u64 v = kPowers.v[tid];
        ct->powers[tid] = v;
        ct->powers32[tid] = static_cast<int>((v + (1ull << 30)) >> 31);
    }
    if (tid < 2) ct->tail[tid] = 0u;
    if (COUNT)
        for (int i = tid; i < kCounters / 8; i += NT) reinterpret_cast<uint4 *>(counters)[i] = make_uint4(0u, 0u, 0u, 0u);
    clear_bins<NT>(pt);
    if (blocks > 1) cluster_arrive();
    grid_wait();
    grid_release();
    // (the settings are here by the time they are used)
    const float temperature = setting(d.temperature_dev, d.temperature, t), top_p = setting(d.top_p_dev, d.top_p, t);
    const float min_p = setting(d.min_p_dev, d.min_p, t), u = d.u_dev[t];
    const int top_k = d.top_k_dev ? d.top_k_dev[t] : d.top_k;

    // ---- the largest logit, the smallest that is not masked (as orders: the least, the greatest)
    u64 best = ~0ull, last = 0ull;
    bool counted = COUNT;  // 16-bit logits are counted by value
    if (COUNT) {
        uint32_t over = 0;  // tokens that were counted, and then are not found
        each_light<NT>(
            pt,
            [&](const float(&v)[4], int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = __float_as_uint(v[i]) >> 16;
                    if (!(v[i] > -INFINITY)) continue;  // masked (many at one place), NaN
                    atomicAdd(counters + (x >> 1), 1u << (16 * (x & 1)));
                    ++over;
                }
            },
            [](const Groups<IN> &, int) {});
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < kCounters / 8; i += NT) {
            const uint4 c = reinterpret_cast<const uint4 *>(counters)[i];
            if ((c.x | c.y | c.z | c.w) == 0) continue;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint32_t m = u4w(c, x >> 1) >> (16 * (x & 1)) & 0xFFFFu;
                over -= m;
                if (m != 0) {
                    const u64 o = order_of(__uint_as_float(static_cast<uint32_t>(8 * i + x) << 16));
                    best = min(best, o), last = max(last, o);
                }
            }
        }
        u64 z0, z1;
        uint32_t z2, all;
        block_scan<NT>(ct, 0, over, z0, z2, z1, all);
        counted = all == 0;  // (else a counter ran over its 16 bits: every token is looked at instead)
    }
    if (!counted) {
        float top = -INFINITY, low = INFINITY;
        each_light<NT>(
            pt,
            [&](const float(&v)[4], int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    top = fmaxf(top, v[i]);  // (NaN is none)
                    if (v[i] > -INFINITY) low = fminf(low, v[i]);
                }
            },
            [](const Groups<IN> &, int) {});
        best = order_of(top);
        last = low == INFINITY ? 0ull : order_of(low);
    }
    if (blocks > 1) cluster_wait();
    gather_range<NT>(ct, best, last, rank, blocks);
    Row r;
    r.max = best == ~0ull ? -INFINITY : logit_of(static_cast<uint32_t>(best));
    const bool nothing = r.max == -INFINITY;
    if (nothing || !(temperature > kGreedy) || top_k == 1) {
        u64 at = ~0ull, none = 0ull;  // the first of the largest
        u64 hits = 0;
        if (!nothing)
            each_light<NT>(
                pt,
                [&](const float(&v)[4], int q) {
                    uint32_t m = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (v[i] == r.max) m |= 1u << i;
                    hits |= static_cast<u64>(m) << (4 * q);
                },
                [&](const Groups<IN> &gr, int g) {
                    if (hits) {
                        const int x = __ffsll(static_cast<long long>(hits)) - 1;
                        at = min(at, static_cast<u64>(first + gr.from + (g + x / gr.VEC * NT) * gr.VEC + x % gr.VEC));
                    }
                    hits = 0;
                });
        if (blocks > 1) cluster_sync();  // what the last exchange left has been read
        gather_range<NT>(ct, at, none, rank, blocks);
        if (rank == 0 && tid == 0) {
            d.token_dev[t] = nothing ? -1 : static_cast<int32_t>(at);
            if (d.prob_dev) d.prob_dev[t] = nothing ? 0.f : 1.f;
        }
        return;
    }
    // log2(e) / t in two floats, from log2(e) in two
    r.ch = 1.44269502f / temperature;
    r.cl = temperature < INFINITY ? (fmaf(-r.ch, temperature, 1.44269502f) + 1.92596303e-8f) / temperature : 0.f;
    r.infinite = r.max == INFINITY;
    if (r.infinite) r.max = 0.f;
    bool exact = true;
    r.least = min_p >= 1.f ? 1ull << kOne : (min_p > 0.f ? part_of(min_p, 1ull << kOne, exact) : 1ull);
    if (!exact) ++r.least;
    const float reach = r.infinite ? 0.f : __fmul_rn(__fsub_rn(r.max, logit_of(static_cast<uint32_t>(last))), r.ch);
    const float range = fminf(reach, kNone);
    r.bins = range > 1e-30f ? (kBins - 1) / range : 0.f;  // (else all in one)
    if (tid == 0) {  // (min-p takes a tail away if it takes any token of a unit)
        ct->most_tail = !(reach < kTailFrom) && r.least == 1 ? d.V / 2 + 2 : 0;
        ct->min_p = min_p;
    }

    // ---- the first pass: every token that counts into its bin
    const bool counts = top_k > 0 || top_p < 1.f;  // (else the one question needs none)
    auto into_bin = [&](float x, float e, uint32_t count) {
        const u64 w = weight(ct, x, e);
        if (w == 0 || w < r.least) return;
        const int bin = bin_of(r, x);
        add_weight(pt.lo, pt.hi, bin, w * count);
        if (counts) atomicAdd(pt.cnt + bin, count);
    };
    if (counted && !r.infinite) {
        // (neighbouring words to neighbouring threads: values that occur lie side by side)
#pragma unroll 1
        for (int i = tid; i < kCounters / 2; i += NT) {
            uint32_t c = counters[i];
#pragma unroll 1
            for (int y = 0; c != 0; ++y, c >>= 16) {
                if ((c & 0xFFFFu) == 0) continue;
                float x, e;
                exponent(r, __uint_as_float(static_cast<uint32_t>(2 * i + y) << 16), x, e);
                into_bin(x, e, c & 0xFFFFu);
            }
        }
    } else {
        // small weights side by side in 32 bits; the others wait in the warp's queue (in the
        // list's place) until there are 32 of them
        const uint32_t least32 = static_cast<uint32_t>(min(r.least, static_cast<u64>(0xFFFFFFFFu)));
        float2 *queue = reinterpret_cast<float2 *>(pt.list) + (tid >> 5) * 64;
        int waiting = 0;
        each_four<NT>(pt, [&](const float(&v)[4]) {
            float x[4], e[4];
            uint32_t w[4], was[4], large = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                exponent(r, r.infinite ? as_infinite(v[i]) : v[i], x[i], e[i]);
                if (x[i] < kSmall) large |= 1u << i;
                w[i] = small_weight(ct, x[i], e[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                was[i] = 0u;
                if (w[i] >= least32) was[i] = atomicAdd(pt.lo + bin_of(r, x[i]), w[i]);
            }
            if (counts) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (w[i] >= least32) atomicAdd(pt.cnt + bin_of(r, x[i]), 1u);
            }
            bool carry = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) carry |= was[i] > ~w[i];
            if (carry) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (was[i] > ~w[i]) atomicAdd(pt.hi + bin_of(r, x[i]), 1u);
            }
#pragma unroll 1
            for (;;) {
                const uint32_t have = __ballot_sync(0xffffffffu, large != 0);
                if (have == 0) break;
                if (large != 0) {
                    const int i = __ffs(large) - 1;
                    large &= large - 1;
                    queue[waiting + __popc(have & ((1u << lane) - 1u))] = make_float2(select4(x, i), select4(e, i));
                }
                waiting += __popc(have);
                __syncwarp();
                if (waiting >= 32) {
                    waiting -= 32;
                    const float2 q = queue[waiting + lane];
                    into_bin(q.x, q.y, 1u);
                    __syncwarp();
                }
            }
        });
        if (lane < waiting) into_bin(queue[lane].x, queue[lane].y, 1u);
    }
    reduce_bins<NT>(pt, rank, blocks);

    // ---- questions, until the first block has found the token
    Chooser<NT, IN> ch{pt, ct, blocks, counts, top_k, top_p, u};
    if (rank == 0) ch.load_bins(ch.w, ch.n, ch.before_w, ch.before_n, ch.z, ch.all_n);
#pragma unroll 1
    for (;;) {
        if (rank == 0 && !ch.go_on()) {
            if (tid == 0) {
                d.token_dev[t] = static_cast<int32_t>(ch.key & (MOE_SAMPLE_MAX_VOCAB - 1));
                if (d.prob_dev) d.prob_dev[t] = static_cast<float>(static_cast<double>(ch.key_w) / static_cast<double>(ch.z));
            }
            if (blocks == 1) return;
            ch.ask(kDone, 0);
        }
        if (blocks > 1)
            cluster_sync();
        else
            __syncthreads();
        if (ct->op == kDone) return;  // (nobody's shared memory is read any more)
        answer<NT>(pt, r, ct, rank, blocks);
    }
}

template <typename IN, int NT, bool COUNT>
cudaError_t launch_one(const Params &p, cudaStream_t st)
{
    const int blocks = p.blocks;
    constexpr int smem = static_cast<int>((sizeof(Control) + 15) / 16 * 16 + 2 * kList * 8 + 3 * kBins * 4) + (COUNT ? kCounters * 2 : 0);
    auto *fn = moe_sample_kernel<IN, NT, COUNT>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(p.d.T * blocks);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

cudaError_t launch_sample(const moe_sample_desc &d, int num_sms, cudaStream_t st)
{
    // The split of a row with the least time by a model of it, in us: a block's fixed part, more in a cluster, and
    // its logits, at 1.4 a thousand (counted 0.23); both grow with the blocks that share an SM or wait
    // for one.  Fitted to 900 times of 16 to 1000 rows of 4000 to 262144 logits: a call takes 2 % more than with
    // the best split of its own (18 % at worst).  Against as many blocks as the SMs hold, fp32: 256 rows of 131075
    // 283 -> 239 us, 100 rows 148 -> 121, 76 rows of 32000 46 -> 35; bf16: 32 rows of 65543 40 -> 35, 100
    // rows of 16000 37 -> 27.
    struct Split {
        int blocks;
        double us;
    };
    auto best = [&](bool count) {
        Split s{1, 0};
        for (int b = 1; b <= kMaxCluster && (b == 1 || d.V > 2048 * b); b *= 2) {
            const double logits = (d.V + b - 1) / b * 1e-3;
            double more, us;  // blocks of an SM above the first
            if (count) {  // each needs an SM's shared memory; clusters of 4 and 8 leave some SMs out
                const int sms = b <= 2 ? num_sms : (b == 4 ? num_sms * 10 / 11 : num_sms * 10 / 13);
                more = std::max(std::ceil(double(d.T) * b / sms) - 1, 0.);
                us = (b > 1 ? 31 : 22) * (1 + 0.73 * more) + 0.23 * logits * (1 + 0.6 * more);
            } else {
                const double x = double(d.T) * b / num_sms;
                more = std::max((x + std::ceil(x)) / 2 - 1, 0.);
                us = (b > 1 ? 16 : 12) * (1 + 0.45 * more) + 1.4 * logits * (1 + 0.4 * more);
            }
            if (b == 1 || us < s.us) s = Split{b, us};
        }
        return s;
    };
    auto params = [&](const Split &s) { return Params{d, (d.V + s.blocks - 1) / s.blocks, s.blocks}; };
    const Split p = best(false);
    if (!d.bf16) return launch_one<float, 512, false>(params(p), st);
    const Split c = best(true);
    return c.us < p.us ? launch_one<uint16_t, 1024, true>(params(c), st) : launch_one<uint16_t, 512, false>(params(p), st);
}

}  // namespace moe
