// moe_kv_attend.cu -- causal attention over the paged 8-bit cache
// (moe_kv_attend).
//
//   o[i, h] = sum_t w_t v[t] / sum_t w_t,   w_t = exp(scale q.k_t - m)
//
// in one pass over the cache with a running maximum m and sum.  A query head
// group's rows (tokens of a sequence x heads that share a kv head) form tiles;
// both products run on mma.sync m16n8k32 with E4M3 operands, straight on the
// cache's codes:
//
//  * q enters as two E4M3 digits, hi + lo, after a power-of-two prescale of the
//    row (largest magnitude into [128, 256)): 8 significant bits are two
//    digits of 4, so the sum is exact down to 2^-10 of the row's largest.
//  * the weights enter the second product as two digits of 256 w vs (vs the
//    page's v scale, over the largest that the maximum allows for), relative
//    error 2^-9; their sum stays in fp32.
//
// The running maximum is taken over log2(weight) + ceil(log2(vs)), so that the
// digits have their range for what is actually added, whatever the pages'
// scales.
//
// Order inside a page is free as long as both products agree: column c of
// score tile j is token 16 (c / 2) + 2 j + c % 2, which makes a lane's 16
// weights of a row the 16 consecutive tokens that it reads of a v row, and a
// lane's k and q elements 32 (head dim 128) or 16 consecutive ones.  k comes by TMA with
// the 128-byte swizzle, v as it lies; all shared-memory reads are 16 bytes
// wide and free of bank conflicts.
//
// Work is split evenly over one block per SM: the units are the pages of all
// (sequence, kv head, row tile) in a row, each block takes an equal run of
// them, and a tile cut by a run's end is joined by the last block that arrives
// at it, in block order (the same bits every run).
//
// Two variants: up to 8 rows, the digits of a row are rows r and r + 8 of the
// MMA's 16 (one MMA for both, each digit with its own accumulator); else 16
// rows and an MMA for each digit.  RW row groups of 16 by 8 / RW page groups
// make up the block's 8 warps: page groups take every (8 / RW)-th page of a
// tile and are added at its end.
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

constexpr int kPage = MOE_KV_PAGE;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32 + 128;  // consumers, and a warpgroup whose first warp is the producer
// Registers a thread of the two kinds keeps: 256 * 216 + 128 * 72 = 64512, what
// the block is launched with (384 threads of 168).
constexpr int kConsumerRegs = 216, kProducerRegs = 72;
constexpr int kMaxStages = 12;
constexpr int kPartRows = kAttendMaxRows;

// What a block knows of every sequence.
struct Seqs {
    long long cum[MOE_KV_MAX_SEQS + 1];  // units before sequence b
    int per_head[MOE_KV_MAX_SEQS];       // units of one kv head
    int q0[MOE_KV_MAX_SEQS], n[MOE_KV_MAX_SEQS], len[MOE_KV_MAX_SEQS];
};
struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    float ks[kMaxStages], vs[kMaxStages];  // scales of the stage's page; ks < 0: no such page
    int abort, last;
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t f16x2)
{
    uint32_t r;
    asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n cvt.u32.u16 %0, t;\n}" : "=r"(r) : "r"(f16x2));
    return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four values (at most 448 in magnitude) as two E4M3 digits: hi the nearest, lo
// the nearest to 2^LO times the rest.
template <int LO>
__device__ __forceinline__ void digits4(float a, float b, float c, float d, uint32_t &hi, uint32_t &lo)
{
    const uint32_t x = cvt_f16x2(a, b), y = cvt_f16x2(c, d);
    const uint32_t hx = cvt_e4m3x2(x), hy = cvt_e4m3x2(y);
    uint32_t rx = hsub2(x, e4m3x2_to_f16x2(static_cast<uint16_t>(hx)));
    uint32_t ry = hsub2(y, e4m3x2_to_f16x2(static_cast<uint16_t>(hy)));
    if (LO) {
        const uint32_t f = (0x3C00u + (LO << 10)) * 0x10001u;
        rx = hmul2(rx, f);
        ry = hmul2(ry, f);
    }
    hi = hx | (hy << 16);
    lo = cvt_e4m3x2(rx) | (cvt_e4m3x2(ry) << 16);
}
constexpr int kLoShift = 5;  // of the low digits where they have accumulators of their own

// Bounded wait; a block that gave up sets its abort flag and goes on without
// waiting, so that every warp still reaches the block's barriers.
__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, const AttendParams &p, Control *ct)
{
    if (mbar_test(bar, parity)) return;
    const uint64_t t0 = gtimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_test(bar, parity)) return;
        if ((it & 31u) == 0) {
            if (*reinterpret_cast<volatile int *>(&ct->abort)) return;
            if (static_cast<long long>(gtimer() - t0) > p.timeout_ns) {
                atomicOr(p.c.ctrl + 2, kErrTimeout);
                *reinterpret_cast<volatile int *>(&ct->abort) = 1;
                return;
            }
        }
    }
}

// Tokens that row r of a sequence sees (r = new token * group + head).
__device__ __forceinline__ int row_sees(int len, int n, int G, int r) { return max(len - n + r / G + 1, 0); }

// Units of row tile j: its pages, or one where its last row sees nothing (the
// tile's zeros still have to be written).
__device__ __forceinline__ int tile_units(int len, int n, int G, int TR, int j)
{
    const int last = min((j + 1) * TR, n * G) - 1;
    return max(1, (row_sees(len, n, G, last) + kPage - 1) / kPage);
}

// A run of units of one tile.
struct Segment {
    int b, h, tile, p0, p1;   // pages [p0, p1) of the tile
    int units;                // units of the whole tile
    long long start;          // first unit of the tile
};

// The tile that unit u lies in, and the run of it up to unit end.
__device__ __forceinline__ Segment locate(const Seqs &s, int B, int G, int TR, long long u, long long end)
{
    Segment g;
    int lo = 0, hi = B - 1;
    while (lo < hi) {  // the last b with cum[b] <= u (u is below cum[B])
        const int mid = (lo + hi + 1) >> 1;
        if (s.cum[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    g.b = lo;
    const int n = s.n[lo], len = s.len[lo];
    const int rel = static_cast<int>(u - s.cum[lo]);
    g.h = rel / s.per_head[lo];
    int r = rel - g.h * s.per_head[lo];
    const int tiles = (n * G + TR - 1) / TR;
    g.tile = 0;
    g.units = tile_units(len, n, G, TR, 0);
    if (tiles > 1) {
        const int lane = threadIdx.x & 31;
        for (int j0 = 0;; j0 += 32) {  // 32 tiles at a time
            const int mine = j0 + lane < tiles ? tile_units(len, n, G, TR, j0 + lane) : 0;
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned m = __ballot_sync(0xffffffffu, sum > r);
            if (m) {
                const int l = __ffs(m) - 1;
                g.tile = j0 + l;
                g.units = __shfl_sync(0xffffffffu, mine, l);
                r -= __shfl_sync(0xffffffffu, sum, l) - g.units;
                break;
            }
            r -= __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    g.start = u - r;
    g.p0 = r;
    g.p1 = static_cast<int>(min(static_cast<long long>(g.units), r + (end - u)));
    return g;
}

// First unit of block c when U units are dealt out to G blocks.
__device__ __forceinline__ long long block_start(long long U, int G, int c)
{
    const long long q = U / G, r = U - q * G;
    return q * c + min(static_cast<long long>(c), r);
}
// The block whose run holds unit u.
__device__ __forceinline__ int block_of(long long U, int G, long long u)
{
    const long long q = U / G, r = U - q * G;
    const long long cut = (q + 1) * r;
    return static_cast<int>(u < cut ? u / (q + 1) : r + (u - cut) / q);
}

// Shared memory: ring of stages (k page, v page), then the control block, the
// sequences, and (page groups) the merge buffer.
template <int D>
struct Layout {
    static constexpr int kStage = 2 * kPage * D;
};

template <int D, int RW, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) moe_kv_attend_kernel(const __grid_constant__ AttendParams p, int NS)
{
    constexpr int PW = kWarps / RW;             // page groups
    constexpr int MR = SPLIT ? 8 : 16;          // query rows of a warp
    constexpr int TR = MR * RW;                 // query rows of a tile
    constexpr int KS = D / 32;                  // K steps of the first product
    constexpr int DT = D / 8;                   // N tiles of the second
    constexpr int kStage = Layout<D>::kStage;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Control *ct = reinterpret_cast<Control *>(smem + NS * kStage);
    Seqs &sq = *reinterpret_cast<Seqs *>(smem + NS * kStage + sizeof(Control));
    float *mrg = reinterpret_cast<float *>(smem + NS * kStage + sizeof(Control) + sizeof(Seqs));
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const KvParams &c = p.c;
    const int G = c.q_heads / c.kv_heads;

    if (tid == 0) {
        ct->abort = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(&ct->full[i], 1);
            mbar_init(&ct->empty[i], RW);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_wait();
    grid_release();

    // ---- the sequences and their units
    for (int b = tid; b < c.B; b += kThreads) {
        const int a0 = c.q_off[b], a1 = c.q_off[b + 1], l = c.kv_len[b];
        const int q0 = min(max(a0, 0), c.N), q1 = min(max(a1, q0), c.N);
        const int len = l < 0 || l > c.max_pages * kPage ? 0 : l;  // out of range: nothing is seen
        if (blockIdx.x == 0 && (q0 != a0 || q1 != a1 || len != l)) atomicOr(c.ctrl + 2, kErrBadIndex);
        sq.q0[b] = q0;
        sq.n[b] = q1 - q0;
        sq.len[b] = len;
        const int rows = (q1 - q0) * G;
        sq.per_head[b] = rows == 0 ? 0 : (rows <= TR ? tile_units(len, q1 - q0, G, TR, 0) : -1);
    }
    __syncthreads();
    for (int b = wid; b < c.B; b += kThreads / 32) {
        if (sq.per_head[b] >= 0) continue;
        const int n = sq.n[b], len = sq.len[b], tiles = (n * G + TR - 1) / TR;
        int sum = 0;
        for (int j = lane; j < tiles; j += 32) sum += tile_units(len, n, G, TR, j);
        sum = __reduce_add_sync(0xffffffffu, sum);
        __syncwarp();
        if (lane == 0) sq.per_head[b] = sum;
    }
    __syncthreads();
    if (wid == 0) {
        long long run = 0;
        for (int b0 = 0; b0 < c.B; b0 += 32) {
            const int b = b0 + lane;
            const long long mine = b < c.B ? static_cast<long long>(sq.per_head[b]) * c.kv_heads : 0;
            long long sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (b < c.B) sq.cum[b] = run + sum - mine;
            run += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) sq.cum[c.B] = run;
    }
    __syncthreads();
    const long long U = sq.cum[c.B];
    const int blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), U));
    if (static_cast<int>(blockIdx.x) >= blocks) return;
    const long long u0 = block_start(U, blocks, blockIdx.x), u1 = block_start(U, blocks, blockIdx.x + 1);

    if (wid >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        if (wid > kWarps) return;
        // ---- producer: 32 pages' ids and scales at a time, then their copies
        int it = 0;
        const uint64_t pol = policy_evict_first();
        for (long long u = u0; u < u1;) {
            const Segment s = locate(sq, c.B, G, TR, u, u1);
            const int len = sq.len[s.b];
            const int pages = (len + kPage - 1) / kPage;
            const int pe = min(s.p1, pages);
            for (int pb = s.p0; pb < pe; pb += 32) {
                int id = -1;
                float ks = -1.f, vs = 0.f;
                if (pb + lane < pe) {
                    id = c.pages[static_cast<size_t>(s.b) * c.max_pages + pb + lane];
                    if (id >= 0 && id < c.n_pages) {
                        ks = c.ks[static_cast<size_t>(id) * c.kv_heads + s.h];
                        vs = c.vs[static_cast<size_t>(id) * c.kv_heads + s.h];
                    } else {
                        id = -1;
                        atomicOr(c.ctrl + 2, kErrBadIndex);
                    }
                }
                const int m = min(32, pe - pb);
                for (int i = 0; i < m; ++i, ++it) {
                    const int st = it % NS;
                    const int pid = __shfl_sync(0xffffffffu, id, i);
                    const float pks = __shfl_sync(0xffffffffu, ks, i), pvs = __shfl_sync(0xffffffffu, vs, i);
                    if (lane == 0) {
                        if (it >= NS) wait_or_abort(&ct->empty[st], (it / NS - 1) & 1, p, ct);
                        if (*reinterpret_cast<volatile int *>(&ct->abort) == 0) {
                            ct->ks[st] = pks;
                            ct->vs[st] = pvs;
                            if (pid < 0) {
                                mbar_arrive(&ct->full[st]);
                            } else {
                                mbar_expect_tx(&ct->full[st], kStage);
                                uint8_t *dst = smem + st * kStage;
                                const size_t ph = static_cast<size_t>(pid) * c.kv_heads + s.h;
                                if (D == 128)
                                    tma2d(dst, &c.tm_k, 0, static_cast<int>(ph * kPage), &ct->full[st], pol);
                                else
                                    bulk_g2s(dst, c.k + ph * (kPage * D), kPage * D, &ct->full[st], pol);
                                bulk_g2s(dst + kPage * D, c.v + ph * (kPage * D), kPage * D, &ct->full[st], pol);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            u += s.p1 - s.p0;
        }
        // every copy is waited for by the warps that use it, unless they gave up:
        // no block ends with a copy into its shared memory in flight
        if (lane == 0 && *reinterpret_cast<volatile int *>(&ct->abort)) {
            const uint64_t t0 = gtimer();
            for (int j = max(it - NS, 0); j < it; ++j)
                while (!mbar_test(&ct->full[j % NS], (j / NS) & 1) && static_cast<long long>(gtimer() - t0) < p.timeout_ns) {
                }
        }
        return;
    }

    // ---- consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    const int rw = wid / PW, pw = wid % PW;
    int it0 = 0;  // pages of this block before the segment
    for (long long u = u0; u < u1;) {
        const Segment s = locate(sq, c.B, G, TR, u, u1);
        const int n = sq.n[s.b], len = sq.len[s.b], rows = n * G, q0 = sq.q0[s.b];
        const int pages = (len + kPage - 1) / kPage, pe = min(s.p1, pages);
        const int r_lo = s.tile * TR + rw * MR + g, r_hi = r_lo + 8;  // this lane's rows (r_hi: 16-row variant)

        // q: two digits of the lane's 32 (16) elements of its rows
        uint32_t qh[2][2 * KS], ql[2][2 * KS];
        float qs[2];
        int sees[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = x ? r_hi : r_lo;
            const bool in = r < rows && (x == 0 || !SPLIT);
            sees[x] = in ? row_sees(len, n, G, r) : 0;
            qs[x] = 0.f;
            if (SPLIT && x) break;
            uint4 w[KS];
            const uint16_t *src = p.q + static_cast<long long>(q0 + r / G) * p.q_stride + (s.h * G + r % G) * D + (D / 4) * t4;
#pragma unroll
            for (int i = 0; i < KS; ++i) w[i] = in ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0u, 0u, 0u, 0u);
            uint32_t am = 0u;
#pragma unroll
            for (int i = 0; i < 4 * KS; ++i) am = __vmaxu2(am, u4w(w[i >> 2], i & 3) & 0x7FFF7FFFu);
            am = max(am >> 16, am & 0xFFFFu);
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
            // largest magnitude into [128, 256); NaN or infinity: NaN digits
            const bool nan = am >= 0x7F80u;
            const int e = am < 0x0080u ? 120 : max(-120, min(120, 7 + 127 - static_cast<int>(am >> 7)));
            const float f = exp2i(e);
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) {
                const uint32_t a = u4w(w[i >> 1], 2 * (i & 1)), b = u4w(w[i >> 1], 2 * (i & 1) + 1);
                digits4<SPLIT ? kLoShift : 0>(bf16_lo(a) * f, bf16_hi(a) * f, bf16_lo(b) * f, bf16_hi(b) * f, qh[x][i], ql[x][i]);
                if (nan) qh[x][i] = 0x7F7F7F7Fu;
            }
            qs[x] = exp2i(-e) * p.scale_log2;
        }
        const int tile_sees = row_sees(len, n, G, s.tile * TR);  // the tile's first row sees the least

        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[DT][4];
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

        for (int pg = s.p0 + pw; pg < pe; pg += PW) {
            const int it = it0 + pg - s.p0, st = it % NS;
            wait_or_abort(&ct->full[st], (it / NS) & 1, p, ct);
            __syncwarp();
            const uint8_t *kp = smem + st * kStage, *vp = kp + kPage * D;
            const float ks = ct->ks[st], vs = ct->vs[st];
            if (ks < 0.f) {  // no such page: nothing sees its tokens
                __syncwarp();
                if (lane == 0) mbar_arrive(&ct->empty[st]);
                continue;
            }
            // the products go step by step over eight independent accumulators, so
            // that an MMA's latency is covered by the ones beside it
            float sc[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[j][x] = 0.f;
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
                uint4 w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int tok = 16 * (g >> 1) + 2 * j + (g & 1);
                    const int gr = D == 128 ? ((2 * t4 + i) ^ (tok & 7)) : t4;
                    w[j] = *reinterpret_cast<const uint4 *>(kp + tok * D + gr * 16);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int a = 4 * i + 2 * y;  // q's words of this K step: a, a + 1
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (SPLIT)
                            mma_e4m3(sc[j], qh[0][a], ql[0][a], qh[0][a + 1], ql[0][a + 1], u4w(w[j], 2 * y), u4w(w[j], 2 * y + 1));
                        else
                            mma_e4m3(sc[j], qh[0][a], qh[1][a], qh[0][a + 1], qh[1][a + 1], u4w(w[j], 2 * y), u4w(w[j], 2 * y + 1));
                    }
                    if (!SPLIT) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            mma_e4m3(sc[j], ql[0][a], ql[1][a], ql[0][a + 1], ql[1][a + 1], u4w(w[j], 2 * y), u4w(w[j], 2 * y + 1));
                    }
                }
            }
            // scores in log2, masked
            const bool edge = (pg + 1) * kPage > tile_sees;
            const uint32_t vb = __float_as_uint(vs);
            const float lv = static_cast<float>(max(-64, static_cast<int>(vb >> 23) - 127 + ((vb & 0x7FFFFFu) ? 1 : 0)));
            constexpr int NX = SPLIT ? 1 : 2;
            float fs[2] = {qs[0] * ks, qs[1] * ks};
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (SPLIT) {
                    sc[j][0] += sc[j][2] * (1.f / (1 << kLoShift));
                    sc[j][1] += sc[j][3] * (1.f / (1 << kLoShift));
                }
#pragma unroll
                for (int x = 0; x < 2 * NX; ++x) sc[j][x] *= fs[x >> 1];
                if (edge) {
                    const int tok = pg * kPage + 16 * t4 + 2 * j;
#pragma unroll
                    for (int x = 0; x < 2 * NX; ++x)
                        if (tok + (x & 1) >= sees[x >> 1]) sc[j][x] = -INFINITY;
                }
#pragma unroll
                for (int x = 0; x < 2 * NX; ++x) mx[x >> 1] = fmaxf(mx[x >> 1], sc[j][x]);
            }
            float ref[2], alpha[2];
            bool grew = false;
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
                mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
                const float mn = fmaxf(m[x], mx[x] + lv);
                ref[x] = mn == -INFINITY ? 0.f : mn;
                alpha[x] = ex2(m[x] - ref[x]);  // m = -inf: 0
                grew |= mn != m[x];
                m[x] = mn;
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int x = 0; x < NX; ++x) l[x] *= alpha[x];
#pragma unroll
                for (int i = 0; i < DT; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[i][x] *= alpha[SPLIT ? 0 : x >> 1];
            }
            const float pv = vs * 256.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int x = 0; x < 2 * NX; ++x) {
                    const float w = ex2(sc[j][x] - ref[x >> 1]);
                    l[x >> 1] += w;
                    sc[j][x] = w * pv;
                }
            uint32_t ph[2][4], pl[2][4];  // [row][word]: the lane's 16 tokens
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    digits4<SPLIT ? kLoShift : 0>(sc[2 * i][2 * x], sc[2 * i][2 * x + 1], sc[2 * i + 1][2 * x],
                                                  sc[2 * i + 1][2 * x + 1], ph[x][i], pl[x][i]);
#pragma unroll
            for (int i0 = 0; i0 < DT; i0 += 8) {
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = *reinterpret_cast<const uint4 *>(vp + (8 * (i0 + i) + g) * kPage + 16 * t4);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (SPLIT)
                            mma_e4m3(o[i0 + i], ph[0][2 * y], pl[0][2 * y], ph[0][2 * y + 1], pl[0][2 * y + 1],
                                     u4w(w[i], 2 * y), u4w(w[i], 2 * y + 1));
                        else
                            mma_e4m3(o[i0 + i], ph[0][2 * y], ph[1][2 * y], ph[0][2 * y + 1], ph[1][2 * y + 1],
                                     u4w(w[i], 2 * y), u4w(w[i], 2 * y + 1));
                    }
                    if (!SPLIT) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            mma_e4m3(o[i0 + i], pl[0][2 * y], pl[1][2 * y], pl[0][2 * y + 1], pl[1][2 * y + 1],
                                     u4w(w[i], 2 * y), u4w(w[i], 2 * y + 1));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ct->empty[st]);
        }
        it0 += max(pe - s.p0, 0);
        u += s.p1 - s.p0;

        // ---- the segment's result: m, l and o / 256 per row
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        }
        // element (x, i) of the lane: row x ? r_hi : r_lo, head dims 8 i + 2 t4 + {0, 1}
        if (SPLIT) {
#pragma unroll
            for (int i = 0; i < DT; ++i) {
                o[i][0] += o[i][2] * (1.f / (1 << kLoShift));
                o[i][1] += o[i][3] * (1.f / (1 << kLoShift));
            }
        }
        constexpr int NX = SPLIT ? 1 : 2;
        if (PW > 1) {
            // page groups: their sums to shared memory, added in page-group order
            float *mo = mrg, *mm = mrg + kWarps * MR * (D + 4), *ml = mm + kWarps * MR;
            asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");  // the last segment's reads are over
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int rr = wid * MR + 8 * x + g;
                if (t4 == 0) {
                    mm[rr] = m[x];
                    ml[rr] = l[x];
                }
#pragma unroll
                for (int i = 0; i < DT; ++i)
                    *reinterpret_cast<float2 *>(mo + rr * (D + 4) + 8 * i + 2 * t4) = make_float2(o[i][2 * x], o[i][2 * x + 1]);
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        }
        const bool whole = s.p0 == 0 && s.p1 == s.units;
        const int c0 = block_of(U, blocks, s.start), c1 = block_of(U, blocks, s.start + s.units - 1);
        // this block's partial: slot 0 continues a tile, slot 1 starts one
        float *part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (s.p0 == 0 ? 1 : 0)) * (kPartRows * (D + 2));
        auto put = [&](int rr, int d, float a, float b, float mv, float lv) {
            // two neighbouring elements of tile row rr
            if (whole) {
                const int r = s.tile * TR + rr;
                if (r < rows) {
                    const float inv = lv > 0.f || lv != lv ? 1.f / (256.f * lv) : 0.f;
                    *reinterpret_cast<uint32_t *>(p.o + (static_cast<size_t>(q0 + r / G) * c.q_heads + s.h * G + r % G) * D + d) =
                        pack_bf16(a * inv, b * inv);
                }
            } else {
                *reinterpret_cast<float2 *>(part + 2 * TR + rr * D + d) = make_float2(a, b);
                if (d == 0) {
                    part[rr] = mv;
                    part[TR + rr] = lv;
                }
            }
        };
        if (PW > 1) {
            const float *mo = mrg, *mm = mrg + kWarps * MR * (D + 4), *ml = mm + kWarps * MR;
            for (int i = tid; i < TR * (D / 2); i += kWarps * 32) {
                const int rr = i / (D / 2), d = 2 * (i % (D / 2));
                const int w0 = (rr / MR) * PW;
                float mv = -INFINITY, lv = 0.f, a = 0.f, b = 0.f;
#pragma unroll
                for (int k = 0; k < PW; ++k) mv = fmaxf(mv, mm[(w0 + k) * MR + rr % MR]);
                const float ref = mv == -INFINITY ? 0.f : mv;
#pragma unroll
                for (int k = 0; k < PW; ++k) {
                    const int q = (w0 + k) * MR + rr % MR;
                    const float f = ex2(mm[q] - ref);
                    const float2 v = *reinterpret_cast<const float2 *>(mo + q * (D + 4) + d);
                    lv += ml[q] * f;
                    a += v.x * f;
                    b += v.y * f;
                }
                put(rr, d, a, b, mv, lv);
            }
        } else {
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int i = 0; i < DT; ++i)
                    put(rw * MR + 8 * x + g, 8 * i + 2 * t4, o[i][2 * x], o[i][2 * x + 1], m[x], l[x]);
        }
        if (whole) continue;
        // ---- a tile cut between blocks c0 .. c1: the last to arrive joins them
        __threadfence();
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        if (tid == 0) {
            const uint32_t old = atom_add_acqrel_gpu(p.count + c0, 1u);
            ct->last = old == static_cast<uint32_t>(c1 - c0);
            if (ct->last) p.count[c0] = 0u;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        if (!ct->last) continue;
        __threadfence();
        for (int i = tid; i < TR * (D / 2); i += kWarps * 32) {
            const int rr = i / (D / 2), d = 2 * (i % (D / 2)), r = s.tile * TR + rr;
            if (r >= rows) continue;
            float mv = -INFINITY, lv = 0.f, a = 0.f, b = 0.f;
            for (int k = c0; k <= c1; ++k) {
                const float *q = p.part + (static_cast<size_t>(k) * 2 + (k == c0 ? 1 : 0)) * (kPartRows * (D + 2));
                const float mk = __ldcg(q + rr), lk = __ldcg(q + TR + rr);
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(q + 2 * TR + rr * D + d));
                const float mn = fmaxf(mv, mk), ref = mn == -INFINITY ? 0.f : mn;
                const float f0 = ex2(mv - ref), f1 = ex2(mk - ref);
                lv = lv * f0 + lk * f1;
                a = a * f0 + v.x * f1;
                b = b * f0 + v.y * f1;
                mv = mn;
            }
            const float inv = lv > 0.f || lv != lv ? 1.f / (256.f * lv) : 0.f;
            *reinterpret_cast<uint32_t *>(p.o + (static_cast<size_t>(q0 + r / G) * c.q_heads + s.h * G + r % G) * D + d) =
                pack_bf16(a * inv, b * inv);
        }
    }
}

template <int D, int RW, bool SPLIT>
cudaError_t launch_one(const AttendParams &p, int grid, int smem_optin, cudaStream_t st)
{
    constexpr int MR = SPLIT ? 8 : 16;
    const int merge = RW < kWarps ? kWarps * MR * (D + 6) * 4 : 0;
    const int fixed = 1024 + static_cast<int>(sizeof(Control) + sizeof(Seqs)) + merge;
    const int ns = std::min(kMaxStages, (smem_optin - fixed) / Layout<D>::kStage);
    const int smem = fixed + ns * Layout<D>::kStage;
    auto *fn = moe_kv_attend_kernel<D, RW, SPLIT>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchCfg l(dim3(grid), dim3(kThreads), smem, st);
    return cudaLaunchKernelEx(&l.cfg, fn, p, ns);
}

template <int D>
cudaError_t launch_d(const AttendParams &p, int grid, int optin, cudaStream_t st)
{
    switch (attend_tile_rows(static_cast<long long>(p.c.max_q) * (p.c.q_heads / p.c.kv_heads))) {
        case 8: return launch_one<D, 1, true>(p, grid, optin, st);
        case 16: return launch_one<D, 1, false>(p, grid, optin, st);
        case 32: return launch_one<D, 2, false>(p, grid, optin, st);
        case 64: return launch_one<D, 4, false>(p, grid, optin, st);
    }
    return launch_one<D, 8, false>(p, grid, optin, st);
}

}  // namespace

int attend_tile_rows(long long rows)
{
    return rows <= 8 ? 8 : (rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128)));
}

cudaError_t launch_kv_attend(const AttendParams &p, int num_sms, int smem_optin, cudaStream_t st)
{
    return p.c.D == 128 ? launch_d<128>(p, num_sms, smem_optin, st) : launch_d<64>(p, num_sms, smem_optin, st);
}

}  // namespace moe
