// moe_kv_attend.cu -- causal attention over the paged 8-bit cache
// (moe_kv_attend) for few query rows: single tokens, short verification runs.
//
//   o[i, h] = sum_t w_t v[t] / sum_t w_t,   w_t = 2^(s_t - m),
//   s_t = log2(e) scale q.k_t
//
// in one pass over the cache with a running maximum m and sum.  The cache's
// bytes bound it: each page and kv head is read once for all query heads that
// share it (a decode batch of ragged lengths, 1.1 GB of cache: 178 us, 93% of the
// measured copy rate; one sequence of 4002 tokens: 11.1 us, its fixed costs).  The E4M3 codes become fp16 in registers (exact) for mma.sync
// m16n8k16; q enters as fp16 after a power-of-two prescale of its row (exact
// for elements down to 2^-28 of the row's largest), the weights as fp16 of 256 w vs (vs: the
// page's v scale over the largest that the maximum allows for); their sum
// stays in fp32, as all accumulators do.  (The tensor cores' additions cut instead of
// rounding: with values of one sign a sum loses 8e-10 of itself for each token that one
// block adds up, 7e-5 over 131072.)  The running maximum is taken over
// s + ceil(log2(vs)), so that the fp16 weights have their range for what is
// actually added, whatever the pages' scales.
//
// A block's 8 warps take the pages of its run in turn, two warps a page (half its
// tokens each: the sooner a page is done, the more of the ring is in flight), with
// their own maximum, sum and accumulators (16 rows x head dim), and add up at a
// tile's end in warp order; nothing but the ring of pages couples them.
//
// Order inside a page is free as long as both products agree: column c of
// score tile j is token 16 (c / 2) + 2 j + c % 2, which makes a lane's weights of
// a row consecutive tokens that it reads of a v row (8 of 16 a warp), and a lane's
// k and q elements 32 (head dim 128) or 16 consecutive ones.  k comes by TMA with
// the 128-byte swizzle, free of bank conflicts; v as it lies, its 8-byte reads
// two to a bank.
#include "moe_internal.h"
#include "moe_layer_internal.h"
#include "moe_ring.h"

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

namespace moe {
namespace {
#include "moe_device.cuh"
#include "moe_layer_device.cuh"

#include "moe_attend.cuh"

constexpr int kWarps = 8;
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 128;  // consumers, and a warpgroup of producers
// Registers a thread of the two kinds keeps: 256 * 216 + 128 * 72 = 64512, what
// the block is launched with (384 threads of 168).
constexpr int kConsumerRegs = 216, kProducerRegs = 72;

// What beginning and ending a tile costs, in pages.
constexpr int kTileCost = 4;
constexpr int kPageWarps = 2;  // warps that share a page: tokens 8 h .. 8 h + 7 of every 16
// Page n of a block is group n % kGroups's, in stage n % NS.  NS is a multiple of
// kGroups, so a stage has one group for good: with another it could be waited
// for a phase ahead (a group can be done with its pages while an earlier page of
// another group is still on its way), and a barrier only tells neighbouring phases apart.
constexpr int kGroups = kWarps / kPageWarps;

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    float ks[kMaxStages], vs[kMaxStages];  // scales of the stage's page; ks < 0: no such page
    int issued[4];  // by a producer warp: one past its last page
    int abort, last;
};

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Columns of the weighted sums that the warps add at a time: what fits beside the ring.
__host__ __device__ constexpr int merge_cols(int D, int NX) { return D < 64 / NX ? D : 64 / NX; }

// NX: query rows of a tile / 8 (1 or 2).  Shared memory: ring of stages (k page,
// v page), the control block, the sequences, the warps' results.  TREE: the new tokens
// are trees, and see the way to their root instead of all before them.
template <int D, int NX, bool TREE>
__global__ void __launch_bounds__(kThreads, 1) moe_kv_attend_kernel(const __grid_constant__ AttendParams p, int NS)
{
    constexpr int TR = 8 * NX;                  // query rows of a tile
    constexpr int KS = D / 16;                  // K steps of the first product
    constexpr int DT = D / 8;                   // N tiles of the second
    constexpr int NJ = 8 / kPageWarps;          // score tiles of a warp
    constexpr int CC = merge_cols(D, NX);
    constexpr int kStage = 2 * kPage * D;
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
            mbar_init(&ct->full[i], 2);  // k and v
            mbar_init(&ct->empty[i], kPageWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_wait();
    grid_release();
    plan_units<kTileCost, TREE>(p, sq, G, TR);
    const long long U = sq.cum[c.B];
    const int blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), U));
    if (static_cast<int>(blockIdx.x) >= blocks) return;
    const long long u0 = block_start(U, blocks, blockIdx.x), u1 = block_start(U, blocks, blockIdx.x + 1);

    if (wid >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        // ---- producers: a page a stage; warps 0 and 2 bring k, 1 and 3 v, of even and
        // odd pages (one thread's issue alone would bound the kernel)
        const bool values = wid & 1;
        const int odd = (wid - kWarps) >> 1;
        int it = 0, issued = 0;
        const uint64_t pol = policy_evict_first();
        for (long long u = u0; u < u1;) {
            const Segment s = locate<kTileCost>(sq, c.B, G, TR, u, u1);
            for (int pb = s.p0; pb < s.pe; pb += 32) {
                const PageInfo pi = load_pages(c, s, pb);
                const int m = min(32, s.pe - pb);
                for (int i = (it & 1) ^ odd; i < m; i += 2) {
                    const int n = it + i, st = n % NS;
                    const int pid = __shfl_sync(0xffffffffu, pi.id, i);
                    const float scale = __shfl_sync(0xffffffffu, values ? pi.vs : pi.ks, i);
                    if (lane == 0) {
                        if (n >= NS) wait_or_abort(&ct->empty[st], (n / NS - 1) & 1, p, &ct->abort);
                        if (*reinterpret_cast<volatile int *>(&ct->abort) == 0) {
                            (values ? ct->vs : ct->ks)[st] = scale;
                            uint8_t *dst = smem + st * kStage + (values ? kPage * D : 0);
                            const size_t ph = static_cast<size_t>(max(pid, 0)) * c.kv_heads + s.h;
                            if (pid < 0) {
                                mbar_arrive(&ct->full[st]);
                            } else {
                                mbar_expect_tx(&ct->full[st], kPage * D);
                                if (values || D == 64)
                                    bulk_g2s(dst, (values ? c.v : c.k) + ph * (kPage * D), kPage * D, &ct->full[st], pol);
                                else
                                    tma2d(dst, &c.tm_k, 0, static_cast<int>(ph * kPage), &ct->full[st], pol);
                            }
                            issued = n + 1;
                        }
                    }
                    __syncwarp();
                }
                it += m;
            }
            u += s.units;
        }
        if (lane == 0) ct->issued[wid - kWarps] = issued;
    } else {
        // ---- consumers
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
        int it0 = 0;  // pages of this block before the segment
        for (long long u = u0; u < u1;) {
            const Segment s = locate<kTileCost>(sq, c.B, G, TR, u, u1);
            u += s.units;
            if (s.p1 == 0) continue;
            const int n = sq.n[s.b], len = sq.len[s.b], rows = n * G, q0 = sq.q0[s.b];

            // q: fp16 of the lane's D / 4 elements of rows g and g + 8 of the tile
            uint32_t qf[2][2 * KS];
            float qs[NX];
            int sees[NX];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = s.tile * TR + 8 * x + g;
                const bool in = x < NX && r < rows;
                uint4 w[KS / 2];
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + static_cast<long long>(q0 + r / G) * p.q_stride +
                                                                   (s.h * G + r % G) * D + (D / 4) * t4);
#pragma unroll
                for (int i = 0; i < KS / 2; ++i) w[i] = in ? src[i] : make_uint4(0u, 0u, 0u, 0u);
                if (x < NX) {
                    uint32_t am = 0u;  // largest magnitude, as bits (16-bit halves)
#pragma unroll
                    for (int i = 0; i < 2 * KS; ++i) am = __vmaxu2(am, u4w(w[i >> 2], i & 3) & 0x7FFF7FFFu);
                    am = max(am >> 16, am & 0xFFFFu);
                    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
                    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
                    const int e = max(-120, min(120, f16_prescale_exp(__uint_as_float(am << 16))));
                    const float f = exp2i(e);
#pragma unroll
                    for (int i = 0; i < 2 * KS; ++i) qf[x][i] = bf16x2_to_f16x2_scaled(u4w(w[i >> 2], i & 3), f);
                    // a NaN or an infinity in the row: NaN scores
                    qs[x < NX ? x : 0] = am >= 0x7F80u ? __int_as_float(0x7FC00000) : exp2i(-e) * p.scale_log2;
                    sees[x < NX ? x : 0] = in ? row_sees(len, n, G, r) : 0;
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * KS; ++i) qf[x][i] = 0u;
                }
            }
            // the tile's first row sees the least; of a tree's tokens each sees what is before the tree
            const int tile_sees = TREE ? max(len - n, 0) : row_sees(len, n, G, s.tile * TR);

            // TREE: parents, a token a lane, loaded ahead of the pages that hold tokens of the tree
            // (walking back from each row there, a load a token: 32 trees of 4 tokens after 8192 in 79.7 us
            // against 76.4; without a tree 73).  A tree of more than 32 tokens comes here only
            // under a max_q that is too small, and is walked.
            int parent = -1;
            if (TREE && lane < n) parent = tree_parent(p, q0, lane);

            float m[NX], l[NX];
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                m[x] = -INFINITY;
                l[x] = 0.f;
            }
            float o[DT][4];
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

            const int half = wid % kPageWarps;
            for (int pg = s.p0 + (wid / kPageWarps + kGroups - it0 % kGroups) % kGroups; pg < s.pe; pg += kGroups) {
                const int it = it0 + pg - s.p0, st = it % NS;
                wait_or_abort(&ct->full[st], (it / NS) & 1, p, &ct->abort);
                __syncwarp();
                const uint8_t *kp = smem + st * kStage, *vp = kp + kPage * D;
                const float ks = ct->ks[st], vs = ct->vs[st];
                if (ks < 0.f) {  // no such page: nothing sees its tokens
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ct->empty[st]);
                    continue;
                }
                // scores: K step by K step over independent accumulators
                float sc[NJ][4];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[j][x] = 0.f;
#pragma unroll
                for (int i = 0; i < KS / 4; ++i) {
                    uint4 w[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int tok = 16 * (g >> 1) + 2 * (NJ * half + j) + (g & 1);
                        const int gr = D == 128 ? ((2 * t4 + i) ^ (tok & 7)) : t4;
                        w[j] = *reinterpret_cast<const uint4 *>(kp + tok * D + gr * 16);
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int a = 2 * (4 * i + y);
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            const uint32_t k4 = u4w(w[j], y);
                            mma16816(sc[j], qf[0][a], qf[1][a], qf[0][a + 1], qf[1][a + 1],
                                     e4m3x2_to_f16x2(static_cast<uint16_t>(k4)), e4m3x2_to_f16x2(static_cast<uint16_t>(k4 >> 16)));
                        }
                    }
                }
                // in log2 units, masked; their maximum
                const bool edge = (pg + 1) * kPage > tile_sees;
                const float lv = scale_log2(vs), pv = vs * 256.f;
                float fs[NX], mx[NX];
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    fs[x] = qs[x] * ks;
                    mx[x] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int x = 0; x < 2 * NX; ++x) {
                        sc[j][x] *= fs[x >> 1];
                        if (!TREE && edge && pg * kPage + 16 * t4 + 2 * (NJ * half + j) + (x & 1) >= sees[x >> 1]) sc[j][x] = -INFINITY;
                        if (!TREE) mx[x >> 1] = fmaxf(mx[x >> 1], sc[j][x]);
                    }
                if (TREE && edge) {
                    // a token's way to the root: its parent's added, and on from the parent's parent
                    uint32_t way = 1u << lane;
                    if (n <= 32)
                        for (int up = parent; __any_sync(0xffffffffu, up >= 0);) {
                            const uint32_t its = __shfl_sync(0xffffffffu, way, up & 31);
                            const int next = __shfl_sync(0xffffffffu, up, up & 31);
                            if (up >= 0) way |= its, up = next;
                        }
#pragma unroll
                    for (int x = 0; x < NX; ++x) {  // the page's tokens that a row sees, the lane's first lowest
                        const int r = s.tile * TR + 8 * x + g;
                        uint64_t w[1] = {0ull};  // (a row past the sequence's sees nothing)
                        if (n <= 32) {
                            const uint32_t its = __shfl_sync(0xffffffffu, way, (r / G) & 31);
                            w[0] = tree_page(r < rows ? its : 0u, pg * kPage - (len - n));
                        } else if (r < rows) {
                            tree_sees<1>(p, q0, len - n, r / G, pg, w);
                        }
                        const uint32_t see = static_cast<uint32_t>(w[0] >> (16 * t4 + 2 * NJ * half));
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if (!((see >> (2 * j + y)) & 1u)) sc[j][2 * x + y] = -INFINITY;
                    }
                    __syncwarp();
                }
                if (TREE)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int x = 0; x < 2 * NX; ++x) mx[x >> 1] = fmaxf(mx[x >> 1], sc[j][x]);
                float ref[NX], alpha[NX];
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
                        for (int x = 0; x < 2 * NX; ++x) o[i][x] *= alpha[x >> 1];
                }
                uint32_t pf[2][NJ];  // weights: [row][token pair]
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (x < NX) {
                            const int y = x < NX ? x : 0;
                            const float a = ex2(sc[j][2 * y] - ref[y]), b = ex2(sc[j][2 * y + 1] - ref[y]);
                            l[y] += a + b;
                            pf[x][j] = cvt_f16x2(a * pv, b * pv);
                        } else {
                            pf[x][j] = 0u;
                        }
                    }
#pragma unroll
                for (int i0 = 0; i0 < DT; i0 += 8) {
                    uint2 w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = *reinterpret_cast<const uint2 *>(vp + (8 * (i0 + i) + g) * kPage + 16 * t4 + 8 * half);
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t v4 = y ? w[i].y : w[i].x;
                            mma16816(o[i0 + i], pf[0][2 * y], pf[1][2 * y], pf[0][2 * y + 1], pf[1][2 * y + 1],
                                     e4m3x2_to_f16x2(static_cast<uint16_t>(v4)), e4m3x2_to_f16x2(static_cast<uint16_t>(v4 >> 16)));
                        }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ct->empty[st]);
            }
            it0 += s.pe - s.p0;

            // ---- the warps' sums to shared memory, added in warp order, CC columns at a time
            float *mo = mrg, *mm = mrg + kWarps * TR * (CC + 4), *ml = mm + kWarps * TR;
            float *part = part_slot(p, blockIdx.x, s.p0 == 0);
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            }
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += CC) {
                __syncwarp();
                asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");  // the last reads are over
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    const int rr = wid * TR + 8 * x + g;
                    if (t4 == 0) {
                        mm[rr] = m[x];
                        ml[rr] = l[x];
                    }
#pragma unroll
                    for (int i = 0; i < CC / 8; ++i)
                        *reinterpret_cast<float2 *>(mo + rr * (CC + 4) + 8 * i + 2 * t4) =
                            make_float2(o[c0 / 8 + i][2 * x], o[c0 / 8 + i][2 * x + 1]);
                }
                __syncwarp();
                asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
                for (int i = tid; i < TR * (CC / 2); i += kConsumers) {
                    const int rr = i / (CC / 2), cc = 2 * (i % (CC / 2)), d = c0 + cc, r = s.tile * TR + rr;
                    float mv = -INFINITY, lv = 0.f, a = 0.f, b = 0.f;
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) mv = fmaxf(mv, mm[k * TR + rr]);
                    const float ref = mv == -INFINITY ? 0.f : mv;
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) {
                        const int q = k * TR + rr;
                        const float f = ex2(mm[q] - ref);
                        const float2 v = *reinterpret_cast<const float2 *>(mo + q * (CC + 4) + cc);
                        lv += ml[q] * f;
                        a += v.x * f;
                        b += v.y * f;
                    }
                    if (!s.whole()) {
                        *reinterpret_cast<float2 *>(part_at(part, TR, rr, d)) = make_float2(a, b);
                        if (d == 0) {
                            part[rr] = mv;
                            part[TR + rr] = lv;
                        }
                    } else if (r < rows) {
                        const float inv = inv_sum(256.f, lv);
                        *reinterpret_cast<uint32_t *>(out_row(p, q0, s.h, G, r) + d) = pack_bf16(a * inv, b * inv);
                    }
                }
            }
            if (!s.whole()) join_tile<D, kConsumers, TR>(p, s, U, blocks, rows, q0, G, 256.f, &ct->last, tid);
        }
    }

    // Every copy was waited for by the warp that uses it, unless the block gave up: no block
    // ends with a copy into its shared memory in flight.  (Asked where all warps have met:
    // nobody waits for a page, and so gives up, any more.)
    __syncwarp();
    __syncthreads();
    if (*reinterpret_cast<volatile int *>(&ct->abort) && (wid == kWarps || wid == kWarps + 2) && lane == 0) {
        const int odd = (wid - kWarps) >> 1;
        const uint64_t t0 = gtimer();
        ring_drain_halves(
            odd, ct->issued[2 * odd], ct->issued[2 * odd + 1], NS, [&](int st) { mbar_arrive(&ct->full[st]); },
            [&](int st, uint32_t parity) {
                while (!mbar_test(&ct->full[st], parity) && static_cast<long long>(gtimer() - t0) < p.timeout_ns) {
                }
            });
    }
}

template <int D, int NX, bool TREE>
cudaError_t launch_one(const AttendParams &p, int grid, int smem_optin, cudaStream_t st)
{
    constexpr int kStage = 2 * kPage * D;
    const int fixed = 1024 + static_cast<int>(sizeof(Control) + sizeof(Seqs)) + kWarps * 8 * NX * (merge_cols(D, NX) + 6) * 4;
    const int ns = std::min(kMaxStages, (smem_optin - fixed) / kStage) / kGroups * kGroups;
    const int smem = fixed + ns * kStage;
    auto *fn = moe_kv_attend_kernel<D, NX, TREE>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchCfg l(dim3(grid), dim3(kThreads), smem, st);
    return cudaLaunchKernelEx(&l.cfg, fn, p, ns);
}

template <bool TREE>
cudaError_t launch_rows(const AttendParams &p, int tile_rows, int num_sms, int smem_optin, cudaStream_t st)
{
    if (p.c.D == 128)
        return tile_rows == 8 ? launch_one<128, 1, TREE>(p, num_sms, smem_optin, st)
                              : launch_one<128, 2, TREE>(p, num_sms, smem_optin, st);
    return tile_rows == 8 ? launch_one<64, 1, TREE>(p, num_sms, smem_optin, st)
                          : launch_one<64, 2, TREE>(p, num_sms, smem_optin, st);
}

}  // namespace

cudaError_t launch_kv_attend_rows(const AttendParams &p, int tile_rows, int num_sms, int smem_optin, cudaStream_t st)
{
    return p.parent ? launch_rows<true>(p, tile_rows, num_sms, smem_optin, st)
                    : launch_rows<false>(p, tile_rows, num_sms, smem_optin, st);
}

}  // namespace moe
