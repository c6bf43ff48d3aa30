// moe_linear_tc.cu -- moe_linear for weights of many rows, on the tensor cores.
//
//   y[t, n] = ts[n] * sum_k E2M1(q[n, k]) * E4M3(s[n, k/16]) * x[t, k]
//
// The same product as moe_linear.cu's kernels compute with mma.sync, where the
// issue of instructions bounded it.  Here a block owns up to four tiles of up to
// 128 rows.  Weights arrive by TMA, 256 elements of K of a tile at a time; two
// warpgroups, a thread a row, turn them into fp16 (E2M1 times E4M3 is exact there)
// and store them to tensor memory as the A operand of tcgen05.mma (shared memory
// would have to take and give each of those bytes, at four times the weights' own);
// tokens are the N axis (16 or 32), staged in shared memory as fp16.  The tiles
// take a piece of K in turn, so x passes by once.  The rows of a tile are the
// block's rows over its tiles, not 128: every block brings the same number of bytes.
//
// 24 tokens, 65543 rows of 4096: 44.7 us, 52% of the rate at which memory could
// bring the weights (66 us with mma.sync).  No unit is full (issue 51%, ALU 43%, DRAM
// 38% in a profile): the eight converting warps' waits bound it, two warps a scheduler with
// little to cover them (loads of codes, their stores to tensor memory, a free buffer, and
// every 512 elements the end of the products, 4 us), then the pass over x that finds
// the tokens' scales (every block reads all of x before its first product, 5 us).
//
// x enters as fp16 after a power-of-two scale of each token, from its largest
// element and undone at the end: bf16's 8 bits are exact down to 2^-31 of the
// token's largest, and what is smaller is off by at most 2^-39 of that largest.
//
// Sums on the tensor cores run over 512 elements of K, then go on in fp32 additions
// that round, in tensor memory beside them: 1.1e-7 of the result's norm at K = 4096,
// as with mma.sync; in one run over all of K, 1e-6 (and 40.4 us).
//
// A wait that runs out (bounded as everywhere) leaves NaN in the block's rows.
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
#include "moe_tcgen05.cuh"

constexpr int kRows = 128;      // of a tile: tensor-memory lanes
constexpr int kTiles = 4;       // of a block
constexpr int kPiece = 256;     // elements of K of a stage
constexpr int kCodes = kRows * kPiece / 2;  // bytes of a stage
constexpr int kThreads = 512;
// first warps of each kind
constexpr int kProducer = 0, kIssuer = 1, kStager = 4, kConverter = 8;  // (two issuers)
constexpr int kTmemCols = 512;
// Pieces of a tile whose products are added up on the tensor cores before the sum
// goes on in fp32 additions that round: a long run there loses a digit.
constexpr int kRun = 2;

// Buffers of A in tensor memory (128 elements of K, 64 columns each) that a
// converting warpgroup has: the columns that accumulators and sums leave.
template <int TN>
__host__ __device__ constexpr int buffers() { return (kTmemCols - 2 * kTiles * TN) / 64 / 2; }
// Stages of weights: an even number, so that a stage always belongs to the same
// warpgroup (a barrier's parity tells neighbouring phases apart, no more).
constexpr int kStages = 10;

struct Control {
    alignas(16) float scale[32], back[32];  // each token's power of two and its inverse
    uint64_t full[kStages], empty[kStages];
    uint64_t x_full[2], x_empty[2];
    uint64_t a_full[2][3], a_empty[2][3];
    uint64_t d_ready, drained[2];
    uint32_t amax[32];          // largest magnitude of each token, as bits
    uint32_t tmem;
    int issued;                 // stages of weights that were issued
    int abort;
};

// Bounded wait; a block that gave up goes on without waiting.
__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, long long timeout_ns, int *abort_flag)
{
    uint64_t t0 = 0;  // (reading the timer takes long: not before many tries have failed)
#pragma unroll 1
    for (uint32_t it = 1; !mbar_test(bar, parity); ++it) {
        if ((it & 31u) != 0) continue;
        if (*reinterpret_cast<volatile int *>(abort_flag)) return;
        const uint64_t t = gtimer();
        if (t0 == 0) t0 = t;
        if (static_cast<long long>(t - t0) > timeout_ns) {
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
            return;
        }
    }
}

// Descriptor of a K-major tile: rows of 128 bytes, swizzled over 128 bytes, 8-row
// groups 1024 bytes apart; the low word holds the address.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// D[128 x N] (+)= A B^T: fp16 operands, A in tensor memory
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d), "r"(a), "r"(b_lo), "r"(kDescHi), "r"(idesc),
        "r"(add)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&u)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}

template <int TN>
__global__ void __launch_bounds__(kThreads, 1) moe_linear_tc_kernel(const __grid_constant__ LinearTcParams tp)
{
    constexpr int NS = kStages, NB = buffers<TN>();
    constexpr int kX = TN * kPiece * 2;  // bytes of a piece of x: four blocks of 64 elements, TN rows of 128 bytes
    extern __shared__ uint8_t smem_raw[];
    uint8_t *codes = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *xbuf = codes + NS * kCodes;
    Control *ct = reinterpret_cast<Control *>(xbuf + 2 * kX);
    const LinearParams &p = tp.l;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int tok0 = blockIdx.y * TN, T = min(p.T - tok0, TN);
    const int row0 = blockIdx.x * tp.tiles * tp.rows, tiles = tp.tiles;  // (tiles past the last row are zeros)
    const int pieces = p.K / kPiece, total = pieces * tiles;
    auto aborted = [&] { return *reinterpret_cast<volatile int *>(&ct->abort) != 0; };
    auto wait = [&](uint64_t *bar, uint32_t parity) { wait_or_abort(bar, parity, tp.timeout_ns, &ct->abort); };

    if (tid == 0) {
        ct->abort = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(&ct->full[i], 1);
            mbar_init(&ct->empty[i], 128);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ct->x_full[b], 128);
            mbar_init(&ct->x_empty[b], 2);
            mbar_init(&ct->drained[b], 1);
            for (int i = 0; i < NB; ++i) {
                mbar_init(&ct->a_full[b][i], 128);
                mbar_init(&ct->a_empty[b][i], 1);
            }
        }
        mbar_init(&ct->d_ready, 2);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < TN) ct->amax[tid] = 0;
    // tensor memory before the next kernel may start: its blocks can take theirs ahead of
    // their wait for this one (as these do), which must not have to wait for them in turn
    if (wid == kIssuer) tc_alloc(&ct->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();
    grid_release();
    const uint32_t tmem = ct->tmem, ta = tmem + kTmemCols - 2 * NB * 64;

    if (wid == kProducer) {
        // ---- weights
        if (lane == 0) {
            const uint64_t pol = gridDim.y > 1 ? policy_evict_last() : policy_evict_first();
            int it = 0;
            for (int k = 0; k < pieces; ++k)
                for (int m = 0; m < tiles; ++m, ++it) {
                    const int st = it % NS;
                    if (it >= NS) wait(&ct->empty[st], (it / NS - 1) & 1);
                    if (aborted()) goto out;  // (what is issued stays a run from the first on)
                    mbar_expect_tx(&ct->full[st], tp.rows * (kPiece / 2));
                    tma2d(codes + st * kCodes, &tp.tm_q, k * (kPiece / 2), row0 + m * tp.rows, &ct->full[st], pol);
                }
        out:
            ct->issued = it;
        }
    } else {
        // ---- each token's largest element: a warp takes 256 elements of a token at a time
        constexpr int kWarps = kThreads / 32 - 1, kBatch = 13;
        struct Item {
            int tok, k;  // (k in pieces)
            __device__ __forceinline__ void next(int pieces)
            {
                for (k += kWarps; k >= pieces; k -= pieces) ++tok;
            }
        };
        Item i{(wid - 1) / pieces, (wid - 1) % pieces};
        while (i.tok < T) {
            uint4 a[kBatch];
            Item j = i;
#pragma unroll
            for (int v = 0; v < kBatch; ++v, j.next(pieces))
                a[v] = j.tok < T ? __ldg(reinterpret_cast<const uint4 *>(
                                       p.x + static_cast<long long>(tok0 + j.tok) * p.x_stride + j.k * kPiece + 8 * lane))
                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int v = 0; v < kBatch; ++v, i.next(pieces)) {
                uint32_t am = 0u;
#pragma unroll
                for (int w = 0; w < 4; ++w) am = __vmaxu2(am, u4w(a[v], w) & 0x7FFF7FFFu);
                am = __reduce_max_sync(0xffffffffu, max(am >> 16, am & 0xFFFFu));
                if (lane == 0 && i.tok < T) atomicMax(&ct->amax[i.tok], am);
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 32) : "memory");
        if (const int tok = tid - 32; tok < TN) {
            const int e = min(126, f16_prescale_exp(__uint_as_float(ct->amax[tok] << 16)));
            ct->scale[tok] = exp2i(e);
            ct->back[tok] = exp2i(-e);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 32) : "memory");
    }

    if (wid == kIssuer || wid == kIssuer + 1) {
        // ---- products, a thread for each converting warpgroup's (one alone would take
        // longer to issue them than they take): no two add to the same accumulator.
        // A block that gave up goes on without waiting, on whatever is there.
        const int w = __shfl_sync(0xffffffffu, wid, 0) - kIssuer;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t xd = (smem_u32(xbuf) >> 4) | (1u << 16);
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(TN >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
        int b = 0;
        uint32_t phase = 0;
        for (int k = 0; k < pieces; ++k) {
            wait(&ct->x_full[k & 1], (k >> 1) & 1);
            for (int it = k * tiles + ((k * tiles ^ w) & 1); it < (k + 1) * tiles; it += 2) {
                const uint32_t d = tm + (tiles == 1 ? w : it - k * tiles) * TN;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    wait(&ct->a_full[w][b], phase);
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t a = tm + kTmemCols - 2 * NB * 64 + (w * NB + b) * 64, x = xd + ((k & 1) * kX + half * (kX / 2)) / 16;
                    const uint32_t add = half > 0 || (tiles == 1 ? k >> 1 : k) % kRun != 0;
                    if (elect_one()) {
                        mma_f16_ts(d, a, x, idesc, add);
#pragma unroll
                        for (int j = 1; j < 8; ++j)
                            mma_f16_ts(d, a + 8 * j, x + (j >> 2) * (TN * 128 / 16) + 2 * (j & 3), idesc, 1);
                        tc_commit(&ct->a_empty[w][b]);
                    }
                    __syncwarp();
                    if (++b == NB) {
                        b = 0;
                        phase ^= 1;
                    }
                }
            }
            if (elect_one()) tc_commit(&ct->x_empty[k & 1]);
        }
        if (elect_one()) tc_commit(&ct->d_ready);
    } else if (wid >= kStager && wid < kConverter) {
        // ---- x: items of 8 elements, item i is token i / 32, elements 8 (i % 32) .. of the piece
        constexpr int kItems = TN * kPiece / 8 / 128;
        const int t = tid - 32 * kStager, g = t & 31;
        float f[kItems];
#pragma unroll
        for (int v = 0; v < kItems; ++v) f[v] = ct->scale[(t >> 5) + 4 * v];
        for (int k = 0; k < pieces; ++k) {
            uint4 a[kItems];
#pragma unroll
            for (int v = 0; v < kItems; ++v) {
                const int tok = (t >> 5) + 4 * v;
                if (tok < T)
                    a[v] = __ldg(reinterpret_cast<const uint4 *>(p.x + static_cast<long long>(tok0 + tok) * p.x_stride +
                                                                 k * kPiece + 8 * g));
            }
            if (k >= 2) wait(&ct->x_empty[k & 1], ((k >> 1) - 1) & 1);
#pragma unroll
            for (int v = 0; v < kItems; ++v) {
                const int tok = (t >> 5) + 4 * v;
                if (tok < T)  // (the columns of other tokens are never written out)
                    *reinterpret_cast<uint4 *>(xbuf + (k & 1) * kX + (g >> 3) * (TN * 128) + tok * 128 +
                                               (((g & 7) ^ (tok & 7)) << 4)) =
                        make_uint4(bf16x2_to_f16x2_scaled(a[v].x, f[v]), bf16x2_to_f16x2_scaled(a[v].y, f[v]),
                                   bf16x2_to_f16x2_scaled(a[v].z, f[v]), bf16x2_to_f16x2_scaled(a[v].w, f[v]));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(&ct->x_full[k & 1]);
        }
    } else if (wid >= kConverter) {
        // ---- weights to fp16 in tensor memory: warpgroup w takes every other stage, a thread a row
        const int row = (tid - 32 * kConverter) & (kRows - 1), w = (wid - kConverter) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(wid & 3) << 21;  // this warp's tensor-memory lanes
        int b = 0, used = 0;
        uint32_t phase = 0;  // of buffer b: how often it has been around
        // a row's scales of a stage: 16 bytes, straight to registers (boxes 16 bytes wide
        // took the TMA unit longer than the codes do), two of the warpgroup's stages ahead
        struct Place {
            int k, m;  // piece and tile of a stage
            __device__ __forceinline__ void next(int tiles)
            {
                for (m += 2; m >= tiles; m -= tiles) ++k;
            }
        } at{w / tiles, w % tiles};
        auto load_scales = [&] {
            const int n = min(row0 + at.m * tp.rows + min(row, tp.rows - 1), p.N - 1);
            const uint4 r = at.k < pieces ? __ldg(reinterpret_cast<const uint4 *>(p.s + static_cast<size_t>(n) * (p.K / 16)) + at.k)
                                          : make_uint4(0u, 0u, 0u, 0u);
            at.next(tiles);
            return r;
        };
        uint4 s1st = load_scales(), s2nd = load_scales();
        // a tile's sum so far: from the accumulator, which the next run starts over, to
        // columns of its own.  The tile's last stage was this warpgroup's last or, with four
        // tiles, the one before; its products are done when its last buffer is free.
        Place now{w / tiles, w % tiles};
        auto keep_sum = [&](int slot, bool more) {
            const int last = used - (tiles == kTiles ? 3 : 1);
            if (last + NB >= used) wait(&ct->a_empty[w][last % NB], (last / NB) & 1);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < TN; c += 16) {
                const uint32_t at = tmem + lanes + slot * TN + c;
                float v[16], u[16];
                uint32_t x[16];
                tc_ld16(at, v);
                if (more) tc_ld16(at + kTiles * TN, u);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(more ? v[j] + u[j] : v[j]);
                tc_st16(at + kTiles * TN, x);
            }
            tc_wait_st();
        };
        int st = w;
        uint32_t round = 0;
        for (int it = w; it < total; it += 2) {
            const uint8_t *src = codes + st * kCodes + row * 128;
            const uint4 s16 = s1st;
            s1st = s2nd;
            s2nd = load_scales();
            if (const int run = tiles == 1 ? now.k >> 1 : now.k; run > 0 && run % kRun == 0)
                keep_sum(tiles == 1 ? w : now.m, run > kRun);
            now.next(tiles);
            wait(&ct->full[st], round);
            uint4 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = *reinterpret_cast<const uint4 *>(src + ((i ^ (row & 7)) << 4));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (used >= NB) wait(&ct->a_empty[w][b], phase ^ 1);
                __syncwarp();
                tc_fence_after();
                const uint32_t dst = ta + lanes + (w * NB + b) * 64;
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // 32 codes, two scales
                    const uint32_t sc = e4m3x2_to_f16x2(static_cast<uint16_t>(u4w(s16, 2 * half + (i >> 1)) >> (16 * (i & 1))));
                    const uint32_t s0 = __byte_perm(sc, 0u, 0x1010), s1 = __byte_perm(sc, 0u, 0x3232);
                    uint32_t h[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e2m1x8_to_f16x2(u4w(q[4 * half + i], j), h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
#pragma unroll
                        for (int z = 0; z < 4; ++z) h[4 * j + z] = hmul2(h[4 * j + z], j < 2 ? s0 : s1);
                    }
                    tc_st16(dst + 16 * i, h);
                    if (half == 0 && i == 0) mbar_arrive(&ct->empty[st]);  // (the codes are in registers)
                }
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&ct->a_full[w][b]);
                ++used;
                if (++b == NB) {
                    b = 0;
                    phase ^= 1;
                }
            }
            if ((st += 2) >= NS) {
                st -= NS;
                round ^= 1;
            }
        }
        // ---- the result: lane is the row, column the token
        float ts[kTiles / 2];
#pragma unroll
        for (int i = 0; i < kTiles / 2; ++i) {
            const int m = w + 2 * i, n = row0 + m * tp.rows + row;
            ts[i] = m < tiles && row < tp.rows && n < p.N ? p.ts[n] : 0.f;
        }
        wait(&ct->d_ready, 0);
        __syncwarp();
        tc_fence_after();
        const float nan = __int_as_float(0x7FC00000);
        const bool poison = aborted(), two = tiles == 1 && pieces > 1;  // two: one tile, each warpgroup's half of K apart
        // sums kept beside the accumulators
        const bool sums = (tiles == 1 ? (pieces + 1) / 2 : pieces) > kRun, sums2 = pieces / 2 > kRun;
#pragma unroll
        for (int i = 0; i < kTiles / 2; ++i) {
            const int m = w + 2 * i, n = row0 + m * tp.rows + row;
            if (m >= tiles) continue;
            const bool in = row < tp.rows && n < p.N;
            const size_t N = p.N;
            size_t o = tok0 * N + n;
#pragma unroll 1
            for (int c = 0; c < T; c += 4, o += 4 * N) {
                float4 v, u[3] = {};
                __syncwarp();
                tc_ld4(tmem + lanes + m * TN + c, v);
                if (sums) tc_ld4(tmem + lanes + (kTiles + m) * TN + c, u[0]);
                if (two) tc_ld4(tmem + lanes + TN + c, u[1]);
                if (two && sums2) tc_ld4(tmem + lanes + (kTiles + 1) * TN + c, u[2]);
                tc_wait_ld();
                if (!in) continue;
                const float4 f = *reinterpret_cast<const float4 *>(&ct->back[c]);
                v = f4add(f4add(v, u[0]), f4add(u[1], u[2]));
                const float y[4] = {v.x * f.x * ts[i], v.y * f.y * ts[i], v.z * f.z * ts[i], v.w * f.w * ts[i]};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (c + j >= T) break;
                    if (p.y_bf16)
                        static_cast<uint16_t *>(p.y)[o + j * N] = static_cast<uint16_t>(pack_bf16(poison ? nan : y[j], 0.f));
                    else
                        static_cast<float *>(p.y)[o + j * N] = poison ? nan : y[j];
                }
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    // No block ends with a copy into its shared memory or a product in flight: each was waited
    // for, unless the block gave up.  (Asked where all warps have met: nobody waits, and
    // so gives up, any more.)
    if (aborted()) {
        const uint64_t t0 = gtimer();
        auto landed = [&](uint64_t *bar, uint32_t parity) {
            while (!mbar_test(bar, parity) && static_cast<long long>(gtimer() - t0) < tp.timeout_ns) {
            }
        };
        if (wid == kProducer && lane == 0)
            ring_drain(ct->issued, NS, [&](int st, uint32_t parity) { landed(&ct->full[st], parity); });
        if ((wid == kIssuer || wid == kIssuer + 1) && elect_one()) {  // (the lane that issued them)
            tc_commit(&ct->drained[wid - kIssuer]);
            landed(&ct->drained[wid - kIssuer], 0);
        }
        __syncwarp();
        __syncthreads();
    }
    if (wid == kIssuer) tc_dealloc(tmem, kTmemCols);
}

template <int TN>
cudaError_t launch_tn(const LinearTcParams &p, int blocks, cudaStream_t st)
{
    constexpr int smem = 1024 + kStages * kCodes + 2 * TN * kPiece * 2 + static_cast<int>(sizeof(Control));
    static_assert(smem <= 227 * 1024, "shared memory of a block");
    static_assert(buffers<TN>() <= 3, "barriers of the buffers of A");
    auto *fn = moe_linear_tc_kernel<TN>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchCfg l(dim3(blocks, (p.l.T + TN - 1) / TN), dim3(kThreads), smem, st);
    return cudaLaunchKernelEx(&l.cfg, fn, p);
}

}  // namespace

LinearTcPlan linear_tc_plan(const LinearParams &p, int num_sms)
{
    // rows a block, from as many full waves of blocks as it takes; spread over its tiles
    const int waves = (p.N + num_sms * kTiles * kRows - 1) / (num_sms * kTiles * kRows);
    const int per = (p.N + num_sms * waves - 1) / (num_sms * waves);
    LinearTcPlan r;
    r.tiles = per <= kRows ? 1 : (per <= 2 * kRows ? 2 : kTiles);  // one, or as many for either warpgroup
    r.rows = (per + r.tiles - 1) / r.tiles;
    r.blocks = (p.N + r.tiles * r.rows - 1) / (r.tiles * r.rows);
    return r;
}

cudaError_t launch_linear_tc(const LinearTcParams &p, int blocks, cudaStream_t st)
{
    return p.l.T <= 16 ? launch_tn<16>(p, blocks, st) : launch_tn<32>(p, blocks, st);
}

}  // namespace moe
