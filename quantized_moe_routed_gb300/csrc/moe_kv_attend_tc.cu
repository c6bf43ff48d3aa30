// moe_kv_attend_tc.cu -- causal attention over the paged 8-bit cache
// (moe_kv_attend) for many query rows: prefill chunks, verification runs.
//
//   o[i, h] = sum_t w_t v[t] / sum_t w_t,   w_t = 2^(s_t - ref),
//   s_t = log2(e) scale q.k_t
//
// A tile is 128 query rows, a step 128 tokens (two pages).  Both products run on
// the tensor cores (tcgen05.mma), their accumulators in tensor memory:
//
//  * S = Q K^T, kind::f8f6f4 on the cache's E4M3 codes as TMA brings them: q enters
//    as two E4M3 digits, hi + lo, after a power-of-two prescale of the row (largest
//    magnitude into [128, 256)): 8 significant bits are two digits of 4, so the
//    sum is exact down to 2^-9 of the row's largest, smaller elements off by 2^-17 of
//    it.  Two digits at twice the 16-bit rate cost what 16-bit operands would.
//  * O += P V, kind::f16: the weights 64 w vs (vs: the page's v scale over the largest
//    that the reference allows for) are rounded to fp16 and written to tensor
//    memory.  v's codes become fp16 (exact) in shared memory; two digits for the
//    weights instead would cost the softmax three more instructions a weight.
//
// The reference is the running maximum of s + ceil(log2(vs)), moved only when a
// step exceeds it by more than 8 (fp16 holds 64 * 2^8), so the accumulators in
// tensor memory are rescaled rarely.
//
// The tensor cores' additions cut what does not fit instead of rounding it: O loses 6e-9 of
// itself a token (weights and values of one sign; 0.6% over a million tokens in one run,
// more than a bf16 output's rounding).  So a run ends after 128 steps: O then goes on in additions
// that round, in the block's place for partial results (no column of tensor memory is
// left), and starts over; 1e-4 is lost.
//
// A group of eight MMAs takes 800 cycles from issue to its barrier, 512 of them at
// work, and a softmax step about 1700: so steps overlap.  Two warpgroups take the
// steps in turn (a thread a row), each with its own S and P in tensor memory; the
// scores of a warpgroup's next step are computed once it has read this one's,
// and P V during the following softmax.  Only the reference goes from step to step, as
// soon as a step's maxima are known.  Two threads bring pages, a warp issues the
// products for S and one those for O, two pairs of warps convert v.  2048 new tokens after
// 16384, 32 heads of 128 on 8: 455 us, 1280 TFLOP/s; a step takes about 1900 cycles, of
// which the tensor cores work 1024 and the exponentials 512; the rest are waits between
// them.  (Before runs ended the chunk took 437 us: ending them costs 2, the code for it in
// the loops the rest.  Measured against 449 then: commits for each page of P, turns for the
// exponentials, four softmax warpgroups, an eighth of the exponentials as polynomials, all
// slower: 484, 537, 524 and 476 us.)  With two row
// tiles a block sharing k and v, tensor memory leaves no room for this (S and P in one
// place): the softmax then waits for the chain from its weights over P V to the next
// scores, 580 us for 2048 x 16384 tokens and 32 heads.
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

#include "moe_attend.cuh"

constexpr int kRows = 128;       // rows of a tile: tensor-memory lanes, threads of a softmax warpgroup
constexpr int kConsumers = 2 * kRows;
constexpr int kThreads = kConsumers + 256;  // and a warpgroup that converts v, one with the producer and the issuers
// Registers a thread of the two kinds keeps: 256 * 200 + 256 * 56 = 65536, what the
// block is launched with (512 threads of 128).
constexpr int kConsumerRegs = 200, kOtherRegs = 56;
constexpr int kKeys = 2 * kPage; // tokens of a step
constexpr float kGain = 64.f;    // of the weights
constexpr float kSlack = 8.f;    // how far a step may exceed the reference (64 * 2^8 is inside fp16)
// Tensor memory: warpgroup b's S at 128 b, its P at 256 + 64 b, O at 384.
constexpr int kTmemCols = 512, kTmemP = 256, kTmemO = 384;
// What beginning and ending a tile (queries, joining, filling and draining) costs,
// in pages: about 14000 cycles against 900 a page.
constexpr int kTileCost = 16;
constexpr int kKStages = 3, kVStages = 4, kFStages = 2;  // steps of k, of v, of v in fp16
constexpr int kRun = 128;        // steps whose weighted sums are added up on the tensor cores: even, so that
                                 // of a segment the same warpgroup ends every run
constexpr int kScales = 8;       // steps whose scales are kept: more than a softmax lags behind the producer

struct Control {
    uint64_t k_full[kKStages], k_empty[kKStages];   // codes of k
    uint64_t v_full[kVStages], v_empty[kVStages];   // codes of v
    uint64_t f_full[kFStages], f_empty[kFStages];   // v in fp16
    uint64_t sc_full[kScales];
    uint64_t q_ready, drained[2];
    uint64_t s_ready[2], s_read[2], ref_ready[2], p_ready[2], o_ready[2];  // of the warpgroups' steps
    float ks[kScales][2], vs[kScales][2];  // scales of a step's pages; ks < 0: no such page
    float qs[kRows];                       // each row's factor from digits to scores (log2 units)
    float ref[2][kRows];                   // the reference after a warpgroup's last step
    float l[2][kRows], lref[2][kRows];     // the warpgroups' sums at a tile's end and what they refer to
    float kref[kRows];                     // what the weighted sums of ended runs refer to
    uint32_t tmem;
    int abort, last;
};

// Matrix descriptors of K-major tiles: rows of 128 bytes with the 128-byte swizzle,
// 8-row groups 1024 bytes apart, or rows of 64 bytes with the 64-byte swizzle, groups
// 512 bytes apart.  The high word is a constant, the low one holds the address, so
// the next step along K is one addition (a lone issuing thread has nothing to
// hide a longer computation behind).
__host__ __device__ constexpr uint32_t desc_hi(int row) { return row == 128 ? (1024u >> 4) | (1u << 14) | (2u << 29) : (512u >> 4) | (1u << 14) | (4u << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }

// D[128 x N] (+)= A B^T: E4M3 operands, both in shared memory
template <bool ADD>
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc),
        "n"(ADD ? 1 : 0)
        : "memory");
}
// The same for fp16 operands, A in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(add)
        : "memory");
}
// Instruction descriptor: fp32 accumulator, E4M3 (kind::f8f6f4) or fp16 (kind::f16)
// A and B, K-major both, M = 128, N = n.
__device__ __forceinline__ uint32_t mma_idesc(int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&r)[32])
{
    uint32_t u[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&u)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}

// Four values (at most 448 in magnitude) as two E4M3 digits: hi the nearest, lo
// the nearest to the rest.
__device__ __forceinline__ void digits4(float a, float b, float c, float d, uint32_t &hi, uint32_t &lo)
{
    asm("{\n .reg .b32 x, y, hx, hy;\n .reg .b16 p, q;\n"
        " cvt.rn.f16x2.f32 x, %3, %2;\n cvt.rn.f16x2.f32 y, %5, %4;\n"
        " cvt.rn.satfinite.e4m3x2.f16x2 p, x;\n cvt.rn.satfinite.e4m3x2.f16x2 q, y;\n mov.b32 %0, {p, q};\n"
        " cvt.rn.f16x2.e4m3x2 hx, p;\n cvt.rn.f16x2.e4m3x2 hy, q;\n"
        " sub.rn.f16x2 x, x, hx;\n sub.rn.f16x2 y, y, hy;\n"
        " cvt.rn.satfinite.e4m3x2.f16x2 p, x;\n cvt.rn.satfinite.e4m3x2.f16x2 q, y;\n mov.b32 %1, {p, q};\n}"
        : "=r"(hi), "=r"(lo)
        : "f"(a), "f"(b), "f"(c), "f"(d));
}

// 16-byte granule gr of row `row` in a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ int granule(int row, int gr)
{
    return row * D + ((D == 128 ? gr ^ (row & 7) : gr ^ ((row >> 1) & 3)) << 4);
}

// Half a query row (two neighbouring threads share a row) as two digits into the tile at dst
// (hi; lo follows kRows * D bytes on); returns the row's factor.
template <int D>
__device__ __forceinline__ float put_query(uint8_t *dst, int row, int half, const uint16_t *src, bool in, float scale)
{
    uint4 w[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
        w[i] = in ? reinterpret_cast<const uint4 *>(src + half * (D / 2))[i] : make_uint4(0u, 0u, 0u, 0u);
    uint32_t am = 0u;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) am = __vmaxu2(am, u4w(w[i >> 2], i & 3) & 0x7FFF7FFFu);
    am = max(am >> 16, am & 0xFFFFu);
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    // largest magnitude into [128, 256)
    const int e = am < 0x0080u ? 120 : max(-120, min(120, 7 + 127 - static_cast<int>(am >> 7)));
    const float f = scale < 0.f ? -exp2i(e) : exp2i(e);  // the scale's sign is in the digits
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = u4w(w[2 * i + (j >> 1)], 2 * (j & 1)), b = u4w(w[2 * i + (j >> 1)], 2 * (j & 1) + 1);
            digits4(bf16_lo(a) * f, bf16_hi(a) * f, bf16_lo(b) * f, bf16_hi(b) * f, hi[j], lo[j]);
        }
        uint8_t *o = dst + granule<D>(row, half * (D / 32) + i);
        *reinterpret_cast<uint4 *>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(o + kRows * D) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    // a NaN or an infinity in the row: NaN scores
    return am >= 0x7F80u ? __int_as_float(0x7FC00000) : exp2i(-e) * fabsf(scale);
}

// Two packed fp32 values.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) moe_kv_attend_tc_kernel(const __grid_constant__ AttendParams p)
{
    constexpr int TR = kRows;
    constexpr int kPageBytes = kPage * D;
    constexpr int kStep = 2 * kPageBytes;  // a step's codes of k, or of v
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *kbuf = smem, *vbuf = kbuf + kKStages * kStep, *fbuf = vbuf + kVStages * kStep, *qbuf = fbuf + kFStages * 2 * kStep;
    Control *ct = reinterpret_cast<Control *>(qbuf + 2 * kRows * D);
    Seqs &sq = *reinterpret_cast<Seqs *>(reinterpret_cast<uint8_t *>(ct) + sizeof(Control));
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const KvParams &c = p.c;
    const int G = c.q_heads / c.kv_heads;
    auto aborted = [&] { return *reinterpret_cast<volatile int *>(&ct->abort) != 0; };

    if (tid == 0) {
        ct->abort = 0;
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&ct->k_full[i], 1);
            mbar_init(&ct->k_empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&ct->v_full[i], 1);
            mbar_init(&ct->v_empty[i], 64);
        }
        for (int i = 0; i < kFStages; ++i) {
            mbar_init(&ct->f_full[i], 64);
            mbar_init(&ct->f_empty[i], 1);
        }
        for (int i = 0; i < kScales; ++i) mbar_init(&ct->sc_full[i], 1);
        mbar_init(&ct->q_ready, kConsumers);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ct->drained[b], 1);
            mbar_init(&ct->s_ready[b], 1);
            mbar_init(&ct->s_read[b], kRows);
            mbar_init(&ct->ref_ready[b], kRows);
            mbar_init(&ct->p_ready[b], kRows);
            mbar_init(&ct->o_ready[b], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // first warps of each kind (where several are ready the older issues, and
    // everything waits for the producer and the issuers)
    constexpr int kProducer = 0, kIssuer = 2, kConverter = 4, kSoftmax = 8;
    // tensor memory before the next kernel may start: its blocks can take theirs ahead of
    // their wait for this one, which must not have to wait for them in turn
    if (wid == kIssuer) tc_alloc(&ct->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct->tmem;
    grid_wait();
    grid_release();
    plan_units<kTileCost>(p, sq, G, TR);
    const long long U = sq.cum[c.B];
    const int blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), U));
    if (static_cast<int>(blockIdx.x) >= blocks) {
        if (wid == kIssuer) tc_dealloc(tmem, kTmemCols);
        return;
    }
    const long long u0 = block_start(U, blocks, blockIdx.x), u1 = block_start(U, blocks, blockIdx.x + 1);

    // No block ends with a copy into its shared memory or a product in flight: each was waited
    // for, unless the block gave up.  Whoever has some in flight asks where all warps have met:
    // nobody waits, and so gives up, any more.  (Each kind of warp comes here from its own end:
    // the same behind their common one slowed the loops, 451 against 437 us for a prefill chunk.)
    auto meet = [&] {
        __syncwarp();
        asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory");
        return aborted();
    };
    auto landed = [&](uint64_t *bar, uint32_t parity, uint64_t t0) {
        while (!mbar_test(bar, parity) && static_cast<long long>(gtimer() - t0) < p.timeout_ns) {
        }
    };

    if (wid < kSoftmax) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (wid >= kConverter) {
            // ---- v's codes to fp16: rows of a head dim, 64 tokens of a page (128 bytes).
            // Two warps a step, in turn (an even number of stages: each is always the same pair's).
            const int t = (tid - 32 * kConverter) & 63, half = (wid - kConverter) >> 1;
            int it = 0;
            for (long long u = u0; u < u1;) {
                const Segment s = locate<kTileCost>(sq, c.B, G, TR, u, u1);
                const int end = it + (s.pe - s.p0 + 1) / 2;
                for (it += (it & 1) ^ half; it < end; it += 2) {
                    const int vs = it % kVStages, f = it % kFStages;
                    wait_or_abort(&ct->v_full[vs], (it / kVStages) & 1, p, &ct->abort);
                    if (it >= kFStages) wait_or_abort(&ct->f_empty[f], (it / kFStages - 1) & 1, p, &ct->abort);
                    __syncwarp();
                    const uint8_t *src = vbuf + vs * kStep;
                    uint8_t *dst = fbuf + f * 2 * kStep;
#pragma unroll 4
                    for (int i = t; i < kStep / 16; i += 64) {  // 16 codes: granule i % 4 of row i / 4
                        const uint4 w = *reinterpret_cast<const uint4 *>(src + i * 16);
                        uint32_t h[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            h[2 * j] = e4m3x2_to_f16x2(static_cast<uint16_t>(u4w(w, j)));
                            h[2 * j + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(u4w(w, j) >> 16));
                        }
                        const int row = i >> 2, gr = 2 * (i & 3);
                        *reinterpret_cast<uint4 *>(dst + row * 128 + ((gr ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4 *>(dst + row * 128 + (((gr + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive(&ct->f_full[f]);
                    mbar_arrive(&ct->v_empty[vs]);
                }
                it = end;
                u += s.units;
            }
            meet();
        } else if (wid < kIssuer) {
            // ---- producers, one of k and one of v: two pages a step; an odd last page
            // comes twice (the second copy is behind every row's mask)
            const bool values = wid != kProducer;
            const int stages = values ? kVStages : kKStages;
            uint64_t *full = values ? ct->v_full : ct->k_full, *empty = values ? ct->v_empty : ct->k_empty;
            int it = 0, st = 0, issued = 0;
            uint32_t phase = 1;
            const uint64_t pol = policy_evict_last();  // other tiles read the page too
            for (long long u = u0; u < u1;) {
                const Segment s = locate<kTileCost>(sq, c.B, G, TR, u, u1);
                for (int pb = s.p0; pb < s.pe; pb += 32) {
                    const PageInfo pi = load_pages(c, s, pb);
                    const int m = min(32, s.pe - pb);
                    for (int i = 0; i < m; i += 2, ++it) {
                        int ph[2];
                        float pks[2], pvs[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int src = min(i + x, m - 1);
                            // a page out of range is masked; page 0 stands in for its codes
                            ph[x] = max(__shfl_sync(0xffffffffu, pi.id, src), 0) * c.kv_heads + s.h;
                            pks[x] = __shfl_sync(0xffffffffu, pi.ks, src);
                            pvs[x] = __shfl_sync(0xffffffffu, pi.vs, src);
                        }
                        if (lane == 0) {
                            if (it >= stages) wait_or_abort(&empty[st], phase, p, &ct->abort);
                            if (!aborted()) {
                                uint8_t *dst = (values ? vbuf : kbuf) + st * kStep;
                                mbar_expect_tx(&full[st], kStep);
                                if (values) {
#pragma unroll
                                    for (int x = 0; x < 2; ++x)
                                        bulk_g2s(dst + x * kPageBytes, c.v + static_cast<size_t>(ph[x]) * kPageBytes, kPageBytes,
                                                 &full[st], pol);
                                } else {
                                    const int sc = it % kScales;
#pragma unroll
                                    for (int x = 0; x < 2; ++x) {
                                        ct->ks[sc][x] = pks[x];
                                        ct->vs[sc][x] = pvs[x];
                                        tma2d(dst + x * kPageBytes, &c.tm_k, 0, ph[x] * kPage, &full[st], pol);
                                    }
                                    mbar_arrive(&ct->sc_full[sc]);
                                }
                                issued = it + 1;
                            }
                        }
                        if (++st == stages) st = 0, phase ^= 1;
                        __syncwarp();
                    }
                }
                u += s.units;
            }
            if (meet() && lane == 0) {
                const uint64_t t0 = gtimer();
                ring_drain(issued, stages, [&](int st, uint32_t parity) { landed(&full[st], parity, t0); });
            }
        } else if (wid == kIssuer || wid == kIssuer + 1) {
            // ---- MMA issue, a warp for S and one for O, an elected lane of each.  A
            // block that gave up goes on without waiting, on whatever is there.
            const bool scores = __shfl_sync(0xffffffffu, wid, 0) == kIssuer;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t qd = desc_lo(smem_u32(qbuf)), kd = desc_lo(smem_u32(kbuf)), fd = desc_lo(smem_u32(fbuf));
            int slot = 0, nseg = 0;      // buffer of the next step; segments so far
            uint32_t phase = 0, n = 0;   // of that buffer; steps so far
            for (long long u = u0; u < u1;) {
                const Segment s = locate<kTileCost>(sq, c.B, G, TR, u, u1);
                const int steps = (s.pe - s.p0 + 1) / 2;
                u += s.units;
                if (steps == 0) continue;  // (the softmax warps bring no queries then)
                if (scores) {
                    wait_or_abort(&ct->q_ready, nseg++ & 1, p, &ct->abort);
                    for (int i = 0; i < steps; ++i, ++n) {
                        const uint32_t b = n & 1, d = tm + 128 * b, k = kd + slot * (kStep / 16);
                        wait_or_abort(&ct->k_full[slot], phase, p, &ct->abort);
                        if (n >= 2) wait_or_abort(&ct->s_read[b], (n / 2 - 1) & 1, p, &ct->abort);
                        __syncwarp();
                        tc_fence_after();
                        if (elect_one()) {
                            mma_f8<false>(d, qd, k, desc_hi(D), mma_idesc(kKeys));
#pragma unroll
                            for (int j = 1; j < D / 32; ++j) mma_f8<true>(d, qd + 2 * j, k + 2 * j, desc_hi(D), mma_idesc(kKeys));
#pragma unroll
                            for (int j = 0; j < D / 32; ++j)
                                mma_f8<true>(d, qd + kRows * D / 16 + 2 * j, k + 2 * j, desc_hi(D), mma_idesc(kKeys));
                            tc_commit(&ct->s_ready[b]);
                            tc_commit(&ct->k_empty[slot]);
                        }
                        __syncwarp();
                        if (++slot == kKStages) slot = 0, phase ^= 1;
                    }
                } else {
                    for (int i = 0; i < steps; ++i, ++n) {
                        const uint32_t b = n & 1, a = tm + kTmemP + 64 * b, f = fd + slot * (2 * kStep / 16);
                        wait_or_abort(&ct->f_full[slot], phase, p, &ct->abort);
                        wait_or_abort(&ct->p_ready[b], (n / 2) & 1, p, &ct->abort);
                        __syncwarp();
                        tc_fence_after();
                        const uint32_t add = i % kRun != 0;
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)  // 16 tokens each: four of each page
                                mma_f16_ts(tm + kTmemO, a + 8 * j, f + (j >> 2) * (2 * kPageBytes / 16) + 2 * (j & 3),
                                           desc_hi(128), mma_idesc(D), j > 0 ? 1 : add);
                            tc_commit(&ct->o_ready[b]);
                            tc_commit(&ct->f_empty[slot]);
                        }
                        __syncwarp();
                        if (++slot == kFStages) slot = 0, phase ^= 1;
                    }
                }
                __syncwarp();
            }
            if (meet() && elect_one()) {  // (the lane that issued them)
                tc_commit(&ct->drained[scores]);
                landed(&ct->drained[scores], 0, gtimer());
            }
        }
    } else {
        // ---- softmax: warpgroup w takes the steps n with n % 2 = w, a thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
        const int ctid = tid - 32 * kSoftmax, row = ctid & (kRows - 1);
        const uint32_t w = ctid / kRows;
        const uint32_t lanes = static_cast<uint32_t>(wid & 3) << 21;  // this warp's tensor-memory lanes
        const uint32_t ts = tmem + lanes + 128 * w, tp = tmem + lanes + kTmemP + 64 * w, to = tmem + lanes + kTmemO;
        uint32_t n0 = 0;  // steps before the segment
        for (long long u = u0; u < u1;) {
            const Segment s = locate<kTileCost>(sq, c.B, G, TR, u, u1);
            u += s.units;
            if (s.p1 == 0) continue;
            const int n = sq.n[s.b], len = sq.len[s.b], rows = n * G, q0 = sq.q0[s.b], row0 = s.tile * TR;
            const int steps = (s.pe - s.p0 + 1) / 2;
            __syncwarp();
            asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");  // the last segment is over
            // Queries only where there are steps: the barrier's phase for them is then one that the
            // scores' issuer has passed before the segment ends.  A segment without
            // steps waits for nothing of the issuer's, so two of them in a row could
            // complete two phases between two of its polls, which a parity cannot tell from none.
            if (steps > 0) {
                const int qr = ctid >> 1, r = row0 + qr;
                const float f = put_query<D>(qbuf, qr, ctid & 1,
                                             p.q + static_cast<long long>(q0 + r / G) * p.q_stride + (s.h * G + r % G) * D,
                                             r < rows, p.scale_log2);
                if ((ctid & 1) == 0) ct->qs[qr] = f;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                mbar_arrive(&ct->q_ready);
                __syncwarp();
                asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
            }
            const int r = row0 + row;
            const int sees = r < rows ? row_sees(len, n, G, r) : 0;
            const float qs = steps > 0 && sees > 0 ? ct->qs[row] : 0.f;
            const int tile_sees = row_sees(len, n, G, row0);  // the least of the tile's rows

            float l = 0.f, lref = -INFINITY;  // this warpgroup's sum and what it refers to
            // (a run's end is a step of the segment's first warpgroup)
            if (w == (n0 & 1)) ct->kref[row] = -INFINITY;
            for (int i = (n0 & 1) == w ? 0 : 1; i < steps; i += 2) {
                const uint32_t k = n0 + i, ph = (k >> 1) & 1, sc = k % kScales;  // step, its barriers' phase
                wait_or_abort(&ct->sc_full[sc], (k / kScales) & 1, p, &ct->abort);
                wait_or_abort(&ct->s_ready[w], ph, p, &ct->abort);
                __syncwarp();
                tc_fence_after();
                float a[4][32];
#pragma unroll
                for (int h = 0; h < 4; ++h) tc_ld32(ts + 32 * h, a[h]);
                const float2 ks = *reinterpret_cast<const float2 *>(ct->ks[sc]), vs = *reinterpret_cast<const float2 *>(ct->vs[sc]);
                const int pg = s.p0 + 2 * i;
                const bool none0 = ks.x < 0.f, none1 = ks.y < 0.f || pg + 1 >= s.pe;  // no such page
                tc_wait_ld();
                tc_fence_before();
                mbar_arrive(&ct->s_read[w]);
                if (none0 || none1 || (pg + 2) * kPage > tile_sees) {
                    const int lim0 = none0 ? 0 : sees - pg * kPage, lim1 = none1 ? 0 : sees - (pg + 1) * kPage;
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * (h & 1) + j >= (h < 2 ? lim0 : lim1)) a[h][j] = -INFINITY;
                }
                // the largest, in log2 units (a row's factor is not negative)
                float fs[2] = {qs * fmaxf(ks.x, 0.f), qs * fmaxf(ks.y, 0.f)};  // (no such page: 0)
                float mx = -INFINITY;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    if (fs[y] == 0.f) fs[y] = 1.17549435e-38f;  // masked scores (-inf) stay what they are
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < 64; j += 8)
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float *v = &a[2 * y + (j >> 5)][j & 31];
                            m4[z] = max3(m4[z], v[z], v[z + 4]);
                        }
                    const float m = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
                    if (m > -INFINITY) mx = fmaxf(mx, fmaf(m, fs[y], scale_log2(y ? vs.y : vs.x)));
                }
                // the reference after the step before, from the other warpgroup
                float ref = -INFINITY;
                if (i > 0) {
                    wait_or_abort(&ct->ref_ready[w ^ 1], ((k - 1) >> 1) & 1, p, &ct->abort);
                    ref = ct->ref[w ^ 1][row];
                }
                const bool move = mx > ref + kSlack;  // (ref = -inf: as soon as anything is seen)
                const float old = ref;
                if (move) ref = mx;
                ct->ref[w][row] = ref;
                mbar_arrive(&ct->ref_ready[w]);
                if (i > 1) {
                    // the last weights in this warpgroup's place have been used.  (Before the
                    // rescaling too: the other warpgroup's barrier is then at most one
                    // phase behind the one waited for there, which is all a parity can tell.)
                    wait_or_abort(&ct->o_ready[w], ph ^ 1, p, &ct->abort);
                    __syncwarp();
                    tc_fence_after();
                }
                const bool ends = i > 0 && i % kRun == 0;  // the run before this step
                const bool moves = i > 0 && __any_sync(0xffffffffu, move);
                if (ends || moves) {
                    // the accumulators follow, between the last step's product and this one's:
                    // they go on under the new reference, or where the ended runs' sums are
                    wait_or_abort(&ct->o_ready[w ^ 1], ((k - 1) >> 1) & 1, p, &ct->abort);
                    __syncwarp();
                    tc_fence_after();
                    const float kref = ct->kref[row];
                    const float f = ends ? (kref == -INFINITY ? 0.f : ex2(kref - old)) : (move ? ex2(old - ref) : 1.f);
#pragma unroll 1
                    for (int h = 0; h < D / 16; ++h) {
                        float v[16];
                        tc_ld16(to + 16 * h, v);
                        tc_wait_ld();
                        if (ends) {
                            float *part = part_slot(p, blockIdx.x, s.p0 == 0);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float4 *at = reinterpret_cast<float4 *>(part_at(part, TR, row, 16 * h + 4 * j));
                                const float4 was = i > kRun ? __ldcg(at) : make_float4(0.f, 0.f, 0.f, 0.f);
                                __stcg(at, make_float4(fmaf(was.x, f, v[4 * j]), fmaf(was.y, f, v[4 * j + 1]),
                                                       fmaf(was.z, f, v[4 * j + 2]), fmaf(was.w, f, v[4 * j + 3])));
                            }
                        } else {
                            uint32_t x[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(v[j] * f);
                            tc_st16(to + 16 * h, x);
                        }
                    }
                    if (ends) ct->kref[row] = old;
                }
                const float base = ref == -INFINITY ? 0.f : ref;
                if (lref != ref) l *= ex2(lref - base);  // (lref = -inf: 0, as l is)
                lref = ref;
                // 64 w vs in fp16; w's sum from the unrounded values
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float pv = fmaxf(y ? vs.y : vs.x, 0x1p-64f) * kGain, add = __log2f(pv) - base;
                    const uint64_t f2 = pack2(fs[y], fs[y]), a2 = pack2(add, add);
                    uint64_t l2[2] = {0, 0};
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int h = 2 * y + hh;
                        uint32_t x[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float e0, e1;
                            unpack2(fma2(pack2(a[h][2 * j], a[h][2 * j + 1]), f2, a2), e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            l2[j & 1] = add2(l2[j & 1], pack2(e0, e1));
                            x[j] = cvt_f16x2(e0, e1);
                        }
                        tc_st16(tp + 16 * h, x);
                    }
                    float e0, e1;
                    unpack2(add2(l2[0], l2[1]), e0, e1);
                    l += (e0 + e1) * (1.f / pv);
                }
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&ct->p_ready[w]);
            }

            // ---- the result: o / 64 in tensor memory, the last reference, the sums
            ct->l[w][row] = l;
            ct->lref[w][row] = lref;
            __syncwarp();
            asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
            n0 += steps;
            float ref = -INFINITY, lsum = 0.f, kf = 0.f;
            if (steps > 0) {
                const uint32_t last = n0 - 1;
                ref = ct->ref[last & 1][row];
                const float base = ref == -INFINITY ? 0.f : ref;
                lsum = ct->l[0][row] * ex2(ct->lref[0][row] - base) + ct->l[1][row] * ex2(ct->lref[1][row] - base);
                if (ct->kref[row] != -INFINITY) kf = ex2(ct->kref[row] - base);
                wait_or_abort(&ct->o_ready[last & 1], (last >> 1) & 1, p, &ct->abort);  // (products end in order)
                __syncwarp();
                tc_fence_after();
            }
            float *part = part_slot(p, blockIdx.x, s.p0 == 0);
            if (!s.whole() && w == 0) {
                part[row] = ref;
                part[TR + row] = lsum;
            }
            const float inv = inv_sum(kGain, lsum);
            uint16_t *orow = out_row(p, q0, s.h, G, min(r, rows - 1));
            // each warpgroup has half the head dims
#pragma unroll 2
            for (int col = D / 2 * w; col < D / 2 * (w + 1); col += 16) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = 0.f;
                if (steps > 0) tc_ld16(to + col, v);
                tc_wait_ld();
                if (steps > kRun) {  // the ended runs
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 was = __ldcg(reinterpret_cast<const float4 *>(part_at(part, TR, row, col + 4 * j)));
                        v[4 * j] = fmaf(was.x, kf, v[4 * j]);
                        v[4 * j + 1] = fmaf(was.y, kf, v[4 * j + 1]);
                        v[4 * j + 2] = fmaf(was.z, kf, v[4 * j + 2]);
                        v[4 * j + 3] = fmaf(was.w, kf, v[4 * j + 3]);
                    }
                }
                if (!s.whole()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float4 *>(part_at(part, TR, row, col + 4 * j)) =
                            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                } else if (r < rows) {
                    uint4 *o = reinterpret_cast<uint4 *>(orow + col);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        o[j] = make_uint4(pack_bf16(v[8 * j] * inv, v[8 * j + 1] * inv),
                                          pack_bf16(v[8 * j + 2] * inv, v[8 * j + 3] * inv),
                                          pack_bf16(v[8 * j + 4] * inv, v[8 * j + 5] * inv),
                                          pack_bf16(v[8 * j + 6] * inv, v[8 * j + 7] * inv));
                }
            }
            tc_fence_before();
            if (!s.whole()) join_tile<D, kConsumers, TR>(p, s, U, blocks, rows, q0, G, kGain, &ct->last, ctid);
        }
        tc_fence_before();
        meet();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (wid == kIssuer) tc_dealloc(tmem, kTmemCols);
}

template <int D>
cudaError_t launch_d(const AttendParams &p, int grid, cudaStream_t st)
{
    // steps of k, of v, of v in fp16 (twice as many bytes), query digits
    constexpr int smem = 1024 + 2 * kPage * D * (kKStages + kVStages + 2 * kFStages) + 2 * kRows * D +
                         static_cast<int>(sizeof(Control) + sizeof(Seqs));
    static_assert(smem <= 227 * 1024, "shared memory of a block");
    auto *fn = moe_kv_attend_tc_kernel<D>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchCfg l(dim3(grid), dim3(kThreads), smem, st);
    return cudaLaunchKernelEx(&l.cfg, fn, p);
}

}  // namespace

cudaError_t launch_kv_attend_tc(const AttendParams &p, int num_sms, cudaStream_t st)
{
    return p.c.D == 128 ? launch_d<128>(p, num_sms, st) : launch_d<64>(p, num_sms, st);
}

}  // namespace moe
