// moe_kv_attend_tc.cu -- causal attention over the paged 8-bit cache
// (moe_kv_attend) for many query rows: prefill chunks, verification runs.
//
//   o[i, h] = sum_t w_t v[t] / sum_t w_t,   w_t = 2^(s_t - ref),
//   s_t = log2(e) scale q.k_t
//
// Both products run on the tensor cores (tcgen05.mma kind::f8f6f4, accumulators
// in tensor memory) straight on the cache's E4M3 codes, which TMA brings into
// shared memory and nothing else touches:
//
//  * S[128 rows x 128 tokens] = Q K^T: q enters as two E4M3 digits, hi + lo,
//    after a power-of-two prescale of the row (largest magnitude into [128,
//    256)): 8 significant bits are two digits of 4, so the sum is exact down
//    to 2^-10 of the row's largest.
//  * O[128 rows x head dim] += P V: the weights 64 w vs (vs: the page's v scale
//    over the largest that the reference allows for) enter as two digits, relative
//    error 2^-9, written to tensor memory over the scores they come from.
//
// Two digits at twice the 16-bit rate cost what 16-bit operands would, without
// converting the cache.  The reference is the running maximum of s + ceil(
// log2(vs)), moved only when a tile exceeds it by more than 2 (the digits hold
// four times the usual largest), so the accumulators in tensor memory are rescaled rarely.
//
// A block runs two streams, each with a warpgroup for the softmax (a thread a
// row) and its own S / P and O in tensor memory, so that one stream's softmax
// and the other's products overlap.  With TWO, the streams are two row tiles
// that share the pages; otherwise they are the even and the odd page pairs of
// one row tile, joined at the end.  One warp brings pages (two a stage), one thread
// issues the MMAs.
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
#include "moe_tcgen05.cuh"

#include "moe_attend.cuh"

constexpr int kRows = 128;       // rows of a stream: tensor-memory lanes
constexpr int kKeys = 2 * kPage; // tokens of a stage
constexpr float kGain = 64.f;    // of the weights' digits
constexpr float kSlack = 2.f;    // how far a tile may exceed the reference (64 * 2^2 = 256 <= 448)
constexpr int kTmemCols = 512;   // stream s: S / P at 256 s, O at 256 s + 128

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_ready, s_ready[2], p_ready[2], o_ready[2], drained;
    float ks[kMaxStages][2], vs[kMaxStages][2];  // scales of the stage's pages; ks < 0: no such page
    float qs[2][kRows];                          // each row's factor from digits to scores (log2 units)
    float m[2][kRows], l[2][kRows];              // the streams' references and sums, for joining them
    uint32_t tmem;
    int abort, last;
};

// D[128 x N] (+)= A B^T with E4M3 operands: A from shared or tensor memory
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Instruction descriptor, kind::f8f6f4: fp32 accumulator, E4M3 A and B, K-major
// both, M = 128, N = n.
__device__ __forceinline__ uint32_t f8_idesc(int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// Matrix descriptor: K-major rows of 64 bytes, 64-byte swizzle, 8-row groups
// 512 bytes apart.
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(4) << 61);
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
// the nearest to the rest.
__device__ __forceinline__ void digits4(float a, float b, float c, float d, uint32_t &hi, uint32_t &lo)
{
    const uint32_t x = cvt_f16x2(a, b), y = cvt_f16x2(c, d);
    const uint32_t hx = cvt_e4m3x2(x), hy = cvt_e4m3x2(y);
    const uint32_t rx = hsub2(x, e4m3x2_to_f16x2(static_cast<uint16_t>(hx)));
    const uint32_t ry = hsub2(y, e4m3x2_to_f16x2(static_cast<uint16_t>(hy)));
    hi = hx | (hy << 16);
    lo = cvt_e4m3x2(rx) | (cvt_e4m3x2(ry) << 16);
}

// 16-byte granule gr of row `row` in a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ int granule(int row, int gr)
{
    return row * D + ((D == 128 ? gr ^ (row & 7) : gr ^ ((row >> 1) & 3)) << 4);
}

// Half a query row (thread pairs share a row) as two digits into the tile at dst
// (hi; lo follows kRows * D bytes on); returns the row's factor.
template <int D>
__device__ __forceinline__ float put_query(uint8_t *dst, int row, int half, const uint16_t *src, bool in, float scale_log2)
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
    const float f = exp2i(e);
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
    return am >= 0x7F80u ? __int_as_float(0x7FC00000) : exp2i(-e) * scale_log2;
}

template <int D, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) moe_kv_attend_tc_kernel(const __grid_constant__ AttendParams p, int NS)
{
    constexpr int TR = TWO ? 2 * kRows : kRows;   // query rows of a tile
    constexpr int kPageBytes = kPage * D;
    constexpr int kStage = 4 * kPageBytes;        // two pages of k, two of v
    constexpr int kQ = 2 * kRows * D;             // a stream's query digits
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = smem + NS * kStage;
    Control *ct = reinterpret_cast<Control *>(qbuf + (TWO ? 2 : 1) * kQ);
    Seqs &sq = *reinterpret_cast<Seqs *>(reinterpret_cast<uint8_t *>(ct) + sizeof(Control));
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const KvParams &c = p.c;
    const int G = c.q_heads / c.kv_heads;

    if (tid == 0) {
        ct->abort = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(&ct->full[i], 1);
            mbar_init(&ct->empty[i], TWO ? 2 : 1);
        }
        mbar_init(&ct->q_ready, kConsumers);
        mbar_init(&ct->drained, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ct->s_ready[s], 1);
            mbar_init(&ct->p_ready[s], kRows);
            mbar_init(&ct->o_ready[s], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_wait();
    grid_release();
    plan_units(p, sq, G, TR);
    const long long U = sq.cum[c.B];
    const int blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), U));
    if (static_cast<int>(blockIdx.x) >= blocks) return;
    const long long u0 = block_start(U, blocks, blockIdx.x), u1 = block_start(U, blocks, blockIdx.x + 1);
    if (wid == 9) tc_alloc(&ct->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct->tmem;

    if (wid >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        if (wid == 8) {
            // ---- producer: two pages a stage; an odd last page comes twice (the
            // second copy is behind every row's mask)
            int it = 0;
            const uint64_t pol = TWO ? policy_evict_last() : policy_evict_first();  // other tiles read the page too
            for (long long u = u0; u < u1;) {
                const Segment s = locate(sq, c.B, G, TR, u, u1);
                for (int pb = s.p0; pb < s.pe; pb += 32) {
                    const PageInfo pi = load_pages(c, s, pb);
                    const int m = min(32, s.pe - pb);
                    for (int i = 0; i < m; i += 2, ++it) {
                        const int st = it % NS;
                        int pid[2];
                        float ks[2], vs[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int src = min(i + x, m - 1);
                            pid[x] = __shfl_sync(0xffffffffu, pi.id, src);
                            ks[x] = __shfl_sync(0xffffffffu, pi.ks, src);
                            vs[x] = __shfl_sync(0xffffffffu, pi.vs, src);
                        }
                        if (lane == 0) {
                            if (it >= NS) wait_or_abort(&ct->empty[st], (it / NS - 1) & 1, p, &ct->abort);
                            if (*reinterpret_cast<volatile int *>(&ct->abort) == 0) {
                                mbar_expect_tx(&ct->full[st], kStage);
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    ct->ks[st][x] = ks[x];
                                    ct->vs[st][x] = vs[x];
                                    // a page out of range is masked; page 0 stands in for its codes
                                    const int ph = max(pid[x], 0) * c.kv_heads + s.h;
                                    uint8_t *dst = smem + st * kStage + x * kPageBytes;
                                    tma2d(dst, &c.tm_k, 0, ph * kPage, &ct->full[st], pol);
                                    tma2d(dst + 2 * kPageBytes, &c.tm_v, 0, ph * D, &ct->full[st], pol);
                                }
                            }
                        }
                        __syncwarp();
                    }
                }
                u += s.p1 - s.p0;
            }
            if (lane == 0 && *reinterpret_cast<volatile int *>(&ct->abort)) {
                // no block ends with a copy into its shared memory in flight
                const uint64_t t0 = gtimer();
                for (int j = max(it - NS, 0); j < it; ++j)
                    while (!mbar_test(&ct->full[j % NS], (j / NS) & 1) &&
                           static_cast<long long>(gtimer() - t0) < p.timeout_ns) {
                    }
            }
        } else if (wid == 9) {
            // ---- MMA issue: one thread (the whole warp finds the segments)
            const uint32_t idesc_s = f8_idesc(kKeys), idesc_o = f8_idesc(D);
            int base = 0, nseg = 0;  // stages before the segment; segments so far
            uint32_t sn[2] = {0, 0};  // steps of each stream so far
            for (long long u = u0; u < u1; ++nseg) {
                const Segment s = locate(sq, c.B, G, TR, u, u1);
                const int stages = (s.pe - s.p0 + 1) / 2;
                const int steps[2] = {TWO ? stages : (stages + 1) / 2, TWO ? stages : stages / 2};
                u += s.p1 - s.p0;
                __syncwarp();
                if (lane != 0) continue;
                wait_or_abort(&ct->q_ready, nseg & 1, p, &ct->abort);
                tc_fence_after();
                auto stage_of = [&](int x, int i) { return base + (TWO ? i : 2 * i + x); };
                auto issue_s = [&](int x, int i) {
                    const int it = stage_of(x, i), st = it % NS;
                    wait_or_abort(&ct->full[st], (it / NS) & 1, p, &ct->abort);
                    if (*reinterpret_cast<volatile int *>(&ct->abort)) return;
                    const uint32_t qa = smem_u32(qbuf) + (TWO ? x * kQ : 0), ka = smem_u32(smem + st * kStage);
#pragma unroll
                    for (int dg = 0; dg < 2; ++dg)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            const uint32_t a = qa + dg * (kRows * D) + 32 * k, b = ka + 32 * k;
                            mma_f8(tmem + 256 * x, D == 128 ? sw128_desc(a) : sw64_desc(a),
                                   D == 128 ? sw128_desc(b) : sw64_desc(b), idesc_s, dg + k > 0);
                        }
                    tc_commit(&ct->s_ready[x]);
                };
                auto issue_o = [&](int x, int i) {
                    const int it = stage_of(x, i), st = it % NS;
                    wait_or_abort(&ct->p_ready[x], (sn[x] + i) & 1, p, &ct->abort);
                    if (*reinterpret_cast<volatile int *>(&ct->abort)) return;
                    tc_fence_after();
                    const uint32_t va = smem_u32(smem + st * kStage) + 2 * kPageBytes;
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 32 tokens each: two of each page
#pragma unroll
                        for (int dg = 0; dg < 2; ++dg)
                            mma_f8_ts(tmem + 256 * x + 128, tmem + 256 * x + 16 * k + 8 * dg,
                                      sw64_desc(va + (k >> 1) * kPageBytes + 32 * (k & 1)), idesc_o, i + k + dg > 0);
                    tc_commit(&ct->o_ready[x]);
                    tc_commit(&ct->empty[st]);
                };
                for (int x = 0; x < 2; ++x)
                    if (steps[x] > 0) issue_s(x, 0);
                for (int i = 0; i < steps[0]; ++i)
                    for (int x = 0; x < 2; ++x)
                        if (i < steps[x]) {
                            issue_o(x, i);
                            if (i + 1 < steps[x]) {
                                // the next scores take the place of these weights
                                wait_or_abort(&ct->o_ready[x], (sn[x] + i) & 1, p, &ct->abort);
                                issue_s(x, i + 1);
                            }
                        }
                for (int x = 0; x < 2; ++x) sn[x] += steps[x];
                base += stages;
            }
            if (lane == 0 && *reinterpret_cast<volatile int *>(&ct->abort)) {
                // no block ends with products in flight
                tc_commit(&ct->drained);
                const uint64_t t0 = gtimer();
                while (!mbar_test(&ct->drained, 0) && static_cast<long long>(gtimer() - t0) < p.timeout_ns) {
                }
            }
        }
    } else {
        // ---- softmax: stream x, a thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
        const int x = wid >> 2, row = tid & (kRows - 1);
        const uint32_t lanes = static_cast<uint32_t>(wid & 3) << 21;  // this warp's tensor-memory lanes
        const uint32_t ts = tmem + 256 * x + lanes, to = ts + 128;
        int base = 0;
        uint32_t sn = 0, on[2] = {0, 0};  // this stream's steps so far; both streams'
        for (long long u = u0; u < u1;) {
            const Segment s = locate(sq, c.B, G, TR, u, u1);
            const int n = sq.n[s.b], len = sq.len[s.b], rows = n * G, q0 = sq.q0[s.b];
            const int stages = (s.pe - s.p0 + 1) / 2;
            const int steps = TWO ? stages : (stages + 1 - x) / 2;
            // queries: 64 rows at a time, two threads a row
            asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");  // both streams are done with the last
            for (int part = 0; part < (TWO ? 2 : 1); ++part) {
                const int qr = 64 * (TWO ? part : x) + (row >> 1);  // row of the 128-row tile
                const int r = s.tile * TR + (TWO ? kRows * x : 0) + qr;
                const float f = put_query<D>(qbuf + (TWO ? x * kQ : 0), qr, row & 1,
                                             p.q + static_cast<long long>(q0 + r / G) * p.q_stride + (s.h * G + r % G) * D,
                                             r < rows, p.scale_log2);
                if ((row & 1) == 0) ct->qs[TWO ? x : 0][qr] = f;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            mbar_arrive(&ct->q_ready);
            asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
            const int r = s.tile * TR + (TWO ? kRows * x : 0) + row;
            const float qs = ct->qs[TWO ? x : 0][row];
            const int sees = r < rows ? row_sees(len, n, G, r) : 0;
            const int tile_sees = row_sees(len, n, G, s.tile * TR + (TWO ? kRows * x : 0));  // the least of the stream's rows

            float ref = -INFINITY, l = 0.f;
            for (int i = 0; i < steps; ++i) {
                const int it = base + (TWO ? i : 2 * i + x), st = it % NS;
                wait_or_abort(&ct->full[st], (it / NS) & 1, p, &ct->abort);  // the pages' scales
                wait_or_abort(&ct->s_ready[x], (sn + i) & 1, p, &ct->abort);
                __syncwarp();
                tc_fence_after();
                const float ks[2] = {ct->ks[st][0], ct->ks[st][1]}, vs[2] = {ct->vs[st][0], ct->vs[st][1]};
                const int tok0 = (s.p0 + 2 * (it - base)) * kPage;
                const bool edge = tok0 + kKeys > tile_sees || tok0 + kKeys > s.pe * kPage || ks[0] < 0.f || ks[1] < 0.f;
                // the last token of each page that this row sees, from the page's first
                int lim[2];
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    lim[y] = ks[y] < 0.f || tok0 + y * kPage >= s.pe * kPage ? 0 : sees - (tok0 + y * kPage);
                // largest of the row
                float mx = -INFINITY;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float a[32];
                    tc_ld32(ts + 32 * h, a);
                    tc_wait_ld();
                    const float fs = qs * ks[h >> 1];
                    float mh = -INFINITY;
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * (h & 1) + j < lim[h >> 1]) mh = fmaxf(mh, a[j] * fs);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) mh = fmaxf(mh, a[j] * fs);
                    }
                    mx = fmaxf(mx, mh + scale_log2(vs[h >> 1]));
                }
                const bool move = mx > ref + kSlack;  // (ref = -inf: as soon as anything is seen)
                if (__any_sync(0xffffffffu, move)) {
                    const float nref = move ? mx : ref;
                    const float f = move ? ex2(ref - nref) : 1.f;
                    l *= f;
                    ref = nref;
                    if (i > 0) {
                        wait_or_abort(&ct->o_ready[x], (sn + i - 1) & 1, p, &ct->abort);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int h = 0; h < D / 32; ++h) {
                            float a[32];
                            tc_ld32(to + 32 * h, a);
                            tc_wait_ld();
                            uint32_t b[2][16];
#pragma unroll
                            for (int j = 0; j < 32; ++j) b[j >> 4][j & 15] = __float_as_uint(a[j] * f);
                            tc_st16(to + 32 * h, b[0]);
                            tc_st16(to + 32 * h + 16, b[1]);
                        }
                        tc_wait_st();
                    }
                }
                const float base_ref = ref == -INFINITY ? 0.f : ref;
                // weights and their digits, 32 tokens at a time, over the scores read
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float a[32];
                    tc_ld32(ts + 32 * h, a);
                    tc_wait_ld();
                    const float fs = qs * ks[h >> 1], pv = vs[h >> 1] * kGain;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float w = ex2(fmaf(a[j], fs, -base_ref));
                        if (edge && 32 * (h & 1) + j >= lim[h >> 1]) w = 0.f;
                        l += w;
                        a[j] = w * pv;
                    }
                    uint32_t dg[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) digits4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3], dg[j], dg[8 + j]);
                    tc_st16(ts + 16 * h, dg);
                }
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&ct->p_ready[x]);
            }
            sn += steps;
            on[0] += TWO ? stages : (stages + 1) / 2;
            on[1] += TWO ? stages : stages / 2;

            // ---- the result: o / 64 in tensor memory, the reference and the sum
            float *part = part_slot(p, blockIdx.x, s.p0 == 0);
            const int rr = TWO ? kRows * x + row : row;
            uint16_t *orow = out_row(p, q0, s.h, G, min(r, rows - 1));
            float f0 = 1.f, f1 = 0.f, lsum = l, msum = ref;
            if (!TWO) {  // both streams' sums
                ct->m[x][row] = ref;
                ct->l[x][row] = l;
                asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
                const float m0 = ct->m[0][row], m1 = ct->m[1][row], mm = fmaxf(m0, m1);
                const float mref = mm == -INFINITY ? 0.f : mm;
                f0 = ex2(m0 - mref);
                f1 = ex2(m1 - mref);
                lsum = ct->l[0][row] * f0 + ct->l[1][row] * f1;
                msum = mm;
            }
            const bool have0 = TWO ? steps > 0 : stages > 0, have1 = !TWO && stages > 1;
            const int x0 = TWO ? x : 0;
            if (have0) wait_or_abort(&ct->o_ready[x0], (on[x0] - 1) & 1, p, &ct->abort);
            if (have1) wait_or_abort(&ct->o_ready[1], (on[1] - 1) & 1, p, &ct->abort);
            __syncwarp();
            tc_fence_after();
            const float inv = inv_sum(kGain, lsum);
            if (!s.whole() && (TWO || x == 0)) {
                part[rr] = msum;
                part[TR + rr] = lsum;
            }
            constexpr int NH = TWO ? D / 32 : D / 64;  // 32-column pieces of this thread: all, or the stream's half
#pragma unroll 1
            for (int h = 0; h < NH; ++h) {
                const int col = 32 * (TWO ? h : NH * x + h);
                float a[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) a[j] = 0.f;
                if (have0) {
                    tc_ld32(tmem + lanes + 256 * x0 + 128 + col, a);
                    tc_wait_ld();
                }
                if (!TWO) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) a[j] *= f0;
                    if (have1) {
                        float b[32];
                        tc_ld32(tmem + lanes + 256 + 128 + col, b);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[j] += b[j] * f1;
                    }
                }
                if (!s.whole()) {
                    float4 *o = reinterpret_cast<float4 *>(part + 2 * TR + rr * D + col);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = make_float4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]);
                } else if (r < rows) {
                    uint4 *o = reinterpret_cast<uint4 *>(orow + col);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[j] = make_uint4(pack_bf16(a[8 * j] * inv, a[8 * j + 1] * inv),
                                          pack_bf16(a[8 * j + 2] * inv, a[8 * j + 3] * inv),
                                          pack_bf16(a[8 * j + 4] * inv, a[8 * j + 5] * inv),
                                          pack_bf16(a[8 * j + 6] * inv, a[8 * j + 7] * inv));
                }
            }
            tc_fence_before();
            if (!s.whole()) join_tile<D>(p, s, U, blocks, TR, rows, q0, G, kGain, &ct->last);
            base += stages;
            u += s.p1 - s.p0;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (wid == 9) tc_dealloc(tmem, kTmemCols);
}

template <int D, bool TWO>
cudaError_t launch_one(const AttendParams &p, int grid, int smem_optin, cudaStream_t st)
{
    constexpr int kStage = 4 * kPage * D;
    const int fixed = 1024 + static_cast<int>(sizeof(Control) + sizeof(Seqs)) + (TWO ? 2 : 1) * 2 * kRows * D;
    const int ns = std::min(kMaxStages, (smem_optin - fixed) / kStage);
    const int smem = fixed + ns * kStage;
    auto *fn = moe_kv_attend_tc_kernel<D, TWO>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchCfg l(dim3(grid), dim3(kThreads), smem, st);
    return cudaLaunchKernelEx(&l.cfg, fn, p, ns);
}

}  // namespace

cudaError_t launch_kv_attend_tc(const AttendParams &p, int tile_rows, int num_sms, int smem_optin, cudaStream_t st)
{
    if (p.c.D == 128)
        return tile_rows == 256 ? launch_one<128, true>(p, num_sms, smem_optin, st)
                                : launch_one<128, false>(p, num_sms, smem_optin, st);
    return tile_rows == 256 ? launch_one<64, true>(p, num_sms, smem_optin, st)
                            : launch_one<64, false>(p, num_sms, smem_optin, st);
}

}  // namespace moe
