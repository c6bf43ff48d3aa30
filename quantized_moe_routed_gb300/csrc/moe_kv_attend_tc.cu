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
// A block runs two streams, each with two warpgroups for the softmax (two
// threads a row, each a page of the stage) and its own S / P and O in tensor memory, so that
// one stream's softmax and the other's products overlap.  With TWO, the streams are two row tiles
// that share the pages; otherwise they are the even and the odd page pairs of
// one row tile, joined at the end.  One warp brings pages (two a stage), one thread a
// stream issues the MMAs.
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

constexpr int kStream = 256;     // softmax threads of a stream
constexpr int kConsumers = 2 * kStream;
constexpr int kThreads = kConsumers + 128;  // and a warpgroup with the producer and the MMA issuers
// Registers a thread of the two kinds keeps: 512 * 104 + 128 * 48 = 59392, within
// what the block is launched with (640 threads of 96).
constexpr int kConsumerRegs = 104, kProducerRegs = 48;
constexpr int kRows = 128;       // rows of a stream: tensor-memory lanes
constexpr int kKeys = 2 * kPage; // tokens of a stage
constexpr float kGain = 64.f;    // of the weights' digits
constexpr float kSlack = 2.f;    // how far a tile may exceed the reference (64 * 2^2 = 256 <= 448)
constexpr int kTmemCols = 512;   // stream s: S / P at 256 s, O at 256 s + 128

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_ready, s_ready[2], p_ready[2], o_ready[2], drained[2];
    float ks[kMaxStages][2], vs[kMaxStages][2];  // scales of the stage's pages; ks < 0: no such page
    float qs[2][kRows];                          // each row's factor from digits to scores (log2 units)
    float mx[2][2][kRows];                       // [stream][page]: largest of a row in a stage's page
    float m[2][kRows], l[2][2][kRows];           // references, and sums of the two pages, at a tile's end
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

// Half a query row (thread pairs share a row) as two digits into the tile at dst
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
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ct->s_ready[s], 1);
            mbar_init(&ct->p_ready[s], kStream);
            mbar_init(&ct->o_ready[s], 1);
            mbar_init(&ct->drained[s], 1);
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
    constexpr int kProducer = kConsumers / 32, kIssuer = kProducer + 1;  // warps
    if (wid == kIssuer) tc_alloc(&ct->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct->tmem;

    if (wid >= kProducer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        if (wid == kProducer) {
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
        } else if (wid == kIssuer || wid == kIssuer + 1) {
            // ---- MMA issue: a thread for each stream (its warp finds the segments), so
            // that a stream waits only for its own
            const int x = wid - kIssuer;
            const uint32_t idesc_s = f8_idesc(kKeys), idesc_o = f8_idesc(D);
            const uint32_t sd = tmem + 256 * x, od = sd + 128;
            int base = 0, nseg = 0;  // stages before the segment; segments so far
            uint32_t sn = 0;         // steps so far
            for (long long u = u0; u < u1; ++nseg) {
                const Segment s = locate(sq, c.B, G, TR, u, u1);
                const int stages = (s.pe - s.p0 + 1) / 2, steps = TWO ? stages : (stages + 1 - x) / 2;
                u += s.p1 - s.p0;
                __syncwarp();
                if (lane != 0) continue;
                wait_or_abort(&ct->q_ready, nseg & 1, p, &ct->abort);
                tc_fence_after();
                const uint32_t qa = smem_u32(qbuf) + (TWO ? x * kQ : 0);
                for (int i = 0; i < steps; ++i, ++sn) {
                    const int it = base + (TWO ? i : 2 * i + x), st = it % NS;
                    const uint32_t ka = smem_u32(smem + st * kStage), va = ka + 2 * kPageBytes;
                    wait_or_abort(&ct->full[st], (it / NS) & 1, p, &ct->abort);
                    // the scores take the place of the last step's weights
                    if (i > 0) wait_or_abort(&ct->o_ready[x], (sn - 1) & 1, p, &ct->abort);
                    if (*reinterpret_cast<volatile int *>(&ct->abort)) continue;
                    tc_fence_after();
#pragma unroll
                    for (int dg = 0; dg < 2; ++dg)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            const uint32_t a = qa + dg * (kRows * D) + 32 * k, b = ka + 32 * k;
                            mma_f8(sd, D == 128 ? sw128_desc(a) : sw64_desc(a), D == 128 ? sw128_desc(b) : sw64_desc(b),
                                   idesc_s, dg + k > 0);
                        }
                    tc_commit(&ct->s_ready[x]);
                    wait_or_abort(&ct->p_ready[x], sn & 1, p, &ct->abort);
                    if (*reinterpret_cast<volatile int *>(&ct->abort)) continue;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 32 tokens each: two of each page
#pragma unroll
                        for (int dg = 0; dg < 2; ++dg)
                            mma_f8_ts(od, sd + 16 * k + 8 * dg, sw64_desc(va + (k >> 1) * kPageBytes + 32 * (k & 1)), idesc_o,
                                      i + k + dg > 0);
                    tc_commit(&ct->o_ready[x]);
                    tc_commit(&ct->empty[st]);
                }
                base += stages;
            }
            if (lane == 0 && *reinterpret_cast<volatile int *>(&ct->abort)) {
                // no block ends with products in flight
                tc_commit(&ct->drained[x]);
                const uint64_t t0 = gtimer();
                while (!mbar_test(&ct->drained[x], 0) && static_cast<long long>(gtimer() - t0) < p.timeout_ns) {
                }
            }
        }
    } else {
        // ---- softmax: stream x, thread pairs (in two warpgroups) share a row; page y
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
        const int x = wid >> 3, y = (wid >> 2) & 1, row = tid & (kRows - 1);
        const uint32_t lanes = static_cast<uint32_t>(wid & 3) << 21;  // this warp's tensor-memory lanes
        const uint32_t ts = tmem + 256 * x + lanes, to = ts + 128;
        auto stream_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(2 + x), "n"(kStream) : "memory"); };
        int base = 0;
        uint32_t sn = 0, on[2] = {0, 0};  // this stream's steps so far; both streams'
        for (long long u = u0; u < u1;) {
            const Segment s = locate(sq, c.B, G, TR, u, u1);
            const int n = sq.n[s.b], len = sq.len[s.b], rows = n * G, q0 = sq.q0[s.b];
            const int stages = (s.pe - s.p0 + 1) / 2;
            const int steps = TWO ? stages : (stages + 1 - x) / 2;
            const int row0 = s.tile * TR + (TWO ? kRows * x : 0);  // of the stream
            // queries: two neighbouring threads a row
            asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");  // both streams are done with the last
            if (TWO || x == 0) {
                const int qr = (tid & (kStream - 1)) >> 1, r = row0 + qr;
                const float f = put_query<D>(qbuf + (TWO ? x * kQ : 0), qr, tid & 1,
                                             p.q + static_cast<long long>(q0 + r / G) * p.q_stride + (s.h * G + r % G) * D,
                                             r < rows, p.scale_log2);
                if ((tid & 1) == 0) ct->qs[TWO ? x : 0][qr] = f;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            mbar_arrive(&ct->q_ready);
            asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
            const int r = row0 + row;
            const float qs = ct->qs[TWO ? x : 0][row];
            const int sees = r < rows ? row_sees(len, n, G, r) : 0;
            const int tile_sees = row_sees(len, n, G, row0);  // the least of the stream's rows

            float ref = -INFINITY, l = 0.f;
            for (int i = 0; i < steps; ++i) {
                const int it = base + (TWO ? i : 2 * i + x), st = it % NS;
                wait_or_abort(&ct->full[st], (it / NS) & 1, p, &ct->abort);  // the page's scales
                wait_or_abort(&ct->s_ready[x], (sn + i) & 1, p, &ct->abort);
                __syncwarp();
                tc_fence_after();
                // the row's scores of this page
                float a[64];
                tc_ld32(ts + 64 * y, *reinterpret_cast<float(*)[32]>(a));
                tc_ld32(ts + 64 * y + 32, *reinterpret_cast<float(*)[32]>(a + 32));
                const float ks = ct->ks[st][y], vs = ct->vs[st][y];
                const int pg = s.p0 + 2 * (it - base) + y;
                const bool none = ks < 0.f || pg >= s.pe;  // no such page
                const float fs = qs * ks;
                tc_wait_ld();
                if (none || (pg + 1) * kPage > tile_sees) {
                    const int lim = none ? 0 : sees - pg * kPage;
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j >= lim) a[j] = -INFINITY;
                }
                // their largest, in log2 units (a row's factor is not negative), with the other page's
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 64; j += 8)
#pragma unroll
                    for (int z = 0; z < 4; ++z) m4[z] = fmaxf(m4[z], fmaxf(a[j + z], a[j + 4 + z]));
                const float mr = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                float mx = mr > -INFINITY ? mr * fs + scale_log2(vs) : -INFINITY;
                ct->mx[x][y][row] = mx;
                tc_fence_before();
                stream_sync();  // (the weights overwrite the other page's scores: they have been read)
                tc_fence_after();
                mx = fmaxf(mx, ct->mx[x][y ^ 1][row]);
                const bool move = mx > ref + kSlack;  // (ref = -inf: as soon as anything is seen)
                if (__any_sync(0xffffffffu, move)) {
                    const float nref = move ? mx : ref;
                    const float f = move ? ex2(ref - nref) : 1.f;
                    l *= f;
                    ref = nref;
                    if (i > 0) {  // this thread's half of the row's accumulators
                        wait_or_abort(&ct->o_ready[x], (sn + i - 1) & 1, p, &ct->abort);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int h = 0; h < D / 32; ++h) {
                            float v[16];
                            uint32_t b[16];
                            tc_ld16(to + (D / 2) * y + 16 * h, v);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) b[j] = __float_as_uint(v[j] * f);
                            tc_st16(to + (D / 2) * y + 16 * h, b);
                        }
                    }
                }
                // 64 w vs as digits, 32 tokens at a time; w's sum from theirs
                const float pv = fmaxf(vs, 0x1p-64f) * kGain;
                const float add = __log2f(pv) - (ref == -INFINITY ? 0.f : ref);
                float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 32 * h; j < 32 * h + 32; ++j) {
                        a[j] = ex2(fmaf(a[j], fs, add));
                        l4[j & 3] += a[j];
                    }
                    uint32_t dg[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float *w = a + 32 * h + 4 * j;
                        digits4(w[0], w[1], w[2], w[3], dg[j], dg[8 + j]);
                    }
                    tc_st16(ts + 32 * y + 16 * h, dg);
                }
                l += ((l4[0] + l4[1]) + (l4[2] + l4[3])) * (1.f / pv);
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&ct->p_ready[x]);
            }
            sn += steps;
            on[0] += TWO ? stages : (stages + 1) / 2;
            on[1] += TWO ? stages : stages / 2;

            // ---- the result: o / 64 in tensor memory, references and sums
            if (y == 0) ct->m[x][row] = ref;
            ct->l[x][y][row] = l;
            asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
            const bool have0 = stages > 0, have1 = !TWO && stages > 1;
            const int x0 = TWO ? x : 0;
            if (have0) wait_or_abort(&ct->o_ready[x0], (on[x0] - 1) & 1, p, &ct->abort);
            if (have1) wait_or_abort(&ct->o_ready[1], (on[1] - 1) & 1, p, &ct->abort);
            __syncwarp();
            tc_fence_after();
            float f0 = 1.f, f1 = 0.f, msum = ref, lsum = ct->l[x0][0][row] + ct->l[x0][1][row];
            if (!TWO) {  // the streams' together
                const float m0 = ct->m[0][row], m1 = ct->m[1][row];
                msum = fmaxf(m0, m1);
                const float mref = msum == -INFINITY ? 0.f : msum;
                f0 = ex2(m0 - mref);
                f1 = ex2(m1 - mref);
                lsum = lsum * f0 + (ct->l[1][0][row] + ct->l[1][1][row]) * f1;
            }
            float *part = part_slot(p, blockIdx.x, s.p0 == 0);
            const int rr = TWO ? kRows * x + row : row;
            if (!s.whole() && y == 0 && (TWO || x == 0)) {
                part[rr] = msum;
                part[TR + rr] = lsum;
            }
            const float inv = inv_sum(kGain, lsum);
            uint16_t *orow = out_row(p, q0, s.h, G, min(r, rows - 1));
            constexpr int kCols = TWO ? D / 2 : D / 4;  // of this thread
            const int col0 = kCols * (TWO ? y : 2 * x + y);
#pragma unroll 1
            for (int col = col0; col < col0 + kCols; col += 16) {
                float v[16], w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = w[j] = 0.f;
                if (have0) tc_ld16(tmem + lanes + 256 * x0 + 128 + col, v);
                if (have1) tc_ld16(tmem + lanes + 256 + 128 + col, w);
                tc_wait_ld();
                if (!TWO) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = v[j] * f0 + w[j] * f1;
                }
                if (!s.whole()) {
                    float4 *o = reinterpret_cast<float4 *>(part + 2 * TR + rr * D + col);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
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
            if (!s.whole()) join_tile<D, kConsumers>(p, s, U, blocks, TR, rows, q0, G, kGain, &ct->last);
            base += stages;
            u += s.p1 - s.p0;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (wid == kIssuer) tc_dealloc(tmem, kTmemCols);
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
