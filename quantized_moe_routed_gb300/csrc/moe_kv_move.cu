// moe_kv_move.cu -- the paged 8-bit cache moved between sequences: keeping the accepted
// ones of a sequence's newest tokens (moe_kv_compact), sequences that go on from others
// (moe_kv_fork).
//
// Codes move as they are; where pages of different scales come together in one, those of
// smaller scale are requantised by the ratio.  Both move little: latency bounds them for
// few sequences, the memory's rate for many.
#include "moe_internal.h"
#include "moe_layer_internal.h"

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {
namespace {
#include "moe_device.cuh"
#include "moe_layer_device.cuh"

constexpr int kPage = MOE_KV_PAGE;
constexpr int kMoveThreads = 256;
constexpr int kTreePages = (MOE_KV_MAX_TREE + kPage - 2) / kPage + 1;  // pages that a tree's tokens can touch

// The factor from codes of scale s to codes of scale to: 1 where nothing has to change
// (a scale that is none leaves the codes alone).
__device__ __forceinline__ float requant_factor(float s, float to) { return s > 0.f && s < to ? s / to : 1.f; }

// A block per (sequence, kv head, k or v).  Pages that receive tokens are done one
// after the other: what one gets is read into registers, from itself and later
// pages, before it is written, and later pages are written later.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) moe_kv_compact_kernel(const CompactParams p)
{
    __shared__ int keep[MOE_KV_MAX_TREE];
    __shared__ int id[kTreePages];
    __shared__ float scale[kTreePages];
    const KvParams &c = p.c;
    grid_wait();
    grid_release();
    const int b = blockIdx.y, tid = threadIdx.x, h = blockIdx.x >> 1;
    const bool values = blockIdx.x & 1;
    const int a0 = c.q_off[b], a1 = c.q_off[b + 1], len = c.kv_len[b], m = p.n_keep[b];
    const int n = a1 - a0, past = len - n;
    bool bad = a0 < 0 || a1 < a0 || a1 > c.N || n > MOE_KV_MAX_TREE || len < 0 || len > c.max_pages * kPage || past < 0 || m < 0 ||
               m > min(n, p.max_keep);
    if (!bad) {  // (the same for all threads)
        const int32_t *row = p.keep + static_cast<size_t>(b) * p.max_keep;
        for (int j = tid; j < m; j += kMoveThreads) {
            const int k = row[j];
            keep[j] = k;
            bad |= k < 0 || k >= n || (j > 0 && row[j - 1] >= k);
        }
        bad = __syncthreads_or(bad);
    }
    const int p0 = past / kPage;
    if (!bad && m > 0) {
        const int pages = (past + keep[m - 1]) / kPage - p0 + 1;  // pages that hold a token that stays
        if (tid < pages) {
            const int page = c.pages[static_cast<size_t>(b) * c.max_pages + p0 + tid];
            bad = page < 0 || page >= c.n_pages;
            id[tid] = page;
            if (!bad) scale[tid] = (values ? c.vs : c.ks)[static_cast<size_t>(page) * c.kv_heads + h];
        }
        bad = __syncthreads_or(bad);
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.kv_len_out[b] = bad ? len : past + m;
        if (bad) atomicOr(c.ctrl + 2, kErrBadIndex);
    }
    if (bad) return;
    int j0 = 0;  // the first token that moves (all after it do)
    while (j0 < m && keep[j0] == j0) ++j0;
    uint8_t *codes = values ? c.v : c.k;
    float *scales = values ? c.vs : c.ks;
    auto page_at = [&](int t) { return codes + (static_cast<size_t>(id[t]) * c.kv_heads + h) * (kPage * D); };
    for (int at = j0; at < m;) {
        // page t of the tree's gets tokens at .. end - 1; it keeps those of its slots before slot0
        const int t = (past + at) / kPage - p0, slot0 = (past + at) % kPage, end = min(m, at + kPage - slot0);
        float to = slot0 > 0 ? scale[t] : 0.f;
        for (int j = at; j < end; ++j) to = fmaxf(to, scale[(past + keep[j]) / kPage - p0]);
        const float fall = requant_factor(scale[t], to);
        uint8_t *dst = page_at(t);
        if (!values) {
            // a granule of 16 codes of a token a thread, twice for a full page
            constexpr int UT = D / 16, IT = kPage * UT / kMoveThreads;
            uint4 w[IT];
#pragma unroll
            for (int x = 0; x < IT; ++x) {
                const int slot = (tid + x * kMoveThreads) / UT, u = (tid + x * kMoveThreads) % UT, j = at + slot - slot0;
                const bool in = j >= at && j < end;
                if (in) {
                    const int pos = past + keep[j], s = pos / kPage - p0;
                    w[x] = reinterpret_cast<const uint4 *>(page_at(s) + (pos % kPage) * D)[u];
                    const float f = requant_factor(scale[s], to);
                    if (f != 1.f) w[x] = requant16(w[x], f);
                } else if (fall != 1.f) {
                    w[x] = requant16(reinterpret_cast<const uint4 *>(dst + slot * D)[u], fall);
                }
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < IT; ++x) {
                const int slot = (tid + x * kMoveThreads) / UT, u = (tid + x * kMoveThreads) % UT, j = at + slot - slot0;
                if ((j >= at && j < end) || fall != 1.f) reinterpret_cast<uint4 *>(dst + slot * D)[u] = w[x];
            }
        } else {
            // four slots of a head dim a word: 16 words a row, a thread has the same four in every row of its
            constexpr int IT = D * (kPage / 4) / kMoveThreads;
            const int s0 = 4 * (tid & 15);
            bool any = fall != 1.f;
            const uint8_t *src[4];
            float f[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = at + s0 + y - slot0;
                src[y] = nullptr;
                f[y] = fall;
                if (j >= at && j < end) {
                    const int pos = past + keep[j], s = pos / kPage - p0;
                    src[y] = page_at(s) + pos % kPage;
                    f[y] = requant_factor(scale[s], to);
                    any = true;
                }
            }
            uint32_t w[IT];
            if (any) {
#pragma unroll
                for (int x = 0; x < IT; ++x) {
                    const int d = (tid >> 4) + x * (kMoveThreads / 16);
                    w[x] = *reinterpret_cast<const uint32_t *>(dst + d * kPage + s0);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        if (src[y])
                            w[x] = (w[x] & ~(0xFFu << (8 * y))) | static_cast<uint32_t>(src[y][d * kPage]) << (8 * y);
                    if (f[0] != 1.f || f[1] != 1.f || f[2] != 1.f || f[3] != 1.f) {
                        const float4 v = e4m3_unpack4(w[x]);
                        w[x] = e4m3_pack4(v.x * f[0], v.y * f[1], v.z * f[2], v.w * f[3]);
                    }
                }
            }
            __syncthreads();
            if (any) {
#pragma unroll
                for (int x = 0; x < IT; ++x)
                    *reinterpret_cast<uint32_t *>(dst + ((tid >> 4) + x * (kMoveThreads / 16)) * kPage + s0) = w[x];
            }
        }
        if (tid == 0) scales[static_cast<size_t>(id[t]) * c.kv_heads + h] = to;
        at = end;
    }
}

// A block per (child, kv head): the head's codes of the page that the child gets for
// its own; the first head's also writes the child's table.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) moe_kv_fork_kernel(const ForkParams p)
{
    const KvParams &c = p.c;
    grid_wait();
    grid_release();
    const int ch = blockIdx.x, tid = threadIdx.x, h = blockIdx.y;
    const int s = p.src[ch], fresh = p.fresh[ch];
    int len = 0, tail = 0, page = -1;
    bool bad = s < 0 || s >= c.B || fresh >= c.n_pages;
    if (!bad) {
        len = c.kv_len[s];
        bad = len < 0 || len > c.max_pages * kPage;
        if (!bad) {
            tail = len / kPage;
            if (fresh >= 0 && len % kPage) {
                page = c.pages[static_cast<size_t>(s) * c.max_pages + tail];
                bad = page < 0 || page >= c.n_pages;
            }
        }
    }
    if (fresh >= 0)
        for (int i = tid; i < ch; i += kMoveThreads) bad |= p.fresh[i] == fresh;
    bad = __syncthreads_or(bad);
    if (!bad && page >= 0) {
        const size_t to = static_cast<size_t>(fresh) * c.kv_heads + h, from = static_cast<size_t>(page) * c.kv_heads + h;
        constexpr int IT = kPage * D / 16 / kMoveThreads;
        const uint4 *ks = reinterpret_cast<const uint4 *>(c.k + from * (kPage * D));
        const uint4 *vs = reinterpret_cast<const uint4 *>(c.v + from * (kPage * D));
        uint4 kw[IT], vw[IT];
#pragma unroll
        for (int x = 0; x < IT; ++x) kw[x] = ks[tid + x * kMoveThreads];
#pragma unroll
        for (int x = 0; x < IT; ++x) vw[x] = vs[tid + x * kMoveThreads];
        uint4 *kd = reinterpret_cast<uint4 *>(c.k + to * (kPage * D)), *vd = reinterpret_cast<uint4 *>(c.v + to * (kPage * D));
#pragma unroll
        for (int x = 0; x < IT; ++x) kd[tid + x * kMoveThreads] = kw[x];
#pragma unroll
        for (int x = 0; x < IT; ++x) vd[tid + x * kMoveThreads] = vw[x];
        if (tid == 0) {
            c.ks[to] = c.ks[from];
            c.vs[to] = c.vs[from];
        }
    }
    if (h != 0) return;
    const int32_t *row = c.pages + static_cast<size_t>(bad ? 0 : s) * c.max_pages;
    int32_t *out = p.pages_out + static_cast<size_t>(ch) * c.max_pages;
    for (int i = tid; i < c.max_pages; i += kMoveThreads) out[i] = bad ? -1 : (i == tail && fresh >= 0 ? fresh : row[i]);
    if (tid == 0) {
        p.kv_len_out[ch] = bad ? 0 : len;
        if (bad) atomicOr(c.ctrl + 2, kErrBadIndex);
    }
}

}  // namespace

cudaError_t launch_kv_compact(const CompactParams &p, cudaStream_t st)
{
    LaunchCfg l(dim3(2 * p.c.kv_heads, p.c.B), dim3(kMoveThreads), 0, st);
    return p.c.D == 128 ? cudaLaunchKernelEx(&l.cfg, moe_kv_compact_kernel<128>, p)
                        : cudaLaunchKernelEx(&l.cfg, moe_kv_compact_kernel<64>, p);
}

cudaError_t launch_kv_fork(const ForkParams &p, cudaStream_t st)
{
    LaunchCfg l(dim3(p.C, p.c.kv_heads), dim3(kMoveThreads), 0, st);
    return p.c.D == 128 ? cudaLaunchKernelEx(&l.cfg, moe_kv_fork_kernel<128>, p)
                        : cudaLaunchKernelEx(&l.cfg, moe_kv_fork_kernel<64>, p);
}

}  // namespace moe
