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

// A block per (sequence, kv head).  Pages that receive tokens are done one after the
// other: what one gets is read into registers, from itself and later pages, before it is
// written, and later pages are written later.  What bounds it is the chain of dependent loads
// (lengths and kept tokens, pages, scales and codes: three in a row): 16 tokens of one
// sequence take 4.4 us, 128 sequences of 60 9.9 us in 1.7 turns of four blocks an SM (13.5 with
// a block for k, one for v and a load more in the chain).
template <int D>
__global__ void __launch_bounds__(kMoveThreads, 4) moe_kv_compact_kernel(const CompactParams p)
{
    static_assert(kMoveThreads >= MOE_KV_MAX_TREE, "a kept token a thread");
    __shared__ int keep[MOE_KV_MAX_TREE];
    __shared__ int id[kTreePages];
    __shared__ float ks[kTreePages], vs[kTreePages];
    const KvParams &c = p.c;
    grid_wait();
    grid_release();
    const int b = blockIdx.y, tid = threadIdx.x, h = blockIdx.x;
    const int mine = tid < p.max_keep ? p.keep[static_cast<size_t>(b) * p.max_keep + tid] : 0;
    const int a0 = c.q_off[b], a1 = c.q_off[b + 1], len = c.kv_len[b], m = p.n_keep[b];
    bool bad = a0 < 0 || a1 < a0 || a1 > c.N || a1 - a0 > MOE_KV_MAX_TREE || len < 0 || len > c.max_pages * kPage;
    const int n = bad ? 0 : a1 - a0, past = len - n;
    bad |= past < 0 || m < 0 || m > min(n, p.max_keep);
    const int p0 = bad ? 0 : past / kPage;  // (the same for all threads so far)
    if (tid < MOE_KV_MAX_TREE) keep[tid] = mine;
    if (tid < kTreePages)
        id[tid] = !bad && p0 + tid < c.max_pages ? c.pages[static_cast<size_t>(b) * c.max_pages + p0 + tid] : -1;
    __syncthreads();
    if (!bad && m > 0) {
        auto is_page = [&](int pos) {
            const int t = pos / kPage - p0;
            return id[t] >= 0 && id[t] < c.n_pages;
        };
        // the pages that a token comes from and goes to have to be some; those between may be anything
        if (tid < m) bad = mine < 0 || mine >= n || (tid > 0 && keep[tid - 1] >= mine) || !is_page(past + mine) || !is_page(past + tid);
    }
    bad = __syncthreads_or(bad);
    if (h == 0 && tid == 0) {
        p.kv_len_out[b] = bad ? len : past + m;
        if (bad) atomicOr(c.ctrl + 2, kErrBadIndex);
    }
    if (bad) return;
    int j0 = 0;  // the first token that moves (all after it do)
    while (j0 < m && keep[j0] == j0) ++j0;
    if (j0 == m) return;
    if (const int pages = (past + keep[m - 1]) / kPage - p0 + 1; tid < pages && id[tid] >= 0 && id[tid] < c.n_pages) {
        const size_t ph = static_cast<size_t>(id[tid]) * c.kv_heads + h;
        ks[tid] = c.ks[ph];
        vs[tid] = c.vs[ph];
    }
    auto codes_at = [&](uint8_t *codes, int t) { return codes + (static_cast<size_t>(id[t]) * c.kv_heads + h) * (kPage * D); };
    // of k a granule of 16 codes of a token a thread, twice for a full page; of v four slots of a head
    // dim, a word, the same four in every row that the thread has
    constexpr int UT = D / 16, KI = kPage * UT / kMoveThreads, VI = D * (kPage / 4) / kMoveThreads;
    const int s0 = 4 * (tid & 15), d0 = tid >> 4;
    for (int at = j0; at < m;) {
        // page t of the tree's gets tokens at .. end - 1; it keeps those of its slots before slot0
        const int t = (past + at) / kPage - p0, slot0 = (past + at) % kPage, end = min(m, at + kPage - slot0);
        uint8_t *kd = codes_at(c.k, t), *vd = codes_at(c.v, t);
        uint4 kw[KI];
        uint32_t vw[VI];
        int kfrom[KI], vfrom[4];  // the page of the tree that a token comes from; -1: none comes
#pragma unroll
        for (int x = 0; x < KI; ++x) {
            const int slot = (tid + x * kMoveThreads) / UT, u = (tid + x * kMoveThreads) % UT, j = at + slot - slot0;
            kfrom[x] = -1;
            if (j >= at && j < end) {
                const int pos = past + keep[j];
                kfrom[x] = pos / kPage - p0;
                kw[x] = reinterpret_cast<const uint4 *>(codes_at(c.k, kfrom[x]) + (pos % kPage) * D)[u];
            }
        }
        const uint8_t *src[4];
        bool some = false;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int j = at + s0 + y - slot0;
            vfrom[y] = -1;
            if (j >= at && j < end) {
                const int pos = past + keep[j];
                vfrom[y] = pos / kPage - p0;
                src[y] = codes_at(c.v, vfrom[y]) + pos % kPage;
                some = true;
            }
        }
        if (some) {
#pragma unroll
            for (int x = 0; x < VI; ++x) {
                const int d = d0 + x * (kMoveThreads / 16);
                vw[x] = *reinterpret_cast<const uint32_t *>(vd + d * kPage + s0);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (vfrom[y] >= 0) vw[x] = (vw[x] & ~(0xFFu << (8 * y))) | static_cast<uint32_t>(src[y][d * kPage]) << (8 * y);
            }
        }
        __syncthreads();  // (the scales are there)
        float kto = slot0 > 0 ? ks[t] : 0.f, vto = slot0 > 0 ? vs[t] : 0.f;
        for (int j = at; j < end; ++j) {
            const int from = (past + keep[j]) / kPage - p0;
            kto = fmaxf(kto, ks[from]);
            vto = fmaxf(vto, vs[from]);
        }
        const float kfall = requant_factor(ks[t], kto), vfall = requant_factor(vs[t], vto);
#pragma unroll
        for (int x = 0; x < KI; ++x) {
            if (kfrom[x] >= 0) {
                const float f = requant_factor(ks[kfrom[x]], kto);
                if (f != 1.f) kw[x] = requant16(kw[x], f);
            } else if (kfall != 1.f) {
                kw[x] = requant16(reinterpret_cast<const uint4 *>(kd)[tid + x * kMoveThreads], kfall);
            }
        }
        if (some || vfall != 1.f) {
            float f[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) f[y] = vfrom[y] >= 0 ? requant_factor(vs[vfrom[y]], vto) : vfall;
#pragma unroll
            for (int x = 0; x < VI; ++x) {
                if (!some) vw[x] = *reinterpret_cast<const uint32_t *>(vd + (d0 + x * (kMoveThreads / 16)) * kPage + s0);
                if (f[0] != 1.f || f[1] != 1.f || f[2] != 1.f || f[3] != 1.f) {
                    const float4 v = e4m3_unpack4(vw[x]);
                    vw[x] = e4m3_pack4(v.x * f[0], v.y * f[1], v.z * f[2], v.w * f[3]);
                }
            }
        }
        __syncthreads();  // all has been read
#pragma unroll
        for (int x = 0; x < KI; ++x)
            if (kfrom[x] >= 0 || kfall != 1.f) reinterpret_cast<uint4 *>(kd)[tid + x * kMoveThreads] = kw[x];
        if (some || vfall != 1.f) {
#pragma unroll
            for (int x = 0; x < VI; ++x) *reinterpret_cast<uint32_t *>(vd + (d0 + x * (kMoveThreads / 16)) * kPage + s0) = vw[x];
        }
        if (tid == 0) {
            const size_t ph = static_cast<size_t>(id[t]) * c.kv_heads + h;
            c.ks[ph] = kto;
            c.vs[ph] = vto;
        }
        at = end;
    }
}

// A block per (child, kv head): the head's codes of the page that the child gets for
// its own; the first head's also writes the child's table.  Three dependent loads (source and fresh
// page, length, table, then codes) bound it: 8 children take 2.6 us; 384 of 8 heads, of which 170 copy a page,
// 7.8 us in 3.4 turns of six blocks an SM, where the 34 MB that they move would take 5.0.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) moe_kv_fork_kernel(const ForkParams p)
{
    const KvParams &c = p.c;
    grid_wait();
    grid_release();
    const int ch = blockIdx.x, tid = threadIdx.x, h = blockIdx.y;
    const int s = p.src[ch], fresh = p.fresh[ch];
    int len = 0, tail = 0, page = -1;
    // an earlier child that gets the same fresh page, or is left the same page (both would append to it if
    // that is partly filled)
    bool twin = false;
    for (int i = tid; i < ch; i += kMoveThreads) twin |= fresh >= 0 ? p.fresh[i] == fresh : p.fresh[i] < 0 && p.src[i] == s;
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
    bad |= twin && (fresh >= 0 || len % kPage != 0);
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
    LaunchCfg l(dim3(p.c.kv_heads, p.c.B), dim3(kMoveThreads), 0, st);
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
