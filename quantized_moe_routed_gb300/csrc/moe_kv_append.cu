// moe_kv_append.cu -- rotation of queries and keys, and the append of keys and
// values to the paged 8-bit cache (moe_kv_append).
//
//   pair (a, b) of a head's rotated part: (a cos - b sin, b cos + a sin)
//   scale of a page and head: 2^e >= largest / 448, never below the one in the
//   page when the page already holds tokens; codes E4M3(value / scale)
//
// One block per (page that gets new tokens, kv head) writes that page's codes
// and scales of k and of v: the scale needs the largest of all new values of
// the page, and its growth the page's old codes, so a page and head is the
// unit that no two blocks share (no atomics, the same bits every run).  Another
// block per (page, kv head) rotates the head group's queries.  Bytes bound it
// for prefill chunks; for single tokens the chain of dependent loads (lengths,
// page id, old scale, codes) does.
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
constexpr int kThreads = 256;
// 448 * 2^60, what the largest scale holds: attention's softmax weights are
// taken relative to the largest (weight x v scale), and this range of scales
// keeps the smallest ones that count inside fp32.
constexpr float kMaxValue = 448.f * 1152921504606846976.f;

// The elements of rotated pair j (j < rot / 2); pairs past it are (2j, 2j + 1).
__device__ __forceinline__ void pair_at(const KvParams &c, int j, int &i0, int &i1)
{
    const bool half = j < c.rot_dim / 2 && !c.rot_inter;
    i0 = half ? j : 2 * j;
    i1 = half ? j + c.rot_dim / 2 : 2 * j + 1;
}

// Rotate pair (a, b) by the table's angle; every product and sum rounded on
// its own, so that the codes are those of the formula in fp32.
__device__ __forceinline__ void rotate(float &a, float &b, float2 cs)
{
    const float ra = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
    const float rb = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
    a = ra;
    b = rb;
}

// cnt tokens of D bf16 (src, stride elements apart) as fp32 into t[cnt][D + 1].
template <int D>
__device__ __forceinline__ void load_tile(float *t, const uint16_t *src, long long stride, int cnt)
{
    for (int i = threadIdx.x; i < cnt * (D / 8); i += kThreads) {
        const int tok = i / (D / 8), c = (i % (D / 8)) * 8;
        const uint4 a = *reinterpret_cast<const uint4 *>(src + tok * stride + c);
        float *o = t + tok * (D + 1) + c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[2 * j] = bf16_lo(u4w(a, j));
            o[2 * j + 1] = bf16_hi(u4w(a, j));
        }
    }
}

// Rotate the tile in place: token i is at position pos0 + i.
template <int D>
__device__ __forceinline__ void rotate_tile(const KvParams &c, float *t, int cnt, int pos0)
{
    const int np = c.rot_dim / 2;
    for (int i = threadIdx.x; i < cnt * np; i += kThreads) {
        const int tok = i / np, j = i % np;
        int i0, i1;
        pair_at(c, j, i0, i1);
        const float2 cs = __ldg(reinterpret_cast<const float2 *>(c.rope + static_cast<size_t>(pos0 + tok) * c.rot_dim) + j);
        rotate(t[tok * (D + 1) + i0], t[tok * (D + 1) + i1], cs);
    }
}

__device__ __forceinline__ float block_max(float v, float *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kThreads / 32; ++i) v = fmaxf(v, red[i]);
    __syncthreads();
    return v;
}

// Sixteen codes times f (a power of two, or a ratio of caller's scales).
__device__ __forceinline__ uint4 requant16(uint4 w, float f)
{
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = e4m3_unpack4(u4w(w, i));
        o[i] = e4m3_pack4(v.x * f, v.y * f, v.z * f, v.w * f);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The page's new scale from the new tokens' largest, and the factor of the
// codes already there (1: they stay).
__device__ __forceinline__ float new_scale(float amax, bool old_tokens, float old, float &factor)
{
    float s = exp2i(scale_exp(amax));
    factor = 1.f;
    if (old_tokens && old > 0.f && old < INFINITY) {
        if (old >= s)
            s = old;
        else
            factor = old / s;
    }
    return s;
}

template <int D>
__global__ void __launch_bounds__(kThreads) moe_kv_append_kernel(const AppendParams p)
{
    extern __shared__ float tile[];  // [2][kPage][D + 1]: k, v (or one query head)
    __shared__ float red[kThreads / 32];
    __shared__ int bad_tok[kPage];
    const KvParams &c = p.c;
    grid_wait();
    grid_release();
    const int b = blockIdx.y, tid = threadIdx.x, hk = c.kv_heads;
    const bool queries = static_cast<int>(blockIdx.z) >= hk;
    const int h = queries ? blockIdx.z - hk : blockIdx.z;
    // the sequence, with offsets and lengths kept inside the step's arrays
    const int q0 = min(max(c.q_off[b], 0), c.N), q1 = min(max(c.q_off[b + 1], q0), c.N);
    const int n = q1 - q0, lens = c.kv_len[b];
    const int len = lens < 0 || lens > c.max_pages * kPage ? 0 : lens;  // out of range: nothing has a position
    const int first = len - n;  // position of the first new token
    if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0 &&
        (q0 != c.q_off[b] || q1 != c.q_off[b + 1] || first < 0 || len != lens))
        atomicOr(c.ctrl + 2, kErrBadIndex);
    if (n == 0) return;
    if (queries && blockIdx.x == 0 && first < 0) {  // new tokens without a position
        const int G = c.q_heads / hk, rows = min(n, -first);
        for (int i = tid; i < rows * G * (D / 8); i += kThreads) {
            const int tok = i / (G * (D / 8)), cc = i % (G * (D / 8)) * 8;
            *reinterpret_cast<uint4 *>(p.q_out + (static_cast<size_t>(q0 + tok) * c.q_heads + h * G) * D + cc) =
                make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const int page0 = max(first, 0) / kPage;
    for (int pg = page0 + blockIdx.x; pg * kPage < len; pg += gridDim.x) {
        const int pos0 = max(pg * kPage, first);                        // first new token of the page
        const int cnt = min(pg * kPage + kPage, len) - pos0;            // new tokens of the page
        const int row0 = q0 + (pos0 - first);                           // its row in q, k and v
        const int slot0 = pos0 - pg * kPage;
        const int id = c.pages[static_cast<size_t>(b) * c.max_pages + pg];
        const bool ok = id >= 0 && id < c.n_pages && (c.rot_dim == 0 || pos0 + cnt <= c.rope_positions);
        if (!ok && tid == 0) atomicOr(c.ctrl + 2, kErrBadIndex);
        if (queries) {
            const int G = c.q_heads / hk;
            for (int g = 0; g < G; ++g) {
                const int hq = h * G + g;
                __syncthreads();
                load_tile<D>(tile, p.q + row0 * p.q_stride + hq * D, p.q_stride, cnt);
                __syncthreads();
                if (ok) rotate_tile<D>(c, tile, cnt, pos0);
                __syncthreads();
                for (int i = tid; i < cnt * (D / 8); i += kThreads) {
                    const int tok = i / (D / 8), cc = (i % (D / 8)) * 8;
                    const float *t = tile + tok * (D + 1) + cc;
                    uint4 o = make_uint4(0u, 0u, 0u, 0u);
                    if (ok)
                        o = make_uint4(pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3]), pack_bf16(t[4], t[5]),
                                       pack_bf16(t[6], t[7]));
                    *reinterpret_cast<uint4 *>(p.q_out + (static_cast<size_t>(row0 + tok) * c.q_heads + hq) * D + cc) = o;
                }
            }
            continue;
        }
        if (!ok) continue;
        float *tk = tile, *tv = tile + kPage * (D + 1);
        const size_t ph = static_cast<size_t>(id) * hk + h;
        const float old_ks = c.ks[ph], old_vs = c.vs[ph];
        __syncthreads();
        if (tid < kPage) bad_tok[tid] = 0;
        load_tile<D>(tk, p.k + row0 * p.k_stride + h * D, p.k_stride, cnt);
        load_tile<D>(tv, p.v + row0 * p.v_stride + h * D, p.v_stride, cnt);
        __syncthreads();
        rotate_tile<D>(c, tk, cnt, pos0);
        __syncthreads();
        for (int i = tid; i < cnt * D; i += kThreads) {
            const int o = (i / D) * (D + 1) + i % D;
            if (!(fabsf(tk[o]) <= kMaxValue) || !(fabsf(tv[o]) <= kMaxValue)) bad_tok[i / D] = 1;
        }
        __syncthreads();
        float ak = 0.f, av = 0.f;
        for (int i = tid; i < cnt * D; i += kThreads) {
            const int o = (i / D) * (D + 1) + i % D;
            if (bad_tok[i / D]) {
                tk[o] = __int_as_float(0x7FC00000);
                tv[o] = 0.f;
            } else {
                ak = fmaxf(ak, fabsf(tk[o]));
                av = fmaxf(av, fabsf(tv[o]));
            }
        }
        ak = block_max(ak, red);
        av = block_max(av, red);
        float fk, fv;
        const float sk = new_scale(ak, slot0 > 0, old_ks, fk), sv = new_scale(av, slot0 > 0, old_vs, fv);
        const float ik = 1.f / sk, iv = 1.f / sv;
        // k: a token's codes are contiguous
        uint8_t *ko = c.k + ph * (kPage * D);
        for (int i = tid; i < kPage * (D / 16); i += kThreads) {
            const int tok = i / (D / 16), cc = (i % (D / 16)) * 16, r = tok - slot0;
            uint4 *dst = reinterpret_cast<uint4 *>(ko + tok * D + cc);
            if (r >= 0 && r < cnt) {
                const float *t = tk + r * (D + 1) + cc;
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = e4m3_pack4(t[4 * j] * ik, t[4 * j + 1] * ik, t[4 * j + 2] * ik, t[4 * j + 3] * ik);
                *dst = make_uint4(o[0], o[1], o[2], o[3]);
            } else if (fk != 1.f) {
                *dst = requant16(*dst, fk);
            }
        }
        // v: a head dimension's codes are contiguous; sixteen tokens at a time
        uint8_t *vo = c.v + ph * (kPage * D);
        for (int i = tid; i < D * (kPage / 16); i += kThreads) {
            const int d = i % D, s0 = (i / D) * 16;
            const int lo = max(slot0 - s0, 0), hi = min(slot0 + cnt - s0, 16);
            uint4 *dst = reinterpret_cast<uint4 *>(vo + d * kPage + s0);
            const bool some = lo < hi;
            if (!some && fv == 1.f) continue;
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (!(lo == 0 && hi == 16)) {
                w = *dst;
                if (fv != 1.f) w = requant16(w, fv);
            }
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t m = 0u, x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int tok = 4 * j + u;
                    const bool in = tok >= lo && tok < hi;
                    x[u] = __float_as_uint(in ? tv[(s0 + tok - slot0) * (D + 1) + d] * iv : 0.f);
                    if (in) m |= 0xFFu << (8 * u);
                }
                o[j] = (e4m3_pack4(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]),
                                   __uint_as_float(x[3])) & m) |
                       (u4w(w, j) & ~m);
            }
            *dst = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (tid == 0) {
            c.ks[ph] = sk;
            c.vs[ph] = sv;
        }
    }
}

template <int D>
cudaError_t launch_d(const AppendParams &p, cudaStream_t st)
{
    const int smem = 2 * kPage * (D + 1) * 4;
    cudaError_t e = cudaFuncSetAttribute(moe_kv_append_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const KvParams &c = p.c;
    // pages a sequence's new tokens can touch; a block walks on where max_q was
    // given too small
    const int pages = std::min(std::max(c.max_q, 1) / kPage + 2, c.max_pages);
    LaunchCfg l(dim3(c.max_q <= 1 ? 1 : pages, c.B, c.kv_heads * (p.q ? 2 : 1)), dim3(kThreads), smem, st);
    return cudaLaunchKernelEx(&l.cfg, moe_kv_append_kernel<D>, p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t st)
{
    return p.c.D == 128 ? launch_d<128>(p, st) : launch_d<64>(p, st);
}

}  // namespace moe
