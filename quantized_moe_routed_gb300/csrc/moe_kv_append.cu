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
// block per (page, kv head) rotates the head group's queries.  The chain of
// dependent loads (lengths, page id, old scale, codes) bounds it, for single tokens
// (24 sequences: 4.75 us) and for chunks (4 x 4096 tokens of 32 + 16 heads of 128:
// 37.0 us, 55% of the rate of a copy of the same bytes), where 64 registers a thread let
// two blocks of 512 share an SM; so the new tokens' loads do not wait for the
// page's id, v stays packed until it is coded (44.5 us otherwise), and what a thread reads
// next, a head of the queries or the page's old codes of v, is under way before it is
// needed (without: 5.0 and 37.9 us; 32 sequences of 60 tokens after 8192, all 128 columns turned,
// 17.3 instead of 15.4, as trees 17.8 instead of 16.4).
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
// 448 * 2^60, what the largest scale holds: attention's softmax weights are
// taken relative to the largest (weight x v scale), and this range of scales
// keeps the smallest ones that count inside fp32.
constexpr float kMaxValue = 448.f * 1152921504606846976.f;

// Which elements a rotation pairs: neighbours; element i of the two halves, where
// 16 divides rot_dim; the same otherwise.
enum Rot { kNone, kNeighbours, kHalves, kOddHalves };

// A unit is 16 elements of a head that a thread holds: 8 from c0 on and 8 from c1
// on, which are each other's partners in the rotated part of kHalves, else lie
// one after the other.
template <Rot ROT>
struct Units {
    int c0, c1;
    __device__ __forceinline__ Units(const KvParams &c, int u)
    {
        const bool apart = ROT == kHalves && u < c.rot_dim / 16;
        c0 = apart ? 8 * u : 16 * u;
        c1 = apart ? c0 + c.rot_dim / 2 : 16 * u + 8;
    }
};

__device__ __forceinline__ uint4 at8(const uint16_t *src) { return *reinterpret_cast<const uint4 *>(src); }

__device__ __forceinline__ void unpack8(float *v, const uint4 &a)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(u4w(a, j));
        v[2 * j + 1] = bf16_hi(u4w(a, j));
    }
}

// The (cos, sin) of the unit's eight pairs (pairs of the table 8 u .. 8 u + 7; (1,
// 0) past the rotated part).
template <Rot ROT>
__device__ __forceinline__ void load_angles(const KvParams &c, float2 (&cs)[8], int pos, int u)
{
    if (ROT == kNone || ROT == kOddHalves) return;
    const float2 *t = reinterpret_cast<const float2 *>(c.rope + static_cast<size_t>(pos) * c.rot_dim) + 8 * u;
    if (ROT == kHalves) {  // eight pairs, or none (turn_unit turns none)
        if (8 * u >= c.rot_dim / 2) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = __ldg(t + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 8 * u + i < c.rot_dim / 2 ? __ldg(t + i) : make_float2(1.f, 0.f);
    }
}

// (a, b) turned: every product and sum rounded on its own, so that the values are
// those of the formula in fp32.
__device__ __forceinline__ float turn_a(float a, float b, float2 cs)
{
    return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float turn_b(float a, float b, float2 cs)
{
    return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// A head's unit (lo, hi: its elements from c0 and from c1 on), rotated.
template <Rot ROT>
__device__ __forceinline__ void turn_unit(const KvParams &c, float (&v)[16], const uint4 &lo, const uint4 &hi,
                                          const uint16_t *head, const Units<ROT> &un, const float2 (&cs)[8], int pos)
{
    unpack8(v, lo);
    unpack8(v + 8, hi);
    if (ROT == kNeighbours) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (un.c0 + 2 * i < c.rot_dim) {
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = turn_a(a, b, cs[i]);
                v[2 * i + 1] = turn_b(a, b, cs[i]);
            }
    } else if (ROT == kHalves) {
        if (un.c0 < c.rot_dim / 2) {  // (a rotated unit begins in the first half)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = v[i], b = v[8 + i];
                v[i] = turn_a(a, b, cs[i]);
                v[8 + i] = turn_b(a, b, cs[i]);
            }
        }
    } else if (ROT == kOddHalves) {
        const int half = c.rot_dim / 2;
        const float2 *t = reinterpret_cast<const float2 *>(c.rope + static_cast<size_t>(pos) * c.rot_dim);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int d = un.c0 + i;
            if (d >= c.rot_dim) continue;
            const float o = __uint_as_float(static_cast<uint32_t>(head[d < half ? d + half : d - half]) << 16);
            v[i] = d < half ? turn_a(v[i], o, __ldg(t + d)) : turn_b(o, v[i], __ldg(t + d - half));
        }
    }
}

// The larger of a and b, or NaN where either is one.
__device__ __forceinline__ float nan_max(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The block's largest of a and of b.
template <int THREADS>
__device__ __forceinline__ void block_max2(float &a, float &b, float *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
        red[2 * w] = a;
        red[2 * w + 1] = b;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        a = fmaxf(a, red[2 * i]);
        b = fmaxf(b, red[2 * i + 1]);
    }
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

// TREE: the new tokens are trees, turned by their depth behind the tokens before the tree.
template <int D, Rot ROT, bool TREE>
__global__ void __launch_bounds__(kPage *D / 16, 2048 / (kPage * D / 16) / 2) moe_kv_append_kernel(const AppendParams p)
{
    constexpr int UT = D / 16;            // units of a token
    constexpr int kThreads = kPage * UT;  // a unit of a full page each
    constexpr int kStride = kPage + 4;          // bytes of a v row in shared memory: no bank twice
    __shared__ uint32_t vt[D * kStride / 4];    // v codes, transposed
    __shared__ float red[2 * kThreads / 32];
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
    // out of range, or too long for a tree: nothing has a position
    const int len = lens < 0 || lens > c.max_pages * kPage || (TREE && n > MOE_KV_MAX_TREE) ? 0 : lens;
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
    struct Page {
        int pos0, cnt;  // first new token of the page, its new tokens
        int row0;       // that token's row in q, k and v
        int slot0, id;  // its slot; the page's id, which the new tokens' loads do not wait for
        bool turns;     // all positions are inside the table
    };
    auto page = [&](int pg) {
        Page r;
        r.pos0 = max(pg * kPage, first);
        r.cnt = min(pg * kPage + kPage, len) - r.pos0;
        r.row0 = q0 + (r.pos0 - first);
        r.slot0 = r.pos0 - pg * kPage;
        r.id = c.pages[static_cast<size_t>(b) * c.max_pages + pg];
        r.turns = c.rot_dim == 0 || r.pos0 + r.cnt <= c.rope_positions;
        return r;
    };
    // The position that turns the token stored at `at` (never behind it: inside the table if that is).
    auto angle_at = [&](int at) {
        if (!TREE || ROT == kNone) return at;
        int depth = 0;
        for (int i = at - first; i >= 0;) {  // (a parent is an earlier token, so this ends)
            const int up = __ldg(p.parent + q0 + i);
            if (up >= i || up < -1) {
                atomicOr(c.ctrl + 2, kErrBadIndex);
                break;
            }
            if (up >= 0) ++depth;
            i = up;
        }
        return max(first + depth, 0);
    };
    // (two loops: in one, what either kind of block needs would be held through the other's)
    if (queries) {
        for (int pg = page0 + blockIdx.x; pg * kPage < len; pg += gridDim.x) {
            const auto [pos0, cnt, row0, slot0, id, turns] = page(pg);
            const int G = c.q_heads / hk;
            if (const int tok = tid / UT, u = tid % UT; tok < cnt) {
                const Units<ROT> un(c, u);
                float2 cs[8];
                const int pos = turns ? angle_at(pos0 + tok) : 0;
                if (turns) load_angles<ROT>(c, cs, pos, u);
                const uint16_t *src = p.q + (row0 + tok) * p.q_stride + h * G * D;
                uint16_t *dst = p.q_out + (static_cast<size_t>(row0 + tok) * c.q_heads + h * G) * D;
                // a head's loads are under way while the one before it is turned
                uint4 lo = at8(src + un.c0), hi = at8(src + un.c1);
#pragma unroll 1
                for (int g = 0; g < G; ++g) {
                    float v[16];
                    const uint4 lo0 = lo, hi0 = hi;
                    if (g + 1 < G) lo = at8(src + (g + 1) * D + un.c0), hi = at8(src + (g + 1) * D + un.c1);
                    if (turns) turn_unit<ROT>(c, v, lo0, hi0, src + g * D, un, cs, pos);
                    // where partners are other elements of the token's UT lanes, all are read before
                    // any is written: the queries may be rotated in place
                    if (ROT == kOddHalves) __syncwarp(((1u << UT) - 1u) << (tid & 31 & ~(UT - 1)));
                    if (!turns || id < 0 || id >= c.n_pages) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = 0.f;
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        *reinterpret_cast<uint4 *>(dst + g * D + (y ? un.c1 : un.c0)) =
                            make_uint4(pack_bf16(v[8 * y], v[8 * y + 1]), pack_bf16(v[8 * y + 2], v[8 * y + 3]),
                                       pack_bf16(v[8 * y + 4], v[8 * y + 5]), pack_bf16(v[8 * y + 6], v[8 * y + 7]));
                }
            }
        }
        return;
    }
    for (int pg = page0 + blockIdx.x; pg * kPage < len; pg += gridDim.x) {
        const auto [pos0, cnt, row0, slot0, id, turns] = page(pg);
        const int tok = tid / UT, u = tid % UT;
        const bool in = tok < cnt;
        const Units<ROT> un(c, u);
        float x[16];  // the thread's unit of k
        uint4 z[2];   // and of v, as it is
        if (in && turns) {
            float2 cs[8];
            const uint4 *zp = reinterpret_cast<const uint4 *>(p.v + (row0 + tok) * p.v_stride + h * D + 16 * u);
            z[0] = zp[0];
            z[1] = zp[1];
            const int pos = angle_at(pos0 + tok);
            load_angles<ROT>(c, cs, pos, u);
            const uint16_t *kp = p.k + (row0 + tok) * p.k_stride + h * D;
            turn_unit<ROT>(c, x, at8(kp + un.c0), at8(kp + un.c1), kp, un, cs, pos);
        }
        if (!turns || id < 0 || id >= c.n_pages) {
            if (tid == 0) atomicOr(c.ctrl + 2, kErrBadIndex);
            continue;
        }
        const size_t ph = static_cast<size_t>(id) * hk + h;
        const float old_ks = c.ks[ph], old_vs = c.vs[ph];
        // v: a head dimension's codes are contiguous; sixteen tokens of one a thread, lo .. hi - 1 of them new
        const int d = tid % D, s0 = (tid / D) * 16, lo = max(slot0 - s0, 0), hi = min(slot0 + cnt - s0, 16);
        uint4 *vo = reinterpret_cast<uint4 *>(c.v + ph * (kPage * D) + d * kPage + s0);
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (lo < hi && (lo > 0 || hi < 16)) w = *vo;
        __syncthreads();  // the last page's readers of shared memory are done
        if (tid < kPage) bad_tok[tid] = 0;
        __syncthreads();
        float ak = 0.f, av = 0.f;
        if (in) {
#pragma unroll
            for (int j = 0; j < 16; ++j) ak = nan_max(ak, fabsf(x[j]));
            uint32_t am = 0u;  // v's largest magnitude, as bits (a NaN's are above infinity's)
#pragma unroll
            for (int j = 0; j < 8; ++j) am = __vmaxu2(am, u4w(z[j >> 2], j & 3) & 0x7FFF7FFFu);
            av = __uint_as_float(max(am >> 16, am & 0xFFFFu) << 16);
            if (!(ak <= kMaxValue) || !(av <= kMaxValue)) bad_tok[tok] = 1;
        }
        __syncthreads();
        if (in && bad_tok[tok] != 0) {
            ak = av = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = __int_as_float(0x7FC00000);
            z[0] = z[1] = make_uint4(0u, 0u, 0u, 0u);
        }
        block_max2<kThreads>(ak, av, red);
        float fk, fv;
        const float sk = new_scale(ak, slot0 > 0, old_ks, fk), sv = new_scale(av, slot0 > 0, old_vs, fv);
        const float ik = 1.f / sk, iv = 1.f / sv;
        // k: a token's codes are contiguous; v goes through shared memory, transposed
        uint8_t *ko = c.k + ph * (kPage * D);
        if (in) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint2 o;
                o.x = e4m3_pack4(x[8 * y] * ik, x[8 * y + 1] * ik, x[8 * y + 2] * ik, x[8 * y + 3] * ik);
                o.y = e4m3_pack4(x[8 * y + 4] * ik, x[8 * y + 5] * ik, x[8 * y + 6] * ik, x[8 * y + 7] * ik);
                *reinterpret_cast<uint2 *>(ko + (slot0 + tok) * D + (y ? un.c1 : un.c0)) = o;
            }
            uint8_t *t = reinterpret_cast<uint8_t *>(vt) + 16 * u * kStride + slot0 + tok;
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const uint32_t z0 = u4w(z[j >> 3], (j >> 1) & 3), z1 = u4w(z[j >> 3], ((j >> 1) & 3) + 1);
                const uint32_t w = e4m3_pack4(bf16_lo(z0) * iv, bf16_hi(z0) * iv, bf16_lo(z1) * iv, bf16_hi(z1) * iv);
#pragma unroll
                for (int b = 0; b < 4; ++b) t[(j + b) * kStride] = static_cast<uint8_t>(w >> (8 * b));
            }
        }
        if (fk != 1.f && (tok < slot0 || tok >= slot0 + cnt)) {  // the page's other codes: a granule a thread
            uint4 *dst = reinterpret_cast<uint4 *>(ko + tid * 16);
            *dst = requant16(*dst, fk);
        }
        __syncthreads();
        if (lo < hi || fv != 1.f) {
            if (lo >= hi) w = *vo;
            if (fv != 1.f) w = requant16(w, fv);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // bytes lo - 4 j .. hi - 4 j - 1 of the word are new
                const int a = min(max(lo - 4 * j, 0), 4), b = min(max(hi - 4 * j, 0), 4);
                const uint32_t m = b <= a ? 0u : (0xFFFFFFFFu >> (32 - 8 * (b - a))) << (8 * a);
                o[j] = (vt[(d * kStride + s0) / 4 + j] & m) | (u4w(w, j) & ~m);
            }
            *vo = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (tid == 0) {
            c.ks[ph] = sk;
            c.vs[ph] = sv;
        }
    }
}

template <int D, Rot ROT, bool TREE>
cudaError_t launch_one(const AppendParams &p, cudaStream_t st)
{
    const KvParams &c = p.c;
    // pages a sequence's new tokens can touch; a block walks on where max_q was
    // given too small
    const int pages = std::min(std::max(c.max_q, 1) / kPage + 2, c.max_pages);
    LaunchCfg l(dim3(c.max_q <= 1 ? 1 : pages, c.B, c.kv_heads * (p.q ? 2 : 1)), dim3(kPage * D / 16), 0, st);
    return cudaLaunchKernelEx(&l.cfg, moe_kv_append_kernel<D, ROT, TREE>, p);
}

template <int D, bool TREE>
cudaError_t launch_d(const AppendParams &p, cudaStream_t st)
{
    if (p.c.rot_dim == 0) return launch_one<D, kNone, TREE>(p, st);
    if (p.c.rot_inter) return launch_one<D, kNeighbours, TREE>(p, st);
    return p.c.rot_dim % 16 == 0 ? launch_one<D, kHalves, TREE>(p, st) : launch_one<D, kOddHalves, TREE>(p, st);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t st)
{
    if (p.parent) return p.c.D == 128 ? launch_d<128, true>(p, st) : launch_d<64, true>(p, st);
    return p.c.D == 128 ? launch_d<128, false>(p, st) : launch_d<64, false>(p, st);
}

}  // namespace moe
