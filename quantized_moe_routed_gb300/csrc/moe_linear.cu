// moe_linear.cu -- matrix-vector products with NVFP4 weights (moe_linear).
//
//   y[t, n] = ts[n] * sum_k E2M1(q[n, k]) * E4M3(s[n, k/16]) * x[t, k]
//
// The weights are read once for up to 24 tokens, so their bytes bound it.  (Weights
// of many rows: moe_linear_tc.cu.)
// They go from global memory to registers (16 bytes a lane, the next loads in
// flight while these are used), become fp16 there (E2M1 times E4M3 is exact in
// fp16) and are the A operand of mma.sync m16n8k16; tokens are the N axis.
//
// One block per SM owns an equal run of the 16-row tiles and keeps the sums of
// up to 32 of them in registers, so that x passes by once per run: a piece of
// K at a time, in shared memory, shared by the block's 16 warps.  With few
// tiles, KW warps share one and take its 128-element chunks of K in turn, their
// sums added in warp order at the end.  (Clusters that split K, their sums added
// through distributed shared memory, measured slower at every size: 8.1 against
// 5.0 us for one token and 2432 rows.)
//
// K is permuted inside a chunk so that a lane's operands are contiguous in
// memory: lane (g, t) of the MMA holds elements 32 t .. 32 t + 31 of rows g and
// g + 8 (and of token g), four in each of the chunk's eight K steps.
//
// x enters as fp16 after a power-of-two prescale of each (token, chunk), taken
// from the largest of the chunk's 128 elements and undone in the fp32
// accumulation: no bf16 value leaves fp16's range, and none loses bits that
// count beside its chunk's largest.
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

constexpr int kWarps = 16;
constexpr int kChunk = 128;  // elements of K a warp takes at a time
constexpr int kMaxMT = 2;    // tiles a warp keeps

struct Shape {
    int KW;       // warps that share a tile
    int tiles;    // 16-row tiles of a block in one pass
    int passes;   // passes of a block over K
    int piece;    // chunks of K in shared memory at a time
    int buffers;  // pieces in shared memory: 1 if that is all of K
    int tshift;   // up to 16 tokens: their number is at most 2^tshift
};

template <int MT>
struct WChunk {
    uint4 q[MT][2];     // rows g and g + 8 of each tile: 32 codes
    uint16_t s[MT][2];  // their two block scales
};

// A lane's place in the weights: byte offsets of its two rows of each tile from
// the pass's first row (a row's scales are an eighth of its codes).
template <int MT>
struct WRows {
    const uint8_t *q, *s;
    uint32_t at[MT][2];
};

template <int MT>
__device__ __forceinline__ void load_chunk(WChunk<MT> &w, const WRows<MT> &r, int tiles, int k, int K)
{
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w.q[m][h] = make_uint4(0u, 0u, 0u, 0u);
            w.s[m][h] = 0;
            if (m < tiles && k < K) {
                const uint32_t o = r.at[m][h] + k / 2;
                w.q[m][h] = __ldcs(reinterpret_cast<const uint4 *>(r.q + o));
                w.s[m][h] = __ldg(reinterpret_cast<const uint16_t *>(r.s + o / 8));
            }
        }
}

// D = A B (+ D unless it is the first): the accumulator starts without a move.
template <bool FIRST>
__device__ __forceinline__ void mma_to(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1)
{
    if (FIRST)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        mma16816(d, a0, a1, a2, a3, b0, b1);
}

// The products of one chunk of M tiles with the tokens' chunk at xs, added to acc
// with the tokens' factors (columns are tokens 2 t4 and 2 t4 + 1).
template <int M, int MT, int NT>
__device__ __forceinline__ void use_chunk(float (&acc)[MT][NT][4], const WChunk<MT> &w, const uint8_t *xs, const float *bk)
{
    float d[M][NT][4];
    uint32_t sc[M][2];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        sc[m][0] = e4m3x2_to_f16x2(w.s[m][0]);
        sc[m][1] = e4m3x2_to_f16x2(w.s[m][1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 8 elements of each row: two K steps
        uint32_t a[M][2][4];
        const uint32_t sel = i < 2 ? 0x1010u : 0x3232u;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                e2m1x8_to_f16x2(u4w(w.q[m][h], i), a[m][h][0], a[m][h][1], a[m][h][2], a[m][h][3]);
                const uint32_t f = __byte_perm(sc[m][h], 0u, sel);
#pragma unroll
                for (int j = 0; j < 4; ++j) a[m][h][j] = hmul2(a[m][h][j], f);
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 b = *reinterpret_cast<const uint4 *>(xs + (n * 4 + i) * 512);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (i == 0)
                    mma_to<true>(d[m][n], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b.x, b.y);
                else
                    mma_to<false>(d[m][n], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b.x, b.y);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) mma_to<false>(d[m][n], a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], b.z, b.w);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float2 f = *reinterpret_cast<const float2 *>(bk + n * 8);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            acc[m][n][0] += d[m][n][0] * f.x;
            acc[m][n][1] += d[m][n][1] * f.y;
            acc[m][n][2] += d[m][n][2] * f.x;
            acc[m][n][3] += d[m][n][3] * f.y;
        }
    }
}

// x in shared memory is the MMA's B operand, [chunk][8 tokens][16 bytes i][lane
// (token, quarter)], with the factors that undo the prescales.  Sixteen threads
// bring a (chunk, token), elements 8 h .. 8 h + 7 each: item i of a piece is token
// i % TP of its chunk i / TP.  Places of tokens past the last one are left as
// they are: the products' columns are independent, and theirs are never written out.
struct XPlace {
    int TP, shift;  // tokens of a chunk's items: 24, or a power of two (its shift)
    __device__ __forceinline__ int chunk(int i) const { return TP == 24 ? i / 24 : i >> shift; }
    __device__ __forceinline__ int token(int i) const { return TP == 24 ? i % 24 : i & (TP - 1); }
};
__device__ __forceinline__ uint4 load_x(const LinearParams &p, const XPlace &xp, int tok0, int T, int c0, int i, int items)
{
    const int tok = xp.token(i), k = (c0 + xp.chunk(i)) * kChunk + 8 * (threadIdx.x & 15);
    if (i >= items || tok >= T || k >= p.K) return make_uint4(0u, 0u, 0u, 0u);
    return __ldg(reinterpret_cast<const uint4 *>(p.x + static_cast<long long>(tok0 + tok) * p.x_stride + k));
}
template <int NT>
__device__ __forceinline__ void store_x(uint4 a, const XPlace &xp, uint8_t *xs, float *back, int i, int items)
{
    const int h = threadIdx.x & 15, tok = xp.token(i), slot = xp.chunk(i);
    uint32_t am = 0u;  // largest magnitude, as bits (16-bit halves)
#pragma unroll
    for (int j = 0; j < 4; ++j) am = __vmaxu2(am, u4w(a, j) & 0x7FFF7FFFu);
    am = max(am >> 16, am & 0xFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (i >= items) return;
    const int e = min(126, f16_prescale_exp(__uint_as_float(am << 16)));
    const float f = exp2i(e);
    *reinterpret_cast<uint4 *>(xs + ((slot * NT + tok / 8) * 4 + h % 4) * 512 + ((tok % 8) * 4 + h / 4) * 16) =
        make_uint4(bf16x2_to_f16x2_scaled(a.x, f), bf16x2_to_f16x2_scaled(a.y, f), bf16x2_to_f16x2_scaled(a.z, f),
                   bf16x2_to_f16x2_scaled(a.w, f));
    if (h == 0) back[slot * NT * 8 + tok] = exp2i(-e);
}

__device__ __forceinline__ void put_output(const LinearParams &p, float v, int n, int tok)
{
    const size_t o = static_cast<size_t>(tok) * p.N + n;
    if (p.y_bf16)
        static_cast<uint16_t *>(p.y)[o] = static_cast<uint16_t>(pack_bf16(v, 0.f));
    else
        static_cast<float *>(p.y)[o] = v;
}

// Few tiles: a block a tile, its warps take the chunks of K in turn.  A warp
// converts its own chunks of x on the way from global memory, which no other
// warp needs: nothing is staged, and the block meets once, for the sums.
template <int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 2 : 1) moe_linear_few_kernel(const LinearParams p)
{
    __shared__ float red[kWarps][NT * 8][17];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int row0 = blockIdx.x * 16, tok0 = blockIdx.y * kLinearMaxT, T = min(p.T - tok0, kLinearMaxT);
    const int r = threadIdx.x & 15, tok = threadIdx.x >> 4;  // of the outputs
    const float ts = row0 + r < p.N ? p.ts[row0 + r] : 0.f;
    float acc[1][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[0][n][i] = 0.f;
    WRows<1> at{p.q + static_cast<size_t>(row0) * (p.K / 2), p.s + static_cast<size_t>(row0) * (p.K / 16), {}};
#pragma unroll
    for (int h = 0; h < 2; ++h) at.at[0][h] = static_cast<uint32_t>(min(8 * h + g, p.N - 1 - row0)) * (p.K / 2);
    WChunk<1> w, wn;
    int k = wid * kChunk + 32 * t4;
    load_chunk<1>(w, at, 1, k, p.K);
    for (int c = wid * kChunk; c < p.K; c += kWarps * kChunk, k += kWarps * kChunk) {
        uint4 a[NT][4];  // the lane's 32 elements of token g of each 8
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool in = n * 8 + g < T && k < p.K;
            const uint4 *xp = reinterpret_cast<const uint4 *>(p.x + static_cast<long long>(tok0 + n * 8 + g) * p.x_stride + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[n][i] = in ? __ldg(xp + i) : make_uint4(0u, 0u, 0u, 0u);
        }
        load_chunk<1>(wn, at, 1, k + kWarps * kChunk, p.K);
        uint32_t sc[2] = {e4m3x2_to_f16x2(w.s[0][0]), e4m3x2_to_f16x2(w.s[0][1])};
        float f[NT], back[NT][2], d[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t am = 0u;  // largest magnitude, as bits (16-bit halves)
#pragma unroll
            for (int i = 0; i < 16; ++i) am = __vmaxu2(am, u4w(a[n][i >> 2], i & 3) & 0x7FFF7FFFu);
            am = max(am >> 16, am & 0xFFFFu);
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const int e = min(126, f16_prescale_exp(__uint_as_float(am << 16)));
            f[n] = exp2i(e);
            // the accumulator's columns are tokens 2 t4 and 2 t4 + 1
            back[n][0] = exp2i(-__shfl_sync(0xffffffffu, e, 8 * t4));
            back[n][1] = exp2i(-__shfl_sync(0xffffffffu, e, 8 * t4 + 4));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 elements of each row: two K steps
            uint32_t b[2][4];
            const uint32_t sel = i < 2 ? 0x1010u : 0x3232u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                e2m1x8_to_f16x2(u4w(w.q[0][h], i), b[h][0], b[h][1], b[h][2], b[h][3]);
                const uint32_t s = __byte_perm(sc[h], 0u, sel);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[h][j] = hmul2(b[h][j], s);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = bf16x2_to_f16x2_scaled(u4w(a[n][i], j), f[n]);
                if (i == 0)
                    mma_to<true>(d[n], b[0][0], b[1][0], b[0][1], b[1][1], x[0], x[1]);
                else
                    mma_to<false>(d[n], b[0][0], b[1][0], b[0][1], b[1][1], x[0], x[1]);
                mma_to<false>(d[n], b[0][2], b[1][2], b[0][3], b[1][3], x[2], x[3]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][n][i] += d[n][i] * back[n][i & 1];
        w = wn;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wid][n * 8 + 2 * t4 + (i & 1)][g + 8 * (i >> 1)] = acc[0][n][i];
    __syncthreads();
    if (tok < T && row0 + r < p.N) {
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) v += red[u][tok][r];
        put_output(p, v * ts, row0 + r, tok0 + tok);
    }
}

// PF: chunks whose loads are in flight beside the one in use.
template <int MT, int NT, int PF>
__global__ void __launch_bounds__(kWarps * 32, 1) moe_linear_kernel(const LinearParams p, const Shape sh)
{
    extern __shared__ uint8_t smem[];  // [buffers][piece] chunks of x, their factors; then the warps' sums
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int tok0 = blockIdx.y * kLinearMaxT, T = min(p.T - tok0, kLinearMaxT);
    const int rw = wid / sh.KW, kw = wid % sh.KW, RW = kWarps / sh.KW;
    const int all_tiles = (p.N + 15) / 16, chunks = (p.K + kChunk - 1) / kChunk;
    const int xbytes = sh.piece * NT * 2048;
    const XPlace xp{NT == 3 ? 24 : 1 << sh.tshift, sh.tshift};
    float *back = reinterpret_cast<float *>(smem + sh.buffers * xbytes);
    grid_wait();
    grid_release();
    for (int pass = 0; pass < sh.passes; ++pass) {
        const int tile0 = (blockIdx.x * sh.passes + pass) * sh.tiles;
        if (tile0 >= all_tiles) return;
        // this warp's tiles: rw, rw + RW, .. of the pass
        const int mine = min(sh.tiles, all_tiles - tile0), tiles = mine <= rw ? 0 : min(MT, (mine - rw + RW - 1) / RW);
        const size_t first_row = 16 * static_cast<size_t>(tile0);
        WRows<MT> at{p.q + first_row * (p.K / 2), p.s + first_row * (p.K / 16), {}};
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                at.at[m][h] = static_cast<uint32_t>(min(16 * (rw + m * RW) + 8 * h + g, p.N - 1 - 16 * tile0)) * (p.K / 2);
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        // rounds: every warp takes a chunk; round j's weights are in w[j % R]
        constexpr int R = PF + 1;
        const int rounds = (chunks + sh.KW - 1) / sh.KW, per_piece = sh.piece / sh.KW;
        WChunk<MT> w[R];
        auto load = [&](WChunk<MT> &to, int j) {
            const int c = kw + j * sh.KW;
            load_chunk<MT>(to, at, c < chunks ? tiles : 0, c * kChunk + 32 * t4, p.K);
        };
        const int hw = threadIdx.x >> 4, items = sh.piece * xp.TP;
        const int my_items = (items + 2 * kWarps - 1) / (2 * kWarps);
        auto stage = [&](int c0, int buf) {
            constexpr int S = MT == 1 ? 8 : 4;
            for (int i = hw; i < my_items * 2 * kWarps; i += S * 2 * kWarps) {
                uint4 a[S];
#pragma unroll
                for (int v = 0; v < S; ++v) a[v] = load_x(p, xp, tok0, T, c0, i + v * 2 * kWarps, items);
#pragma unroll
                for (int v = 0; v < S; ++v)
                    if (i - hw + v * 2 * kWarps < items)
                        store_x<NT>(a[v], xp, smem + buf * xbytes, back + buf * sh.piece * NT * 8, i + v * 2 * kWarps, items);
            }
        };
        if (pass == 0 || sh.buffers > 1) {  // (all of K in one piece: it is there from the first pass)
            if (pass > 0) __syncthreads();
            stage(0, 0);
        }
        // a thread has one row of the outputs and every step-th token
        const int nrows = sh.tiles * 16, step = max(kWarps * 32 / nrows, 1);
        const int r = threadIdx.x % nrows, first = threadIdx.x / nrows, n = 16 * tile0 + r;
        const float ts = first < step && n < p.N ? p.ts[n] : 0.f;
#pragma unroll
        for (int i = 0; i < PF; ++i) load(w[i], i);
        int left = 0, buf = 1;  // rounds to the next piece; the piece in use
        for (int j0 = 0; j0 < rounds; j0 += R) {
#pragma unroll
            for (int v = 0; v < R; ++v) {
                const int j = j0 + v;
                if (j >= rounds) break;
                if (left == 0) {
                    // the piece in the other buffer is staged and this one's readers are done
                    __syncthreads();
                    buf ^= 1;
                    left = per_piece;
                    if (MT == 1 && j + per_piece < rounds) stage((j + per_piece) * sh.KW, buf ^ 1);
                }
                // many tiles: an item of the next piece a round, its load in flight
                // during the products (a piece has at least as many rounds as items)
                const int xc = (j + left) * sh.KW, xi = hw + (per_piece - left) * 2 * kWarps;
                const bool more = MT > 1 && j + left < rounds && per_piece - left < my_items;
                uint4 xa;
                if (more) xa = load_x(p, xp, tok0, T, xc, xi, items);
                const int c = kw + j * sh.KW, slot = kw + (per_piece - left) * sh.KW;  // chunk of the run, of the piece
                --left;
                load(w[(v + PF) % R], j + PF);
                if (c < chunks) {
                    const uint8_t *xs = smem + buf * xbytes + slot * NT * 2048 + lane * 16;
                    const float *bk = back + (buf * sh.piece + slot) * NT * 8 + 2 * t4;
                    if (tiles == MT)
                        use_chunk<MT, MT, NT>(acc, w[v], xs, bk);
                    else if (tiles > 0)
                        use_chunk<1, MT, NT>(acc, w[v], xs, bk);
                }
                if (more) store_x<NT>(xa, xp, smem + (buf ^ 1) * xbytes, back + (buf ^ 1) * sh.piece * NT * 8, xi, items);
            }
        }
        // sums of the KW warps of a tile, and out
        const bool last = pass + 1 == sh.passes;
        float *red = reinterpret_cast<float *>(smem + (last ? 0 : sh.buffers * (xbytes + sh.piece * NT * 32)));
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[((m * kWarps + wid) * NT * 8 + n * 8 + 2 * t4 + (i & 1)) * 17 + g + 8 * (i >> 1)] = acc[m][n][i];
        __syncthreads();
        auto warp_sum = [&](int r, int tok) {
            const float *a = red + (((r / 16 / RW) * kWarps + (r / 16 % RW) * sh.KW) * NT * 8 + tok) * 17 + r % 16;
            float v = 0.f;
            for (int u = 0; u < sh.KW; ++u) v += a[u * NT * 8 * 17];
            return v;
        };
        if (first < step && n < p.N)
            for (int tok = first; tok < T; tok += step) put_output(p, warp_sum(r, tok) * ts, n, tok0 + tok);
    }
}

template <int MT, int NT>
cudaError_t launch_mn(const LinearParams &p, const Shape &sh, int blocks, cudaStream_t st)
{
    const int x = sh.buffers * sh.piece * (NT * 2048 + NT * 32);
    const int red = MT * kWarps * NT * 8 * 17 * 4;
    const int smem = sh.passes > 1 ? x + red : std::max(x, red);
    auto *fn = moe_linear_kernel<MT, NT, MT == 2 ? 1 : (NT == 1 ? 3 : 2)>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchCfg l(dim3(blocks, (p.T + kLinearMaxT - 1) / kLinearMaxT), dim3(kWarps * 32), smem, st);
    return cudaLaunchKernelEx(&l.cfg, fn, p, sh);
}

}  // namespace

cudaError_t launch_linear(const LinearParams &p, int num_sms, cudaStream_t st)
{
    const int nt = p.T <= 8 ? 1 : (p.T <= 16 ? 2 : 3);
    const int all = (p.N + 15) / 16, chunks = (p.K + kChunk - 1) / kChunk;
    Shape sh{};
    const int share = (all + num_sms - 1) / num_sms;  // tiles of a block
    // a block a tile while they are few; its own conversion of x, which every tile
    // repeats, costs more than staging x for many.  Measured at K = 4096, few
    // against staged: one token, 2 tiles an SM 6.2 / 7.7 us, 3 tiles 8.0 / 8.9, 4
    // tiles 13.2 / 10.5; 24 tokens, 1 tile 8.1 / 14.1, 2 tiles 15.1 / 16.4, 3 tiles 20.6 / 18.1
    if (share <= (nt == 1 ? 3 : 2)) {
        LaunchCfg l(dim3(all, (p.T + kLinearMaxT - 1) / kLinearMaxT), dim3(kWarps * 32), 0, st);
        auto *fn = nt == 1 ? moe_linear_few_kernel<1> : (nt == 2 ? moe_linear_few_kernel<2> : moe_linear_few_kernel<3>);
        return cudaLaunchKernelEx(&l.cfg, fn, p);
    }
    sh.passes = (share + kWarps * kMaxMT - 1) / (kWarps * kMaxMT);
    sh.tiles = (share + sh.passes - 1) / sh.passes;
    while (sh.tshift < 4 && (1 << sh.tshift) < std::min(p.T, kLinearMaxT)) ++sh.tshift;
    // x: all of K where it fits (200 KB, beside the sums of a further pass or two tiles a
    // warp 64 KB), else two pieces of 16 chunks (8 for 24 tokens and two tiles a warp)
    const bool one = sh.tiles <= kWarps && sh.passes == 1;
    const bool whole = chunks * nt * (2048 + 32) <= (one ? 200 : 64) * 1024;
    const int piece = nt == 3 && !one ? 8 : 16, most = std::min(chunks, whole ? kWarps : piece);
    sh.KW = 1;
    while (sh.tiles * sh.KW * 2 <= kWarps && sh.KW * 2 <= most) sh.KW *= 2;
    sh.piece = whole ? (chunks + sh.KW - 1) / sh.KW * sh.KW : piece;
    sh.buffers = whole ? 1 : 2;
    const int blocks = (all + sh.tiles * sh.passes - 1) / (sh.tiles * sh.passes);
    const bool two = sh.tiles > kWarps / sh.KW;
    if (nt == 1) return two ? launch_mn<2, 1>(p, sh, blocks, st) : launch_mn<1, 1>(p, sh, blocks, st);
    if (nt == 2) return two ? launch_mn<2, 2>(p, sh, blocks, st) : launch_mn<1, 2>(p, sh, blocks, st);
    return two ? launch_mn<2, 3>(p, sh, blocks, st) : launch_mn<1, 3>(p, sh, blocks, st);
}

}  // namespace moe
