// moe_linear.cu -- matrix-vector products with NVFP4 weights (moe_linear).
//
//   y[t, n] = ts[n] * sum_k E2M1(q[n, k]) * E4M3(s[n, k/16]) * x[t, k]
//
// The weights are read once for up to 24 tokens, so their bytes bound it.
// They go from global memory to registers (16 bytes a lane, the next chunk's
// loads in flight while this one is used), become fp16 there (E2M1 times E4M3
// is exact in fp16) and are the A operand of mma.sync m16n8k16; tokens are the
// N axis.  A block computes 16 * MT rows, its 8 warps take every eighth chunk
// of 128 elements of K, and the block adds their sums in warp order.
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

#include <cstdint>

namespace moe {
namespace {
#include "moe_device.cuh"
#include "moe_layer_device.cuh"

constexpr int kWarps = 8;
constexpr int kChunk = 128;  // elements of K a warp takes at a time

template <int MT>
struct WChunk {
    uint4 q[MT][2];     // rows g and g + 8 of each 16-row tile: 32 codes
    uint16_t s[MT][2];  // their two block scales
};

template <int MT>
__device__ __forceinline__ void load_chunk(WChunk<MT> &w, const LinearParams &p, int row0, int g, int k)
{
    const bool in = k < p.K;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = min(row0 + 16 * m + 8 * h + g, p.N - 1);
            w.q[m][h] = make_uint4(0u, 0u, 0u, 0u);
            w.s[m][h] = 0;
            if (in) {
                w.q[m][h] = __ldcs(reinterpret_cast<const uint4 *>(p.q + static_cast<size_t>(r) * (p.K / 2) + k / 2));
                w.s[m][h] = __ldg(reinterpret_cast<const uint16_t *>(p.s + static_cast<size_t>(r) * (p.K / 16) + k / 16));
            }
        }
}

template <int MT, int NT>
__global__ void __launch_bounds__(kWarps * 32) moe_linear_kernel(const LinearParams p)
{
    __shared__ float red[kWarps][NT * 8][16 * MT + 1];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int row0 = blockIdx.x * 16 * MT, tok0 = blockIdx.y * kLinearMaxT;
    const int T = min(p.T - tok0, kLinearMaxT);
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

    WChunk<MT> w, wn;
    int k = wid * kChunk + 32 * t4;
    load_chunk<MT>(w, p, row0, g, k);
    for (int c = wid * kChunk; c < p.K; c += kWarps * kChunk, k += kWarps * kChunk) {
        // x of this chunk: the lane's 32 elements of token g of each 8-token tile
        uint32_t xb[NT][16];
        float back[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint4 a[4];
            const int tok = n * 8 + g;
            const bool in = tok < T && k < p.K;
            const uint4 *xp = reinterpret_cast<const uint4 *>(p.x + static_cast<long long>(tok0 + tok) * p.x_stride + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = in ? __ldg(xp + i) : make_uint4(0u, 0u, 0u, 0u);
            uint32_t am = 0u;  // largest magnitude, as bits (16-bit halves)
#pragma unroll
            for (int i = 0; i < 16; ++i) am = __vmaxu2(am, u4w(a[i >> 2], i & 3) & 0x7FFF7FFFu);
            am = max(am >> 16, am & 0xFFFFu);
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const int e = min(126, f16_prescale_exp(__uint_as_float(am << 16)));
            const float f = exp2i(e);
#pragma unroll
            for (int i = 0; i < 16; ++i) xb[n][i] = bf16x2_to_f16x2_scaled(u4w(a[i >> 2], i & 3), f);
            // the accumulator's columns are tokens 2 t4 and 2 t4 + 1
            back[n][0] = exp2i(-__shfl_sync(0xffffffffu, e, 8 * t4));
            back[n][1] = exp2i(-__shfl_sync(0xffffffffu, e, 8 * t4 + 4));
        }
        load_chunk<MT>(wn, p, row0, g, k + kWarps * kChunk);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[n][i] = 0.f;
            const uint32_t s0 = e4m3x2_to_f16x2(w.s[m][0]), s1 = e4m3x2_to_f16x2(w.s[m][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 8 elements of each row: two K steps
                uint32_t a0[4], a1[4];
                e2m1x8_to_f16x2(u4w(w.q[m][0], i), a0[0], a0[1], a0[2], a0[3]);
                e2m1x8_to_f16x2(u4w(w.q[m][1], i), a1[0], a1[1], a1[2], a1[3]);
                const uint32_t sel = i < 2 ? 0x1010u : 0x3232u;
                const uint32_t f0 = __byte_perm(s0, 0u, sel), f1 = __byte_perm(s1, 0u, sel);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a0[j] = hmul2(a0[j], f0);
                    a1[j] = hmul2(a1[j], f1);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816(d[n], a0[0], a1[0], a0[1], a1[1], xb[n][4 * i], xb[n][4 * i + 1]);
                    mma16816(d[n], a0[2], a1[2], a0[3], a1[3], xb[n][4 * i + 2], xb[n][4 * i + 3]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[m][n][0] += d[n][0] * back[n][0];
                acc[m][n][1] += d[n][1] * back[n][1];
                acc[m][n][2] += d[n][2] * back[n][0];
                acc[m][n][3] += d[n][3] * back[n][1];
            }
        }
        w = wn;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[wid][n * 8 + 2 * t4 + (i & 1)][16 * m + g + 8 * (i >> 1)] = acc[m][n][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * 16 * MT; i += kWarps * 32) {
        const int r = i % (16 * MT), tok = i / (16 * MT);
        if (tok >= T || row0 + r >= p.N) continue;
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) v += red[u][tok][r];
        v *= p.ts[row0 + r];
        const size_t o = static_cast<size_t>(tok0 + tok) * p.N + row0 + r;
        if (p.y_bf16)
            static_cast<uint16_t *>(p.y)[o] = static_cast<uint16_t>(pack_bf16(v, 0.f));
        else
            static_cast<float *>(p.y)[o] = v;
    }
}

template <int MT, int NT>
cudaError_t launch_mn(const LinearParams &p, cudaStream_t st)
{
    LaunchCfg l(dim3((p.N + 16 * MT - 1) / (16 * MT), (p.T + kLinearMaxT - 1) / kLinearMaxT), dim3(kWarps * 32), 0, st);
    return cudaLaunchKernelEx(&l.cfg, moe_linear_kernel<MT, NT>, p);
}

}  // namespace

cudaError_t launch_linear(const LinearParams &p, int num_sms, cudaStream_t st)
{
    const int nt = p.T <= 8 ? 1 : (p.T <= 16 ? 2 : 3);
    // taller blocks share the conversion of x among more rows; short ones give
    // every SM a block where there are few rows
    const bool tall = p.N >= 64 * 2 * num_sms;
    if (nt == 1) return tall ? launch_mn<2, 1>(p, st) : launch_mn<1, 1>(p, st);
    if (nt == 2) return tall ? launch_mn<4, 2>(p, st) : launch_mn<1, 2>(p, st);
    return tall ? launch_mn<2, 3>(p, st) : launch_mn<1, 3>(p, st);
}

}  // namespace moe
