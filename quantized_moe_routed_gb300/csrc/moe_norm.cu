// moe_norm.cu -- residual addition and root-mean-square norm (moe_norm).
//
//   s = x + r;  y = s / sqrt(mean(s^2) + eps) * w;  r_out = bf16(s)
//   bf16(y) and / or E4M3(y / 2^e) with one power of two for 128 columns
//
// One block per row; a row stays in registers between the sum of squares and
// the output, so every input is read once and every output written once: the
// copy bandwidth bounds it for many rows (8191 rows of 4096, bf16 with a residual,
// both outputs: 54 us, 5.6 TB/s; more or fewer blocks an SM change nothing), the
// launch and one block's chain of load, reduction and store for few (one row: 1.9 us).
#include "moe_internal.h"
#include "moe_layer_internal.h"

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {
namespace {
#include "moe_device.cuh"
#include "moe_layer_device.cuh"

// NV: groups of 8 consecutive elements a thread holds (group i of thread t is
// elements 8 * (i * blockDim + t) ..).
template <int NV, bool X32>
__global__ void __launch_bounds__(512) moe_norm_kernel(const NormParams p)
{
    __shared__ float red[16];
    grid_wait();
    grid_release();
    const int t = blockIdx.x, H = p.H, tid = threadIdx.x;
    const size_t row = static_cast<size_t>(t) * H;
    float s[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * blockDim.x + tid);
        if (c < H) {
            if (X32) {
                const float4 *xp = reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + t * p.x_stride + c);
                const float4 a = xp[0], b = xp[1];
                s[i][0] = a.x, s[i][1] = a.y, s[i][2] = a.z, s[i][3] = a.w;
                s[i][4] = b.x, s[i][5] = b.y, s[i][6] = b.z, s[i][7] = b.w;
            } else {
                const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + t * p.x_stride + c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][2 * j] = bf16_lo(u4w(a, j));
                    s[i][2 * j + 1] = bf16_hi(u4w(a, j));
                }
            }
            if (p.r) {
                const uint4 a = *reinterpret_cast<const uint4 *>(p.r + row + c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][2 * j] += bf16_lo(u4w(a, j));
                    s[i][2 * j + 1] += bf16_hi(u4w(a, j));
                }
            }
            if (p.r_out)
                *reinterpret_cast<uint4 *>(p.r_out + row + c) =
                    make_uint4(pack_bf16(s[i][0], s[i][1]), pack_bf16(s[i][2], s[i][3]), pack_bf16(s[i][4], s[i][5]),
                               pack_bf16(s[i][6], s[i][7]));
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += s[i][j] * s[i][j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] = 0.f;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const int nw = blockDim.x >> 5;
    if ((tid & 31) == 0) red[tid >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < nw; ++i) ss += red[i];
    const float rs = rsqrtf(ss / static_cast<float>(H) + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * blockDim.x + tid);
        const bool in = c < H;
        if (in) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p.w + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][2 * j] = s[i][2 * j] * rs * bf16_lo(u4w(a, j));
                s[i][2 * j + 1] = s[i][2 * j + 1] * rs * bf16_hi(u4w(a, j));
            }
            if (p.y)
                *reinterpret_cast<uint4 *>(p.y + row + c) =
                    make_uint4(pack_bf16(s[i][0], s[i][1]), pack_bf16(s[i][2], s[i][3]), pack_bf16(s[i][4], s[i][5]),
                               pack_bf16(s[i][6], s[i][7]));
        }
        if (p.q) {
            // a block of 128 columns is 16 neighbouring threads (H is a multiple
            // of 128, so a block is inside the row as a whole or not at all)
            float am = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = fabsf(s[i][j]);
                if (a < INFINITY) am = fmaxf(am, a);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            const int e = scale_exp(am);
            const float f = exp2i(-e);
            if (in) {
                uint2 o;
                o.x = e4m3_pack4(s[i][0] * f, s[i][1] * f, s[i][2] * f, s[i][3] * f);
                o.y = e4m3_pack4(s[i][4] * f, s[i][5] * f, s[i][6] * f, s[i][7] * f);
                *reinterpret_cast<uint2 *>(p.q + row + c) = o;
                if ((c & 127) == 0) p.q_scale[(row + c) >> 7] = exp2i(e);
            }
        }
    }
}

template <int NV>
cudaError_t launch_nv(const NormParams &p, int threads, cudaStream_t st)
{
    LaunchCfg l(dim3(p.T), dim3(threads), 0, st);
    return p.x_f32 ? cudaLaunchKernelEx(&l.cfg, moe_norm_kernel<NV, true>, p)
                   : cudaLaunchKernelEx(&l.cfg, moe_norm_kernel<NV, false>, p);
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, cudaStream_t st)
{
    const int groups = p.H / 8;
    // as few groups a thread as 512 threads allow
    const int nv = (groups + 511) / 512;
    const int threads = ((groups + nv - 1) / nv + 31) / 32 * 32;
    if (nv == 1) return launch_nv<1>(p, threads, st);
    if (nv == 2) return launch_nv<2>(p, threads, st);
    if (nv == 3) return launch_nv<3>(p, threads, st);
    return launch_nv<4>(p, threads, st);
}

}  // namespace moe
