// moe_layer_device.cuh -- device pieces the layer operators share: launches
// that may start while the previous kernel drains, bf16 and E4M3 conversions
// and the power-of-two scale of an 8-bit block.  Included inside
// namespace moe { namespace { ... } }, after moe_device.cuh.
#pragma once

// The kernel may have been launched before the previous one on the stream
// ended: nothing is read or written before this.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel on the stream start its launch (its own wait holds it
// back until this grid has ended).
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two values -> two E4M3 codes (lo in the low byte): nearest, ties to even,
// saturating at 448, NaN to the NaN code.
__device__ __forceinline__ uint32_t e4m3_pack2(float lo, float hi)
{
    uint32_t r;
    asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n cvt.u32.u16 %0, t;\n}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d)
{
    return e4m3_pack2(a, b) | (e4m3_pack2(c, d) << 16);
}
// Four E4M3 codes -> four values.
__device__ __forceinline__ float4 e4m3_unpack4(uint32_t w)
{
    const uint32_t l = e4m3x2_to_f16x2(static_cast<uint16_t>(w)), h = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&l));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return make_float4(a.x, a.y, b.x, b.y);
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

// Exponent e of the smallest power of two with a <= 448 * 2^e, at least -64
// (a >= 0, finite).  448 = 1.75 * 2^8, so with a = m * 2^E it is E - 8, or
// E - 7 where m > 1.75.
__device__ __forceinline__ int scale_exp(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
    return max(-64, e);  // a subnormal or zero a lands here too
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One lane of a converged warp, the same every time.  A warp that stays together
// and elects the lane that issues keeps descriptors and addresses in uniform
// registers; a branch on the lane's number costs a move a product and operand.
__device__ __forceinline__ bool elect_one()
{
    uint32_t is;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(is));
    return is != 0;
}

// Launch configuration shared by the operators: programmatic dependent launch
// (every kernel calls grid_wait before its first access).
struct LaunchCfg {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    LaunchCfg(dim3 grid, dim3 block, size_t smem, cudaStream_t st)
    {
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};
