// rows.cuh -- what the kernels on rows of values share: eight values as they lie
// in memory and in F32, and a launch whose blocks may start before the grid in
// front of them ends (each kernel waits for it before it reads).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace splitk {

constexpr int kVec = 8;   // values a thread takes at once

template <typename T>
struct Pack;   // kVec values as they lie in memory
template <>
struct Pack<float> {
    float4 a, b;
};
template <>
struct Pack<__half> {
    uint4 a;
};
template <>
struct Pack<__nv_bfloat16> {
    uint4 a;
};

__device__ __forceinline__ void unpack(const Pack<float> &p, float (&v)[kVec])
{
    v[0] = p.a.x, v[1] = p.a.y, v[2] = p.a.z, v[3] = p.a.w;
    v[4] = p.b.x, v[5] = p.b.y, v[6] = p.b.z, v[7] = p.b.w;
}
__device__ __forceinline__ void pack(const float (&v)[kVec], Pack<float> &p)
{
    p.a = make_float4(v[0], v[1], v[2], v[3]);
    p.b = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void unpack(const Pack<__half> &p, float (&v)[kVec])
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&p.a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void pack(const float (&v)[kVec], Pack<__half> &p)
{
    __half2 *h = reinterpret_cast<__half2 *>(&p.a);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16> &p, float (&v)[kVec])
{
    // a BF16 is the upper half of its F32
    const uint32_t u[4] = {p.a.x, p.a.y, p.a.z, p.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}
__device__ __forceinline__ void pack(const float (&v)[kVec], Pack<__nv_bfloat16> &p)
{
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&p.a);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
}

inline cudaLaunchConfig_t config(unsigned grid, unsigned block, cudaStream_t stream, cudaLaunchAttribute *attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace splitk
