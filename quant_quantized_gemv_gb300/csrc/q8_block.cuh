// q8_block.cuh -- the quantization of 32-value blocks that every q8 plane is
// written with (producers.cu states the formula and its source).
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace mq {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int q8_code(float v, float di)
{
    int q = __float2int_rn(v * di);  // round half to even, like rintf
    return max(-128, min(127, q));
}

// Quantize 4 values held by this lane; 8 lanes (aligned group) form a block.
// gid = global index of this lane's 4-value group (block = gid / 8).
__device__ __forceinline__ void quantize4(float4 v, bool valid, long long gid, uint8_t *q8,
                                          unsigned d_off, unsigned sum_off)
{
    float am = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
    am = fmaxf(am, __shfl_xor_sync(kFull, am, 1));
    am = fmaxf(am, __shfl_xor_sync(kFull, am, 2));
    am = fmaxf(am, __shfl_xor_sync(kFull, am, 4));
    const float d = am / 127.0f;
    const float di = (d != 0.0f) ? 1.0f / d : 0.0f;
    const int q0 = q8_code(v.x, di), q1 = q8_code(v.y, di);
    const int q2 = q8_code(v.z, di), q3 = q8_code(v.w, di);
    int s = q0 + q1 + q2 + q3;
    s += __shfl_xor_sync(kFull, s, 1);
    s += __shfl_xor_sync(kFull, s, 2);
    s += __shfl_xor_sync(kFull, s, 4);
    if (!valid) return;
    const uint32_t packed = (uint32_t)(q0 & 0xff) | ((uint32_t)(q1 & 0xff) << 8) |
                            ((uint32_t)(q2 & 0xff) << 16) | ((uint32_t)(q3 & 0xff) << 24);
    reinterpret_cast<uint32_t *>(q8)[gid] = packed;
    if ((gid & 7) == 0) {
        const long long b = gid >> 3;
        reinterpret_cast<__half *>(q8 + d_off)[b] = __float2half_rn(d);
        reinterpret_cast<int *>(q8 + sum_off)[b] = s;
    }
}

}  // namespace
}  // namespace mq
