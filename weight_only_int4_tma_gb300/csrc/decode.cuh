// Shared pieces of the decoder-layer kernels (norm.cu, rope.cu, attn.cu): 16-bit value
// conversions, reductions and the programmatic dependent launch.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "launch_math.h"
#include "ptx.cuh"

namespace w4g {

constexpr int kDecInvalidArg = -1;  // w4a16_status W4A16_ERR_INVALID_ARG

// DT: 0 fp16, 1 bf16.
template <int DT>
__device__ __forceinline__ float dec_to_f32(uint16_t b) {
    if constexpr (DT == 0) return __half2float(__ushort_as_half(b));
    else return __bfloat162float(__ushort_as_bfloat16(b));
}
template <int DT>
__device__ __forceinline__ uint16_t dec_from_f32(float v) {
    if constexpr (DT == 0) return __half_as_ushort(__float2half_rn(v));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Two values rounded and packed, lo in the low half.
template <int DT>
__device__ __forceinline__ uint32_t dec_pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (DT == 0) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 values to E4M3, round to nearest even, saturated to +-448 (lo in the low byte).
__device__ __forceinline__ uint32_t dec_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two E4M3 values (low 16 bits) to an fp16 pair, exact.
__device__ __forceinline__ uint32_t dec_e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// Launch that may begin while the stream's previous kernel still runs (every kernel here
// calls grid_dep_wait() before its first access to memory).  Returns a w4a16_status.
template <typename... KArgs, typename... Args>
int launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                     cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) == cudaSuccess ? 0 : -3;
}

}  // namespace w4g
