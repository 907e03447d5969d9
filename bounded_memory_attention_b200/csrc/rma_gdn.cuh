// Device helpers shared by the gated-delta-rule kernels.
#pragma once

#include <cuda_bf16.h>

#include "rma_internal.cuh"

namespace rma {

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
    const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&v);
    return __bfloat1622float2(h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Tokens of sequence b, clamped to [0, n]; `report`: this thread sets the status bit.
__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int n, uint32_t* status, bool report) {
    if (!lens) return n;
    const int len = lens[b];
    if (report && (len < 0 || len > n)) atomicOr(status, (unsigned)RMA_STATUS_BAD_LENGTH);
    return min(max(len, 0), n);
}

// g = -alpha softplus(a + dt) and beta = sigmoid(b), alpha = exp(a_log).  g is held at -128 or above:
// exp(-128) is 0 in FP32 already, and the chunked form takes differences of sums of g, which an
// infinity would make NaN.  A NaN stays one.
__device__ __forceinline__ void gates(uint16_t a, uint16_t b, float alpha, float dt, float& g, float& beta) {
    const float z = bf16_float(a) + dt;
    const float sp = fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
    const float x = -alpha * sp;
    g = x < -128.f ? -128.f : x;
    beta = 1.f / (1.f + expf(-bf16_float(b)));
}

// A launch that may be scheduled while the kernel before it on the stream finishes (its kernels
// wait with griddepcontrol.wait before they touch global memory).
struct PdlLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    PdlLaunch(unsigned grid, unsigned threads, size_t smem, cudaStream_t stream) {
        cfg.gridDim = dim3(grid, 1, 1);
        cfg.blockDim = dim3(threads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    PdlLaunch(const PdlLaunch&) = delete;
    PdlLaunch& operator=(const PdlLaunch&) = delete;
};

}  // namespace rma
