// Helpers shared by the kernels of the layers around RMA attention.
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

// ---- powers of two ----
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // |e| <= 126
// the exponent of a scale that brings values of magnitude up to m into [.., 2^top): both it and its
// negative are exponents of normal numbers, whatever m is
__device__ __forceinline__ int scale_of_exponent(int e, int top) { return top - 1 - min(max(e, -110), 127); }
__device__ __forceinline__ int scale_exponent(float m, int top) { return scale_of_exponent(exponent_of(m), top); }

constexpr int kRowTop = 4;   // the largest value of a scaled row (of keys, queries) is below 2^kRowTop

// What a row's values times 2^e have to be multiplied by to be x / sqrt(sum x^2 + eps), `sum` the sum of the scaled
// squares.  One form keeps large rows from overflowing, the other rows far below eps, scaled, from eps = infinity.
__device__ __forceinline__ float scaled_rsqrt(float sum, int e, float eps) {
    const float f = pow2(e), inv = pow2(-e);
    return e <= 0 || (e <= 60 && eps <= 1.f) || eps == 0.f ? 1.f / sqrtf(sum + eps * f * f) : inv / sqrtf(sum * inv * inv + eps);
}

// Whether sum x^2 (+ eps) may be used as it came out of FP32: no square has overflowed, and those that were flushed
// do not count.  A NaN may not.
__device__ __forceinline__ bool plain_sum(float v) { return v > 0x1p-90f && v < 0x1p110f; }

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
