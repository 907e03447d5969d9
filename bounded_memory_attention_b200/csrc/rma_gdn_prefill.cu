// rma_gdn_prefill: the gated delta rule over a block of tokens, in chunks of 64 on the tensor cores.
//
// Within a chunk that starts from state S0 (key x value), with G_i the sum of the log decays g up to
// token i, k, q normalised and u_i = beta_i (v_i - S_{i-1}^T k_i e^{g_i}) the recurrence's updates:
//   (1 + A) U = diag(beta) (V - diag(e^G) K S0),  A_ij = beta_i e^{G_i - G_j} (k_i . k_j), j < i;
//   O  = scale (diag(e^G) Q S0 + P U),            P_ij = e^{G_i - G_j} (q_i . k_j), j <= i;
//   S1 = e^{G_C} S0 + sum_j e^{G_C - G_j} k_j u_j^T.
// With T = (1 + A)^-1 diag(beta), U = T (V - diag(e^G) K S0).
//
// Two launches.
//
// 1. gdn_prep_kernel, a CTA per (chunk, sequence, key head): everything that does not depend on the
//    state.  Norms of q and k; K K^T and Q K^T once per key head; per value head of it the decays, T
//    and P, written to the workspace as the operand images (128-byte swizzle) of the second launch.
// 2. gdn_scan_kernel, a CTA per (sequence, value head), walking over the chunks with the state on chip.
//    All products are transposed, so that a tensor-memory lane is a value column and every A operand is
//    in tensor memory, M = 128 (tcgen05, one elected thread issuing):
//      W^T = S0^T K^T [128 x 64];  X^T = V^T - c1 W^T;  U^T = X^T T^T;  O^T = c2 S0^T Q^T + U^T P^T;
//      S1^T = e^{G_C} S0^T + (c3 U)^T K [128 x 128].
//    A thread holds half of its lane's state, 64 values, in registers in FP32, and all scalings of
//    its lane are its own.
//
// Precision.  The state is carried on, so its products keep FP32's precision: the factors that change
// (S0, X, U) and T go to the tensor cores as pairs of FP16 (hi + lo, 22 bits), each lane or row scaled by
// a power of two so that its largest value is near FP16's upper end, which leaves 2^-39 of the largest as
// the smallest step.  K and Q are BF16 values, which are exact in FP16 once their row is scaled the same
// way, and the norms are factors of the rows.  Products of two pairs leave out lo x lo (2^-22).  What
// only reaches the BF16 output (Q S0 and P U) takes hi alone, 2^-11, an eighth of the output's own rounding.
// Decays are e^(difference of sums): the sums are FP64, since a strong decay (g down to -128) next to a
// weak one would take the weak one's digits in FP32.
#include <cuda.h>
#include <cuda_fp16.h>

#include "rma_gdn.cuh"
#include "sm100_ptx.cuh"

namespace rma {
namespace {

constexpr int kC = 64;                        // tokens of a chunk
constexpr int kTile = kC * 128;               // 64 rows of 64 FP16: one operand image
// a (chunk, key head) block of the workspace: K columns 0-63, 64-127, Q columns 0-63, 64-127
constexpr int kKQBytes = 4 * kTile;
// a (chunk, value head) block: T hi, T lo, P, then FP32 scalars
constexpr int kTPBytes = 3 * kTile + 1536;
constexpr int kOffTLo = kTile, kOffP = 2 * kTile, kOffScal = 3 * kTile;
// scalars: factors of token i in W (c1), Q S0 (c2), U' (c3), the scales of T's and P's rows, e^{G_C}
constexpr int kC1 = 0, kC2 = 64, kC3 = 128, kTS = 192, kPS = 256, kEC = 320;

// ---- powers of two ----
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // |e| <= 126
// the exponent of a scale that brings values of magnitude up to m into [.., 2^top): both it and its
// negative are exponents of normal numbers, whatever m is
__device__ __forceinline__ int scale_of_exponent(int e, int top) { return top - 1 - min(max(e, -110), 127); }
__device__ __forceinline__ int scale_exponent(float m, int top) { return scale_of_exponent(exponent_of(m), top); }

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// the pair (hi, lo) of two values
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = half2_bits(a - f.x, b - f.y);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// byte offset of 16-byte piece `piece` (8 values) of row `row` in an operand image
__device__ __forceinline__ int piece_at(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

// ---------------------------------------------------------------------------
// launch 1
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kHeadsAtOnce = 8;    // value heads whose gates are computed together, one per warp

struct __align__(1024) PrepSmem {
    uint8_t kq[kKQBytes];
    float A[kC][kC + 1];
    float T[kC][kC + 1];
    float Y[32][33];
    double G[kHeadsAtOnce][kC];
    float beta[kHeadsAtOnce][kC];
    float rk[kC], rq[kC];
};

__global__ void __launch_bounds__(kPrepThreads) gdn_prep_kernel(const __grid_constant__ DeltaArgs a, int NC) {
    extern __shared__ uint8_t smem_raw[];
    PrepSmem& s = *reinterpret_cast<PrepSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kh = blockIdx.x % a.HK;
    const int b = (blockIdx.x / a.HK) % a.B;
    const int c = blockIdx.x / a.HK / a.B;
    grid_dep_wait();
    grid_dep_launch();
    const int len = seq_len(a.lens, b, a.n, a.status, c == 0 && kh == 0 && tid == 0);
    const int t0 = c * kC;
    const int valid = min(len - t0, kC);
    if (valid <= 0) return;
    const int R = a.HV / a.HK;

    // K and Q rows into FP16 images, a half-warp per row, with the row's norm
    {
        const int sub = lane >> 4, l16 = lane & 15;
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int m = it >> 2;                                    // 0: K, 1: Q
            const int row = (it & 3) * 16 + warp * 2 + sub;
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (row < valid)
                raw = *reinterpret_cast<const uint4*>(a.qkv + ((int64_t)b * a.n + t0 + row) * a.C +
                                                      (m ? kh : a.HK + kh) * kGdnDim + 8 * l16);
            const float2 p0 = unpack_bf16(raw.x), p1 = unpack_bf16(raw.y), p2 = unpack_bf16(raw.z), p3 = unpack_bf16(raw.w);
            float x[8] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[i]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const int e = scale_exponent(mx, 8);
            const float f = pow2(e), inv = pow2(-e);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= f;
                ss = fmaf(x[i], x[i], ss);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            *reinterpret_cast<uint4*>(s.kq + (2 * m + (l16 >> 3)) * kTile + piece_at(row, l16 & 7)) =
                make_uint4(half2_bits(x[0], x[1]), half2_bits(x[2], x[3]), half2_bits(x[4], x[5]), half2_bits(x[6], x[7]));
            if (l16 == 0) {
                // 1 / sqrt(sum x^2 + eps) times the row's scale; the sum is of scaled values, so the one
                // form keeps large rows from overflowing and the other rows far below eps from NaN
                float r = inv;
                if (a.l2norm) {
                    if (e <= 60 || a.l2_eps == 0.f) r = 1.f / sqrtf(ss + a.l2_eps * f * f);
                    else r = inv / sqrtf(ss * inv * inv + a.l2_eps);
                }
                if (row >= valid) r = 0.f;
                if (m) s.rq[row] = r * a.scale;
                else s.rk[row] = r;
            }
        }
    }
    __syncthreads();
    // the images to the workspace
    uint8_t* kq_out = a.ws + (((int64_t)b * a.HK + kh) * NC + c) * kKQBytes;
    for (int i = tid; i < kKQBytes / 16; i += kPrepThreads)
        reinterpret_cast<uint4*>(kq_out)[i] = reinterpret_cast<const uint4*>(s.kq)[i];
    uint8_t* tp_base = a.ws + (int64_t)a.B * a.HK * NC * kKQBytes;

    // rows 16 rb .. + 15 of K K^T (warps 0-3) or Q K^T (warps 4-7): acc[nt] = columns 8 nt ..
    const int rb = warp & 3, m = warp >> 2;
    float acc[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    {
        const uint32_t kbase = ptx::smem_u32(s.kq), abase = kbase + 2 * m * kTile;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t fa[4];
            ldsm4(abase + (ks >> 2) * kTile + piece_at(16 * rb + (lane & 15), (ks & 3) * 2 + (lane >> 4)), fa);
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                if (np <= rb) {   // columns above the diagonal block are not used
                    uint32_t fb[4];
                    ldsm4(kbase + (ks >> 2) * kTile +
                              piece_at(16 * np + (lane & 7) + ((lane >> 4) << 3), (ks & 3) * 2 + ((lane >> 3) & 1)), fb);
                    mma_f16(acc[2 * np], fa, fb[0], fb[1]);
                    mma_f16(acc[2 * np + 1], fa, fb[2], fb[3]);
                }
            }
        }
    }

    for (int r0 = 0; r0 < R; r0 += kHeadsAtOnce) {
        // gates of up to 8 value heads, a warp each: two tokens a lane, running sums in FP64
        __syncthreads();
        if (r0 + warp < R) {
            const int h = kh * R + r0 + warp;
            const float alpha = expf(a.a_log[h]), dt = a.dt_bias[h];
            float g[2], bt[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                g[i] = 0.f;
                bt[i] = 0.f;
                if (t < valid) {
                    const int64_t at = ((int64_t)b * a.n + t0 + t) * a.ab_stride + h;
                    gates(a.a[at], a.b[at], alpha, dt, g[i], bt[i]);
                }
            }
            const double own = (double)g[0] + (double)g[1];
            double run = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += up;
            }
            s.G[warp][2 * lane] = run - own + (double)g[0];
            s.G[warp][2 * lane + 1] = run;
            s.beta[warp][2 * lane] = bt[0];
            s.beta[warp][2 * lane + 1] = bt[1];
        }
        for (int r = r0; r < min(r0 + kHeadsAtOnce, R); ++r) {
            __syncthreads();
            const double* G = s.G[r - r0];
            const float* beta = s.beta[r - r0];
            uint8_t* out = tp_base + (((int64_t)b * a.HV + kh * R + r) * NC + c) * kTPBytes;
            float* scal = reinterpret_cast<float*>(out + kOffScal);
            const int i0 = 16 * rb + (lane >> 2);
            if (m == 0) {
                // A, strictly below the diagonal
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = i0 + 8 * half;
                    const double Gi = G[i];
                    const float f = beta[i] * s.rk[i];
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int j = 8 * nt + 2 * (lane & 3) + x;
                            float v = 0.f;
                            if (j < i) v = f * s.rk[j] * __expf((float)(Gi - G[j])) * acc[nt][2 * half + x];
                            s.A[i][j] = v;
                        }
                }
            } else {
                // P, and its rows' scales
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = i0 + 8 * half;
                    const double Gi = G[i];
                    const float f = s.rq[i];
                    float p[16], mx = 0.f;
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int j = 8 * nt + 2 * (lane & 3) + x;
                            float v = 0.f;
                            if (j <= i) v = f * s.rk[j] * __expf((float)(Gi - G[j])) * acc[nt][2 * half + x];
                            p[2 * nt + x] = v;
                            mx = fmaxf(mx, fabsf(v));
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const int e = scale_exponent(mx, 8);
                    const float sc = pow2(e);
                    if ((lane & 3) == 0) scal[kPS + i] = pow2(-e);
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
                        *reinterpret_cast<uint32_t*>(out + kOffP + piece_at(i, nt) + 4 * (lane & 3)) =
                            half2_bits(p[2 * nt] * sc, p[2 * nt + 1] * sc);
                }
            }
            if (tid < kC) {
                const float since = __expf((float)G[tid]), until = __expf((float)(G[kC - 1] - G[tid]));
                scal[kC1 + tid] = since * s.rk[tid];
                scal[kC2 + tid] = since * s.rq[tid];
                scal[kC3 + tid] = until * s.rk[tid];
                if (tid == 0) scal[kEC] = __expf((float)G[kC - 1]);
            }
            __syncthreads();
            // inverse of (1 + A): its four 16 x 16 diagonal blocks by substitution, a thread per column
            if (tid < kC) {
                const int o = tid & ~15, j = tid & 15;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
                for (int l = 0; l < 15; ++l)
#pragma unroll
                    for (int i = l + 1; i < 16; ++i) x[i] = fmaf(-s.A[o + i][o + l], x[l], x[i]);
#pragma unroll
                for (int i = 0; i < 16; ++i) s.T[o + i][o + j] = x[i];
            }
            __syncthreads();
            // pairs of 16 into 32: T21 = -T22 (A21 T11)
            {
                const int o = (tid >> 7) * 32, i = (tid & 127) >> 3, j = (tid & 7) * 2;
                float y0 = 0.f, y1 = 0.f;
#pragma unroll
                for (int l = 0; l < 16; ++l) {
                    const float v = s.A[o + 16 + i][o + l];
                    y0 = fmaf(v, s.T[o + l][o + j], y0);
                    y1 = fmaf(v, s.T[o + l][o + j + 1], y1);
                }
                s.Y[(tid >> 7) * 16 + i][j] = y0;
                s.Y[(tid >> 7) * 16 + i][j + 1] = y1;
                // the quarter above the diagonal, which the next product reads
                s.T[o + i][o + 16 + j] = 0.f;
                s.T[o + i][o + 16 + j + 1] = 0.f;
                __syncthreads();
                float z0 = 0.f, z1 = 0.f;
#pragma unroll
                for (int l = 0; l < 16; ++l) {
                    const float v = s.T[o + 16 + i][o + 16 + l];
                    z0 = fmaf(v, s.Y[(tid >> 7) * 16 + l][j], z0);
                    z1 = fmaf(v, s.Y[(tid >> 7) * 16 + l][j + 1], z1);
                }
                s.T[o + 16 + i][o + j] = -z0;
                s.T[o + 16 + i][o + j + 1] = -z1;
            }
            __syncthreads();
            // and 32 into 64, 2 x 2 values a thread
            {
                const int i = (tid >> 4) * 2, j = (tid & 15) * 2;
                float y[2][2] = {};
#pragma unroll 8
                for (int l = 0; l < 32; ++l) {
                    const float u0 = s.A[32 + i][l], u1 = s.A[33 + i][l], v0 = s.T[l][j], v1 = s.T[l][j + 1];
                    y[0][0] = fmaf(u0, v0, y[0][0]); y[0][1] = fmaf(u0, v1, y[0][1]);
                    y[1][0] = fmaf(u1, v0, y[1][0]); y[1][1] = fmaf(u1, v1, y[1][1]);
                }
                __syncthreads();
                s.Y[i][j] = y[0][0]; s.Y[i][j + 1] = y[0][1];
                s.Y[i + 1][j] = y[1][0]; s.Y[i + 1][j + 1] = y[1][1];
                s.T[i][32 + j] = s.T[i][33 + j] = s.T[i + 1][32 + j] = s.T[i + 1][33 + j] = 0.f;
                __syncthreads();
                float z[2][2] = {};
#pragma unroll 8
                for (int l = 0; l < 32; ++l) {
                    const float u0 = s.T[32 + i][32 + l], u1 = s.T[33 + i][32 + l], v0 = s.Y[l][j], v1 = s.Y[l][j + 1];
                    z[0][0] = fmaf(u0, v0, z[0][0]); z[0][1] = fmaf(u0, v1, z[0][1]);
                    z[1][0] = fmaf(u1, v0, z[1][0]); z[1][1] = fmaf(u1, v1, z[1][1]);
                }
                s.T[32 + i][j] = -z[0][0]; s.T[32 + i][j + 1] = -z[0][1];
                s.T[33 + i][j] = -z[1][0]; s.T[33 + i][j + 1] = -z[1][1];
            }
            __syncthreads();
            // T's rows with beta's columns, scaled and split: four threads a row, 16 columns each
            {
                const int i = tid >> 2, j0 = (tid & 3) * 16;
                float v[16], mx = 0.f;
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    v[x] = s.T[i][j0 + x] * beta[j0 + x];
                    mx = fmaxf(mx, fabsf(v[x]));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int e = scale_exponent(mx, 8);
                const float sc = pow2(e);
                if ((tid & 3) == 0) scal[kTS + i] = pow2(-e);
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) split2(v[2 * x] * sc, v[2 * x + 1] * sc, hi[x], lo[x]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int at = piece_at(i, (j0 >> 3) + x);
                    *reinterpret_cast<uint4*>(out + at) = make_uint4(hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
                    *reinterpret_cast<uint4*>(out + kOffTLo + at) = make_uint4(lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// launch 2
// ---------------------------------------------------------------------------
constexpr int kStageTP = kKQBytes;                        // offsets in a stage
constexpr int kStageV = (kKQBytes + kTPBytes + 1023) / 1024 * 1024;
constexpr int kStageBytes = kStageV + kC * kGdnDim * 2;
constexpr int kStages = 3;
constexpr int kScanBar = kStages * kStageBytes;
constexpr int kScanMax = kScanBar + 256;                  // exponents of lane maxima: [4 exchanges][2 halves][128]
constexpr int kScanSmem = kScanMax + 4 * 2 * 128 + 1024;
constexpr int kWarpLoad = 8, kWarpMma = 9;
constexpr int kScanThreads = 320;
static_assert(kScanSmem <= 227 * 1024, "shared memory per CTA");

// tensor memory columns: S0 as hi [0, 64) and lo [64, 128), then the state's increment [0, 128) in FP32;
// W; X, then the scaled U, as hi and lo (32 each); Q S0; U, then P U; U as hi
constexpr uint32_t kTmS = 0, kTmW = 128, kTmX = 192, kTmQ = 256, kTmU = 320, kTmUh = 384, kTmCols = 512;

enum ScanBar {
    kbFull = 0,      // [3] the stage's loads landed (tx bytes)
    kbEmpty = 3,     // [3] 8 warps have read the stage, and every product that reads it is complete
    kbS = 6,         // 8 warps: S0 in tensor memory
    kbX = 7,         // 8 warps: X in tensor memory
    kbU = 8,         // 8 warps: U and the scaled U in tensor memory
    kbWDone = 9,     // commits: W; Q S0; U; the state's increment; P U
    kbQDone = 10,
    kbUDone = 11,
    kbDDone = 12,
    kbPDone = 13,
    kbDrain = 14,    // commit after the last product, also of an abandoned CTA
    kScanBars = 15
};

__global__ void __launch_bounds__(kScanThreads, 1) gdn_scan_kernel(const __grid_constant__ DeltaArgs a, int NC) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x, b = unit / a.HV, h = unit % a.HV, kh = h / (a.HV / a.HK);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kScanBar);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + kScanBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int8_t* maxima = reinterpret_cast<int8_t*>(smem + kScanMax);
    grid_dep_wait();
    grid_dep_launch();
    const int len = seq_len(a.lens, b, a.n, a.status, false);
    if (len == 0) return;
    const int nc = (len + kC - 1) / kC;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&bars[kbFull + i], 1);
            ptx::mbar_init(&bars[kbEmpty + i], 8);
        }
        for (int i = kbS; i <= kbU; ++i) ptx::mbar_init(&bars[i], 8);
        for (int i = kbWDone; i < kScanBars; ++i) ptx::mbar_init(&bars[i], 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc1(tmem_holder, kTmCols);
        ptx::tmem_relinquish1();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    bool ok = true;

    if (warp == kWarpLoad) {
        // ---------------- loads: a stage is the chunk's K and Q, its T, P and scalars, and its V rows ----------------
        const uint8_t* kq = a.ws + ((int64_t)b * a.HK + kh) * NC * kKQBytes;
        const uint8_t* tp = a.ws + (int64_t)a.B * a.HK * NC * kKQBytes + (int64_t)unit * NC * kTPBytes;
        const uint16_t* v = a.qkv + (int64_t)b * a.n * a.C + (2 * a.HK + h) * kGdnDim;
        int issued = 0;
        for (int c = 0; c < nc; ++c) {
            const int st = c % kStages;
            if (c >= kStages && !ptx::mbar_wait_warp(&bars[kbEmpty + st], (c / kStages - 1) & 1, abort_flag, a.status)) break;
            issued = c + 1;
            uint8_t* stage = smem + st * kStageBytes;
            const int rows = min(len - c * kC, kC);
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(&bars[kbFull + st], kKQBytes + kTPBytes + rows * kGdnDim * 2);
                ptx::bulk_load(stage, kq + (int64_t)c * kKQBytes, kKQBytes, &bars[kbFull + st]);
                ptx::bulk_load(stage + kStageTP, tp + (int64_t)c * kTPBytes, kTPBytes, &bars[kbFull + st]);
            }
            __syncwarp();
            for (int i = lane; i < rows; i += 32)
                ptx::bulk_load(stage + kStageV + i * kGdnDim * 2, v + (int64_t)(c * kC + i) * a.C, kGdnDim * 2, &bars[kbFull + st]);
        }
        // what was asked for has landed before the CTA ends
        for (int c = max(0, issued - kStages); c < issued; ++c)
            ptx::mbar_wait_drain(&bars[kbFull + c % kStages], (c / kStages) & 1, a.status);
    } else if (warp == kWarpMma) {
        // ---------------- products ----------------
        constexpr uint32_t id64 = ptx::idesc_f16_f32(128, 64, false, false);
        constexpr uint32_t id128 = ptx::idesc_f16_f32(128, 128, false, true);
        auto kmajor = [](uint32_t base, int ks) {   // 16 values of the rows of an image
            return ptx::smem_desc(base + ks * 32, 16, 1024, ptx::kSwizzle128B);
        };
        for (int c = 0; c < nc; ++c) {
            const int st = c % kStages;
            const uint32_t kb = ptx::smem_u32(smem + st * kStageBytes), tb = kb + kStageTP;
            ok = ptx::mbar_wait_warp(&bars[kbFull + st], (c / kStages) & 1, abort_flag, a.status);
            if (!ok) break;
            ok = ptx::mbar_wait_warp(&bars[kbS], c & 1, abort_flag, a.status);
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                for (int ks = 0; ks < 8; ++ks)
                    ptx::mma_ts1(tmem + kTmW, tmem + kTmS + 8 * ks, kmajor(kb + (ks >> 2) * kTile, ks & 3), id64, ks > 0);
                for (int ks = 0; ks < 8; ++ks)
                    ptx::mma_ts1(tmem + kTmW, tmem + kTmS + 64 + 8 * ks, kmajor(kb + (ks >> 2) * kTile, ks & 3), id64, 1);
                ptx::mma_commit1(&bars[kbWDone]);
                for (int ks = 0; ks < 8; ++ks)
                    ptx::mma_ts1(tmem + kTmQ, tmem + kTmS + 8 * ks, kmajor(kb + (2 + (ks >> 2)) * kTile, ks & 3), id64, ks > 0);
                ptx::mma_commit1(&bars[kbQDone]);
            }
            __syncwarp();
            ok = ptx::mbar_wait_warp(&bars[kbX], c & 1, abort_flag, a.status);
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                for (int ks = 0; ks < 4; ++ks) {
                    ptx::mma_ts1(tmem + kTmU, tmem + kTmX + 8 * ks, kmajor(tb, ks), id64, ks > 0);
                    ptx::mma_ts1(tmem + kTmU, tmem + kTmX + 32 + 8 * ks, kmajor(tb, ks), id64, 1);
                    ptx::mma_ts1(tmem + kTmU, tmem + kTmX + 8 * ks, kmajor(tb + kOffTLo, ks), id64, 1);
                }
                ptx::mma_commit1(&bars[kbUDone]);
            }
            __syncwarp();
            ok = ptx::mbar_wait_warp(&bars[kbU], c & 1, abort_flag, a.status);
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t kd = ptx::smem_desc(kb + ks * 16 * 128, kTile, 1024, ptx::kSwizzle128B);
                    ptx::mma_ts1(tmem + kTmS, tmem + kTmX + 8 * ks, kd, id128, ks > 0);
                    ptx::mma_ts1(tmem + kTmS, tmem + kTmX + 32 + 8 * ks, kd, id128, 1);
                }
                ptx::mma_commit1(&bars[kbDDone]);
                for (int ks = 0; ks < 4; ++ks)
                    ptx::mma_ts1(tmem + kTmU, tmem + kTmUh + 8 * ks, kmajor(tb + kOffP, ks), id64, ks > 0);
                ptx::mma_commit1(&bars[kbPDone]);
            }
            __syncwarp();
        }
        if (lane == 0) ptx::mma_commit1(&bars[kbDrain]);
        __syncwarp();
        ptx::mbar_wait_drain(&bars[kbDrain], 0, a.status);
    } else {
        // ---------------- a thread: lane (value column) `row`, half `wg` of the keys or tokens ----------------
        const int wg = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int pair_bar = 1 + (warp & 3);
        // the scale of this lane's values, whose largest in this half is m, from both halves' exponents:
        // offered, exchanged (which also orders the two warps' tensor-memory accesses), taken
        auto offer = [&](int which, float m) {
            maxima[(2 * which + wg) * 128 + row] = (int8_t)min(max(exponent_of(m), -110), 127);
        };
        auto exchange = [&]() {
            ptx::tc_fence_before();
            ptx::named_bar_sync(pair_bar, 64);
            ptx::tc_fence_after();
        };
        auto take = [&](int which) {
            return scale_of_exponent(max(maxima[2 * which * 128 + row], maxima[(2 * which + 1) * 128 + row]), 15);
        };
        auto signal = [&](int bar) {
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars[bar]);
        };
        float S[64];
        float* gs = a.state + ((int64_t)unit * kGdnDim + 64 * wg) * kGdnDim + row;
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = gs[i * kGdnDim];
        float inv_s = 1.f;
        auto put_state = [&]() {
            float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 64; ++i) m[i & 3] = fmaxf(m[i & 3], fabsf(S[i]));
            offer(0, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
            exchange();
            const int e = take(0);
            const float f = pow2(e);
            inv_s = pow2(-e);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(S[32 * p + 2 * i] * f, S[32 * p + 2 * i + 1] * f, hi[i], lo[i]);
                ptx::tmem_st16(tl + kTmS + 32 * wg + 16 * p, hi);
                ptx::tmem_st16(tl + kTmS + 64 + 32 * wg + 16 * p, lo);
            }
            signal(kbS);
        };
        put_state();
        for (int c = 0; c < nc; ++c) {
            const int st = c % kStages;
            const uint8_t* stage = smem + st * kStageBytes;
            const float* scal = reinterpret_cast<const float*>(stage + kStageTP + kOffScal);
            const uint16_t* vs = reinterpret_cast<const uint16_t*>(stage + kStageV) + 32 * wg * kGdnDim + row;
            const int left = len - c * kC - 32 * wg;   // tokens of this half
            // (an abandoned CTA goes on through its barriers, on values that nobody uses)
            ok = ptx::mbar_wait_warp(&bars[kbFull + st], (c / kStages) & 1, abort_flag, a.status) && ok;
            uint32_t x[32];
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = bf16_float(vs[i * kGdnDim]);
            ok = ptx::mbar_wait_warp(&bars[kbWDone], c & 1, abort_flag, a.status) && ok;
            ptx::tc_fence_after();
            ptx::tmem_ld32(tl + kTmW + 32 * wg, x);
            ptx::tmem_wait_ld();
            float inv_x;
            {
                float m[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float w = __uint_as_float(x[i]) * inv_s;
                    const float d = i < left ? fmaf(-scal[kC1 + 32 * wg + i], w, v[i]) : 0.f;
                    v[i] = d;
                    m[i & 1] = fmaxf(m[i & 1], fabsf(d));
                }
                offer(1, fmaxf(m[0], m[1]));
                exchange();
                const int e = take(1);
                const float f = pow2(e);
                inv_x = pow2(-e);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(v[2 * i] * f, v[2 * i + 1] * f, hi[i], lo[i]);
                ptx::tmem_st16(tl + kTmX + 16 * wg, hi);
                ptx::tmem_st16(tl + kTmX + 32 + 16 * wg, lo);
                signal(kbX);
            }
            // Q S0 while U is computed
            float o[32];
            ok = ptx::mbar_wait_warp(&bars[kbQDone], c & 1, abort_flag, a.status) && ok;
            ptx::tc_fence_after();
            ptx::tmem_ld32(tl + kTmQ + 32 * wg, x);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(x[i]) * inv_s * scal[kC2 + 32 * wg + i];
            // U, and U scaled for the state
            ok = ptx::mbar_wait_warp(&bars[kbUDone], c & 1, abort_flag, a.status) && ok;
            ptx::tc_fence_after();
            ptx::tmem_ld32(tl + kTmU + 32 * wg, x);
            ptx::tmem_wait_ld();
            float inv_u, inv_d;
            {
                float mu = 0.f, md = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float u = __uint_as_float(x[i]) * inv_x * scal[kTS + 32 * wg + i];
                    x[i] = __float_as_uint(u);
                    v[i] = u * scal[kC3 + 32 * wg + i];
                    mu = fmaxf(mu, fabsf(u));
                    md = fmaxf(md, fabsf(v[i]));
                }
                offer(2, md);
                offer(3, mu);
                exchange();
                const int ed = take(2), eu = take(3);
                const float fd = pow2(ed), fu = pow2(eu);
                inv_d = pow2(-ed);
                inv_u = pow2(-eu);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(v[2 * i] * fd, v[2 * i + 1] * fd, hi[i], lo[i]);
                ptx::tmem_st16(tl + kTmX + 16 * wg, hi);
                ptx::tmem_st16(tl + kTmX + 32 + 16 * wg, lo);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    hi[i] = half2_bits(__uint_as_float(x[2 * i]) * fu, __uint_as_float(x[2 * i + 1]) * fu);
                ptx::tmem_st16(tl + kTmUh + 16 * wg, hi);
                signal(kbU);
            }
            // the state
            const float keep = scal[kEC];
            ok = ptx::mbar_wait_warp(&bars[kbDDone], c & 1, abort_flag, a.status) && ok;
            ptx::tc_fence_after();
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                ptx::tmem_ld32(tl + kTmS + 64 * wg + 32 * p, x);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) S[32 * p + i] = fmaf(S[32 * p + i], keep, __uint_as_float(x[i]) * inv_d);
            }
            if (c + 1 < nc) put_state();
            // the outputs
            ok = ptx::mbar_wait_warp(&bars[kbPDone], c & 1, abort_flag, a.status) && ok;
            ptx::tc_fence_after();
            ptx::tmem_ld32(tl + kTmU + 32 * wg, x);
            ptx::tmem_wait_ld();
            uint16_t* out = a.out + (((int64_t)b * a.n + c * kC + 32 * wg) * a.HV + h) * kGdnDim + row;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float y = fmaf(__uint_as_float(x[i]) * inv_u, scal[kPS + 32 * wg + i], o[i]);
                if (i < left) out[(int64_t)i * a.HV * kGdnDim] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars[kbEmpty + st]);
        }
        if (ok) {
#pragma unroll
            for (int i = 0; i < 64; ++i) gs[i * kGdnDim] = S[i];
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWarpMma) ptx::tmem_dealloc1(tmem, kTmCols);
}

}  // namespace

size_t gdn_prefill_workspace_bytes(const rma_gdn_config& c, int n) {
    if (n < kGdnChunkedFrom) return 256;
    const size_t NC = (n + kC - 1) / kC;
    const size_t bytes = NC * c.batch * ((size_t)c.n_k_heads * kKQBytes + (size_t)c.n_v_heads * kTPBytes);
    return (bytes + 255) / 256 * 256;
}

cudaError_t launch_gdn_prefill(const DeltaArgs& a, cudaStream_t stream) {
    if (a.n < kGdnChunkedFrom) return launch_gdn_recurrent(a, stream);
    const int NC = (a.n + kC - 1) / kC;
    const int64_t grid = (int64_t)NC * a.B * a.HK;
    if (grid > 0x7fffffffll) return cudaErrorNotSupported;
    const size_t prep_smem = sizeof(PrepSmem) + 1024;
    static SmemLimit prep_limit(reinterpret_cast<const void*>(gdn_prep_kernel));
    static SmemLimit scan_limit(reinterpret_cast<const void*>(gdn_scan_kernel));
    cudaError_t e = prep_limit.ensure(prep_smem);
    if (e == cudaSuccess) e = scan_limit.ensure(kScanSmem);
    if (e != cudaSuccess) return e;
    PdlLaunch prep((unsigned)grid, kPrepThreads, prep_smem, stream);
    e = cudaLaunchKernelEx(&prep.cfg, gdn_prep_kernel, a, NC);
    if (e != cudaSuccess) return e;
    PdlLaunch scan((unsigned)(a.B * a.HV), kScanThreads, kScanSmem, stream);
    return cudaLaunchKernelEx(&scan.cfg, gdn_scan_kernel, a, NC);
}

}  // namespace rma
