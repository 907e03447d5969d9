// rma_qk_norm_rope: per-head RMS norm of queries and keys, then the position rotation.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  for the rotated pairs (u, v) of a head:
//   (y_u c - y_v s, y_v c + y_u s),  c, s = cos, sin of position * inv_freq[i].
//
// Memory bound: every value is read once and written once, 4 bytes in all.  A CTA takes one KV group's 4
// query heads and its key, a warp each, 8 values (16 bytes) a lane, of one or several consecutive tokens:
// all loads are issued first, then the angles of the group's tokens are computed, a thread each, while
// they are in flight; the sum of squares is one warp reduction.  A product of a far position and a
// frequency has an absolute error of half an ulp of the angle, 0.008 rad at 2^18 in FP32, so the product
// and its reduction to a fraction of a turn are in FP64; the fraction's sine and cosine then need FP32
// only.  Partners in another lane come by shuffles, or through the warp's row of shared memory where a lane's
// eight values do not have one side (rotary_dim / 2 not a multiple of 8).
//
// Measured on one B200, 4 groups: 1.9 us for one token, 5.1 us for 512 sequences of one token (64 values
// rotated; 2,048 CTAs, of which 8 fit an SM: 1.7 waves), 15.2 us for 8 x 256 tokens with all 256 rotated (42 MB,
// 2.8 TB/s; 14.8 before the sums were checked for what FP32 holds).  The last is 3.5 waves of short
// CTAs that issue in 78% of the cycles, about a third of it for the angles, which every group computes for
// itself (its counter is its own).  Two FP32 values an instruction and one table for four groups gave 14.0 us
// there but 5.5 us for the 512.

#include "rma_gdn.cuh"

namespace rma {
namespace {

constexpr int kHeads = kQPerGroup + 1;   // of one group: its queries and its key
constexpr int kRopeThreads = 32 * kHeads;

// Where pair p of a half-split rotation lies in the tables: a lane takes eight in a row, as two fours, and the
// lanes' first fours lie side by side (eight in a row each put all lanes on four banks: 8-way conflicts, which
// held 2,048 tokens to 20 us).
__device__ __forceinline__ int at_pair(int p) { return ((p >> 2) & 1) * 64 + ((p >> 3) << 2) + (p & 3); }

__device__ __forceinline__ void unpack8(const uint4& raw, float (&x)[8]) {
    const float2 p0 = unpack_bf16(raw.x), p1 = unpack_bf16(raw.y), p2 = unpack_bf16(raw.z), p3 = unpack_bf16(raw.w);
    x[0] = p0.x; x[1] = p0.y; x[2] = p1.x; x[3] = p1.y;
    x[4] = p2.x; x[5] = p2.y; x[6] = p3.x; x[7] = p3.y;
}

template <int T>   // tokens of a CTA
__global__ void __launch_bounds__(kRopeThreads, 8) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float cs[T][kHeadDim / 2], sn[T][kHeadDim / 2];
    __shared__ __align__(16) float rows[kHeads][kHeadDim];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.x % a.G;
    const int64_t tok0 = (int64_t)(blockIdx.x / a.G) * T;   // of b n + i
    const int count = (int)min((int64_t)T, (int64_t)a.B * a.n - tok0);
    grid_dep_wait();
    grid_dep_launch();

    const bool is_k = warp == kQPerGroup;
    const int64_t stride = is_k ? a.k_stride : a.q_stride;
    const uint16_t* src = (is_k ? a.k + (int64_t)g * kHeadDim : a.q + (int64_t)(g * kQPerGroup + warp) * kHeadDim) + tok0 * stride;
    uint4 raw[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (t < count) raw[t] = reinterpret_cast<const uint4*>(src + t * stride)[lane];
    const float4* w4 = reinterpret_cast<const float4*>(is_k ? a.w_k : a.w_q) + 2 * lane;
    const float4 wa = __ldg(w4), wb = __ldg(w4 + 1);
    const float w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};

    const int half = a.half;
    for (int i = threadIdx.x; i < half * count; i += kRopeThreads) {
        const int t = T == 1 ? 0 : i / half, f = T == 1 ? i : i - t * half;
        const int64_t tok = tok0 + t;
        int64_t pos;
        if (a.positions) {
            pos = a.positions[tok];
        } else {
            const int64_t b = tok / a.n;
            const int c = a.counters[(b * a.G + g) * 4];
            if (c < 0 && f == 0) atomicOr(a.status, (unsigned)RMA_STATUS_BAD_COUNTERS);
            pos = (int64_t)max(c, 0) + (tok - b * a.n);
        }
        const double turns = (double)pos * (a.inv_freq[f] * 0.15915494309189533577);   // 1 / (2 pi)
        const int at = a.interleaved ? f : at_pair(f);
        sincospif(2.f * (float)(turns - rint(turns)), &sn[t][at], &cs[t][at]);
    }
    __syncthreads();

    const int64_t dst_stride = (int64_t)a.G * kHeadDim * (is_k ? 1 : kQPerGroup);
    uint16_t* dst = (is_k ? a.k_out + (int64_t)g * kHeadDim : a.q_out + (int64_t)(g * kQPerGroup + warp) * kHeadDim) + tok0 * dst_stride;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        if (t >= count) break;
        float x[8];
        unpack8(raw[t], x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        float mean = ss * (1.f / kHeadDim) + a.eps;
        if (!plain_sum(mean)) {   // squares that FP32 does not hold: all values times a power of two, which r takes back
            const float f = mean >= 1.f ? 0x1p-80f : 0x1p80f;
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= f;
                ss = fmaf(x[i], x[i], ss);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            mean = ss * (1.f / kHeadDim) + a.eps * f * f;
        }
        const float r = 1.f / sqrtf(mean);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];

        const int d0 = 8 * lane;
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = 4 * lane + i;
                if (p < half) {
                    const float u = x[2 * i], v = x[2 * i + 1], c = cs[t][p], s = sn[t][p];
                    x[2 * i] = u * c - v * s;
                    x[2 * i + 1] = v * c + u * s;
                }
            }
        } else if (half > 0) {
            if ((half & 7) == 0) {   // a lane's values have one side each, and their partners are one lane's
                const bool first = d0 < half, mine = d0 < 2 * half;
                const int other = mine ? (first ? lane + half / 8 : lane - half / 8) : lane;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], other);
                if (mine) {
                    const int p = (first ? d0 : d0 - half) >> 1;   // eight pairs, in two fours (at_pair)
                    const float4 c0 = *reinterpret_cast<const float4*>(&cs[t][p]), c1 = *reinterpret_cast<const float4*>(&cs[t][p + 64]);
                    const float4 s0 = *reinterpret_cast<const float4*>(&sn[t][p]), s1 = *reinterpret_cast<const float4*>(&sn[t][p + 64]);
                    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = first ? x[i] * c[i] - y[i] * s[i] : x[i] * c[i] + y[i] * s[i];
                }
            } else {
                float4* row = reinterpret_cast<float4*>(rows[warp]) + 2 * lane;
                __syncwarp();   // the token before has been read
                row[0] = make_float4(x[0], x[1], x[2], x[3]);
                row[1] = make_float4(x[4], x[5], x[6], x[7]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = d0 + i;
                    if (d < half) x[i] = x[i] * cs[t][at_pair(d)] - rows[warp][d + half] * sn[t][at_pair(d)];
                    else if (d < 2 * half) x[i] = x[i] * cs[t][at_pair(d - half)] + rows[warp][d - half] * sn[t][at_pair(d - half)];
                }
            }
        }
        reinterpret_cast<uint4*>(dst + t * dst_stride)[lane] =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream) {
    // Few tokens: one a CTA, as many CTAs as there can be.  Many: two, whose loads are both in flight (8 x 256
    // tokens of 4 groups, 42 MB: 17.7 us with one, 15.2 with two at 8 CTAs an SM, 15.5 at 7).
    const int64_t tokens = (int64_t)a.B * a.n;
    const bool many = tokens * a.G >= 4096;
    const PdlLaunch l((unsigned)((many ? (tokens + 1) / 2 : tokens) * a.G), kRopeThreads, 0, stream);
    return many ? cudaLaunchKernelEx(&l.cfg, qk_norm_rope_kernel<2>, a) : cudaLaunchKernelEx(&l.cfg, qk_norm_rope_kernel<1>, a);
}

}  // namespace rma
