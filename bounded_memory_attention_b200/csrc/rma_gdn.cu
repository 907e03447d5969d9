// The gated-delta-rule layers: the short convolution, and the delta rule token by token.
#include "rma_gdn.cuh"

namespace rma {
namespace {

// ---------------------------------------------------------------------------
// rma_gdn_conv: z[t] = bias + sum_j w[j] x[t - 3 + j], out = silu(z), and the three-row state.
//
// Memory bound: 2 bytes read and 2 written per (token, channel), the state's 12 bytes per channel
// and sequence.  A thread keeps 4 or 8 channels' weights in registers.  Blocks of tokens: it walks
// down a tile with the last three rows in registers, the next four rows always on their way, so a row
// is read once per tile plus three rows of overlap.  Single tokens: it walks over sequences instead, so
// that the weights (16 bytes a channel, more than the activations) are fetched once per several, two
// sequences' loads in flight.  The state is read by the first tile only and written by the same
// threads, after their reads.
//
// Measured on one B200, 8,192 channels: 4 ragged prompts of up to 2,048 tokens, 7,202 in all (237 MB), 44.8 us,
// 5.3 TB/s; 512 single tokens (67 MB) 14.0 us, 4.8 TB/s: 2,048 CTAs, of which 9 fit an SM (110 registers), 1.5 waves.
// Blocks issue in 69% of the cycles and their special-function pipe is as busy, so eight CTAs of an SM are needed to
// cover the loads (at 64 registers, of which one is spilled).  Slower there: tiles of 16 or 64 tokens (47.6, 46.3), two
// or eight rows on their way (48, 62), 16 rows through shared memory (50).
// ---------------------------------------------------------------------------
constexpr int kConvThreads = 128;
constexpr int kTokenThreads = 64;
constexpr int kConvTile = 32;     // tokens of a tile
constexpr int kConvRows = 4;      // rows on their way

// z / (1 + exp(-z)).  The approximate forms that flush denormals are two instructions of the slow pipe and no
// more; exp(-z) is infinite below z = -88, where the quotient is -0, and its flush to 0 above 87 changes nothing.
__device__ __forceinline__ float silu(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(1.f + e));
    return z * r;
}

// V channels of a row: 4 (8 bytes) or 8 (16 bytes)
template <int V>
struct ConvRow {
    uint32_t r[V / 2];
    __device__ __forceinline__ static ConvRow load(const uint16_t* p) {
        ConvRow x;
        if constexpr (V == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            x.r[0] = v.x; x.r[1] = v.y; x.r[2] = v.z; x.r[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            x.r[0] = v.x; x.r[1] = v.y;
        }
        return x;
    }
    __device__ __forceinline__ void store(uint16_t* p) const {
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
    }
    __device__ __forceinline__ void floats(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 v = unpack_bf16(r[i]);
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
    }
};

template <int V>
struct ConvWeights {
    float w[V][4], bias[V];
    __device__ __forceinline__ void load(const ConvArgs& a, int c) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(a.w) + c + i);
            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
            bias[i] = 0.f;
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 u = __ldg(reinterpret_cast<const float4*>(a.bias + c) + i);
                bias[4 * i] = u.x; bias[4 * i + 1] = u.y; bias[4 * i + 2] = u.z; bias[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ ConvRow<V> out(const float (&p0)[V], const float (&p1)[V], const float (&p2)[V], const float (&p3)[V]) const {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float z = fmaf(w[i][0], p0[i], bias[i]);
            z = fmaf(w[i][1], p1[i], z);
            z = fmaf(w[i][2], p2[i], z);
            y[i] = silu(fmaf(w[i][3], p3[i], z));
        }
        ConvRow<V> o;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) o.r[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
        return o;
    }
};

__global__ void __launch_bounds__(kConvThreads, 8) gdn_conv_kernel(const __grid_constant__ ConvArgs a, int tiles, int cblocks) {
    constexpr int V = 4;   // 8 leave fewer warps resident: 53 us for the prompts above where 4 took 48
    grid_dep_wait();
    grid_dep_launch();
    const int cb = blockIdx.x % cblocks;
    const int tl = (blockIdx.x / cblocks) % tiles;
    const int b = blockIdx.x / cblocks / tiles;
    const int c = (cb * kConvThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    const int t0 = tl * kConvTile;
    const int len = seq_len(a.lens, b, a.n, a.status, tl == 0 && cb == 0 && threadIdx.x == 0);
    if (t0 >= len) return;
    const uint16_t* x = a.x + (int64_t)b * a.n * a.x_stride + c;
    uint16_t* st = a.state + (int64_t)b * 3 * a.C + c;
    uint16_t* out = a.out + (int64_t)b * a.n * a.C + c;
    auto row = [&](int t) { return ConvRow<V>::load(x + (int64_t)t * a.x_stride); };
    const int end = min(t0 + kConvTile, len);
    ConvRow<V> next[kConvRows], h[3];
#pragma unroll
    for (int i = 0; i < kConvRows; ++i)
        if (t0 + i < end) next[i] = row(t0 + i);
    ConvWeights<V> w;
    w.load(a, c);
    if (t0 == 0) {
#pragma unroll
        for (int j = 0; j < 3; ++j) h[j] = ConvRow<V>::load(st + (int64_t)j * a.C);
        // the last three rows of (state, x): row len + j of the two in sequence
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int i = len + j;
            const ConvRow<V> v = i >= 3 ? row(i - 3) : (i == 1 ? h[1] : h[2]);
            v.store(st + (int64_t)j * a.C);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j) h[j] = row(t0 - 3 + j);
    }
    float p0[V], p1[V], p2[V];
    h[0].floats(p0);
    h[1].floats(p1);
    h[2].floats(p2);
    uint16_t* o = out + (int64_t)t0 * a.C;
    auto one = [&](const ConvRow<V>& r) {
        float p3[V];
        r.floats(p3);
        w.out(p0, p1, p2, p3).store(o);
        o += a.C;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            p0[k] = p1[k];
            p1[k] = p2[k];
            p2[k] = p3[k];
        }
    };
    int t = t0;
    const uint16_t* xn = x + (int64_t)(t0 + kConvRows) * a.x_stride;
    for (; t + 2 * kConvRows <= end; t += kConvRows) {   // these rows and the next are all there
        ConvRow<V> cur[kConvRows];
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) {
            cur[i] = next[i];
            next[i] = ConvRow<V>::load(xn);
            xn += a.x_stride;
        }
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) one(cur[i]);
    }
    for (; t < end; t += kConvRows) {
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) {
            if (t + i < end) {
                one(next[i]);
                if (t + kConvRows + i < end) next[i] = row(t + kConvRows + i);
            }
        }
    }
}

// n == 1: `seqs` sequences a thread, two at a time
__global__ void __launch_bounds__(kTokenThreads) gdn_conv_token_kernel(const __grid_constant__ ConvArgs a, int seqs, int cblocks) {
    constexpr int V = 8;
    grid_dep_wait();
    grid_dep_launch();
    const int cb = blockIdx.x % cblocks;
    const int b0 = (blockIdx.x / cblocks) * seqs, b1 = min(b0 + seqs, a.B);
    const int c = (cb * kTokenThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    ConvWeights<V> w;
    w.load(a, c);
    for (int b = b0; b < b1; b += 2) {
        ConvRow<V> x[2], h[2][3];
        bool on[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            on[i] = b + i < b1 && seq_len(a.lens, b + i, 1, a.status, cb == 0 && threadIdx.x == 0) > 0;
            if (on[i]) {
                x[i] = ConvRow<V>::load(a.x + (int64_t)(b + i) * a.x_stride + c);
#pragma unroll
                for (int j = 0; j < 3; ++j) h[i][j] = ConvRow<V>::load(a.state + ((int64_t)(b + i) * 3 + j) * a.C + c);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!on[i]) continue;
            uint16_t* st = a.state + (int64_t)(b + i) * 3 * a.C + c;
            h[i][1].store(st);
            h[i][2].store(st + a.C);
            x[i].store(st + 2 * (int64_t)a.C);
            float p0[V], p1[V], p2[V], p3[V];
            h[i][0].floats(p0);
            h[i][1].floats(p1);
            h[i][2].floats(p2);
            x[i].floats(p3);
            w.out(p0, p1, p2, p3).store(a.out + (int64_t)(b + i) * a.C + c);
        }
    }
}

// ---------------------------------------------------------------------------
// The delta rule token by token (rma_gdn_decode_step, and prefill blocks too short for chunks).
//
//   S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = S^T q = (e^g S)^T q + (k.q) u,
//
// so one pass over the decayed state gives both products and the update follows in registers: the
// state is read once and written once, which is the bound (64 KiB each way per value head).  A CTA
// holds SLICE value columns of one (sequence, value head), all 128 key rows, in registers; columns
// never meet, so a small batch splits a head over 4 CTAs.  Sums over the key rows go through
// shuffles and one exchange in shared memory.  Everything is FP32.
//
// Measured on one B200, one token: 3.1 us for one sequence of 32 value heads (4 CTAs a head), 7.6 us for 37
// of 6 heads (29 MB, 3.8 TB/s; 888 CTAs, of which 4 fit an SM: 1.5 waves), 317 us for 512 of 32 heads (2.16 GB, 6.8 TB/s).
// ---------------------------------------------------------------------------
constexpr int kRecThreads = 256;
constexpr int kRecWarps = kRecThreads / 32;

template <int SLICE>
__global__ void __launch_bounds__(kRecThreads) gdn_recurrent_kernel(const __grid_constant__ DeltaArgs a) {
    constexpr int kLanes = SLICE / 4;                 // lanes of one key row, 4 columns each
    constexpr int kSub = 32 / kLanes;                 // key rows of a warp at a time
    constexpr int kRows = kGdnDim / (kRecWarps * kSub);
    constexpr int kSlices = kGdnDim / SLICE;
    __shared__ __align__(16) float sk[2][kGdnDim], sq[2][kGdnDim];
    __shared__ __align__(16) float red[2][kRecWarps][2][SLICE];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / kSlices, slice = blockIdx.x % kSlices;
    const int b = unit / a.HV, h = unit % a.HV;
    const int kh = h / (a.HV / a.HK);
    const int len = seq_len(a.lens, b, a.n, a.status, h == 0 && slice == 0 && threadIdx.x == 0);
    if (len == 0) return;
    const int col = 4 * (lane % kLanes), sub = lane / kLanes;
    float* S = a.state + ((int64_t)unit * kGdnDim) * kGdnDim + slice * SLICE + col;
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        s[i] = *reinterpret_cast<const float4*>(S + ((i * kRecWarps + warp) * kSub + sub) * kGdnDim);
    const float alpha = expf(a.a_log[h]), dt = a.dt_bias[h];

    for (int t = 0; t < len; ++t) {
        const int buf = t & 1;
        const int64_t tok = (int64_t)b * a.n + t;
        const uint16_t* x = a.qkv + tok * a.C;
        const uint2 qr = *reinterpret_cast<const uint2*>(x + kh * kGdnDim + 4 * lane);
        const uint2 kr = *reinterpret_cast<const uint2*>(x + (a.HK + kh) * kGdnDim + 4 * lane);
        const uint2 vr = *reinterpret_cast<const uint2*>(x + (2 * a.HK + h) * kGdnDim + slice * SLICE + col);
        float decay, beta;
        gates(a.a[tok * a.ab_stride + h], a.b[tok * a.ab_stride + h], alpha, dt, decay, beta);
        decay = expf(decay);
        const float2 qa = unpack_bf16(qr.x), qb = unpack_bf16(qr.y), ka = unpack_bf16(kr.x), kb = unpack_bf16(kr.y);
        float qq = qa.x * qa.x + qa.y * qa.y + qb.x * qb.x + qb.y * qb.y;
        float kk = ka.x * ka.x + ka.y * ka.y + kb.x * kb.x + kb.y * kb.y;
        float kq = qa.x * ka.x + qa.y * ka.y + qb.x * kb.x + qb.y * kb.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            qq += __shfl_xor_sync(0xffffffffu, qq, o);
            kk += __shfl_xor_sync(0xffffffffu, kk, o);
            kq += __shfl_xor_sync(0xffffffffu, kq, o);
        }
        float4 kv = make_float4(ka.x, ka.y, kb.x, kb.y), qv = make_float4(qa.x, qa.y, qb.x, qb.y);
        float rq, rk, fu = 1.f;   // fu: a factor of k.q that is applied to u first
        if (a.l2norm ? plain_sum(qq + a.l2_eps) && plain_sum(kk + a.l2_eps) : qq < 0x1p110f && kk < 0x1p110f) {
            rq = (a.l2norm ? 1.f / sqrtf(qq + a.l2_eps) : 1.f) * a.scale;
            rk = a.l2norm ? 1.f / sqrtf(kk + a.l2_eps) : 1.f;
            kq *= rq * rk;
        } else {   // values whose squares or products FP32 does not hold: scaled by powers of two, as the chunks do
            float mq = fmaxf(fmaxf(fabsf(qv.x), fabsf(qv.y)), fmaxf(fabsf(qv.z), fabsf(qv.w)));
            float mk = fmaxf(fmaxf(fabsf(kv.x), fabsf(kv.y)), fmaxf(fabsf(kv.z), fabsf(kv.w)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
                mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
            }
            const int eq = scale_exponent(mq, kRowTop), ek = scale_exponent(mk, kRowTop);
            const float fq = pow2(eq), fk = pow2(ek);
            qv = make_float4(qv.x * fq, qv.y * fq, qv.z * fq, qv.w * fq);
            kv = make_float4(kv.x * fk, kv.y * fk, kv.z * fk, kv.w * fk);
            qq = qv.x * qv.x + qv.y * qv.y + qv.z * qv.z + qv.w * qv.w;
            kk = kv.x * kv.x + kv.y * kv.y + kv.z * kv.z + kv.w * kv.w;
            kq = qv.x * kv.x + qv.y * kv.y + qv.z * kv.z + qv.w * kv.w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                qq += __shfl_xor_sync(0xffffffffu, qq, o);
                kk += __shfl_xor_sync(0xffffffffu, kk, o);
                kq += __shfl_xor_sync(0xffffffffu, kq, o);
            }
            rq = (a.l2norm ? scaled_rsqrt(qq, eq, a.l2_eps) : pow2(-eq)) * a.scale;
            rk = a.l2norm ? scaled_rsqrt(kk, ek, a.l2_eps) : pow2(-ek);
            kq *= rq;
            fu = rk;
        }
        if (warp == 0) *reinterpret_cast<float4*>(&sk[buf][4 * lane]) = make_float4(kv.x * rk, kv.y * rk, kv.z * rk, kv.w * rk);
        if (warp == 1) *reinterpret_cast<float4*>(&sq[buf][4 * lane]) = make_float4(qv.x * rq, qv.y * rq, qv.z * rq, qv.w * rq);
        __syncthreads();
        float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = (i * kRecWarps + warp) * kSub + sub;
            const float k = sk[buf][r], q = sq[buf][r];
            s[i].x *= decay; s[i].y *= decay; s[i].z *= decay; s[i].w *= decay;
            pk.x = fmaf(k, s[i].x, pk.x); pk.y = fmaf(k, s[i].y, pk.y);
            pk.z = fmaf(k, s[i].z, pk.z); pk.w = fmaf(k, s[i].w, pk.w);
            pq.x = fmaf(q, s[i].x, pq.x); pq.y = fmaf(q, s[i].y, pq.y);
            pq.z = fmaf(q, s[i].z, pq.z); pq.w = fmaf(q, s[i].w, pq.w);
        }
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) {
            pk.x += __shfl_xor_sync(0xffffffffu, pk.x, o); pk.y += __shfl_xor_sync(0xffffffffu, pk.y, o);
            pk.z += __shfl_xor_sync(0xffffffffu, pk.z, o); pk.w += __shfl_xor_sync(0xffffffffu, pk.w, o);
            pq.x += __shfl_xor_sync(0xffffffffu, pq.x, o); pq.y += __shfl_xor_sync(0xffffffffu, pq.y, o);
            pq.z += __shfl_xor_sync(0xffffffffu, pq.z, o); pq.w += __shfl_xor_sync(0xffffffffu, pq.w, o);
        }
        if (sub == 0) {
            *reinterpret_cast<float4*>(&red[buf][warp][0][col]) = pk;
            *reinterpret_cast<float4*>(&red[buf][warp][1][col]) = pq;
        }
        __syncthreads();
        pk = pq = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kRecWarps; ++w) {
            const float4 x0 = *reinterpret_cast<const float4*>(&red[buf][w][0][col]);
            const float4 x1 = *reinterpret_cast<const float4*>(&red[buf][w][1][col]);
            pk.x += x0.x; pk.y += x0.y; pk.z += x0.z; pk.w += x0.w;
            pq.x += x1.x; pq.y += x1.y; pq.z += x1.z; pq.w += x1.w;
        }
        const float2 va = unpack_bf16(vr.x), vb = unpack_bf16(vr.y);
        const float4 u = make_float4(beta * (va.x - pk.x), beta * (va.y - pk.y), beta * (vb.x - pk.z), beta * (vb.y - pk.w));
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float k = sk[buf][(i * kRecWarps + warp) * kSub + sub];
            s[i].x = fmaf(k, u.x, s[i].x); s[i].y = fmaf(k, u.y, s[i].y);
            s[i].z = fmaf(k, u.z, s[i].z); s[i].w = fmaf(k, u.w, s[i].w);
        }
        if (warp == 0 && sub == 0)
            *reinterpret_cast<uint2*>(a.out + (tok * a.HV + h) * kGdnDim + slice * SLICE + col) =
                make_uint2(pack_bf16(fmaf(kq, fu * u.x, pq.x), fmaf(kq, fu * u.y, pq.y)),
                           pack_bf16(fmaf(kq, fu * u.z, pq.z), fmaf(kq, fu * u.w, pq.w)));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        *reinterpret_cast<float4*>(S + ((i * kRecWarps + warp) * kSub + sub) * kGdnDim) = s[i];
}

}  // namespace

cudaError_t launch_gdn_conv(const ConvArgs& a, cudaStream_t stream) {
    auto blocks = [&](int per_cta) { return (a.C + per_cta - 1) / per_cta; };
    if (a.n == 1) {
        const int seqs = a.B >= 256 ? 4 : (a.B >= 64 ? 2 : 1), cblocks = blocks(8 * kTokenThreads);
        const int64_t grid = (int64_t)cblocks * ((a.B + seqs - 1) / seqs);
        if (grid > 0x7fffffffll) return cudaErrorNotSupported;
        PdlLaunch l((unsigned)grid, kTokenThreads, 0, stream);
        return cudaLaunchKernelEx(&l.cfg, gdn_conv_token_kernel, a, seqs, cblocks);
    }
    const int tiles = (a.n + kConvTile - 1) / kConvTile, cblocks = blocks(4 * kConvThreads);
    const int64_t grid = (int64_t)cblocks * tiles * a.B;
    if (grid > 0x7fffffffll) return cudaErrorNotSupported;
    PdlLaunch l((unsigned)grid, kConvThreads, 0, stream);
    return cudaLaunchKernelEx(&l.cfg, gdn_conv_kernel, a, tiles, cblocks);
}

cudaError_t launch_gdn_recurrent(const DeltaArgs& a, cudaStream_t stream) {
    const int64_t units = (int64_t)a.B * a.HV;
    if (units >= 2 * (int64_t)a.sm_count) {
        PdlLaunch l((unsigned)units, kRecThreads, 0, stream);
        return cudaLaunchKernelEx(&l.cfg, gdn_recurrent_kernel<128>, a);
    }
    PdlLaunch l((unsigned)(4 * units), kRecThreads, 0, stream);
    return cudaLaunchKernelEx(&l.cfg, gdn_recurrent_kernel<32>, a);
}

}  // namespace rma
