// rma_gdn_prefill: the gated delta rule over a block of tokens, in chunks of 64 on the tensor cores.
//
// Within a chunk that starts from state S0 (key x value), with G_i the sum of the log decays g up to
// token i, k, q normalised and u_i = beta_i (v_i - S_{i-1}^T k_i e^{g_i}) the recurrence's updates:
//   (1 + A) U = diag(beta) (V - diag(e^G) K S0),  A_ij = beta_i e^{G_i - G_j} (k_i . k_j), j < i;
//   O  = scale (diag(e^G) Q S0 + P U),            P_ij = e^{G_i - G_j} (q_i . k_j), j <= i;
//   S1 = e^{G_C} S0 + sum_j e^{G_C - G_j} k_j u_j^T.
// With T = (1 + A)^-1 diag(beta), U = T (V - diag(e^G) K S0).
//
// Two launches, or for few heads both in one (gdn_joint_kernel).
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
// the smallest step.  K and Q are BF16 values, which FP16 holds exactly, once their row is scaled the same way, down to
// 2^-20 of the row's largest, and to 2^-28 of it below; the norms are factors of the rows.  Products of two pairs leave
// out lo x lo (2^-22).  The products that only reach the output (Q S0 and P U) are made of pairs as well: with the high
// parts alone, 2^-12 of each term, one output in nine was rounded to a neighbour of what FP32 gives (now 1 in 5,000).
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
// a (chunk, value head) block: T (hi and lo by turns, 8 rows each), P hi, then FP32 scalars.  All are lower triangular,
// so rows 0-31 of columns 32-63 are zeros that no product takes.  P lo stands there: its columns 0-31 in the places
// of T's, 8 rows after 8 rows, the rest in those of P hi.
constexpr int kTPBytes = 3 * kTile + 1024;
constexpr int kOffTLo = 1024, kOffP = 2 * kTile, kOffScal = 3 * kTile;
// scalars: factors of token i in W (c1), Q S0 (c2) and U' (c3); then single values: e^{G_C}, the inverse
// scales of T and P, and the bounds that the scan takes its scales from (see there)
constexpr int kC1 = 0, kC2 = 64, kC3 = 128, kEC = 192, kTS = 193, kPS = 194, kBW = 196, kBT = 197, kBS = 198;

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

// 2^x to 2^-22: as near as the pairs that its results are multiplied into, and one instruction.  (Results below 2^-126,
// flushed to 0, are decays of what has faded.)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// The warp's index, in a register that is known to be the same in all lanes: what follows from it (roles,
// barriers, rows) is computed once for the warp.
__device__ __forceinline__ int warp_index() { return __reduce_max_sync(0xffffffffu, (int)(threadIdx.x >> 5)); }

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

// four 8 x 8 matrices of 16-bit values, transposed: lane l's address takes column l & 7 of matrix l >> 3
__device__ __forceinline__ void stsm4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}
// Ask for `bytes` (a multiple of 16) at a 16-byte aligned global address to be brought into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(reinterpret_cast<uint64_t>(p)), "r"(bytes)
                 : "memory");
}
// TMA store of one box from shared memory (bulk-group completion).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(ptx::smem_u32(src))
                 : "memory");
}

// byte offset of 16-byte piece `piece` (8 values) of row `row` in an operand image
__device__ __forceinline__ int piece_at(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }
// the same of T hi
__device__ __forceinline__ int t_at(int row, int piece) { return piece_at(row, piece) + (row >> 3) * 1024; }
// where a piece of P lo stands in a (chunk, value head) block; rows 0-31 have pieces 0-3 only
__device__ __forceinline__ int p_lo_at(int row, int piece) {
    return piece < 4 ? piece_at(row, piece + 4) : kOffP + piece_at(row - 32, piece);
}

// ---------------------------------------------------------------------------
// launch 1
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kHeadsAtOnce = 4;    // value heads whose gates are computed together, one per warp
constexpr int kLd = kC + 4;        // row of a matrix that the tensor cores' fragments are read from

// Measured on one B200: 89 us for 8,192 tokens of 16 key and 32 value heads, 2,048 CTAs.  It issues in half of
// the cycles, 25,000 warp instructions a CTA; what stalls it are the group's barriers between the short phases
// (24 warps an SM, which registers and shared memory both limit) and shared memory, half of its wavefronts.
// K K^T and Q K^T by tcgen05 instead of mma.sync took the same time: the products are a small part.  So did fewer
// instructions (two FP32 values each, sums of |K| from the norms), the inverse over four warps instead of two, and
// the gates off the critical path.
//
// Two groups of four warps, each with a value head of its own at a time.
struct __align__(1024) PrepSmem {
    union {
        uint8_t kq[kKQBytes];           // operand images of K and Q
        float prod[2][kC][kC];          // then K K^T and Q K^T, 16-byte pieces permuted (prod_at)
    };
    float T[2][kC][kLd];                // A, overwritten by its inverse block by block
    float Gh[kHeadsAtOnce][kC], Gl[kHeadsAtOnce][kC];   // sums of g log2(e), as the sum of two floats
    float beta[kHeadsAtOnce][kC];
    float rk[kC], rq[kC], ks[kC];       // row factors of K and Q, sums of |K|
    float kn[kC], qn[kC];               // norms of the rows with their factors
    float tsum[2][kC], c1[2][kC], c3[2][kC];
    uint32_t tmax[2];
};
static_assert(3 * (sizeof(PrepSmem) + 2048) <= 228 * 1024, "three CTAs an SM");

__device__ __forceinline__ int prod_at(int row, int col) {
    return row * kC + ((((col >> 2) ^ ((row & 7) << 1)) << 2) | (col & 3));
}

// TF32 with FP32's precision: a value as hi + lo, products without lo x lo (2^-22)
struct Tf {
    uint32_t hi, lo;
};
// hi is rounded to 11 bits, halves away from zero, by integer operations, since the conversion instruction is a slow one
// (8 x 256 tokens of 16 and 32 heads took 3% longer with it).  The remainder has 12 bits, so cutting it to 11 errs no
// more than rounding it would, and it keeps a NaN a NaN: hi turns the NaN of FP32 arithmetic, all ones, into a zero.
__device__ __forceinline__ Tf tf_split(float x) {
    Tf t;
    t.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    t.lo = __float_as_uint(x - __uint_as_float(t.hi)) & 0xffffe000u;
    return t;
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d += A[16 x 8] B[8 x 8], A's rows kLd floats apart, B as fragment: b0 = B[lane % 4][lane / 4], b1 four rows on
struct Acc {   // the products of the high parts, and the two corrections
    float d[4], u[4], v[4];
    __device__ __forceinline__ Acc() {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = u[i] = v[i] = 0.f;
    }
    __device__ __forceinline__ void sum(float (&r)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = d[i] + (u[i] + v[i]);
    }
};
__device__ __forceinline__ void mma_fp32(Acc& acc, const float* A, float b0, float b1, int lane) {
    const float* p = A + (lane >> 2) * kLd + (lane & 3);
    const Tf a0 = tf_split(p[0]), a1 = tf_split(p[8 * kLd]), a2 = tf_split(p[4]), a3 = tf_split(p[8 * kLd + 4]);
    const Tf c0 = tf_split(b0), c1 = tf_split(b1);
    mma_tf32(acc.u, a0.lo, a1.lo, a2.lo, a3.lo, c0.hi, c1.hi);
    mma_tf32(acc.v, a0.hi, a1.hi, a2.hi, a3.hi, c0.lo, c1.lo);
    mma_tf32(acc.d, a0.hi, a1.hi, a2.hi, a3.hi, c0.hi, c1.hi);
}
// rows 8 half .. of a 16 x 8 accumulator, as a B fragment
__device__ __forceinline__ void as_b(const float (&d)[4], int half, int lane, float& b0, float& b1) {
    const int src = (lane & 3) * 4 + (lane >> 3);   // the lane that holds row lane % 4, column lane / 4
    const float u0 = __shfl_sync(0xffffffffu, half ? d[2] : d[0], src), u1 = __shfl_sync(0xffffffffu, half ? d[3] : d[1], src);
    const float v0 = __shfl_sync(0xffffffffu, half ? d[2] : d[0], src + 16), v1 = __shfl_sync(0xffffffffu, half ? d[3] : d[1], src + 16);
    b0 = (lane >> 2) & 1 ? u1 : u0;
    b1 = (lane >> 2) & 1 ? v1 : v0;
}
// -d to rows lane / 4 and + 8 of T
__device__ __forceinline__ void put_neg(float* T, const float (&d)[4], int lane) {
    float* t = T + (lane >> 2) * kLd + 2 * (lane & 3);
    *reinterpret_cast<float2*>(t) = make_float2(-d[0], -d[1]);
    *reinterpret_cast<float2*>(t + 8 * kLd) = make_float2(-d[2], -d[3]);
}

// T = (1 + A)^-1 in place, A strictly lower triangular 64 x 64 (zeros elsewhere); the group's four warps.
//   Diagonal blocks of 16 by substitution, a lane per column; then pairs of blocks twice over,
//   T21 = -T22 A21 T11, on the tensor cores: to 32 by a warp each, to 64 by all four, 8 columns each.
//   The product in between goes from accumulators to operands by shuffles.
__device__ __forceinline__ void invert(float (*T)[kLd], int warp, int lane, int bar) {
    const int br = lane & 3, bc = lane >> 2;   // this lane's row and column in a B fragment
    if (warp < 2) {
        const int o = 32 * warp;
        {
            const int q = o + (lane & 16), j = lane & 15;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
            for (int l = 0; l < 15; ++l)
#pragma unroll
                for (int i = l + 1; i < 16; ++i) x[i] = fmaf(-T[q + i][q + l], x[l], x[i]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) T[q + i][q + j] = x[i];
            __syncwarp();
        }
        Acc y[2], z[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int ks = nt; ks < 2; ++ks) {   // T11's columns 8 nt .. are 0 above row 8 nt
                const float* t = &T[o + 8 * ks + br][o + 8 * nt + bc];
                mma_fp32(y[nt], &T[o + 16][o + 8 * ks], t[0], t[4 * kLd], lane);
            }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            float d[4];
            y[nt].sum(d);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                float b0, b1;
                as_b(d, ks, lane, b0, b1);
                mma_fp32(z[nt], &T[o + 16][o + 16 + 8 * ks], b0, b1, lane);
            }
        }
        __syncwarp();   // A21 has been read
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            float e[4];
            z[nt].sum(e);
            put_neg(&T[o + 16][o + 8 * nt], e, lane);
        }
    }
    ptx::named_bar_sync(bar, 128);
    {
        const int n0 = 8 * warp;
        float d[2][4];
        {
            Acc y[2];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                if (ks >= warp) {
                    const float* t = &T[8 * ks + br][n0 + bc];
                    const float b0 = t[0], b1 = t[4 * kLd];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) mma_fp32(y[mt], &T[32 + 16 * mt][8 * ks], b0, b1, lane);
                }
            y[0].sum(d[0]);
            y[1].sum(d[1]);
        }
        ptx::named_bar_sync(bar, 128);   // A21 has been read
        Acc z[2];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            float b0, b1;
            as_b(d[ks >> 1], ks & 1, lane, b0, b1);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
                if (ks < 2 * mt + 2) mma_fp32(z[mt], &T[32 + 16 * mt][32 + 8 * ks], b0, b1, lane);
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float e[4];
            z[mt].sum(e);
            put_neg(&T[32 + 16 * mt][n0], e, lane);
        }
    }
    ptx::named_bar_sync(bar, 128);
}

// Item `item` (chunk, sequence, key head) by 256 threads, all of a CTA's or a slot's, `tid` and `warp` among them.
// Named barriers: kAlone 1 and 2, otherwise three from bar0 on.
template <bool kAlone>
__device__ __forceinline__ void prep_item(const DeltaArgs& a, PrepSmem& s, int NC, uint32_t item, int tid, int warp, int bar0) {
    const int lane = tid & 31;
    auto sync = [&] {
        if constexpr (kAlone) __syncthreads();
        else ptx::named_bar_sync(bar0, kPrepThreads);
    };
    const int kh = item % (uint32_t)a.HK;
    const int b = (item / (uint32_t)a.HK) % (uint32_t)a.B;
    const int c = item / (uint32_t)a.HK / (uint32_t)a.B;
    const int len = seq_len(a.lens, b, a.n, a.status, c == 0 && kh == 0 && tid == 0);
    const int t0 = c * kC;
    const int valid = min(len - t0, kC);
    if (valid <= 0) return;
    const int R = a.HV / a.HK;
    uint8_t* kq_out = a.ws + (((int64_t)b * a.HK + kh) * NC + c) * kKQBytes;
    uint8_t* tp_base = a.ws + (int64_t)a.B * a.HK * NC * kKQBytes;

    // gates of up to kHeadsAtOnce value heads from r0, a warp each: two tokens a lane, running sums in FP64
    auto head_gates = [&](int r0) {
        if (warp >= kHeadsAtOnce || r0 + warp >= R) return;
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
        // sums of g log2(e): decays are powers of two from here on
        const double e0 = (double)g[0] * 1.4426950408889634, e1 = (double)g[1] * 1.4426950408889634, own = e0 + e1;
        double run = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
        }
        const double G[2] = {run - own + e0, run};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float hi = (float)G[i];
            s.Gh[warp][2 * lane + i] = hi;
            s.Gl[warp][2 * lane + i] = (float)(G[i] - (double)hi);
            s.beta[warp][2 * lane + i] = bt[i];
        }
    };

    // K and Q rows into FP16 images, eight lanes a row, with the row's norm
    {
        const int l8 = lane & 7, row0 = warp * 4 + (lane >> 3);
        uint4 raw[4][2];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int row = (it & 1) * 32 + row0;   // it >> 1: 0 K, 1 Q
            raw[it][0] = raw[it][1] = make_uint4(0, 0, 0, 0);
            if (row < valid) {
                const uint4* p = reinterpret_cast<const uint4*>(a.qkv + ((int64_t)b * a.n + t0 + row) * a.C +
                                                                ((it >> 1) ? kh : a.HK + kh) * kGdnDim) + l8;
                raw[it][0] = p[0];
                raw[it][1] = p[8];
            }
        }
        head_gates(0);
        // (the four rows of these lanes go in step, so that their shuffles overlap)
        float mx[4], ss[4], sa[4];
        auto values = [&](int it, float (&x)[16]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 p0 = unpack_bf16(raw[it][i].x), p1 = unpack_bf16(raw[it][i].y);
                const float2 p2 = unpack_bf16(raw[it][i].z), p3 = unpack_bf16(raw[it][i].w);
                x[8 * i] = p0.x; x[8 * i + 1] = p0.y; x[8 * i + 2] = p1.x; x[8 * i + 3] = p1.y;
                x[8 * i + 4] = p2.x; x[8 * i + 5] = p2.y; x[8 * i + 6] = p3.x; x[8 * i + 7] = p3.y;
            }
        };
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            float x[16];
            values(it, x);
            mx[it] = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) asm("max.abs.f32 %0, %0, %1, %2;\n" : "+f"(mx[it]) : "f"(x[i]), "f"(x[i + 1]));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
            for (int it = 0; it < 4; ++it) mx[it] = fmaxf(mx[it], __shfl_xor_sync(0xffffffffu, mx[it], o));
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int m = it >> 1, row = (it & 1) * 32 + row0;
            const float f = pow2(scale_exponent(mx[it], kRowTop));
            float x[16];
            values(it, x);
            ss[it] = 0.f;
            sa[it] = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] *= f;
                ss[it] = fmaf(x[i], x[i], ss[it]);
                sa[it] += fabsf(x[i]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = (2 * m + i) * kTile + piece_at(row, l8);
                const uint4 v = make_uint4(half2_bits(x[8 * i], x[8 * i + 1]), half2_bits(x[8 * i + 2], x[8 * i + 3]),
                                           half2_bits(x[8 * i + 4], x[8 * i + 5]), half2_bits(x[8 * i + 6], x[8 * i + 7]));
                *reinterpret_cast<uint4*>(s.kq + at) = v;
                *reinterpret_cast<uint4*>(kq_out + at) = v;
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                ss[it] += __shfl_xor_sync(0xffffffffu, ss[it], o);
                sa[it] += __shfl_xor_sync(0xffffffffu, sa[it], o);
            }
        // lanes 0-3 of the eight finish a row each
        {
            float ssr = ss[0], sar = sa[0], mxr = mx[0];
#pragma unroll
            for (int it = 1; it < 4; ++it)
                if (l8 == it) ssr = ss[it], sar = sa[it], mxr = mx[it];
            if (l8 < 4) {
                const int m = l8 >> 1, row = (l8 & 1) * 32 + row0, e = scale_exponent(mxr, kRowTop);
                const float inv = pow2(-e);
                float r = a.l2norm ? scaled_rsqrt(ssr, e, a.l2_eps) : inv;
                if (row >= valid) r = 0.f;
                if (m) {
                    r *= a.scale;
                    s.rq[row] = r;
                    s.qn[row] = fabsf(r) * sqrtf(ssr);
                } else {
                    s.rk[row] = r;
                    s.ks[row] = sar;
                    s.kn[row] = r * sqrtf(ssr);
                }
            }
        }
    }
    sync();

    // rows 16 rb .. + 15 of K K^T (warps 0-3) or Q K^T (warps 4-7), up to the diagonal block
    {
        const int rb = warp & 3, m = warp >> 2;
        float acc[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
        const uint32_t kbase = ptx::smem_u32(s.kq), abase = kbase + 2 * m * kTile;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t fa[4];
            ldsm4(abase + (ks >> 2) * kTile + piece_at(16 * rb + (lane & 15), (ks & 3) * 2 + (lane >> 4)), fa);
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                if (np <= rb) {
                    uint32_t fb[4];
                    ldsm4(kbase + (ks >> 2) * kTile +
                              piece_at(16 * np + (lane & 7) + ((lane >> 4) << 3), (ks & 3) * 2 + ((lane >> 3) & 1)), fb);
                    mma_f16(acc[2 * np], fa, fb[0], fb[1]);
                    mma_f16(acc[2 * np + 1], fa, fb[2], fb[3]);
                }
            }
        }
        sync();   // the images have been read
        float* prod = &s.prod[m][0][0];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const int row = 16 * rb + (lane >> 2), col = 8 * nt + 2 * (lane & 3);
            *reinterpret_cast<float2*>(prod + prod_at(row, col)) = make_float2(acc[nt][0], acc[nt][1]);
            *reinterpret_cast<float2*>(prod + prod_at(row + 8, col)) = make_float2(acc[nt][2], acc[nt][3]);
        }
    }
    // P is scaled by its bound, the largest norms of Q and K
    float pmax;
    {
        float q = fmaxf(s.qn[lane], s.qn[lane + 32]), k = fmaxf(s.kn[lane], s.kn[lane + 32]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, o));
            k = fmaxf(k, __shfl_xor_sync(0xffffffffu, k, o));
        }
        pmax = q * k;
    }
    const int ep = scale_exponent(pmax, 8);
    const float p_scale = pow2(ep);
    sync();

    const int grp = warp >> 2, gt = tid & 127, gw = warp & 3, bar = (kAlone ? 1 : bar0 + 1) + grp;
    for (int r0 = 0; r0 < R; r0 += kHeadsAtOnce) {
        if (r0 > 0) {
            sync();
            head_gates(r0);
            sync();
        }
        for (int r = r0 + grp; r < min(r0 + kHeadsAtOnce, R); r += 2) {
            const float *Gh = s.Gh[r - r0], *Gl = s.Gl[r - r0], *beta = s.beta[r - r0];
            uint8_t* out = tp_base + (((int64_t)b * a.HV + kh * R + r) * NC + c) * kTPBytes;
            float* scal = reinterpret_cast<float*>(out + kOffScal);
            float (*T)[kLd] = s.T[grp];
            // A (strictly below the diagonal) and P, eight columns of a row at a time.  Below the diagonal's
            // pieces e^{G_i - G_j} is the product of e^{G_i - G_r} and e^{G_r - G_j}, r the piece's last column:
            // j <= r < i, so neither exceeds 1.
            const int p = gt & 7;
            const float *k_k = &s.prod[0][0][0], *q_k = &s.prod[1][0][0];
            {
                const float rh = Gh[8 * p + 7], rl = Gl[8 * p + 7];
                float cf[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    cf[x] = s.rk[8 * p + x] * ex2((rh - Gh[8 * p + x]) + (rl - Gl[8 * p + x]));
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    const int i = (gt >> 3) + 16 * k;
                    if ((i >> 3) == p) continue;   // the diagonal's
                    float A[8], P[8];
                    if (p < (i >> 3)) {
                        const float ei = ex2((Gh[i] - rh) + (Gl[i] - rl));
                        const float fa = beta[i] * s.rk[i] * ei, fp = s.rq[i] * p_scale * ei;
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float4 kk = *reinterpret_cast<const float4*>(k_k + prod_at(i, 8 * p + 4 * y));
                            const float4 qk = *reinterpret_cast<const float4*>(q_k + prod_at(i, 8 * p + 4 * y));
                            A[4 * y] = fa * cf[4 * y] * kk.x; A[4 * y + 1] = fa * cf[4 * y + 1] * kk.y;
                            A[4 * y + 2] = fa * cf[4 * y + 2] * kk.z; A[4 * y + 3] = fa * cf[4 * y + 3] * kk.w;
                            P[4 * y] = fp * cf[4 * y] * qk.x; P[4 * y + 1] = fp * cf[4 * y + 1] * qk.y;
                            P[4 * y + 2] = fp * cf[4 * y + 2] * qk.z; P[4 * y + 3] = fp * cf[4 * y + 3] * qk.w;
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 8; ++x) A[x] = P[x] = 0.f;
                    }
                    *reinterpret_cast<float4*>(&T[i][8 * p]) = make_float4(A[0], A[1], A[2], A[3]);
                    *reinterpret_cast<float4*>(&T[i][8 * p + 4]) = make_float4(A[4], A[5], A[6], A[7]);
                    if (i >= 32 || p < 4) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) split2(P[2 * x], P[2 * x + 1], hi[x], lo[x]);
                        *reinterpret_cast<uint4*>(out + kOffP + piece_at(i, p)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(out + p_lo_at(i, p)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
            {
                const int i = gt >> 1, j0 = (i & ~7) + 4 * (gt & 1);   // half a piece of the diagonal
                const float4 kk4 = *reinterpret_cast<const float4*>(k_k + prod_at(i, j0));
                const float4 qk4 = *reinterpret_cast<const float4*>(q_k + prod_at(i, j0));
                const float kk[4] = {kk4.x, kk4.y, kk4.z, kk4.w}, qk[4] = {qk4.x, qk4.y, qk4.z, qk4.w};
                const float gh = Gh[i], gl = Gl[i], fa = beta[i] * s.rk[i], fp = s.rq[i] * p_scale;
                float A[4], P[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = j0 + x;
                    const float d = s.rk[j] * ex2((gh - Gh[j]) + (gl - Gl[j]));
                    A[x] = j < i ? fa * d * kk[x] : 0.f;
                    P[x] = j <= i ? fp * d * qk[x] : 0.f;
                }
                *reinterpret_cast<float4*>(&T[i][j0]) = make_float4(A[0], A[1], A[2], A[3]);
                uint32_t hi[2], lo[2];
                split2(P[0], P[1], hi[0], lo[0]);
                split2(P[2], P[3], hi[1], lo[1]);
                *reinterpret_cast<uint2*>(out + kOffP + piece_at(i, i >> 3) + 8 * (gt & 1)) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(out + p_lo_at(i, i >> 3) + 8 * (gt & 1)) = make_uint2(lo[0], lo[1]);
            }
            if (gt < kC) {
                const float since = ex2(Gh[gt] + Gl[gt]);
                const float until = ex2((Gh[kC - 1] - Gh[gt]) + (Gl[kC - 1] - Gl[gt]));
                scal[kC1 + gt] = s.c1[grp][gt] = since * s.rk[gt];
                scal[kC2 + gt] = since * s.rq[gt];
                scal[kC3 + gt] = s.c3[grp][gt] = until * s.rk[gt];
                if (gt == kC - 1) scal[kEC] = since;
            }
            if (gt == 0) s.tmax[grp] = 0u;
            ptx::named_bar_sync(bar, 128);
            invert(T, gw, lane, bar);
            // T with beta's columns, its rows' sums; scaled, split, to the workspace.  With normed keys no value
            // of it exceeds 1: u_i for a single x_j = 1 is beta_i k_i . (contractions) k_j beta_j.
            {
                const float4 b0 = *reinterpret_cast<const float4*>(beta + 8 * p), b1 = *reinterpret_cast<const float4*>(beta + 8 * p + 4);
                float tmax = 1.f;
                if (!a.l2norm) {
                    float mx = 0.f;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const float4 t0 = *reinterpret_cast<const float4*>(&T[(gt >> 3) + 16 * k][8 * p]);
                        const float4 t1 = *reinterpret_cast<const float4*>(&T[(gt >> 3) + 16 * k][8 * p + 4]);
                        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(t0.x * b0.x), fabsf(t0.y * b0.y)), fmaxf(fabsf(t0.z * b0.z), fabsf(t0.w * b0.w))));
                        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(t1.x * b1.x), fabsf(t1.y * b1.y)), fmaxf(fabsf(t1.z * b1.z), fabsf(t1.w * b1.w))));
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    if (lane == 0) atomicMax(&s.tmax[grp], __float_as_uint(mx));
                    ptx::named_bar_sync(bar, 128);
                    tmax = __uint_as_float(s.tmax[grp]);
                }
                const int e = scale_exponent(tmax, 8);
                const float sc = pow2(e);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    const int i = (gt >> 3) + 16 * k;
                    const float4 t0 = *reinterpret_cast<const float4*>(&T[i][8 * p]), t1 = *reinterpret_cast<const float4*>(&T[i][8 * p + 4]);
                    const float v[8] = {t0.x * b0.x, t0.y * b0.y, t0.z * b0.z, t0.w * b0.w, t1.x * b1.x, t1.y * b1.y, t1.z * b1.z, t1.w * b1.w};
                    float sum = 0.f;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        sum += fabsf(v[2 * x]) + fabsf(v[2 * x + 1]);
                        split2(v[2 * x] * sc, v[2 * x + 1] * sc, hi[x], lo[x]);
                    }
                    if (i >= 32 || p < 4) {   // elsewhere P lo stands
                        *reinterpret_cast<uint4*>(out + t_at(i, p)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(out + kOffTLo + t_at(i, p)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (p == 0) s.tsum[grp][i] = sum;
                }
                ptx::named_bar_sync(bar, 128);
                if (gw == 0) {
                    float bw = 0.f, bt = 0.f, bs = 0.f;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int t = lane + 32 * x;
                        bw = fmaxf(bw, s.c1[grp][t] * s.ks[t]);
                        bt = fmaxf(bt, s.tsum[grp][t]);
                        bs += s.c3[grp][t] * s.tsum[grp][t];
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        bw = fmaxf(bw, __shfl_xor_sync(0xffffffffu, bw, o));
                        bt = fmaxf(bt, __shfl_xor_sync(0xffffffffu, bt, o));
                        bs += __shfl_xor_sync(0xffffffffu, bs, o);
                    }
                    if (lane == 0) {
                        scal[kTS] = pow2(-e);
                        scal[kPS] = pow2(-ep);
                        scal[kBW] = bw;
                        scal[kBT] = bt;
                        scal[kBS] = bs * (1 << kRowTop);
                    }
                }
            }
            ptx::named_bar_sync(bar, 128);   // before the next head's A
        }
    }
}

__global__ void __launch_bounds__(kPrepThreads, 3) gdn_prep_kernel(const __grid_constant__ DeltaArgs a, int NC) {
    extern __shared__ uint8_t smem_raw[];
    PrepSmem& s = *reinterpret_cast<PrepSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    grid_dep_wait();
    grid_dep_launch();
    prep_item<true>(a, s, NC, blockIdx.x, threadIdx.x, warp_index(), 0);
}

// ---------------------------------------------------------------------------
// launch 2
//
// Bound by latency: the chunks of a head follow one another, 2.5 us each (4,900 cycles: the state's update and
// split 1,000, wait for W 500, X 680, wait for U 550, its splits 900, V and the increment 1,050), and a CTA starts and
// ends in 8 us.  Measured on one B200: 330 us for 8,192 tokens of one sequence (32 CTAs), 37 us for 8 x 256
// (256 CTAs on 148 SMs).  What shortened the chain: products issued by one elected lane of a converged
// warp (39 cycles an instruction; from a branch of one lane 103), scales from bounds that the first launch computes
// instead of maxima over the chunk, outputs left to warps of their own, registers moved to the warps that hold the
// state (other splits: 3% and 6% slower), and little code: one copy of each loop, short waits, since the instruction
// cache misses on 10% of the requests as it is.  CTAs that take several heads in turn were no faster.
// ---------------------------------------------------------------------------
constexpr int kStageTP = kKQBytes;                        // offsets in a stage
constexpr int kStageV = (kKQBytes + kTPBytes + 1023) / 1024 * 1024;   // V rows; then, in their place, the outputs
constexpr int kStageBytes = kStageV + kC * kGdnDim * 2;
constexpr int kStages = 3;
constexpr int kScanBar = kStages * kStageBytes;
constexpr int kScanMax = kScanBar + 256;                  // lane maxima: [state, V][2 halves][128]
constexpr int kScanExp = kScanMax + 2 * 2 * 128 * 4;      // exponents of scales, for the output warps: [2 chunks][S0, U][128]
constexpr int kScanSmem = kScanExp + 2 * 2 * 128 + 1024;
constexpr int kMaxOrder = 64;                             // sequences that are ordered by length
// warps 0-3 and 4-7: state, X and U, by halves; warps 8-11: outputs; warp 12 loads, warp 13 issues the products
constexpr int kWarpOut = 8, kWarpLoad = 12, kWarpMma = 13;
constexpr int kScanThreads = 512;
// registers a thread after the split, of 128 at launch: 2 x 192 + 88 + 40 = 4 x 128
constexpr int kRegsMain = 192, kRegsOut = 88, kRegsRest = 40;
static_assert(2 * kRegsMain + kRegsOut + kRegsRest <= 4 * 128, "the split must fit what the launch has");
static_assert(kScanSmem <= 227 * 1024, "shared memory per CTA");

// Tensor memory columns; a half is 64 keys of the state, or 32 tokens of the rest.  A thread overwrites
// only columns that it has read itself, and only after the products that read them are complete.
//   S   [0, 128)    per half: S0 as hi, lo (32 + 32); then the state's increment (64, FP32)
//   W   [128, 192)  per half: W (32); then the scaled U as hi, lo (16 + 16)
//   X   [192, 256)  per half: X as hi, lo (16 + 16)
//   U   [256, 320)  U by the first half's X; then U as hi, lo, hi, lo (8 each, of 16 tokens) per half
//   Q S0 [320, 384),  P U [384, 448) by the first half's U
//   [448, 480) U of the second half's tokens by their own X,  [480, 512) their P U by their own U
constexpr uint32_t kTmS = 0, kTmW = 128, kTmX = 192, kTmU = 256, kTmCols = 512;

// The accumulators: first column and width.  Products onto one accumulator follow one another without a commit and a
// wait between them, which the architecture promises to keep in order only where accumulator and shape are the same.  So
// each has one width, none shares a column with another, and products take them from here alone.
struct Accumulator {
    uint32_t column, width;
};
enum { kAccD, kAccW, kAccU, kAccQ, kAccP, kAccU2, kAccP2, kAccumulators };
constexpr Accumulator kAcc[kAccumulators] = {{kTmS, 128}, {kTmW, 64}, {kTmU, 64}, {320, 64}, {384, 64}, {448, 32}, {480, 32}};
constexpr bool disjoint() {
    for (int i = 0; i < kAccumulators; ++i) {
        if (kAcc[i].column + kAcc[i].width > kTmCols) return false;
        for (int j = 0; j < i; ++j)
            if (kAcc[i].column < kAcc[j].column + kAcc[j].width && kAcc[j].column < kAcc[i].column + kAcc[i].width) return false;
    }
    return true;
}
static_assert(disjoint(), "two accumulators share columns");
// D[tmem] (+)= A[tmem] * B, M = 128, B's rows (or columns, if transposed) in eights kStride bytes apart
template <int kA, bool kTransposed = false, uint32_t kStride = 1024>
__device__ __forceinline__ void product(uint32_t a_tmem, uint32_t b, bool add, uint32_t go) {
    ptx::mma_ts1<kStride>(kAcc[kA].column, a_tmem, b, ptx::idesc_f16_f32(128, kAcc[kA].width, false, kTransposed), add, go);
}

// named barriers: the output warps, once a chunk; a warp and the other half's, twice in all (4).  No thread passes one more
// or fewer times after it has given up on a wait than before.
constexpr int kBarOut = 1, kBarBoth = 2;

enum ScanBar {
    kbFull = 0,      // [3] the stage's loads landed (tx bytes)
    kbEmpty = 3,     // [3] 8 warps and the stores are done with the stage (and every product that reads it)
    kbS = 6,         // [2] 4 warps: their half of S0 in tensor memory, and their lane maxima
    kbX = 8,         // [2] 4 warps: X
    kbU = 10,        // [2] 4 warps: U and the scaled U
    kbO = 12,        // 4 warps: Q S0 and P U read
    kbWDone = 13,    // commits: W
    kbUDone = 14,    // [2] U of a half's tokens (and all before, Q S0 among it)
    kbDDone = 16,    // the state's increment
    kbPDone = 17,    // P U, and with it every product of the chunk
    kbDrain = 18,    // commit after the last product, also of an abandoned CTA
    kScanBars = 19
};

struct ScanMaps {
    CUtensorMap v;     // qkv as [batch n][C]: boxes of 128 columns x 64 rows, linear
    CUtensorMap out;   // out as [batch n][HV 128]: boxes of 64 columns x 64 rows, 128-byte swizzle
};

static_assert(8 * kScanBars + 8 <= kScanMax - kScanBar, "barriers, tensor memory's address and the abort flag");

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

// two FP32 operations an instruction
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 pack2(uint32_t a, uint32_t b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// the FP16 pair (hi, lo) of two values
__device__ __forceinline__ void split2(f2 v, uint32_t& hi, uint32_t& lo) {
    const float2 x = unpack2(v);
    hi = half2_bits(x.x, x.y);
    float d0, d1;   // hi - x
    asm("sub.rn.f32.f16 %0, %1, %2;\n" : "=f"(d0) : "h"((uint16_t)(hi & 0xffffu)), "f"(x.x));
    asm("sub.rn.f32.f16 %0, %1, %2;\n" : "=f"(d1) : "h"((uint16_t)(hi >> 16)), "f"(x.y));
    lo = half2_bits(-d0, -d1);
}
__device__ __forceinline__ float absmax(float m, f2 v) {
    const float2 x = unpack2(v);
    asm("max.abs.f32 %0, %0, %1, %2;\n" : "+f"(m) : "f"(x.x), "f"(x.y));
    return m;
}
// four consecutive floats of shared memory, as two pairs
__device__ __forceinline__ void lds4(const float* p, f2& a, f2& b) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    a = v.x;
    b = v.y;
}

// ptx::mbar_wait_warp in less code, of which the scan has twenty copies (8,192 tokens of 32 heads: 348 us, 395 with the
// longer form; the instruction caches).  A wait that gives up raises the CTA's abort flag, which every store looks at, and
// from which the status is set once, at the end.  kVerdict: false in all lanes if any has given up.  The clock's low word
// wraps above the limit.
template <bool kVerdict>
__device__ __forceinline__ bool scan_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    static_assert(ptx::kWaitLimitCycles < 0xffffffffll, "measured by the clock's low word");
    const uint32_t t0 = (uint32_t)clock();
    bool ok = true;
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*abort || (uint32_t)clock() - t0 > (uint32_t)ptx::kWaitLimitCycles) {
            *abort = 1;
            ok = false;
            break;
        }
    }
    if constexpr (kVerdict) return __all_sync(0xffffffffu, ok);
    __syncwarp();
    return ok;
}

// Wait, bounded as the waits on barriers are, until another CTA has set the flag.  By a whole warp, with one verdict.
__device__ __forceinline__ bool item_ready(const uint32_t* flag, volatile int* abort) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        const long long t0 = clock64();
        uint32_t v;
        while (true) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(v) : "l"(flag) : "memory");
            if (v != 0) break;
            if (*abort || clock64() - t0 > ptx::kWaitLimitCycles) {
                *abort = 1;
                ok = false;
                break;
            }
            __nanosleep(64);
        }
        asm volatile("fence.proxy.async;\n" ::: "memory");   // the loads that follow are another proxy's
    }
    return __all_sync(0xffffffffu, ok);
}

// Head `index` of `heads`, in the order (sequence, value head).  `ready`: NULL where the first launch is complete;
// otherwise a flag per item of it, which the same launch's other CTAs set.
__device__ __forceinline__ void scan_head(const DeltaArgs& a, const ScanMaps& maps, int NC, int index, int heads,
                                          const uint32_t* ready) {
    extern __shared__ uint8_t smem_raw[];
    // the same place as a shared-memory address and as a pointer
    const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (smem_base - ptx::smem_u32(smem_raw));
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kScanBar);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + kScanBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    float* maxima = reinterpret_cast<float*>(smem + kScanMax);
    int8_t* exps = reinterpret_cast<int8_t*>(smem + kScanExp);
    // More heads than multiprocessors and lengths that differ: the longest sequences' CTAs first, so that what
    // is dealt out last is short.
    const int h = index % a.HV, kh = h / (a.HV / a.HK);
    int b = index / a.HV;
    const bool ordered = a.lens && a.B > 1 && a.B <= kMaxOrder && heads > a.sm_count;
    if (!ordered && tid == 0)   // the state towards L2, before anything is waited for
        prefetch_l2(a.state + (int64_t)index * kGdnDim * kGdnDim, kGdnDim * kGdnDim * 4);
    grid_dep_wait();
    grid_dep_launch();
    if (ordered) {
        int* ls = reinterpret_cast<int*>(smem);
        if (tid < a.B) ls[tid] = seq_len(a.lens, tid, a.n, a.status, false);
        __syncthreads();
        if (tid < a.B) {
            const int mine = ls[tid];
            int rank = 0;
            for (int j = 0; j < a.B; ++j) rank += ls[j] > mine || (ls[j] == mine && j < tid);
            if (rank == b) ls[kMaxOrder] = tid;
        }
        __syncthreads();
        b = ls[kMaxOrder];
        __syncthreads();   // before the stages take this memory
        if (tid == 0) prefetch_l2(a.state + ((int64_t)b * a.HV + h) * kGdnDim * kGdnDim, kGdnDim * kGdnDim * 4);
    }
    b = __reduce_max_sync(0xffffffffu, b);   // known to be the same in all lanes
    const int unit = b * a.HV + h;
    const int len = seq_len(a.lens, b, a.n, a.status, false);
    if (len == 0) return;
    const int nc = (len + kC - 1) / kC;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&bars[kbFull + i], 1);
            ptx::mbar_init(&bars[kbEmpty + i], 9);
        }
        for (int i = kbS; i <= kbO; ++i) ptx::mbar_init(&bars[i], 4);
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
    // all of tensor memory is this CTA's, so its first column is 0: the products' operands are then constants
    constexpr uint32_t tmem = 0;

    if (warp >= kWarpLoad) {
        regs_down<kRegsRest>();
        if (warp == kWarpLoad) {
            // ---------------- loads: a stage is the chunk's K and Q, its T, P and scalars, and its V rows ----------------
            const uint8_t* kq = a.ws + ((int64_t)b * a.HK + kh) * NC * kKQBytes;
            const uint8_t* tp = a.ws + (int64_t)a.B * a.HK * NC * kKQBytes + (int64_t)unit * NC * kTPBytes;
            int issued = 0;
            for (int c = 0; c < nc; ++c) {
                const int st = c % kStages;
                if (c >= kStages && !scan_wait<true>(&bars[kbEmpty + st], (c / kStages - 1) & 1, abort_flag)) break;
                // the state and the first chunk come first: they are what the start waits for
                if (c == 1 && !scan_wait<true>(&bars[kbS], 0, abort_flag)) break;
                if (ready && !item_ready(ready + ((int64_t)c * a.B + b) * a.HK + kh, abort_flag)) break;
                issued = c + 1;
                uint8_t* stage = smem + st * kStageBytes;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(&bars[kbFull + st], kKQBytes + kTPBytes + kC * kGdnDim * 2);
                    ptx::bulk_load(stage, kq + (int64_t)c * kKQBytes, kKQBytes, &bars[kbFull + st]);
                    ptx::bulk_load(stage + kStageTP, tp + (int64_t)c * kTPBytes, kTPBytes, &bars[kbFull + st]);
                    // 64 rows, also past the sequence's end (not used) or the tensor's (zeros)
                    ptx::tma_load_2d(stage + kStageV, &maps.v, &bars[kbFull + st], (2 * a.HK + h) * kGdnDim, b * a.n + c * kC);
                }
                __syncwarp();
            }
            // what was asked for has landed before the CTA ends
            for (int c = max(0, issued - kStages); c < issued; ++c)
                ptx::mbar_wait_drain(&bars[kbFull + c % kStages], (c / kStages) & 1, a.status);
        } else if (warp == kWarpMma) {
            // ---------------- products ----------------
            // The warp computes the operands together and one elected lane issues: a branch taken by one
            // lane instead costs about 100 cycles an instruction, three times what its product takes.
            // T and P are lower triangular: the first half's tokens take the first half's rows and columns only, and
            // what the second half's add for their own goes to accumulators of its own.  An instruction takes about 39
            // cycles with 64 or 32 columns, 64 with 128.
            constexpr uint32_t kImage = kTile >> 4, kHalfRows = (32 * 128) >> 4, kHalfT = 2 * kHalfRows, kTStride = 2048, kTLo = kOffTLo >> 4, kP = kOffP >> 4;
            const uint32_t go = ptx::elect_one();
            // (The loop over the chunks is not unrolled by stage: three copies of it crowd the other roles out of
            // the instruction caches, which costs more than constant operands save.)
            for (int c = 0; c < nc; ++c) {
                const int st = c % kStages;
                const uint32_t kb = smem_base + st * kStageBytes, tb = kb + kStageTP;
                // low words of the descriptors: address and leading offset (the state's increment takes K by
                // columns).  16 values of the rows of an image are 32 bytes: 2 in the address field
                const uint32_t dk = (kb >> 4) | (1u << 16), dt = (tb >> 4) | (1u << 16), dd = (kb >> 4) | ((uint32_t)(kTile >> 4) << 16);
                auto wait = [&](int bar, int phase) {
                    const bool there = scan_wait<true>(&bars[bar], phase & 1, abort_flag);
                    ptx::tc_fence_after();
                    return there;
                };
                if (!wait(kbFull + st, c / kStages)) break;
                // the chunk before is complete: the scaled U lies where W goes
                if (c > 0 && !wait(kbPDone, c - 1)) break;
                // W, as the halves of the state arrive
                if (!wait(kbS, c)) break;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)   // hi, then lo
                    product<kAccW>(kTmS + 8 * ks, dk + 2 * (ks & 3), ks > 0, go);
                if (!wait(kbS + 1, c)) break;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    product<kAccW>(kTmS + 64 + 8 * ks, dk + kImage + 2 * (ks & 3), true, go);
                ptx::mma_commit1(&bars[kbWDone], go);
                if (c > 0 && !wait(kbO, c - 1)) break;
#pragma unroll
                for (int ks = 0; ks < 16; ++ks)   // per half of the keys: hi, then lo
                    product<kAccQ>(kTmS + 8 * ks, dk + (2 + (ks >> 3)) * kImage + 2 * (ks & 3), ks > 0, go);
                // U: the first half's X for all tokens, then the second half's for its own
                if (!wait(kbX, c)) break;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const uint32_t x = kTmX + 8 * ks, t = dt + 2 * ks;
                    product<kAccU, false, kTStride>(x, t, ks > 0, go);
                    product<kAccU, false, kTStride>(x + 16, t, true, go);
                    product<kAccU, false, kTStride>(x, t + kTLo, true, go);
                }
                ptx::mma_commit1(&bars[kbUDone], go);
                if (!wait(kbX + 1, c)) break;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const uint32_t x = kTmX + 32 + 8 * ks, t = dt + kHalfT + 4 + 2 * ks;
                    product<kAccU2, false, kTStride>(x, t, ks > 0, go);
                    product<kAccU2, false, kTStride>(x + 16, t, true, go);
                    product<kAccU2, false, kTStride>(x, t + kTLo, true, go);
                }
                ptx::mma_commit1(&bars[kbUDone + 1], go);
                // the state's increment, a half of the tokens after the other (16 rows of K are 2 KiB)
                auto increment = [&](int h) {
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        product<kAccD, true>(kTmW + 32 * h + 8 * ks, dd + 128 * (2 * h + ks), h > 0 || ks > 0, go);
                        product<kAccD, true>(kTmW + 32 * h + 16 + 8 * ks, dd + 128 * (2 * h + ks), true, go);
                    }
                };
                if (!wait(kbU, c)) break;
                increment(0);
                if (!wait(kbU + 1, c)) break;
                increment(1);
                ptx::mma_commit1(&bars[kbDDone], go);
                // P U, as U
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const uint32_t u = kTmU + 16 * ks, p = dt + kP + 2 * ks;
                    product<kAccP>(u, p, ks > 0, go);
                    product<kAccP>(u + 8, p, true, go);
                    product<kAccP>(u, dt + 4 + 2 * ks, true, go);
                }
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const uint32_t u = kTmU + 32 + 16 * ks, p = dt + kP + kHalfRows + 4 + 2 * ks;
                    product<kAccP2>(u, p, ks > 0, go);
                    product<kAccP2>(u + 8, p, true, go);
                    product<kAccP2>(u, dt + kP + 4 + 2 * ks, true, go);
                }
                ptx::mma_commit1(&bars[kbPDone], go);
            }
            ptx::mma_commit1(&bars[kbDrain], go);
            __syncwarp();
            ptx::mbar_wait_drain(&bars[kbDrain], 0, a.status);
        }
    } else if (warp >= kWarpOut) {
        regs_down<kRegsOut>();
        // ---------------- outputs: a warp's 32 lanes (value columns), read as fragments of 16 x 8 ----------------
        const int w = warp & 3, col0 = 32 * w;
        const uint32_t tl = tmem + ((uint32_t)col0 << 16);
        // stmatrix: this lane's row (a token, within two groups of 8) in the swizzled image of its 64 columns
        const int st_row = ((lane & 7) + ((lane >> 4) << 3)) * 128 + (w >> 1) * kTile;
        const int st_piece = (w & 1) * 4 + ((lane >> 3) & 1);
        for (int c = 0; c < nc; ++c) {
            const int st = c % kStages;
            uint8_t* stage = smem + st * kStageBytes;
            const float* scal = reinterpret_cast<const float*>(stage + kStageTP + kOffScal);
            const int left = len - c * kC;
            scan_wait<false>(&bars[kbFull + st], (c / kStages) & 1, abort_flag);
            scan_wait<false>(&bars[kbU], c & 1, abort_flag);   // the scales
            const float inv_p = scal[kPS];
            scan_wait<false>(&bars[kbPDone], c & 1, abort_flag);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int hl = 0; hl < 2; ++hl) {            // 16 columns
                f2 is[2], iu[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int8_t* e = exps + (c & 1) * 256 + col0 + 16 * hl + 8 * r + (lane >> 2);
                    const float fs = pow2(-(int)e[0]), fu = pow2(-(int)e[128]) * inv_p;
                    is[r] = pack2(fs, fs);
                    iu[r] = pack2(fu, fu);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) {           // 32 tokens
                    uint32_t q[16], y[16], o[8];
                    ptx::tmem_ld_frag4(tl + ((uint32_t)(16 * hl) << 16) + kAcc[kAccQ].column + 32 * p, q);
                    ptx::tmem_ld_frag4(tl + ((uint32_t)(16 * hl) << 16) + kAcc[kAccP].column + 32 * p, y);
                    if (p == 1) {                       // by both halves' U
                        uint32_t z[16];
                        ptx::tmem_ld_frag4(tl + ((uint32_t)(16 * hl) << 16) + kAcc[kAccP2].column, z);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) + __uint_as_float(z[i]));
                    }
                    ptx::tmem_wait_ld();
                    if (hl == 1 && p == 1) {            // Q S0 and P U are read
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&bars[kbO]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f2 c2 = *reinterpret_cast<const f2*>(scal + kC2 + 32 * p + 8 * j + 2 * (lane & 3));
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const f2 x = mul2(pack2(q[4 * j + 2 * r], q[4 * j + 2 * r + 1]), mul2(c2, is[r]));
                            const float2 v = unpack2(fma2(pack2(y[4 * j + 2 * r], y[4 * j + 2 * r + 1]), iu[r], x));
                            o[2 * j + r] = pack_bf16(v.x, v.y);
                        }
                    }
                    const uint32_t to = ptx::smem_u32(stage + kStageV) + st_row + 32 * p * 128 +
                                        (((st_piece + 2 * hl) ^ (lane & 7)) << 4);
                    stsm4_trans(to, o[0], o[1], o[2], o[3]);
                    stsm4_trans(to + 16 * 128, o[4], o[5], o[6], o[7]);
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::named_bar_sync(kBarOut, 128);
            if (*abort_flag) {
                // a wait has given up: what stands in the stage is nobody's output
            } else if (left >= kC) {
                if (warp == kWarpOut && lane < 2) {
                    tma_store_2d(&maps.out, stage + kStageV + lane * kTile, h * kGdnDim + 64 * lane, b * a.n + c * kC);
                    ptx::bulk_commit();
                    ptx::bulk_wait_read_all();
                }
            } else {   // the last chunk: rows past the sequence's end stay as they are
                for (int i = tid - 32 * kWarpOut; i < 16 * left; i += 128) {
                    const int t = i >> 4, piece = i & 15;
                    const uint4 x = *reinterpret_cast<const uint4*>(stage + kStageV + (piece >> 3) * kTile + piece_at(t, piece & 7));
                    *reinterpret_cast<uint4*>(a.out + (((int64_t)b * a.n + c * kC + t) * a.HV + h) * kGdnDim + 8 * piece) = x;
                }
            }
            __syncwarp();
            if (warp == kWarpOut && lane == 0) ptx::mbar_arrive(&bars[kbEmpty + st]);
        }
    } else {
        regs_up<kRegsMain>();
        // ---------------- a thread: lane (value column) `row`, half `wg` of the keys or tokens ----------------
        // The halves run one behind the other, so that one's arithmetic covers the other's products.
        const int wg = warp >> 2, w = warp & 3, row = 32 * w + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * w) << 16);
        auto signal = [&](int bar) {
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars[bar + wg]);
        };
        // this half's largest values of the lane's state and V, offered to the other half and taken from it.  What the
        // other half has offered for a chunk is there when its state is (kbS): a bounded wait, as all that stand
        // between the chunks.  (By named barriers, two arrivals of a warp that has given up on its waits could complete
        // one without the other half's warp, which would then wait for good.)
        auto offer = [&](float ms, float mv) {
            maxima[wg * 128 + row] = ms;
            maxima[(2 + wg) * 128 + row] = mv;
        };
        auto take = [&](float& ms, float& mv) {
            ms = fmaxf(ms, maxima[(wg ^ 1) * 128 + row]);
            mv = fmaxf(mv, maxima[(2 + (wg ^ 1)) * 128 + row]);
        };
        // this half's V rows of chunk c
        f2 v[16];
        auto get_v = [&](int c) {
            const uint16_t* vs = reinterpret_cast<const uint16_t*>(smem + (c % kStages) * kStageBytes + kStageV) + 32 * wg * kGdnDim + row;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = pack2(bf16_float(vs[2 * i * kGdnDim]), bf16_float(vs[(2 * i + 1) * kGdnDim]));
            const int left = len - c * kC - 32 * wg;
            if (left < 32) {   // tokens past the end, whatever stands there (their K is 0, so their X will be)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 d = unpack2(v[i]);
                    v[i] = pack2(2 * i < left ? d.x : 0.f, 2 * i + 1 < left ? d.y : 0.f);
                }
            }
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 16; ++i) m[i & 1] = absmax(m[i & 1], v[i]);
            return fmaxf(m[0], m[1]);
        };
        // The lane's scales are powers of two from bounds on its values, all known before the products they
        // are for: of the state at the start (its own maximum), of X (V and the keys' sums), of U and the
        // state at the end (X and T's sums).  A bound may be some binades loose: the pairs reach 2^-39 of it.
        f2 S[32];   // times 2^es: keys 64 wg + 2 i, 2 i + 1
        int es;
        float* gs = a.state + ((int64_t)unit * kGdnDim + 64 * wg) * kGdnDim + row;
        float smax = 0.f, vmax = 0.f;
        {
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = pack2(gs[2 * i * kGdnDim], gs[(2 * i + 1) * kGdnDim]);
#pragma unroll
            for (int i = 0; i < 32; ++i) smax = absmax(smax, S[i]);
            offer(smax, 0.f);
            ptx::named_bar_sync(kBarBoth + w, 64);
            take(smax, vmax);
            ptx::named_bar_sync(kBarBoth + w, 64);   // both have taken, before the next offer
            es = scale_exponent(smax, 15);
            smax *= pow2(es);   // scaled, as the state is
            const f2 f = pack2(pow2(es), pow2(es));
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = mul2(S[i], f);
        }
        constexpr float kCap = 1.2676506e30f;   // 2^100: a factor beyond it multiplies a zero, and must not be infinite
        // Step -1 only brings the state and the first V in.
#pragma unroll 1
        for (int c = -1; c < nc; ++c) {
          uint32_t x[32];
          float ck = 1.f;
          int es1 = es;
          if (c >= 0) {
            const int st = c % kStages;
            const float* one = reinterpret_cast<const float*>(smem + st * kStageBytes + kStageTP + kOffScal);
            const float* scal = one + 32 * wg;   // this half's tokens
            // while W is computed: the bounds and the scales
            scan_wait<false>(&bars[kbS + (wg ^ 1)], c & 1, abort_flag);
            take(smax, vmax);
            const float inv_s = pow2(-es);
            smax *= inv_s;
            const float keep = one[kEC], bx = fmaf(one[kBW], smax, vmax);
            const int ex = scale_exponent(bx, 15), eu = scale_exponent(one[kBT] * bx, 15);
            es1 = scale_exponent(fmaf(one[kBS], bx, keep * smax), 15);
            const float fx = pow2(ex), from_x = pow2(-ex) * one[kTS];
            const float cw = -fminf(inv_s * fx, kCap);                // W to X's scale
            const float cu = fminf(pow2(eu) * from_x, kCap);          // U's accumulator to U's scale
            const float cd = fminf(pow2(es1) * from_x, kCap);         // and, with c3, to the new state's
            ck = fminf(keep * inv_s * pow2(es1), kCap);               // the state to its new scale
            if (wg == 0) exps[(c & 1) * 256 + 128 + row] = (int8_t)eu;
            {
                const f2 f = pack2(fx, fx);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], f);
            }
            // X
            // (an abandoned CTA goes on through its barriers, on values that nobody uses)
            scan_wait<false>(&bars[kbWDone], c & 1, abort_flag);
            ptx::tc_fence_after();
            ptx::tmem_ld32(tl + kTmW + 32 * wg, x);
            ptx::tmem_wait_ld();
            {
                const f2 cw2 = pack2(cw, cw);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    f2 c1[2];
                    lds4(scal + kC1 + 2 * i, c1[0], c1[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        split2(fma2(pack2(x[2 * (i + j)], x[2 * (i + j) + 1]), mul2(c1[j], cw2), v[i + j]), hi[i + j], lo[i + j]);
                }
                ptx::tmem_st16(tl + kTmX + 32 * wg, hi);
                ptx::tmem_st16(tl + kTmX + 32 * wg + 16, lo);
                signal(kbX);
            }
            // U, and U scaled for the state
            scan_wait<false>(&bars[kbUDone + wg], c & 1, abort_flag);
            ptx::tc_fence_after();
            {
                const f2 cu2 = pack2(cu, cu), cd2 = pack2(cd, cd);
#pragma unroll 1
                for (int p = 0; p < 2; ++p) {
                    uint32_t u[16], hi[8], lo[8];
                    ptx::tmem_ld16(tl + kTmU + 32 * wg + 16 * p, u);
                    if (wg == 1) {   // by both halves' X
                        uint32_t y[16];
                        ptx::tmem_ld16(tl + kAcc[kAccU2].column + 16 * p, y);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(y[i]));
                    } else {
                        ptx::tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        f2 c3[2];
                        lds4(scal + kC3 + 16 * p + 2 * i, c3[0], c3[1]);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            split2(mul2(pack2(u[2 * (i + j)], u[2 * (i + j) + 1]), mul2(c3[j], cd2)), hi[i + j], lo[i + j]);
                    }
                    ptx::tmem_st8(tl + kTmW + 32 * wg + 8 * p, hi);
                    ptx::tmem_st8(tl + kTmW + 32 * wg + 16 + 8 * p, lo);
#pragma unroll
                    for (int i = 0; i < 8; ++i) split2(mul2(pack2(u[2 * i], u[2 * i + 1]), cu2), hi[i], lo[i]);
                    ptx::tmem_st8(tl + kTmU + 32 * wg + 16 * p, hi);
                    ptx::tmem_st8(tl + kTmU + 32 * wg + 16 * p + 8, lo);
                }
                signal(kbU);
            }
            if (lane == 0) ptx::mbar_arrive(&bars[kbEmpty + st]);   // (the output warps wait for the products)
          }
            // while the increment is computed: the next chunk's V
            if (c + 1 < nc) {
                scan_wait<false>(&bars[kbFull + (c + 1) % kStages], ((c + 1) / kStages) & 1, abort_flag);
                vmax = get_v(c + 1);
            }
            // the state
            if (c >= 0) {
                scan_wait<false>(&bars[kbDDone], c & 1, abort_flag);
                ptx::tc_fence_after();
                es = es1;
                const f2 k2 = pack2(ck, ck);
                float m[2] = {0.f, 0.f};
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    ptx::tmem_ld32(tl + kTmS + 64 * wg + 32 * p, x);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        S[16 * p + i] = fma2(S[16 * p + i], k2, pack2(x[2 * i], x[2 * i + 1]));
                        m[i & 1] = absmax(m[i & 1], S[16 * p + i]);
                    }
                }
                smax = fmaxf(m[0], m[1]);
            }
            if (c + 1 < nc) {
                offer(smax, vmax);
                if (wg == 0) exps[((c + 1) & 1) * 256 + row] = (int8_t)es;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) split2(S[16 * p + i], hi[i], lo[i]);
                    ptx::tmem_st16(tl + kTmS + 64 * wg + 16 * p, hi);
                    ptx::tmem_st16(tl + kTmS + 64 * wg + 32 + 16 * p, lo);
                }
                signal(kbS);
            }
        }
        if (*abort_flag == 0) {   // no wait of this CTA has given up
            const float f = pow2(-es);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float2 y = unpack2(S[i]);
                gs[2 * i * kGdnDim] = y.x * f;
                gs[(2 * i + 1) * kGdnDim] = y.y * f;
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWarpMma) ptx::tmem_dealloc1(tmem, kTmCols);
    if (tid == 0 && *abort_flag) atomicOr(a.status, (unsigned)RMA_STATUS_TIMEOUT);
}

__global__ void __launch_bounds__(kScanThreads, 1) gdn_scan_kernel(const __grid_constant__ DeltaArgs a,
                                                                   const __grid_constant__ ScanMaps maps, int NC) {
    scan_head(a, maps, NC, blockIdx.x, gridDim.x, nullptr);
}

// ---------------------------------------------------------------------------
// Both in one launch, for few heads and many chunks: a CTA an SM, the first ones the heads of launch 2, the others two
// items at a time of launch 1, chunk by chunk.  A finished item sets its flag, and a head's loads wait for it.  The
// launch is cooperative, so that all CTAs are there, and those that are waited for do not wait themselves.
//
// Measured on one B200, 16 key and 32 value heads: 348 us for 8,192 tokens (419 in two launches), 107 (115) for 2,048;
// two sequences of 4,096 tokens 206 (257).
// ---------------------------------------------------------------------------
constexpr int kPrepSlot = (sizeof(PrepSmem) + 1023) / 1024 * 1024;
static_assert(2 * kPrepThreads == kScanThreads && 2 * kPrepSlot + 1024 <= kScanSmem, "two items in a CTA of the scan's size");

__global__ void __launch_bounds__(kScanThreads, 1) gdn_joint_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ ScanMaps maps,
                                                                    int NC, uint32_t* ready) {
    extern __shared__ uint8_t smem_raw[];
    const int heads = a.B * a.HV, workers = gridDim.x - heads;
    grid_dep_launch();
    // The heads first: the first CTAs of a launch are placed in pairs on neighbours, far from the other pairs, and take
    // 4,200 cycles a chunk (4,500 beside the others' work).  On every other SM they took up to 5,700.
    if ((int)blockIdx.x < heads) {
        scan_head(a, maps, NC, blockIdx.x, heads, ready);
        return;
    }
    const int index = blockIdx.x - heads;
    const int w = warp_index(), slot = w >> 3, tid = threadIdx.x & (kPrepThreads - 1);
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PrepSmem& s = *reinterpret_cast<PrepSmem*>(base + slot * kPrepSlot);
    const int items = NC * a.B * a.HK;
    const int bar0 = 1 + 3 * slot;
    for (int item = index + slot * workers; item < items; item += 2 * workers) {
        prep_item<false>(a, s, NC, item, tid, w & 7, bar0);
        ptx::named_bar_sync(bar0, kPrepThreads);   // also before the next item's shared memory
        if (tid == 0) asm volatile("st.release.gpu.global.u32 [%0], %1;\n" ::"l"(ready + item), "r"(1u) : "memory");
    }
}

// A 2-D BF16 tensor of `rows` rows of `cols` values, boxes of bc columns x 64 rows.
bool make_map2(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t bc, CUtensorMapSwizzle swizzle) {
    TensorMapEncodeFn fn = tensor_map_encode();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * 2};
    const cuuint32_t box[2] = {bc, kC};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// the operands, then a flag per item
static size_t operand_bytes(size_t NC, size_t B, size_t HK, size_t HV) {
    return (NC * B * (HK * kKQBytes + HV * kTPBytes) + 255) / 256 * 256;
}

size_t gdn_prefill_workspace_bytes(const rma_gdn_config& c, int n) {
    if (n < kGdnChunkedFrom) return 256;
    const size_t NC = (n + kC - 1) / kC;
    return operand_bytes(NC, c.batch, c.n_k_heads, c.n_v_heads) + (NC * c.batch * c.n_k_heads * 4 + 255) / 256 * 256;
}

// Heads on at most half of the multiprocessors, 32 chunks or more, and the others keep ahead of the heads: an item
// with two value heads takes 12 us, two items at a time a CTA, a chunk of the scan 2.5 us.  And more items than launch 1
// runs at once, three an SM, since with fewer it is over in the time of one: 2,048 tokens of 8 and 16 heads (256 items)
// 104 us here, 100 in two launches, 8,192 of 2 and 4 (256) 344 and 342; 2,048 of 16 and 16 (512) 102 and 108, 8,192 of 4
// and 4 (512) 342 and 352.
static bool in_one_launch(const DeltaArgs& a, int NC) {
    const int heads = a.B * a.HV, rest = a.sm_count - heads;
    return NC >= 32 && (int64_t)NC * a.B * a.HK > 3 * a.sm_count && rest >= heads && 5ll * a.B * a.HK * ((a.HV / a.HK + 1) / 2) <= 2 * rest;
}

cudaError_t launch_gdn_prefill(const DeltaArgs& a, cudaStream_t stream) {
    const bool few = (int64_t)a.B * a.HV * 4 <= a.sm_count;
    if (a.n < (few ? kGdnChunkedFromFew : kGdnChunkedFrom)) return launch_gdn_recurrent(a, stream);
    const int NC = (a.n + kC - 1) / kC;
    const int64_t grid = (int64_t)NC * a.B * a.HK;
    if (grid > 0x7fffffffll) return cudaErrorNotSupported;
    const size_t prep_smem = sizeof(PrepSmem) + 1024;
    static SmemLimit prep_limit(reinterpret_cast<const void*>(gdn_prep_kernel));
    static SmemLimit scan_limit(reinterpret_cast<const void*>(gdn_scan_kernel));
    cudaError_t e = prep_limit.ensure(prep_smem);
    if (e == cudaSuccess) e = scan_limit.ensure(kScanSmem);
    if (e != cudaSuccess) return e;
    ScanMaps maps;
    const uint64_t rows = (uint64_t)a.B * a.n;
    if (!make_map2(&maps.v, a.qkv, a.C, rows, kGdnDim, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map2(&maps.out, a.out, (uint64_t)a.HV * kGdnDim, rows, 64, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (in_one_launch(a, NC)) {
        static SmemLimit joint_limit(reinterpret_cast<const void*>(gdn_joint_kernel));
        e = joint_limit.ensure(kScanSmem);
        if (e != cudaSuccess) return e;
        uint32_t* ready = reinterpret_cast<uint32_t*>(a.ws + operand_bytes(NC, a.B, a.HK, a.HV));
        e = cudaMemsetAsync(ready, 0, grid * 4, stream);
        if (e != cudaSuccess) return e;
        PdlLaunch l((unsigned)a.sm_count, kScanThreads, kScanSmem, stream);
        l.attr[0].id = cudaLaunchAttributeCooperative;
        l.attr[0].val.cooperative = 1;
        e = cudaLaunchKernelEx(&l.cfg, gdn_joint_kernel, a, maps, NC, ready);
        if (e != cudaErrorCooperativeLaunchTooLarge) return e;
        cudaGetLastError();   // a context that has not all of the device's multiprocessors
    }
    PdlLaunch prep((unsigned)grid, kPrepThreads, prep_smem, stream);
    e = cudaLaunchKernelEx(&prep.cfg, gdn_prep_kernel, a, NC);
    if (e != cudaSuccess) return e;
    PdlLaunch scan((unsigned)(a.B * a.HV), kScanThreads, kScanSmem, stream);
    return cudaLaunchKernelEx(&scan.cfg, gdn_scan_kernel, a, maps, NC);
}

}  // namespace rma
