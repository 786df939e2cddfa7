// The gated delta rule on gfx950 matrix cores, chunk by chunk.
//
// Per batch row and head, with a (P x N) state S, keys k, queries q, values v,
// the step's decay a_t = exp(dt_t A) and the write strength beta_t:
//
//   S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T,   y_t = S_t q_t
//
// For a chunk of C = 64 tokens that starts at state S, with G_i the running
// sum of log a inside the chunk and Gam_ij = exp(G_i - G_j) for i >= j:
//
//   E = strictly lower part of (K K^T * Gam),   R = (I + diag(beta) E)^-1
//   X = V - exp(G) K S^T,   U = R (beta X)             (C x P: what is written)
//   Y = exp(G) Q S^T + lower part of (Q K^T * Gam) U
//   S' = exp(G_C) S + (exp(G_C - G) U)^T K
//
// and backwards from dY and D' = dL/dS':
//
//   dU = (lower part of (Q K^T * Gam))^T dY + exp(G_C - G) K D'^T
//   W = R^T dU,   dV = beta W
//   D = exp(G_C) D' + (exp(G) dY)^T Q - (exp(G) beta W)^T K
//   dq = exp(G) dY S + (dY U^T * Gam) K
//   dk = [row] -exp(G) beta W S - (beta W U^T * Gam) K
//      + [col] exp(G_C - G) U D' + (dY U^T * Gam)^T Q - (beta W U^T * Gam)^T K
//   dbeta_i = W_i . V_i - exp(G_i) k_i . (W S)_i - sum_{j<i} E_ij W_i . U_j
//   d(log a_t) = exp(G_C) <D', S>
//      + sum_{j<t} exp(G_C - G_j) k_j . (U D')_j
//      + sum_{i>=t} exp(G_i) (q_i . (dY S)_i - beta_i k_i . (W S)_i)
//      + sum_{i>=t>j} ((dY U^T)_ij (Q K^T * Gam)_ij - (beta W U^T)_ij E_ij)
//
// Every term of the last sum has exp(log a_t) as a factor, and so has what its
// rounding leaves. (Shorter is <D', S'> + sum_{i>=t} (q_i . dq_i + k_i . row_i -
// k_i . col_i), but its terms do not have that factor and cancel: a decay of
// exp(-16) would keep no digit.)
//
// Keys and queries of unit length are rows scaled by rk, rq: the scales (and
// the query scale) ride on the fp32 tables, so that K and Q stay exact bf16
// operands.
//
// What is fp32 stays fp32 through the matrix cores: a computed operand is
// split into three bf16 parts (24 significant bits) and products of parts
// below 2^-24 are left out, so a state or a parameter's gradient is as exact
// as fp32 arithmetic gives it, and a bf16 output is rounded once, from that.
//
// Kernels:
//  * gdr_prep_kernel, one workgroup per chunk and head, every chunk at once:
//    the tables, R (16 x 16 diagonal blocks by substitution, the blocks below
//    by fp32 MFMA) and the decayed scores.
//  * gdr_fwd_kernel / gdr_rev_kernel walk the chunks forwards / backwards. A
//    column p of the state depends on no other, and a wave holds 16 columns of
//    S^T as MFMA accumulators (lane = column, 4 consecutive n). Every product
//    contracts over tokens or n, and an accumulator is the next product's
//    operand in the same lane (the contraction index runs in the order in
//    which a lane holds it), so a wave never exchanges data with another.
//  * gdr_grad_kernel, one workgroup per chunk and group of heads, every chunk
//    at once: dq, dk, dbeta and the decay's gradient from the stored S, D', U
//    and W; gdr_reduce_kernel adds dA and ddt_bias in a fixed order.
#pragma once

#include "matrix_ops.hpp"
#include "scan_kernels.hpp"

namespace ssm_detail {

constexpr int kGdrC = 64;         // tokens per chunk
constexpr int kGdrTiles = 10;     // lower 16 x 16 tiles of a chunk's C x C matrices
constexpr int kGdrTab = 13;       // fp32 tables per token and head
enum GdrTable {
    kTHk, kTHq, kTTk, kTBeta,     // exp(G) rk, exp(G) rq, exp(G_C - G) rk, beta
    kTHead, kTGhi, kTGlo,         // exp(G); G / ln 2 as a sum of two floats
    kTRk, kTRq, kTUq,             // rk, rq * scale, rq alone
    kTStep, kTDstep, kTDbeta      // the step, d step / d dt, d strength / d beta
};

struct GdrParams {
    const uint16_t *q, *k, *v, *dt, *beta, *dy;   // bf16 bit patterns
    const float *A, *dt_bias, *h0, *dh_last;
    uint16_t *y, *dq, *dk, *dv, *ddt, *dbeta;
    float *h_last, *dA, *ddt_bias, *dh0;
    // workspace
    float *tab;            // (bh, chunk, table, token)
    float *R, *score;      // (bh, chunk, tile, 16, 16)
    float *S, *D;          // (bh, chunk, P, N): S at the chunk's start, D' at its end
    float *U, *W;          // (bh, chunk, P, token)
    float *part;           // (bh, chunk, 2): the chunk's dA and ddt_bias
    int64_t qs, ks, vs, dts, bs;   // elements between tokens
    int64_t L;
    int nc, batch, H, G, hpg, P;
    int dt_softplus, beta_sigmoid, qk_norm;
    float scale, qk_eps;
};

// With fewer than 8 computing waves a workgroup of the kernels that walk the chunks
// has as many helpers, which do the staging: a computing wave's time per chunk is
// then its own arithmetic. With 8 (two to a SIMD) there are no registers for
// helpers, and the two waves of a SIMD stage at different times instead.
constexpr int gdr_helpers(int nw) { return nw < 8 ? nw : 0; }

#ifdef SSM_GDR_INSTANTIATE

constexpr int kGdrPad = 8;                 // LDS row padding of K, Q (elements)
constexpr int kGdrRS = kGdrC + 4;          // LDS row stride of C x C operands: 8-byte reads down a column of rows free of conflicts
constexpr int kGdrPlane = kGdrC * kGdrRS;  // one bf16 part of one
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ ssd_f32x4 gdr_zero4() { return ssd_f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }

// a and b rounded to a bf16 pair, and what the rounding left of them (exact). The
// pair is opaque to the compiler, which would otherwise round a once more, alone,
// to take it apart (a tenth of the walks' vector instructions). Remainders by
// dot products of the pair with (-1, 0) and (0, -1) would be 2 instructions less
// per pair, and measured the same.
__device__ __forceinline__ uint32_t gdr_take(float &a, float &b) {
    uint32_t pair = ssd_pack(a, b);
    asm("" : "+v"(pair));
    a -= __uint_as_float(pair << 16);
    b -= __uint_as_float(pair & 0xffff0000u);
    return pair;
}

// v as PARTS bf16 operands whose sum carries 8 PARTS significant bits
template <int PARTS> struct GdrSplit { ssd_bf16x8 part[PARTS]; };

template <int PARTS>
__device__ __forceinline__ GdrSplit<PARTS> gdr_split(const float (&v)[8]) {
    GdrSplit<PARTS> out;
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = k + 1 < PARTS ? gdr_take(r[2 * e], r[2 * e + 1]) : ssd_pack(r[2 * e], r[2 * e + 1]);
        }
        out.part[k] = __builtin_bit_cast(ssd_bf16x8, uint4{w[0], w[1], w[2], w[3]});
    }
    return out;
}

template <int PARTS>
__device__ __forceinline__ GdrSplit<PARTS> gdr_split(const ssd_f32x4 &a, const ssd_f32x4 &b) {
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return gdr_split<PARTS>(v);
}

// products of parts i, j with i + j < max(PA, PB): the others are below the
// last bit that the parts carry. Small products first.
template <int PA, int PB>
__device__ __forceinline__ ssd_f32x4 gdr_mfma(const GdrSplit<PA> &a, const GdrSplit<PB> &b, ssd_f32x4 c) {
    constexpr int M = PA > PB ? PA : PB;
#pragma unroll
    for (int s = M - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < PA; ++i)
            if (s - i >= 0 && s - i < PB) c = ssd_mfma(a.part[i], b.part[s - i], c);
    return c;
}

__device__ __forceinline__ GdrSplit<1> gdr_whole(const ssd_bf16x8 &v) {
    GdrSplit<1> o;
    o.part[0] = v;
    return o;
}

// A row's operand whose contraction index runs as c = 32 s + 16 (e / 4) + 4 g4
// + e % 4: two 8-byte reads 16 elements apart
__device__ __forceinline__ ssd_bf16x8 gdr_ld_perm(const uint16_t *p) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    const uint2 b = *reinterpret_cast<const uint2 *>(p + 16);
    return __builtin_bit_cast(ssd_bf16x8, uint4{a.x, a.y, b.x, b.y});
}

template <int PARTS>
__device__ __forceinline__ GdrSplit<PARTS> gdr_ld_perm_parts(const uint16_t *p, int plane) {
    GdrSplit<PARTS> o;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) o.part[k] = gdr_ld_perm(p + k * plane);
    return o;
}

// A column's operand in the same order, from a row-major tile (r16: the lane's
// place in its group of 16)
__device__ __forceinline__ ssd_bf16x8 gdr_ld_col(const uint16_t *tile, int stride, int row0, int col0, int r16) {
    const uint16_t *p = tile + (row0 + (r16 >> 2)) * stride + col0 + 4 * (r16 & 3);
    return ssd_ld_tr2(p, p + 16 * stride);
}

template <int PARTS>
__device__ __forceinline__ GdrSplit<PARTS> gdr_ld_col_parts(const uint16_t *tile, int stride, int row0, int col0,
                                                           int r16, int plane) {
    GdrSplit<PARTS> o;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) o.part[k] = gdr_ld_col(tile + k * plane, stride, row0, col0, r16);
    return o;
}

// 4 floats as PARTS bf16 planes in LDS
template <int PARTS>
__device__ __forceinline__ void gdr_store_parts(uint16_t *dst, int plane, float4 v) {
    float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        const uint2 w = k + 1 < PARTS ? uint2{gdr_take(r[0], r[1]), gdr_take(r[2], r[3])}
                                      : uint2{ssd_pack(r[0], r[1]), ssd_pack(r[2], r[3])};
        *reinterpret_cast<uint2 *>(dst + k * plane) = w;
    }
}

// Sum over a row of 16 lanes, in every lane of it (DPP rotations by 8, 4, 2, 1)
template <int CTRL> __device__ __forceinline__ float gdr_add_rot(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float gdr_sum16(float v) {
    v = gdr_add_rot<0x128>(v);
    v = gdr_add_rot<0x124>(v);
    v = gdr_add_rot<0x122>(v);
    return gdr_add_rot<0x121>(v);
}

// Inclusive prefix sum over the 64 lanes in 64 bits (DPP shifts within rows of
// 16, then the row totals carried across)
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double gdr_dpp_add(double v, bool take) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROW_MASK, 0xF, false);
    const double u = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    return take ? v + u : v;
}
__device__ __forceinline__ double gdr_prefix64(double v, int lane) {
    const int r = lane & 15;
    v = gdr_dpp_add<0x111, 0xF>(v, r >= 1);
    v = gdr_dpp_add<0x112, 0xF>(v, r >= 2);
    v = gdr_dpp_add<0x114, 0xF>(v, r >= 4);
    v = gdr_dpp_add<0x118, 0xF>(v, r >= 8);
    v = gdr_dpp_add<0x142, 0xA>(v, (lane & 16) != 0);
    v = gdr_dpp_add<0x143, 0xC>(v, (lane & 32) != 0);
    return v;
}
// lane 63's value, in every lane
__device__ __forceinline__ double gdr_last64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// tile (T, J), J <= T, of a C x C lower triangular matrix
__device__ __forceinline__ constexpr int gdr_tile(int T, int J) { return T * (T + 1) / 2 + J; }

__device__ __forceinline__ int gdr_valid(const GdrParams &p, int ci) {
    return (int)min<int64_t>(kGdrC, p.L - (int64_t)ci * kGdrC);
}

// A chunk's token rows (width W elements) into LDS rows of stride `ls`; rows
// past the sequence's end read zero by the buffer's range
template <int W>
__device__ __forceinline__ void gdr_stage_rows(uint16_t *dst, int ls, const uint16_t *src, int64_t stride, int nv,
                                               int tid, int threads) {
    const __amdgpu_buffer_rsrc_t r = ssd_buffer(src, 2u * ((uint32_t)(nv - 1) * (uint32_t)stride + W));
    constexpr int PR = W / 8;
    for (int q = tid; q < kGdrC * PR; q += threads) {
        const int row = q / PR, c = 8 * (q % PR);
        // rows past the last valid one have offsets past the range
        const uint4 v = row < nv ? ssd_bload16(r, 2u * ((uint32_t)row * (uint32_t)stride + c)) : uint4{0, 0, 0, 0};
        *reinterpret_cast<uint4 *>(dst + row * ls + c) = v;
    }
}

// The step, its derivative by dt, the write strength and its derivative by beta
struct GdrStep { float step, dstep, beta, dbeta; };
__device__ __forceinline__ GdrStep gdr_step_of(float dt, float beta, float bias, int softplus, int sigmoid) {
    GdrStep o;
    const float raw = dt + bias;
    o.step = raw;
    o.dstep = 1.0f;
    if (softplus) {
        o.step = fmaxf(raw, 0.0f) + log1pf(expf(-fabsf(raw)));
        o.dstep = 1.0f / (1.0f + expf(-raw));
    }
    o.beta = beta;
    o.dbeta = 1.0f;
    if (sigmoid) {
        o.beta = 1.0f / (1.0f + expf(-beta));
        o.dbeta = o.beta * (1.0f / (1.0f + expf(beta)));
    }
    return o;
}

// ---------------------------------------------------------------------------
// Tables, R and scores of one chunk and head. Everything before the first
// barrier is independent: K and Q go to LDS, row lengths are summed from the
// pieces on their way, and wave 0 forms the step's tables while they arrive. T
// and R take the place of K and Q, so that four workgroups fit a CU (they hide
// each other's latencies, which bound this kernel).
template <int N>
__global__ __launch_bounds__(256) void gdr_prep_kernel(const GdrParams p) {
    constexpr int KS = N + kGdrPad, KI = kGdrC * N / 8 / 256, LPR = N / 8;   // lanes per row
    constexpr int TS = kGdrC + 4;          // fp32 row stride of T and R
    union Lds {
        struct { uint16_t k[kGdrC * KS], q[kGdrC * KS]; } in;
        struct { float t[kGdrC * TS], r[kGdrC * TS]; } sys;
    };
    __shared__ __attribute__((aligned(16))) Lds u;
    __shared__ __attribute__((aligned(16))) float sGh[kGdrC], sGl[kGdrC], sB[kGdrC], sRk[kGdrC], sUq[kGdrC];
    __shared__ float sHead[kGdrC], sTail[kGdrC];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int64_t id = blockIdx.x;                // (b, h) major, chunk minor
    const int ci = (int)(id % p.nc);
    const int bh = (int)(id / p.nc);
    const int b = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int nv = gdr_valid(p, ci);
    const int64_t row0 = (int64_t)b * p.L + (int64_t)ci * kGdrC;
    float *tab = p.tab + id * (kGdrTab * kGdrC);
    {
        const uint32_t ks = (uint32_t)p.ks, qs = (uint32_t)p.qs;
        const __amdgpu_buffer_rsrc_t rk =
            ssd_buffer(p.k + row0 * p.ks + (int64_t)g * N, 2u * ((uint32_t)(nv - 1) * ks + N));
        const __amdgpu_buffer_rsrc_t rq =
            ssd_buffer(p.q + row0 * p.qs + (int64_t)g * N, 2u * ((uint32_t)(nv - 1) * qs + N));
        uint4 kr[KI], qr[KI];
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const uint32_t x = i * 256 + tid, row = x / LPR, c = 8 * (x % LPR);
            kr[i] = ssd_bload16(rk, 2u * (row * ks + c));
            qr[i] = ssd_bload16(rq, 2u * (row * qs + c));
        }
        if (w == 0) {
            GdrStep s = {0.0f, 0.0f, 0.0f, 0.0f};
            if (lane < nv)
                s = gdr_step_of(ssd_bf(p.dt[(row0 + lane) * p.dts + h]), ssd_bf(p.beta[(row0 + lane) * p.bs + h]),
                                p.dt_bias ? p.dt_bias[h] : 0.0f, p.dt_softplus, p.beta_sigmoid);
            // the running sum in 64 bits: differences of it are exponents, and a
            // rounding of the sum would be an error relative to the product
            // (a decay below 2^-1024 is 0 with any state: held there, a reset of any
            // size leaves the later differences their digits. The comparison lets a
            // NaN through, as a maximum would not. Rows past the end decay nothing.)
            double log_a = (double)s.step * (double)p.A[h] * 1.4426950408889634074;
            log_a = log_a < -1024.0 ? -1024.0 : log_a;
            const double G = gdr_prefix64(lane < nv ? log_a : 0.0, lane);
            const double Gc = gdr_last64(G);
            const float hi = (float)G, lo = (float)(G - (double)hi);
            sGh[lane] = hi;
            sGl[lane] = lo;
            sB[lane] = s.beta;
            const float head = __builtin_amdgcn_exp2f(hi);
            sHead[lane] = head;
            sTail[lane] = __builtin_amdgcn_exp2f((float)(Gc - G));
            tab[kTBeta * kGdrC + lane] = s.beta;
            tab[kTHead * kGdrC + lane] = head;
            tab[kTGhi * kGdrC + lane] = hi;
            tab[kTGlo * kGdrC + lane] = lo;
            tab[kTStep * kGdrC + lane] = s.step;
            tab[kTDstep * kGdrC + lane] = s.dstep;
            tab[kTDbeta * kGdrC + lane] = s.dbeta;
        }
        auto square = [](const uint4 &v) {
            const uint32_t e[4] = {v.x, v.y, v.z, v.w};
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = ssd_bf(e[k]), c = __uint_as_float(e[k] & 0xffff0000u);
                s = fmaf(a, a, fmaf(c, c, s));
            }
            return s;
        };
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int x = i * 256 + tid, row = x / LPR, o = row * KS + 8 * (x % LPR);
            *reinterpret_cast<uint4 *>(&u.in.k[o]) = kr[i];
            *reinterpret_cast<uint4 *>(&u.in.q[o]) = qr[i];
            if (p.qk_norm) {
                float k2 = square(kr[i]), q2 = square(qr[i]);
                if (LPR == 16) {
                    k2 = gdr_sum16(k2);
                    q2 = gdr_sum16(q2);
                } else {
#pragma unroll
                    for (int o2 = 1; o2 < 8; o2 <<= 1) {
                        k2 += __shfl_xor(k2, o2);
                        q2 += __shfl_xor(q2, o2);
                    }
                }
                if (x % LPR == 0) {
                    sRk[row] = 1.0f / sqrtf(k2 + p.qk_eps);
                    sUq[row] = 1.0f / sqrtf(q2 + p.qk_eps);
                }
            } else if (x % LPR == 0) {
                sRk[row] = sUq[row] = 1.0f;
            }
        }
    }
    __syncthreads();
    if (w == 3) {
        const float rk = sRk[lane], uq = sUq[lane], rq = uq * p.scale;
        tab[kTHk * kGdrC + lane] = sHead[lane] * rk;
        tab[kTHq * kGdrC + lane] = sHead[lane] * rq;
        tab[kTTk * kGdrC + lane] = sTail[lane] * rk;
        tab[kTRk * kGdrC + lane] = rk;
        tab[kTRq * kGdrC + lane] = rq;
        tab[kTUq * kGdrC + lane] = uq;
    }
    // tiles w, w + 4, w + 8, held transposed: row i = 16 T + r16 is the lane's,
    // columns j = 16 J + 4 g4 .. + 3
    ssd_f32x4 kk[3], qk[3];
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const int x = w + 4 * t;
        kk[t] = qk[t] = gdr_zero4();
        if (x >= kGdrTiles) continue;
        const int T = x >= 6 ? 3 : x >= 3 ? 2 : x >= 1 ? 1 : 0, J = x - T * (T + 1) / 2;
#pragma unroll
        for (int s = 0; s < N / 32; ++s) {
            const ssd_bf16x8 kj = ssd_ld16(&u.in.k[(16 * J + r16) * KS + 32 * s + 8 * g4]);
            kk[t] = ssd_mfma(kj, ssd_ld16(&u.in.k[(16 * T + r16) * KS + 32 * s + 8 * g4]), kk[t]);
            qk[t] = ssd_mfma(kj, ssd_ld16(&u.in.q[(16 * T + r16) * KS + 32 * s + 8 * g4]), qk[t]);
        }
    }
    __syncthreads();
    float *sT = u.sys.t, *sR = u.sys.r;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const int x = w + 4 * t;
        if (x >= kGdrTiles) continue;
        const int T = x >= 6 ? 3 : x >= 3 ? 2 : x >= 1 ? 1 : 0, J = x - T * (T + 1) / 2;
        const int i = 16 * T + r16, j0 = 16 * J + 4 * g4;
        const float gh = sGh[i], gl = sGl[i], ki = sRk[i] * sB[i], qi = sUq[i] * p.scale;
        const float4 ghj = *reinterpret_cast<const float4 *>(&sGh[j0]), glj = *reinterpret_cast<const float4 *>(&sGl[j0]);
        const float4 rkj = *reinterpret_cast<const float4 *>(&sRk[j0]);
        const float gj[4] = {ghj.x, ghj.y, ghj.z, ghj.w}, lj[4] = {glj.x, glj.y, glj.z, glj.w};
        const float rj[4] = {rkj.x, rkj.y, rkj.z, rkj.w};
        ssd_f32x4 tt, sc;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            // above the diagonal exp2(-inf): no branch
            const float e = i >= j0 + r ? (gh - gj[r]) + (gl - lj[r]) : -__builtin_inff();
            const float gam = __builtin_amdgcn_exp2f(e) * rj[r];
            tt[r] = i > j0 + r ? kk[t][r] * gam * ki : 0.0f;
            sc[r] = qk[t][r] * gam * qi;
        }
        *reinterpret_cast<ssd_f32x4 *>(&sT[i * TS + j0]) = tt;
        *reinterpret_cast<ssd_f32x4 *>(p.score + id * (kGdrTiles * 256) + 256 * x + 16 * r16 + 4 * g4) = sc;
    }
    __syncthreads();
    {
        // (I + T)^-1 of diagonal block w, a column per lane, by substitution
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == r16 ? 1.0f : 0.0f;
            float row[16];
#pragma unroll
            for (int k = 0; k < i; k += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(&sT[(16 * w + i) * TS + 16 * w + k]);
                row[k] = f.x; row[k + 1] = f.y; row[k + 2] = f.z; row[k + 3] = f.w;
            }
#pragma unroll
            for (int k = 0; k < i; ++k) v = fmaf(-row[k], x[k], v);
            x[i] = v;
        }
        if (g4 == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) sR[(16 * w + i) * TS + 16 * w + r16] = x[i];
    }
    __syncthreads();
    // block column w below the diagonal: R_iw = -R_ii sum_k T_ik R_kw
    for (int i = w + 1; i < 4; ++i) {
        ssd_f32x4 acc = gdr_zero4();
        for (int k = w; k < i; ++k)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(sT[(16 * i + r16) * TS + 16 * k + 4 * s + g4],
                                                           sR[(16 * k + 4 * s + g4) * TS + 16 * w + r16], acc, 0, 0, 0);
        ssd_f32x4 out = gdr_zero4();
#pragma unroll
        for (int s = 0; s < 4; ++s)
            out = __builtin_amdgcn_mfma_f32_16x16x4f32(-sR[(16 * i + r16) * TS + 16 * i + 4 * g4 + s], acc[s], out, 0, 0,
                                                       0);
#pragma unroll
        for (int r = 0; r < 4; ++r) sR[(16 * i + 4 * g4 + r) * TS + 16 * w + r16] = out[r];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    float *R = p.R + id * (kGdrTiles * 256);
    for (int x = tid; x < kGdrTiles * 64; x += 256) {
        const int t = x >> 6, i = (x >> 2) & 15, c = x & 3;
        const int T = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0, J = t - T * (T + 1) / 2;
        *reinterpret_cast<float4 *>(R + 4 * x) =
            *reinterpret_cast<const float4 *>(&sR[(16 * T + i) * TS + 16 * J + 4 * c]);
    }
}

// the two tiles above the diagonal that share a 32-token operand with one on it
template <int PARTS>
__device__ __forceinline__ void gdr_zero_upper(uint16_t *dst, int tid, int threads) {
    for (int q = tid; q < PARTS * 2 * 64; q += threads) {
        const int plane = q >> 7, t = (q >> 6) & 1, i = (q >> 2) & 15, c = q & 3;
        *reinterpret_cast<uint2 *>(dst + plane * kGdrPlane + (32 * t + i) * kGdrRS + 32 * t + 16 + 4 * c) =
            uint2{0u, 0u};
    }
}

__device__ __forceinline__ ssd_f32x4 gdr_ld4(const float *p) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    return ssd_f32x4{v.x, v.y, v.z, v.w};
}

// ---------------------------------------------------------------------------
// The kernels that walk the chunks.
//
// A workgroup of NW waves takes 16 NW columns of one head. The next chunk's
// rows and matrices are loaded into registers while this one is computed, and
// written to the other half of double-buffered LDS (the C x C matrices split
// into bf16 planes on the way) at the start of the next, so a chunk costs one
// barrier and no wait on memory.
//
// The matrix cores round a sum towards minus infinity (measured: states had a
// mean error of -4e-8 of their mean size, positive and negative ones alike),
// which over many chunks would add up where the gradient of the decay sums
// them. So the state's sign alternates: odd chunks hold -S, through the signs
// of the scales that are applied anyway, and the errors cancel.

// LDS of one chunk: K and Q rows; the lower tiles of R and of the scores in three
// parts; the first four tables and the decay over the whole chunk.
//
// Layouts are chosen for the banks (64 of 4 bytes): with padded rows the walk
// spent more LDS cycles on conflicts than on data (7.4 of 12 thousand per chunk; so
// laid out, 2.0 thousand are left, 254 per wave with its 127 LDS instructions).
//  * A 16 x 16 tile is kept as units of 4 columns, unit column by unit column, rows
//    8 apart swapped in the last two unit columns: 16 lanes that read a unit column
//    (an operand's rows) or a 4 x 4 square of units (a transposing read) touch
//    every bank once.
//  * A row of K or Q is kept in 16-byte pieces, each the columns 4 g .. + 3 and 16 +
//    4 g .. + 3 of a block of 32 (an operand's lane reads just that), at a place
//    exchanged by the row's low bits, so that the pieces of 16 rows, and the squares
//    of a transposing read, lie in different banks.
constexpr int kGdrPart = kGdrTiles * 256;   // elements of one part of a C x C matrix
template <int N> struct GdrChunkLds {
    uint16_t k[kGdrC * N], q[kGdrC * N];
    uint16_t r[3 * kGdrPart], a[3 * kGdrPart];
    float tab[4 * kGdrC];
    float end[4];
};

// element offset of row `row`, unit column c of a tile
__device__ __forceinline__ constexpr int gdr_unit(int row, int c) { return 4 * (16 * c + (row ^ ((c & 2) << 2))); }

// element offset of piece `piece` (4 block + g) of a row of K or Q
template <int N> __device__ __forceinline__ constexpr int gdr_piece(int row, int piece) {
    const int x = N == 128 ? (row & 3) << 2 | ((row >> 2) & 3) : (row & 2) << 1 | ((row >> 2) & 3);
    return row * N + 8 * (piece ^ x);
}

// the operand of rows 16 T + r16, columns 32 s + 16 (e / 4) + 4 g4 + e % 4
template <int N> __device__ __forceinline__ ssd_bf16x8 gdr_ld_row(const uint16_t *m, int T, int s, int r16, int g4) {
    return ssd_ld16(m + 16 * T * N + gdr_piece<N>(r16, 4 * s + g4));
}

// the operand of column 16 nt + r16, rows 32 s + 16 (e / 4) + 4 g4 + e % 4
template <int N> __device__ __forceinline__ ssd_bf16x8 gdr_ld_column(const uint16_t *m, int nt, int s, int r16, int g4) {
    const uint16_t *p = m + 32 * s * N + gdr_piece<N>(4 * g4 + (r16 >> 2), 4 * (nt >> 1) + (r16 & 3)) + 4 * (nt & 1);
    return ssd_ld_tr2(p, p + 16 * N);
}

// rows of row tile T, columns of tiles 2 s and 2 s + 1, of a lower triangular matrix
template <int PARTS>
__device__ __forceinline__ GdrSplit<PARTS> gdr_ld_tile_rows(const uint16_t *m, int T, int s, int r16, int g4) {
    GdrSplit<PARTS> o;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        const uint16_t *p = m + k * kGdrPart + gdr_unit(r16, g4);
        const uint2 a = *reinterpret_cast<const uint2 *>(p + 256 * gdr_tile(T, 2 * s));
        uint2 b = {0u, 0u};
        if (2 * s + 1 <= T) b = *reinterpret_cast<const uint2 *>(p + 256 * gdr_tile(T, 2 * s + 1));
        o.part[k] = __builtin_bit_cast(ssd_bf16x8, uint4{a.x, a.y, b.x, b.y});
    }
    return o;
}

// columns of column tile T, rows of tiles 2 s and 2 s + 1
template <int PARTS>
__device__ __forceinline__ GdrSplit<PARTS> gdr_ld_tile_cols(const uint16_t *m, int T, int s, int r16, int g4) {
    GdrSplit<PARTS> o;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        const uint16_t *p = m + k * kGdrPart + gdr_unit(4 * g4 + (r16 >> 2), r16 & 3);
        uint2 a = {0u, 0u};
        if (2 * s >= T) a = ssd_ld_tr(p + 256 * gdr_tile(2 * s, T));
        const uint2 b = ssd_ld_tr(p + 256 * gdr_tile(2 * s + 1, T));
        o.part[k] = __builtin_bit_cast(ssd_bf16x8, uint4{a.x, a.y, b.x, b.y});
    }
    return o;
}

// A wave's own 16 columns of V (or dY), a chunk ahead in registers (half a row
// per lane), turned through a 64 x 16 tile of LDS that no other wave touches
struct GdrColumns {
    uint4 v[2];
    __device__ __forceinline__ void load(const GdrParams &p, const uint16_t *col, int64_t stride, int64_t rowb, int ci,
                                         int lane) {
        const uint32_t nv = (uint32_t)gdr_valid(p, ci), st = (uint32_t)stride;
        const __amdgpu_buffer_rsrc_t r = ssd_buffer(col + (rowb + (int64_t)ci * kGdrC) * stride, 2u * ((nv - 1) * st + 16));
        const uint32_t o = 2u * ((uint32_t)(lane >> 1) * st + 8u * (lane & 1));
        v[0] = ssd_bload16(r, o);
        v[1] = ssd_bload16(r, o + 64u * st);
    }
    // the lane's column of rows 16 T + 4 g4 .. + 3, for every T
    __device__ __forceinline__ void turn(uint16_t *tile, int lane, uint2 (&out)[4]) const {
        const int r16 = lane & 15, g4 = lane >> 4;
        // half h of row i: unit columns 2 h and 2 h + 1 of tile i / 16
        uint16_t *at = tile + 256 * (lane >> 5);
        const int row = (lane >> 1) & 15, c = 2 * (lane & 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<uint2 *>(at + 512 * i + gdr_unit(row, c)) = uint2{v[i].x, v[i].y};
            *reinterpret_cast<uint2 *>(at + 512 * i + gdr_unit(row, c + 1)) = uint2{v[i].z, v[i].w};
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int T = 0; T < 4; ++T) out[T] = ssd_ld_tr(tile + 256 * T + gdr_unit(4 * g4 + (r16 >> 2), r16 & 3));
    }
};

template <int N, int NW> struct GdrChunkRegs {
    static constexpr int TH = 64 * NW;
    static constexpr int KI = kGdrC * N / 8 / TH, RI = (kGdrTiles * 64 + TH - 1) / TH, TI = (4 * kGdrC + TH - 1) / TH;
    uint4 k[KI], q[KI];
    float4 r[RI], a[RI];
    float tab[TI], end;
    __device__ __forceinline__ void load(const GdrParams &p, int b, int g, int64_t id, int ci, int tid) {
        const uint32_t nv = (uint32_t)gdr_valid(p, ci);
        const int64_t row0 = (int64_t)b * p.L + (int64_t)ci * kGdrC;
        const uint32_t ks = (uint32_t)p.ks, qs = (uint32_t)p.qs;
        // rows past the end have offsets past the ranges: they read zero
        const __amdgpu_buffer_rsrc_t rk = ssd_buffer(p.k + row0 * p.ks + (int64_t)g * N, 2u * ((nv - 1) * ks + N));
        const __amdgpu_buffer_rsrc_t rq = ssd_buffer(p.q + row0 * p.qs + (int64_t)g * N, 2u * ((nv - 1) * qs + N));
        const __amdgpu_buffer_rsrc_t rr = ssd_buffer(p.R + id * kGdrPart, kGdrPart * 4);
        const __amdgpu_buffer_rsrc_t ra = ssd_buffer(p.score + id * kGdrPart, kGdrPart * 4);
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const uint32_t x = i * TH + tid, row = x / (N / 8), c = 8 * (x % (N / 8));
            k[i] = ssd_bload16(rk, 2u * (row * ks + c));
            q[i] = ssd_bload16(rq, 2u * (row * qs + c));
        }
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            r[i] = __builtin_bit_cast(float4, ssd_bload16(rr, 16u * (i * TH + tid)));
            a[i] = __builtin_bit_cast(float4, ssd_bload16(ra, 16u * (i * TH + tid)));
        }
        const float *t = p.tab + id * (kGdrTab * kGdrC);
#pragma unroll
        for (int i = 0; i < TI; ++i) tab[i] = t[(i * TH + tid) & (4 * kGdrC - 1)];
        end = t[kTHead * kGdrC + kGdrC - 1];
    }
    __device__ __forceinline__ void store(GdrChunkLds<N> &s, int tid) const {
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            // columns 8 j .. + 7 of a row: halves of two pieces
            const int x = i * TH + tid, row = x / (N / 8), j = x % (N / 8);
            const int o0 = gdr_piece<N>(row & 15, 4 * (j >> 2) + 2 * (j & 1)) + (row & ~15) * N + 4 * ((j >> 1) & 1);
            const int o1 = gdr_piece<N>(row & 15, 4 * (j >> 2) + 2 * (j & 1) + 1) + (row & ~15) * N + 4 * ((j >> 1) & 1);
            *reinterpret_cast<uint2 *>(&s.k[o0]) = uint2{k[i].x, k[i].y};
            *reinterpret_cast<uint2 *>(&s.k[o1]) = uint2{k[i].z, k[i].w};
            *reinterpret_cast<uint2 *>(&s.q[o0]) = uint2{q[i].x, q[i].y};
            *reinterpret_cast<uint2 *>(&s.q[o1]) = uint2{q[i].z, q[i].w};
        }
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            const int x = i * TH + tid;
            if (x < kGdrTiles * 64) {
                const int o = 256 * (x >> 6) + gdr_unit((x >> 2) & 15, x & 3);
                gdr_store_parts<3>(&s.r[o], kGdrPart, r[i]);
                gdr_store_parts<3>(&s.a[o], kGdrPart, a[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < TI; ++i)
            if (TH * TI == 4 * kGdrC || i * TH + tid < 4 * kGdrC) s.tab[i * TH + tid] = tab[i];
        if (tid == 0) s.end[0] = end;
    }
};

// Products of parts are issued small ones first, each over every T in turn, so that
// consecutive instructions do not wait for one another.
//
// Measured: 256 heads of 128 x 128 on 8192 tokens 0.85-0.90 ms, 7 us a chunk, for
// which a wave issues 1000 vector instructions and 216 MFMAs (3500 cycles), two waves
// to a SIMD: bound by issue and the matrix cores together. With the kept states, 256
// heads on 2048 tokens 0.31 ms for 1.4 GB, 4.6 TB/s: bound by memory. 16 heads of 96
// x 128 with helpers 3.9 us a chunk, of which 1.4 us are MFMAs: bound by the chain
// S -> K S -> R X -> K^T U -> S through one wave. (32 columns per wave would halve the
// LDS reads but spill: 2.4 against 1.2 ms when measured. y from two parts of S, U and
// the scores would be 6% faster, and a bf16 step beside the rounded exact value in
// 0.34% of its elements instead of 0.01%.)
// SAVE: keep S and U for the gradients; WANT_Y: write y (the backward's recomputation does not)
template <int N, bool SAVE, bool WANT_Y, int NW>
__global__ __launch_bounds__(64 * (NW + gdr_helpers(NW))) void gdr_fwd_kernel(const GdrParams p, int splits) {
    constexpr int NT = N / 16;
    __shared__ __attribute__((aligned(16))) GdrChunkLds<N> lds[2];
    __shared__ __attribute__((aligned(16))) uint16_t sV[NW][kGdrC * 16];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int bh = blockIdx.x / splits, split = blockIdx.x % splits;
    const int b = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int p0 = 16 * (split * NW + w);
    constexpr bool HELP = gdr_helpers(NW) > 0;
    const int sid = HELP ? tid - 64 * NW : tid;   // place among the staging threads
    const bool live = w < NW && p0 < p.P;
    const int64_t sbase = ((int64_t)bh * p.P + p0 + r16) * N;
    const uint32_t ysr = (uint32_t)(p.H * p.P);
    const int64_t id0 = (int64_t)bh * p.nc, rowb = (int64_t)b * p.L;
    ssd_f32x4 S[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        S[nt] = live && p.h0 ? gdr_ld4(p.h0 + sbase + 16 * nt + 4 * g4) : gdr_zero4();
    const uint16_t *vcol = p.v + (int64_t)h * p.P + p0;
    GdrChunkRegs<N, NW> regs;
    GdrColumns vr;
    if (live) vr.load(p, vcol, p.vs, rowb, 0, lane);
    if (!HELP || w >= NW) {
        regs.load(p, b, g, id0, 0, sid);
        regs.store(lds[0], sid);
        if (p.nc > 1) regs.load(p, b, g, id0 + 1, 1, sid);
    }
    __syncthreads();
    float sign = 1.0f;
    const bool early = HELP ? w >= NW : w < 4, late = !HELP && !early;
    for (int ci = 0; ci < p.nc; ++ci) {
        const GdrChunkLds<N> &L = lds[ci & 1];
        const int nv = gdr_valid(p, ci);
        const int64_t id = id0 + ci;
        const int64_t row0 = rowb + (int64_t)ci * kGdrC;
        auto stage = [&]() {
            if (ci + 1 < p.nc) regs.store(lds[(ci + 1) & 1], sid);
            if (ci + 2 < p.nc) regs.load(p, b, g, id + 2, ci + 2, sid);
        };
        if (early) stage();
        ssd_f32x4 X[4], Y[4], U[4];
        if (live) {
            uint2 vw[4];
            vr.turn(sV[w], lane, vw);
            if (ci + 1 < p.nc) vr.load(p, vcol, p.vs, rowb, ci + 1, lane);
            if constexpr (SAVE) {
                float *dst = p.S + (id * p.P + p0 + r16) * N + 4 * g4;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) *reinterpret_cast<ssd_f32x4 *>(dst + 16 * nt) = S[nt] * sign;
            }
#pragma unroll
            for (int T = 0; T < 4; ++T) X[T] = Y[T] = U[T] = gdr_zero4();
#pragma unroll
            for (int s = 0; s < N / 32; ++s) {
                const GdrSplit<3> so = gdr_split<3>(S[2 * s], S[2 * s + 1]);
                ssd_bf16x8 ko[4], qo[4];
#pragma unroll
                for (int T = 0; T < 4; ++T) {
                    ko[T] = gdr_ld_row<N>(L.k, T, s, r16, g4);
                    if constexpr (WANT_Y) qo[T] = gdr_ld_row<N>(L.q, T, s, r16, g4);
                }
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int T = 0; T < 4; ++T) {
                        X[T] = ssd_mfma(ko[T], so.part[k], X[T]);
                        if constexpr (WANT_Y) Y[T] = ssd_mfma(so.part[k], qo[T], Y[T]);
                    }
            }
            // beta X
#pragma unroll
            for (int T = 0; T < 4; ++T) {
                const ssd_f32x4 hk = gdr_ld4(&L.tab[kTHk * kGdrC + 16 * T + 4 * g4]);
                const ssd_f32x4 be = gdr_ld4(&L.tab[kTBeta * kGdrC + 16 * T + 4 * g4]);
                const float vc[4] = {ssd_bf(vw[T].x), __uint_as_float(vw[T].x & 0xffff0000u), ssd_bf(vw[T].y),
                                     __uint_as_float(vw[T].y & 0xffff0000u)};
#pragma unroll
                for (int r = 0; r < 4; ++r) X[T][r] = be[r] * (sign * vc[r] - hk[r] * X[T][r]);
            }
            // U = R (beta X)
            {
                const GdrSplit<3> xo[2] = {gdr_split<3>(X[0], X[1]), gdr_split<3>(X[2], X[3])};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    GdrSplit<3> ro[4];
#pragma unroll
                    for (int T = 2 * s; T < 4; ++T)
                        ro[T] = gdr_ld_tile_rows<3>(L.r, T, s, r16, g4);
#pragma unroll
                    for (int k = 2; k >= 0; --k)
#pragma unroll
                        for (int i = 0; i <= k; ++i)
#pragma unroll
                            for (int T = 2 * s; T < 4; ++T) U[T] = ssd_mfma(ro[T].part[i], xo[s].part[k - i], U[T]);
                }
            }
            if constexpr (SAVE) {
                float *dst = p.U + (id * p.P + p0 + r16) * kGdrC + 4 * g4;
#pragma unroll
                for (int T = 0; T < 4; ++T) *reinterpret_cast<ssd_f32x4 *>(dst + 16 * T) = U[T] * sign;
            }
        }
        if (late) stage();
        if (live) {
            // Y^T = exp(G) S Q^T + U^T A^T
            if constexpr (WANT_Y) {
                const __amdgpu_buffer_rsrc_t ry = ssd_buffer(p.y + (row0 * p.H + h) * p.P,
                                                             2u * ((uint32_t)(nv - 1) * ysr + (uint32_t)p.P));
                const GdrSplit<3> uo[2] = {gdr_split<3>(U[0], U[1]), gdr_split<3>(U[2], U[3])};
#pragma unroll
                for (int T = 0; T < 4; ++T) Y[T] *= L.tab[kTHq * kGdrC + 16 * T + r16];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    GdrSplit<3> ao[4];
#pragma unroll
                    for (int T = 2 * s; T < 4; ++T)
                        ao[T] = gdr_ld_tile_rows<3>(L.a, T, s, r16, g4);
#pragma unroll
                    for (int k = 2; k >= 0; --k)
#pragma unroll
                        for (int i = 0; i <= k; ++i)
#pragma unroll
                            for (int T = 2 * s; T < 4; ++T) Y[T] = ssd_mfma(uo[s].part[k - i], ao[T].part[i], Y[T]);
                }
                // rows past the end are dropped by the buffer's range
#pragma unroll
                for (int T = 0; T < 4; ++T)
                    ssd_bstore8(ry, 2u * ((uint32_t)(16 * T + r16) * ysr + p0 + 4 * g4),
                                uint2{ssd_pack(sign * Y[T][0], sign * Y[T][1]), ssd_pack(sign * Y[T][2], sign * Y[T][3])});
            }
            // -S' = -exp(G_C) S - K^T (exp(G_C - G) U)
#pragma unroll
            for (int T = 0; T < 4; ++T) U[T] *= -gdr_ld4(&L.tab[kTTk * kGdrC + 16 * T + 4 * g4]);
            const float end = -L.end[0];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) S[nt] *= end;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const GdrSplit<3> uo = gdr_split<3>(U[2 * s], U[2 * s + 1]);
                ssd_bf16x8 ko[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) ko[nt] = gdr_ld_column<N>(L.k, nt, s, r16, g4);
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) S[nt] = ssd_mfma(ko[nt], uo.part[k], S[nt]);
            }
        }
        sign = -sign;
        __syncthreads();
    }
    if (live && p.h_last)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<ssd_f32x4 *>(p.h_last + sbase + 16 * nt + 4 * g4) = S[nt] * sign;
}

// ---------------------------------------------------------------------------
// Backwards over the chunks: D' of every chunk, W, dv and dh0. 256 heads of 128 x
// 128 on 2048 tokens: 0.28-0.31 ms for 1.4 GB, 4.6-5.1 TB/s, bound by memory; 48 heads 129 us,
// 4.0 us a chunk, bound by the chain through a wave as the forward is.
template <int N, int NW>
__global__ __launch_bounds__(64 * (NW + gdr_helpers(NW))) void gdr_rev_kernel(const GdrParams p, int splits) {
    constexpr int NT = N / 16;
    __shared__ __attribute__((aligned(16))) GdrChunkLds<N> lds[2];
    __shared__ __attribute__((aligned(16))) uint16_t sV[NW][kGdrC * 16];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int bh = blockIdx.x / splits, split = blockIdx.x % splits;
    const int b = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int p0 = 16 * (split * NW + w);
    constexpr bool HELP = gdr_helpers(NW) > 0;
    const int sid = HELP ? tid - 64 * NW : tid;   // place among the staging threads
    const bool live = w < NW && p0 < p.P;
    const int64_t sbase = ((int64_t)bh * p.P + p0 + r16) * N;
    const uint32_t ys = (uint32_t)(p.H * p.P);
    const int64_t id0 = (int64_t)bh * p.nc, rowb = (int64_t)b * p.L;
    ssd_f32x4 D[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        D[nt] = live && p.dh_last ? gdr_ld4(p.dh_last + sbase + 16 * nt + 4 * g4) : gdr_zero4();
    // operands that pick tile 0 or 1 of a pair: W^T in bf16 from an operand
    GdrSplit<1> pick[2];
    {
        float one[2][8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int t = 0; t < 2; ++t) one[t][e] = (e >> 2) == t && 4 * g4 + (e & 3) == r16 ? 1.0f : 0.0f;
        pick[0] = gdr_split<1>(one[0]);
        pick[1] = gdr_split<1>(one[1]);
    }
    const uint16_t *ycol = p.dy + (int64_t)h * p.P + p0;
    const int last = p.nc - 1;
    GdrChunkRegs<N, NW> regs;
    GdrColumns yr;
    if (live) yr.load(p, ycol, ys, rowb, last, lane);
    if (!HELP || w >= NW) {
        regs.load(p, b, g, id0 + last, last, sid);
        regs.store(lds[last & 1], sid);
        if (last > 0) regs.load(p, b, g, id0 + last - 1, last - 1, sid);
    }
    __syncthreads();
    float sign = 1.0f;
    const bool early = HELP ? w >= NW : w < 4, late = !HELP && !early;   // as in the forward
    for (int ci = last; ci >= 0; --ci) {
        const GdrChunkLds<N> &L = lds[ci & 1];
        const int nv = gdr_valid(p, ci);
        const int64_t id = id0 + ci;
        const int64_t row0 = rowb + (int64_t)ci * kGdrC;
        auto stage = [&]() {
            if (ci > 0) regs.store(lds[(ci - 1) & 1], sid);
            if (ci > 1) regs.load(p, b, g, id - 2, ci - 2, sid);
        };
        if (early) stage();
        const uint32_t flip = sign < 0.0f ? 0x80008000u : 0u;
        uint4 yw[2];
        ssd_f32x4 W[4];
        if (live) {
            // dY with the chunk's sign, as operands
            uint2 yt[4];
            yr.turn(sV[w], lane, yt);
            if (ci > 0) yr.load(p, ycol, ys, rowb, ci - 1, lane);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                yw[s] = uint4{yt[2 * s].x ^ flip, yt[2 * s].y ^ flip, yt[2 * s + 1].x ^ flip, yt[2 * s + 1].y ^ flip};
            {
                float *dst = p.D + (id * p.P + p0 + r16) * N + 4 * g4;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) *reinterpret_cast<ssd_f32x4 *>(dst + 16 * nt) = D[nt] * sign;
            }
            // dU = exp(G_C - G) K D'^T + A^T dY
            ssd_f32x4 dU[4];
#pragma unroll
            for (int T = 0; T < 4; ++T) dU[T] = W[T] = gdr_zero4();
#pragma unroll
            for (int s = 0; s < N / 32; ++s) {
                const GdrSplit<3> so = gdr_split<3>(D[2 * s], D[2 * s + 1]);
                ssd_bf16x8 ko[4];
#pragma unroll
                for (int T = 0; T < 4; ++T) ko[T] = gdr_ld_row<N>(L.k, T, s, r16, g4);
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int T = 0; T < 4; ++T) dU[T] = ssd_mfma(ko[T], so.part[k], dU[T]);
            }
#pragma unroll
            for (int T = 0; T < 4; ++T) dU[T] *= gdr_ld4(&L.tab[kTTk * kGdrC + 16 * T + 4 * g4]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const ssd_bf16x8 yo = __builtin_bit_cast(ssd_bf16x8, yw[s]);
                GdrSplit<3> ao[4];
#pragma unroll
                for (int T = 0; T < 2 * s + 2; ++T)
                    ao[T] = gdr_ld_tile_cols<3>(L.a, T, s, r16, g4);
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int T = 0; T < 2 * s + 2; ++T) dU[T] = ssd_mfma(ao[T].part[k], yo, dU[T]);
            }
            // W = R^T dU
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const GdrSplit<3> uo = gdr_split<3>(dU[2 * s], dU[2 * s + 1]);
                GdrSplit<3> ro[4];
#pragma unroll
                for (int T = 0; T < 2 * s + 2; ++T)
                    ro[T] = gdr_ld_tile_cols<3>(L.r, T, s, r16, g4);
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                    for (int i = 0; i <= k; ++i)
#pragma unroll
                        for (int T = 0; T < 2 * s + 2; ++T) W[T] = ssd_mfma(ro[T].part[i], uo.part[k - i], W[T]);
            }
            {
                float *dst = p.W + (id * p.P + p0 + r16) * kGdrC + 4 * g4;
#pragma unroll
                for (int T = 0; T < 4; ++T) *reinterpret_cast<ssd_f32x4 *>(dst + 16 * T) = W[T] * sign;
            }
        }
        if (late) stage();
        if (live) {
            // dv = beta W, rounded, turned so that a lane holds 4 columns of a row
            // (rows past the end dropped by the range)
#pragma unroll
            for (int T = 0; T < 4; ++T) W[T] *= gdr_ld4(&L.tab[kTBeta * kGdrC + 16 * T + 4 * g4]);
            {
                const __amdgpu_buffer_rsrc_t rdv =
                    ssd_buffer(p.dv + (row0 * p.H + h) * p.P, 2u * ((uint32_t)(nv - 1) * ys + (uint32_t)p.P));
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const GdrSplit<1> wo = gdr_split<1>(W[2 * s], W[2 * s + 1]);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const ssd_f32x4 o = ssd_mfma(wo.part[0], pick[t].part[0], gdr_zero4());
                        const int i = 16 * (2 * s + t) + r16;
                        ssd_bstore8(rdv, 2u * ((uint32_t)i * ys + p0 + 4 * g4),
                                    uint2{ssd_pack(o[0], o[1]) ^ flip, ssd_pack(o[2], o[3]) ^ flip});
                    }
                }
            }
            // the two sources of -D
            ssd_f32x4 dY[4];
#pragma unroll
            for (int T = 0; T < 4; ++T) {
                const uint32_t y0 = T & 1 ? yw[T / 2].z : yw[T / 2].x, y1 = T & 1 ? yw[T / 2].w : yw[T / 2].y;
                const ssd_f32x4 y = {ssd_bf(y0), __uint_as_float(y0 & 0xffff0000u), ssd_bf(y1),
                                     __uint_as_float(y1 & 0xffff0000u)};
                W[T] *= gdr_ld4(&L.tab[kTHk * kGdrC + 16 * T + 4 * g4]);
                dY[T] = y * -gdr_ld4(&L.tab[kTHq * kGdrC + 16 * T + 4 * g4]);
            }
            const float end = -L.end[0];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) D[nt] *= end;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const GdrSplit<3> wo = gdr_split<3>(W[2 * s], W[2 * s + 1]);
                const GdrSplit<3> qo = gdr_split<3>(dY[2 * s], dY[2 * s + 1]);
#pragma unroll
                for (int n0 = 0; n0 < NT; n0 += 4) {
                    ssd_bf16x8 ko[4], qr[4];
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        ko[nt] = gdr_ld_column<N>(L.k, n0 + nt, s, r16, g4);
                        qr[nt] = gdr_ld_column<N>(L.q, n0 + nt, s, r16, g4);
                    }
#pragma unroll
                    for (int k = 2; k >= 0; --k)
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt) {
                            D[n0 + nt] = ssd_mfma(ko[nt], wo.part[k], D[n0 + nt]);
                            D[n0 + nt] = ssd_mfma(qr[nt], qo.part[k], D[n0 + nt]);
                        }
                }
            }
        }
        sign = -sign;
        __syncthreads();
    }
    if (live && p.dh0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<ssd_f32x4 *>(p.dh0 + sbase + 16 * nt + 4 * g4) = D[nt] * sign;
}

// ---------------------------------------------------------------------------
// dq, dk, dbeta, ddt of one chunk and group. Wave w holds n tile w; the heads
// of the group follow one another and add into dq and dk in that order. What a
// chunk needs of S, D', U and W (192 KB a head) is read once, 32 columns p ahead of
// their use. 8192 chunks and heads of 128 x 128: 0.91-0.93 ms for 2.0 GB, 2.2 TB/s: the
// reads of a workgroup (one per CU, for its LDS) stop while it forms the pair
// products and row sums, and with several heads to a group 26 registers spill. (The
// decays' gradient from <D', S'> and dq, dk would be 8% faster and lose its digits
// where a decay is strong.) Measured and not kept: walking the chunks with the next
// one's reads in flight (2% faster with one head per group, 1% slower with two: the
// registers), two n tiles per wave (1.5 ms), LDS without bank conflicts here (2%
// slower: the exchanged addresses cost more than the conflicts).
// ONE: a head per group, whose dq and dk need no second accumulators.
template <int N, bool ONE>
__global__ __launch_bounds__(4 * N) void gdr_grad_kernel(const GdrParams p) {
    constexpr int KS = N + kGdrPad, NW = N / 16, TH = 64 * NW, PL = kGdrPlane;
    constexpr int PB = 32;                 // columns p per step
    constexpr int TW = (kGdrTiles + NW - 1) / NW;   // C x C tiles per wave, at most
    constexpr int YS = PB + 8;             // LDS row stride of dY, V (token rows)
    constexpr int UPL = PB * kGdrRS;       // plane of U, W ([p][token])
    constexpr int UI = PB * kGdrC / 4 / TH, YI = (kGdrC * PB / 8 + TH - 1) / TH;
    // a step's columns: U, W in three parts, dY, V
    struct Step { uint16_t u[3 * UPL], w[3 * UPL], dy[kGdrC * YS], v[kGdrC * YS]; };
    // dY U^T and W U^T, decayed and scaled, once the steps are done, and what each
    // pair of tokens adds to the gradient of the decays between them
    constexpr int DS = kGdrC + 4;
    struct Pairs { uint16_t a[3 * PL], e[3 * PL]; float d[kGdrC * DS]; };
    union StepsOrPairs { Step step[2]; Pairs pairs; };
    __shared__ __attribute__((aligned(16))) uint16_t sK[kGdrC * KS], sQ[kGdrC * KS];
    __shared__ __attribute__((aligned(16))) StepsOrPairs sX;
    __shared__ __attribute__((aligned(16))) float sTab[kGdrTab * kGdrC];
    // per wave: q . (dY S), k . (W S), k . (U D') of its columns n; the pairs' sums of its rows
    __shared__ __attribute__((aligned(16))) float sDot[NW][4][kGdrC];
    __shared__ float sEs[4][kGdrC];        // sum_j E_ij W_i . U_j per column tile
    __shared__ float sWv[kGdrC];
    __shared__ double sDs[NW];
    uint16_t *const sPA = sX.pairs.a, *const sPE = sX.pairs.e;
    float *const sPD = sX.pairs.d;
    int tid = threadIdx.x;
    int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    int r16 = lane & 15, g4 = lane >> 4;
    const int ci = (int)(blockIdx.x % p.nc);
    const int bg = (int)(blockIdx.x / p.nc);
    const int b = bg / p.G, g = bg % p.G;
    const int nv = gdr_valid(p, ci);
    const int64_t row0 = (int64_t)b * p.L + (int64_t)ci * kGdrC;
    const uint32_t ys = (uint32_t)(p.H * p.P), vs = (uint32_t)p.vs;
    const int n0 = 16 * w;

    // what a step reads, one step ahead in registers; reads past the columns or
    // tokens that exist give zero
    float4 ur[UI], wr[UI];
    uint4 yr[YI], vr[YI];
    float sn[8], dn[8];
    auto load = [&](int h, int c0) {
        const int64_t id = (int64_t)(b * p.H + h) * p.nc + ci;
        const uint32_t pw = (uint32_t)min(PB, p.P - c0);
        const __amdgpu_buffer_rsrc_t ru = ssd_buffer(p.U + (id * p.P + c0) * kGdrC, pw * kGdrC * 4);
        const __amdgpu_buffer_rsrc_t rw = ssd_buffer(p.W + (id * p.P + c0) * kGdrC, pw * kGdrC * 4);
        const __amdgpu_buffer_rsrc_t rs = ssd_buffer(p.S + (id * p.P + c0) * N, pw * N * 4);
        const __amdgpu_buffer_rsrc_t rd = ssd_buffer(p.D + (id * p.P + c0) * N, pw * N * 4);
        const __amdgpu_buffer_rsrc_t ry =
            ssd_buffer(p.dy + (row0 * p.H + h) * p.P + c0, 2u * ((uint32_t)(nv - 1) * ys + pw));
        const __amdgpu_buffer_rsrc_t rv =
            ssd_buffer(p.v + row0 * p.vs + (int64_t)h * p.P + c0, 2u * ((uint32_t)(nv - 1) * vs + pw));
#pragma unroll
        for (int i = 0; i < UI; ++i) {
            ur[i] = __builtin_bit_cast(float4, ssd_bload16(ru, 16u * (i * TH + tid)));
            wr[i] = __builtin_bit_cast(float4, ssd_bload16(rw, 16u * (i * TH + tid)));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t o = 4u * ((uint32_t)(16 * (e >> 2) + 4 * g4 + (e & 3)) * N + n0 + r16);
            sn[e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (int)o, 0, 0));
            dn[e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rd, (int)o, 0, 0));
        }
#pragma unroll
        for (int i = 0; i < YI; ++i) {
            const uint32_t x = i * TH + tid, row = x / (PB / 8), c = 8 * (x % (PB / 8));
            const bool in = row < kGdrC && c < pw;
            yr[i] = ssd_bload16(ry, in ? 2u * (row * ys + c) : 0x7fffffffu);
            vr[i] = ssd_bload16(rv, in ? 2u * (row * vs + c) : 0x7fffffffu);
        }
    };
    // Every second step's products are taken negative (U and S carry the sign),
    // each step's in a sum of its own, and in every second chunk the others: the
    // matrix cores round towards minus infinity, and so their errors cancel
    // instead of adding up in the decays' gradient.
    auto store = [&](Step &s, float flip) {
#pragma unroll
        for (int i = 0; i < UI; ++i) {
            const int x = i * TH + tid, o = (x / (kGdrC / 4)) * kGdrRS + 4 * (x % (kGdrC / 4));
            gdr_store_parts<3>(&s.u[o], UPL, make_float4(flip * ur[i].x, flip * ur[i].y, flip * ur[i].z, flip * ur[i].w));
            gdr_store_parts<3>(&s.w[o], UPL, wr[i]);
        }
#pragma unroll
        for (int i = 0; i < YI; ++i) {
            const int x = i * TH + tid, o = (x / (PB / 8)) * YS + 8 * (x % (PB / 8));
            if (x < kGdrC * PB / 8) {
                *reinterpret_cast<uint4 *>(&s.dy[o]) = yr[i];
                *reinterpret_cast<uint4 *>(&s.v[o]) = vr[i];
            }
        }
    };
    // Addresses and conditions from the wave's and lane's place are formed where they
    // are used: hoisted out of the loops they would fill the registers.
    auto fresh = [&]() { asm volatile("" : "+v"(r16), "+v"(g4), "+v"(tid), "+v"(lane), "+s"(w)); };
    load(g * p.hpg, 0);
    gdr_stage_rows<N>(sK, KS, p.k + row0 * p.ks + (int64_t)g * N, p.ks, nv, tid, TH);
    gdr_stage_rows<N>(sQ, KS, p.q + row0 * p.qs + (int64_t)g * N, p.qs, nv, tid, TH);
    ssd_f32x4 dq[4], dk[4];
#pragma unroll
    for (int T = 0; T < 4; ++T) dq[T] = dk[T] = gdr_zero4();
    for (int hh = 0; hh < p.hpg; ++hh) {
        const int h = g * p.hpg + hh;
        const int bh = b * p.H + h;
        const int64_t id = (int64_t)bh * p.nc + ci;
        // products over p: dY S, W S, U D' (this wave's n), dY U^T and W U^T
        // (C x C lower tiles dealt over the waves), W V^T (its diagonal)
        ssd_f32x4 aq[4], ar[4], ac[4], pa[TW], pw[TW], wv = gdr_zero4();
#pragma unroll
        for (int T = 0; T < 4; ++T) aq[T] = ar[T] = ac[T] = gdr_zero4();
#pragma unroll
        for (int t = 0; t < TW; ++t) pa[t] = pw[t] = gdr_zero4();
        double ds = 0.0;                   // <D', S> of this wave's columns n
        __syncthreads();                   // the head before is done with sTab and sX
        for (int q = tid; q < kGdrTab * kGdrC; q += TH) sTab[q] = p.tab[id * (kGdrTab * kGdrC) + q];
        const float first = ci & 1 ? -1.0f : 1.0f;
        store(sX.step[0], first);
        for (int c0 = 0, buf = 0; c0 < p.P; c0 += PB, buf ^= 1) {
            const float flip = buf ? -first : first;
            fresh();
            // S and D' columns n0 + r16, rows p = c0 + 16 (e / 4) + 4 g4 + e % 4
            GdrSplit<3> so, dd;
            {
                float sv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ds = fma((double)sn[e], (double)dn[e], ds);
                    sv[e] = sn[e] * flip;
                }
                so = gdr_split<3>(sv);
                dd = gdr_split<3>(dn);
            }
            // the next step's reads: the next head's first behind the last
            if (c0 + PB < p.P) load(h, c0 + PB);
            else if (hh + 1 < p.hpg) load(h + 1, 0);
            __syncthreads();
            const Step &X = sX.step[buf];
            fresh();
#pragma unroll
            for (int T = 0; T < 4; ++T) {
                const GdrSplit<1> yo = gdr_whole(gdr_ld_perm(&X.dy[(16 * T + r16) * YS + 4 * g4]));
                const GdrSplit<3> uo = gdr_ld_col_parts<3>(X.u, kGdrRS, 4 * g4, 16 * T, r16, UPL);
                const GdrSplit<3> wo = gdr_ld_col_parts<3>(X.w, kGdrRS, 4 * g4, 16 * T, r16, UPL);
                ssd_f32x4 tq = gdr_zero4(), tr = gdr_zero4(), tc = gdr_zero4();
#pragma unroll
                for (int k = 2; k >= 0; --k) {
#pragma unroll
                    for (int i = 0; i <= k; ++i) {
                        tr = ssd_mfma(wo.part[i], so.part[k - i], tr);
                        tc = ssd_mfma(uo.part[i], dd.part[k - i], tc);
                    }
                    tq = ssd_mfma(yo.part[0], so.part[k], tq);
                }
                aq[T] += tq * flip;
                ar[T] += tr * flip;
                ac[T] += tc * flip;
                __builtin_amdgcn_sched_barrier(0);   // one tile's operands in registers at a time
            }
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                const int q = w + NW * t;
                if (q < kGdrTiles) {
                    const int T = q >= 6 ? 3 : q >= 3 ? 2 : q >= 1 ? 1 : 0, J = q - T * (T + 1) / 2;
                    const GdrSplit<3> uo = gdr_ld_col_parts<3>(X.u, kGdrRS, 4 * g4, 16 * J, r16, UPL);
                    const GdrSplit<1> yo = gdr_whole(gdr_ld_perm(&X.dy[(16 * T + r16) * YS + 4 * g4]));
                    const GdrSplit<3> wo = gdr_ld_col_parts<3>(X.w, kGdrRS, 4 * g4, 16 * T, r16, UPL);
                    pa[t] += gdr_mfma(uo, yo, gdr_zero4()) * flip;
                    pw[t] += gdr_mfma(uo, wo, gdr_zero4()) * flip;
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            // (waves 0 and 1 hold two tiles: the diagonal goes to the others)
            if (w >= NW - 4) {
                const int T = w - (NW - 4);
                const GdrSplit<3> wo = gdr_ld_col_parts<3>(X.w, kGdrRS, 4 * g4, 16 * T, r16, UPL);
                wv = gdr_mfma(wo, gdr_whole(gdr_ld_perm(&X.v[(16 * T + r16) * YS + 4 * g4])), wv);
            }
            if (c0 + PB < p.P) store(sX.step[buf ^ 1], -flip);
        }
        fresh();
        __syncthreads();                   // every wave is done with the steps: their place holds the pairs
        gdr_zero_upper<3>(sPA, tid, TH);
        gdr_zero_upper<3>(sPE, tid, TH);
        // row i = 16 w + 4 g4 + r, column 16 w + r16: the diagonal of W V^T
        if (w >= NW - 4 && (r16 >> 2) == g4) {
            const int r = r16 & 3;
            sWv[16 * (w - (NW - 4)) + r16] = r == 0 ? wv[0] : r == 1 ? wv[1] : r == 2 ? wv[2] : wv[3];
        }
        // C x C: decayed and scaled. A tile is held transposed: row i = 16 T + r16
        // is the lane's, columns j = 16 J + 4 g4 .. + 3
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            const int q = w + NW * t;
            if (q >= kGdrTiles) break;
            const int T = q >= 6 ? 3 : q >= 3 ? 2 : q >= 1 ? 1 : 0, J = q - T * (T + 1) / 2;
            ssd_f32x4 kk = gdr_zero4(), qk = gdr_zero4();
#pragma unroll
            for (int s = 0; s < N / 32; ++s) {
                const ssd_bf16x8 kj = ssd_ld16(&sK[(16 * J + r16) * KS + 32 * s + 8 * g4]);
                kk = ssd_mfma(kj, ssd_ld16(&sK[(16 * T + r16) * KS + 32 * s + 8 * g4]), kk);
                qk = ssd_mfma(kj, ssd_ld16(&sQ[(16 * T + r16) * KS + 32 * s + 8 * g4]), qk);
            }
            const int i = 16 * T + r16, j0 = 16 * J + 4 * g4;
            const float ghi = sTab[kTGhi * kGdrC + i], gli = sTab[kTGlo * kGdrC + i], rki = sTab[kTRk * kGdrC + i];
            const float rqi = sTab[kTRq * kGdrC + i], bei = sTab[kTBeta * kGdrC + i];
            const ssd_f32x4 ghj = gdr_ld4(&sTab[kTGhi * kGdrC + j0]), glj = gdr_ld4(&sTab[kTGlo * kGdrC + j0]);
            const ssd_f32x4 rkj = gdr_ld4(&sTab[kTRk * kGdrC + j0]);
            float a[4], e[4], d[4], es = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // above the diagonal exp2(-inf): no branch
                const float x = i >= j0 + r ? (ghi - ghj[r]) + (gli - glj[r]) : -__builtin_inff();
                const float gam = __builtin_amdgcn_exp2f(x) * rkj[r];
                a[r] = pa[t][r] * gam * rqi;
                const float ev = i > j0 + r ? pw[t][r] * gam * rki : 0.0f;
                es = fmaf(ev, kk[r], es);          // sum_j E_ij W_i . U_j
                e[r] = ev * bei;                   // subtracted below
                d[r] = i > j0 + r ? fmaf(a[r], qk[r], -e[r] * kk[r]) : 0.0f;
            }
            es += __shfl_xor(es, 16);
            es += __shfl_xor(es, 32);
            if (g4 == 0) sEs[J][i] = es;
            gdr_store_parts<3>(&sPA[i * kGdrRS + j0], PL, make_float4(a[0], a[1], a[2], a[3]));
            gdr_store_parts<3>(&sPE[i * kGdrRS + j0], PL, make_float4(e[0], e[1], e[2], e[3]));
            *reinterpret_cast<float4 *>(&sPD[i * DS + j0]) = make_float4(d[0], d[1], d[2], d[3]);
            __builtin_amdgcn_sched_barrier(0);
        }
        fresh();
        __syncthreads();
        // what the pairs i >= t > j add for token t (the lane): a row's sum up to t,
        // rows from t on
        {
            float sum = 0.0f;
#pragma unroll 1
            for (int i = w; i < kGdrC; i += NW) {
                const float d = lane > 0 && lane <= i ? sPD[i * DS + lane - 1] : 0.0f;
                const float upto = ssd_prefix_sum(d, lane);
                sum += lane <= i ? upto : 0.0f;
            }
            sDot[w][3][lane] = sum;
        }
        // products over tokens, scaled by the tokens' rows. The K and Q operands
        // are the wave's columns n of rows 16 T + 4 g4 + r as well: element
        // 4 (T % 2) + r of operand T / 2.
        ssd_bf16x8 ko[2], qo[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            ko[s] = gdr_ld_col(sK, KS, 32 * s + 4 * g4, n0, r16);
            qo[s] = gdr_ld_col(sQ, KS, 32 * s + 4 * g4, n0, r16);
        }
#pragma unroll
        for (int T = 0; T < 4; ++T) {
            // the products with S and D', and what they add to the decays' gradient
            aq[T] *= gdr_ld4(&sTab[kTHq * kGdrC + 16 * T + 4 * g4]);
            ar[T] *= gdr_ld4(&sTab[kTHk * kGdrC + 16 * T + 4 * g4]);
            ac[T] *= gdr_ld4(&sTab[kTTk * kGdrC + 16 * T + 4 * g4]);
            {
                ssd_f32x4 qs, kw, ku;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float kv = (float)ko[T / 2][4 * (T % 2) + r], qv = (float)qo[T / 2][4 * (T % 2) + r];
                    qs[r] = gdr_sum16(qv * aq[T][r]);
                    kw[r] = gdr_sum16(kv * ar[T][r]);
                    ku[r] = gdr_sum16(kv * ac[T][r]);
                }
                if (r16 == 0) {
                    *reinterpret_cast<ssd_f32x4 *>(&sDot[w][0][16 * T + 4 * g4]) = qs;
                    *reinterpret_cast<ssd_f32x4 *>(&sDot[w][1][16 * T + 4 * g4]) = kw;
                    *reinterpret_cast<ssd_f32x4 *>(&sDot[w][2][16 * T + 4 * g4]) = ku;
                }
            }
            ac[T] -= ar[T] * gdr_ld4(&sTab[kTBeta * kGdrC + 16 * T + 4 * g4]);
            __builtin_amdgcn_sched_barrier(0);
            ssd_f32x4 tq = gdr_zero4(), tr = gdr_zero4(), te = gdr_zero4(), ta = gdr_zero4();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s <= T / 2) {
                    const GdrSplit<3> ao = gdr_ld_perm_parts<3>(&sPA[(16 * T + r16) * kGdrRS + 32 * s + 4 * g4], PL);
                    const GdrSplit<3> eo = gdr_ld_perm_parts<3>(&sPE[(16 * T + r16) * kGdrRS + 32 * s + 4 * g4], PL);
#pragma unroll
                    for (int k = 2; k >= 0; --k) {
                        tq = ssd_mfma(ao.part[k], ko[s], tq);
                        tr = ssd_mfma(eo.part[k], ko[s], tr);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                if (s >= T / 2) {
                    const GdrSplit<3> eo = gdr_ld_col_parts<3>(sPE, kGdrRS, 32 * s + 4 * g4, 16 * T, r16, PL);
                    const GdrSplit<3> ao = gdr_ld_col_parts<3>(sPA, kGdrRS, 32 * s + 4 * g4, 16 * T, r16, PL);
#pragma unroll
                    for (int k = 2; k >= 0; --k) {
                        te = ssd_mfma(eo.part[k], ko[s], te);
                        ta = ssd_mfma(ao.part[k], qo[s], ta);
                    }
                }
            }
            aq[T] += tq;
            ac[T] += ta - te - tr;
            dq[T] = ONE ? aq[T] : dq[T] + aq[T];
            dk[T] = ONE ? ac[T] : dk[T] + ac[T];
            __builtin_amdgcn_sched_barrier(0);
        }
        ds = gdr_last64(gdr_prefix64(ds, lane));
        if (lane == 0) sDs[w] = ds;
        __syncthreads();
        if (w == 0) {
            // sums that run on from the tokens before (of U D') and back from those
            // behind (of S, whose lanes count from the last token)
            const int back = kGdrC - 1 - lane;
            double whole = 0.0, before = 0.0, behind = 0.0, pairs = 0.0, kwb = 0.0;
            float kw = 0.0f, es = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                whole += sDs[k];
                before += lane > 0 ? sDot[k][2][lane - 1] : 0.0f;
                behind += sDot[k][0][back];
                kwb += sDot[k][1][back];
                kw += sDot[k][1][lane];
                pairs += sDot[k][3][lane];
            }
#pragma unroll
            for (int J = 0; J < 4; ++J) es += J <= lane / 16 ? sEs[J][lane] : 0.0f;
            behind = gdr_prefix64(behind - (double)sTab[kTBeta * kGdrC + back] * kwb, lane);
            before = gdr_prefix64(before, lane);
            const float dlog = (float)(whole * (double)sTab[kTHead * kGdrC + kGdrC - 1] + before + __shfl(behind, back) + pairs);
            const float step = sTab[kTStep * kGdrC + lane];
            const float ddt = dlog * p.A[h] * sTab[kTDstep * kGdrC + lane];
            double pA = lane < nv && dlog != 0.0f ? (double)dlog * step : 0.0;   // (step may be infinite)
            double pb = lane < nv ? (double)ddt : 0.0;
            if (lane < nv) {
                const int64_t o = (row0 + lane) * p.H + h;
                p.ddt[o] = ssd_to_bf(ddt);
                p.dbeta[o] = ssd_to_bf((sWv[lane] - kw - es) * sTab[kTDbeta * kGdrC + lane]);
            }
            pA = gdr_last64(gdr_prefix64(pA, lane));
            pb = gdr_last64(gdr_prefix64(pb, lane));
            if (lane == 0) {
                p.part[2 * id] = (float)pA;
                p.part[2 * id + 1] = (float)pb;
            }
        }
    }
    // the gradients of the rows as given: through the unit lengths, whose rows'
    // products with their gradients all waves need
    if (p.qk_norm) {
        __syncthreads();
#pragma unroll
        for (int T = 0; T < 4; ++T) {
            ssd_f32x4 qd, kd;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                qd[r] = gdr_sum16(ssd_bf(sQ[(16 * T + 4 * g4 + r) * KS + n0 + r16]) * dq[T][r]);
                kd[r] = gdr_sum16(ssd_bf(sK[(16 * T + 4 * g4 + r) * KS + n0 + r16]) * dk[T][r]);
            }
            if (r16 == 0) {
                *reinterpret_cast<ssd_f32x4 *>(&sDot[w][0][16 * T + 4 * g4]) = qd;
                *reinterpret_cast<ssd_f32x4 *>(&sDot[w][1][16 * T + 4 * g4]) = kd;
            }
        }
        __syncthreads();
        if (tid < 2 * kGdrC) {
            // rq^2 q . dq and rk^2 k . dk of row tid % 64, into the table's place
            const int of = tid >> 6;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) sum += sDot[k][of][lane];
            const float u = sTab[(of ? kTRk : kTUq) * kGdrC + lane];
            sTab[(of ? kTRk : kTUq) * kGdrC + lane] = u * u * sum;
        }
        __syncthreads();
    }
    const uint32_t gs = (uint32_t)(p.G * N);
    const __amdgpu_buffer_rsrc_t rdq = ssd_buffer(p.dq + (row0 * p.G + g) * N, 2u * ((uint32_t)(nv - 1) * gs + N));
    const __amdgpu_buffer_rsrc_t rdk = ssd_buffer(p.dk + (row0 * p.G + g) * N, 2u * ((uint32_t)(nv - 1) * gs + N));
#pragma unroll
    for (int T = 0; T < 4; ++T) {
        ssd_f32x4 fq = gdr_zero4(), fk = gdr_zero4();
        if (p.qk_norm) {
            fq = gdr_ld4(&sTab[kTUq * kGdrC + 16 * T + 4 * g4]);
            fk = gdr_ld4(&sTab[kTRk * kGdrC + 16 * T + 4 * g4]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * T + 4 * g4 + r;
            const float a = dq[T][r] - fq[r] * ssd_bf(sQ[i * KS + n0 + r16]);
            const float c = dk[T][r] - fk[r] * ssd_bf(sK[i * KS + n0 + r16]);
            // rows past the end are dropped by the buffers' ranges
            const int o = (int)(2u * ((uint32_t)i * gs + n0 + r16));
            __builtin_amdgcn_raw_buffer_store_b16(ssd_to_bf(a), rdq, o, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b16(ssd_to_bf(c), rdk, o, 0, 0);
        }
    }
}

// dA and ddt_bias of head h: the chunks' parts, batch row by batch row
static __global__ __launch_bounds__(256) void gdr_reduce_kernel(const GdrParams p) {
    __shared__ double s[2][256];
    const int h = blockIdx.x, tid = threadIdx.x;
    double a = 0.0, c = 0.0;
    const int64_t n = (int64_t)p.batch * p.nc;
    for (int64_t q = tid; q < n; q += 256) {
        const int64_t id = ((q / p.nc) * p.H + h) * p.nc + q % p.nc;
        a += p.part[2 * id];
        c += p.part[2 * id + 1];
    }
    s[0][tid] = a;
    s[1][tid] = c;
    __syncthreads();
    for (int o = 128; o >= 1; o >>= 1) {
        if (tid < o) {
            s[0][tid] += s[0][tid + o];
            s[1][tid] += s[1][tid + o];
        }
        __syncthreads();
    }
    if (tid == 0) {
        p.dA[h] = (float)s[0][0];
        if (p.ddt_bias) p.ddt_bias[h] = (float)s[1][0];
    }
}

#endif  // SSM_GDR_INSTANTIATE

}  // namespace ssm_detail
