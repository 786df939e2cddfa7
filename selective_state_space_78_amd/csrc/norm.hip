// The norms around a mixer block: the residual add and RMS norm before it, the
// gated RMS norm behind it, and their gradients (include/ssm_scan.h states
// them). Every one is bound by memory: a row is read once, kept in registers
// between its sums and its outputs, and every output is written once.
//
// A row (of one group) is taken by LPS lanes, each holding NV pieces of VEC
// consecutive channels: a part of a wave for short rows (a norm per head), a
// wave up to 2048 channels, a workgroup up to 8192. Longer rows, and rows of
// unaligned channels beyond 1024, are read twice (the second time from L2).
// Pieces are 16 bytes of the narrower type when the channels, the strides and
// the pointers allow it, single channels otherwise.
//
// Backward: with n = f / rms and the incoming w dy, one pass over the row gives
// sum f^2 and sum f w dy, which determine df = (w dy - n mean(n w dy)) / rms. The
// sums over rows (dweight, dscale) are kept per channel in registers while a
// workgroup walks its rows, added across the workgroup's row slots in LDS and
// written as one partial row per workgroup; norm_reduce_kernel adds those in a
// fixed order, so no result depends on timing.
//
// Measured, at a device copy rate of 5.0 to 5.4 TB/s: 65536 rows of 32 groups of 128
// bf16 channels forward 0.28 ms (5.8 TB/s), backward 0.57 ms (4.7 TB/s); 8192 rows
// of 768 with an fp32 residual forward 13 us, backward 24 us and its sums 6.5 us (the
// tensors stay in the cache). Single channels (widths that are no multiple of a
// piece): 1.3 to 1.8 TB/s in bf16, 2.9 to 3.5 in fp32. The next segment's reads ahead of this one's sums
// measured 7% slower (registers), stores past the cache 3% faster, but what comes
// next reads these outputs.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "ssm_scan.h"
#include "abi_util.hpp"
#include "matrix_ops.hpp"
#include "scan_kernels.hpp"

namespace {

using namespace ssm_detail;

constexpr int kMaxWg = 1024;       // workgroups that walk rows in a backward: 4 per CU

struct NormParams {
    const void *x, *z, *res, *dy, *dr;   // res: the residual (forward), r (backward)
    const float *scale, *weight;
    void *r, *y, *dx, *dz, *dres;
    float *dweight, *dscale, *part;      // part: (workgroup, dweight and dscale, dim)
    float *stat;                         // long rows' backward: (row, 2)
    int64_t rows, groups, dim;           // rows of x; groups and channels per row
    int64_t xs, zs;
    float eps, inv_dim;
    int gate_first, shared;
    int slabs;                           // backward: workgroups per group
};

template <typename T, int VEC>
__device__ __forceinline__ void ld(const void *base, int64_t off, float (&v)[VEC]) {
    const T *p = static_cast<const T *>(base) + off;
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 2) v[0] = ssd_bf(*p);
        else v[0] = *p;
    } else if constexpr (sizeof(T) == 2) {
        static_assert(VEC == 8);
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p + e);
            v[e] = a.x; v[e + 1] = a.y; v[e + 2] = a.z; v[e + 3] = a.w;
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void st(void *base, int64_t off, const float (&v)[VEC]) {
    T *p = static_cast<T *>(base) + off;
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 2) *p = ssd_to_bf(v[0]);
        else *p = v[0];
    } else if constexpr (sizeof(T) == 2) {
        static_assert(VEC == 8);
        *reinterpret_cast<uint4 *>(p) =
            uint4{ssd_pack(v[0], v[1]), ssd_pack(v[2], v[3]), ssd_pack(v[4], v[5]), ssd_pack(v[6], v[7])};
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) *reinterpret_cast<float4 *>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
}

// row and group of a segment; segments fit 32 bits (64-bit division costs more than
// a short row's arithmetic)
__device__ __forceinline__ void place(int64_t seg, int64_t groups, int64_t &row, int64_t &g) {
    const uint32_t q = (uint32_t)seg / (uint32_t)groups;
    row = q;
    g = (uint32_t)seg - q * (uint32_t)groups;
}

template <typename T> __device__ __forceinline__ float rounded(float v) {
    if constexpr (sizeof(T) == 2) return ssd_bf(ssd_to_bf(v));
    else return v;
}

// Sums of a and b over the LPS lanes of a row (all threads of the workgroup
// call it together when LPS is 256)
template <int LPS>
__device__ __forceinline__ void row_sum(float &a, float &b, float (*buf)[2]) {
#pragma unroll
    for (int o = 1; o < (LPS < 64 ? LPS : 64); o <<= 1) {
        a += __shfl_xor(a, o);
        b += __shfl_xor(b, o);
    }
    if constexpr (LPS == 256) {
        const int w = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            buf[w][0] = a;
            buf[w][1] = b;
        }
        __syncthreads();
        a = (buf[0][0] + buf[1][0]) + (buf[2][0] + buf[3][0]);
        b = (buf[0][1] + buf[1][1]) + (buf[2][1] + buf[3][1]);
    }
}

// The logistic sigmoid to a few half steps at any z: the exponent's product is taken
// to twice fp32's digits (rounded to fp32 its exponential would be |z| half steps
// off), and 1 + e scaled so that the reciprocal stays a normal number up to e's
// overflow. (65536 rows of 32 x 128, forward and backward: with expf and a division
// 1070 us, so 865, y within 6 half steps of its own size at gates to 1e-36.)
__device__ __forceinline__ float sigm(float z) {
    constexpr float kLog2eLow = 1.92596299e-8f, kScale = 1.0f / 256.0f;
    const float c = __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f), t = c * -kLog2e;
    const float low = fmaf(c, -kLog2eLow, fmaf(c, -kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t) * fmaf(low, 0.69314718f, 1.0f);
    return __builtin_amdgcn_rcpf(fmaf(e, kScale, kScale)) * kScale;
}

// What is normed, and what its gradient needs, of VEC channels. A policy per
// operator: T is the element type, R the residual's.
template <typename T_, typename R_> struct Pre {
    typedef T_ T;
    typedef R_ R;
    static constexpr bool kGated = false;
    template <int VEC>
    static __device__ __forceinline__ void normed(const NormParams &p, int64_t row, int64_t g, int64_t c, float (&f)[VEC],
                                                  float (&)[VEC]) {
        float x[VEC];
        ld<T, VEC>(p.x, row * p.xs + c, x);
        if (p.scale) {
            float s[VEC];
            ld<float, VEC>(p.scale, c, s);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] *= s[e];
        }
        if (p.res) {
            ld<R, VEC>(p.res, row * p.dim + c, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] += x[e];
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = x[e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = rounded<R>(f[e]);
        if (p.r) st<R, VEC>(p.r, row * p.dim + c, f);
    }
};

template <typename T_> struct Gated {
    typedef T_ T;
    typedef T_ R;
    static constexpr bool kGated = true;
    // f, and the gate silu(z) (1 without z)
    template <int VEC>
    static __device__ __forceinline__ void normed(const NormParams &p, int64_t row, int64_t g, int64_t c, float (&f)[VEC],
                                                  float (&gate)[VEC]) {
        ld<T, VEC>(p.x, row * p.xs + g * p.dim + c, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) gate[e] = 1.0f;
        if (p.z) {
            float z[VEC];
            ld<T, VEC>(p.z, row * p.zs + g * p.dim + c, z);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                gate[e] = z[e] * sigm(z[e]);
                if (p.gate_first) f[e] *= gate[e];
            }
        }
    }
};

// ---------------------------------------------------------------------------
// Forward: a workgroup of 256 threads takes 256 / LPS rows. NV pieces per lane
// in registers; NV == 0: the row is read twice.
template <typename P, int VEC, int LPS, int NV>
__global__ __launch_bounds__(256) void norm_fwd_kernel(const NormParams p) {
    __shared__ float buf[4][2];
    constexpr int RPW = 256 / LPS;
    const int l = threadIdx.x % LPS;
    const int64_t seg = (int64_t)blockIdx.x * RPW + threadIdx.x / LPS;
    const bool live = seg < p.rows * p.groups;
    int64_t row, g;
    place(live ? seg : 0, p.groups, row, g);
    const float *wt = p.weight + (P::kGated && !p.shared ? g * p.dim : 0);
    const int64_t yo = row * p.groups * p.dim + g * p.dim;
    float ss = 0.0f, unused = 0.0f;
    auto finish = [&](int64_t c, const float (&f)[VEC], const float (&gate)[VEC], float inv) {
        float wv[VEC], y[VEC];
        ld<float, VEC>(wt, c, wv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            y[e] = f[e] * inv * wv[e];
            if (P::kGated && !p.gate_first) y[e] *= gate[e];
        }
        st<typename P::T, VEC>(p.y, yo + c, y);
    };
    if constexpr (NV > 0) {
        float f[NV][VEC], gate[P::kGated ? NV : 1][VEC];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = (int64_t)(v * LPS + l) * VEC;
            if (live && c < p.dim) {
                P::template normed<VEC>(p, row, g, c, f[v], gate[P::kGated ? v : 0]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = fmaf(f[v][e], f[v][e], ss);
            }
        }
        row_sum<LPS>(ss, unused, buf);
        const float inv = 1.0f / sqrtf(ss * p.inv_dim + p.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = (int64_t)(v * LPS + l) * VEC;
            if (live && c < p.dim) finish(c, f[v], gate[P::kGated ? v : 0], inv);
        }
    } else {
        float f[VEC], gate[VEC];
        for (int64_t c = (int64_t)l * VEC; c < p.dim; c += (int64_t)LPS * VEC) {
            P::template normed<VEC>(p, row, g, c, f, gate);
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss = fmaf(f[e], f[e], ss);
        }
        row_sum<LPS>(ss, unused, buf);
        const float inv = 1.0f / sqrtf(ss * p.inv_dim + p.eps);
        for (int64_t c = (int64_t)l * VEC; c < p.dim; c += (int64_t)LPS * VEC) {
            // the residual may have been overwritten by r, which is then what was normed
            if constexpr (P::kGated) P::template normed<VEC>(p, row, g, c, f, gate);
            else if (p.r) ld<typename P::R, VEC>(p.r, row * p.dim + c, f);
            else P::template normed<VEC>(p, row, g, c, f, gate);
            finish(c, f, gate, inv);
        }
    }
}

// ---------------------------------------------------------------------------
// Backward of VEC channels: what is read (kept until the row's sums are known),
// then, given 1/rms and m = mean(n w dy), the outputs and what the channels add
// to dweight and dscale.
template <typename P, int VEC> struct BwdIn {
    float f[VEC], up[VEC];             // normed, incoming (before weight)
    float x[VEC], z[VEC], dy[VEC];     // gated: as read; prenorm: x with a scale, dr in z
};

template <typename P, int VEC>
__device__ __forceinline__ void bwd_load(const NormParams &p, int64_t row, int64_t g, int64_t c, BwdIn<P, VEC> &o) {
    typedef typename P::T T;
    const int64_t yo = row * p.groups * p.dim + g * p.dim + c;
    ld<T, VEC>(p.dy, yo, o.dy);
    if constexpr (P::kGated) {
        ld<T, VEC>(p.x, row * p.xs + g * p.dim + c, o.x);
        if (p.z) ld<T, VEC>(p.z, row * p.zs + g * p.dim + c, o.z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float gate = p.z ? o.z[e] * sigm(o.z[e]) : 1.0f;
            o.f[e] = p.gate_first ? o.x[e] * gate : o.x[e];
            o.up[e] = p.gate_first ? o.dy[e] : o.dy[e] * gate;
        }
    } else {
        ld<typename P::R, VEC>(p.res, row * p.dim + c, o.f);
        if (p.dr) ld<typename P::R, VEC>(p.dr, yo, o.z);
        if (p.scale) ld<T, VEC>(p.x, row * p.xs + c, o.x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.up[e] = o.dy[e];
    }
}

template <typename P, int VEC>
__device__ __forceinline__ void bwd_finish(const NormParams &p, int64_t row, int64_t g, int64_t c, const BwdIn<P, VEC> &in,
                                           const float (&wt)[VEC], float inv, float m, float (&dw)[VEC], float (&dsc)[VEC]) {
    typedef typename P::T T;
    const int64_t yo = row * p.groups * p.dim + g * p.dim + c;
    float df[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const float n = in.f[e] * inv;
        df[e] = inv * (in.up[e] * wt[e] - n * m);
        dw[e] = fmaf(in.up[e], n, dw[e]);
    }
    if constexpr (P::kGated) {
        if (p.z) {
            float dx[VEC], dz[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float z = in.z[e], s = sigm(z);
                const float dgate = s * (1.0f + z * (1.0f - s));
                dx[e] = p.gate_first ? df[e] * z * s : df[e];
                dz[e] = (p.gate_first ? df[e] * in.x[e] : in.dy[e] * in.f[e] * inv * wt[e]) * dgate;
            }
            st<T, VEC>(p.dz, yo, dz);
            st<T, VEC>(p.dx, yo, dx);
        } else {
            st<T, VEC>(p.dx, yo, df);
        }
    } else {
        if (p.dr) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) df[e] += in.z[e];
        }
        if (p.dres) st<typename P::R, VEC>(p.dres, yo, df);
        if (p.scale) {
            float s[VEC];
            ld<float, VEC>(p.scale, c, s);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                dsc[e] = fmaf(df[e], in.x[e], dsc[e]);
                df[e] *= s[e];
            }
        }
        st<T, VEC>(p.dx, yo, df);
    }
}

// A workgroup walks the rows of one group (every row and group in order with a
// shared weight) in steps of slabs * RPW; its channels' sums stay in registers.
template <typename P, int VEC, int LPS, int NV>
__global__ __launch_bounds__(256) void norm_bwd_kernel(const NormParams p) {
    __shared__ float buf[4][2];
    constexpr int RPW = 256 / LPS;
    __shared__ float acc[RPW > 1 ? 256 * VEC * NV : 1];
    const int l = threadIdx.x % LPS, slot = threadIdx.x / LPS;
    const bool fixed = P::kGated && !p.shared;          // a workgroup per group
    const int64_t gfix = fixed ? blockIdx.x % p.groups : 0;
    const int64_t slab = fixed ? blockIdx.x / p.groups : blockIdx.x;
    const int64_t total = fixed ? p.rows : p.rows * p.groups;
    float wt[NV][VEC], dw[NV][VEC], dsc[P::kGated ? 1 : NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = (int64_t)(v * LPS + l) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) wt[v][e] = dw[v][e] = dsc[P::kGated ? 0 : v][e] = 0.0f;
        if (c < p.dim) ld<float, VEC>(p.weight, gfix * p.dim + c, wt[v]);
    }
    for (int64_t s0 = slab * RPW; s0 < total; s0 += (int64_t)p.slabs * RPW) {
        const int64_t seg = s0 + slot;
        const bool live = seg < total;
        int64_t row = live ? seg : 0, g = gfix;
        if (!fixed) place(live ? seg : 0, p.groups, row, g);
        BwdIn<P, VEC> in[NV];
        float ss = 0.0f, sw = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = (int64_t)(v * LPS + l) * VEC;
            if (live && c < p.dim) {
                bwd_load<P, VEC>(p, row, g, c, in[v]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    ss = fmaf(in[v].f[e], in[v].f[e], ss);
                    sw = fmaf(in[v].f[e], in[v].up[e] * wt[v][e], sw);
                }
            }
        }
        row_sum<LPS>(ss, sw, buf);
        const float inv = 1.0f / sqrtf(ss * p.inv_dim + p.eps);
        const float m = inv * sw * p.inv_dim;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = (int64_t)(v * LPS + l) * VEC;
            if (live && c < p.dim) bwd_finish<P, VEC>(p, row, g, c, in[v], wt[v], inv, m, dw[v], dsc[P::kGated ? 0 : v]);
        }
    }
    // the row slots' sums, in order
    const int64_t outs = P::kGated ? 1 : 2;
    float *part = p.part + (slab * outs * (fixed ? p.groups : 1) + gfix) * p.dim;
    auto join = [&](const float (&d)[NV][VEC], float *dst) {
        if constexpr (RPW > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[slot * (LPS * VEC * NV) + (v * LPS + l) * VEC + e] = d[v][e];
            __syncthreads();
            for (int64_t c = threadIdx.x; c < p.dim; c += 256) {
                float s = 0.0f;
                for (int k = 0; k < RPW; ++k) s += acc[k * (LPS * VEC * NV) + c];
                dst[c] = s;
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int64_t c = (int64_t)(v * LPS + l) * VEC;
                if (c < p.dim)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) dst[c + e] = d[v][e];
            }
        }
    };
    join(dw, part);
    if constexpr (!P::kGated) {
        if (p.scale) join(dsc, part + p.dim);
    }
}

// Long rows: 1 / rms and m of every row, then a workgroup per block of channels
// and slab of rows.
template <typename P, int VEC>
__global__ __launch_bounds__(256) void norm_bwd_stat_kernel(const NormParams p) {
    __shared__ float buf[4][2];
    const int64_t seg = blockIdx.x;
    int64_t row, g;
    place(seg, p.groups, row, g);
    const float *weight = p.weight + (P::kGated && !p.shared ? g * p.dim : 0);
    float ss = 0.0f, sw = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.dim; c += 256 * VEC) {
        BwdIn<P, VEC> in;
        float wt[VEC];
        bwd_load<P, VEC>(p, row, g, c, in);
        ld<float, VEC>(weight, c, wt);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            ss = fmaf(in.f[e], in.f[e], ss);
            sw = fmaf(in.f[e], in.up[e] * wt[e], sw);
        }
    }
    row_sum<256>(ss, sw, buf);
    if (threadIdx.x == 0) {
        const float inv = 1.0f / sqrtf(ss * p.inv_dim + p.eps);
        p.stat[2 * seg] = inv;
        p.stat[2 * seg + 1] = inv * sw * p.inv_dim;
    }
}

template <typename P, int VEC>
__global__ __launch_bounds__(256) void norm_bwd_cols_kernel(const NormParams p) {
    const int64_t cb = (p.dim + 256 * VEC - 1) / (256 * VEC);       // channel blocks of a row
    const bool fixed = P::kGated && !p.shared;
    const int64_t c = ((int64_t)(blockIdx.x % cb) * 256 + threadIdx.x) * VEC;
    const int64_t rest = blockIdx.x / cb;
    const int64_t gfix = fixed ? rest % p.groups : 0, slab = fixed ? rest / p.groups : rest;
    const int64_t total = fixed ? p.rows : p.rows * p.groups;
    if (c >= p.dim) return;
    float wt[VEC], dw[VEC], dsc[VEC];
    ld<float, VEC>(p.weight, gfix * p.dim + c, wt);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[e] = dsc[e] = 0.0f;
    for (int64_t s = slab; s < total; s += p.slabs) {
        int64_t row = s, g = gfix;
        if (!fixed) place(s, p.groups, row, g);
        const int64_t seg = fixed ? row * p.groups + g : s;
        BwdIn<P, VEC> in;
        bwd_load<P, VEC>(p, row, g, c, in);
        bwd_finish<P, VEC>(p, row, g, c, in, wt, p.stat[2 * seg], p.stat[2 * seg + 1], dw, dsc);
    }
    const int64_t outs = P::kGated ? 1 : 2;
    float *part = p.part + (slab * outs * (fixed ? p.groups : 1) + gfix) * p.dim + c;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        part[e] = dw[e];
        if (!P::kGated && p.scale) part[p.dim + e] = dsc[e];
    }
}

// Column sums of the partial rows (slabs of `cols` floats): 16 columns and 64 runs
// of slabs per workgroup, each run in order, then the runs pairwise
constexpr int kRunCols = 16, kRuns = 64;
__global__ __launch_bounds__(kRunCols * kRuns) void norm_reduce_kernel(const float *part, int slabs, int64_t cols,
                                                                       int64_t first, float *o0, float *o1) {
    __shared__ float s[kRuns][kRunCols];
    const int l = threadIdx.x % kRunCols, run = threadIdx.x / kRunCols;
    const int64_t c = (int64_t)blockIdx.x * kRunCols + l;
    float a = 0.0f;
    if (c < cols)
        for (int k = run; k < slabs; k += kRuns) a += part[(int64_t)k * cols + c];
    s[run][l] = a;
    for (int o = kRuns / 2; o >= 1; o >>= 1) {
        __syncthreads();
        if (run < o) s[run][l] += s[run + o][l];
    }
    if (run == 0 && c < cols) {
        if (c < first) o0[c] = s[0][l];
        else if (o1) o1[c - first] = s[0][l];
    }
}

// ---------------------------------------------------------------------------
// Launching

struct Shape {
    int lps, nv;    // nv 0: long rows
};

// The narrowest team of lanes that holds a row in at most 4 pieces per lane
Shape shape_for(int64_t dim, int vec) {
    const int64_t pieces = (dim + vec - 1) / vec;
    if (pieces <= 8) return {8, 1};
    if (pieces <= 16) return {16, 1};
    if (pieces <= 32) return {32, 1};
    if (pieces <= 64) return {64, 1};
    if (pieces <= 128) return {64, 2};
    if (pieces <= 256) return {64, 4};
    if (pieces <= 512) return {256, 2};
    if (pieces <= 1024) return {256, 4};
    return {256, 0};
}

#define NORM_SHAPES(X) X(8, 1) X(16, 1) X(32, 1) X(64, 1) X(64, 2) X(64, 4) X(256, 2) X(256, 4)

template <typename P, int VEC>
hipError_t launch_fwd(const NormParams &p, hipStream_t st) {
    const Shape s = shape_for(p.dim, VEC);
    const int64_t blocks = (p.rows * p.groups + 256 / s.lps - 1) / (256 / s.lps);
    if (!grid_ok(blocks, 256)) return hipErrorInvalidConfiguration;
#define NORM_CASE(LPS, NV)                                                                                              \
    if (s.lps == LPS && s.nv == NV)                                                                                    \
        hipLaunchKernelGGL((norm_fwd_kernel<P, VEC, LPS, NV>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    NORM_SHAPES(NORM_CASE)
    NORM_CASE(256, 0)
#undef NORM_CASE
    return hipGetLastError();
}

// Workgroups per group that walk rows: enough for the chip, at most the rows
int slabs_for(int64_t rows, int64_t groups, int64_t dim, bool fixed, int vec) {
    const Shape s = shape_for(dim, vec);
    const int64_t walks = fixed ? groups : 1, total = fixed ? rows : rows * groups;
    const int64_t rpw = s.nv == 0 ? 1 : 256 / s.lps;
    const int64_t cb = s.nv == 0 ? (dim + 256 * vec - 1) / (256 * vec) : 1;
    const int64_t want = std::max<int64_t>(1, kMaxWg / std::max<int64_t>(1, walks * cb));
    return (int)std::max<int64_t>(1, std::min((total + rpw - 1) / rpw, want));
}

template <typename P, int VEC>
hipError_t launch_bwd(NormParams &p, hipStream_t st) {
    const bool fixed = P::kGated && !p.shared;
    const Shape s = shape_for(p.dim, VEC);
    p.slabs = slabs_for(p.rows, p.groups, p.dim, fixed, VEC);
    const int64_t walks = fixed ? p.groups : 1;
    const int64_t cols = (P::kGated ? 1 : 2) * walks * p.dim;
    // without a scale the second half of a partial row is not written, and not read
    const int64_t sums = ((P::kGated || p.scale ? cols : p.dim) + kRunCols - 1) / kRunCols;
    if (!grid_ok(sums, kRunCols * kRuns)) return hipErrorInvalidConfiguration;
    if (s.nv == 0) {
        const int64_t cb = (p.dim + 256 * VEC - 1) / (256 * VEC);
        const int64_t b1 = p.rows * p.groups, b2 = cb * walks * p.slabs;
        if (!grid_ok(b1, 256) || !grid_ok(b2, 256)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((norm_bwd_stat_kernel<P, VEC>), dim3((unsigned)b1), dim3(256), 0, st, p);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((norm_bwd_cols_kernel<P, VEC>), dim3((unsigned)b2), dim3(256), 0, st, p);
    } else {
        const int64_t blocks = walks * p.slabs;
        if (!grid_ok(blocks, 256)) return hipErrorInvalidConfiguration;
#define NORM_CASE(LPS, NV)                                                                                              \
    if (s.lps == LPS && s.nv == NV)                                                                                    \
        hipLaunchKernelGGL((norm_bwd_kernel<P, VEC, LPS, NV>), dim3((unsigned)blocks), dim3(256), 0, st, p);
        NORM_SHAPES(NORM_CASE)
#undef NORM_CASE
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)sums), dim3(kRunCols * kRuns), 0, st, p.part, p.slabs, cols,
                       P::kGated ? cols : p.dim, p.dweight, p.dscale);
    return hipGetLastError();
}

size_t bwd_bytes(int64_t rows, int64_t groups, int64_t dim, bool gated, bool shared) {
    if (rows == 0) return 0;
    const bool fixed = gated && !shared;
    const int64_t cols = (gated ? 1 : 2) * (fixed ? groups : 1) * dim;
    // the slabs and the path depend on the piece width, which the pointers decide
    const int64_t slabs = std::max(slabs_for(rows, groups, dim, fixed, 1),
                                   std::max(slabs_for(rows, groups, dim, fixed, 4), slabs_for(rows, groups, dim, fixed, 8)));
    return align256((size_t)slabs * cols * 4) + align256((size_t)rows * groups * 8);
}

bool dtype_ok(int t) { return t == SSM_F32 || t == SSM_BF16; }
size_t esize(int t) { return t == SSM_BF16 ? 2 : 4; }

// One output may equal one input exactly (same address and size)
bool clash(Range out, const Range *in, int n, const void *same = nullptr) {
    for (int k = 0; k < n; ++k)
        if (overlaps(out, in[k]) && !(same != nullptr && in[k].lo == (uintptr_t)same && in[k].lo == out.lo && in[k].hi == out.hi))
            return true;
    return false;
}

int check_pre(const ssm_prenorm_desc *desc) {
    if (desc == nullptr) return SSM_ERR_NULL;
    const ssm_prenorm_desc &d = *desc;
    int64_t n;
    if (d.rows < 0 || d.dim < 1 || d.dim > (1 << 20) || d.x_stride < 0 || (d.x_stride != 0 && d.x_stride < d.dim))
        return SSM_ERR_SHAPE;
    if (!mul_ok(d.rows, std::max<int64_t>(d.x_stride, d.dim), &n) || n > INT64_MAX / 16 || d.rows > INT32_MAX)
        return SSM_ERR_SHAPE;
    if (!dtype_ok(d.dtype) || !dtype_ok(d.residual_dtype)) return SSM_ERR_DTYPE;
    if (d.residual_dtype != d.dtype && d.residual_dtype != SSM_F32) return SSM_ERR_UNSUPPORTED;
    if (!(d.eps >= 0.0f) || d.eps > 3e38f || d.reserved != 0) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

int check_gated(const ssm_gated_norm_desc *desc) {
    if (desc == nullptr) return SSM_ERR_NULL;
    const ssm_gated_norm_desc &d = *desc;
    int64_t w, n, segs;
    if (d.rows < 0 || d.groups < 1 || d.dim < 1 || d.dim > (1 << 20) || !mul_ok(d.groups, d.dim, &w) || w > INT32_MAX)
        return SSM_ERR_SHAPE;
    if (d.x_stride < 0 || d.z_stride < 0 || (d.x_stride != 0 && d.x_stride < w) || (d.z_stride != 0 && d.z_stride < w))
        return SSM_ERR_SHAPE;
    if (!mul_ok(d.rows, std::max(w, std::max(d.x_stride, d.z_stride)), &n) || n > INT64_MAX / 16 ||
        !mul_ok(d.rows, d.groups, &segs) || segs > INT32_MAX)
        return SSM_ERR_SHAPE;
    if (!dtype_ok(d.dtype)) return SSM_ERR_DTYPE;
    if ((d.gate_first & ~1) || (d.weight_shared & ~1) || !(d.eps >= 0.0f) || d.eps > 3e38f) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

// Whether rows move in 16-byte pieces of the narrower type (`vec` elements)
bool wide(int64_t dim, int vec, const int64_t *strides, int ns, const void *const *ptr, int np) {
    if (dim % vec != 0) return false;
    for (int k = 0; k < ns; ++k)
        if (strides[k] % vec != 0) return false;
    for (int k = 0; k < np; ++k)
        if (ptr[k] && !aligned(ptr[k], 16)) return false;
    return true;
}

int64_t span(int64_t rows, int64_t stride, int64_t width) { return rows > 0 ? (rows - 1) * stride + width : 0; }

template <bool BWD, typename P, int VEC>
hipError_t go(NormParams &p, hipStream_t st) {
    if constexpr (BWD) return launch_bwd<P, VEC>(p, st);
    else return launch_fwd<P, VEC>(p, st);
}

template <bool BWD>
hipError_t go_pre(const ssm_prenorm_desc &d, NormParams &p, bool w, hipStream_t st) {
    if (d.dtype == SSM_F32) return w ? go<BWD, Pre<float, float>, 4>(p, st) : go<BWD, Pre<float, float>, 1>(p, st);
    if (d.residual_dtype == SSM_F32)
        return w ? go<BWD, Pre<uint16_t, float>, 8>(p, st) : go<BWD, Pre<uint16_t, float>, 1>(p, st);
    return w ? go<BWD, Pre<uint16_t, uint16_t>, 8>(p, st) : go<BWD, Pre<uint16_t, uint16_t>, 1>(p, st);
}

template <bool BWD>
hipError_t go_gated(const ssm_gated_norm_desc &d, NormParams &p, bool w, hipStream_t st) {
    if (d.dtype == SSM_F32) return w ? go<BWD, Gated<float>, 4>(p, st) : go<BWD, Gated<float>, 1>(p, st);
    return w ? go<BWD, Gated<uint16_t>, 8>(p, st) : go<BWD, Gated<uint16_t>, 1>(p, st);
}

// What a launch came to; sizes that need too many work items are refused before the first
int status(hipError_t e) {
    return e == hipSuccess ? SSM_OK : e == hipErrorInvalidConfiguration ? SSM_ERR_SHAPE : SSM_ERR_HIP;
}

NormParams params_of(const ssm_prenorm_desc &d) {
    NormParams p{};
    p.rows = d.rows;
    p.groups = 1;
    p.dim = d.dim;
    p.xs = d.x_stride ? d.x_stride : d.dim;
    p.eps = d.eps;
    p.inv_dim = 1.0f / (float)d.dim;
    return p;
}

NormParams params_of(const ssm_gated_norm_desc &d) {
    NormParams p{};
    p.rows = d.rows;
    p.groups = d.groups;
    p.dim = d.dim;
    p.xs = d.x_stride ? d.x_stride : d.groups * d.dim;
    p.zs = d.z_stride ? d.z_stride : d.groups * d.dim;
    p.eps = d.eps;
    p.inv_dim = 1.0f / (float)d.dim;
    p.gate_first = d.gate_first;
    p.shared = d.weight_shared;
    return p;
}

// No rows: sums over them are 0
__global__ __launch_bounds__(256) void norm_zero_kernel(float *a, int64_t n, float *b, int64_t m) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) a[i] = 0.0f;
    if (b != nullptr && i < m) b[i] = 0.0f;
}

int zero_sums(float *a, int64_t n, float *b, int64_t m, hipStream_t st) {
    if (!grid_ok((std::max(n, m) + 255) / 256, 256)) return SSM_ERR_SHAPE;
    hipLaunchKernelGGL(norm_zero_kernel, dim3((unsigned)((std::max(n, m) + 255) / 256)), dim3(256), 0, st, a, n, b, m);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace

extern "C" int ssm_prenorm_fwd(const ssm_prenorm_desc *desc, const void *x, const void *residual, const float *scale,
                               const float *weight, void *r, void *y, hipStream_t stream) {
    if (const int rc = check_pre(desc)) return rc;
    const ssm_prenorm_desc &d = *desc;
    if (d.rows == 0) return SSM_OK;
    if (x == nullptr || weight == nullptr || y == nullptr) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype), er = esize(d.residual_dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(residual, er) || !aligned(r, er) || !aligned(scale, 4) ||
        !aligned(weight, 4))
        return SSM_ERR_ALIGN;
    NormParams p = params_of(d);
    const int64_t n = d.rows * d.dim;
    const Range in[] = {range_of(x, span(d.rows, p.xs, d.dim) * e), range_of(residual, n * er), range_of(scale, d.dim * 4),
                        range_of(weight, d.dim * 4)};
    const Range ry = range_of(y, n * e), rr = range_of(r, n * er);
    if (clash(ry, in, 4) || clash(rr, in, 4, residual) || overlaps(ry, rr)) return SSM_ERR_ALIAS;
    p.x = x;
    p.res = residual;
    p.scale = scale;
    p.weight = weight;
    p.r = r;
    p.y = y;
    const void *ptr[] = {x, residual, scale, weight, r, y};
    const bool w = wide(d.dim, d.dtype == SSM_F32 ? 4 : 8, &p.xs, 1, ptr, 6);
    return status(go_pre<false>(d, p, w, stream));
}

extern "C" size_t ssm_prenorm_bwd_workspace_size(const ssm_prenorm_desc *desc) {
    if (check_pre(desc) != SSM_OK) return 0;
    return bwd_bytes(desc->rows, 1, desc->dim, false, false);
}

extern "C" int ssm_prenorm_bwd(const ssm_prenorm_desc *desc, const void *dy, const void *r, const void *dr, const void *x,
                               const float *scale, const float *weight, void *dx, void *dresidual, float *dweight,
                               float *dscale, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (const int rc = check_pre(desc)) return rc;
    const ssm_prenorm_desc &d = *desc;
    if (dweight == nullptr || (scale != nullptr && dscale == nullptr)) return SSM_ERR_NULL;
    if (!aligned(dweight, 4) || (scale && !aligned(dscale, 4))) return SSM_ERR_ALIGN;
    if (d.rows == 0) return zero_sums(dweight, d.dim, scale ? dscale : nullptr, d.dim, stream);
    if (dy == nullptr || r == nullptr || weight == nullptr || dx == nullptr || (scale && x == nullptr)) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype), er = esize(d.residual_dtype);
    if (!aligned(dy, e) || !aligned(dx, e) || !aligned(r, er) || !aligned(dr, er) || !aligned(dresidual, er) ||
        (scale && (!aligned(x, e) || !aligned(scale, 4))) || !aligned(weight, 4))
        return SSM_ERR_ALIGN;
    const size_t need = bwd_bytes(d.rows, 1, d.dim, false, false);
    if (workspace == nullptr || workspace_bytes < need) return SSM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
    NormParams p = params_of(d);
    const int64_t n = d.rows * d.dim;
    const Range ws = range_of(workspace, need);
    const Range in[] = {range_of(dy, n * e), range_of(r, n * er), range_of(dr, n * er),
                        range_of(x, scale ? span(d.rows, p.xs, d.dim) * e : 0), range_of(scale, scale ? d.dim * 4 : 0),
                        range_of(weight, d.dim * 4), ws};
    const Range out[] = {range_of(dx, n * e), range_of(dresidual, dresidual ? n * er : 0), range_of(dweight, d.dim * 4),
                         range_of(dscale, scale ? d.dim * 4 : 0)};
    for (int k = 0; k < 4; ++k) {
        if (clash(out[k], in, 7, k == 1 ? dr : nullptr)) return SSM_ERR_ALIAS;
        for (int j = 0; j < k; ++j)
            if (overlaps(out[k], out[j])) return SSM_ERR_ALIAS;
    }
    for (int k = 0; k < 6; ++k)
        if (overlaps(ws, in[k])) return SSM_ERR_ALIAS;
    p.dy = dy;
    p.res = r;
    p.dr = dr;
    p.x = x;
    p.scale = scale;
    p.weight = weight;
    p.dx = dx;
    p.dres = dresidual;
    p.dweight = dweight;
    p.dscale = scale ? dscale : nullptr;
    p.stat = static_cast<float *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + align256((size_t)d.rows * 8));
    const void *ptr[] = {dy, r, dr, scale ? x : nullptr, scale, weight, dx, dresidual};
    const bool w = wide(d.dim, d.dtype == SSM_F32 ? 4 : 8, &p.xs, scale ? 1 : 0, ptr, 8);
    return status(go_pre<true>(d, p, w, stream));
}

extern "C" int ssm_gated_norm_fwd(const ssm_gated_norm_desc *desc, const void *x, const void *z, const float *weight,
                                  void *y, hipStream_t stream) {
    if (const int rc = check_gated(desc)) return rc;
    const ssm_gated_norm_desc &d = *desc;
    if (d.rows == 0) return SSM_OK;
    if (x == nullptr || weight == nullptr || y == nullptr) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype);
    if (!aligned(x, e) || !aligned(z, e) || !aligned(y, e) || !aligned(weight, 4)) return SSM_ERR_ALIGN;
    NormParams p = params_of(d);
    const int64_t width = d.groups * d.dim;
    const Range in[] = {range_of(x, span(d.rows, p.xs, width) * e), range_of(z, span(d.rows, p.zs, width) * e),
                        range_of(weight, (d.weight_shared ? d.dim : width) * 4)};
    if (clash(range_of(y, d.rows * width * e), in, 3)) return SSM_ERR_ALIAS;
    p.x = x;
    p.z = z;
    p.weight = weight;
    p.y = y;
    const int64_t strides[] = {p.xs, z ? p.zs : 0};
    const void *ptr[] = {x, z, weight, y};
    const bool w = wide(d.dim, d.dtype == SSM_F32 ? 4 : 8, strides, 2, ptr, 4);
    return status(go_gated<false>(d, p, w, stream));
}

extern "C" size_t ssm_gated_norm_bwd_workspace_size(const ssm_gated_norm_desc *desc) {
    if (check_gated(desc) != SSM_OK) return 0;
    return bwd_bytes(desc->rows, desc->groups, desc->dim, true, desc->weight_shared != 0);
}

extern "C" int ssm_gated_norm_bwd(const ssm_gated_norm_desc *desc, const void *dy, const void *x, const void *z,
                                  const float *weight, void *dx, void *dz, float *dweight, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
    if (const int rc = check_gated(desc)) return rc;
    const ssm_gated_norm_desc &d = *desc;
    const int64_t width = d.groups * d.dim, wn = d.weight_shared ? d.dim : width;
    if (dweight == nullptr) return SSM_ERR_NULL;
    if (!aligned(dweight, 4)) return SSM_ERR_ALIGN;
    if (d.rows == 0) return zero_sums(dweight, wn, nullptr, 0, stream);
    if (dy == nullptr || x == nullptr || weight == nullptr || dx == nullptr || (z && dz == nullptr)) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype);
    if (!aligned(dy, e) || !aligned(x, e) || !aligned(z, e) || !aligned(dx, e) || (z && !aligned(dz, e)) ||
        !aligned(weight, 4))
        return SSM_ERR_ALIGN;
    const size_t need = bwd_bytes(d.rows, d.groups, d.dim, true, d.weight_shared != 0);
    if (workspace == nullptr || workspace_bytes < need) return SSM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
    NormParams p = params_of(d);
    const int64_t n = d.rows * width;
    const Range ws = range_of(workspace, need);
    const Range in[] = {range_of(dy, n * e), range_of(x, span(d.rows, p.xs, width) * e),
                        range_of(z, z ? span(d.rows, p.zs, width) * e : 0), range_of(weight, wn * 4), ws};
    const Range out[] = {range_of(dx, n * e), range_of(dz, z ? n * e : 0), range_of(dweight, wn * 4)};
    for (int k = 0; k < 3; ++k) {
        if (clash(out[k], in, 5)) return SSM_ERR_ALIAS;
        for (int j = 0; j < k; ++j)
            if (overlaps(out[k], out[j])) return SSM_ERR_ALIAS;
    }
    for (int k = 0; k < 4; ++k)
        if (overlaps(ws, in[k])) return SSM_ERR_ALIAS;
    p.dy = dy;
    p.x = x;
    p.z = z;
    p.weight = weight;
    p.dx = dx;
    p.dz = dz;
    p.dweight = dweight;
    p.stat = static_cast<float *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + align256((size_t)d.rows * d.groups * 8));
    const int64_t strides[] = {p.xs, z ? p.zs : 0};
    const void *ptr[] = {dy, x, z, weight, dx, z ? dz : nullptr};
    const bool w = wide(d.dim, d.dtype == SSM_F32 ? 4 : 8, strides, 2, ptr, 6);
    return status(go_gated<true>(d, p, w, stream));
}
