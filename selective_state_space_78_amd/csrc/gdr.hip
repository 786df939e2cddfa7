// C entries of the gated delta rule (include/ssm_scan.h states it) and its
// one-token step; the chunked kernels are in gdr_kernels.hpp.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ssm_scan.h"
#include "abi_util.hpp"
#include "gdr_launch.hpp"

namespace {

using namespace ssm_detail;

// ---------------------------------------------------------------------------
// One token. Per state row p, u = w (v - a S_p . k) and
//   S_p' = a S_p + u k,  y_p = scale (a S_p . q + u k . q),
// so one read of the row gives both products and it is written once. N / 4
// lanes hold a row as 16-byte pieces; a workgroup takes 32 (N 128) or 64 (N
// 64) rows of a head, so the loads of a thread's 4 rows are in flight together
// and q and k are read once for them. Bound by memory: 256 users x 40 heads of
// 128 x 128 (1.35 GB) 0.233-0.240 ms, 5.6-5.8 TB/s; one user x 32 heads 5 us.
struct GdrStepParams {
    const uint16_t *q, *k, *v, *dt, *beta;
    const float *A, *dt_bias, *h;
    float *h_out;
    uint16_t *y;
    int64_t qs, ks, vs, dts, bs;
    int H, G, hpg, P;
    int dt_softplus, beta_sigmoid, qk_norm;
    float scale, qk_eps;
};

constexpr int kStepRows = 4;   // rows per thread

template <int N>
__global__ __launch_bounds__(256) void gdr_step_kernel(const GdrStepParams p, int blocks_per_head) {
    constexpr int LPR = N / 4, RPW = 256 / LPR;
    const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int64_t bh = blockIdx.x / blocks_per_head;
    const int p0 = (int)(blockIdx.x % blocks_per_head) * (RPW * kStepRows) + slot;
    const int h = (int)(bh % p.H), g = h / p.hpg;
    const int64_t b = bh / p.H;
    auto bf = [](uint32_t v) { return __uint_as_float(v << 16); };
    float4 s[kStepRows];
    float vv[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int pr = p0 + r * RPW;
        s[r] = pr < p.P ? *reinterpret_cast<const float4 *>(p.h + (bh * p.P + pr) * N + 4 * l) : float4{0, 0, 0, 0};
        vv[r] = pr < p.P ? bf(p.v[b * p.vs + (int64_t)h * p.P + pr]) : 0.0f;
    }
    const uint2 kw = *reinterpret_cast<const uint2 *>(p.k + b * p.ks + (int64_t)g * N + 4 * l);
    const uint2 qw = *reinterpret_cast<const uint2 *>(p.q + b * p.qs + (int64_t)g * N + 4 * l);
    float kv[4] = {bf(kw.x & 0xffffu), __uint_as_float(kw.x & 0xffff0000u), bf(kw.y & 0xffffu),
                   __uint_as_float(kw.y & 0xffff0000u)};
    float qv[4] = {bf(qw.x & 0xffffu), __uint_as_float(qw.x & 0xffff0000u), bf(qw.y & 0xffffu),
                   __uint_as_float(qw.y & 0xffff0000u)};
    float raw = bf(p.dt[b * p.dts + h]) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
    float w = bf(p.beta[b * p.bs + h]);
    if (p.dt_softplus) raw = fmaxf(raw, 0.0f) + log1pf(expf(-fabsf(raw)));
    if (p.beta_sigmoid) w = 1.0f / (1.0f + expf(-w));
    const float a = expf(raw * p.A[h]);
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        kk = fmaf(kv[e], kv[e], kk);
        qq = fmaf(qv[e], qv[e], qq);
        kq = fmaf(kv[e], qv[e], kq);
    }
    float sk[kStepRows], sq[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        sk[r] = fmaf(s[r].w, kv[3], fmaf(s[r].z, kv[2], fmaf(s[r].y, kv[1], s[r].x * kv[0])));
        sq[r] = fmaf(s[r].w, qv[3], fmaf(s[r].z, qv[2], fmaf(s[r].y, qv[1], s[r].x * qv[0])));
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) {
        kk += __shfl_xor(kk, o);
        qq += __shfl_xor(qq, o);
        kq += __shfl_xor(kq, o);
#pragma unroll
        for (int r = 0; r < kStepRows; ++r) {
            sk[r] += __shfl_xor(sk[r], o);
            sq[r] += __shfl_xor(sq[r], o);
        }
    }
    const float rk = p.qk_norm ? 1.0f / sqrtf(kk + p.qk_eps) : 1.0f;
    const float rq = p.scale * (p.qk_norm ? 1.0f / sqrtf(qq + p.qk_eps) : 1.0f);
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int pr = p0 + r * RPW;
        if (pr >= p.P) continue;
        const float u = w * (vv[r] - a * rk * sk[r]);
        const float c = u * rk;
        float4 o;
        o.x = fmaf(a, s[r].x, c * kv[0]);
        o.y = fmaf(a, s[r].y, c * kv[1]);
        o.z = fmaf(a, s[r].z, c * kv[2]);
        o.w = fmaf(a, s[r].w, c * kv[3]);
        *reinterpret_cast<float4 *>(p.h_out + (bh * p.P + pr) * N + 4 * l) = o;
        if (l == 0) p.y[bh * p.P + pr] = ssd_to_bf(rq * fmaf(a, sq[r], c * kq));
    }
}

// No tokens: the state passes through, sums over them are 0
__global__ __launch_bounds__(256) void gdr_empty_kernel(const float *from, float *to, int64_t n, float *dA, float *db,
                                                        int H) {
    const int64_t step = (int64_t)gridDim.x * 256, end = n > H ? n : H;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < end; i += step) {
        if (to != nullptr && i < n) to[i] = from != nullptr ? from[i] : 0.0f;
        if (dA != nullptr && i < H) dA[i] = 0.0f;
        if (db != nullptr && i < H) db[i] = 0.0f;
    }
}

unsigned empty_blocks(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, 8192); }

// ---------------------------------------------------------------------------
// Descriptors, layouts

struct Sizes {
    int64_t tokens, heads, state, nc;      // batch * seqlen, batch * H, elements of a state, chunks
    int64_t qs, ks, vs, dts, bs;           // resolved strides
};

// one: a single token, whose kernel addresses rows in 64 bits
int check(const ssm_gdr_desc *desc, Sizes *s, bool one = false) {
    if (desc == nullptr) return SSM_ERR_NULL;
    const ssm_gdr_desc &d = *desc;
    if (d.batch < 0 || d.seqlen < 0 || d.nheads < 1 || d.ngroups < 1 || d.nheads % d.ngroups != 0) return SSM_ERR_SHAPE;
    if (d.dtype != SSM_F32 && d.dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (d.dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    if (d.headdim < 16 || d.headdim > 256 || d.headdim % 16 != 0 || (d.dstate != 64 && d.dstate != 128))
        return SSM_ERR_UNSUPPORTED;
    if ((d.dt_softplus & ~1) || (d.beta_sigmoid & ~1) || (d.qk_norm & ~1) || !std::isfinite(d.scale))
        return SSM_ERR_UNSUPPORTED;
    if (d.qk_norm && !(d.qk_eps > 0.0f && std::isfinite(d.qk_eps))) return SSM_ERR_UNSUPPORTED;
    const int64_t H = d.nheads, G = d.ngroups, P = d.headdim, N = d.dstate;
    const int64_t width[] = {G * N, G * N, H * P, H, H};
    const int64_t given[] = {d.q_stride, d.k_stride, d.v_stride, d.dt_stride, d.beta_stride};
    int64_t *out[] = {&s->qs, &s->ks, &s->vs, &s->dts, &s->bs};
    int64_t n;
    if (!mul_ok(d.batch, d.seqlen, &s->tokens) || !mul_ok(d.batch, H, &s->heads) ||
        !mul_ok(s->heads, P * N, &s->state) || s->state > INT64_MAX / 16)
        return SSM_ERR_SHAPE;
    for (int k = 0; k < 5; ++k) {
        // a chunk's rows are addressed by 32-bit byte offsets
        if (given[k] < 0 || (given[k] != 0 && given[k] < width[k])) return SSM_ERR_SHAPE;
        *out[k] = given[k] ? given[k] : width[k];
        if ((!one && *out[k] > (INT32_MAX / 2) / kGdrC) || !mul_ok(s->tokens, *out[k], &n) || n > INT64_MAX / 4)
            return SSM_ERR_SHAPE;
    }
    if (!mul_ok(s->tokens, H * P, &n) || H * P > (INT32_MAX / 2) / kGdrC) return SSM_ERR_SHAPE;
    s->nc = (d.seqlen + kGdrC - 1) / kGdrC;
    // one workgroup per chunk and head; the workspace's bytes fit
    if (!mul_ok(s->heads, std::max<int64_t>(s->nc, 16), &n) || n > INT32_MAX) return SSM_ERR_SHAPE;
    if (!one && s->tokens > 0 && !gdr_fwd_grids_ok(s->heads, s->nc, d.headdim)) return SSM_ERR_SHAPE;
    return SSM_OK;
}

struct Layout {
    size_t tab, R, score, S, U, D, W, part, fwd, total;
};

Layout layout_of(const ssm_gdr_desc &d, const Sizes &s) {
    const size_t chunks = (size_t)s.heads * s.nc, P = d.headdim, N = d.dstate;
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at += align256(floats * 4);
        return here;
    };
    l.tab = take(chunks * kGdrTab * kGdrC);
    l.R = take(chunks * kGdrTiles * 256);
    l.score = take(chunks * kGdrTiles * 256);
    l.fwd = at;
    l.S = take(chunks * P * N);
    l.U = take(chunks * P * kGdrC);
    l.D = take(chunks * P * N);
    l.W = take(chunks * P * kGdrC);
    l.part = take(chunks * 2);
    l.total = at;
    return l;
}

GdrParams params_of(const ssm_gdr_desc &d, const Sizes &s, const Layout &l, void *workspace) {
    GdrParams p{};
    char *ws = static_cast<char *>(workspace);
    p.tab = reinterpret_cast<float *>(ws + l.tab);
    p.R = reinterpret_cast<float *>(ws + l.R);
    p.score = reinterpret_cast<float *>(ws + l.score);
    p.S = reinterpret_cast<float *>(ws + l.S);
    p.U = reinterpret_cast<float *>(ws + l.U);
    p.D = reinterpret_cast<float *>(ws + l.D);
    p.W = reinterpret_cast<float *>(ws + l.W);
    p.part = reinterpret_cast<float *>(ws + l.part);
    p.qs = s.qs;
    p.ks = s.ks;
    p.vs = s.vs;
    p.dts = s.dts;
    p.bs = s.bs;
    p.L = d.seqlen;
    p.nc = (int)s.nc;
    p.batch = (int)d.batch;
    p.H = d.nheads;
    p.G = d.ngroups;
    p.hpg = d.nheads / d.ngroups;
    p.P = d.headdim;
    p.dt_bias = d.dt_bias;
    p.dt_softplus = d.dt_softplus;
    p.beta_sigmoid = d.beta_sigmoid;
    p.qk_norm = d.qk_norm;
    p.scale = d.scale;
    p.qk_eps = d.qk_eps;
    return p;
}

hipError_t prep(const GdrParams &p, int N, hipStream_t st) {
    return N == 64 ? gdr_prep_launch<64>(p, st) : gdr_prep_launch<128>(p, st);
}
hipError_t fwd(const GdrParams &p, int N, bool save, hipStream_t st) {
    return N == 64 ? gdr_fwd_launch<64>(p, save, st) : gdr_fwd_launch<128>(p, save, st);
}
hipError_t bwd(const GdrParams &p, int N, hipStream_t st) {
    return N == 64 ? gdr_bwd_launch<64>(p, st) : gdr_bwd_launch<128>(p, st);
}

int64_t span(int64_t rows, int64_t stride, int64_t width) { return rows > 0 ? (rows - 1) * stride + width : 0; }

// Pointers and ranges that the calls over a sequence share. `in` gets the
// inputs' ranges, h0 the last.
int check_inputs(const ssm_gdr_desc &d, const Sizes &s, const void *q, const void *k, const void *v, const void *dt,
                 const void *beta, const float *A, const float *h0, Range *in) {
    if (A == nullptr) return SSM_ERR_NULL;
    if (s.tokens > 0 && (q == nullptr || k == nullptr || v == nullptr || dt == nullptr || beta == nullptr))
        return SSM_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(h0, 16) || !aligned(dt, 2) ||
        !aligned(beta, 2) || !aligned(A, 4) || !aligned(d.dt_bias, 4) || s.qs % 8 || s.ks % 8 || s.vs % 8)
        return SSM_ERR_ALIGN;
    const int64_t H = d.nheads, gn = (int64_t)d.ngroups * d.dstate, hp = H * d.headdim;
    in[0] = range_of(q, span(s.tokens, s.qs, gn) * 2);
    in[1] = range_of(k, span(s.tokens, s.ks, gn) * 2);
    in[2] = range_of(v, span(s.tokens, s.vs, hp) * 2);
    in[3] = range_of(dt, span(s.tokens, s.dts, H) * 2);
    in[4] = range_of(beta, span(s.tokens, s.bs, H) * 2);
    in[5] = range_of(A, H * 4);
    in[6] = range_of(d.dt_bias, H * 4);
    in[7] = range_of(h0, s.state * 4);
    return SSM_OK;
}

int run_fwd(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt, const void *beta,
            const float *A, const float *h0, void *y, float *h_last, void *workspace, size_t workspace_bytes, bool save,
            hipStream_t stream) {
    Sizes s;
    if (const int rc = check(desc, &s)) return rc;
    const ssm_gdr_desc &d = *desc;
    if (s.heads == 0) return SSM_OK;
    Range in[9];
    if (const int rc = check_inputs(d, s, q, k, v, dt, beta, A, h0, in)) return rc;
    if (s.tokens > 0 && y == nullptr) return SSM_ERR_NULL;
    if (!aligned(y, 16) || !aligned(h_last, 16)) return SSM_ERR_ALIGN;
    const Range ry = range_of(y, s.tokens * d.nheads * d.headdim * 2), rh = range_of(h_last, s.state * 4);
    const Layout l = layout_of(d, s);
    const size_t need = s.tokens == 0 ? 0 : save ? l.total : l.fwd;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
    const Range ws = range_of(workspace, (int64_t)need);
    for (int i = 0; i < 8; ++i) {
        if (overlaps(ry, in[i]) || overlaps(ws, in[i])) return SSM_ERR_ALIAS;
        if (overlaps(rh, in[i]) && !(i == 7 && h_last == h0)) return SSM_ERR_ALIAS;
    }
    if (overlaps(ry, rh) || overlaps(ws, ry) || overlaps(ws, rh)) return SSM_ERR_ALIAS;
    if (s.tokens == 0) {
        if (h_last == nullptr || h_last == h0) return SSM_OK;
        hipLaunchKernelGGL(gdr_empty_kernel, dim3(empty_blocks(s.state)), dim3(256), 0, stream, h0, h_last, s.state,
                           nullptr, nullptr, 0);
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    }
    GdrParams p = params_of(d, s, l, workspace);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.dt = static_cast<const uint16_t *>(dt);
    p.beta = static_cast<const uint16_t *>(beta);
    p.A = A;
    p.h0 = h0;
    p.y = static_cast<uint16_t *>(y);
    p.h_last = h_last;
    if (prep(p, d.dstate, stream) != hipSuccess) return SSM_ERR_HIP;
    return fwd(p, d.dstate, save, stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int run_bwd(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt, const void *beta,
            const float *A, const float *h0, const void *dy, const float *dh_last, void *dq, void *dk, void *dv,
            void *ddt, void *dbeta, float *dA, float *ddt_bias, float *dh0, void *workspace, size_t workspace_bytes,
            bool saved, hipStream_t stream) {
    Sizes s;
    if (const int rc = check(desc, &s)) return rc;
    const ssm_gdr_desc &d = *desc;
    if (s.tokens > 0 && !gdr_bwd_grids_ok(d.batch * d.ngroups, s.nc, d.nheads, d.dstate)) return SSM_ERR_SHAPE;
    const int64_t H = d.nheads, gn = (int64_t)d.ngroups * d.dstate, hp = H * d.headdim;
    Range in[11];
    if (const int rc = check_inputs(d, s, q, k, v, dt, beta, A, h0, in)) return rc;
    if (dA == nullptr || (d.dt_bias != nullptr && ddt_bias == nullptr)) return SSM_ERR_NULL;
    if (s.tokens > 0 && (dy == nullptr || dq == nullptr || dk == nullptr || dv == nullptr || ddt == nullptr ||
                         dbeta == nullptr))
        return SSM_ERR_NULL;
    if (d.dt_bias == nullptr) ddt_bias = nullptr;
    if (!aligned(dy, 16) || !aligned(dh_last, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
        !aligned(ddt, 2) || !aligned(dbeta, 2) || !aligned(dA, 4) || !aligned(ddt_bias, 4) || !aligned(dh0, 16))
        return SSM_ERR_ALIGN;
    const Layout l = layout_of(d, s);
    const size_t need = s.tokens == 0 ? 0 : l.total;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
    in[8] = range_of(dy, s.tokens * hp * 2);
    in[9] = range_of(workspace, (int64_t)need);
    in[10] = range_of(dh_last, s.state * 4);
    const Range out[] = {range_of(dq, s.tokens * gn * 2), range_of(dk, s.tokens * gn * 2), range_of(dv, s.tokens * hp * 2),
                         range_of(ddt, s.tokens * H * 2), range_of(dbeta, s.tokens * H * 2), range_of(dA, H * 4),
                         range_of(ddt_bias, H * 4), range_of(dh0, s.state * 4)};
    for (int o = 0; o < 8; ++o) {
        for (int i = 0; i < 11; ++i)
            if (overlaps(out[o], in[i]) && !(o == 7 && i == 10 && dh0 == dh_last)) return SSM_ERR_ALIAS;
        for (int j = 0; j < o; ++j)
            if (overlaps(out[o], out[j])) return SSM_ERR_ALIAS;
    }
    for (int i = 0; i < 11; ++i)
        if (i != 9 && overlaps(in[9], in[i])) return SSM_ERR_ALIAS;
    if (s.tokens == 0) {
        hipLaunchKernelGGL(gdr_empty_kernel, dim3(empty_blocks(std::max<int64_t>(s.state, H))), dim3(256), 0, stream,
                           dh_last, dh0 == dh_last ? nullptr : dh0, s.state, dA, ddt_bias, (int)H);
        return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    }
    GdrParams p = params_of(d, s, l, workspace);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.dt = static_cast<const uint16_t *>(dt);
    p.beta = static_cast<const uint16_t *>(beta);
    p.A = A;
    p.h0 = h0;
    p.dy = static_cast<const uint16_t *>(dy);
    p.dh_last = dh_last;
    p.dq = static_cast<uint16_t *>(dq);
    p.dk = static_cast<uint16_t *>(dk);
    p.dv = static_cast<uint16_t *>(dv);
    p.ddt = static_cast<uint16_t *>(ddt);
    p.dbeta = static_cast<uint16_t *>(dbeta);
    p.dA = dA;
    p.ddt_bias = ddt_bias;
    p.dh0 = dh0;
    if (!saved) {
        // the states and U of the forward; it stores no y
        if (prep(p, d.dstate, stream) != hipSuccess) return SSM_ERR_HIP;
        if (fwd(p, d.dstate, true, stream) != hipSuccess) return SSM_ERR_HIP;
    }
    return bwd(p, d.dstate, stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace

extern "C" size_t ssm_gdr_workspace_size(const ssm_gdr_desc *desc) {
    Sizes s;
    if (check(desc, &s) != SSM_OK || s.tokens == 0) return 0;
    return layout_of(*desc, s).fwd;
}

extern "C" size_t ssm_gdr_bwd_workspace_size(const ssm_gdr_desc *desc) {
    Sizes s;
    if (check(desc, &s) != SSM_OK || s.tokens == 0) return 0;
    return layout_of(*desc, s).total;
}

extern "C" int ssm_gdr_fwd(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                           const void *beta, const float *A, const float *h0, void *y, float *h_last, void *workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    return run_fwd(desc, q, k, v, dt, beta, A, h0, y, h_last, workspace, workspace_bytes, false, stream);
}

extern "C" int ssm_gdr_fwd_save(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                                const void *beta, const float *A, const float *h0, void *y, float *h_last,
                                void *workspace, size_t workspace_bytes, hipStream_t stream) {
    return run_fwd(desc, q, k, v, dt, beta, A, h0, y, h_last, workspace, workspace_bytes, true, stream);
}

extern "C" int ssm_gdr_bwd(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                           const void *beta, const float *A, const float *h0, const void *dy, const float *dh_last,
                           void *dq, void *dk, void *dv, void *ddt, void *dbeta, float *dA, float *ddt_bias, float *dh0,
                           void *workspace, size_t workspace_bytes, hipStream_t stream) {
    return run_bwd(desc, q, k, v, dt, beta, A, h0, dy, dh_last, dq, dk, dv, ddt, dbeta, dA, ddt_bias, dh0, workspace,
                   workspace_bytes, false, stream);
}

extern "C" int ssm_gdr_bwd_saved(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v, const void *dt,
                                 const void *beta, const float *A, const float *h0, const void *dy,
                                 const float *dh_last, void *dq, void *dk, void *dv, void *ddt, void *dbeta, float *dA,
                                 float *ddt_bias, float *dh0, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
    return run_bwd(desc, q, k, v, dt, beta, A, h0, dy, dh_last, dq, dk, dv, ddt, dbeta, dA, ddt_bias, dh0, workspace,
                   workspace_bytes, true, stream);
}

extern "C" int ssm_gdr_state_update(const ssm_gdr_desc *desc, const void *q, const void *k, const void *v,
                                    const void *dt, const void *beta, const float *A, const float *h, float *h_out,
                                    void *y, hipStream_t stream) {
    Sizes s;
    if (const int rc = check(desc, &s, true)) return rc;
    const ssm_gdr_desc &d = *desc;
    if (d.seqlen != 1) return SSM_ERR_SHAPE;
    if (s.heads == 0) return SSM_OK;
    if (q == nullptr || k == nullptr || v == nullptr || dt == nullptr || beta == nullptr || A == nullptr ||
        h == nullptr || h_out == nullptr || y == nullptr)
        return SSM_ERR_NULL;
    if (!aligned(q, 8) || !aligned(k, 8) || !aligned(v, 2) || !aligned(dt, 2) || !aligned(beta, 2) || !aligned(A, 4) ||
        !aligned(d.dt_bias, 4) || !aligned(h, 16) || !aligned(h_out, 16) || !aligned(y, 2) || s.qs % 4 || s.ks % 4)
        return SSM_ERR_ALIGN;
    const int64_t H = d.nheads, gn = (int64_t)d.ngroups * d.dstate, hp = H * d.headdim, B = d.batch;
    const Range in[] = {range_of(q, span(B, s.qs, gn) * 2), range_of(k, span(B, s.ks, gn) * 2),
                        range_of(v, span(B, s.vs, hp) * 2), range_of(dt, span(B, s.dts, H) * 2),
                        range_of(beta, span(B, s.bs, H) * 2), range_of(A, H * 4), range_of(d.dt_bias, H * 4),
                        range_of(h, s.state * 4)};
    const Range ro = range_of(h_out, s.state * 4), ry = range_of(y, B * hp * 2);
    for (int i = 0; i < 8; ++i) {
        if (overlaps(ry, in[i])) return SSM_ERR_ALIAS;
        if (overlaps(ro, in[i]) && !(i == 7 && h_out == h)) return SSM_ERR_ALIAS;
    }
    if (overlaps(ry, ro)) return SSM_ERR_ALIAS;
    GdrStepParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.dt = static_cast<const uint16_t *>(dt);
    p.beta = static_cast<const uint16_t *>(beta);
    p.A = A;
    p.dt_bias = d.dt_bias;
    p.h = h;
    p.h_out = h_out;
    p.y = static_cast<uint16_t *>(y);
    p.qs = s.qs;
    p.ks = s.ks;
    p.vs = s.vs;
    p.dts = s.dts;
    p.bs = s.bs;
    p.H = d.nheads;
    p.G = d.ngroups;
    p.hpg = d.nheads / d.ngroups;
    p.P = d.headdim;
    p.dt_softplus = d.dt_softplus;
    p.beta_sigmoid = d.beta_sigmoid;
    p.qk_norm = d.qk_norm;
    p.scale = d.scale;
    p.qk_eps = d.qk_eps;
    const int rows = (d.dstate == 64 ? 16 : 8) * kStepRows, bph = (d.headdim + rows - 1) / rows;
    const int64_t blocks = s.heads * bph;
    if (!grid_ok(blocks, 256)) return SSM_ERR_SHAPE;
    if (d.dstate == 64)
        hipLaunchKernelGGL((gdr_step_kernel<64>), dim3((unsigned)blocks), dim3(256), 0, stream, p, bph);
    else
        hipLaunchKernelGGL((gdr_step_kernel<128>), dim3((unsigned)blocks), dim3(256), 0, stream, p, bph);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}
