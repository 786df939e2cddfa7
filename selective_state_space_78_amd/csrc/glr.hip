// The gated linear recurrence (include/ssm_scan.h states it): per channel,
//
//   s = rate softplus(lam) sigmoid(rgate),  a = exp(-s),  m = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + m_t sigmoid(igate_t) x_t,   y_t = h_t gate_t
//
// A run of tokens maps the state before it to the state behind it by h -> P h + H
// with P the product of its decays, and maps compose. A workgroup takes one chunk of
// tokens of a tile of channels: 16 streams (8 in the backward) of TT tokens, two to a
// wave, each lane VEC channels. Every lane forms its tokens' a and b = m i x once, into registers,
// and its stream's map; the streams' maps meet in LDS, the chunk's in device memory,
// and with the state before its stream a lane runs h = a h + b over its registers.
// Inputs are read once and outputs written once, however few the channels.
//
// Chunks of one sequence are joined by looking back: a workgroup publishes its
// chunk's map, then takes the state behind the nearest chunk whose state is known and
// applies the maps of the chunks between in their order of time, the same operations
// on the same values as the one-by-one chain; results do not depend on timing.
// Workgroups take their chunk from a counter, in order of time, so that a workgroup
// waits only for ones that have started, and every wait ends. What is published is
// one word that is valid by itself (all bits set: not there yet), stored and read by
// relaxed device-scope atomics: no fence, no cache write-back.
//
// Backward: g_t = dy_t gate_t + a_{t+1} g_{t+1}, by the same maps from the end, with
// the states recomputed from the ones that the forward kept every 64 tokens. With
// w = a (a i x s / m - s h_{t-1}):  dx = g m i, digate = g m i x (1 - i), drgate =
// g w (1 - r), dlam = sigmoid(lam) / softplus(lam) sum g w. s / m goes to 0 with s,
// so an open recurrence gate (a = 1) has gradients.
//
// 1 - a is a polynomial in s up to 1/2 and a its difference from 1: decays near 1 are
// then rounded once, without the exponential's own error, which would add up over
// 1 / (1 - a) tokens, and m keeps its digits.
//
// A reset (a = 0 whatever the gate, m = 1) is carried as a decay of -0: it takes
// nothing of the state before it, were that infinite.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "ssm_scan.h"
#include "abi_util.hpp"
#include "matrix_ops.hpp"
#include "scan_kernels.hpp"

// Products and sums are fused where fmaf says so and nowhere else: every form of a kernel
// (single channels, pairs) then rounds alike
#pragma clang fp contract(off)

namespace {

using namespace ssm_detail;

constexpr int kRow = 32;                                  // lanes to a token's row of a tile
constexpr int kFwdStreams = 16, kBwdStreams = 8;          // to a workgroup, of kRow lanes each
constexpr int kBwdTokens = 8;                             // of a stream
constexpr int kKeep = kBwdStreams * kBwdTokens;           // tokens from one kept state to the next
constexpr int kBack = 8;                                  // chunks that are looked back over
// Bytes of one tensor beyond which reads and writes go past the cache: half of it (8 x 8192 x 4096
// bf16 436 -> 415 us, 131072 x 5120 1134 -> 1097 us; the training pass on 4 x 2048 x 1536, which
// stays in it, 100 -> 109 us)
constexpr int64_t kCached = (int64_t)128 << 20;
constexpr int64_t kMaxStride = (1 << 24) - 1;             // lane offsets stay in 32 bits
constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.92596299e-8f;   // and its next digits

struct GlrParams {
    const void *x, *rg, *ig, *gate, *dy;
    const float *lam, *h0, *dh_last;
    const uint8_t *reset;
    void *y, *dx, *drg, *dig, *dgate;
    float *h_last, *dh0, *dlam;
    float *keep, *part;          // (batch, kept, dim) states; (batch, chunks, dim) sums for dlam
    unsigned long long *map;     // (chunk, batch, dim) P and H of a chunk
    uint32_t *state;             // (chunk, batch, dim) the state behind a chunk
    uint32_t *ticket;            // NULL with one chunk
    int64_t L, dim, xs, rs, is, gs;
    int batch, chunks, tiles, kept, past;
    float rate;
};

template <typename T, int VEC> struct Raw;
template <> struct Raw<uint16_t, 1> { typedef uint16_t type; };
template <> struct Raw<uint16_t, 2> { typedef uint32_t type; };
template <> struct Raw<float, 1> { typedef float type; };
template <> struct Raw<float, 2> { typedef float2 type; };

template <int VEC> __device__ __forceinline__ void widen(uint16_t r, float (&v)[VEC]) { v[0] = ssd_bf(r); }
__device__ __forceinline__ void widen(uint32_t r, float (&v)[2]) {
    v[0] = __uint_as_float(r << 16);
    v[1] = __uint_as_float(r & 0xffff0000u);
}
template <int VEC> __device__ __forceinline__ void widen(float r, float (&v)[VEC]) { v[0] = r; }
__device__ __forceinline__ void widen(float2 r, float (&v)[2]) { v[0] = r.x; v[1] = r.y; }

__device__ __forceinline__ void narrow(const float (&v)[1], uint16_t &r) { r = ssd_to_bf(v[0]); }
__device__ __forceinline__ void narrow(const float (&v)[2], uint32_t &r) { r = ssd_pack(v[0], v[1]); }
__device__ __forceinline__ void narrow(const float (&v)[1], float &r) { r = v[0]; }
__device__ __forceinline__ void narrow(const float (&v)[2], float2 &r) { r = make_float2(v[0], v[1]); }

template <int VEC> __device__ __forceinline__ void ldf(const float *p, float (&v)[VEC]) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) v[c] = p[c];
}
template <int VEC> __device__ __forceinline__ void stf(float *p, const float (&v)[VEC]) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) p[c] = v[c];
}

__device__ __forceinline__ float soft_plus(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))) + (v != v ? v : 0.0f); }

// sigmoid; e = exp(-v) (infinite where the sigmoid is 0). With fp32 gates the exponent is taken
// to twice fp32's digits, as its rounding leaves e off by |v| half steps: a few at any v then.
// Where gates have 16 bits, which tell them to 2^-9, it is rounded (8 x 8192 x 4096 415 us, in
// full 448; fp32 takes the same time either way).
template <typename T> __device__ __forceinline__ float sigm(float v, float &e) {
    const float t = v * -kLog2e;
    e = __builtin_amdgcn_exp2f(t);
    if constexpr (sizeof(T) == 4) {
        const float low = fmaf(v, -kLog2eLow, fmaf(v, -kLog2e, -t));
        e *= fmaf(__builtin_amdgcn_fmed3f(low, -1.0f, 1.0f), 0.69314718f, 1.0f);      // infinities stay
    }
    return __builtin_amdgcn_rcpf(1.0f + e);
}
// 1 - sigmoid to its own digits
__device__ __forceinline__ float one_minus(float sig, float e) { return e > 1.0f ? 1.0f - sig : e * sig; }

// a = exp(-s) and w = 1 - a^2, 0 <= s < 1/2: 1 - a = s - s^2 / 2 + ..., fitted to 1.5e-9 of itself
__device__ __forceinline__ float decay_near(float s, float &w) {
    float q = fmaf(s, -0.0011259224265813828f, 0.008193295449018478f);
    q = fmaf(s, q, -0.04163204878568649f);
    q = fmaf(s, q, 0.16666288673877716f);
    q = fmaf(s, q, -0.49999985098838806f);
    const float em = fmaf(s, s * q, s), a = 1.0f - em;
    w = fmaf(em, a, em);
    return a;
}

// The same for s beyond (and NaN)
__device__ __forceinline__ void decay_far(float s, float &a, float &w) {
    const float ex = __builtin_amdgcn_exp2f(s * -kLog2e), em = 1.0f - ex;
    if (!(s < 0.5f)) {
        a = ex;
        w = fmaf(em, ex, em);
    }
}

// Whether every rate of the wave keeps s below 1/2 (decays that last more than 1.6 tokens
// with the gate open, as trained and initial ones do): the exponential is then left out.
template <int VEC> __device__ __forceinline__ bool all_near(const float (&k)[VEC]) {
    bool y = true;
#pragma unroll
    for (int c = 0; c < VEC; ++c) y = y && k[c] < 0.5f;
    return __all(y);
}

// Has the compiler form v at this point
__device__ __forceinline__ void here(float &v) { asm volatile("" : "+v"(v)); }

// Has the compiler take what was read as it is from here on, not what was formed of it
__device__ __forceinline__ void again(uint32_t &v) { asm volatile("" : "+v"(v)); }
template <typename R> __device__ __forceinline__ void again(R &) {}   // other types take no fewer registers

__device__ __forceinline__ bool is_reset(float P) { return __float_as_uint(P) == 0x80000000u; }

// The state behind a run from the one before it
template <bool RESET> __device__ __forceinline__ float behind(float P, float H, float h) {
    const float v = fmaf(P, h, H);
    if constexpr (RESET) return is_reset(P) ? H : v;
    else return v;
}
// The decay of two runs
template <bool RESET> __device__ __forceinline__ float both(float P, float Q) {
    if constexpr (RESET) return is_reset(P) || is_reset(Q) ? -0.0f : P * Q;
    else return P * Q;
}

constexpr uint32_t kNone = 0xffffffffu;
__device__ __forceinline__ uint32_t word_of(float v) {
    const uint32_t u = __float_as_uint(v);
    return u == kNone ? 0x7fc00000u : u;
}

template <typename W> __device__ __forceinline__ W peek(const W *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W> __device__ __forceinline__ void post(W *p, W v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Streams' maps of a chunk, and the state before it
template <int VEC, int NS> struct Shared {
    float2 map[NS][kRow * VEC];
    float2 back[kBack][64];      // a lane's own
    float start[kRow * VEC];
    float rate[kRow * VEC];
    uint32_t tile;
};

// The chunk's place: tiles in order of time (of the direction), batch rows and channels within
struct Place {
    int k, b;         // chunk in order of the direction, batch row
    int64_t c0;       // first channel
};

template <int VEC, int NS> __device__ __forceinline__ Place place(const GlrParams &p, Shared<VEC, NS> &sh) {
    uint32_t t = blockIdx.x;
    if (p.ticket) {
        if (threadIdx.x == 0) sh.tile = atomicAdd(p.ticket, 1u);
        __syncthreads();
        t = __builtin_amdgcn_readfirstlane(sh.tile);
    }
    const uint32_t per = (uint32_t)p.batch * (uint32_t)p.tiles;
    Place q;
    q.k = (int)(t / per);
    t -= (uint32_t)q.k * per;
    q.b = (int)(t / (uint32_t)p.tiles);
    q.c0 = (int64_t)(t - (uint32_t)q.b * (uint32_t)p.tiles) * (kRow * VEC);
    return q;
}

// Wave 0, a channel to a lane: the chunk's map from its streams', in order of the
// direction; the state before the chunk by looking back; the state behind it published.
// `first` is the state before the sequence (NULL: 0). Lanes past the channels go along
// with the last one.
template <bool RESET, bool REV, int VEC, int NS>
__device__ __forceinline__ void join_chunks(const GlrParams &p, Shared<VEC, NS> &sh, const Place &at, const float *first, int lane) {
    const int l = lane < kRow * VEC ? lane : kRow * VEC - 1;
    const int64_t ch = min(at.c0 + l, p.dim - 1);
    const bool write = at.c0 + lane < p.dim && lane < kRow * VEC, last = at.k == p.chunks - 1;
    float P = 1.0f, H = 0.0f, h = 0.0f;
    if (!last) {
#pragma unroll 4
        for (int s = 0; s < NS; ++s) {
            const float2 m = sh.map[REV ? NS - 1 - s : s][l];
            H = behind<RESET>(m.x, m.y, H);
            P = both<RESET>(P, m.x);
        }
    }
    const int64_t row = (int64_t)p.batch * p.dim;
    const int64_t mine = ((int64_t)at.k * p.batch + at.b) * p.dim + ch;
    if (at.k == 0) {
        if (first) h = first[(int64_t)at.b * p.dim + ch];
    } else {
        bool published = last;
        int w = 0;                            // chunks back whose maps lie in sh.back
        int64_t there = mine - row;           // not reached before chunk 0, whose state comes first
        for (;;) {
            const uint32_t s = peek(p.state + there);
            if (__all(s != kNone)) {
                h = __uint_as_float(s);
                break;
            }
            if (!published) {
                if (write) post(p.map + mine, (unsigned long long)word_of(P) | ((unsigned long long)word_of(H) << 32));
                published = true;
            }
            // chunk 0 publishes no map: its state is all that there is to wait for
            if (w < kBack && at.k - 1 - w > 0) {
                const unsigned long long m = peek(p.map + there);
                if (__all(m != ~0ull)) {
                    sh.back[w][lane] = make_float2(__uint_as_float((uint32_t)m), __uint_as_float((uint32_t)(m >> 32)));
                    there -= row;
                    ++w;
                    continue;
                }
            }
            __builtin_amdgcn_s_sleep(1);
        }
        while (--w >= 0) h = behind<RESET>(sh.back[w][lane].x, sh.back[w][lane].y, h);
    }
    if (!last && write) post(p.state + mine, word_of(behind<RESET>(P, H, h)));
    if (lane < kRow * VEC) sh.start[lane] = h;
}

// The state before a stream, in order of the direction
template <bool RESET, bool REV, int VEC, int NS>
__device__ __forceinline__ void stream_start(const Shared<VEC, NS> &sh, int wave, int half, int l, float (&h)[VEC]) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) h[c] = sh.start[l + c];
    if constexpr (!REV) {
        for (int s = 0; s < 2 * wave; ++s)
#pragma unroll
            for (int c = 0; c < VEC; ++c) h[c] = behind<RESET>(sh.map[s][l + c].x, sh.map[s][l + c].y, h[c]);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float v = behind<RESET>(sh.map[2 * wave][l + c].x, sh.map[2 * wave][l + c].y, h[c]);
            h[c] = half ? v : h[c];
        }
    } else {
        for (int s = NS - 1; s > 2 * wave + 1; --s)
#pragma unroll
            for (int c = 0; c < VEC; ++c) h[c] = behind<RESET>(sh.map[s][l + c].x, sh.map[s][l + c].y, h[c]);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float v = behind<RESET>(sh.map[2 * wave + 1][l + c].x, sh.map[2 * wave + 1][l + c].y, h[c]);
            h[c] = half ? h[c] : v;
        }
    }
}

// PAST: past the cache, which the tensor does not fit
template <bool PAST, typename R> __device__ __forceinline__ R bload(__amdgpu_buffer_rsrc_t r, uint32_t lane_off, uint32_t off) {
    constexpr int aux = PAST ? 2 : 0;
    if constexpr (sizeof(R) == 2) return __builtin_bit_cast(R, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)lane_off, (int)off, aux));
    else if constexpr (sizeof(R) == 4) return __builtin_bit_cast(R, __builtin_amdgcn_raw_buffer_load_b32(r, (int)lane_off, (int)off, aux));
    else return __builtin_bit_cast(R, __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane_off, (int)off, aux));
}
template <bool PAST, typename R> __device__ __forceinline__ void bstore(__amdgpu_buffer_rsrc_t r, uint32_t lane_off, uint32_t off, R v) {
    constexpr int aux = PAST ? 2 : 0;
    if constexpr (sizeof(R) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), r, (int)lane_off, (int)off, aux);
    else if constexpr (sizeof(R) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, (int)lane_off, (int)off, aux);
    else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(ssd_u32x2, v), r, (int)lane_off, (int)off, aux);
}

// A wave's rows of one tensor, from its first token's: a lane offset that stays, and the
// token's own, which is the same for the wave (a scalar register: no address arithmetic in
// the lanes). Offsets reach 32 rows: below 2^31 bytes. In the last, ragged chunk, rows past
// the end read the last row.
struct Rows {
    __amdgpu_buffer_rsrc_t r;
    uint32_t off, step;

    __device__ __forceinline__ Rows(const void *base, int64_t row0, int64_t stride, uint32_t half_rows, int64_t ch, int esz)
        : r(ssd_buffer(static_cast<const char *>(base) + row0 * stride * esz, 0xffffffffu)),
          off((half_rows * (uint32_t)stride + (uint32_t)ch) * (uint32_t)esz), step((uint32_t)stride * (uint32_t)esz) {}

    template <typename R, int TT>
    __device__ __forceinline__ void load(bool whole, bool past, uint32_t half_rows, int64_t left, R (&out)[TT]) const {
        if (whole && past) {
#pragma unroll
            for (int j = 0; j < TT; ++j) out[j] = bload<true, R>(r, off, j * step);
        } else if (whole) {
#pragma unroll
            for (int j = 0; j < TT; ++j) out[j] = bload<false, R>(r, off, j * step);
        } else {
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                const uint32_t back = (uint32_t)max((int64_t)0, (int64_t)half_rows + j - (left - 1));   // rows past the last
                out[j] = bload<false, R>(r, off + (j - back) * step, 0);
            }
        }
    }

    template <typename R> __device__ __forceinline__ void store(bool past, int j, R v) const {
        if (past) bstore<true, R>(r, off, j * step, v);
        else bstore<false, R>(r, off, j * step, v);
    }
};

// Forward: TT tokens to a stream. y NULL: the kept states and h_last alone. Bound by memory:
// 8 x 8192 x 4096 in bf16 405 to 417 us from run to run (figures beside one another, here and in
// other comments, are of one run), 2.15 GB at 5.15 to 5.3 TB/s; one row of 131072 x 5120 1097 us, 4.9.
// How many tokens a stream takes: fwd_tokens.
template <typename T, int VEC, int TT, bool RESET>
__global__ __launch_bounds__(kFwdStreams * kRow, 4) void glr_fwd_kernel(GlrParams p) {
    typedef typename Raw<T, VEC>::type R;
    constexpr int CT = kFwdStreams * TT;
    __shared__ Shared<VEC, kFwdStreams> sh;
    const Place at = place(p, sh);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
    const int l = (lane & (kRow - 1)) * VEC;
    const bool ok = at.c0 + l < p.dim;
    const int64_t ch = ok ? at.c0 + l : p.dim - VEC;
    const int64_t t0 = (int64_t)at.k * CT + wave * 2 * TT;            // the wave's first token
    const bool whole = (int64_t)at.k * CT + CT <= p.L;
    const int64_t left = p.L - t0;                                    // tokens from there to the end
    const int64_t row0 = (int64_t)at.b * p.L + (left > 0 ? t0 : p.L - 1);
    const int64_t lf = left > 0 ? left : 1;
    const uint32_t hr = half * TT;

    R rx[TT], rr[TT], ri[TT];
    Rows(p.rg, row0, p.rs, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, rr);
    Rows(p.ig, row0, p.is, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, ri);
    Rows(p.x, row0, p.xs, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, rx);
    if (threadIdx.x < kRow * VEC) sh.rate[threadIdx.x] = p.rate * soft_plus(p.lam[min(at.c0 + (int64_t)threadIdx.x, p.dim - 1)]);
    __syncthreads();
    float k[VEC];
    ldf<VEC>(sh.rate + l, k);
    uint32_t first = 0;      // bit j: token j starts a sequence
    if constexpr (RESET) {
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int64_t r = min((int64_t)hr + j, lf - 1);
            first |= (p.reset[row0 + r] ? 1u : 0u) << j;
        }
    }
    float a[TT][VEC], b[TT][VEC], P[VEC], H[VEC];
    const bool near = all_near<VEC>(k);
#pragma unroll
    for (int c = 0; c < VEC; ++c) { P[c] = 1.0f; H[c] = 0.0f; }
#pragma unroll
    for (int j0 = 0; j0 < TT; j0 += 2) {
        float s[2][VEC], w[2][VEC];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float r[VEC];
            widen(rr[j0 + n], r);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                float e;
                s[n][c] = k[c] * sigm<T>(r[c], e);
                a[j0 + n][c] = decay_near(s[n][c], w[n][c]);
            }
        }
        if (!near) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int c = 0; c < VEC; ++c) decay_far(s[n][c], a[j0 + n][c], w[n][c]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j = j0 + n;
            float x[VEC], i[VEC];
            widen(rx[j], x);
            widen(ri[j], i);
            const bool in = whole || (int64_t)hr + j < left;
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                float e, m = __builtin_amdgcn_sqrtf(w[n][c]);
                if constexpr (RESET) {
                    if ((first >> j) & 1) { a[j][c] = -0.0f; m = 1.0f; }
                }
                b[j][c] = m * sigm<T>(i[c], e) * x[c];
                if (!in) { a[j][c] = 1.0f; b[j][c] = 0.0f; }
                H[c] = behind<RESET>(a[j][c], b[j][c], H[c]);
                P[c] = both<RESET>(P[c], a[j][c]);
            }
        }
        // a few tokens' chains at a time: all of them at once do not fit the registers
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) sh.map[2 * wave + half][l + c] = make_float2(P[c], H[c]);
    __syncthreads();
    const int64_t bd = (int64_t)at.b * p.dim + ch;
    if (wave == 0) join_chunks<RESET, false>(p, sh, at, p.h0, lane);
    __syncthreads();
    float h[VEC];
    stream_start<RESET, false>(sh, wave, half, l, h);
    if (!ok) return;
    if (p.keep) {
        const int64_t t = t0 + hr;
        if (t % kKeep == 0 && t < p.L) stf<VEC>(p.keep + ((int64_t)at.b * p.kept + t / kKeep) * p.dim + ch, h);
    }
    if (p.y) {
        R rg[TT];
        if (p.gate) Rows(p.gate, row0, p.gs, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, rg);
        const Rows out(p.y, row0, p.dim, hr, ch, sizeof(T));
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            float v[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[c] = h[c] = behind<RESET>(a[j][c], b[j][c], h[c]);
            if (p.gate) {
                float g[VEC];
                widen(rg[j], g);
#pragma unroll
                for (int c = 0; c < VEC; ++c) v[c] *= g[c];
            }
            R o;
            narrow(v, o);
            if (whole || (int64_t)hr + j < left) out.store(p.past != 0, j, o);
        }
    } else {
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int c = 0; c < VEC; ++c) h[c] = behind<RESET>(a[j][c], b[j][c], h[c]);
    }
    // tokens past the end leave the state as it is
    if (p.h_last && at.k == p.chunks - 1 && 2 * wave + half == kFwdStreams - 1) stf<VEC>(p.h_last + bd, h);
}

// Backward: chunks of kKeep tokens from the end, the states before a lane's tokens recomputed into
// registers. 4 x 2048 x 1536 in bf16 with a gate 59 us, 230 MB at 3.9 TB/s: the arithmetic of two
// sigmoids, the decay and four gradients (80 instructions to a value, 26 us of issue at 2.4 GHz)
// stands beside the memory. Three workgroups a CU, two where pairs of fp32 and a gate would spill
// (training on 4 x 2048 x 1536 161 us, with three 177; without a gate 129 either way).
template <typename T, int VEC, bool RESET, bool GATE>
__global__ __launch_bounds__(kBwdStreams * kRow, sizeof(T) * VEC == 8 && GATE ? 2 : 3) void glr_bwd_kernel(GlrParams p) {
    typedef typename Raw<T, VEC>::type R;
    constexpr int TT = kBwdTokens, CT = kKeep;
    __shared__ Shared<VEC, kBwdStreams> sh;
    __shared__ float sum[kBwdStreams][kRow * VEC];
    const Place at = place(p, sh);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
    const int l = (lane & (kRow - 1)) * VEC;
    const int chunk = p.chunks - 1 - at.k;
    const bool ok = at.c0 + l < p.dim;
    const int64_t ch = ok ? at.c0 + l : p.dim - VEC;
    const int64_t t0 = (int64_t)chunk * CT + wave * 2 * TT;
    const bool whole = (int64_t)chunk * CT + CT <= p.L;
    const int64_t left = p.L - t0;
    const int64_t row0 = (int64_t)at.b * p.L + (left > 0 ? t0 : p.L - 1);
    const int64_t lf = left > 0 ? left : 1;
    const uint32_t hr = half * TT;

    R rx[TT], rr[TT], ri[TT], rdy[TT], rga[TT];
    Rows(p.rg, row0, p.rs, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, rr);
    Rows(p.ig, row0, p.is, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, ri);
    Rows(p.x, row0, p.xs, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, rx);
    Rows(p.dy, row0, p.dim, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, rdy);
    if constexpr (GATE) Rows(p.gate, row0, p.gs, hr, ch, sizeof(T)).load(whole, p.past != 0, hr, lf, rga);
    if (threadIdx.x < kRow * VEC) sh.rate[threadIdx.x] = p.rate * soft_plus(p.lam[min(at.c0 + (int64_t)threadIdx.x, p.dim - 1)]);
    __syncthreads();
    float k[VEC];
    ldf<VEC>(sh.rate + l, k);
    uint32_t first = 0;
    if constexpr (RESET) {
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int64_t r = min((int64_t)hr + j, lf - 1);
            first |= (p.reset[row0 + r] ? 1u : 0u) << j;
        }
    }
    // Per token, beside x, dy and the gate as they were read: a; m i; 1 - i, then g's factor of
    // digate; 1 - r; s, then w; a i x s / m. b = m i x and dy gate are formed again at each use.
    float a[TT][VEC], mi[TT][VEC], oi[TT][VEC], orr[TT][VEC], sw[TT][VEC], u[TT][VEC];
    auto input = [&](int j, float (&b)[VEC]) {
        widen(rx[j], b);
#pragma unroll
        for (int c = 0; c < VEC; ++c) b[c] *= mi[j][c];
    };
    auto incoming = [&](int j, const float (&from)[VEC], float (&g)[VEC]) {       // dy gate + from
        float dy[VEC], ga[VEC];
        widen(rdy[j], dy);
        if constexpr (GATE) widen(rga[j], ga);
#pragma unroll
        for (int c = 0; c < VEC; ++c) g[c] = GATE ? fmaf(dy[c], ga[c], from[c]) : dy[c] + from[c];
    };
    float P[VEC], H[VEC], G[VEC];
    const bool near = all_near<VEC>(k);
#pragma unroll
    for (int c = 0; c < VEC; ++c) { P[c] = 1.0f; H[c] = 0.0f; }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        float x[VEC], r[VEC], i[VEC], sr[VEC], er[VEC], w[VEC], b[VEC];
        widen(rr[j], r);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            sr[c] = sigm<T>(r[c], er[c]);
            sw[j][c] = k[c] * sr[c];
            a[j][c] = decay_near(sw[j][c], w[c]);
        }
        if (!near) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                decay_far(sw[j][c], a[j][c], w[c]);
                sw[j][c] = fminf(sw[j][c], 1e4f);          // a is 0 there
            }
        }
        const bool in = whole || (int64_t)hr + j < left;
        if (!in) {
            rx[j] = R{};
            rdy[j] = R{};
            if constexpr (GATE) rga[j] = R{};
        }
        widen(rx[j], x);
        widen(ri[j], i);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            float ei;
            const float si = sigm<T>(i[c], ei), inv = __builtin_amdgcn_rsqf(w[c]);
            const bool still = w[c] < 1.17549435e-38f;     // a gate that lets nothing in or out
            float m = still ? 0.0f : w[c] * inv;
            const float q = still ? 0.0f : sw[j][c] * inv;
            u[j][c] = a[j][c] * (si * x[c]) * q;
            if constexpr (RESET) {
                if ((first >> j) & 1) { a[j][c] = -0.0f; m = 1.0f; u[j][c] = 0.0f; sw[j][c] = 0.0f; }
            }
            mi[j][c] = m * si;
            oi[j][c] = one_minus(si, ei);
            orr[j][c] = one_minus(sr[c], er[c]);
            if (!in) { a[j][c] = 1.0f; mi[j][c] = 0.0f; }
            // formed here: put off to where it is used, each would keep two values alive instead of one
            here(oi[j][c]);
            here(orr[j][c]);
            here(u[j][c]);
            here(mi[j][c]);
        }
        input(j, b);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            H[c] = behind<RESET>(a[j][c], b[c], H[c]);
            P[c] = both<RESET>(P[c], a[j][c]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // what flows out of the stream towards the past, of what flows in at its end
#pragma unroll
    for (int j = 0; j < TT; ++j) again(rx[j]);
#pragma unroll
    for (int c = 0; c < VEC; ++c) G[c] = 0.0f;
#pragma unroll
    for (int j = TT - 1; j >= 0; --j) {
        float g[VEC];
        incoming(j, G, g);
#pragma unroll
        for (int c = 0; c < VEC; ++c) G[c] = RESET && is_reset(a[j][c]) ? 0.0f : a[j][c] * g[c];
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        again(rdy[j]);
        if constexpr (GATE) again(rga[j]);
    }
    // the states: from the kept one, in the chunk alone
#pragma unroll
    for (int c = 0; c < VEC; ++c) sh.map[2 * wave + half][l + c] = make_float2(P[c], H[c]);
    const int64_t bd = (int64_t)at.b * p.dim + ch;
    if (wave == 0 && lane < kRow) {
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            sh.start[l + c] = chunk == 0 ? (p.h0 ? p.h0[bd + c] : 0.0f) : p.keep[((int64_t)at.b * p.kept + chunk) * p.dim + ch + c];
    }
    __syncthreads();
    float h[VEC];
    stream_start<RESET, false>(sh, wave, half, l, h);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < VEC; ++c) sh.map[2 * wave + half][l + c] = make_float2(P[c], G[c]);
    __syncthreads();
    if (wave == 0) join_chunks<RESET, true>(p, sh, at, p.dh_last, lane);
    const Rows outg(GATE ? p.dgate : p.dx, row0, p.dim, hr, ch, sizeof(T));
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        float dg[VEC], b[VEC];
        input(j, b);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            // a reset reads nothing of the state before it: its s and u are 0
            const float t = RESET && is_reset(a[j][c]) ? 0.0f : a[j][c] * fmaf(-sw[j][c], h[c], u[j][c]);
            h[c] = behind<RESET>(a[j][c], b[c], h[c]);
            sw[j][c] = t;
            oi[j][c] *= b[c];
        }
        if constexpr (GATE) {
            float dy[VEC];
            widen(rdy[j], dy);
#pragma unroll
            for (int c = 0; c < VEC; ++c) dg[c] = dy[c] * h[c];
            R o;
            narrow(dg, o);
            if (ok && (whole || (int64_t)hr + j < left)) outg.store(p.past != 0, j, o);
        }
    }
    __syncthreads();
    const Rows outx(p.dx, row0, p.dim, hr, ch, sizeof(T)), outr(p.drg, row0, p.dim, hr, ch, sizeof(T)),
        outi(p.dig, row0, p.dim, hr, ch, sizeof(T));
    float c_in[VEC], dl[VEC];
    stream_start<RESET, true>(sh, wave, half, l, c_in);
#pragma unroll
    for (int c = 0; c < VEC; ++c) dl[c] = 0.0f;
#pragma unroll
    for (int j = TT - 1; j >= 0; --j) {
        const bool in = whole || (int64_t)hr + j < left;
        float vx[VEC], vr[VEC], vi[VEC], g[VEC];
        incoming(j, c_in, g);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            c_in[c] = RESET && is_reset(a[j][c]) ? 0.0f : a[j][c] * g[c];
            vx[c] = g[c] * mi[j][c];
            vi[c] = g[c] * oi[j][c];
            const float t = g[c] * sw[j][c];
            vr[c] = t * orr[j][c];
            dl[c] += in ? t : 0.0f;
        }
        R ox, orv, oiv;
        narrow(vx, ox);
        narrow(vr, orv);
        narrow(vi, oiv);
        if (ok && in) {
            outx.store(p.past != 0, j, ox);
            outr.store(p.past != 0, j, orv);
            outi.store(p.past != 0, j, oiv);
        }
    }
    if (p.dh0 && chunk == 0 && wave == 0 && half == 0 && ok) stf<VEC>(p.dh0 + bd, c_in);
#pragma unroll
    for (int c = 0; c < VEC; ++c) sum[2 * wave + half][l + c] = dl[c];
    __syncthreads();
    if (threadIdx.x < kRow * VEC && at.c0 + (int64_t)threadIdx.x < p.dim) {
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < kBwdStreams; ++s) v += sum[s][threadIdx.x];
        p.part[((int64_t)at.b * p.chunks + chunk) * p.dim + at.c0 + threadIdx.x] = v;
    }
}

// dlam from the chunks' sums, in 64 bits and a fixed order: 16 channels by 64 runs of rows
constexpr int kSumCols = 16, kSumRuns = 64;
__global__ __launch_bounds__(kSumCols * kSumRuns) void glr_sum_kernel(const float *part, int64_t n, int64_t dim,
                                                                     const float *lam, float *dlam) {
    __shared__ double s[kSumRuns][kSumCols];
    const int l = threadIdx.x % kSumCols, run = threadIdx.x / kSumCols;
    const int64_t c = (int64_t)blockIdx.x * kSumCols + l;
    double v = 0.0;
    if (c < dim)
        for (int64_t k = run; k < n; k += kSumRuns) v += part[k * dim + c];
    s[run][l] = v;
    for (int o = kSumRuns / 2; o >= 1; o >>= 1) {
        __syncthreads();
        if (run < o) s[run][l] += s[run + o][l];
    }
    if (run == 0 && c < dim) {
        // sigmoid(lam) / softplus(lam), 1 towards minus infinity
        const float x = lam[c], e = expf(-fabsf(x)), sig = (x >= 0.0f ? 1.0f : e) / (1.0f + e), sp = soft_plus(x);
        dlam[c] = (float)(s[0][l] * (sp < 1e-30f ? 1.0 : (double)sig / (double)sp));
    }
}

// Counter to 0, what chunks publish to "not there"
__global__ __launch_bounds__(256) void glr_clear_kernel(uint4 *at, int64_t n) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const uint32_t v = k < 16 ? 0u : kNone;
    if (k < n) at[k] = uint4{v, v, v, v};
}

// One token: bound by its launch and its trips to memory, one for softplus(lam) and the first row and one for
// each further row of a lane, which waits for the stores of the one before (256 x 5120 in bf16 with a
// gate, two rows to a lane, 7.4 us for 24 MB; after one another in a graph 6.1, fp32 7.0 to 7.2).
// A lane takes VEC channels of `rows_per` batch rows, so that softplus(lam) is formed once for them.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrParams p, const float *h, float *h_out, int rows_per) {
    typedef typename Raw<T, VEC>::type R;
    const int64_t ch = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
    if (ch >= p.dim) return;
    float k[VEC];
    ldf<VEC>(p.lam + ch, k);
#pragma unroll
    for (int c = 0; c < VEC; ++c) k[c] = p.rate * soft_plus(k[c]);
    const int64_t b1 = min((int64_t)(blockIdx.y + 1) * rows_per, (int64_t)p.batch);
    for (int64_t b = (int64_t)blockIdx.y * rows_per; b < b1; ++b) {
        const T *px = static_cast<const T *>(p.x), *pr = static_cast<const T *>(p.rg), *pi = static_cast<const T *>(p.ig);
        float x[VEC], r[VEC], i[VEC], g[VEC], s0[VEC], v[VEC];
        widen(*reinterpret_cast<const R *>(px + b * p.xs + ch), x);
        widen(*reinterpret_cast<const R *>(pr + b * p.rs + ch), r);
        widen(*reinterpret_cast<const R *>(pi + b * p.is + ch), i);
        if (p.gate) widen(*reinterpret_cast<const R *>(static_cast<const T *>(p.gate) + b * p.gs + ch), g);
        ldf<VEC>(h + b * p.dim + ch, s0);
        const bool first = p.reset && p.reset[b];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            float e, w;
            const float s = k[c] * sigm<T>(r[c], e);
            float a = decay_near(s, w);
            decay_far(s, a, w);
            const float ix = sigm<T>(i[c], e) * x[c];
            s0[c] = first ? ix : fmaf(a, s0[c], __builtin_amdgcn_sqrtf(w) * ix);
            v[c] = p.gate ? s0[c] * g[c] : s0[c];
        }
        stf<VEC>(h_out + b * p.dim + ch, s0);
        R o;
        narrow(v, o);
        *reinterpret_cast<R *>(static_cast<T *>(p.y) + b * p.dim + ch) = o;
    }
}

// ---------------------------------------------------------------------------
// Launching

// Tokens to a stream of the forward: 16 halve what joining chunks costs (8 x 8192 x 4096 bf16
// 415 us, with 8 461), where they fit the registers of four waves a SIMD: not in fp32 (8 x 8192 x 4096
// 974 us, with 8 741), nor with resets (4 x 4096 x 2048 bf16 149 us, with 8 81; without resets 62)
int fwd_tokens(int dtype, bool reset) { return (dtype == SSM_BF16 && !reset ? 16 : 8) * kFwdStreams; }
int64_t chunks_of(int64_t L, int tokens) { return (L + tokens - 1) / tokens; }

// A workspace: the backward's kept states and sums, then what chunks publish: the
// counter, the maps, the states
struct Layout {
    size_t part, sync, map, state, total;
};

Layout layout(const ssm_glr_desc &d, bool bwd, int64_t chunks) {
    const size_t bd = (size_t)d.batch * (size_t)d.dim;
    Layout l{};
    if (bwd) {
        l.part = align256((size_t)chunks_of(d.seqlen, kKeep) * bd * 4);
        l.sync = 2 * l.part;
    }
    l.map = l.sync + 256;
    l.state = l.map + align256((size_t)chunks * bd * 8);
    l.total = chunks > 1 ? l.state + align256((size_t)chunks * bd * 4) : l.sync;
    return l;
}

// Bytes that any call with this descriptor needs
size_t bytes_of(const ssm_glr_desc &d, bool bwd) {
    return layout(d, bwd, chunks_of(d.seqlen, bwd ? kKeep : fwd_tokens(d.dtype, true))).total;
}

int64_t tiles_of(int64_t dim, int vec) { return (dim + kRow * vec - 1) / (kRow * vec); }

size_t esize(int t) { return t == SSM_BF16 ? 2 : 4; }

int check(const ssm_glr_desc *desc) {
    if (desc == nullptr) return SSM_ERR_NULL;
    const ssm_glr_desc &d = *desc;
    if (d.batch < 0 || d.seqlen < 0 || d.dim < 1 || d.dim > kMaxStride) return SSM_ERR_SHAPE;
    int64_t n = 0, m;
    const int64_t strides[] = {d.x_stride, d.rgate_stride, d.igate_stride, d.gate_stride};
    for (int64_t s : strides) {
        if (s < 0 || (s != 0 && s < d.dim) || s > kMaxStride) return SSM_ERR_SHAPE;
        n = std::max(n, s);
    }
    if (!mul_ok(d.batch, d.seqlen, &m) || !mul_ok(m, std::max(n, d.dim), &n) || n > INT64_MAX / 64) return SSM_ERR_SHAPE;
    if (d.batch > INT32_MAX || d.seqlen > ((int64_t)1 << 37)) return SSM_ERR_SHAPE;
    if (d.dtype != SSM_F32 && d.dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (!(d.rate >= 0.0f) || d.rate > 3e38f) return SSM_ERR_UNSUPPORTED;
    // every launch below 2^32 work items, with the narrowest pieces
    if (!mul_ok(d.batch, tiles_of(d.dim, 1), &n) || !mul_ok(n, std::max<int64_t>(1, chunks_of(d.seqlen, kKeep)), &n) ||
        !grid_ok(n, kFwdStreams * kRow))
        return SSM_ERR_SHAPE;
    int64_t cells;
    if (!mul_ok(d.batch * d.dim, chunks_of(d.seqlen, kKeep), &cells) || !grid_ok(cells / 256 + 64, 256)) return SSM_ERR_SHAPE;
    return SSM_OK;
}

int64_t stride_of(int64_t s, int64_t dim) { return s ? s : dim; }
int64_t span(int64_t rows, int64_t stride, int64_t width) { return rows > 0 ? (rows - 1) * stride + width : 0; }

GlrParams params_of(const ssm_glr_desc &d) {
    GlrParams p{};
    p.L = d.seqlen;
    p.dim = d.dim;
    p.batch = (int)d.batch;
    p.xs = stride_of(d.x_stride, d.dim);
    p.rs = stride_of(d.rgate_stride, d.dim);
    p.is = stride_of(d.igate_stride, d.dim);
    p.gs = stride_of(d.gate_stride, d.dim);
    p.rate = d.rate;
    p.kept = (int)chunks_of(d.seqlen, kKeep);
    p.past = d.batch * d.seqlen * d.dim * (int64_t)esize(d.dtype) > kCached;
    return p;
}

// Whether lanes move two channels at a time
bool pairs(const ssm_glr_desc &d, const GlrParams &p, const void *const *ptr, int n) {
    if (d.dim % 2 || p.xs % 2 || p.rs % 2 || p.is % 2 || (p.gate && p.gs % 2)) return false;
    for (int k = 0; k < n; ++k)
        if (ptr[k] && !aligned(ptr[k], 2 * esize(d.dtype))) return false;
    return true;
}

hipError_t set_sync(const ssm_glr_desc &d, GlrParams &p, char *ws, bool bwd, int64_t chunks, hipStream_t st) {
    p.chunks = (int)chunks;
    p.ticket = nullptr;
    if (chunks <= 1) return hipSuccess;
    const Layout l = layout(d, bwd, chunks);
    p.ticket = reinterpret_cast<uint32_t *>(ws + l.sync);
    p.map = reinterpret_cast<unsigned long long *>(ws + l.map);
    p.state = reinterpret_cast<uint32_t *>(ws + l.state);
    const int64_t n = (int64_t)(l.total - l.sync) / 16;
    hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st,
                       reinterpret_cast<uint4 *>(ws + l.sync), n);
    return hipGetLastError();
}

template <typename T, int VEC, int TT> void launch_fwd(const GlrParams &p, unsigned blocks, hipStream_t st) {
    if (p.reset) hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, 8, true>), dim3(blocks), dim3(kFwdStreams * kRow), 0, st, p);
    else hipLaunchKernelGGL((glr_fwd_kernel<T, VEC, TT, false>), dim3(blocks), dim3(kFwdStreams * kRow), 0, st, p);
}

int run_fwd(const ssm_glr_desc &d, GlrParams &p, bool two, char *ws, bool save, hipStream_t st) {
    const int64_t chunks = chunks_of(d.seqlen, fwd_tokens(d.dtype, p.reset != nullptr));
    if (set_sync(d, p, ws, save, chunks, st) != hipSuccess) return SSM_ERR_HIP;
    p.tiles = (int)tiles_of(d.dim, two ? 2 : 1);
    const unsigned blocks = (unsigned)((int64_t)p.tiles * p.batch * p.chunks);
    if (d.dtype == SSM_BF16) two ? launch_fwd<uint16_t, 2, 16>(p, blocks, st) : launch_fwd<uint16_t, 1, 16>(p, blocks, st);
    else two ? launch_fwd<float, 2, 8>(p, blocks, st) : launch_fwd<float, 1, 8>(p, blocks, st);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

template <typename T, int VEC> void launch_bwd(const GlrParams &p, unsigned blocks, hipStream_t st) {
#define GLR_CASE(RESET, GATE) \
    hipLaunchKernelGGL((glr_bwd_kernel<T, VEC, RESET, GATE>), dim3(blocks), dim3(kBwdStreams * kRow), 0, st, p)
    if (p.reset) {
        if (p.gate) GLR_CASE(true, true);
        else GLR_CASE(true, false);
    } else {
        if (p.gate) GLR_CASE(false, true);
        else GLR_CASE(false, false);
    }
#undef GLR_CASE
}

// No tokens: the last state is the first, and the gradients of what no token reads are 0
__global__ __launch_bounds__(256) void glr_pass_kernel(const float *from, float *to, int64_t n, float *zero, int64_t m) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (to && k < n) to[k] = from ? from[k] : 0.0f;
    if (zero && k < m) zero[k] = 0.0f;
}

int pass_state(const float *from, float *to, int64_t n, float *zero, int64_t m, hipStream_t st) {
    const int64_t blocks = (std::max(to ? n : 0, zero ? m : 0) + 255) / 256;
    if (blocks == 0) return SSM_OK;
    if (!grid_ok(blocks, 256)) return SSM_ERR_SHAPE;
    hipLaunchKernelGGL(glr_pass_kernel, dim3((unsigned)blocks), dim3(256), 0, st, from, to, n, zero, m);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

struct Inputs {
    const void *x, *rg, *ig, *gate;
    const float *lam, *h0;
    const uint8_t *reset;
};

// Ranges of what both directions read
int inputs_of(const ssm_glr_desc &d, const GlrParams &p, const Inputs &in, Range *r) {
    const int64_t rows = d.batch * d.seqlen, e = (int64_t)esize(d.dtype);
    r[0] = range_of(in.x, span(rows, p.xs, d.dim) * e);
    r[1] = range_of(in.rg, span(rows, p.rs, d.dim) * e);
    r[2] = range_of(in.ig, span(rows, p.is, d.dim) * e);
    r[3] = range_of(in.gate, span(rows, p.gs, d.dim) * e);
    r[4] = range_of(in.lam, d.dim * 4);
    r[5] = range_of(in.reset, rows);
    r[6] = range_of(in.h0, d.batch * d.dim * 4);
    return 7;
}

bool same(Range a, Range b) { return a.lo == b.lo && a.hi == b.hi; }

int forward(const ssm_glr_desc *desc, const Inputs &in, void *y, float *h_last, void *workspace, size_t bytes, bool save,
            hipStream_t st) {
    if (const int rc = check(desc)) return rc;
    const ssm_glr_desc &d = *desc;
    const int64_t bd = d.batch * d.dim, rows = d.batch * d.seqlen;
    if (!aligned(in.h0, 4) || !aligned(h_last, 4)) return SSM_ERR_ALIGN;
    const Range rl = range_of(h_last, bd * 4), r0 = range_of(in.h0, bd * 4);
    if (overlaps(rl, r0) && !same(rl, r0)) return SSM_ERR_ALIAS;
    if (bd == 0) return SSM_OK;
    if (d.seqlen == 0) return h_last == in.h0 ? SSM_OK : pass_state(in.h0, h_last, bd, nullptr, 0, st);
    if (!in.x || !in.rg || !in.ig || !in.lam || !y) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype);
    if (!aligned(in.x, e) || !aligned(in.rg, e) || !aligned(in.ig, e) || !aligned(in.gate, e) || !aligned(in.lam, 4) ||
        !aligned(y, e))
        return SSM_ERR_ALIGN;
    const size_t need = bytes_of(d, save);
    if (need && (!workspace || bytes < need)) return SSM_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
    GlrParams p = params_of(d);
    Range r[8];
    const int n = inputs_of(d, p, in, r);
    const Range ry = range_of(y, rows * d.dim * (int64_t)e), ws = range_of(workspace, (int64_t)need);
    for (int k = 0; k < n; ++k)
        if (overlaps(ry, r[k]) || overlaps(ws, r[k]) || (k < 6 && overlaps(rl, r[k]))) return SSM_ERR_ALIAS;
    if (overlaps(ry, rl) || overlaps(ws, ry) || overlaps(ws, rl)) return SSM_ERR_ALIAS;
    p.x = in.x; p.rg = in.rg; p.ig = in.ig; p.gate = in.gate; p.lam = in.lam; p.h0 = in.h0; p.reset = in.reset;
    p.y = y;
    p.h_last = h_last;
    char *w = static_cast<char *>(workspace);
    if (save) p.keep = reinterpret_cast<float *>(w);
    const void *ptr[] = {in.x, in.rg, in.ig, in.gate, y};
    return run_fwd(d, p, pairs(d, p, ptr, 5), w, save, st);
}

int backward(const ssm_glr_desc *desc, const Inputs &in, const void *dy, const float *dh_last, void *dx, void *drg, void *dig,
             void *dgate, float *dlam, float *dh0, void *workspace, size_t bytes, bool saved, hipStream_t st) {
    if (const int rc = check(desc)) return rc;
    const ssm_glr_desc &d = *desc;
    const int64_t bd = d.batch * d.dim, rows = d.batch * d.seqlen;
    if (!dlam) return SSM_ERR_NULL;
    if (!aligned(dlam, 4) || !aligned(dh0, 4) || !aligned(dh_last, 4) || !aligned(in.h0, 4)) return SSM_ERR_ALIGN;
    const Range rdl = range_of(dlam, d.dim * 4), rd0 = range_of(dh0, bd * 4), rdh = range_of(dh_last, bd * 4);
    if ((overlaps(rd0, rdh) && !same(rd0, rdh)) || overlaps(rdl, rd0) || overlaps(rdl, rdh)) return SSM_ERR_ALIAS;
    if (rows == 0) return pass_state(dh_last, dh0 == dh_last ? nullptr : dh0, bd, dlam, d.dim, st);
    if (!in.x || !in.rg || !in.ig || !in.lam || !dy || !dx || !drg || !dig || (in.gate && !dgate)) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype);
    const void *typed[] = {in.x, in.rg, in.ig, in.gate, dy, dx, drg, dig, in.gate ? dgate : nullptr};
    for (const void *q : typed)
        if (!aligned(q, e)) return SSM_ERR_ALIGN;
    if (!aligned(in.lam, 4)) return SSM_ERR_ALIGN;
    const size_t need = bytes_of(d, true);
    if (!workspace || bytes < need) return SSM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
    GlrParams p = params_of(d);
    Range r[10];
    int n = inputs_of(d, p, in, r);
    const int64_t full = rows * d.dim * (int64_t)e;
    r[n++] = range_of(dy, full);
    r[n++] = rdh;
    const Range ws = range_of(workspace, (int64_t)need);
    const Range out[] = {range_of(dx, full), range_of(drg, full), range_of(dig, full), range_of(dgate, in.gate ? full : 0), rdl, rd0};
    for (int k = 0; k < 6; ++k) {
        for (int j = 0; j < n; ++j)
            if (overlaps(out[k], r[j]) && !(k == 5 && j == n - 1)) return SSM_ERR_ALIAS;
        for (int j = 0; j < k; ++j)
            if (overlaps(out[k], out[j])) return SSM_ERR_ALIAS;
        if (overlaps(out[k], ws)) return SSM_ERR_ALIAS;
    }
    for (int j = 0; j < n; ++j)
        if (overlaps(ws, r[j])) return SSM_ERR_ALIAS;
    p.x = in.x; p.rg = in.rg; p.ig = in.ig; p.gate = in.gate; p.lam = in.lam; p.h0 = in.h0; p.reset = in.reset;
    char *w = static_cast<char *>(workspace);
    p.keep = reinterpret_cast<float *>(w);
    const bool two = pairs(d, p, typed, 9);
    if (!saved) {
        const int rc = run_fwd(d, p, two, w, true, st);
        if (rc != SSM_OK) return rc;
    }
    p.dy = dy; p.dh_last = dh_last; p.dx = dx; p.drg = drg; p.dig = dig; p.dgate = dgate; p.dh0 = dh0;
    const int64_t chunks = chunks_of(d.seqlen, kKeep);
    p.part = reinterpret_cast<float *>(w + layout(d, true, chunks).part);
    if (set_sync(d, p, w, true, chunks, st) != hipSuccess) return SSM_ERR_HIP;
    p.tiles = (int)tiles_of(d.dim, two ? 2 : 1);
    const unsigned blocks = (unsigned)((int64_t)p.tiles * p.batch * p.chunks);
    if (d.dtype == SSM_BF16) two ? launch_bwd<uint16_t, 2>(p, blocks, st) : launch_bwd<uint16_t, 1>(p, blocks, st);
    else two ? launch_bwd<float, 2>(p, blocks, st) : launch_bwd<float, 1>(p, blocks, st);
    if (hipGetLastError() != hipSuccess) return SSM_ERR_HIP;
    hipLaunchKernelGGL(glr_sum_kernel, dim3((unsigned)((d.dim + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumRuns), 0, st,
                       p.part, (int64_t)p.batch * p.chunks, d.dim, in.lam, dlam);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace

extern "C" size_t ssm_glr_workspace_size(const ssm_glr_desc *desc) {
    if (check(desc) != SSM_OK || desc->batch == 0 || desc->seqlen == 0) return 0;
    return bytes_of(*desc, false);
}

extern "C" size_t ssm_glr_bwd_workspace_size(const ssm_glr_desc *desc) {
    if (check(desc) != SSM_OK || desc->batch == 0 || desc->seqlen == 0) return 0;
    return bytes_of(*desc, true);
}

extern "C" int ssm_glr_fwd(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                           const float *h0, const void *gate, const uint8_t *reset, void *y, float *h_last, void *workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    return forward(desc, Inputs{x, rgate, igate, gate, lam, h0, reset}, y, h_last, workspace, workspace_bytes, false, stream);
}

extern "C" int ssm_glr_fwd_save(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                                const float *h0, const void *gate, const uint8_t *reset, void *y, float *h_last,
                                void *workspace, size_t workspace_bytes, hipStream_t stream) {
    return forward(desc, Inputs{x, rgate, igate, gate, lam, h0, reset}, y, h_last, workspace, workspace_bytes, true, stream);
}

extern "C" int ssm_glr_bwd(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                           const float *h0, const void *gate, const uint8_t *reset, const void *dy, const float *dh_last,
                           void *dx, void *drgate, void *digate, void *dgate, float *dlam, float *dh0, void *workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    return backward(desc, Inputs{x, rgate, igate, gate, lam, h0, reset}, dy, dh_last, dx, drgate, digate, dgate, dlam, dh0,
                    workspace, workspace_bytes, false, stream);
}

extern "C" int ssm_glr_bwd_saved(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate, const float *lam,
                                 const float *h0, const void *gate, const uint8_t *reset, const void *dy,
                                 const float *dh_last, void *dx, void *drgate, void *digate, void *dgate, float *dlam,
                                 float *dh0, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    return backward(desc, Inputs{x, rgate, igate, gate, lam, h0, reset}, dy, dh_last, dx, drgate, digate, dgate, dlam, dh0,
                    workspace, workspace_bytes, true, stream);
}

extern "C" int ssm_glr_state_update(const ssm_glr_desc *desc, const void *x, const void *rgate, const void *igate,
                                    const float *lam, const void *gate, const uint8_t *reset, const float *h, float *h_out,
                                    void *y, hipStream_t stream) {
    if (const int rc = check(desc)) return rc;
    const ssm_glr_desc &d = *desc;
    if (d.seqlen != 1) return SSM_ERR_SHAPE;
    if (d.batch == 0) return SSM_OK;
    if (!x || !rgate || !igate || !lam || !h || !h_out || !y) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype);
    const void *typed[] = {x, rgate, igate, gate, y};
    for (const void *q : typed)
        if (!aligned(q, e)) return SSM_ERR_ALIGN;
    if (!aligned(lam, 4) || !aligned(h, 4) || !aligned(h_out, 4)) return SSM_ERR_ALIGN;
    GlrParams p = params_of(d);
    Range r[8];
    const int n = inputs_of(d, p, Inputs{x, rgate, igate, gate, lam, h, reset}, r);
    const Range ry = range_of(y, d.batch * d.dim * (int64_t)e), ro = range_of(h_out, d.batch * d.dim * 4);
    for (int k = 0; k < n; ++k)
        if (overlaps(ry, r[k]) || (overlaps(ro, r[k]) && !(k == 6 && same(ro, r[k])))) return SSM_ERR_ALIAS;
    if (overlaps(ry, ro)) return SSM_ERR_ALIAS;
    p.x = x; p.rg = rgate; p.ig = igate; p.gate = gate; p.lam = lam; p.reset = reset;
    p.y = y;
    const bool two = pairs(d, p, typed, 5);
    const int64_t bx = (d.dim + 256 * (two ? 2 : 1) - 1) / (256 * (two ? 2 : 1));
    // rows to a lane: as many as leave four workgroups to a CU
    int rows_per = 1;
    while (rows_per < 16 && bx * ((d.batch + 2 * rows_per - 1) / (2 * rows_per)) >= 1024) rows_per *= 2;
    while ((d.batch + rows_per - 1) / rows_per > 65535) rows_per *= 2;
    const dim3 grid((unsigned)bx, (unsigned)((d.batch + rows_per - 1) / rows_per));
    if (d.dtype == SSM_BF16) {
        if (two) hipLaunchKernelGGL((glr_step_kernel<uint16_t, 2>), grid, dim3(256), 0, stream, p, h, h_out, rows_per);
        else hipLaunchKernelGGL((glr_step_kernel<uint16_t, 1>), grid, dim3(256), 0, stream, p, h, h_out, rows_per);
    } else {
        if (two) hipLaunchKernelGGL((glr_step_kernel<float, 2>), grid, dim3(256), 0, stream, p, h, h_out, rows_per);
        else hipLaunchKernelGGL((glr_step_kernel<float, 1>), grid, dim3(256), 0, stream, p, h, h_out, rows_per);
    }
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}
