// Matrix products of the projections on the matrix cores, with what follows them
// done on the accumulators.
//
//   out[j][i] = f(sum over r of P(i, r) Q(j, r))
//
// P runs along a row of the output, Q along its rows. Each operand is stored with r
// running along its rows ("kept") or with i (j) running along them ("turned"): y = x W^T
// has both kept, dx = dpre W has W turned, dW = dpre^T x both.
//
// A workgroup takes a BI x BJ tile and walks r in steps of 128 bytes (64 values of 16
// bits, 32 of 32). A step's two tiles come straight from memory into LDS, 16 bytes a lane,
// into one of two buffers while the waves multiply out of the other; the pair swaps at a
// barrier. Pieces of 16 bytes are laid out by an exclusive or with bits of their row, so
// that the reads of a fragment spread over all banks; a lane picks its piece's address in
// memory to suit, since the piece's place in LDS goes by the lane. Turned bf16 tiles are
// read with the transposing LDS reads. bf16 products use the 16x16x32 instruction, fp32 ones
// 16x16x4: full precision, four to a 16-byte piece.
//
// The sums then go through LDS, each wave's by itself, to lanes of 8 consecutive values of
// an output row: bias, activation and residual are applied there, in fp32, and rows leave
// in 16-byte stores of whole lines (16384 x 2048 -> 4096 writing pre as well 239 us; stored
// from the accumulators, 8 bytes a lane over 16 rows, 329).
//
// Bound by the matrix cores at the large sizes: 8192^3 in bf16 takes 758 us (1450 TFLOP/s),
// products running in 71 % of its cycles, the rest at the steps' barriers; fp32 4096^3 930 to 944 us
// (146 to 148 TFLOP/s). Four waves of 128 x 128 instead of eight of 128 x 64 halve what is read from
// LDS, and read a step ahead: 8192^3 took 5 % longer so, with four buffers of 64 bytes of r 4 %.
//
// Where tiles are few the reduction is split over workgroups: each writes its fp32 sums,
// and a second kernel adds them in order and finishes as the first would.
#pragma once

#include <type_traits>

#include "matrix_ops.hpp"

namespace ssm_detail {

enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSigmoid = 3 };

struct ProjParams {
    const void *p, *q;          // operands
    int64_t ldp, ldq;           // elements from row to row
    int64_t gp, gq;             // and from group to group
    int64_t I, J, R;
    const float *bias;          // (groups, I) or NULL
    const void *res;            // of the output's type, or NULL
    void *pre, *out;            // pre (of the operands' type) may be NULL
    int64_t ldo, go;            // elements from output row to row, from group to group
    float *part;                // splits > 1: (split, group, J, I)
    int ti, tj, groups, splits, steps;   // tiles; steps of r to a split
    int act, wide, eight;       // wide: the output is fp32; eight: groups of 8 columns lie on 16-byte addresses
    int past;                   // the output goes past the cache
};

constexpr float kGeluK = 1.5957691216057308f;   // 2 sqrt(2 / pi): z (1 + tanh(u)) / 2 = z sigmoid(2 u)
constexpr double kGelu1 = -1.5957691216057308 * 1.4426950408889634, kGelu3 = kGelu1 * 0.044715;   // of z and z^3, as a power of 2

// The sigmoid that the activation multiplies z by (or is): of z, for gelu of 2 sqrt(2 / pi)
// (z + 0.044715 z^3); e is the exponential of its negative argument. Rounding the argument
// leaves e off by as many half steps as the argument is large. T of 16 bits rounds more than
// that; of fp32 the argument is taken to twice its digits, and 1 + e scaled so that its
// reciprocal stays a normal number up to e's overflow: a few half steps at any z.
template <typename T, int ACT> __device__ __forceinline__ float proj_gate(float z, float &e) {
#pragma clang fp contract(off)      // what a product rounds away is added once
    constexpr float c = -1.4426950408889634f;
    if constexpr (sizeof(T) == 2) {
        e = __builtin_amdgcn_exp2f(z * (ACT == kActGelu ? fmaf(z * z, (float)kGelu3, (float)kGelu1) : c));
        return __builtin_amdgcn_rcpf(1.0f + e);
    } else {
        float t, low;
        if constexpr (ACT == kActGelu) {
            constexpr float c1 = (float)kGelu1, d1 = (float)(kGelu1 - c1), c3 = (float)kGelu3, d3 = (float)(kGelu3 - c3);
            const float q = z * z, w = z * q, wl = fmaf(z, q, -w) + z * fmaf(z, z, -q);
            const float a = z * c1, b = w * c3, bb = (t = a + b) - a;
            low = ((a - (t - bb)) + (b - bb)) + fmaf(z, d1, fmaf(z, c1, -a)) + fmaf(wl, c3, fmaf(w, d3, fmaf(w, c3, -b)));
        } else {
            t = z * c;
            low = fmaf(z, -1.92596299e-8f, fmaf(z, c, -t));
        }
        e = __builtin_amdgcn_exp2f(t) * fmaf(__builtin_amdgcn_fmed3f(low, -1.0f, 1.0f), 0.69314718f, 1.0f);   // infinities stay
        constexpr float kScale = 1.0f / 256.0f;
        return __builtin_amdgcn_rcpf(fmaf(e, kScale, kScale)) * kScale;
    }
}

// f(activation as a constant): one branch for all values that it is done for
template <typename F> __device__ __forceinline__ void proj_with(int act, F f) {
    if (act == kActSilu) f(std::integral_constant<int, kActSilu>());
    else if (act == kActGelu) f(std::integral_constant<int, kActGelu>());
    else if (act == kActSigmoid) f(std::integral_constant<int, kActSigmoid>());
}

template <typename T, int N> __device__ __forceinline__ void proj_act(float (&v)[N], int act) {
    proj_with(act, [&](auto a) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float e;
            const float s = proj_gate<T, decltype(a)::value>(v[n], e);
            v[n] = decltype(a)::value == kActSigmoid ? s : v[n] * s;
        }
    });
}

template <typename T> __device__ __forceinline__ void proj_store4(void *base, int64_t at, const float (&v)[4]) {
    T *o = static_cast<T *>(base) + at;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2 *>(o) = uint2{ssd_pack(v[0], v[1]), ssd_pack(v[2], v[3])};
    else *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
}
template <typename T> __device__ __forceinline__ void proj_store1(void *base, int64_t at, float v) {
    T *o = static_cast<T *>(base) + at;
    if constexpr (sizeof(T) == 2) *o = ssd_to_bf(v);
    else *o = v;
}
template <typename T> __device__ __forceinline__ float proj_load1(const void *base, int64_t at) {
    const T *o = static_cast<const T *>(base) + at;
    if constexpr (sizeof(T) == 2) return ssd_bf(*o);
    else return *o;
}
template <typename T> __device__ __forceinline__ void proj_load4(const void *base, int64_t at, float (&v)[4]) {
    const T *o = static_cast<const T *>(base) + at;
    if constexpr (sizeof(T) == 2) {
        const uint2 r = *reinterpret_cast<const uint2 *>(o);
        v[0] = __uint_as_float(r.x << 16);
        v[1] = __uint_as_float(r.x & 0xffff0000u);
        v[2] = __uint_as_float(r.y << 16);
        v[3] = __uint_as_float(r.y & 0xffff0000u);
    } else {
        const float4 r = *reinterpret_cast<const float4 *>(o);
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
    }
}

// PAST: past the cache
template <bool PAST> __device__ __forceinline__ void proj_put(void *to, uint4 v) {
    if constexpr (PAST) __builtin_nontemporal_store(__builtin_bit_cast(ssd_u32x4, v), static_cast<ssd_u32x4 *>(to));
    else *static_cast<uint4 *>(to) = v;
}
template <typename T, int N, bool PAST = false> __device__ __forceinline__ void proj_store(void *base, int64_t at, const float (&v)[N]) {
    T *o = static_cast<T *>(base) + at;
    if constexpr (N == 1) {
        proj_store1<T>(base, at, v[0]);
    } else if constexpr (sizeof(T) == 2) {
        proj_put<PAST>(o, uint4{ssd_pack(v[0], v[1]), ssd_pack(v[2], v[3]), ssd_pack(v[4], v[5]), ssd_pack(v[6], v[7])});
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 4)
            proj_put<PAST>(o + e, uint4{__float_as_uint(v[e]), __float_as_uint(v[e + 1]), __float_as_uint(v[e + 2]), __float_as_uint(v[e + 3])});
    }
}
template <typename T, int N> __device__ __forceinline__ void proj_load(const void *base, int64_t at, float (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = proj_load1<T>(base, at);
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            float r[4];
            proj_load4<T>(base, at + e, r);
#pragma unroll
            for (int c = 0; c < 4; ++c) v[e + c] = r[c];
        }
    }
}

// The sums of N columns from i of output row j (1, or 8 on 16-byte addresses), finished and stored
template <typename T, int N>
__device__ __forceinline__ void proj_finish(const ProjParams &a, int g, int64_t j, int64_t i, const float (&bias)[N], float (&v)[N]) {
    const int64_t at = g * a.go + j * a.ldo + i;
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] += bias[e];
    if (a.pre) proj_store<T, N, true>(a.pre, at, v);       // nothing reads it before the backward
    proj_act<T, N>(v, a.act);
    if (a.res) {
        float r[N];
        if (a.wide) proj_load<float, N>(a.res, at, r);
        else proj_load<T, N>(a.res, at, r);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] += r[e];
    }
    if (a.wide) proj_store<float, N>(a.out, at, v);
    else if (a.past) proj_store<T, N, true>(a.out, at, v);
    else proj_store<T, N>(a.out, at, v);
}

template <int N> __device__ __forceinline__ void proj_bias(const ProjParams &a, int g, int64_t i, float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = a.bias && i + e < a.I ? a.bias[g * a.I + i + e] : 0.0f;
}

typedef __attribute__((address_space(3))) void proj_lds;

// One operand's tile of B rows (kept) or columns (turned), W waves
template <typename T, bool TURNED, int B, int W, bool FAST> struct ProjTile {
    static constexpr int kEach = 16 / (int)sizeof(T);              // values to a piece
    static constexpr int kStep = 128 / (int)sizeof(T);             // values of r to a step
    static constexpr int kBytes = B * 128;
    static constexpr int kLoads = kBytes / 16 / 64 / W;            // pieces to a lane
    static constexpr int kRowPieces = TURNED ? B / kEach : 8;
    static_assert(kLoads * 16 * 64 * W == kBytes);

    const char *base;      // the tile at r = 0
    int64_t ld;            // elements
    int64_t left;          // rows (columns) from the tile's first to the operand's last
    uint32_t off[kLoads];

    // Where piece c of a row lies in it
    static __device__ __forceinline__ int swap(int c, int row) {
        if constexpr (!TURNED) return c ^ (row & 7);
        else if constexpr (sizeof(T) == 4) return c ^ (((row >> 2) & 3) << 2);
        else if constexpr (B >= 128) return c ^ (((row & 3) | (((row >> 3) & 1) << 2)) << 1);
        else return c ^ ((((row >> 1) & 1) | (((row >> 3) & 1) << 1)) << 1);
    }
    static __device__ __forceinline__ int row_of(int wave, int lane, int n) { return ((wave * kLoads + n) * 64 + lane) / kRowPieces; }
    static __device__ __forceinline__ int piece_of(int wave, int lane, int n) {
        return swap(((wave * kLoads + n) * 64 + lane) % kRowPieces, row_of(wave, lane, n));
    }

    __device__ __forceinline__ void start(const void *p, int64_t first, int64_t count, int64_t ld_, int wave, int lane) {
        ld = ld_;
        left = count - first;
        base = static_cast<const char *>(p) + (TURNED ? first : first * ld) * (int64_t)sizeof(T);
        if constexpr (FAST) {
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const int row = row_of(wave, lane, n), c = piece_of(wave, lane, n);
                // rows and columns past the operand's read its last ones, and a piece that its end cuts
                // reads on into the next row (the last row's step comes by fetch); their products are not stored
                if constexpr (TURNED)
                    off[n] = (uint32_t)(row * ld + min((int64_t)c * kEach, (left - 1) / kEach * kEach)) * (uint32_t)sizeof(T);
                else
                    off[n] = (uint32_t)(min((int64_t)row, left - 1) * ld + c * kEach) * (uint32_t)sizeof(T);
            }
        }
    }

    // Step s (values of r from s kStep), all of it inside the operand, straight into LDS
    __device__ __forceinline__ void load(char *lds, int64_t s, int wave) const {
        const char *b = base + s * kStep * (TURNED ? ld : 1) * (int64_t)sizeof(T);
        // every lane's offset is inside the operand: the buffer's own bound is all that 32 bits reach
        const __amdgpu_buffer_rsrc_t r = ssd_buffer(b, 0xffffffffu);
#pragma unroll
        for (int n = 0; n < kLoads; ++n)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (proj_lds *)(lds + (wave * kLoads + n) * 1024), 16, (int)off[n], 0, 0, 0);
    }

    // The value of 16 bytes without its first ones, which its last take the place of, zeros behind
    static __device__ __forceinline__ uint4 moved(const uint4 &v, int bytes) {
        const uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
        const int by = bytes * 8;
        const uint64_t l = by >= 64 ? hi >> (by - 64) : by == 0 ? lo : lo >> by | hi << (64 - by), h = by >= 64 ? 0 : hi >> by;
        return uint4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
    }

    // Any step, into registers: values past the last r are zeros, and so are whole pieces past the
    // operand. Pieces inside are read at whatever address they have.
    __device__ __forceinline__ void fetch(uint4 (&v)[kLoads], int64_t s, int64_t R, int wave, int lane) const {
        const int64_t r0 = s * kStep;
        const char *b = base + (TURNED ? r0 * ld : r0) * (int64_t)sizeof(T);
        if constexpr (FAST) {
            // a piece that the end cuts is read as the 16 bytes before the end, and moved down
            const int64_t end = TURNED ? left : R - r0;
            const int rest = (int)((TURNED ? left : R) % kEach), back = rest ? (kEach - rest) * (int)sizeof(T) : 0;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const int row = row_of(wave, lane, n), c = piece_of(wave, lane, n) * kEach;
                v[n] = uint4{0, 0, 0, 0};
                const bool any = c < end && (!TURNED || r0 + row < R), part = c + kEach > end;
                if (any) __builtin_memcpy(&v[n], b + off[n] - (part ? back : 0), 16);
                if (rest) v[n] = part ? moved(v[n], back) : v[n];
            }
        } else {
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const int row = row_of(wave, lane, n), c = piece_of(wave, lane, n) * kEach;
                v[n] = uint4{0, 0, 0, 0};
                const char *at = b + ((int64_t)row * ld + c) * (int64_t)sizeof(T);
                const int64_t in = TURNED ? (r0 + row < R ? left - c : 0) : (row < left ? R - r0 - c : 0);   // values of the piece
                if (in >= kEach) {
                    __builtin_memcpy(&v[n], at, 16);
                } else if (in > 0) {
                    T w[kEach];
#pragma unroll
                    for (int e = 0; e < kEach; ++e) w[e] = e < in ? reinterpret_cast<const T *>(at)[e] : T(0);
                    __builtin_memcpy(&v[n], w, 16);
                }
            }
        }
    }

    __device__ __forceinline__ void put(char *lds, const uint4 (&v)[kLoads], int wave, int lane) const {
#pragma unroll
        for (int n = 0; n < kLoads; ++n) *reinterpret_cast<uint4 *>(lds + ((wave * kLoads + n) * 64 + lane) * 16) = v[n];
    }

    // Where a lane's part of a wave's first fragment lies (the fragment's 16 rows or columns
    // begin at `at`, a multiple of all that the wave's fragments span). Fragment f and the step's
    // half h are told apart by an exclusive or and an addition of constants.
    static __device__ __forceinline__ uint32_t place(int at, int lane) {
        const int s = lane & 15, g = lane >> 4;
        if constexpr (!TURNED) {
            return (uint32_t)((at + s) * 128 + ((g ^ (s & 7)) << 4));
        } else if constexpr (sizeof(T) == 2) {
            const int row = 8 * g + (s >> 2);
            return (uint32_t)(row * (B * 2) + swap(at / 8 + ((s >> 1) & 1), row) * 16 + (s & 1) * 8);
        } else {
            const int row = 4 * g;
            return (uint32_t)(row * (B * 4) + swap((at + s) >> 2, row) * 16 + (s & 3) * 4);
        }
    }

    // Fragment f: r running over 4 groups of kEach values, one to each 16 lanes
    static __device__ __forceinline__ uint4 read(const char *lds, uint32_t place, int f, int h) {
        if constexpr (!TURNED) {
            return *reinterpret_cast<const uint4 *>(lds + (place ^ (uint32_t)(h * 64)) + f * 2048);
        } else if constexpr (sizeof(T) == 2) {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(lds + (place ^ (uint32_t)(f * 32)) + h * (64 * B));
            return __builtin_bit_cast(uint4, ssd_ld_tr2(p, p + 4 * B));
        } else {
            const char *p = lds + (place ^ (uint32_t)(f * 64)) + h * (64 * B);
            return uint4{*reinterpret_cast<const uint32_t *>(p), *reinterpret_cast<const uint32_t *>(p + B * 4),
                         *reinterpret_cast<const uint32_t *>(p + B * 8), *reinterpret_cast<const uint32_t *>(p + B * 12)};
        }
    }
};

template <typename T> __device__ __forceinline__ void proj_mul(const uint4 &p, const uint4 &q, ssd_f32x4 &c) {
    if constexpr (sizeof(T) == 2) {
        c = ssd_mfma(__builtin_bit_cast(ssd_bf16x8, p), __builtin_bit_cast(ssd_bf16x8, q), c);
    } else {
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(p.x), __uint_as_float(q.x), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(p.y), __uint_as_float(q.y), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(p.z), __uint_as_float(q.z), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(p.w), __uint_as_float(q.w), c, 0, 0, 0);
    }
}

// A barrier behind which every wave's loads into LDS are there: a wave waits for its own
// first. (The compiler waits where a wave itself reads what it loaded, which may be behind
// the barrier, where others' are read too.)
__device__ __forceinline__ void proj_arrived() {
    __builtin_amdgcn_s_waitcnt(0x0f70);      // vmcnt 0; the other counters as they are
    __syncthreads();
}

template <int BI, int BJ> struct ProjShape {
    static constexpr int kWI = BI == 256 ? 64 : BI / 2, kWJ = BJ / 2;     // a wave's part of the tile
    static constexpr int kWaves = (BI / kWI) * (BJ / kWJ);
};

template <typename T, bool TP, bool TQ, int BI, int BJ, bool FAST>
__global__ __launch_bounds__((ProjShape<BI, BJ>::kWaves * 64)) void proj_kernel(ProjParams a) {
    typedef ProjShape<BI, BJ> S;
    constexpr int FI = S::kWI / 16, FJ = S::kWJ / 16;
    typedef ProjTile<T, TP, BI, S::kWaves, FAST> TileP;
    typedef ProjTile<T, TQ, BJ, S::kWaves, FAST> TileQ;
    // two objects, so that the compiler knows a load into one from a read of the other
    __shared__ __attribute__((aligned(1024))) char one[TileP::kBytes + TileQ::kBytes];
    __shared__ __attribute__((aligned(1024))) char two[FAST ? TileP::kBytes + TileQ::kBytes : 16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;

    // Workgroups go to the 8 XCDs in turn: each gets a run of consecutive tiles, 8 rows of tiles deep
    const uint32_t all = gridDim.x, x = blockIdx.x & 7u, part = all / 8, rest = all % 8;
    uint32_t t = x * part + min(x, rest) + blockIdx.x / 8;
    const uint32_t per = (uint32_t)a.ti * (uint32_t)a.tj;
    const uint32_t lot = t / per;
    t -= lot * per;
    const int split = (int)(lot % (uint32_t)a.splits), g = (int)(lot / (uint32_t)a.splits);
    const uint32_t band = t / (8u * a.ti), depth = min(8u, (uint32_t)a.tj - band * 8u);
    t -= band * 8u * a.ti;
    const int64_t j0 = (int64_t)(band * 8u + t % depth) * BJ, i0 = (int64_t)(t / depth) * BI;

    TileP tp;
    TileQ tq;
    tp.start(static_cast<const T *>(a.p) + g * a.gp, i0, a.I, a.ldp, wave, lane);
    tq.start(static_cast<const T *>(a.q) + g * a.gq, j0, a.J, a.ldq, wave, lane);
    const int wi = wave % (BI / S::kWI) * S::kWI, wj = wave / (BI / S::kWI) * S::kWJ;
    const uint32_t place_p = TileP::place(wi, lane), place_q = TileQ::place(wj, lane);
    const int64_t every = (a.R + TileP::kStep - 1) / TileP::kStep;
    const int64_t s0 = (int64_t)split * a.steps, s1 = min(s0 + a.steps, every);

    ssd_f32x4 acc[FJ][FI];
#pragma unroll
    for (int f = 0; f < FJ; ++f)
#pragma unroll
        for (int e = 0; e < FI; ++e) acc[f][e] = ssd_f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    uint4 vp[TileP::kLoads], vq[TileQ::kLoads];
    auto fetch = [&](int64_t s) {
        tp.fetch(vp, s, a.R, wave, lane);
        tq.fetch(vq, s, a.R, wave, lane);
    };
    auto put = [&](char *to) {
        tp.put(to, vp, wave, lane);
        tq.put(to + TileP::kBytes, vq, wave, lane);
    };
    auto load = [&](char *to, int64_t s) {
        tp.load(to, s, wave);
        tq.load(to + TileP::kBytes, s, wave);
    };
    auto multiply = [&](const char *from) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 p[FI], q[FJ];
#pragma unroll
            for (int e = 0; e < FI; ++e) p[e] = TileP::read(from, place_p, e, h);
#pragma unroll
            for (int f = 0; f < FJ; ++f) q[f] = TileQ::read(from + TileP::kBytes, place_q, f, h);
#pragma unroll
            for (int f = 0; f < FJ; ++f)
#pragma unroll
                for (int e = 0; e < FI; ++e) proj_mul<T>(p[e], q[f], acc[f][e]);
            // both operands turned: one half's fragments in registers at a time, or they spill (8192^3: 0.83 ms,
            // without 1.29; with one turned or none the halves overlap and gain 2%)
            if constexpr (BI == 256 && TP && TQ && sizeof(T) == 2) __builtin_amdgcn_sched_barrier(0);
        }
    };
    if constexpr (FAST) {
        // A ragged last step, and one more where the whole ones are odd in number, go first and by
        // themselves; the rest in pairs, each step loaded while the one before is multiplied.
        const bool cut = (TP && a.I % TileP::kEach) || (TQ && a.J % TileQ::kEach);
        const int64_t s2 = max(s0, min(s1, (cut ? a.R - 1 : a.R) / TileP::kStep));
        const int odd = (int)((s2 - s0) & 1), alone = odd + (s1 > s2);
        for (int k = 0; k < alone; ++k) {
            if (odd && k == alone - 1) {
                load(two, s0);
                proj_arrived();
            } else {
                fetch(s1 - 1);
                put(two);
                __syncthreads();
            }
            multiply(two);
            __syncthreads();
        }
        int64_t s = s0 + odd;
        if (s < s2) {
            load(one, s);
            load(two, s + 1);
            proj_arrived();
            for (;; s += 2) {
                multiply(one);
                proj_arrived();
                const bool more = s + 2 < s2;
                if (more) load(one, s + 2);
                multiply(two);
                proj_arrived();
                if (!more) break;
                load(two, s + 3);
            }
        }
    } else if (s0 < s1) {
        // through registers: the next step is on its way while this one is multiplied
        fetch(s0);
        for (int64_t s = s0; s < s1; ++s) {
            put(one);
            __syncthreads();
            if (s + 1 < s1) fetch(s + 1);
            multiply(one);
            __syncthreads();
        }
    }

    // A wave's sums in parts of RJ rows: rows of WI floats, their 16-byte pieces laid out by an
    // exclusive or with the row's low bits.
    constexpr int WI = S::kWI, RJ = S::kWJ > 64 ? 64 : S::kWJ, kPart = RJ * WI * 4;
    constexpr int kIn = (TileP::kBytes + TileQ::kBytes) / kPart;      // waves that fit the first object
    static_assert(kIn >= S::kWaves || (FAST && 2 * kIn >= S::kWaves));
    char *mine = kIn >= S::kWaves || wave < kIn ? one + wave * kPart : two + (wave - kIn) * kPart;
    float *sums = a.splits > 1 ? a.part + ((int64_t)split * a.groups + g) * a.J * a.I : nullptr;
#pragma unroll
    for (int part = 0; part < S::kWJ / RJ; ++part) {
        const int64_t jp = j0 + wj + part * RJ;
#pragma unroll
        for (int f = 0; f < RJ / 16; ++f)
#pragma unroll
            for (int e = 0; e < FI; ++e) {
                const int row = 16 * f + (lane & 15), c = 4 * e + (lane >> 4);
                const ssd_f32x4 &v = acc[part * (RJ / 16) + f][e];
                *reinterpret_cast<float4 *>(mine + row * (WI * 4) + ((c ^ (row & 7)) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
            }
        __builtin_amdgcn_wave_barrier();
        if (a.eight) {
            constexpr int kAcross = WI / 8, kRows = 64 / kAcross;     // lanes to a row, rows at a time
            const int c = 2 * (lane % kAcross), r0 = lane / kAcross;
            const int64_t i = i0 + wi + 4 * c;
            float bias[8];
            proj_bias<8>(a, g, i, bias);
#pragma unroll 2
            for (int n = 0; n < RJ; n += kRows) {
                const int row = n + r0;
                const char *at = mine + row * (WI * 4);
                const float4 x = *reinterpret_cast<const float4 *>(at + ((c ^ (row & 7)) << 4));
                const float4 y = *reinterpret_cast<const float4 *>(at + (((c + 1) ^ (row & 7)) << 4));
                float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                const int64_t j = jp + row;
                if (j < a.J && i < a.I) {
                    if (sums) proj_store<float, 8>(sums, j * a.I + i, v);
                    else proj_finish<T, 8>(a, g, j, i, bias, v);
                }
            }
        } else {
            constexpr int kRows = 64 / WI;
            const int c = lane % WI;
            const int64_t i = i0 + wi + c;
            float bias[1];
            proj_bias<1>(a, g, i, bias);
#pragma unroll 2
            for (int n = 0; n < RJ; n += kRows) {
                const int row = n + lane / WI;
                float v[1] = {*reinterpret_cast<const float *>(mine + row * (WI * 4) + (((c >> 2) ^ (row & 7)) << 4) + (c & 3) * 4)};
                const int64_t j = jp + row;
                if (j < a.J && i < a.I) {
                    if (sums) sums[j * a.I + i] = v[0];
                    else proj_finish<T, 1>(a, g, j, i, bias, v);
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Splits added in order, and finished: 8 columns of a row to a lane, or one
template <typename T, int N> __global__ __launch_bounds__(256) void proj_join_kernel(ProjParams a) {
    const uint32_t cols = (uint32_t)(a.I / N);
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, row = k / cols;
    if (row >= (int64_t)a.groups * a.J) return;
    const int64_t i = (k - row * cols) * N, g = row / a.J, j = row - g * a.J;
    float v[N], bias[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = 0.0f;
    const int64_t step = (int64_t)a.groups * a.J * a.I;
    const float *p = a.part + row * a.I + i;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s, p += step) {
        float r[N];
        proj_load<float, N>(p, 0, r);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] += r[e];
    }
    proj_bias<N>(a, (int)g, i, bias);
    proj_finish<T, N>(a, (int)g, j, i, bias, v);
}

// One row: the weight is read once, 16 bytes a lane along r at any address, two of its rows to
// a wave, four pieces of each on their way at once (one after another 6.0 us); the products are
// ordinary fp32 ones. Bound by the weight's bytes (4096 -> 4096 in bf16 5.0 us, out of the cache;
// by the matrix instructions of the next kernel 7.0, 768 -> 1536 3.2 either way).
template <typename T> __global__ __launch_bounds__(256) void proj_one_row_kernel(ProjParams a) {
    constexpr int E = 16 / (int)sizeof(T), NI = 2;
    const int lane = threadIdx.x & 63;
    const int64_t total = a.groups * a.I;
    const int64_t n0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * NI;
    if (n0 >= total) return;
    float acc[NI];
    const T *w[NI], *x[NI];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const int64_t i = min(n0 + n, total - 1), g = i / a.I;
        w[n] = static_cast<const T *>(a.p) + g * a.gp + (i - g * a.I) * a.ldp;
        x[n] = static_cast<const T *>(a.q) + g * a.gq;
        acc[n] = 0.0f;
    }
    const bool apart = x[1] != x[0];        // the wave's two rows lie in two groups
    auto get = [](const T *p) {
        uint4 v;
        __builtin_memcpy(&v, p, 16);
        return v;
    };
    auto wide = [](const uint4 &r, float (&v)[E]) {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 2) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            } else {
                v[e] = __uint_as_float(u[e]);
            }
        }
    };
    const int64_t whole = a.R / E * E;
    int64_t r = (int64_t)lane * E;
    // N pieces on their way at once
    auto run = [&](auto count) {
        constexpr int N = decltype(count)::value;
        uint4 vw[N][NI], vx[N], vo[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
#pragma unroll
            for (int n = 0; n < NI; ++n) vw[k][n] = get(w[n] + r + k * 64 * E);
            vx[k] = get(x[0] + r + k * 64 * E);
            vo[k] = vx[k];
        }
        if (apart) {
#pragma unroll
            for (int k = 0; k < N; ++k) vo[k] = get(x[1] + r + k * 64 * E);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float w0[E], w1[E], x0[E], x1[E];
            wide(vw[k][0], w0);
            wide(vw[k][1], w1);
            wide(vx[k], x0);
            wide(vo[k], x1);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                acc[0] = fmaf(w0[e], x0[e], acc[0]);
                acc[1] = fmaf(w1[e], x1[e], acc[1]);
            }
        }
        r += N * 64 * E;
    };
    while (r + 3 * 64 * E < whole) run(std::integral_constant<int, 4>());
    while (r < whole) run(std::integral_constant<int, 1>());
    if (whole + lane < a.R) {
#pragma unroll
        for (int n = 0; n < NI; ++n) acc[n] = fmaf(proj_load1<T>(w[n], whole + lane), proj_load1<T>(x[n], whole + lane), acc[n]);
    }
#pragma unroll
    for (int n = 0; n < NI; ++n)
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) acc[n] += __shfl_xor(acc[n], o);
    if (lane >= NI || n0 + lane >= total) return;
    const int64_t g = (n0 + lane) / a.I, i = n0 + lane - g * a.I;
    float v[1] = {lane == 0 ? acc[0] : acc[1]}, bias[1];
    proj_bias<1>(a, (int)g, i, bias);
    proj_finish<T, 1>(a, (int)g, 0, i, bias, v);
}

// Up to 16 rows: the weight is read once, into registers, 16 bytes a lane along r at any address.
// A workgroup takes 16 of its rows, the waves share r in runs of pairs of steps (whole lines); their
// sums are added in LDS in order. Lanes read four to a row, next to one another, and hand over, by
// ds_bpermute, to the lane that the matrix instruction has the piece in. Read there directly,
// neighbouring lanes in different rows, loads pass one lane at a time: 8 rows 4096 -> 4096 in bf16
// 8.3 us, 16 rows 9.6; so 6.0 and 6.2; in tiles 10.2 to 10.5. 8 rows 768 -> 1536 2.9 us, in tiles 5.6.
// fp32 4096 -> 4096 14.3 to 14.6 us for 2 to 16 rows; read directly 16 rows took 16.8, but 2 rows 12.2.
template <typename T, int W> __global__ __launch_bounds__(W * 64) void proj_few_rows_kernel(ProjParams a) {
    constexpr int E = 16 / (int)sizeof(T), kStep = 4 * E;
    __shared__ float4 sum[W][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, s = lane & 15, q = lane >> 4;
    const uint32_t g = blockIdx.x / (uint32_t)a.ti;
    const int64_t i0 = (int64_t)(blockIdx.x - g * (uint32_t)a.ti) * 16;
    // rows past the last read it again; their products are not stored
    const T *w = static_cast<const T *>(a.p) + g * a.gp + min(i0 + s, a.I - 1) * a.ldp + q * E;
    const T *x = static_cast<const T *>(a.q) + g * a.gq + min((int64_t)s, a.J - 1) * a.ldq + q * E;
    const int64_t steps = a.R / kStep, each = (steps + 2 * W - 1) / (2 * W) * 2;
    const int64_t k0 = min(wave * each, steps), k1 = min(k0 + each, steps);
    ssd_f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    // the lane that read what this lane multiplies, and what this lane reads
    const int back = (lane & 15) * 16 + (lane >> 4) * 4;
    const T *wl = static_cast<const T *>(a.p) + g * a.gp + min(i0 + (lane >> 2), a.I - 1) * a.ldp + (lane & 3) * E;
    const T *xl = static_cast<const T *>(a.q) + g * a.gq + min((int64_t)(lane >> 2), a.J - 1) * a.ldq + (lane & 3) * E;
    auto get = [](const T *p) {
        uint4 v;
        __builtin_memcpy(&v, p, 16);
        return v;
    };
    auto turned = [&](const uint4 &v) {
        return uint4{(uint32_t)__builtin_amdgcn_ds_bpermute(back, (int)v.x), (uint32_t)__builtin_amdgcn_ds_bpermute(back, (int)v.y),
                     (uint32_t)__builtin_amdgcn_ds_bpermute(back, (int)v.z), (uint32_t)__builtin_amdgcn_ds_bpermute(back, (int)v.w)};
    };
    int64_t k = k0;
    auto run = [&](auto count) {
        constexpr int N = decltype(count)::value;
        if (k + N > k1) return;
        uint4 vw[N], vx[N];
#pragma unroll
        for (int n = 0; n < N; ++n) vw[n] = get(wl + (k + n) * kStep);
#pragma unroll
        for (int n = 0; n < N; ++n) vx[n] = get(xl + (k + n) * kStep);
#pragma unroll
        for (int n = 0; n < N; ++n) proj_mul<T>(turned(vw[n]), turned(vx[n]), acc);
        k += N;
    };
    while (k + 8 <= k1) run(std::integral_constant<int, 8>());
    run(std::integral_constant<int, 4>());
    run(std::integral_constant<int, 2>());
    run(std::integral_constant<int, 1>());
    if (wave == W - 1 && steps * kStep < a.R) {
        const int64_t at = steps * kStep, in = a.R - at - q * E;      // values of the lane's piece
        T tw[E], tx[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            tw[e] = e < in ? w[at + e] : T(0);
            tx[e] = e < in ? x[at + e] : T(0);
        }
        uint4 vw, vx;
        __builtin_memcpy(&vw, tw, 16);
        __builtin_memcpy(&vx, tx, 16);
        proj_mul<T>(vw, vx, acc);
    }
    sum[wave][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (threadIdx.x >= 256) return;
    const int i = threadIdx.x & 15, j = threadIdx.x >> 4;
    if (j >= a.J || i0 + i >= a.I) return;
    float v[1] = {0.0f}, bias[1];
#pragma unroll
    for (int n = 0; n < W; ++n) v[0] += reinterpret_cast<const float *>(&sum[n][(i >> 2) * 16 + j])[i & 3];
    proj_bias<1>(a, (int)g, i0 + i, bias);
    proj_finish<T, 1>(a, (int)g, j, i0 + i, bias, v);
}

}  // namespace ssm_detail
