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
// P is the instruction's first operand, so a lane holds 4 consecutive values of an output
// row: bias, activation and residual are applied there, and stores are 8 or 16 bytes.
//
// Where tiles are few the reduction is split over workgroups: each writes its fp32 sums,
// and a second kernel adds them in order and finishes as the first would.
#pragma once

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
    int act, wide, four;        // wide: the output is fp32; four: groups of 4 columns move as one
};

__device__ __forceinline__ float proj_sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

constexpr float kGeluK = 1.5957691216057308f;   // 2 sqrt(2 / pi): z (1 + tanh(u)) / 2 = z sigmoid(2 u)

__device__ __forceinline__ float proj_act(float z, int act) {
    if (act == kActSilu) return z * proj_sigmoid(z);
    if (act == kActGelu) return z * proj_sigmoid(kGeluK * fmaf(0.044715f * z * z, z, z));
    return act == kActSigmoid ? proj_sigmoid(z) : z;
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

// pre of columns i..i+3 of output row j (with FOUR all below I, moved as one), finished and stored
template <typename T, bool FOUR>
__device__ __forceinline__ void proj_finish(const ProjParams &a, int g, int64_t j, int64_t i, float (&v)[4]) {
    const int64_t at = g * a.go + j * a.ldo + i;
    if constexpr (FOUR) {
        if (a.pre) proj_store4<T>(a.pre, at, v);
        if (a.act != kActNone) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = proj_act(v[e], a.act);
        }
        if (a.res) {
            float r[4];
            if (a.wide) proj_load4<float>(a.res, at, r);
            else proj_load4<T>(a.res, at, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += r[e];
        }
        if (a.wide) proj_store4<float>(a.out, at, v);
        else proj_store4<T>(a.out, at, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i + e < a.I) {
                if (a.pre) proj_store1<T>(a.pre, at + e, v[e]);
                float y = proj_act(v[e], a.act);
                if (a.res) y += a.wide ? proj_load1<float>(a.res, at + e) : proj_load1<T>(a.res, at + e);
                if (a.wide) proj_store1<float>(a.out, at + e, y);
                else proj_store1<T>(a.out, at + e, y);
            }
        }
    }
}

// The bias of columns i..i+3
__device__ __forceinline__ void proj_bias(const ProjParams &a, int g, int64_t i, float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = a.bias && i + e < a.I ? a.bias[g * a.I + i + e] : 0.0f;
}

template <bool FOUR> __device__ __forceinline__ void proj_keep(float *o, int64_t left, const float (&v)[4]) {
    if constexpr (FOUR) {
        *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < left) o[c] = v[c];
    }
}

typedef __attribute__((address_space(3))) void proj_lds;
typedef const __attribute__((address_space(1))) void proj_glb;

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
                // rows and columns past the operand's read its last ones; their products are not stored
                if constexpr (TURNED)
                    off[n] = (uint32_t)(row * ld + min((int64_t)c * kEach, left - kEach)) * (uint32_t)sizeof(T);
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

    // Any step, values past the last r as zeros
    __device__ __forceinline__ void load_any(char *lds, int64_t s, int64_t R, int wave, int lane) const {
        const int64_t r0 = s * kStep;
        const char *b = base + (TURNED ? r0 * ld : r0) * (int64_t)sizeof(T);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int row = row_of(wave, lane, n), c = piece_of(wave, lane, n) * kEach;
            uint4 w = uint4{0, 0, 0, 0};
            if constexpr (FAST) {
                // a piece is on one side of the end whole
                if (r0 + (TURNED ? row : c) < R) w = *reinterpret_cast<const uint4 *>(b + off[n]);
            } else {
                T v[kEach];
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const bool in = TURNED ? r0 + row < R && c + e < left : r0 + c + e < R && row < left;
                    v[e] = in ? *reinterpret_cast<const T *>(b + ((int64_t)row * ld + c + e) * (int64_t)sizeof(T)) : T(0);
                }
                __builtin_memcpy(&w, v, 16);
            }
            *reinterpret_cast<uint4 *>(lds + ((wave * kLoads + n) * 64 + lane) * 16) = w;
        }
    }

    // Fragment of the 16 rows (columns) from `at`, of the step's half h: r running over
    // 4 groups of kEach values, one to each 16 lanes
    static __device__ __forceinline__ uint4 read(const char *lds, int at, int h, int lane) {
        const int s = lane & 15, g = lane >> 4;
        if constexpr (!TURNED) {
            return *reinterpret_cast<const uint4 *>(lds + (at + s) * 128 + (((4 * h + g) ^ (s & 7)) << 4));
        } else if constexpr (sizeof(T) == 2) {
            const int row = 32 * h + 8 * g + (s >> 2);
            const int c = swap(at / 8 + ((s >> 1) & 1), row);
            const uint16_t *p = reinterpret_cast<const uint16_t *>(lds + row * (B * 2) + c * 16 + (s & 1) * 8);
            return __builtin_bit_cast(uint4, ssd_ld_tr2(p, p + 4 * B));
        } else {
            const int row = 16 * h + 4 * g;
            const char *p = lds + row * (B * 4) + swap((at + s) >> 2, row) * 16 + (s & 3) * 4;
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

template <int BI, int BJ> struct ProjShape {
    static constexpr int kWI = BI == 256 ? 64 : BI / 2, kWJ = BJ / 2;     // a wave's part of the tile
    static constexpr int kWaves = (BI / kWI) * (BJ / kWJ);
};

template <typename T, bool TP, bool TQ, int BI, int BJ, bool FAST>
__global__ __launch_bounds__((ProjShape<BI, BJ>::kWaves * 64)) void proj_kernel(ProjParams a) {
    typedef ProjShape<BI, BJ> S;
    constexpr int FI = S::kWI / 16, FJ = S::kWJ / 16;
    constexpr bool FOUR = BI > 64;      // outputs that do not move in fours get the smallest tile
    typedef ProjTile<T, TP, BI, S::kWaves, FAST> TileP;
    typedef ProjTile<T, TQ, BJ, S::kWaves, FAST> TileQ;
    // two objects, so that the compiler knows a load into one from a read of the other
    __shared__ __attribute__((aligned(1024))) char one[TileP::kBytes + TileQ::kBytes];
    __shared__ __attribute__((aligned(1024))) char two[TileP::kBytes + TileQ::kBytes];
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
    const int64_t every = (a.R + TileP::kStep - 1) / TileP::kStep;
    const int64_t s0 = (int64_t)split * a.steps, s1 = min(s0 + a.steps, every);

    ssd_f32x4 acc[FJ][FI];
#pragma unroll
    for (int f = 0; f < FJ; ++f)
#pragma unroll
        for (int e = 0; e < FI; ++e) acc[f][e] = ssd_f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto load_any = [&](char *to, int64_t s) {
        tp.load_any(to, s, a.R, wave, lane);
        tq.load_any(to + TileP::kBytes, s, a.R, wave, lane);
    };
    auto load = [&](char *to, int64_t s) {
        if constexpr (FAST) {
            tp.load(to, s, wave);
            tq.load(to + TileP::kBytes, s, wave);
        } else {
            load_any(to, s);
        }
    };
    auto multiply = [&](const char *from) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 p[FI], q[FJ];
#pragma unroll
            for (int e = 0; e < FI; ++e) p[e] = TileP::read(from, wi + 16 * e, h, lane);
#pragma unroll
            for (int f = 0; f < FJ; ++f) q[f] = TileQ::read(from + TileP::kBytes, wj + 16 * f, h, lane);
#pragma unroll
            for (int f = 0; f < FJ; ++f)
#pragma unroll
                for (int e = 0; e < FI; ++e) proj_mul<T>(p[e], q[f], acc[f][e]);
            // one half's fragments in registers at a time
            if constexpr (BI == 256) __builtin_amdgcn_sched_barrier(0);
        }
    };
    // A ragged last step, and one more where the whole ones are odd in number, go first
    // and by themselves; the rest in pairs, each step loaded while the one before is multiplied.
    const int64_t s2 = max(s0, min(s1, a.R / TileP::kStep));
    const int odd = (int)((s2 - s0) & 1), alone = odd + (s1 > s2);
    for (int k = 0; k < alone; ++k) {
        load_any(two, odd && k == alone - 1 ? s0 : s1 - 1);
        __syncthreads();
        multiply(two);
        __syncthreads();
    }
    int64_t s = s0 + odd;
    if (s < s2) {
        load(one, s);
        __syncthreads();
        for (; s < s2; s += 2) {
            load(two, s + 1);
            multiply(one);
            __syncthreads();
            if (s + 2 < s2) load(one, s + 2);
            multiply(two);
            __syncthreads();
        }
    }

    const int64_t jl = j0 + wj + (lane & 15), il = i0 + wi + 4 * (lane >> 4);
    if (a.splits > 1) {
        float *sums = a.part + ((int64_t)split * a.groups + g) * a.J * a.I;
#pragma unroll
        for (int f = 0; f < FJ; ++f)
#pragma unroll
            for (int e = 0; e < FI; ++e) {
                const int64_t j = jl + 16 * f, i = il + 16 * e;
                const float v[4] = {acc[f][e][0], acc[f][e][1], acc[f][e][2], acc[f][e][3]};
                if (j < a.J && i < a.I) proj_keep<FOUR>(sums + j * a.I + i, a.I - i, v);
            }
        return;
    }
    float bias[FI][4];
#pragma unroll
    for (int e = 0; e < FI; ++e) proj_bias(a, g, il + 16 * e, bias[e]);
#pragma unroll
    for (int f = 0; f < FJ; ++f)
#pragma unroll
        for (int e = 0; e < FI; ++e) {
            const int64_t j = jl + 16 * f, i = il + 16 * e;
            float v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = acc[f][e][c] + bias[e][c];
            if (j < a.J && i < a.I) {
                if constexpr (FOUR) proj_finish<T, true>(a, g, j, i, v);
                else if (a.four) proj_finish<T, true>(a, g, j, i, v);
                else proj_finish<T, false>(a, g, j, i, v);
            }
        }
}

// Splits added in order, and finished: 4 columns of a row to a lane
template <typename T> __global__ __launch_bounds__(256) void proj_join_kernel(ProjParams a) {
    const uint32_t cols = (uint32_t)((a.I + 3) / 4);
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, row = k / cols;
    if (row >= (int64_t)a.groups * a.J) return;
    const int64_t i = (k - row * cols) * 4, g = row / a.J, j = row - g * a.J;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t step = (int64_t)a.groups * a.J * a.I;
    const float *p = a.part + row * a.I + i;
    for (int s = 0; s < a.splits; ++s, p += step) {
        if ((a.I & 3) == 0) {
            const float4 r = *reinterpret_cast<const float4 *>(p);
            v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += i + e < a.I ? p[e] : 0.0f;
        }
    }
    float b[4];
    proj_bias(a, (int)g, i, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += b[e];
    if (a.four) proj_finish<T, true>(a, (int)g, j, i, v);
    else proj_finish<T, false>(a, (int)g, j, i, v);
}

// A few rows (up to MJ): the weight is read once, 16 bytes a lane along r (one value
// where rows are not aligned), two of its rows to a wave; the products are ordinary
// fp32 ones. Bound by the weight's bytes.
template <typename T, int MJ, bool FAST> __global__ __launch_bounds__(256) void proj_few_kernel(ProjParams a) {
    constexpr int E = FAST ? 16 / (int)sizeof(T) : 1, NI = 2;
    const int lane = threadIdx.x & 63;
    const int64_t total = a.groups * a.I;
    const int64_t n0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * NI;
    if (n0 >= total) return;
    float acc[NI][MJ];
    const T *w[NI], *x[NI];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const int64_t i = min(n0 + n, total - 1), g = i / a.I;
        w[n] = static_cast<const T *>(a.p) + g * a.gp + (i - g * a.I) * a.ldp;
        x[n] = static_cast<const T *>(a.q) + g * a.gq;
#pragma unroll
        for (int m = 0; m < MJ; ++m) acc[n][m] = 0.0f;
    }
    auto get = [](const T *p, float (&v)[E]) {
        if constexpr (!FAST) {
            v[0] = proj_load1<T>(p, 0);
        } else if constexpr (sizeof(T) == 2) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p);
            const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const float4 r = *reinterpret_cast<const float4 *>(p);
            v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
        }
    };
#pragma unroll 4
    for (int64_t r = (int64_t)lane * E; r < a.R; r += 64 * E) {
        float wv[NI][E];
#pragma unroll
        for (int n = 0; n < NI; ++n) get(w[n] + r, wv[n]);
#pragma unroll
        for (int m = 0; m < MJ; ++m) {
            if (m >= a.J) break;
            float xv[E];
            get(x[0] + m * a.ldq + r, xv);
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                // the wave's two rows lie in two groups only where one ends
                if (n > 0 && x[n] != x[0]) get(x[n] + m * a.ldq + r, xv);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[n][m] = fmaf(wv[n][e], xv[e], acc[n][m]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NI; ++n)
#pragma unroll
        for (int m = 0; m < MJ; ++m)
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) acc[n][m] += __shfl_xor(acc[n][m], o);
    // one output to a lane
    float v = 0.0f;
#pragma unroll
    for (int n = 0; n < NI; ++n)
#pragma unroll
        for (int m = 0; m < MJ; ++m) v = lane == n * MJ + m ? acc[n][m] : v;
    const int n = lane / MJ, m = lane % MJ;
    if (n >= NI || m >= a.J || n0 + n >= total) return;
    const int64_t g = (n0 + n) / a.I, i = n0 + n - g * a.I;
    if (a.bias) v += a.bias[n0 + n];
    const int64_t at = g * a.go + m * a.ldo + i;
    if (a.pre) proj_store1<T>(a.pre, at, v);
    v = proj_act(v, a.act);
    if (a.res) v += a.wide ? proj_load1<float>(a.res, at) : proj_load1<T>(a.res, at);
    if (a.wide) proj_store1<float>(a.out, at, v);
    else proj_store1<T>(a.out, at, v);
}

}  // namespace ssm_detail
