// The projections' C entries, their launches and the first pass of the backward
// (include/ssm_scan.h states them; proj_kernels.hpp has the products).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "ssm_scan.h"
#include "abi_util.hpp"
#include "proj_kernels.hpp"
#include "scan_kernels.hpp"

namespace {

using namespace ssm_detail;

constexpr int64_t kMaxWidth = ((int64_t)1 << 22) - 1;   // of a row: a tile's lane offsets stay in 32 bits
constexpr int kCus = 256, kMostSplits = 64;
// Bytes of a 16-bit output beyond which it goes past the cache. A product and one that reads its
// output: 65536 x 1024 -> 2048 (268 MB) 530 -> 507 us, 16384 x 2048 -> 4096 (134 MB) 455 -> 449;
// 16384 x 2560 -> 2560 (84 MB) 416 -> 421, 16384 x 1024 -> 2560 (84 MB) 166 -> 175. fp32 gains nowhere
// (16384 x 768 -> 2048, 134 MB, 737 -> 743).
constexpr int64_t kCached = (int64_t)100 << 20;

size_t esize(int t) { return t == SSM_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// dpre = dy act'(pre), and its sums over rows. A workgroup takes 64 lanes' columns
// of a slab of rows, four rows at a time; the slabs' sums are added by proj_sum_kernel.

// Beyond 100 the slopes are at their ends, 0 and 1: there z's powers, which the vanishing
// 1 - s or s stands before, are taken at 100 and do not overflow.
template <typename T, int ACT> __device__ __forceinline__ float act_grad(float z) {
    float e;
    const float s = proj_gate<T, ACT>(z, e);
    const float r = e > 1.0f ? 1.0f - s : e * s;          // 1 - s to its own digits
    z = __builtin_amdgcn_fmed3f(z, -100.0f, 100.0f);      // NaN is in s
    if constexpr (ACT == kActSilu) return s * fmaf(z, r, 1.0f);
    if constexpr (ACT == kActGelu) return fmaf(z * s * r, kGeluK * fmaf(3.0f * 0.044715f * z, z, 1.0f), s);
    return s * r;
}

struct DpreParams {
    const void *dy, *pre;
    void *dpre;                 // NULL: not written
    float *part;                // (slab, columns), or NULL
    int64_t rows, cols, per;    // rows of a slab
    int act;
};

template <typename T, typename D, int VEC> __global__ __launch_bounds__(256) void proj_dpre_kernel(DpreParams a) {
    __shared__ float sum[4][64 * VEC];
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = ((int64_t)blockIdx.x * 64 + l) * VEC;
    const int64_t r1 = min((int64_t)(blockIdx.y + 1) * a.per, a.rows);
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = 0.0f;
    if (c < a.cols) {
#pragma unroll 4
        for (int64_t r = (int64_t)blockIdx.y * a.per + w; r < r1; r += 4) {
            const int64_t at = r * a.cols + c;
            float d[VEC], z[VEC];
            if constexpr (VEC == 4) proj_load4<D>(a.dy, at, d);
            else d[0] = proj_load1<D>(a.dy, at);
            if (a.act != kActNone) {
                if constexpr (VEC == 4) proj_load4<T>(a.pre, at, z);
                else z[0] = proj_load1<T>(a.pre, at);
                proj_with(a.act, [&](auto act) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] *= act_grad<T, decltype(act)::value>(z[e]);
                });
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] += d[e];
            if (a.dpre) {
                if constexpr (VEC == 4) proj_store4<T>(a.dpre, at, d);
                else proj_store1<T>(a.dpre, at, d[0]);
            }
        }
    }
    if (a.part == nullptr) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[w][l * VEC + e] = s[e];
    __syncthreads();
    for (int k = threadIdx.x; k < 64 * VEC; k += 256) {
        const int64_t col = (int64_t)blockIdx.x * 64 * VEC + k;
        if (col < a.cols) a.part[(int64_t)blockIdx.y * a.cols + col] = (sum[0][k] + sum[1][k]) + (sum[2][k] + sum[3][k]);
    }
}

// 16 columns by 64 runs of slabs, in 64 bits
constexpr int kSumCols = 16, kSumRuns = 64;
__global__ __launch_bounds__(kSumCols * kSumRuns) void proj_sum_kernel(const float *part, int64_t slabs, int64_t cols, float *out) {
    __shared__ double s[kSumRuns][kSumCols];
    const int l = threadIdx.x % kSumCols, run = threadIdx.x / kSumCols;
    const int64_t c = (int64_t)blockIdx.x * kSumCols + l;
    double v = 0.0;
    if (c < cols)
        for (int64_t k = run; k < slabs; k += kSumRuns) v += part[k * cols + c];
    s[run][l] = v;
    for (int o = kSumRuns / 2; o >= 1; o >>= 1) {
        __syncthreads();
        if (run < o) s[run][l] += s[run + o][l];
    }
    if (run == 0 && c < cols) out[c] = (float)s[0][l];
}

__global__ __launch_bounds__(256) void proj_zero_kernel(void *p, int64_t bytes) {
    for (int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2; k < bytes; k += (int64_t)gridDim.x * 512)
        *reinterpret_cast<uint16_t *>(static_cast<char *>(p) + k) = 0;
}

// ---------------------------------------------------------------------------
// Products: which tile, how many splits

struct Tiling {
    int tile;         // 256, 128 or 64: a tile's sides
    int64_t splits, steps;      // steps of r to a split
    double us;        // as planned
};

// The time of a product of J x I outputs over R, in us, from how many workgroups a CU
// gets: it holds `hold` of a tile at once, and a step of 128 bytes of r takes it
// step[k] with k + 1 of them, next to `fixed` for a workgroup's first loads and its
// output. Splits add their sums' traffic and a launch. It puts tiles in their order; the
// times themselves come out 0.85 to 1.3 times what it says (the 12 groups below: 11.5 with 128,
// 11.3 with 64). Measured (bf16, us, tiles of 256 / 128 / 64, one split): 16384 x 2048 -> 4096 216-234 / 264 / 361; 8192 x 768 -> 1536 27.4
// / 29.0 / 32.9; 16384 x 64 -> 4096 41.6 / 45.0 / 48.7; 2048 x 2048 -> 2048 47 (2 splits
// 41) / 27.4 / 27.4; 8192 x 12 groups of 128 -> 128 25.4 / 16.1 / 14.5; 2048 x 768 -> 1536
// 24.1 / 12.8 / 10.8; 512 x 2048 -> 2048 45 / 21.9 / 12.2 (2 splits 33 / 21.0 / 16.9);
// dweight of 8192 x 768 -> 1536 175 / 92 / 63, in 8 splits 44 / 43 / -, as planned (128, 6 splits) 35;
// fp32 8192 x 768 -> 1536 187 / 146 / 144.
Tiling plan_for(int64_t I, int64_t J, int64_t R, int64_t groups, int dtype) {
    struct Kind { int side, hold; double step[4], fixed; };
    static const Kind narrow[] = {{256, 1, {1.75}, 8.0}, {128, 2, {0.75, 1.0}, 4.0}, {64, 4, {0.3, 0.42, 0.58, 0.74}, 2.3}};
    static const Kind wide[] = {{256, 1, {7.3}, 12.0}, {128, 2, {2.2, 4.1}, 5.0}, {64, 4, {0.9, 1.2, 1.6, 2.1}, 2.5}};
    const int64_t every = ceil_div(R, dtype == SSM_BF16 ? 64 : 32);
    Tiling best{128, 1, every, 1e300};
    for (const Kind &k : dtype == SSM_BF16 ? narrow : wide) {
        const int64_t tiles = ceil_div(I, k.side) * ceil_div(J, k.side) * groups;
        for (int64_t s = 1; s <= kMostSplits && s <= every; s = s < 4 ? s + 1 : s + s / 2) {
            if (s > 1 && tiles * s > 4 * kCus * k.hold) break;
            // an even number of steps to a split: they go in pairs
            const int64_t each = s == 1 ? every : 2 * ceil_div(every, 2 * s), splits = ceil_div(every, each);
            const double steps = (double)each;
            const int64_t on = ceil_div(tiles * splits, kCus), rest = on % k.hold;
            double t = (double)(on / k.hold) * (steps * k.step[k.hold - 1] + k.fixed);
            if (rest) t += steps * k.step[rest - 1] + k.fixed;
            if (splits > 1) t += 3.5 + (double)I * J * groups * (8.0 * splits + 4.0) / 4.5e6;
            if (t < best.us) best = Tiling{k.side, splits, each, t};
        }
    }
    return best;
}

int64_t part_bytes(int64_t I, int64_t J, int64_t groups, const Tiling &pl) {
    return pl.splits > 1 ? (int64_t)align256((size_t)(pl.splits * groups * J * I * 4)) : 0;
}

constexpr int kFew = 16;    // rows that the forward can take without tiles, reading the weight once

// Whether it does: not where the weight's rows are so long that the waves of a workgroup are longer
// at theirs than split tiles take. By the weight's rows in KB and workgroups a CU; measured in us
// without tiles / with: one row 4096 -> 2048 4.2 / 9.9, 65536 -> 16 19.1 / 13.7; 8 rows 4096 -> 4096
// 6.0 / 10.2, 8192 -> 1024 7.8 / 9.6, 8192 -> 256 7.6 / 8.8 (taken with), 16384 -> 512 13.0 / 10.4,
// 65536 -> 256 50 / 18.5; fp32 4096 -> 4096 14.4 / 23.8, 8192 -> 512 14.7 / 12.0. The time
// without tiles is rough: fp32 4096 -> 4096 comes out as 7.9.
bool without_tiles(const ssm_proj_desc &d, const Tiling &pl) {
    if (d.rows > kFew) return false;
    const double kb = (double)d.in * (d.dtype == SSM_BF16 ? 2 : 4) / 1024;
    const int64_t each = d.rows == 1 ? 32 : 16;      // outputs that share a CU's pace
    const double turns = (double)ceil_div(d.groups * ceil_div(d.out, each), kCus);
    return (d.rows == 1 ? 2.7 + kb * 0.13 * turns : 2.3 + kb * 0.35 * turns) <= pl.us;
}

template <typename T, bool TP, bool TQ, bool FAST>
hipError_t launch_tiles(ProjParams &a, int tile, hipStream_t st) {
    a.ti = (int)ceil_div(a.I, tile);
    a.tj = (int)ceil_div(a.J, tile);
    const unsigned blocks = (unsigned)((int64_t)a.ti * a.tj * a.groups * a.splits);
    if constexpr (FAST) {
        if (tile == 256) hipLaunchKernelGGL((proj_kernel<T, TP, TQ, 256, 256, true>), dim3(blocks), dim3(512), 0, st, a);
        else if (tile == 128) hipLaunchKernelGGL((proj_kernel<T, TP, TQ, 128, 128, true>), dim3(blocks), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((proj_kernel<T, TP, TQ, 64, 64, true>), dim3(blocks), dim3(256), 0, st, a);
    } else {
        hipLaunchKernelGGL((proj_kernel<T, TP, TQ, 64, 64, false>), dim3(blocks), dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

template <typename T, bool TP, bool TQ> hipError_t product(ProjParams &a, Tiling pl, int dtype, hipStream_t st) {
    const int64_t each = 16 / (int64_t)sizeof(T);
    // whether pieces of 16 bytes lie on 4-byte addresses, and rows hold one at least; others go through
    // registers (8192 x 772 -> 1536 in bf16 35 us, through registers 73)
    auto dwords = [&](const void *p, int64_t ld, int64_t g, int64_t n) {
        return aligned(p, 4) && ld * (int64_t)sizeof(T) % 4 == 0 && (a.groups == 1 || g * (int64_t)sizeof(T) % 4 == 0) && n >= each;
    };
    const bool fast = dwords(a.p, a.ldp, a.gp, TP ? a.I : a.R) && dwords(a.q, a.ldq, a.gq, TQ ? a.J : a.R);
    a.splits = (int)pl.splits;
    a.steps = (int)pl.steps;
    a.past = !a.wide && a.groups * a.J * a.I * 2 > kCached;
    const hipError_t e = fast ? launch_tiles<T, TP, TQ, true>(a, pl.tile, st) : launch_tiles<T, TP, TQ, false>(a, 64, st);
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t n = (int64_t)a.groups * a.J * a.I;
    if (a.eight) hipLaunchKernelGGL((proj_join_kernel<T, 8>), dim3((unsigned)ceil_div(n / 8, 256)), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((proj_join_kernel<T, 1>), dim3((unsigned)ceil_div(n, 256)), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T> hipError_t few(ProjParams &a, hipStream_t st) {
    if (a.J <= 1) {
        hipLaunchKernelGGL((proj_one_row_kernel<T>), dim3((unsigned)ceil_div(a.groups * a.I, 8)), dim3(256), 0, st, a);
    } else {
        a.ti = (int)ceil_div(a.I, 16);
        hipLaunchKernelGGL((proj_few_rows_kernel<T, 8>), dim3((unsigned)(a.groups * (int64_t)a.ti)), dim3(512), 0, st, a);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Checks

bool type_ok(int t) { return t == SSM_F32 || t == SSM_BF16; }

int check(const ssm_proj_desc *desc) {
    if (desc == nullptr) return SSM_ERR_NULL;
    const ssm_proj_desc &d = *desc;
    if (d.rows < 0 || d.groups < 1 || d.in < 1 || d.out < 1 || d.x_stride < 0) return SSM_ERR_SHAPE;
    int64_t ki, ko, n;
    if (!mul_ok(d.groups, d.in, &ki) || !mul_ok(d.groups, d.out, &ko) || ki > kMaxWidth || ko > kMaxWidth ||
        d.x_stride > kMaxWidth || (d.x_stride != 0 && d.x_stride < ki) || d.rows > INT32_MAX)
        return SSM_ERR_SHAPE;
    if (!type_ok(d.dtype) || !type_ok(d.y_dtype)) return SSM_ERR_DTYPE;
    if (d.y_dtype != d.dtype && d.y_dtype != SSM_F32) return SSM_ERR_UNSUPPORTED;
    if (d.activation < SSM_ACT_NONE || d.activation > SSM_ACT_SIGMOID || d.reserved != 0) return SSM_ERR_UNSUPPORTED;
    // the smallest tiles of every product in the largest number of splits, and the joining pass, below 2^32 work items
    if (!mul_ok(d.rows, std::max(ki, ko), &n) || n > ((int64_t)1 << 38)) return SSM_ERR_SHAPE;
    const int64_t ti = ceil_div(d.in, 64), to = ceil_div(d.out, 64), tr = ceil_div(d.rows, 64);
    if (!grid_ok(std::max(tr * std::max(ti, to), ti * to) * d.groups, 256 * 2) ||
        !grid_ok(ceil_div(std::max(std::max(d.rows * ki, d.rows * ko), d.in * ko), 256), 256))
        return SSM_ERR_SHAPE;
    return SSM_OK;
}

int64_t span(int64_t rows, int64_t stride, int64_t width) { return rows > 0 ? (rows - 1) * stride + width : 0; }

// Rows of an odd number of 16-bit values begin between 4-byte words, from where nothing goes
// straight into LDS. Such operands are first copied, their rows padded to whole pieces, where the
// product is long enough for that: a launch and twice the bytes against its planned time again, at
// least (gradients of 7447 x 155 -> 3200 through registers 93 and 77 us, with copies 34 and 32; 8192 x 767 -> 1535
// 83 and 66, its gradients 96 and 101 and 55 each). Rows of less than a piece go through registers
// padded or not, and are left where they are: `row` is the shorter one of a product's operands
// (50000 x 5 -> 515 forward 47.6 us, with copies 52.4; both gradients of 200000 x 7 -> 2048 496, with 507).
int64_t padded(int64_t width) { return ceil_div(width, 8) * 8; }

bool worth_copies(const Tiling &pl, int64_t row, int64_t bytes) { return row >= 8 && pl.us > 6.0 + (double)bytes / 2.0e6; }

// One 16-byte piece of the copy to a lane; pieces lie row by row, group by group
__global__ __launch_bounds__(256) void proj_pad_kernel(const uint16_t *from, uint4 *to, uint32_t pieces, int width, uint32_t groups,
                                                       int64_t ld, int64_t group) {
    const uint32_t k = blockIdx.x * 256 + threadIdx.x;
    if (k >= pieces) return;
    const uint32_t across = (uint32_t)(width + 7) / 8, line = k / across, row = line / groups, g = line - row * groups;
    const int c = (int)(k - line * across) * 8, in = width - c;
    const uint16_t *at = from + row * ld + g * group + c;
    uint4 v{0, 0, 0, 0};
    if (in >= 8) {
        __builtin_memcpy(&v, at, 16);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < in ? at[e] : 0;
        v = uint4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
    }
    to[k] = v;
}

hipError_t pad(const void *from, char *to, int64_t rows, int64_t width, int64_t groups, int64_t ld, int64_t group, hipStream_t st) {
    const int64_t pieces = rows * groups * (padded(width) / 8);
    hipLaunchKernelGGL(proj_pad_kernel, dim3((unsigned)ceil_div(pieces, 256)), dim3(256), 0, st, static_cast<const uint16_t *>(from),
                       reinterpret_cast<uint4 *>(to), (uint32_t)pieces, (int)width, (uint32_t)groups, ld, group);
    return hipGetLastError();
}

int64_t copy_bytes(int64_t rows, int64_t groups, int64_t width) { return (int64_t)align256((size_t)(rows * groups * padded(width) * 2)); }

// Bytes of the operands' copies, 0 for one that is read where it is
struct Copies {
    int64_t w, x, dz;
};

bool odd_x(const ssm_proj_desc &d) { return d.dtype == SSM_BF16 && (d.in % 2 || d.x_stride % 2); }
bool odd_in(const ssm_proj_desc &d) { return d.dtype == SSM_BF16 && d.in % 2; }
bool odd_out(const ssm_proj_desc &d) { return d.dtype == SSM_BF16 && d.out % 2; }

struct ForwardPlan {
    Tiling tiles;
    bool few;
    Copies copies;
    int64_t part, total;        // bytes: splits' sums; all
};

ForwardPlan forward_plan(const ssm_proj_desc &d) {
    ForwardPlan f{plan_for(d.out, d.rows, d.in, d.groups, d.dtype), false, {0, 0, 0}, 0, 0};
    f.few = without_tiles(d, f.tiles);
    if (f.few) return f;
    f.part = part_bytes(d.out, d.rows, d.groups, f.tiles);
    Copies c{odd_in(d) ? copy_bytes(d.groups * d.out, 1, d.in) : 0, odd_x(d) ? copy_bytes(d.rows, d.groups, d.in) : 0, 0};
    if (worth_copies(f.tiles, d.in, c.w + c.x)) f.copies = c;
    f.total = f.part + f.copies.w + f.copies.x;
    return f;
}

struct BackPlan {
    Tiling dx, dw;
    int64_t slabs, per;         // of dpre's pass
    Copies copies;
    int64_t sums, part, total;  // bytes: the slabs' sums; splits' sums; all
};

BackPlan back_plan(const ssm_proj_desc &d) {
    BackPlan b;
    b.dx = plan_for(d.in, d.rows, d.out, d.groups, d.dtype);
    b.dw = plan_for(d.in, d.out, d.rows, d.groups, d.dtype);
    // enough slabs for four workgroups to a CU, of 16 rows at least
    const int64_t cols = d.groups * d.out, blocks = ceil_div(cols, 256);
    b.slabs = std::max<int64_t>(1, std::min(ceil_div(d.rows, 16), ceil_div(4 * kCus, blocks)));
    b.per = ceil_div(d.rows, b.slabs);
    b.slabs = ceil_div(d.rows, b.per);
    b.sums = (int64_t)align256((size_t)(b.slabs * cols * 4));
    b.part = std::max(part_bytes(d.in, d.rows, d.groups, b.dx), part_bytes(d.in, d.out, d.groups, b.dw));
    const Copies c{odd_in(d) ? copy_bytes(d.groups * d.out, 1, d.in) : 0, odd_x(d) ? copy_bytes(d.rows, d.groups, d.in) : 0,
                   odd_out(d) ? copy_bytes(d.rows, d.groups, d.out) : 0};
    const int64_t row = std::min(d.in, d.out);
    const bool dx = worth_copies(b.dx, row, c.w + c.dz), dw = worth_copies(b.dw, row, c.x + c.dz);
    b.copies = Copies{dx ? c.w : 0, dw ? c.x : 0, dx && dw ? c.dz : 0};
    // dz is copied for both products or for none: one that goes without leaves the other's no use
    if (c.dz && !b.copies.dz) b.copies = Copies{0, 0, 0};
    b.total = b.sums + b.part + b.copies.w + b.copies.x + b.copies.dz;
    return b;
}

template <typename T, typename D> hipError_t dpre_pass(const DpreParams &a, int64_t slabs, bool four, hipStream_t st) {
    if (four)
        hipLaunchKernelGGL((proj_dpre_kernel<T, D, 4>), dim3((unsigned)ceil_div(a.cols, 256), (unsigned)slabs), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((proj_dpre_kernel<T, D, 1>), dim3((unsigned)ceil_div(a.cols, 64), (unsigned)slabs), dim3(256), 0, st, a);
    return hipGetLastError();
}

int zero(void *p, int64_t bytes, hipStream_t st) {
    if (p == nullptr || bytes == 0) return SSM_OK;
    hipLaunchKernelGGL(proj_zero_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(bytes, 512), 1 << 20)), dim3(256), 0, st, p, bytes);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

}  // namespace

extern "C" size_t ssm_proj_workspace_size(const ssm_proj_desc *desc) {
    if (check(desc) != SSM_OK || desc->rows == 0) return 0;
    const ssm_proj_desc &d = *desc;
    return (size_t)forward_plan(d).total;
}

extern "C" size_t ssm_proj_bwd_workspace_size(const ssm_proj_desc *desc) {
    if (check(desc) != SSM_OK || desc->rows == 0) return 0;
    return (size_t)back_plan(*desc).total;
}

extern "C" int ssm_proj_fwd(const ssm_proj_desc *desc, const void *x, const void *weight, const float *bias, const void *residual,
                            void *pre, void *y, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (const int rc = check(desc)) return rc;
    const ssm_proj_desc &d = *desc;
    if (d.rows == 0) return SSM_OK;
    if (!x || !weight || !y) return SSM_ERR_NULL;
    const size_t e = esize(d.dtype), ey = esize(d.y_dtype);
    if (!aligned(x, e) || !aligned(weight, e) || !aligned(pre, e) || !aligned(bias, 4) || !aligned(residual, ey) || !aligned(y, ey))
        return SSM_ERR_ALIGN;
    const int64_t xs = d.x_stride ? d.x_stride : d.groups * d.in, n = d.rows * d.groups * d.out;
    const ForwardPlan f = forward_plan(d);
    const int64_t need = f.total;
    if (need && (!workspace || workspace_bytes < (size_t)need)) return SSM_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
    const Range in[] = {range_of(x, span(d.rows, xs, d.groups * d.in) * e), range_of(weight, d.groups * d.in * d.out * e),
                        range_of(bias, d.groups * d.out * 4), range_of(residual, n * ey)};
    const Range ry = range_of(y, n * ey), rp = range_of(pre, n * e), ws = range_of(workspace, need);
    for (int k = 0; k < 4; ++k) {
        const bool same = k == 3 && in[k].lo == ry.lo;      // a residual updated in place
        if ((overlaps(ry, in[k]) && !same) || overlaps(rp, in[k]) || overlaps(ws, in[k])) return SSM_ERR_ALIAS;
    }
    if (overlaps(ry, rp) || overlaps(ws, ry) || overlaps(ws, rp)) return SSM_ERR_ALIAS;
    ProjParams a{};
    a.p = weight;
    a.q = x;
    a.ldp = d.in;
    a.ldq = xs;
    a.gp = d.in * d.out;
    a.gq = d.in;
    a.I = d.out;
    a.J = d.rows;
    a.R = d.in;
    a.bias = bias;
    a.res = residual;
    a.pre = pre;
    a.out = y;
    a.ldo = d.groups * d.out;
    a.go = d.out;
    a.part = static_cast<float *>(workspace);
    a.groups = (int)d.groups;
    a.splits = 1;
    a.act = d.activation;
    a.wide = d.y_dtype == SSM_F32;
    a.eight = d.out % 8 == 0 && aligned(y, 16) && aligned(residual, 16) && aligned(pre, 16);
    if (f.few) return status(d.dtype == SSM_BF16 ? few<uint16_t>(a, stream) : few<float>(a, stream));
    char *copy = static_cast<char *>(workspace) + f.part;
    if (f.copies.w) {
        if (pad(weight, copy, d.groups * d.out, d.in, 1, d.in, 0, stream) != hipSuccess) return SSM_ERR_HIP;
        a.p = copy;
        a.ldp = padded(d.in);
        a.gp = d.out * a.ldp;
        copy += f.copies.w;
    }
    if (f.copies.x) {
        if (pad(x, copy, d.rows, d.in, d.groups, xs, d.in, stream) != hipSuccess) return SSM_ERR_HIP;
        a.q = copy;
        a.gq = padded(d.in);
        a.ldq = d.groups * a.gq;
    }
    return status(d.dtype == SSM_BF16 ? product<uint16_t, false, false>(a, f.tiles, d.dtype, stream)
                                      : product<float, false, false>(a, f.tiles, d.dtype, stream));
}

extern "C" int ssm_proj_bwd(const ssm_proj_desc *desc, const void *dy, const void *x, const void *weight, const void *pre,
                            void *dpre, void *dx, void *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    if (const int rc = check(desc)) return rc;
    const ssm_proj_desc &d = *desc;
    const size_t e = esize(d.dtype), ey = esize(d.y_dtype);
    const int64_t ko = d.groups * d.out, ki = d.groups * d.in, wn = d.groups * d.in * d.out;
    if (!aligned(dweight, e) || !aligned(dbias, 4)) return SSM_ERR_ALIGN;
    if (d.rows == 0) {
        const Range rw = range_of(dweight, wn * e), rb = range_of(dbias, ko * 4);
        if (overlaps(rw, rb)) return SSM_ERR_ALIAS;
        const int rc = zero(dweight, wn * (int64_t)e, stream);
        return rc != SSM_OK ? rc : zero(dbias, ko * 4, stream);
    }
    const bool act = d.activation != SSM_ACT_NONE, made = act || d.y_dtype != d.dtype;
    if (!dy || (act && !pre) || (made && !dpre) || (dx && !weight) || (dweight && !x)) return SSM_ERR_NULL;
    if (!aligned(dy, ey) || (act && !aligned(pre, e)) || (made && !aligned(dpre, e)) || !aligned(dx, e) || !aligned(x, e) ||
        !aligned(weight, e))
        return SSM_ERR_ALIGN;
    const BackPlan b = back_plan(d);
    if (b.total && (!workspace || workspace_bytes < (size_t)b.total)) return SSM_ERR_WORKSPACE;
    if (b.total && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
    const int64_t xs = d.x_stride ? d.x_stride : ki;
    const Range ws = range_of(workspace, b.total);
    const Range in[] = {range_of(dy, d.rows * ko * ey), range_of(act ? pre : nullptr, d.rows * ko * e),
                        range_of(dweight ? x : nullptr, span(d.rows, xs, ki) * e), range_of(dx ? weight : nullptr, wn * e), ws};
    const Range out[] = {range_of(made ? dpre : nullptr, d.rows * ko * e), range_of(dx, d.rows * ki * e),
                         range_of(dweight, wn * e), range_of(dbias, ko * 4)};
    for (int k = 0; k < 4; ++k) {
        for (int j = 0; j < 5; ++j)
            if (overlaps(out[k], in[j])) return SSM_ERR_ALIAS;
        for (int j = 0; j < k; ++j)
            if (overlaps(out[k], out[j])) return SSM_ERR_ALIAS;
    }
    for (int j = 0; j < 4; ++j)
        if (overlaps(ws, in[j])) return SSM_ERR_ALIAS;
    const bool bf = d.dtype == SSM_BF16;
    float *sums = static_cast<float *>(workspace), *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + b.sums);
    if (made || dbias) {
        DpreParams q{dy, act ? pre : nullptr, made ? dpre : nullptr, dbias ? sums : nullptr, d.rows, ko, b.per, d.activation};
        const bool four = ko % 4 == 0 && aligned(dy, 4 * ey) && (!act || aligned(pre, 4 * e)) && (!made || aligned(dpre, 4 * e));
        const hipError_t r = !bf                   ? dpre_pass<float, float>(q, b.slabs, four, stream)
                             : d.y_dtype == SSM_F32 ? dpre_pass<uint16_t, float>(q, b.slabs, four, stream)
                                                    : dpre_pass<uint16_t, uint16_t>(q, b.slabs, four, stream);
        if (r != hipSuccess) return SSM_ERR_HIP;
        if (dbias) {
            hipLaunchKernelGGL(proj_sum_kernel, dim3((unsigned)ceil_div(ko, kSumCols)), dim3(kSumCols * kSumRuns), 0, stream, sums,
                               b.slabs, ko, dbias);
            if (hipGetLastError() != hipSuccess) return SSM_ERR_HIP;
        }
    }
    const void *dz = made ? dpre : dy;
    ProjParams a{};
    a.groups = (int)d.groups;
    a.part = part;
    a.q = dz;
    a.ldq = ko;
    a.gq = d.out;
    a.wide = !bf;
    char *copy = reinterpret_cast<char *>(part) + b.part;
    if (b.copies.dz && (dx || dweight)) {
        if (pad(dz, copy, d.rows, d.out, d.groups, ko, d.out, stream) != hipSuccess) return SSM_ERR_HIP;
        a.q = copy;
        a.gq = padded(d.out);
        a.ldq = d.groups * a.gq;
        copy += b.copies.dz;
    }
    if (dx) {
        a.p = weight;
        a.ldp = d.in;
        a.gp = d.in * d.out;
        if (b.copies.w) {
            if (pad(weight, copy, d.groups * d.out, d.in, 1, d.in, 0, stream) != hipSuccess) return SSM_ERR_HIP;
            a.p = copy;
            a.ldp = padded(d.in);
            a.gp = d.out * a.ldp;
        }
        a.I = d.in;
        a.J = d.rows;
        a.R = d.out;
        a.out = dx;
        a.ldo = ki;
        a.go = d.in;
        a.eight = d.in % 8 == 0 && aligned(dx, 16);
        const hipError_t r = bf ? product<uint16_t, true, false>(a, b.dx, d.dtype, stream) : product<float, true, false>(a, b.dx, d.dtype, stream);
        if (r != hipSuccess) return SSM_ERR_HIP;
    }
    if (dweight) {
        a.p = x;
        a.ldp = xs;
        a.gp = d.in;
        if (b.copies.x) {
            copy += b.copies.w;
            if (pad(x, copy, d.rows, d.in, d.groups, xs, d.in, stream) != hipSuccess) return SSM_ERR_HIP;
            a.p = copy;
            a.gp = padded(d.in);
            a.ldp = d.groups * a.gp;
        }
        a.I = d.in;
        a.J = d.out;
        a.R = d.rows;
        a.out = dweight;
        a.ldo = d.in;
        a.go = d.in * d.out;
        a.eight = d.in % 8 == 0 && aligned(dweight, 16);
        const hipError_t r = bf ? product<uint16_t, true, true>(a, b.dw, d.dtype, stream) : product<float, true, true>(a, b.dw, d.dtype, stream);
        if (r != hipSuccess) return SSM_ERR_HIP;
    }
    return SSM_OK;
}
