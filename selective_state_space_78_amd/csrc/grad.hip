// The norm over many gradient tensors and their clipping by it (include/ssm_scan.h
// states them): one reading for the sum of squares, one reading and writing for the
// scaling; bound by memory.
//
// Tensors reach the kernels by value, up to kPer to a launch, so a call copies and
// keeps nothing. A launch cuts its tensors into pieces of kPiece elements and gives
// each workgroup a run of consecutive ones: it looks its first tensor up once and
// walks on from there. Elements move in 16 bytes from the first aligned one on;
// tensors whose source and destination are aligned differently move one by one.
//
// Squares are taken and added in 64 bits: no gradient overflows or vanishes in its
// square, and the order of sums, fixed here, matters to no digit of the fp32 norm. Each workgroup
// leaves one partial sum; those of the scaling add all of them, in the same order,
// instead of waiting for a launch that does (beyond one launch's worth a launch does, or
// every workgroup would read as much again in sums). They ask for their first elements before
// they add, and walk launches and runs backwards: what the sum read last is read first,
// out of the cache.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdlib.h>

#include <algorithm>

#include "ssm_scan.h"
#include "abi_util.hpp"
#include "matrix_ops.hpp"
#include "scan_kernels.hpp"

namespace {

using namespace ssm_detail;

constexpr int kPer = 128;            // tensors to a launch: their table is part of the kernel's arguments
constexpr int kThreads = 256;
constexpr int kWgs = 1024;           // workgroups to a launch at most: 4 to a CU
constexpr int kPiece = 8192;         // elements
// Bytes of gradients beyond which the scaling goes past the cache, which then keeps what the sum
// read last (600 MB of fp32 367 -> 345 us, 2.4 GB of bf16 1.50 -> 1.42 ms; 54 MB in the cache 28.6 us either way)
constexpr int64_t kCached = (int64_t)128 << 20;
constexpr int64_t kLongest = (int64_t)1 << 35;   // elements of a tensor: a launch's pieces stay in 32 bits

struct Table {
    const void *in[kPer];
    void *out[kPer];
    int64_t n[kPer];
    uint32_t first[kPer + 1];        // piece
    uint32_t wide[kPer / 32];        // bit: fp32
    int count;
};

__device__ __forceinline__ bool is_wide(const Table &t, int k) { return (t.wide[k >> 5] >> (k & 31)) & 1; }

// The run of pieces of this workgroup
__device__ __forceinline__ void run_of(const Table &t, uint32_t &p0, uint32_t &p1) {
    const uint32_t all = t.first[t.count];
    p0 = (uint32_t)((uint64_t)all * blockIdx.x / gridDim.x);
    p1 = (uint32_t)((uint64_t)all * (blockIdx.x + 1) / gridDim.x);
}

// The last tensor that begins at or before a piece (tensors without pieces are passed over)
__device__ __forceinline__ int find(const Table &t, uint32_t piece) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (t.first[m] <= piece) lo = m;
        else hi = m - 1;
    }
    return lo;
}

// Elements before the first 16-byte aligned one (all of them when no later one is to move so)
template <typename T> __device__ __forceinline__ int64_t head_of(const void *in, const void *out, int64_t n) {
    const uint32_t a = (uint32_t)(uintptr_t)in & 15u, b = (uint32_t)(uintptr_t)out & 15u;
    if (a != b) return n;
    return min(n, (int64_t)((16u - a) & 15u) / (int64_t)sizeof(T));
}

template <typename T> __device__ __forceinline__ float value(const T *p) {
    if constexpr (sizeof(T) == 2) return ssd_bf(*p);
    else return *p;
}

template <typename T> __device__ __forceinline__ void put(T *p, float v) {
    if constexpr (sizeof(T) == 2) *p = ssd_to_bf(v);
    else *p = v;
}

template <typename T> struct Words {
    static constexpr int kEach = 16 / sizeof(T), kIter = kPiece / (kEach * kThreads);
};

template <typename T> __device__ __forceinline__ void words(const uint4 &r, float (&v)[16 / sizeof(T)]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        } else {
            v[e] = __uint_as_float(w[e]);
        }
    }
}

// One piece: elements [e0, e1) of a tensor, e0 a multiple of kPiece. Their 16-byte
// words are those of the elements from `head` on; what is left over on both sides
// goes one by one. SCALE writes in * factor() to out (asked for once the reads are under
// way), else squares are added to sum.
template <typename T, bool SCALE, typename F>
__device__ __forceinline__ void piece(const T *in, T *out, int64_t n, int64_t e0, F factor, bool past, double &sum) {
    typedef Words<T> W;
    const int64_t e1 = min(e0 + kPiece, n);
    const int64_t head = head_of<T>(in, SCALE ? out : in, n);
    // first and behind the last whole word in [e0, e1)
    int64_t w0 = e0 <= head ? head : head + (e0 - head + W::kEach - 1) / W::kEach * W::kEach;
    w0 = min(w0, e1);
    const int nw = (int)((e1 - w0) / W::kEach);
    const int64_t w1 = w0 + (int64_t)nw * W::kEach;
    const uint4 *src = reinterpret_cast<const uint4 *>(in + w0);
    uint4 r[W::kIter];
#pragma unroll
    for (int k = 0; k < W::kIter; ++k) {
        const int at = k * kThreads + (int)threadIdx.x;
        if (at >= nw) continue;
        if (SCALE && past) r[k] = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const ssd_u32x4 *>(src) + at));
        else r[k] = src[at];
    }
    const float coef = SCALE ? factor() : 0.0f;
    // in place, a factor of 1 leaves what is there
    if (SCALE && coef == 1.0f && in == out) return;
#pragma unroll
    for (int k = 0; k < W::kIter; ++k) {
        const int at = k * kThreads + (int)threadIdx.x;
        if (at >= nw) continue;
        float v[W::kEach];
        words<T>(r[k], v);
        if constexpr (SCALE) {
            uint4 o;
            if constexpr (sizeof(T) == 2) {
                o = uint4{ssd_pack(v[0] * coef, v[1] * coef), ssd_pack(v[2] * coef, v[3] * coef),
                          ssd_pack(v[4] * coef, v[5] * coef), ssd_pack(v[6] * coef, v[7] * coef)};
            } else {
                o = uint4{__float_as_uint(v[0] * coef), __float_as_uint(v[1] * coef), __float_as_uint(v[2] * coef),
                          __float_as_uint(v[3] * coef)};
            }
            if (past) __builtin_nontemporal_store(__builtin_bit_cast(ssd_u32x4, o), reinterpret_cast<ssd_u32x4 *>(out + w0) + at);
            else reinterpret_cast<uint4 *>(out + w0)[at] = o;
        } else {
#pragma unroll
            for (int e = 0; e < W::kEach; ++e) sum = fma((double)v[e], (double)v[e], sum);
        }
    }
    auto one = [&](int64_t e) {
        const float v = value<T>(in + e);
        if constexpr (SCALE) put<T>(out + e, v * coef);
        else sum = fma((double)v, (double)v, sum);
    };
    for (int64_t e = e0 + threadIdx.x; e < w0; e += kThreads) one(e);
    for (int64_t e = w1 + threadIdx.x; e < e1; e += kThreads) one(e);
}

// The sum over a workgroup's threads, to all of them
__device__ __forceinline__ double wg_sum(double v, double *s) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = 0.0;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) r += s[w];
    return r;
}

__global__ __launch_bounds__(kThreads) void grad_square_kernel(Table t, double *part) {
    __shared__ double s[kThreads / 64];
    uint32_t p0, p1;
    run_of(t, p0, p1);
    double sum = 0.0;
    int k = find(t, p0);
    for (uint32_t p = p0; p < p1; ++p) {
        while (p >= t.first[k + 1]) ++k;
        const int64_t e0 = (int64_t)(p - t.first[k]) * kPiece;
        auto none = [] { return 0.0f; };
        if (is_wide(t, k)) piece<float, false>(static_cast<const float *>(t.in[k]), nullptr, t.n[k], e0, none, false, sum);
        else piece<uint16_t, false>(static_cast<const uint16_t *>(t.in[k]), nullptr, t.n[k], e0, none, false, sum);
    }
    sum = wg_sum(sum, s);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The sum of all partial sums, the same in every workgroup of 256 that forms it
__device__ __forceinline__ double total(const double *part, int n, double *s) {
    double v = 0.0;
    for (int k = threadIdx.x; k < n; k += kThreads) v += part[k];
    return wg_sum(v, s);
}

// The norm, and the sum again where `sum` is given
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double *part, int n, float *norm, double *sum) {
    __shared__ double s[kThreads / 64];
    const double v = total(part, n, s);
    if (threadIdx.x != 0) return;
    *norm = (float)sqrt(v);
    if (sum) *sum = v;
}

// parts > 0: the norm is formed from the partial sums, and written where `write` is set; else it is read
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(Table t, const double *part, int parts, float *norm, int write,
                                                              float max_norm, float eps, int past) {
    __shared__ double s[kThreads / 64];
    bool known = false;
    float coef = 0.0f;
    auto factor = [&] {
        if (!known) {
            known = true;
            double v = parts > 0 ? sqrt(total(part, parts, s)) : (double)*norm;
            const float shown = (float)v;
            if (write && blockIdx.x == 0 && threadIdx.x == 0) *norm = shown;
            if (isinf(shown)) v = shown;      // beyond fp32 it is infinity, as the caller is told
            const double d = v + (double)eps, c = (double)max_norm / d;
            coef = c >= 1.0 || d == 0.0 ? 1.0f : (float)c;      // NaN stays
        }
        return coef;
    };
    uint32_t p0, p1;
    run_of(t, p0, p1);
    if (p0 >= p1) return;
    double none = 0.0;
    int k = find(t, p1 - 1);
    for (uint32_t p = p1; p-- > p0;) {
        while (p < t.first[k]) --k;
        const int64_t e0 = (int64_t)(p - t.first[k]) * kPiece;
        if (is_wide(t, k))
            piece<float, true>(static_cast<const float *>(t.in[k]), static_cast<float *>(t.out[k]), t.n[k], e0, factor, past != 0, none);
        else
            piece<uint16_t, true>(static_cast<const uint16_t *>(t.in[k]), static_cast<uint16_t *>(t.out[k]), t.n[k], e0, factor, past != 0, none);
    }
}

// ---------------------------------------------------------------------------
// Launching

struct List {
    int64_t count;
    const void *const *in;
    void *const *out;          // NULL: none is written
    const int64_t *n;
    const int32_t *dtype;
};

size_t esize(int t) { return t == SSM_BF16 ? 2 : 4; }
int64_t launches(int64_t count) { return (count + kPer - 1) / kPer; }
int64_t part_bytes(int64_t count) { return launches(count) * kWgs * (int64_t)sizeof(double) + (count ? 256 : 0); }   // and the sum

int check(const List &l) {
    if (l.count < 0 || l.count > (1 << 20)) return SSM_ERR_SHAPE;
    if (l.count == 0) return SSM_OK;
    if (!l.in || !l.n || !l.dtype) return SSM_ERR_NULL;
    for (int64_t k = 0; k < l.count; ++k) {
        if (l.n[k] < 0 || l.n[k] > kLongest) return SSM_ERR_SHAPE;
        if (l.dtype[k] != SSM_F32 && l.dtype[k] != SSM_BF16) return SSM_ERR_DTYPE;
    }
    for (int64_t k = 0; k < l.count; ++k) {
        if (l.n[k] == 0) continue;
        if (!l.in[k] || (l.out && !l.out[k])) return SSM_ERR_NULL;
        if (!aligned(l.in[k], esize(l.dtype[k])) || (l.out && !aligned(l.out[k], esize(l.dtype[k])))) return SSM_ERR_ALIGN;
    }
    return SSM_OK;
}

struct Item {
    uintptr_t lo, hi;
    int64_t owner;
    bool written;
};

// Whether anything written overlaps anything else, but a gradient written to itself.
// Sorted by address: a range overlaps an earlier one exactly if it begins before the
// furthest end so far.
int clashes(const List &l, Range norm, Range ws) {
    const int64_t most = 2 * l.count + 2;
    Item *v = static_cast<Item *>(malloc((size_t)most * sizeof(Item)));
    if (!v) return SSM_ERR_SHAPE;
    int64_t m = 0;
    auto add = [&](Range r, int64_t owner, bool written) {
        if (r.lo != 0 && r.lo < r.hi) v[m++] = Item{r.lo, r.hi, owner, written};
    };
    for (int64_t k = 0; k < l.count; ++k) {
        const int64_t bytes = l.n[k] * (int64_t)esize(l.dtype[k]);
        const Range a = range_of(l.in[k], bytes);
        if (!l.out) {
            add(a, k, false);
            continue;
        }
        const Range b = range_of(l.out[k], bytes);
        add(b, k, true);
        if (a.lo != b.lo) add(a, k, false);
    }
    add(norm, l.count, true);
    add(ws, l.count + 1, true);
    std::sort(v, v + m, [](const Item &a, const Item &b) { return a.lo < b.lo; });
    uintptr_t any = 0, out = 0;      // ends of all, and of what is written, so far
    bool bad = false;
    for (int64_t k = 0; k < m && !bad; ++k) {
        bad = v[k].lo < out || (v[k].written && v[k].lo < any);
        any = std::max(any, v[k].hi);
        if (v[k].written) out = std::max(out, v[k].hi);
    }
    free(v);
    return bad ? SSM_ERR_ALIAS : SSM_OK;
}

// The k-th launch's table, and its workgroups
unsigned table(const List &l, int64_t launch, Table &t) {
    const int64_t k0 = launch * kPer;
    t.count = (int)std::min<int64_t>(kPer, l.count - k0);
    for (uint32_t &w : t.wide) w = 0;
    uint32_t at = 0;
    for (int k = 0; k < t.count; ++k) {
        t.in[k] = l.in[k0 + k];
        t.out[k] = l.out ? l.out[k0 + k] : nullptr;
        t.n[k] = l.n[k0 + k];
        t.first[k] = at;
        if (l.dtype[k0 + k] == SSM_F32) t.wide[k >> 5] |= 1u << (k & 31);
        at += (uint32_t)((t.n[k] + kPiece - 1) / kPiece);
    }
    t.first[t.count] = at;
    return std::min<uint32_t>(at, kWgs);
}

// Partial sums of every launch, one after another; their number
int squares(const List &l, double *part, int &parts, hipStream_t st) {
    parts = 0;
    Table t;
    for (int64_t k = 0; k < launches(l.count); ++k) {
        const unsigned wgs = table(l, k, t);
        if (wgs == 0) continue;
        hipLaunchKernelGGL(grad_square_kernel, dim3(wgs), dim3(kThreads), 0, st, t, part + parts);
        if (hipGetLastError() != hipSuccess) return SSM_ERR_HIP;
        parts += (int)wgs;
    }
    return SSM_OK;
}

int scale(const List &l, const double *part, int parts, float *norm, bool write, float max_norm, float eps, hipStream_t st) {
    Table t;
    int64_t bytes = 0;
    for (int64_t k = 0; k < l.count; ++k) bytes += l.n[k] * (int64_t)esize(l.dtype[k]);
    const bool past = bytes > kCached;
    for (int64_t k = launches(l.count) - 1; k >= 0; --k) {
        const unsigned wgs = table(l, k, t);
        if (wgs == 0) continue;
        hipLaunchKernelGGL(grad_scale_kernel, dim3(wgs), dim3(kThreads), 0, st, t, part, parts, norm, (int)write, max_norm, eps, (int)past);
        if (hipGetLastError() != hipSuccess) return SSM_ERR_HIP;
        write = false;
    }
    return SSM_OK;
}

int norm_of(const double *part, int parts, float *norm, double *sum, hipStream_t st) {
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0, st, part, parts, norm, sum);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

bool factor_ok(float max_norm, float eps) { return max_norm >= 0.0f && max_norm <= 3e38f && eps >= 0.0f && eps <= 3e38f; }

}  // namespace

extern "C" size_t ssm_grad_workspace_size(int64_t count) {
    return count < 1 || count > (1 << 20) ? 0 : (size_t)part_bytes(count);
}

extern "C" int ssm_grad_norm(int64_t count, const void *const *grads, const int64_t *sizes, const int32_t *dtypes, float *norm,
                             void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const List l{count, grads, nullptr, sizes, dtypes};
    if (const int rc = check(l)) return rc;
    if (!norm) return SSM_ERR_NULL;
    if (!aligned(norm, 4)) return SSM_ERR_ALIGN;
    const int64_t need = part_bytes(count);
    if (need && (!workspace || workspace_bytes < (size_t)need)) return SSM_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
    if (const int rc = clashes(l, range_of(norm, 4), range_of(workspace, need))) return rc;
    int parts = 0;
    if (const int rc = squares(l, static_cast<double *>(workspace), parts, stream)) return rc;
    return norm_of(static_cast<double *>(workspace), parts, norm, nullptr, stream);
}

extern "C" int ssm_grad_clip(int64_t count, const void *const *grads, void *const *out, const int64_t *sizes,
                             const int32_t *dtypes, float max_norm, float eps, float *norm, void *workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    const List l{count, grads, out, sizes, dtypes};
    if (count > 0 && !out) return SSM_ERR_NULL;
    if (const int rc = check(l)) return rc;
    if (!factor_ok(max_norm, eps)) return SSM_ERR_UNSUPPORTED;
    if (!norm) return SSM_ERR_NULL;
    if (!aligned(norm, 4)) return SSM_ERR_ALIGN;
    const int64_t need = part_bytes(count);
    if (need && (!workspace || workspace_bytes < (size_t)need)) return SSM_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
    if (const int rc = clashes(l, range_of(norm, 4), range_of(workspace, need))) return rc;
    double *part = static_cast<double *>(workspace);
    int parts = 0;
    if (const int rc = squares(l, part, parts, stream)) return rc;
    if (parts == 0) return norm_of(part, 0, norm, nullptr, stream);
    if (parts <= kWgs) return scale(l, part, parts, norm, true, max_norm, eps, stream);
    double *sum = part + parts;
    if (const int rc = norm_of(part, parts, norm, sum, stream)) return rc;
    return scale(l, sum, 1, norm, false, max_norm, eps, stream);
}

extern "C" int ssm_grad_scale(int64_t count, const void *const *grads, void *const *out, const int64_t *sizes,
                              const int32_t *dtypes, const float *norm, float max_norm, float eps, hipStream_t stream) {
    const List l{count, grads, out, sizes, dtypes};
    if (count > 0 && !out) return SSM_ERR_NULL;
    if (const int rc = check(l)) return rc;
    if (!factor_ok(max_norm, eps)) return SSM_ERR_UNSUPPORTED;
    if (!norm) return SSM_ERR_NULL;
    if (!aligned(norm, 4)) return SSM_ERR_ALIGN;
    if (const int rc = clashes(l, range_of(norm, 4), Range{0, 0})) return rc;
    return scale(l, nullptr, 0, const_cast<float *>(norm), false, max_norm, eps, stream);
}
