// Launches of the gated delta rule's kernels.
#pragma once

#include "abi_util.hpp"
#include "gdr_kernels.hpp"

namespace ssm_detail {

constexpr int kGdrCus = 256;

// workgroups per head of a walk with nw computing waves (of 16 columns) each
inline int gdr_splits(int P, int nw) { return (P / 16 + nw - 1) / nw; }

// Computing waves per workgroup of the kernels that walk the chunks of `heads` heads.
// LDS allows one workgroup per CU, so the rounds over the CUs count, times what a
// chunk takes: taken as 1.1 times as long with 4 waves as with 2, and 1.7 times with
// 8. Measured, 2 / 4 / 8 waves, us a chunk: forward 3.8 / 3.7 / 5.6 (N 128) and 2.9 /
// 2.7 / 4.4 (N 64), with kept states 4.0 / 4.8 / 6.6 and 3.1 / 3.1 / 5.4, backwards
// 4.0 / 5.3 / 6.9 and 3.0 / 3.2 / 5.2 (with 4 and N 128 12 to 17 registers spill).
// Over 24 to 320 heads of 64 and 128 columns, each N, the choice is within 12% of the
// best of the three, but for 320 heads of 128 x 128, where 3 rounds of 4 and 2 of 8
// count as much: 20% and 26% with kept states and backwards.
inline int gdr_waves(int64_t heads, int P) {
    auto time = [&](int nw, double chunk) { return (double)((heads * gdr_splits(P, nw) + kGdrCus - 1) / kGdrCus) * chunk; };
    const double t2 = time(2, 1.0), t4 = time(4, 1.1), t8 = time(8, 1.7);
    return t2 <= t4 && t2 <= t8 ? 2 : t4 <= t8 ? 4 : 8;
}

// Whether the launches over `chunks` chunks in each of `heads` heads stay below 2^32
// work items
inline bool gdr_fwd_grids_ok(int64_t heads, int64_t chunks, int P) {
    const int nw = gdr_waves(heads, P);
    return grid_ok(heads * chunks, 256) && grid_ok(heads * gdr_splits(P, nw), 64 * (nw + gdr_helpers(nw)));
}
inline bool gdr_bwd_grids_ok(int64_t groups, int64_t chunks, int H, int N) {
    return grid_ok(groups * chunks, 4 * N) && grid_ok(H, 256);
}

#ifdef SSM_GDR_INSTANTIATE

template <int N>
hipError_t gdr_prep_launch(const GdrParams &p, hipStream_t st) {
    const int64_t blocks = (int64_t)p.batch * p.H * p.nc;
    hipLaunchKernelGGL((gdr_prep_kernel<N>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    return hipGetLastError();
}

template <int N, int NW>
void gdr_fwd_nw(const GdrParams &p, bool save, hipStream_t st) {
    const int splits = gdr_splits(p.P, NW);
    const dim3 grid((unsigned)((int64_t)p.batch * p.H * splits));
    if (save && p.y == nullptr)
        hipLaunchKernelGGL((gdr_fwd_kernel<N, true, false, NW>), grid, dim3(64 * (NW + gdr_helpers(NW))), 0, st, p, splits);
    else if (save)
        hipLaunchKernelGGL((gdr_fwd_kernel<N, true, true, NW>), grid, dim3(64 * (NW + gdr_helpers(NW))), 0, st, p, splits);
    else
        hipLaunchKernelGGL((gdr_fwd_kernel<N, false, true, NW>), grid, dim3(64 * (NW + gdr_helpers(NW))), 0, st, p, splits);
}

template <int N>
hipError_t gdr_fwd_launch(const GdrParams &p, bool save, hipStream_t st) {
    const int nw = gdr_waves((int64_t)p.batch * p.H, p.P);
    if (nw == 8) gdr_fwd_nw<N, 8>(p, save, st);
    else if (nw == 4) gdr_fwd_nw<N, 4>(p, save, st);
    else gdr_fwd_nw<N, 2>(p, save, st);
    return hipGetLastError();
}

template <int N, int NW>
void gdr_rev_nw(const GdrParams &p, hipStream_t st) {
    const int splits = gdr_splits(p.P, NW);
    hipLaunchKernelGGL((gdr_rev_kernel<N, NW>), dim3((unsigned)((int64_t)p.batch * p.H * splits)),
                       dim3(64 * (NW + gdr_helpers(NW))), 0, st, p, splits);
}

template <int N>
hipError_t gdr_bwd_launch(const GdrParams &p, hipStream_t st) {
    const int nw = gdr_waves((int64_t)p.batch * p.H, p.P);
    if (nw == 8) gdr_rev_nw<N, 8>(p, st);
    else if (nw == 4) gdr_rev_nw<N, 4>(p, st);
    else gdr_rev_nw<N, 2>(p, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((int64_t)p.batch * p.G * p.nc));
    if (p.hpg == 1)
        hipLaunchKernelGGL((gdr_grad_kernel<N, true>), grid, dim3(4 * N), 0, st, p);
    else
        hipLaunchKernelGGL((gdr_grad_kernel<N, false>), grid, dim3(4 * N), 0, st, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gdr_reduce_kernel, dim3((unsigned)p.H), dim3(256), 0, st, p);
    return hipGetLastError();
}

#else

template <int N> hipError_t gdr_prep_launch(const GdrParams &p, hipStream_t st);
template <int N> hipError_t gdr_fwd_launch(const GdrParams &p, bool save, hipStream_t st);
template <int N> hipError_t gdr_bwd_launch(const GdrParams &p, hipStream_t st);

#endif

}  // namespace ssm_detail
