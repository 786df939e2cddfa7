// Launches of the gated delta rule's kernels.
#pragma once

#include "gdr_kernels.hpp"

namespace ssm_detail {

#ifdef SSM_GDR_INSTANTIATE

// Waves (of 16 columns) per workgroup of the kernels that walk the chunks: 8
// when that leaves a workgroup for most CUs, else 4, so that a head's columns
// spread over two
inline int gdr_waves(const GdrParams &p) {
    const int64_t heads = (int64_t)p.batch * p.H;
    return p.P > 64 && heads * ((p.P / 16 + 7) / 8) >= 192 ? 8 : 4;
}

template <int N>
hipError_t gdr_prep_launch(const GdrParams &p, hipStream_t st) {
    const int64_t blocks = (int64_t)p.batch * p.H * p.nc;
    hipLaunchKernelGGL((gdr_prep_kernel<N>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    return hipGetLastError();
}

template <int N, int NW>
void gdr_fwd_nw(const GdrParams &p, bool save, hipStream_t st) {
    const int splits = (p.P / 16 + NW - 1) / NW;
    const dim3 grid((unsigned)((int64_t)p.batch * p.H * splits));
    if (save)
        hipLaunchKernelGGL((gdr_fwd_kernel<N, true, NW>), grid, dim3(64 * NW), 0, st, p, splits);
    else
        hipLaunchKernelGGL((gdr_fwd_kernel<N, false, NW>), grid, dim3(64 * NW), 0, st, p, splits);
}

template <int N>
hipError_t gdr_fwd_launch(const GdrParams &p, bool save, hipStream_t st) {
    if (gdr_waves(p) == 8) gdr_fwd_nw<N, 8>(p, save, st);
    else gdr_fwd_nw<N, 4>(p, save, st);
    return hipGetLastError();
}

template <int N, int NW>
void gdr_rev_nw(const GdrParams &p, hipStream_t st) {
    const int splits = (p.P / 16 + NW - 1) / NW;
    hipLaunchKernelGGL((gdr_rev_kernel<N, NW>), dim3((unsigned)((int64_t)p.batch * p.H * splits)), dim3(64 * NW), 0, st,
                       p, splits);
}

template <int N>
hipError_t gdr_bwd_launch(const GdrParams &p, hipStream_t st) {
    if (gdr_waves(p) == 8) gdr_rev_nw<N, 8>(p, st);
    else gdr_rev_nw<N, 4>(p, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdr_grad_kernel<N>), dim3((unsigned)((int64_t)p.batch * p.G * p.nc)), dim3(4 * N), 0, st, p);
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
