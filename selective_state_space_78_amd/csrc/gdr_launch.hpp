// Launches of the gated delta rule's kernels.
#pragma once

#include "gdr_kernels.hpp"

namespace ssm_detail {

#ifdef SSM_GDR_INSTANTIATE

// Waves per workgroup of the kernels that walk the chunks: 16 columns each
inline int gdr_waves(int P) { return P / 16 < 4 ? P / 16 : 4; }

template <int N>
hipError_t gdr_prep_launch(const GdrParams &p, hipStream_t st) {
    const int64_t blocks = (int64_t)p.batch * p.H * p.nc;
    hipLaunchKernelGGL((gdr_prep_kernel<N>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    return hipGetLastError();
}

template <int N>
hipError_t gdr_fwd_launch(const GdrParams &p, bool save, hipStream_t st) {
    const int nw = gdr_waves(p.P), splits = (p.P / 16 + nw - 1) / nw;
    const dim3 grid((unsigned)((int64_t)p.batch * p.H * splits));
    if (save)
        hipLaunchKernelGGL((gdr_fwd_kernel<N, true>), grid, dim3(64 * nw), 0, st, p, splits);
    else
        hipLaunchKernelGGL((gdr_fwd_kernel<N, false>), grid, dim3(64 * nw), 0, st, p, splits);
    return hipGetLastError();
}

template <int N>
hipError_t gdr_bwd_launch(const GdrParams &p, hipStream_t st) {
    const int nw = gdr_waves(p.P), splits = (p.P / 16 + nw - 1) / nw;
    hipLaunchKernelGGL((gdr_rev_kernel<N>), dim3((unsigned)((int64_t)p.batch * p.H * splits)), dim3(64 * nw), 0, st, p,
                       splits);
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
