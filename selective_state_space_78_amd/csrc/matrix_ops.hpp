// Pieces shared by the matrix-core kernels: bf16 operands and their splits,
// the 16x16x32 MFMA, transposing LDS reads, wave prefix sums and range-checked
// buffer accesses.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace ssm_detail {

typedef __bf16 ssd_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 ssd_bf16x2 __attribute__((ext_vector_type(2)));
typedef float ssd_f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float ssd_bf(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

__device__ __forceinline__ uint16_t ssd_to_bf(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ __forceinline__ uint32_t ssd_pack(float lo, float hi) {
    const ssd_bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ ssd_f32x4 ssd_mfma(const ssd_bf16x8 &a, const ssd_bf16x8 &b, const ssd_f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ ssd_bf16x8 ssd_ld16(const uint16_t *p) {
    return __builtin_bit_cast(ssd_bf16x8, *reinterpret_cast<const uint4 *>(p));
}

// Transposing LDS read (ds_read_b64_tr_b16): within each group of 16 lanes,
// lane s supplies the address of 4 consecutive 16-bit values V_s[0..3], and
// lane 4q + c receives V_q[c], V_{q+4}[c], V_{q+8}[c], V_{q+12}[c]. With lane s
// pointing at row r0 + (s >> 2), columns c0 + 4 (s & 3) of a row-major tile,
// lane 4q + c gets column c0 + 4q + c of rows r0 .. r0 + 3: a column of the
// tile, as a matrix-core operand whose K runs along the rows needs it.
__device__ __forceinline__ uint2 ssd_ld_tr(const uint16_t *p) {
    typedef short v4i16 __attribute__((ext_vector_type(4)));
    const v4i16 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16 *)(p));
    return __builtin_bit_cast(uint2, v);
}

// Two transposing reads (K positions 0..3 and 4..7) as one operand.
__device__ __forceinline__ ssd_bf16x8 ssd_ld_tr2(const uint16_t *p0, const uint16_t *p1) {
    const uint2 a = ssd_ld_tr(p0);
    const uint2 b = ssd_ld_tr(p1);
    const uint4 v = {a.x, a.y, b.x, b.y};
    return __builtin_bit_cast(ssd_bf16x8, v);
}

// Inclusive prefix sum over the 64 lanes of a wave: Kogge-Stone steps within
// rows of 16 (DPP row shifts), then the row totals carried across rows (DPP
// row broadcasts of lanes 15 and 31). Lanes without a source add 0.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float ssd_dpp_add(float v, bool take) {
    const float u = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                                          ROW_MASK, 0xF, false));
    return take ? v + u : v;
}

__device__ __forceinline__ float ssd_prefix_sum(float v, int lane) {
    const int r = lane & 15;
    v = ssd_dpp_add<0x111, 0xF>(v, r >= 1);              // row_shr:1
    v = ssd_dpp_add<0x112, 0xF>(v, r >= 2);              // row_shr:2
    v = ssd_dpp_add<0x114, 0xF>(v, r >= 4);              // row_shr:4
    v = ssd_dpp_add<0x118, 0xF>(v, r >= 8);              // row_shr:8
    v = ssd_dpp_add<0x142, 0xA>(v, (lane & 16) != 0);    // row_bcast:15 -> rows 1, 3
    v = ssd_dpp_add<0x143, 0xC>(v, (lane & 32) != 0);    // row_bcast:31 -> rows 2, 3
    return v;
}

// Two floats as the hi and lo words of packed bf16 pairs whose sums carry 16
// significant bits: hi is the pair rounded to bf16, lo the two remainders
// rounded to bf16.
__device__ __forceinline__ void ssd_split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = ssd_pack(a, b);
    const float ra = a - __uint_as_float(hi << 16);
    const float rb = b - __uint_as_float(hi & 0xffff0000u);
    lo = ssd_pack(ra, rb);
}

typedef unsigned int ssd_u32x4 __attribute__((ext_vector_type(4)));

// A raw buffer of `bytes` bytes at `base` (dword 3: 32-bit data format, the
// setting for untyped access on gfx9). Buffer instructions check every access
// against that size: loads past it return zero and stores past it are
// dropped. Rows past the end of the sequence then need no branch, and the
// compiler's wait counts, which must assume the shortest path through a
// branch, stay exact.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t ssd_buffer(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ uint4 ssd_bload16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const ssd_u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
    return uint4{v.x, v.y, v.z, v.w};
}

__device__ __forceinline__ void ssd_bstore16(__amdgpu_buffer_rsrc_t r, uint32_t off, const uint4 &v) {
    __builtin_amdgcn_raw_buffer_store_b128(ssd_u32x4{v.x, v.y, v.z, v.w}, r, (int)off, 0, 0);
}

typedef unsigned int ssd_u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint2 ssd_bload8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const ssd_u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
    return uint2{v.x, v.y};
}

__device__ __forceinline__ void ssd_bstore8(__amdgpu_buffer_rsrc_t r, uint32_t off, const uint2 &v) {
    __builtin_amdgcn_raw_buffer_store_b64(ssd_u32x2{v.x, v.y}, r, (int)off, 0, 0);
}

}  // namespace ssm_detail
