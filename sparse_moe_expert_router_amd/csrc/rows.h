// Pieces shared by the kernels that work on rows held in registers (norm.hip,
// balance.hip; not part of the ABI).
#pragma once

#include "common.h"

namespace moe {

typedef float f32x8_t __attribute__((ext_vector_type(8)));

template <int kCtrl>
__device__ __forceinline__ float dpp_f32(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xF, 0xF, false));
}

__device__ __forceinline__ float readlane_f32(float v, int l) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
}

// Sum over the 16 lanes of a row of lanes, in every lane of it (fixed order).
__device__ __forceinline__ float sum16_f32(float v) {
    v += dpp_f32<0xB1>(v);   // quad_perm 1,0,3,2
    v += dpp_f32<0x4E>(v);   // quad_perm 2,3,0,1
    v += dpp_f32<0x141>(v);  // row_half_mirror
    v += dpp_f32<0x140>(v);  // row_mirror
    return v;
}

// Sum over the 64 lanes of a wave whose lanes are all active (fixed order); uniform.
__device__ __forceinline__ float wave_sum_f32(float v) {
    v = sum16_f32(v);
    return (readlane_f32(v, 0) + readlane_f32(v, 16)) + (readlane_f32(v, 32) + readlane_f32(v, 48));
}

// Eight consecutive values of a bf16 or fp32 row (16-byte aligned).
__device__ __forceinline__ f32x8_t load8(const void* p, int64_t i, int f32) {
    f32x8_t v;
    if (f32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        const uint4 a = s[0], b = s[1];
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
    return v;
}

__device__ __forceinline__ uint4 pack8(f32x8_t v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Eight consecutive values, rounded once to the row's type.
__device__ __forceinline__ void store8(void* p, int64_t i, int f32, f32x8_t v) {
    if (f32) {
        f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i);
        o[0] = __builtin_shufflevector(v, v, 0, 1, 2, 3);
        o[1] = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = pack8(v);
    }
}

// Column sums of a [rows][pitch] fp32 matrix by 1024 threads (p0, q), p0 < 128
// and q < 8, for the four columns at `base`: rows p0, p0 + 128, .., with eight
// loads on their way at a time (one after another, 1024 rows took 20 us);
// then the 128 sums of a column through `red`, in a fixed order.  Every thread
// writes red[p0][q] and passes a barrier in between; the result is p0 = 0's.
__device__ __forceinline__ f32x4_t sum_rows(const float* base, int rows, int pitch, int p0) {
    f32x4_t v = f32x4_t(0.0f);
    for (int p = p0; p < rows; p += 8 * 128) {
        f32x4_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = *reinterpret_cast<const f32x4_t*>(base + (size_t)(p + 128 * i < rows ? p + 128 * i : p) * pitch);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p + 128 * i < rows) v += u[i];
    }
    return v;
}
__device__ __forceinline__ f32x4_t sum_128(f32x4_t v, f32x4_t (*red)[8], int p0, int q) {
    if (p0 < 16) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += red[p0 + 16 * i][q];
        red[p0][q] = v;
    }
    __syncthreads();
    if (p0 == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) v += red[i][q];
    }
    return v;
}

}  // namespace moe
