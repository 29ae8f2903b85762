// quant.hpp -- the 8-bit row format on the device: e4m3 codes with one E8M0
// scale (a power of two) for each block of 128 columns.
#pragma once

#include "moonep_internal.hpp"

namespace moonep {

constexpr int32_t kQuantBlock = 128;

// Bytes of one row's scales: a dword for each four blocks.
__host__ __device__ inline int32_t scale_row_bytes(int32_t cols)
{
    return (int32_t)(4 * (((int64_t)cols + 4 * kQuantBlock - 1) / (4 * kQuantBlock)));
}

// E8M0 byte of a block from the fp32 bits of its largest magnitude: the least
// exponent e with amax <= 448 * 2^e.  448 = 1.75 * 2^8, so e is the exponent of
// amax less 8, and one more where its mantissa is above 1.75: adding
// 2^23 - 1 - 0x600000 carries into the exponent exactly there.  As integers,
// infinity and NaN are above every finite magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits)
{
    const int32_t b = (int32_t)((amax_bits + 0x1FFFFFu) >> 23) - 8;
    const uint32_t byte = amax_bits == 0 ? 127u : (uint32_t)(b < 1 ? 1 : b);
    return amax_bits >= 0x7F800000u ? 255u : byte;
}

// 2^(127 - byte), exact for every byte below 254 (scale_byte gives at most 247
// to a finite block).
__device__ __forceinline__ float inverse_scale(uint32_t byte)
{
    return __uint_as_float((254u - byte) << 23);
}

// Four scaled values to e4m3 codes, to nearest even; all NaN for byte 255.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d, float inv,
                                              uint32_t byte)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
    return byte == 255u ? 0x7F7F7F7Fu : (uint32_t)r;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// All-reduce over the 16 lanes of a DPP row: row_ror:n rotates within it.
constexpr int kDppRowRor1 = 0x121, kDppRowRor2 = 0x122, kDppRowRor4 = 0x124, kDppRowRor8 = 0x128;

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, true);
}

__device__ __forceinline__ uint32_t row16_max(uint32_t v)
{
    v = max(v, dpp<kDppRowRor8>(v));
    v = max(v, dpp<kDppRowRor4>(v));
    v = max(v, dpp<kDppRowRor2>(v));
    return max(v, dpp<kDppRowRor1>(v));
}

__device__ __forceinline__ uint32_t row16_min(uint32_t v)
{
    v = min(v, dpp<kDppRowRor8>(v));
    v = min(v, dpp<kDppRowRor4>(v));
    v = min(v, dpp<kDppRowRor2>(v));
    return min(v, dpp<kDppRowRor1>(v));
}

__device__ __forceinline__ float row16_sum(float v)
{
    v += __uint_as_float(dpp<kDppRowRor8>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kDppRowRor4>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kDppRowRor2>(__float_as_uint(v)));
    return v + __uint_as_float(dpp<kDppRowRor1>(__float_as_uint(v)));
}

// The first lane's value in all 16 lanes of a DPP row (row_newbcast:0).
constexpr int kDppRowBcast0 = 0x150;

__device__ __forceinline__ float row16_first(float v)
{
    return __uint_as_float(dpp<kDppRowBcast0>(__float_as_uint(v)));
}

// The scale bytes of the four 16-lane rows of a wave as one dword (uniform).
__device__ __forceinline__ uint32_t gather_scale_dword(uint32_t byte)
{
    const uint32_t b0 = (uint32_t)__builtin_amdgcn_readlane((int)byte, 0);
    const uint32_t b1 = (uint32_t)__builtin_amdgcn_readlane((int)byte, 16);
    const uint32_t b2 = (uint32_t)__builtin_amdgcn_readlane((int)byte, 32);
    const uint32_t b3 = (uint32_t)__builtin_amdgcn_readlane((int)byte, 48);
    return b0 | (b1 << 8) | (b2 << 16) | (b3 << 24);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A workgroup barrier that waits for this wave's LDS operations only: a
// __syncthreads would also wait for every load in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace moonep
