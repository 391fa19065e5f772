// value_types.h -- loads and stores of f32, bf16 and f16 values as f32 (gfx950).
// DT is enum rad_dtype: 0 f32, 1 bf16, 2 f16.  Offsets count values.
#pragma once

#include "rad_device.h"

namespace rad {

constexpr int kDtF32 = 0, kDtBf16 = 1, kDtF16 = 2;

constexpr int dt_bytes(int dt) { return dt == kDtF32 ? 4 : 2; }

__device__ __forceinline__ uint32_t bf16_round(float f) {   // nearest even; bits in the low half
    return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f)));
}
__device__ __forceinline__ uint32_t f16_round(float f) {
    return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(f)));
}
__device__ __forceinline__ float f16_widen(uint32_t bits) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

template <int DT>
__device__ __forceinline__ uint32_t round16(float f) {
    static_assert(DT != kDtF32, "a 16-bit type");
    if constexpr (DT == kDtBf16) return bf16_round(f);
    else return f16_round(f);
}
template <int DT>
__device__ __forceinline__ float widen16(uint32_t bits) {
    if constexpr (DT == kDtBf16) return __uint_as_float(bits << 16);
    else return f16_widen(bits);
}
// f rounded to the type, as f32
template <int DT>
__device__ __forceinline__ float rounded(float f) {
    if constexpr (DT == kDtF32) return f;
    else return widen16<DT>(round16<DT>(f));
}

typedef float nt_float4 __attribute__((ext_vector_type(4)));
typedef unsigned int nt_uint2 __attribute__((ext_vector_type(2)));

// Four consecutive values (16 or 8 bytes, aligned to that); NT: nontemporal.
template <int DT, bool NT = false>
__device__ __forceinline__ float4 load4(const void *base, int64_t i) {
    if constexpr (DT == kDtF32) {
        const nt_float4 *p = reinterpret_cast<const nt_float4 *>(static_cast<const float *>(base) + i);
        nt_float4 v;
        if constexpr (NT) v = __builtin_nontemporal_load(p);
        else v = *p;
        return make_float4(v.x, v.y, v.z, v.w);
    } else {
        const nt_uint2 *p = reinterpret_cast<const nt_uint2 *>(static_cast<const uint16_t *>(base) + i);
        nt_uint2 v;
        if constexpr (NT) v = __builtin_nontemporal_load(p);
        else v = *p;
        return make_float4(widen16<DT>(v.x & 0xFFFFu), widen16<DT>(v.x >> 16), widen16<DT>(v.y & 0xFFFFu),
                           widen16<DT>(v.y >> 16));
    }
}
template <int DT, bool NT = false>
__device__ __forceinline__ void store4(void *base, int64_t i, float4 f) {
    if constexpr (DT == kDtF32) {
        nt_float4 *p = reinterpret_cast<nt_float4 *>(static_cast<float *>(base) + i);
        const nt_float4 v{f.x, f.y, f.z, f.w};
        if constexpr (NT) __builtin_nontemporal_store(v, p);
        else *p = v;
    } else {
        nt_uint2 *p = reinterpret_cast<nt_uint2 *>(static_cast<uint16_t *>(base) + i);
        const nt_uint2 v{round16<DT>(f.x) | (round16<DT>(f.y) << 16), round16<DT>(f.z) | (round16<DT>(f.w) << 16)};
        if constexpr (NT) __builtin_nontemporal_store(v, p);
        else *p = v;
    }
}

}  // namespace rad
