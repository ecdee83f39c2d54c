// io8.h -- eight consecutive elements of a float32 or bfloat16 row as floats
// in registers, and back (bfloat16 rounds to nearest, ties to even).
#pragma once
#include "mesa_device.h"

namespace mesa {

struct f32x8 { float v[8]; };

__device__ __forceinline__ f32x8 load8(const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return f32x8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ f32x8 load8(const bf16_t* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    f32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[2 * i] = __uint_as_float(w[i] << 16);
        r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(bf16_t* p, float x) {
    p->bits = __builtin_bit_cast(uint16_t, (__bf16)x);
}
__device__ __forceinline__ void store8(float* p, const f32x8& r) {
    *reinterpret_cast<f32x4*>(p) = f32x4{r.v[0], r.v[1], r.v[2], r.v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{r.v[4], r.v[5], r.v[6], r.v[7]};
}
__device__ __forceinline__ void store8(bf16_t* p, const f32x8& r) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(r.v[0], r.v[1]), bf16_pair(r.v[2], r.v[3]),
                                              bf16_pair(r.v[4], r.v[5]), bf16_pair(r.v[6], r.v[7]));
}

// The same at any element alignment, of the first `left` of the eight elements
// (the others read as zeros and are not written).  With WHOLE, left is 8 or
// more; without it a row's last, ragged piece goes element by element, which
// costs a branch at every access.  The stores are streaming ones: the outputs
// are larger than the caches, or too small for it to matter.
typedef float f32x4_el __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_el __attribute__((ext_vector_type(4), aligned(2)));
template <bool WHOLE>
__device__ __forceinline__ f32x8 load8_upto(const float* p, int left) {
    f32x8 r{};
    if (WHOLE || left >= 8) {
        const f32x4_el a = reinterpret_cast<const f32x4_el*>(p)[0], b = reinterpret_cast<const f32x4_el*>(p)[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) { r.v[e] = a[e]; r.v[4 + e] = b[e]; }
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) r.v[e] = p[e];
    }
    return r;
}
template <bool WHOLE>
__device__ __forceinline__ f32x8 load8_upto(const bf16_t* p, int left) {
    f32x8 r{};
    if (WHOLE || left >= 8) {
        const u32x4_el w = *reinterpret_cast<const u32x4_el*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[2 * i] = __uint_as_float(w[i] << 16);
            r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) r.v[e] = to_f32(p[e]);
    }
    return r;
}
template <bool WHOLE>
__device__ __forceinline__ void store8_upto(float* p, const f32x8& r, int left) {
    if (WHOLE || left >= 8) {
        __builtin_nontemporal_store(f32x4_el{r.v[0], r.v[1], r.v[2], r.v[3]}, reinterpret_cast<f32x4_el*>(p));
        __builtin_nontemporal_store(f32x4_el{r.v[4], r.v[5], r.v[6], r.v[7]}, reinterpret_cast<f32x4_el*>(p) + 1);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) p[e] = r.v[e];
    }
}
template <bool WHOLE>
__device__ __forceinline__ void store8_upto(bf16_t* p, const f32x8& r, int left) {
    if (WHOLE || left >= 8) {
        __builtin_nontemporal_store(u32x4_el{bf16_pair(r.v[0], r.v[1]), bf16_pair(r.v[2], r.v[3]),
                                             bf16_pair(r.v[4], r.v[5]), bf16_pair(r.v[6], r.v[7])},
                                    reinterpret_cast<u32x4_el*>(p));
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) store1(p + e, r.v[e]);
    }
}

}  // namespace mesa
