// mixer_device.h -- element access and reductions of the mixer kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace rssm {
namespace {

typedef float f8v __attribute__((ext_vector_type(8)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
// Rows taken from a projection's output start at any element, so wide
// accesses promise no more alignment than an element's; the hardware accepts
// 16-byte accesses at such addresses.
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u4u __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements of type T: raw8 as stored, and widened to fp32.
template <typename T> struct vec8;

template <> struct vec8<float> {
    struct raw8 { f4u a, b; };
    static __device__ __forceinline__ raw8 load(const float *p) {
        return {*reinterpret_cast<const f4u *>(p), *reinterpret_cast<const f4u *>(p + 4)};
    }
    // for data that is read once: does not displace what is in the caches
    static __device__ __forceinline__ raw8 load_once(const float *p) {
        return {__builtin_nontemporal_load(reinterpret_cast<const f4u *>(p)),
                __builtin_nontemporal_load(reinterpret_cast<const f4u *>(p + 4))};
    }
    static __device__ __forceinline__ raw8 zero() { return {(f4u)0.f, (f4u)0.f}; }
    static __device__ __forceinline__ void store_raw(float *p, const raw8 &r) {
        *reinterpret_cast<f4u *>(p) = r.a;
        *reinterpret_cast<f4u *>(p + 4) = r.b;
    }
    static __device__ __forceinline__ f8v widen(const raw8 &r) {
        return f8v{r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    }
    static __device__ __forceinline__ void store(float *p, f8v v) {
        *reinterpret_cast<f4u *>(p) = f4u{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f4u *>(p + 4) = f4u{v[4], v[5], v[6], v[7]};
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
};

template <> struct vec8<uint16_t> {   // bf16, carried as its 16 bits
    typedef u4u raw8;
    static __device__ __forceinline__ raw8 load(const uint16_t *p) { return *reinterpret_cast<const u4u *>(p); }
    static __device__ __forceinline__ raw8 load_once(const uint16_t *p) {
        return __builtin_nontemporal_load(reinterpret_cast<const u4u *>(p));
    }
    static __device__ __forceinline__ raw8 zero() { return (u4u)0u; }
    static __device__ __forceinline__ void store_raw(uint16_t *p, const raw8 &r) { *reinterpret_cast<u4u *>(p) = r; }
    static __device__ __forceinline__ f8v widen(const raw8 &r) {
        f8v v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
        return v;
    }
    // one rounding to nearest even
    static __device__ __forceinline__ void store(uint16_t *p, f8v v) {
        *reinterpret_cast<u4u *>(p) = __builtin_bit_cast(u4u, __builtin_convertvector(v, b8v));
    }
    static __device__ __forceinline__ float get(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
    static __device__ __forceinline__ void put(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
};

// Up to eight elements at p, `left` of them inside the row (zeros past them);
// FULL: eight or none.
template <bool FULL, typename T>
__device__ __forceinline__ f8v load_part(const T *p, int left) {
    f8v v = (f8v)0.f;
    if constexpr (FULL) {
        if (left > 0) v = vec8<T>::widen(vec8<T>::load(p));
        return v;
    }
    if (left >= 8) return vec8<T>::widen(vec8<T>::load(p));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) v[i] = vec8<T>::get(p + i);
    return v;
}

template <bool FULL, typename T>
__device__ __forceinline__ void store_part(T *p, f8v v, int left) {
    if (FULL || left >= 8) {
        vec8<T>::store(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) vec8<T>::put(p + i, v[i]);
}

// v sigmoid(v).  For v below -87.3 the reciprocal is below the smallest normal
// number and is flushed: results of less than 1.2e-36 in size become zero.
__device__ __forceinline__ float silu(float v) { return v * __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

}  // namespace
}  // namespace rssm
