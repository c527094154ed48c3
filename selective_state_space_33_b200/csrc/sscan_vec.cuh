// sscan_vec.cuh -- V neighbouring elements of an fp32 or bf16 row in one access (2 to 16
// bytes), widened to fp32 and rounded back (to nearest even).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

namespace sscan {

template <int B> struct Raw;
template <> struct Raw<2> { using type = unsigned short; };
template <> struct Raw<4> { using type = unsigned int; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };

template <typename T, int V>
struct Vec {
    using R = typename Raw<V * sizeof(T)>::type;
    R r;
    // through the read-only path: the kernel writes nothing at this address
    __device__ __forceinline__ void load(const T* p) { r = __ldg(reinterpret_cast<const R*>(p)); }
    // memory that this thread itself overwrites later
    __device__ __forceinline__ void load_rw(const T* p) { r = *reinterpret_cast<const R*>(p); }
    __device__ __forceinline__ void zero() { r = R{}; }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<R*>(p) = r; }
    __device__ __forceinline__ void get(float (&x)[V]) const {
        if constexpr (sizeof(T) == 4) {
            const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = f[v];
        } else if constexpr (V == 1) {
            x[0] = __uint_as_float((unsigned int)r << 16);
        } else {
            const unsigned int* w = reinterpret_cast<const unsigned int*>(&r);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) {
                x[2 * v] = __uint_as_float(w[v] << 16);
                x[2 * v + 1] = __uint_as_float(w[v] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&x)[V]) {
        if constexpr (sizeof(T) == 4) {
            float* f = reinterpret_cast<float*>(&r);
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = x[v];
        } else if constexpr (V == 1) {
            r = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
        } else {
            unsigned int* w = reinterpret_cast<unsigned int*>(&r);
#pragma unroll
            for (int v = 0; v < V / 2; ++v) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * v], x[2 * v + 1]);
                w[v] = *reinterpret_cast<const unsigned int*>(&t);
            }
        }
    }
};

template <int V, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[V]) {
    Vec<T, V> t;
    t.load(p);
    t.get(x);
}

// V neighbouring elements of a shared-memory tile.
template <int V, typename T>
__device__ __forceinline__ void load_shared(const T* p, float (&x)[V]) {
    Vec<T, V> t;
    t.load_rw(p);
    t.get(x);
}

template <int V, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
    Vec<T, V> t;
    t.set(x);
    t.store(p);
}

}  // namespace sscan
