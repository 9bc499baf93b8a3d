// Element types of the many-token operators (fp16, bf16, fp32 activations):
// conversions, and vectors of elements moved as one access.
#pragma once

#include "common.hpp"

namespace spmv {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct F16 {
    typedef _Float16 T;
    static constexpr int CODE = SPMV_F16;
};
struct BF16 {
    typedef __bf16 T;
    static constexpr int CODE = SPMV_BF16;
};
struct F32 {
    typedef float T;
    static constexpr int CODE = SPMV_F32;
};

inline bool dtype_ok(int32_t d) { return d == SPMV_F16 || d == SPMV_BF16 || d == SPMV_F32; }
// A grid holds fewer than 2^32 threads.
inline spmv_status check_grid(int64_t blocks, int threads = 256) {
    if (blocks > (int64_t)(UINT32_MAX / (unsigned)threads))
        return fail(SPMV_ERR_OVERFLOW, "the launch would need 2^32 threads or more");
    return SPMV_OK;
}
inline size_t dtype_size(int32_t d) { return d == SPMV_F32 ? 4 : 2; }

// N elements of type E, loaded and stored with one aligned access.
template <typename E, int N>
struct alignas(sizeof(typename E::T) * N) Vec {
    typename E::T v[N];
};

template <typename E, int N>
__device__ __forceinline__ Vec<E, N> load_vec(const typename E::T *p) {
    return *reinterpret_cast<const Vec<E, N> *>(p);
}
template <typename E, int N>
__device__ __forceinline__ void store_vec(typename E::T *p, const Vec<E, N> &v) {
    *reinterpret_cast<Vec<E, N> *>(p) = v;
}

// The same for 16 bytes at an address aligned to one element only (global
// memory takes such accesses on gfx950), and for data that is read or written
// once and need not stay in the caches.
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <typename E, int N>
__device__ __forceinline__ Vec<E, N> load_any(const typename E::T *p) {
    if constexpr (sizeof(Vec<E, N>) == 16)
        return __builtin_bit_cast(Vec<E, N>, (u32x4) * reinterpret_cast<const u32x4_any *>(p));
    else
        return load_vec<E, N>(p);
}
template <typename E, int N>
__device__ __forceinline__ Vec<E, N> load_once(const typename E::T *p) {
    if constexpr (sizeof(Vec<E, N>) == 16)
        return __builtin_bit_cast(Vec<E, N>, (u32x4)__builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p)));
    else
        return load_vec<E, N>(p);
}
template <typename E, int N>
__device__ __forceinline__ void store_any(typename E::T *p, const Vec<E, N> &v) {
    if constexpr (sizeof(Vec<E, N>) == 16)
        *reinterpret_cast<u32x4_any *>(p) = __builtin_bit_cast(u32x4, v);
    else
        store_vec<E, N>(p, v);
}
template <typename E, int N>
__device__ __forceinline__ void store_once(typename E::T *p, const Vec<E, N> &v) {
    if constexpr (sizeof(Vec<E, N>) == 16)
        __builtin_nontemporal_store((u32x4_any)__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4_any *>(p));
    else
        store_vec<E, N>(p, v);
}

}  // namespace spmv
