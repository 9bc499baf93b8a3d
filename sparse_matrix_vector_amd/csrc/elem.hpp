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

}  // namespace spmv
