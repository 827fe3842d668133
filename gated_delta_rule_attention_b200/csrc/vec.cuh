// vec.cuh -- a few neighbouring values of a row as one vector access.
#pragma once

#include "la_internal.cuh"

namespace la {

// V values as they lie in memory; accesses of up to 16 bytes each (tensors start on 16-byte
// boundaries, not on wider ones).
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, V> *>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &x) {
    *reinterpret_cast<Pack<T, V> *>(p) = x;
}

}  // namespace la
