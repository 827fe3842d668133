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

// n / d for 0 <= n < 2^31 by a product: with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (hi32(n m) + n) >> s (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994; the sum stays below 2^32 for these n).
struct FastDiv {
    unsigned d = 1, m = 1, s = 0;
    FastDiv() = default;
    explicit FastDiv(unsigned by) : d(by) {
        while (s < 31 && (1u << s) < d) ++s;
        m = (unsigned)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    }
    __device__ __forceinline__ unsigned operator()(unsigned n) const { return (__umulhi(n, m) + n) >> s; }
};

}  // namespace la
