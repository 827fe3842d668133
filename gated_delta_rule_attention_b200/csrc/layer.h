// layer.h -- what the operators around the attention share (scan.cu, rotary.cu, norm.cu, and their
// C entry points in abi_layer.cu): launch arguments, launchers, vector accesses.
#pragma once

#include "la_internal.cuh"

namespace la {

// The gated linear recurrence with a vector state.  The forward pass can keep the state in
// front of every kScanCheckpoint-th row for the backward pass.
constexpr int kScanCheckpoint = 32;
struct ScanArgs {
    int dtype;
    int B, T, C;             // step: B sequences of one token
    const void *x;
    const float *gate;
    const float *state_in;   // nullptr: zeros
    float *state_out;        // may be state_in
    void *h;
    float *ckpt;             // [B, ceil(T / kScanCheckpoint), C] or nullptr
    bool blend;
    cudaStream_t stream;
    const int *codes = nullptr;   // packed sequences: the row codes of launch_scan_rows
};
struct ScanBackwardArgs {
    int dtype;
    int B, T, C;
    const void *x, *dh;
    const float *gate, *ckpt, *dstate;
    void *dx;
    float *dgate, *dstate0;
    bool blend;
    cudaStream_t stream;
};

struct RotaryArgs {
    int dtype;
    int B, T, Hq, Hk, d, r;
    const void *q, *k;       // k: nullptr with Hk = 0
    void *yq, *yk;           // may be q, k where the layouts agree
    const double *freqs;     // [r / 2]
    const int *positions;    // [B, T] or nullptr: start + t
    long long start;
    float scale;
    bool interleaved, transpose, x_tokens, y_tokens;
    cudaStream_t stream;
};

struct NormArgs {
    int dtype;
    int B, H, T, C;          // x [B, H, T, C] -> y [B, T, H, C]
    const void *x, *residual;   // residual: nullptr or (H = 1) the stream
    const float *w;
    void *h, *y;
    float *scales;
    bool fp8;
    int group;               // columns a scale: 0 (the row) or 128
    float eps;
    cudaStream_t stream;
};
struct NormBackwardArgs {
    int dtype;
    int B, H, T, C;
    const void *h, *dy, *dres;
    const float *w;
    void *dx;
    float *dw, *partial;
    float eps;
    cudaStream_t stream;
};

// Launchers return cudaSuccess or the launch error.  They assume validated arguments.
cudaError_t launch_rotary(const RotaryArgs &a);
cudaError_t launch_norm(const NormArgs &a);
cudaError_t launch_norm_backward(const NormBackwardArgs &a);
size_t norm_backward_partial_bytes(long long rows, int C);
cudaError_t launch_scan(const ScanArgs &a);
cudaError_t launch_scan_step(const ScanArgs &a);
cudaError_t launch_scan_backward(const ScanBackwardArgs &a);
// Packed sequences: the code of every row, checks of the offsets; the state of every empty
// sequence is zeroed (zero_state: the state, or nullptr to leave it).
size_t scan_codes_bytes(int T);
cudaError_t launch_scan_rows(const ScanArgs &a, const int *cu, int N, int *codes, float *zero_state);

// ------------------------------------------------------------------------------- device side

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
