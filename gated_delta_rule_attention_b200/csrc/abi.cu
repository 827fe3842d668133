// abi.cu -- the extern "C" boundary of liblinattn (declared in include/la.h).
//
// Host-side only: argument validation, chunk resolution, dispatch to a kernel launcher
// on the caller's stream, and the device failure word.  No entry point allocates
// device memory or keeps a pointer past its return.
#include "la_internal.cuh"

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <utility>

namespace la {

static std::atomic<unsigned long long> g_launches{0};
void note_launches(unsigned n) { g_launches.fetch_add(n, std::memory_order_relaxed); }

__device__ unsigned g_device_error;

unsigned *device_error_word() {
    constexpr int kMaxDevices = 64;
    static unsigned *addr[kMaxDevices] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
        addr[dev] = static_cast<unsigned *>(p);
    }
    return addr[dev];
}

namespace {

constexpr long long kMaxElems = 1ll << 40;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// True if `p` is memory the current device can address as global memory.
bool device_pointer(const void *p) {
    if (!p) return false;
    cudaPointerAttributes attr;
    const cudaError_t err = cudaPointerGetAttributes(&attr, p);
    if (err != cudaSuccess) {
        (void)cudaGetLastError();  // clear the non-sticky error this query may leave
        return false;
    }
    if (attr.type == cudaMemoryTypeManaged) return true;
    if (attr.type != cudaMemoryTypeDevice) return false;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    return attr.device == dev;
}

bool tensor_ok(const void *p, uintptr_t align) { return p && aligned(p, align) && device_pointer(p); }

la_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

// Modes that take beta (the delta rule).
bool delta_mode(int mode) { return mode == LA_MODE_GATED_DELTA || mode == LA_MODE_KDA; }
// The RetNet mode is the scalar-gate mode with one constant gate per head.
int internal_mode(int mode) { return mode == LA_MODE_RETNET ? (int)LA_MODE_GATED : mode; }

bool dims_ok(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

// Bytes of a call's gate tensor: per token (a scalar, or d_k values in the per-channel mode)
// or one value per head (the constant-decay mode).
size_t gate_bytes(int mode, long long tokens_x_heads, int H, int d_k) {
    if (mode == LA_MODE_RETNET) return sizeof(float) * (size_t)H;
    return sizeof(float) * (size_t)tokens_x_heads * (mode == LA_MODE_KDA ? d_k : 1);
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" la_status_t la_prefill(la_mode_t mode, la_dtype_t dtype, int B, int H, int T, int d_k,
                                  int d_v, const void *q, const void *k, const void *v,
                                  const float *gate, const float *beta, float *state, float *z,
                                  void *o, int chunk, unsigned flags, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    timer_reset();
    if (mode < LA_MODE_ELU1_NORM || mode > LA_MODE_RETNET) return LA_ERR_INVALID_ARG;
    if (mode == LA_MODE_RETNET && !tensor_ok(gate, 4)) return LA_ERR_INVALID_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 0) return LA_ERR_INVALID_ARG;
    if (flags & ~LA_FLAG_INIT_STATE) return LA_ERR_INVALID_ARG;
    if (chunk < 0) return LA_ERR_INVALID_ARG;
    if (!dims_ok(d_k, d_v)) return LA_ERR_UNSUPPORTED;
    const long long BH = (long long)B * H;
    if (BH > INT32_MAX || BH * T * (long long)(d_k > d_v ? d_k : d_v) > kMaxElems)
        return LA_ERR_INVALID_ARG;
    const bool init = (flags & LA_FLAG_INIT_STATE) != 0;
    if (!tensor_ok(state, 16)) return LA_ERR_INVALID_ARG;
    if (mode == LA_MODE_ELU1_NORM && !tensor_ok(z, 16)) return LA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (init) return LA_OK;
        cudaError_t e = cudaMemsetAsync(state, 0, sizeof(float) * BH * d_v * d_k, st);
        if (e == cudaSuccess && mode == LA_MODE_ELU1_NORM)
            e = cudaMemsetAsync(z, 0, sizeof(float) * BH * d_k, st);
        return from_cuda(e);
    }
    if (!tensor_ok(q, 16) || !tensor_ok(k, 16) || !tensor_ok(v, 16) || !tensor_ok(o, 16))
        return LA_ERR_INVALID_ARG;
    if (mode != LA_MODE_ELU1_NORM && gate && !tensor_ok(gate, 4)) return LA_ERR_INVALID_ARG;
    if (delta_mode(mode) && !tensor_ok(beta, 4)) return LA_ERR_INVALID_ARG;
    {
        const size_t es = dtype == LA_BF16 ? 2 : 4, th = (size_t)BH * T;
        const bool z_used = mode == LA_MODE_ELU1_NORM;
        if (!writes_disjoint({{o, th * d_v * es}, {state, sizeof(float) * BH * d_v * d_k},
                              {z_used ? z : nullptr, sizeof(float) * BH * d_k}},
                             {{q, th * d_k * es}, {k, th * d_k * es}, {v, th * d_v * es},
                              {z_used ? nullptr : gate, gate_bytes(mode, (long long)th, H, d_k)},
                              {delta_mode(mode) ? beta : nullptr, sizeof(float) * th},
                              {workspace, workspace ? workspace_bytes : 0}}))
            return LA_ERR_INVALID_ARG;
    }

    PrefillArgs a;
    a.mode = internal_mode(mode);
    a.gate_heads = (mode == LA_MODE_RETNET) ? H : 0;
    a.dtype = dtype;
    a.B = B; a.H = H; a.T = T; a.dk = d_k; a.dv = d_v;
    a.q = q; a.k = k; a.v = v;
    a.gate = (mode == LA_MODE_ELU1_NORM) ? nullptr : gate;
    a.beta = delta_mode(mode) ? beta : nullptr;
    a.state = state;
    a.z = (mode == LA_MODE_ELU1_NORM) ? z : nullptr;
    a.o = o;
    a.init_state = init;
    a.stream = st;
    if (workspace && workspace_bytes && !tensor_ok(workspace, 16)) return LA_ERR_INVALID_ARG;
    if (prefill_tc_supports(internal_mode(mode), dtype, d_k, d_v, chunk)) {
        a.chunk = 64;
        return from_cuda(launch_prefill_tc(a, workspace, workspace ? workspace_bytes : 0));
    }
    int resolved = 0;
    if (!prefill_simt_supports(dtype, d_k, d_v, chunk, &resolved)) return LA_ERR_UNSUPPORTED;
    a.chunk = resolved;
    return from_cuda(launch_prefill_simt(a));
}

extern "C" la_status_t la_prefill_varlen(la_mode_t mode, la_dtype_t dtype, int N, int H, int T,
                                         int d_k, int d_v, const int *cu_seqlens, const void *q,
                                         const void *k, const void *v, const float *gate,
                                         const float *beta, float *state, float *z, void *o,
                                         int chunk, unsigned flags, void *stream) {
    timer_reset();
    if (mode < LA_MODE_ELU1_NORM || mode > LA_MODE_RETNET) return LA_ERR_INVALID_ARG;
    if (mode == LA_MODE_RETNET && !tensor_ok(gate, 4)) return LA_ERR_INVALID_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (N < 1 || H < 1 || T < 0) return LA_ERR_INVALID_ARG;
    if (flags & ~LA_FLAG_INIT_STATE) return LA_ERR_INVALID_ARG;
    if (chunk < 0) return LA_ERR_INVALID_ARG;
    if (!dims_ok(d_k, d_v)) return LA_ERR_UNSUPPORTED;
    if ((long long)N * H > INT32_MAX || (long long)H * T * (d_k > d_v ? d_k : d_v) > kMaxElems)
        return LA_ERR_INVALID_ARG;
    const bool init = (flags & LA_FLAG_INIT_STATE) != 0;
    if (!tensor_ok(cu_seqlens, 4) || !tensor_ok(state, 16)) return LA_ERR_INVALID_ARG;
    if (mode == LA_MODE_ELU1_NORM && !tensor_ok(z, 16)) return LA_ERR_INVALID_ARG;
    if (T > 0) {
        if (!tensor_ok(q, 16) || !tensor_ok(k, 16) || !tensor_ok(v, 16) || !tensor_ok(o, 16))
            return LA_ERR_INVALID_ARG;
        if (mode != LA_MODE_ELU1_NORM && gate && !tensor_ok(gate, 4)) return LA_ERR_INVALID_ARG;
        if (delta_mode(mode) && !tensor_ok(beta, 4)) return LA_ERR_INVALID_ARG;
    }
    {
        const size_t es = dtype == LA_BF16 ? 2 : 4, th = (size_t)H * T;
        const bool z_used = mode == LA_MODE_ELU1_NORM;
        if (!writes_disjoint({{T > 0 ? o : nullptr, th * d_v * es},
                              {state, sizeof(float) * N * H * d_v * d_k},
                              {z_used ? z : nullptr, sizeof(float) * N * H * d_k}},
                             {{cu_seqlens, sizeof(int) * (N + 1)},
                              {T > 0 ? q : nullptr, th * d_k * es}, {T > 0 ? k : nullptr, th * d_k * es},
                              {T > 0 ? v : nullptr, th * d_v * es},
                              {z_used || T == 0 ? nullptr : gate, gate_bytes(mode, (long long)th, H, d_k)},
                              {delta_mode(mode) && T > 0 ? beta : nullptr, sizeof(float) * th}}))
            return LA_ERR_INVALID_ARG;
    }
    PrefillArgs a;
    a.mode = internal_mode(mode);
    a.gate_heads = (mode == LA_MODE_RETNET) ? H : 0;
    a.dtype = dtype;
    a.B = 1; a.H = H; a.T = T; a.dk = d_k; a.dv = d_v;
    a.q = q; a.k = k; a.v = v;
    a.gate = (mode == LA_MODE_ELU1_NORM) ? nullptr : gate;
    a.beta = delta_mode(mode) ? beta : nullptr;
    a.state = state;
    a.z = (mode == LA_MODE_ELU1_NORM) ? z : nullptr;
    a.o = o;
    a.init_state = init;
    a.stream = static_cast<cudaStream_t>(stream);
    a.cu = cu_seqlens;
    a.nseq = N;
    if (T == 0) {   // every sequence is empty
        if (init) return LA_OK;
        return from_cuda(launch_zero_empty_sequences(a));
    }
    if (prefill_tc_supports(internal_mode(mode), dtype, d_k, d_v, chunk)) {
        a.chunk = 64;
        cudaError_t e = launch_prefill_tc(a, nullptr, 0);
        if (e == cudaSuccess && !init) e = launch_zero_empty_sequences(a);
        return from_cuda(e);
    }
    int resolved = 0;
    if (!prefill_simt_supports(dtype, d_k, d_v, chunk, &resolved)) return LA_ERR_UNSUPPORTED;
    a.chunk = resolved;
    return from_cuda(launch_prefill_simt(a));
}

extern "C" size_t la_prefill_workspace_size(la_mode_t mode, la_dtype_t dtype, int B, int H, int T,
                                            int d_k, int d_v, int chunk) {
    if (mode < LA_MODE_ELU1_NORM || mode > LA_MODE_RETNET || B < 1 || H < 1 || T < 1)
        return 0;
    if (!prefill_tc_supports(internal_mode(mode), dtype, d_k, d_v, chunk)) return 0;
    return prefill_tc_workspace_bytes(internal_mode(mode), B, H, T);
}

extern "C" la_status_t la_decode_step(la_mode_t mode, la_dtype_t dtype, int N, int H, int d_k,
                                      int d_v, const void *q, const void *k, const void *v,
                                      const float *gate, const float *beta, float *state,
                                      float *z, void *o, void *stream) {
    timer_reset();
    if (mode < LA_MODE_ELU1_NORM || mode > LA_MODE_RETNET) return LA_ERR_INVALID_ARG;
    if (mode == LA_MODE_RETNET && !tensor_ok(gate, 4)) return LA_ERR_INVALID_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (N < 1 || H < 1) return LA_ERR_INVALID_ARG;
    if (!dims_ok(d_k, d_v)) return LA_ERR_UNSUPPORTED;
    const long long NH = (long long)N * H;
    if (NH > INT32_MAX) return LA_ERR_INVALID_ARG;
    const uintptr_t io_align = dtype == LA_BF16 ? 2 : 4;
    if (!tensor_ok(q, io_align) || !tensor_ok(k, io_align) || !tensor_ok(v, io_align) ||
        !tensor_ok(o, io_align) || !tensor_ok(state, 16))
        return LA_ERR_INVALID_ARG;
    if (mode == LA_MODE_ELU1_NORM && !tensor_ok(z, 16)) return LA_ERR_INVALID_ARG;
    if (mode != LA_MODE_ELU1_NORM && gate && !tensor_ok(gate, 4)) return LA_ERR_INVALID_ARG;
    if (delta_mode(mode) && !tensor_ok(beta, 4)) return LA_ERR_INVALID_ARG;
    {
        const size_t es = dtype == LA_BF16 ? 2 : 4;
        const bool z_used = mode == LA_MODE_ELU1_NORM;
        if (!writes_disjoint({{o, (size_t)NH * d_v * es}, {state, sizeof(float) * NH * d_v * d_k},
                              {z_used ? z : nullptr, sizeof(float) * NH * d_k}},
                             {{q, (size_t)NH * d_k * es}, {k, (size_t)NH * d_k * es},
                              {v, (size_t)NH * d_v * es},
                              {z_used ? nullptr : gate, gate_bytes(mode, NH, H, d_k)},
                              {delta_mode(mode) ? beta : nullptr, sizeof(float) * NH}}))
            return LA_ERR_INVALID_ARG;
    }
    DecodeArgs a;
    a.mode = internal_mode(mode);
    a.gate_heads = (mode == LA_MODE_RETNET) ? H : 0;
    a.dtype = dtype;
    a.N = N; a.H = H; a.dk = d_k; a.dv = d_v;
    a.q = q; a.k = k; a.v = v;
    a.gate = (mode == LA_MODE_ELU1_NORM) ? nullptr : gate;
    a.beta = delta_mode(mode) ? beta : nullptr;
    a.state = state;
    a.z = (mode == LA_MODE_ELU1_NORM) ? z : nullptr;
    a.o = o;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(launch_decode(a));
}

extern "C" la_status_t la_short_conv(la_dtype_t dtype, int B, int T, int H, int d, int width,
                                     const void *x, const float *w, const void *window_in,
                                     void *window_out, void *y, unsigned flags, void *stream) {
    timer_reset();
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (B < 1 || T < 0 || H < 1 || width < 1 || width > 4) return LA_ERR_INVALID_ARG;
    if (flags & ~(LA_CONV_SILU | LA_CONV_L2NORM)) return LA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return LA_ERR_UNSUPPORTED;
    const long long C = (long long)H * d;
    if (C > INT32_MAX || (long long)B * T * C > kMaxElems) return LA_ERR_INVALID_ARG;
    if (!tensor_ok(w, 4)) return LA_ERR_INVALID_ARG;
    const size_t es = dtype == LA_BF16 ? 2 : 4;
    const size_t win_bytes = (size_t)B * (width - 1) * C * es;
    const void *win_in = width > 1 ? window_in : nullptr;
    void *win_out = width > 1 ? window_out : nullptr;
    if (win_in && !tensor_ok(win_in, 16)) return LA_ERR_INVALID_ARG;
    if (win_out && !tensor_ok(win_out, 16)) return LA_ERR_INVALID_ARG;
    if (win_in != win_out && overlap(win_in, win_bytes, win_out, win_bytes)) return LA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (!win_out || win_out == win_in) return LA_OK;
        return from_cuda(win_in ? cudaMemcpyAsync(win_out, win_in, win_bytes, cudaMemcpyDeviceToDevice, st)
                                : cudaMemsetAsync(win_out, 0, win_bytes, st));
    }
    if (!tensor_ok(x, 16) || !tensor_ok(y, 16)) return LA_ERR_INVALID_ARG;
    const size_t xy_bytes = (size_t)B * T * C * es;
    if (overlap(x, xy_bytes, y, xy_bytes) || overlap(y, xy_bytes, win_in, win_bytes) ||
        overlap(y, xy_bytes, win_out, win_bytes) || overlap(x, xy_bytes, win_out, win_bytes))
        return LA_ERR_INVALID_ARG;
    ConvArgs a;
    a.dtype = dtype;
    a.B = B; a.T = T; a.H = H; a.d = d; a.width = width;
    a.step = false;
    a.silu = (flags & LA_CONV_SILU) != 0;
    a.l2norm = (flags & LA_CONV_L2NORM) != 0;
    a.x = x; a.w = w; a.win_in = win_in; a.win_out = win_out; a.y = y;
    a.stream = st;
    return from_cuda(launch_short_conv(a));
}

extern "C" la_status_t la_short_conv_varlen(la_dtype_t dtype, int N, int T, int H, int d,
                                            int width, const int *cu_seqlens, const void *x,
                                            const float *w, const void *window_in,
                                            void *window_out, void *y, unsigned flags,
                                            void *stream) {
    timer_reset();
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (N < 1 || T < 0 || H < 1 || width < 1 || width > 4) return LA_ERR_INVALID_ARG;
    if (flags & ~(LA_CONV_SILU | LA_CONV_L2NORM)) return LA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return LA_ERR_UNSUPPORTED;
    const long long C = (long long)H * d;
    if (C > INT32_MAX || (long long)T * C > kMaxElems || (long long)N * C * width > kMaxElems)
        return LA_ERR_INVALID_ARG;
    if (!tensor_ok(w, 4) || !tensor_ok(cu_seqlens, 4)) return LA_ERR_INVALID_ARG;
    const size_t es = dtype == LA_BF16 ? 2 : 4;
    const size_t win_bytes = (size_t)N * (width - 1) * C * es;
    const void *win_in = width > 1 ? window_in : nullptr;
    void *win_out = width > 1 ? window_out : nullptr;
    if (win_in && !tensor_ok(win_in, 16)) return LA_ERR_INVALID_ARG;
    if (win_out && !tensor_ok(win_out, 16)) return LA_ERR_INVALID_ARG;
    if (win_in != win_out && overlap(win_in, win_bytes, win_out, win_bytes)) return LA_ERR_INVALID_ARG;
    if (T > 0) {
        if (!tensor_ok(x, 16) || !tensor_ok(y, 16)) return LA_ERR_INVALID_ARG;
        const size_t xy_bytes = (size_t)T * C * es;
        if (overlap(x, xy_bytes, y, xy_bytes) || overlap(y, xy_bytes, win_in, win_bytes) ||
            overlap(y, xy_bytes, win_out, win_bytes) || overlap(x, xy_bytes, win_out, win_bytes))
            return LA_ERR_INVALID_ARG;
    }
    ConvArgs a;
    a.dtype = dtype;
    a.B = N; a.T = T; a.H = H; a.d = d; a.width = width;
    a.step = false;
    a.silu = (flags & LA_CONV_SILU) != 0;
    a.l2norm = (flags & LA_CONV_L2NORM) != 0;
    a.x = x; a.w = w; a.win_in = win_in; a.win_out = win_out; a.y = y;
    a.stream = static_cast<cudaStream_t>(stream);
    a.cu = cu_seqlens;
    return from_cuda(launch_short_conv(a));
}

extern "C" la_status_t la_short_conv_step(la_dtype_t dtype, int N, int H, int d, int width,
                                          const void *x, const float *w, void *window, void *y,
                                          unsigned flags, void *stream) {
    timer_reset();
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (N < 1 || H < 1 || width < 1 || width > 4) return LA_ERR_INVALID_ARG;
    if (flags & ~(LA_CONV_SILU | LA_CONV_L2NORM)) return LA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return LA_ERR_UNSUPPORTED;
    const long long C = (long long)H * d;
    if (C > INT32_MAX || (long long)N * C * width > kMaxElems) return LA_ERR_INVALID_ARG;
    if (!tensor_ok(w, 4) || !tensor_ok(x, 16) || !tensor_ok(y, 16)) return LA_ERR_INVALID_ARG;
    void *win = width > 1 ? window : nullptr;
    if (width > 1 && !tensor_ok(win, 16)) return LA_ERR_INVALID_ARG;
    const size_t es = dtype == LA_BF16 ? 2 : 4;
    const size_t xy_bytes = (size_t)N * C * es, win_bytes = (size_t)N * (width - 1) * C * es;
    if (overlap(x, xy_bytes, y, xy_bytes) || overlap(win, win_bytes, x, xy_bytes) ||
        overlap(win, win_bytes, y, xy_bytes))
        return LA_ERR_INVALID_ARG;
    ConvArgs a;
    a.dtype = dtype;
    a.B = N; a.T = 1; a.H = H; a.d = d; a.width = width;
    a.step = true;
    a.silu = (flags & LA_CONV_SILU) != 0;
    a.l2norm = (flags & LA_CONV_L2NORM) != 0;
    a.x = x; a.w = w; a.win_in = win; a.win_out = win; a.y = y;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(launch_short_conv(a));
}

extern "C" la_status_t la_check_status(void *stream) {
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return LA_ERR_CUDA;
    unsigned *word = device_error_word();
    if (!word) return LA_ERR_CUDA;
    unsigned host = 0;
    if (cudaMemcpy(&host, word, sizeof(host), cudaMemcpyDeviceToHost) != cudaSuccess)
        return LA_ERR_CUDA;
    if (host == 0) return LA_OK;
    const unsigned zero = 0;
    if (cudaMemcpy(word, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
        return LA_ERR_CUDA;
    if (host & kErrTimeout) return LA_ERR_TIMEOUT;
    if (host & kErrBadInput) return LA_ERR_INVALID_ARG;
    return LA_ERR_CUDA;
}

extern "C" const char *la_status_string(la_status_t s) {
    switch (s) {
        case LA_OK: return "LA_OK: success";
        case LA_ERR_INVALID_ARG: return "LA_ERR_INVALID_ARG: invalid argument (pointer, size, mode or dtype)";
        case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED: no kernel for this combination";
        case LA_ERR_CUDA: return "LA_ERR_CUDA: CUDA runtime error";
        case LA_ERR_TIMEOUT: return "LA_ERR_TIMEOUT: a kernel's bounded wait ran out";
    }
    return "unknown la_status_t";
}

extern "C" int la_version(void) { return 100; }

extern "C" unsigned long long la_kernel_launches(void) {
    return g_launches.load(std::memory_order_relaxed);
}

extern "C" size_t la_prefill_conv_workspace_size(int B, int H, int T) {
    if (B < 1 || H < 1 || T < 1 || (long long)B * H > INT32_MAX) return 0;
    return prefill_gdn_workspace_bytes(B * H, T);
}

extern "C" la_status_t la_prefill_conv(la_dtype_t dtype, int B, int H, int T, int d, int width,
                                       const void *xq, const void *xk, const void *xv, const float *wq,
                                       const float *wk, const float *wv, const void *window_in,
                                       void *window_out, unsigned flags_qk, unsigned flags_v, void *y,
                                       const float *gate, const float *beta, float *state, void *o,
                                       unsigned flags, void *workspace, size_t workspace_bytes,
                                       void *stream) {
    timer_reset();
    if (dtype != LA_BF16) return dtype == LA_F32 ? LA_ERR_UNSUPPORTED : LA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 1 || width < 1 || width > 4) return LA_ERR_INVALID_ARG;
    if (d != 128) return d == 64 ? LA_ERR_UNSUPPORTED : LA_ERR_INVALID_ARG;
    if ((flags & ~LA_FLAG_INIT_STATE) || ((flags_qk | flags_v) & ~(LA_CONV_SILU | LA_CONV_L2NORM)))
        return LA_ERR_INVALID_ARG;
    const long long BH = (long long)B * H;
    if (BH > INT32_MAX || BH * T * d > kMaxElems) return LA_ERR_INVALID_ARG;
    const void *need16[] = {xq, xk, xv, y, o, state, workspace};
    for (const void *p : need16)
        if (!tensor_ok(p, 16)) return LA_ERR_INVALID_ARG;
    const float *need4[] = {wq, wk, wv, beta};
    for (const float *p : need4)
        if (!tensor_ok(p, 4)) return LA_ERR_INVALID_ARG;
    if (gate && !tensor_ok(gate, 4)) return LA_ERR_INVALID_ARG;
    if (width > 1) {
        if (window_in && !tensor_ok(window_in, 16)) return LA_ERR_INVALID_ARG;
        if (window_out && !tensor_ok(window_out, 16)) return LA_ERR_INVALID_ARG;
    }
    if (workspace_bytes < la_prefill_conv_workspace_size(B, H, T)) return LA_ERR_INVALID_ARG;
    const size_t th = (size_t)BH * T, xb = th * d * 2, win = (size_t)3 * B * (width - 1) * H * d * 2;
    const size_t wb = sizeof(float) * (size_t)H * d * width;
    if (!writes_disjoint({{y, 3 * xb}, {o, xb}, {state, sizeof(float) * BH * d * d},
                          {width > 1 ? window_out : nullptr, win}, {workspace, workspace_bytes}},
                         {{xq, xb}, {xk, xb}, {xv, xb}, {wq, wb}, {wk, wb}, {wv, wb},
                          {width > 1 ? window_in : nullptr, win}, {gate, sizeof(float) * th},
                          {beta, sizeof(float) * th}}))
        return LA_ERR_INVALID_ARG;
    PrefillArgs a;
    a.mode = LA_MODE_GATED_DELTA;
    a.dtype = LA_BF16;
    a.B = B; a.H = H; a.T = T; a.dk = d; a.dv = d;
    const __nv_bfloat16 *yb = static_cast<const __nv_bfloat16 *>(y);
    a.q = yb;
    a.k = yb + th * d;
    a.v = yb + 2 * th * d;
    a.gate = gate;
    a.beta = beta;
    a.state = state;
    a.z = nullptr;
    a.o = o;
    a.chunk = 64;
    a.init_state = (flags & LA_FLAG_INIT_STATE) != 0;
    a.stream = static_cast<cudaStream_t>(stream);
    ConvSpec cs;
    cs.x[0] = xq; cs.x[1] = xk; cs.x[2] = xv;
    cs.w[0] = wq; cs.w[1] = wk; cs.w[2] = wv;
    cs.win_in = width > 1 ? window_in : nullptr;
    cs.win_out = width > 1 ? window_out : nullptr;
    cs.y = y;
    cs.width = width;
    cs.fqk = flags_qk;
    cs.fv = flags_v;
    return from_cuda(launch_prefill_gdn_conv(a, cs, workspace, workspace_bytes));
}

// ---------------------------------------------------------------- gated linear recurrence

namespace {

// Checks shared by the dense forms: dtype, flags, sizes.
bool scan_sizes_ok(int dtype, int B, int T, int C, unsigned flags, unsigned allowed) {
    if (dtype != LA_F32 && dtype != LA_BF16) return false;
    if (flags & ~allowed) return false;
    return B >= 1 && T >= 0 && C >= 1 && (long long)B * C <= kMaxElems && (long long)B * T <= kMaxElems / C;
}
// Element alignment is enough: the kernels take narrower vectors where a tensor's start asks for it.
bool scan_io_ok(int dtype, const void *p) { return tensor_ok(p, dtype == LA_BF16 ? 2 : 4); }
size_t checkpoint_bytes(int B, int T, int C) {
    return sizeof(float) * (size_t)B * (((size_t)T + kScanCheckpoint - 1) / kScanCheckpoint) * C;
}

}  // namespace

extern "C" la_status_t la_linear_scan(la_dtype_t dtype, int B, int T, int C, const void *x, const float *gate,
                                      float *state, void *h, float *checkpoints, unsigned flags, void *stream) {
    timer_reset();
    if (!scan_sizes_ok(dtype, B, T, C, flags, LA_FLAG_INIT_STATE | LA_SCAN_BLEND)) return LA_ERR_INVALID_ARG;
    if (!tensor_ok(state, 4)) return LA_ERR_INVALID_ARG;
    const bool init = (flags & LA_FLAG_INIT_STATE) != 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t sb = sizeof(float) * (size_t)B * C;
    if (T == 0) return init ? LA_OK : from_cuda(cudaMemsetAsync(state, 0, sb, st));
    if (!scan_io_ok(dtype, x) || !tensor_ok(gate, 4) || !scan_io_ok(dtype, h) ||
        (checkpoints && !tensor_ok(checkpoints, 4)))
        return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)B * T * C, io = n * (dtype == LA_BF16 ? 2 : 4);
    if (!writes_disjoint({{h, io}, {state, sb}, {checkpoints, checkpoint_bytes(B, T, C)}},
                         {{x, io}, {gate, sizeof(float) * n}}))
        return LA_ERR_INVALID_ARG;
    ScanArgs a;
    a.dtype = dtype;
    a.B = B; a.T = T; a.C = C;
    a.x = x; a.gate = gate;
    a.state_in = init ? state : nullptr;
    a.state_out = state;
    a.h = h;
    a.ckpt = checkpoints;
    a.blend = (flags & LA_SCAN_BLEND) != 0;
    a.stream = st;
    return from_cuda(launch_scan(a));
}

extern "C" size_t la_linear_scan_varlen_workspace_size(int T) { return T < 1 ? 0 : scan_codes_bytes(T); }

extern "C" la_status_t la_linear_scan_varlen(la_dtype_t dtype, int N, int T, int C, const int *cu_seqlens,
                                             const void *x, const float *gate, float *state, void *h,
                                             unsigned flags, void *workspace, size_t workspace_bytes, void *stream) {
    timer_reset();
    // a row's sequence number shares a 32-bit code with two flags; the codes are padded rows
    if (N < 1 || N >= (1 << 29) || T > INT32_MAX - 512) return LA_ERR_INVALID_ARG;
    if (!scan_sizes_ok(dtype, 1, T, C, flags, LA_FLAG_INIT_STATE | LA_SCAN_BLEND) || (long long)N > kMaxElems / C)
        return LA_ERR_INVALID_ARG;
    if (!tensor_ok(cu_seqlens, 4) || !tensor_ok(state, 4)) return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)T * C, io = n * (dtype == LA_BF16 ? 2 : 4);
    if (T > 0) {
        if (!scan_io_ok(dtype, x) || !tensor_ok(gate, 4) || !scan_io_ok(dtype, h) || !tensor_ok(workspace, 16) ||
            workspace_bytes < la_linear_scan_varlen_workspace_size(T))
            return LA_ERR_INVALID_ARG;
    }
    if (!writes_disjoint({{T > 0 ? h : nullptr, io}, {state, sizeof(float) * (size_t)N * C},
                          {T > 0 ? workspace : nullptr, workspace_bytes}},
                         {{cu_seqlens, sizeof(int) * ((size_t)N + 1)}, {T > 0 ? x : nullptr, io},
                          {T > 0 ? gate : nullptr, sizeof(float) * n}}))
        return LA_ERR_INVALID_ARG;
    const bool init = (flags & LA_FLAG_INIT_STATE) != 0;
    ScanArgs a;
    a.dtype = dtype;
    a.B = 1; a.T = T; a.C = C;
    a.x = x; a.gate = gate;
    a.state_in = init ? state : nullptr;
    a.state_out = state;
    a.h = h;
    a.ckpt = nullptr;
    a.blend = (flags & LA_SCAN_BLEND) != 0;
    a.stream = static_cast<cudaStream_t>(stream);
    int *codes = static_cast<int *>(workspace);
    cudaError_t e = launch_scan_rows(a, cu_seqlens, N, codes, init ? nullptr : state);
    if (e != cudaSuccess || T == 0) return from_cuda(e);
    a.codes = codes;
    return from_cuda(launch_scan(a));
}

extern "C" la_status_t la_linear_scan_step(la_dtype_t dtype, int N, int C, const void *x, const float *gate,
                                           float *state, void *h, unsigned flags, void *stream) {
    timer_reset();
    if (!scan_sizes_ok(dtype, N, 1, C, flags, LA_SCAN_BLEND)) return LA_ERR_INVALID_ARG;
    if (!scan_io_ok(dtype, x) || !tensor_ok(gate, 4) || !tensor_ok(state, 4) || !scan_io_ok(dtype, h))
        return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)N * C, io = n * (dtype == LA_BF16 ? 2 : 4);
    if (!writes_disjoint({{h, io}, {state, sizeof(float) * n}}, {{x, io}, {gate, sizeof(float) * n}}))
        return LA_ERR_INVALID_ARG;
    ScanArgs a;
    a.dtype = dtype;
    a.B = N; a.T = 1; a.C = C;
    a.x = x; a.gate = gate;
    a.state_in = a.state_out = state;
    a.h = h;
    a.ckpt = nullptr;
    a.blend = (flags & LA_SCAN_BLEND) != 0;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(launch_scan_step(a));
}

extern "C" size_t la_linear_scan_backward_workspace_size(int B, int T, int C) {
    return B < 1 || T < 1 || C < 1 ? 0 : checkpoint_bytes(B, T, C);
}

extern "C" la_status_t la_linear_scan_backward(la_dtype_t dtype, int B, int T, int C, const void *x,
                                               const float *gate, const float *state0,
                                               const float *checkpoints, const void *dh, const float *dstate,
                                               void *dx, float *dgate, float *dstate0, unsigned flags,
                                               void *workspace, size_t workspace_bytes, void *stream) {
    timer_reset();
    if (!scan_sizes_ok(dtype, B, T, C, flags, LA_SCAN_BLEND) || T < 1) return LA_ERR_INVALID_ARG;
    const void *need[] = {x, dh, dx};
    for (const void *q : need)
        if (!scan_io_ok(dtype, q)) return LA_ERR_INVALID_ARG;
    if (!tensor_ok(gate, 4) || !(checkpoints ? tensor_ok(checkpoints, 4) : tensor_ok(workspace, 16)))
        return LA_ERR_INVALID_ARG;
    const float *may[] = {checkpoints ? nullptr : state0, dstate, dgate, dstate0};
    for (const float *q : may)
        if (q && !tensor_ok(q, 4)) return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)B * T * C, io = n * (dtype == LA_BF16 ? 2 : 4), sb = sizeof(float) * (size_t)B * C;
    const size_t kb = checkpoint_bytes(B, T, C);
    if (!checkpoints && workspace_bytes < kb) return LA_ERR_INVALID_ARG;
    if (!writes_disjoint({{dx, io}, {dgate, sizeof(float) * n}, {dstate0, sb},
                          {checkpoints ? nullptr : workspace, workspace_bytes}},
                         {{x, io}, {gate, sizeof(float) * n}, {dh, io}, {dstate, sb}, {checkpoints, kb},
                          {checkpoints ? nullptr : state0, sb}}))
        return LA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool blend = (flags & LA_SCAN_BLEND) != 0;
    if (!checkpoints) {   // the forward walk once more, for the kept states alone
        ScanArgs f;
        f.dtype = dtype;
        f.B = B; f.T = T; f.C = C;
        f.x = x; f.gate = gate;
        f.state_in = state0;
        f.state_out = nullptr;
        f.h = nullptr;
        f.ckpt = static_cast<float *>(workspace);
        f.blend = blend;
        f.stream = st;
        const cudaError_t e = launch_scan(f);
        if (e != cudaSuccess) return from_cuda(e);
        checkpoints = f.ckpt;
    }
    ScanBackwardArgs a;
    a.dtype = dtype;
    a.B = B; a.T = T; a.C = C;
    a.x = x; a.dh = dh;
    a.gate = gate; a.ckpt = checkpoints; a.dstate = dstate;
    a.dx = dx; a.dgate = dgate; a.dstate0 = dstate0;
    a.blend = blend;
    a.stream = st;
    return from_cuda(launch_scan_backward(a));
}

// ---------------------------------------------------------------- rotary positions

extern "C" la_status_t la_rotary(la_dtype_t dtype, int B, int T, int H_q, int H_k, int d, int rotary_dim,
                                 const void *q, const void *k, const double *freqs, const int *positions,
                                 int start, float scale, void *y_q, void *y_k, unsigned flags, void *stream) {
    timer_reset();
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (flags & ~(LA_ROT_INTERLEAVED | LA_ROT_TRANSPOSE | LA_ROT_X_TOKENS | LA_ROT_Y_TOKENS)) return LA_ERR_INVALID_ARG;
    if (B < 1 || T < 0 || H_q < 1 || H_k < 0 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > d)
        return LA_ERR_INVALID_ARG;
    if (d > 512) return LA_ERR_UNSUPPORTED;
    const long long most = H_q > H_k ? H_q : H_k;
    if ((long long)B * T > kMaxElems / (most * d)) return LA_ERR_INVALID_ARG;
    if (T == 0) return LA_OK;
    if (!tensor_ok(freqs, 8) || (positions && !tensor_ok(positions, 4))) return LA_ERR_INVALID_ARG;
    if (!tensor_ok(q, 16) || !tensor_ok(y_q, 16)) return LA_ERR_INVALID_ARG;
    if (H_k && (!tensor_ok(k, 16) || !tensor_ok(y_k, 16))) return LA_ERR_INVALID_ARG;
    if (!H_k) k = y_k = nullptr;
    const bool xt = (flags & LA_ROT_X_TOKENS) != 0, yt = (flags & LA_ROT_Y_TOKENS) != 0;
    const size_t row = (size_t)B * T * d * (dtype == LA_BF16 ? 2 : 4), qb = row * H_q, kb = row * H_k;
    // in place (each value is read and written by one thread) where the layouts agree
    const void *rq = (y_q == q && xt == yt) ? nullptr : q, *rk = (y_k == k && xt == yt) ? nullptr : k;
    if (!writes_disjoint({{y_q, qb}, {y_k, kb}},
                         {{rq, qb}, {rk, kb}, {freqs, sizeof(double) * (rotary_dim / 2)},
                          {positions, sizeof(int) * (size_t)B * T}}))
        return LA_ERR_INVALID_ARG;
    RotaryArgs a;
    a.dtype = dtype;
    a.B = B; a.T = T; a.Hq = H_q; a.Hk = H_k; a.d = d; a.r = rotary_dim;
    a.q = q; a.k = k; a.yq = y_q; a.yk = y_k;
    a.freqs = freqs;
    a.positions = positions;
    a.start = start;
    a.scale = scale;
    a.interleaved = (flags & LA_ROT_INTERLEAVED) != 0;
    a.transpose = (flags & LA_ROT_TRANSPOSE) != 0;
    a.x_tokens = xt;
    a.y_tokens = yt;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(launch_rotary(a));
}

// ---------------------------------------------------------------- RMS norm

namespace {

constexpr int kMaxNormColumns = 16384;

la_status_t norm_sizes(int dtype, int B, int H, int T, int C, float eps) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 0 || C < 1 || !(eps >= 0.f)) return LA_ERR_INVALID_ARG;
    if (C > kMaxNormColumns) return LA_ERR_UNSUPPORTED;
    if ((long long)B * H > kMaxElems / C || (T > 0 && (long long)B * H * C > kMaxElems / T)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

}  // namespace

extern "C" la_status_t la_rms_norm(la_dtype_t dtype, int B, int H, int T, int C, const void *x,
                                   const void *residual, const float *w, float eps, void *residual_out, void *y,
                                   float *scales, int group, unsigned flags, void *stream) {
    timer_reset();
    if (flags & ~LA_NORM_FP8) return LA_ERR_INVALID_ARG;
    const la_status_t sized = norm_sizes(dtype, B, H, T, C, eps);
    if (sized != LA_OK) return sized;
    const bool fp8 = (flags & LA_NORM_FP8) != 0;
    if (group != 0 && (!fp8 || group != 128 || C % 128)) return LA_ERR_INVALID_ARG;
    if (residual && H != 1) return LA_ERR_INVALID_ARG;
    if (T == 0) return LA_OK;
    if (!tensor_ok(x, 16) || !tensor_ok(w, 16) || !tensor_ok(y, 16) || (fp8 && !tensor_ok(scales, 4)))
        return LA_ERR_INVALID_ARG;
    if (residual && (!tensor_ok(residual, 16) || !tensor_ok(residual_out, 16))) return LA_ERR_INVALID_ARG;
    if (!residual) residual_out = nullptr;
    if (!fp8) scales = nullptr;
    const size_t es = dtype == LA_BF16 ? 2 : 4, rows = (size_t)B * H * T, xb = rows * C * es;
    // the stream may be updated in place: a thread stores what it alone has read
    const void *rx = residual_out == x ? nullptr : x, *rr = residual_out == residual ? nullptr : residual;
    if (!writes_disjoint({{y, rows * C * (fp8 ? 1 : es)}, {residual_out, xb},
                          {scales, sizeof(float) * rows * (group ? C / group : 1)}},
                         {{rx, xb}, {rr, xb}, {w, sizeof(float) * (size_t)C}}))
        return LA_ERR_INVALID_ARG;
    NormArgs a;
    a.dtype = dtype;
    a.B = B; a.H = H; a.T = T; a.C = C;
    a.x = x; a.residual = residual; a.w = w;
    a.h = residual_out; a.y = y; a.scales = scales;
    a.fp8 = fp8;
    a.group = group;
    a.eps = eps;
    a.stream = static_cast<cudaStream_t>(stream);
    return from_cuda(launch_norm(a));
}

extern "C" size_t la_rms_norm_backward_workspace_size(int B, int H, int T, int C) {
    if (norm_sizes(LA_F32, B, H, T, C, 0.f) != LA_OK || T == 0) return 0;
    return norm_backward_partial_bytes((long long)B * H * T, C);
}

extern "C" la_status_t la_rms_norm_backward(la_dtype_t dtype, int B, int H, int T, int C, const void *h,
                                            const float *w, float eps, const void *dy, const void *dresidual,
                                            void *dx, float *dw, void *workspace, size_t workspace_bytes,
                                            void *stream) {
    timer_reset();
    const la_status_t sized = norm_sizes(dtype, B, H, T, C, eps);
    if (sized != LA_OK) return sized;
    if (!tensor_ok(dw, 16)) return LA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return from_cuda(cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)C, st));
    const void *need[] = {h, w, dy, dx, workspace};
    for (const void *q : need)
        if (!tensor_ok(q, 16)) return LA_ERR_INVALID_ARG;
    if (dresidual && !tensor_ok(dresidual, 16)) return LA_ERR_INVALID_ARG;
    if (workspace_bytes < la_rms_norm_backward_workspace_size(B, H, T, C)) return LA_ERR_INVALID_ARG;
    const size_t xb = (size_t)B * H * T * C * (dtype == LA_BF16 ? 2 : 4), wb = sizeof(float) * (size_t)C;
    if (!writes_disjoint({{dx, xb}, {dw, wb}, {workspace, workspace_bytes}},
                         {{h, xb}, {w, wb}, {dy, xb}, {dresidual, xb}}))
        return LA_ERR_INVALID_ARG;
    NormBackwardArgs a;
    a.dtype = dtype;
    a.B = B; a.H = H; a.T = T; a.C = C;
    a.h = h; a.dy = dy; a.dres = dresidual; a.w = w;
    a.dx = dx; a.dw = dw;
    a.partial = static_cast<float *>(workspace);
    a.eps = eps;
    a.stream = st;
    return from_cuda(launch_norm_backward(a));
}
