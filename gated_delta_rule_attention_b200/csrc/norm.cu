// norm.cu -- the root-mean-square norm with the residual's addition (la_rms_norm), an output in
// 8 bits with scales, and its gradients (la_rms_norm_backward).
//
// Section "Memory must forget: decay and gates": modern variants drop the denominator and
// normalise after the attention (rows of d, head-major in, token-major out for the output
// projection); the same norm stands in front of a layer's projections, where the residual
// stream takes in the last layer's output.  For a row of C values,
//
//   h = x + residual (rounded to the stream's type, as it is stored; without residual h = x),
//   y = h rstd w,   rstd = 1 / sqrt(mean h^2 + eps),
//
// and with 8-bit output q = y / scale in e4m3, scale = max |y| / 448 over the row or over each
// 128 columns.  Backwards, with n = h rstd and p = dy w,
//
//   dx = rstd (p - n mean(p n)) (+ the stored stream's own gradient),   dw = sum_rows dy n.
//
// The norm takes the rounded h, so that the gradient, which has only the stored stream, belongs
// to exactly the y that was computed.
//
// Bound by HBM: a row is read once into registers (as stored, widened where used), its one or
// two sums go through the threads of the row (shuffles within a warp or a part of one, shared
// memory for a row of a whole CTA), and it is written once.  Threads of a row: C / 8 up to a
// warp, then up to eight vectors a lane, then a CTA a row; rows are taken in a loop, so the
// weights stay in L1.  dw: every thread keeps its columns' sums over its CTA's rows in
// registers, each CTA writes one row of partial sums, and a second kernel adds those in a fixed
// order.
#include "la_internal.cuh"
#include "vec.cuh"

#include <cuda_fp8.h>

namespace la {
namespace {

constexpr float kFp8Max = 448.f;   // largest e4m3 value
constexpr int kMaxPartials = 148 * 4;

struct NormParams {
    const void *x, *residual;
    const float *w;
    void *h;          // the stored stream, with a residual
    void *y;          // I/O dtype, or e4m3 bytes
    float *scales;    // [rows, C / group]
    long long rows;   // B * H * T
    int H, T, C;
    int group;        // 8-bit output: columns a scale
    float eps, inv_c;
};

struct NormBackwardParams {
    const void *h, *dy, *dres;
    const float *w;
    void *dx;
    float *partial;   // [blocks, C]
    long long rows;
    int H, T, C;
    float eps, inv_c;
};

// Row of y for row i of x: (b, head, t) -> (b, t, head).
__device__ __forceinline__ long long out_row(long long i, int H, int T) {
    if (H == 1) return i;
    const long long bh = i / T, t = i - bh * T, b = bh / H;
    return (b * T + t) * H + (bh - b * H);
}

// Sum and maximum over the NT threads of a row, the same in each of them.  NT > 32: one row a
// CTA; `box` is one of two alternating areas, so a row's reads never meet the next row's writes.
template <int NT>
__device__ __forceinline__ float2 row_sum(float2 v, float2 *box) {
#pragma unroll
    for (int off = (NT < 32 ? NT : 32) / 2; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(~0u, v.x, off);
        v.y += __shfl_xor_sync(~0u, v.y, off);
    }
    if (NT > 32) {
        if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) v.x += box[i].x, v.y += box[i].y;
    }
    return v;
}
template <int NT>
__device__ __forceinline__ float2 row_sum_max(float2 v, float2 *box) {   // x summed, y's maximum
#pragma unroll
    for (int off = (NT < 32 ? NT : 32) / 2; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(~0u, v.x, off);
        v.y = fmaxf(v.y, __shfl_xor_sync(~0u, v.y, off));
    }
    if (NT > 32) {
        if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) v.x += box[i].x, v.y = fmaxf(v.y, box[i].y);
    }
    return v;
}

// Scale of a group whose largest |y| is `top`: 1 for zeros, and never so small that its
// reciprocal overflows.
__device__ __forceinline__ float fp8_scale(float top) {
    return top > 0.f ? fmaxf(top / kFp8Max, 1.17549435e-38f) : 1.f;
}

template <int V>
__device__ __forceinline__ void store_fp8(unsigned char *p, const float (&y)[V], float inv) {
    if constexpr (V == 1) {
        p[0] = __nv_cvt_float_to_fp8(y[0] * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j] * inv, y[4 * j + 1] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j + 2] * inv, y[4 * j + 3] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[j] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// V values a vector, K vectors a thread, NT threads a row, ROWS rows in flight a thread.
// GROUPS: 8-bit output with a scale for each p.group columns (128: 16 neighbouring lanes);
// otherwise with FP8 a scale a row.
template <typename IO, int V, int K, int NT, int ROWS, bool RES, bool FP8, bool GROUPS>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_kernel(const NormParams p) {
    constexpr int kBlock = NT < 256 ? 256 : NT;
    constexpr int kRowsBlock = NT <= 32 ? kBlock / NT : 1;
    static_assert(NT <= 32 || NT == kBlock, "a row has part of a warp, a warp or a CTA");
    using X = Pack<IO, V>;
    __shared__ float2 box[2][NT > 32 ? NT / 32 : 1];
    const int t = threadIdx.x % NT;
    const long long stride = (long long)gridDim.x * kRowsBlock * ROWS;
    const int C = p.C;
    int turn = 0;
    // the loop runs by whole blocks: threads without a row take part in the shuffles
    for (long long base = (long long)blockIdx.x * kRowsBlock * ROWS; base < p.rows; base += stride) {
        X x[ROWS][K], r[RES ? ROWS : 1][RES ? K : 1];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const long long i = base + q * kRowsBlock + threadIdx.x / NT;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + t) * V;
                if (i < p.rows && c < C) {
                    x[q][k] = load_pack<IO, V>(static_cast<const IO *>(p.x) + i * C + c);
                    if (RES) r[RES ? q : 0][RES ? k : 0] = load_pack<IO, V>(static_cast<const IO *>(p.residual) + i * C + c);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        x[q][k].v[j] = from_f32<IO>(0.f);
                        if (RES) r[RES ? q : 0][RES ? k : 0].v[j] = from_f32<IO>(0.f);
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const long long i = base + q * kRowsBlock + threadIdx.x / NT;
            const bool live = i < p.rows;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + t) * V;
                if (RES) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        x[q][k].v[j] = from_f32<IO>(to_f32(x[q][k].v[j]) + to_f32(r[RES ? q : 0][RES ? k : 0].v[j]));
                    if (live && c < C) store_pack<IO, V>(static_cast<IO *>(p.h) + i * C + c, x[q][k]);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float f = to_f32(x[q][k].v[j]);
                    sum.x = fmaf(f, f, sum.x);
                    if (FP8 && !GROUPS && c < C) sum.y = fmaxf(sum.y, fabsf(f * p.w[c + j]));
                }
            }
            sum = FP8 && !GROUPS ? row_sum_max<NT>(sum, box[turn]) : row_sum<NT>(sum, box[turn]);
            turn ^= 1;
            const float rstd = rsqrtf(fmaf(sum.x, p.inv_c, p.eps));
            const long long o = out_row(live ? i : 0, p.H, p.T) * C;
            float inv = 1.f;
            if (FP8 && !GROUPS) {
                const float scale = fp8_scale(sum.y * rstd);
                inv = 1.f / scale;
                if (live && t == 0) p.scales[o / C] = scale;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + t) * V;
                float y[V];
                float top = 0.f;
                if (c < C) {
                    const Pack<float, V> w = load_pack<float, V>(p.w + c);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        y[j] = to_f32(x[q][k].v[j]) * rstd * w.v[j];
                        top = fmaxf(top, fabsf(y[j]));
                    }
                }
                if (FP8 && GROUPS) {
#pragma unroll
                    for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, off));
                    const float scale = fp8_scale(top);
                    inv = 1.f / scale;
                    if (live && c < C && (threadIdx.x & 15) == 0) p.scales[(o + c) / 128] = scale;
                }
                if (live && c < C) {
                    if constexpr (FP8) {
                        store_fp8<V>(static_cast<unsigned char *>(p.y) + o + c, y, inv);
                    } else {
                        X out;
#pragma unroll
                        for (int j = 0; j < V; ++j) out.v[j] = from_f32<IO>(y[j]);
                        store_pack<IO, V>(static_cast<IO *>(p.y) + o + c, out);
                    }
                }
            }
        }
    }
}

template <typename IO, int V, int K, int NT, int ROWS, bool DRES>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_backward_kernel(const NormBackwardParams p) {
    constexpr int kBlock = NT < 256 ? 256 : NT;
    constexpr int kRowsBlock = NT <= 32 ? kBlock / NT : 1;
    static_assert(NT <= 32 || NT == kBlock, "a row has part of a warp, a warp or a CTA");
    using X = Pack<IO, V>;
    __shared__ float2 box[2][NT > 32 ? NT / 32 : 1];
    __shared__ float fold[NT <= 32 ? kBlock * K * V : 1];
    const int t = threadIdx.x % NT;
    const long long stride = (long long)gridDim.x * kRowsBlock * ROWS;
    const int C = p.C;
    float dw[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][j] = 0.f;
    int turn = 0;
    for (long long base = (long long)blockIdx.x * kRowsBlock * ROWS; base < p.rows; base += stride) {
        X x[ROWS][K], g[ROWS][K], r[DRES ? ROWS : 1][DRES ? K : 1];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const long long i = base + q * kRowsBlock + threadIdx.x / NT;
            const long long o = i < p.rows ? out_row(i, p.H, p.T) * C : 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + t) * V;
                if (i < p.rows && c < C) {
                    x[q][k] = load_pack<IO, V>(static_cast<const IO *>(p.h) + i * C + c);
                    g[q][k] = load_pack<IO, V>(static_cast<const IO *>(p.dy) + o + c);
                    if (DRES) r[DRES ? q : 0][DRES ? k : 0] = load_pack<IO, V>(static_cast<const IO *>(p.dres) + i * C + c);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) x[q][k].v[j] = g[q][k].v[j] = from_f32<IO>(0.f);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const long long i = base + q * kRowsBlock + threadIdx.x / NT;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + t) * V;
                if (c < C) {
                    const Pack<float, V> w = load_pack<float, V>(p.w + c);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float f = to_f32(x[q][k].v[j]);
                        sum.x = fmaf(f, f, sum.x);
                        sum.y = fmaf(to_f32(g[q][k].v[j]) * w.v[j], f, sum.y);
                    }
                }
            }
            sum = row_sum<NT>(sum, box[turn]);
            turn ^= 1;
            const float rstd = rsqrtf(fmaf(sum.x, p.inv_c, p.eps));
            const float mean = sum.y * rstd * p.inv_c;   // mean(p n)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + t) * V;
                if (i < p.rows && c < C) {
                    const Pack<float, V> w = load_pack<float, V>(p.w + c);
                    X out;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float n = to_f32(x[q][k].v[j]) * rstd, d = to_f32(g[q][k].v[j]);
                        dw[k][j] = fmaf(d, n, dw[k][j]);
                        float v = rstd * (d * w.v[j] - n * mean);
                        if (DRES) v += to_f32(r[DRES ? q : 0][DRES ? k : 0].v[j]);
                        out.v[j] = from_f32<IO>(v);
                    }
                    store_pack<IO, V>(static_cast<IO *>(p.dx) + i * C + c, out);
                }
            }
        }
    }
    // the CTA's row of partial sums
    float *partial = p.partial + (long long)blockIdx.x * C;
    if constexpr (NT <= 32) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) fold[(threadIdx.x / NT) * (K * NT * V) + (k * NT + t) * V + j] = dw[k][j];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += kBlock) {
            float s = 0.f;
            for (int q = 0; q < kRowsBlock; ++q) s += fold[q * (K * NT * V) + c];
            partial[c] = s;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * NT + t) * V;
            if (c < C) {
                Pack<float, V> s;
#pragma unroll
                for (int j = 0; j < V; ++j) s.v[j] = dw[k][j];
                store_pack<float, V>(partial + c, s);
            }
        }
    }
}

// dw = the sum of the CTAs' partial rows: 8 columns a CTA, 32 threads a column.
__global__ void __launch_bounds__(256) norm_weight_kernel(int blocks, int C, const float *__restrict__ partial,
                                                         float *__restrict__ dw) {
    __shared__ float box[32][9];
    const int c = blockIdx.x * 8 + threadIdx.x % 8, q = threadIdx.x / 8;
    float s = 0.f;
    if (c < C)
        for (int i = q; i < blocks; i += 32) s += partial[(long long)i * C + c];
    box[q][threadIdx.x % 8] = s;
    __syncthreads();
    if (threadIdx.x < 8 && blockIdx.x * 8 + threadIdx.x < C) {
        float total = 0.f;
        for (int i = 0; i < 32; ++i) total += box[i][threadIdx.x];
        dw[blockIdx.x * 8 + threadIdx.x] = total;
    }
}

// ------------------------------------------------------------------------------- host side

// Blocks for `rows` rows: all at once up to what the SMs hold, then in a loop.
template <typename F>
unsigned loop_blocks(F kernel, int threads, long long rows, int rows_block) {
    int per_sm = 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0) != cudaSuccess) {
        (void)cudaGetLastError();
        per_sm = 1;
    }
    const long long need = (rows + rows_block - 1) / rows_block, most = 148ll * (per_sm < 1 ? 1 : per_sm);
    return (unsigned)(need < most ? need : most);
}

template <typename IO, int V, int K, int NT, int ROWS, bool RES, bool FP8, bool GROUPS>
cudaError_t launch_forward(const NormArgs &a) {
    constexpr int kBlock = NT < 256 ? 256 : NT, kRowsBlock = NT <= 32 ? kBlock / NT : 1;
    NormParams p;
    p.x = a.x; p.residual = a.residual; p.w = a.w;
    p.h = a.h; p.y = a.y; p.scales = a.scales;
    p.rows = (long long)a.B * a.H * a.T;
    p.H = a.H; p.T = a.T; p.C = a.C;
    p.group = a.group;
    p.eps = a.eps;
    p.inv_c = 1.f / (float)a.C;
    auto kernel = norm_kernel<IO, V, K, NT, ROWS, RES, FP8, GROUPS>;
    const unsigned blocks = loop_blocks(kernel, kBlock, p.rows, kRowsBlock * ROWS);
    timer_begin(a.stream);
    kernel<<<blocks, kBlock, 0, a.stream>>>(p);
    timer_end(a.stream);
    note_launches(1);
    return cudaGetLastError();
}

template <typename IO, int V, int K, int NT, int ROWS>
cudaError_t forward_kind(const NormArgs &a) {
    if (!a.fp8) {
        return a.residual ? launch_forward<IO, V, K, NT, ROWS, true, false, false>(a)
                          : launch_forward<IO, V, K, NT, ROWS, false, false, false>(a);
    }
    if constexpr (V == 8 && NT >= 16) {
        if (a.group == 128)
            return a.residual ? launch_forward<IO, V, K, NT, ROWS, true, true, true>(a)
                              : launch_forward<IO, V, K, NT, ROWS, false, true, true>(a);
    }
    return a.residual ? launch_forward<IO, V, K, NT, ROWS, true, true, false>(a)
                      : launch_forward<IO, V, K, NT, ROWS, false, true, false>(a);
}

template <typename IO>
cudaError_t forward_io(const NormArgs &a) {
    const int C = a.C;
    if (C % 8) {
        if (C <= 256) return forward_kind<IO, 1, 8, 32, 1>(a);
        if (C <= 2048) return forward_kind<IO, 1, 8, 256, 1>(a);
        return forward_kind<IO, 1, 16, 1024, 1>(a);
    }
    if (C <= 64) return forward_kind<IO, 8, 1, 8, 4>(a);
    if (C <= 128) return forward_kind<IO, 8, 1, 16, 4>(a);
    if (C <= 256) return forward_kind<IO, 8, 1, 32, 4>(a);
    if (C <= 512) return forward_kind<IO, 8, 2, 32, 2>(a);
    if (C <= 1024) return forward_kind<IO, 8, 4, 32, 1>(a);
    if (C <= 2048) return forward_kind<IO, 8, 1, 256, 1>(a);
    if (C <= 4096) return forward_kind<IO, 8, 2, 256, 1>(a);
    if (C <= 8192) return forward_kind<IO, 8, 4, 256, 1>(a);
    return forward_kind<IO, 8, 4, 512, 1>(a);
}

template <typename IO, int V, int K, int NT, int ROWS, bool DRES>
cudaError_t launch_backward(const NormBackwardArgs &a) {
    constexpr int kBlock = NT < 256 ? 256 : NT, kRowsBlock = NT <= 32 ? kBlock / NT : 1;
    NormBackwardParams p;
    p.h = a.h; p.dy = a.dy; p.dres = a.dres; p.w = a.w;
    p.dx = a.dx; p.partial = a.partial;
    p.rows = (long long)a.B * a.H * a.T;
    p.H = a.H; p.T = a.T; p.C = a.C;
    p.eps = a.eps;
    p.inv_c = 1.f / (float)a.C;
    auto kernel = norm_backward_kernel<IO, V, K, NT, ROWS, DRES>;
    unsigned blocks = loop_blocks(kernel, kBlock, p.rows, kRowsBlock * ROWS);
    if (blocks > (unsigned)kMaxPartials) blocks = kMaxPartials;
    timer_begin(a.stream);
    kernel<<<blocks, kBlock, 0, a.stream>>>(p);
    timer_end(a.stream);
    note_launches(1);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    timer_begin(a.stream);
    norm_weight_kernel<<<(unsigned)((a.C + 7) / 8), 256, 0, a.stream>>>((int)blocks, a.C, a.partial, a.dw);
    timer_end(a.stream);
    note_launches(1);
    return cudaGetLastError();
}

template <typename IO, int V, int K, int NT, int ROWS>
cudaError_t backward_kind(const NormBackwardArgs &a) {
    return a.dres ? launch_backward<IO, V, K, NT, ROWS, true>(a) : launch_backward<IO, V, K, NT, ROWS, false>(a);
}

template <typename IO>
cudaError_t backward_io(const NormBackwardArgs &a) {
    const int C = a.C;
    if (C % 8) {
        if (C <= 256) return backward_kind<IO, 1, 8, 32, 1>(a);
        if (C <= 2048) return backward_kind<IO, 1, 8, 256, 1>(a);
        return backward_kind<IO, 1, 16, 1024, 1>(a);
    }
    if (C <= 64) return backward_kind<IO, 8, 1, 8, 2>(a);
    if (C <= 128) return backward_kind<IO, 8, 1, 16, 2>(a);
    if (C <= 256) return backward_kind<IO, 8, 1, 32, 2>(a);
    if (C <= 512) return backward_kind<IO, 8, 2, 32, 1>(a);
    if (C <= 2048) return backward_kind<IO, 8, 1, 256, 1>(a);
    if (C <= 4096) return backward_kind<IO, 8, 1, 512, 1>(a);
    if (C <= 8192) return backward_kind<IO, 8, 1, 1024, 1>(a);
    return backward_kind<IO, 8, 2, 1024, 1>(a);
}

}  // namespace

size_t norm_backward_partial_bytes(long long rows, int C) {
    const long long n = rows < kMaxPartials ? rows : kMaxPartials;
    return sizeof(float) * (size_t)n * C;
}

cudaError_t launch_norm(const NormArgs &a) {
    return a.dtype == LA_BF16 ? forward_io<__nv_bfloat16>(a) : forward_io<float>(a);
}

cudaError_t launch_norm_backward(const NormBackwardArgs &a) {
    return a.dtype == LA_BF16 ? backward_io<__nv_bfloat16>(a) : backward_io<float>(a);
}

}  // namespace la
