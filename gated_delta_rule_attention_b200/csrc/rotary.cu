// rotary.cu -- rotary positions of q and k (la_rotary).
//
// Constant-decay (RetNet) layers, section "Memory must forget: decay and gates", and the
// softmax layers of the hybrids, section "Hybrids of 2025: Qwen3-Next and Kimi Linear", turn
// the first r values of every head in pairs (u, v) by an angle that grows with the position:
//
//   u' = s (u cos - v sin),  v' = s (u sin + v cos),   angle = position * freqs[j], j < r / 2,
//
// with (u, v) = (x_{2j}, x_{2j+1}) (interleaved) or (x_j, x_{j + r/2}) (halves); the other
// d - r values pass through.  The gradient is the transposed rotation (sin with the other
// sign).  As in the short convolution, rows come token-major from a projection and leave
// head-major for the attention kernels (or the other way round for the gradient).
//
// The angle of a far position needs more than fp32: position * freqs / (2 pi) is formed in
// fp64 (a relative error of 2^-52, so less than 1e-6 of a turn at position 2^31), its whole
// turns are dropped, and the rest of a turn, at most 1/2, goes to sincospif.
//
// Bound by HBM: every value is read once and written once, two products a value.  A thread
// owns eight pairs (two 16-byte vectors of bf16) of one token, forms their eight angles once
// and applies them to every HS-th head of q and of k, several heads' loads in flight; the
// HS threads of a token that hold the same pairs, and then the pairs of a head, are
// neighbours, so a warp reads and writes whole 256-byte head rows.
#include "la_internal.cuh"
#include "vec.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // heads in flight

struct RotaryParams {
    const void *x[2];      // q, k
    void *y[2];
    int heads[2];
    const double *freqs;
    const int *positions;  // [B, T], or nullptr: start + t
    long long start;
    long long tokens, T;   // B * T, T
    int d, r;
    int units;             // threads of one head row
    int HS;                // threads of one token that share its heads
    float scale, sign;
    bool x_tokens, y_tokens;
};

// sin and cos of position * f.
__device__ __forceinline__ void angle(double pos, double f, float &sn, float &cs) {
    constexpr double kInvTwoPi = 0.15915494309189533577;
    double turns = pos * (f * kInvTwoPi);
    turns -= rint(turns);
    sincospif(2.f * (float)turns, &sn, &cs);
}

// Element offset of head 0 of a token, and the stride from head to head.
__device__ __forceinline__ long long row_of(bool token_major, long long b, long long t, long long T, int H, int d,
                                            long long &head_stride) {
    head_stride = token_major ? d : T * d;
    return token_major ? (b * T + t) * (long long)H * d : (b * H * T + t) * d;
}

// PAIRS pairs a thread: 8 (rows in 16-byte vectors; r a multiple of 16, d of 8), or 1.
// Units behind the rotated ones copy 2 * PAIRS values (none when in place).
template <typename IO, int PAIRS, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
    using X = Pack<IO, PAIRS>;
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
    long long rest;
    int u, hs;
    if (p.tokens * p.units * p.HS <= UINT32_MAX) {
        const unsigned i = (unsigned)idx;
        u = i % (unsigned)p.units;
        hs = i / (unsigned)p.units % (unsigned)p.HS;
        rest = i / (unsigned)p.units / (unsigned)p.HS;
    } else {
        u = (int)(idx % p.units);
        hs = (int)(idx / p.units % p.HS);
        rest = idx / p.units / p.HS;
    }
    if (rest >= p.tokens) return;
    const long long b = rest / p.T, t = rest - b * p.T;
    const int turned = p.r / (2 * PAIRS);
    const bool turn = u < turned;
    // the two vectors of the thread in a head row
    int e0, e1;
    if (turn) {
        e0 = INTERLEAVED ? u * 2 * PAIRS : u * PAIRS;
        e1 = INTERLEAVED ? e0 + PAIRS : e0 + p.r / 2;
    } else {
        e0 = p.r + (u - turned) * 2 * PAIRS;
        e1 = e0 + PAIRS;
    }
    const bool second = e1 < p.d;   // false: the last copied vector of a row stands alone
    float cs[PAIRS], sn[PAIRS];
    if (turn) {
        const double pos = (double)(p.positions ? (long long)p.positions[rest] : p.start + t);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            angle(pos, p.freqs[u * PAIRS + j], sn[j], cs[j]);
            cs[j] *= p.scale;
            sn[j] *= p.scale * p.sign;
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int H = p.heads[which];
        if (H == 0) continue;
        long long xh, yh;
        const IO *x = static_cast<const IO *>(p.x[which]) + row_of(p.x_tokens, b, t, p.T, H, p.d, xh);
        IO *y = static_cast<IO *>(p.y[which]) + row_of(p.y_tokens, b, t, p.T, H, p.d, yh);
        for (int h0 = hs; h0 < H; h0 += kUnroll * p.HS) {
            X v0[kUnroll], v1[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int h = h0 + i * p.HS;
                if (h < H) {
                    v0[i] = load_pack<IO, PAIRS>(x + h * xh + e0);
                    if (second) v1[i] = load_pack<IO, PAIRS>(x + h * xh + e1);
                }
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int h = h0 + i * p.HS;
                if (h >= H) break;
                if (turn) {
#pragma unroll
                    for (int j = 0; j < PAIRS; ++j) {
                        // interleaved pairs lie next to each other across the two vectors
                        IO &a = INTERLEAVED ? (2 * j < PAIRS ? v0[i].v[(2 * j) % PAIRS] : v1[i].v[(2 * j) % PAIRS])
                                            : v0[i].v[j];
                        IO &c = INTERLEAVED ? (2 * j + 1 < PAIRS ? v0[i].v[(2 * j + 1) % PAIRS]
                                                                 : v1[i].v[(2 * j + 1) % PAIRS])
                                            : v1[i].v[j];
                        const float fa = to_f32(a), fc = to_f32(c);
                        a = from_f32<IO>(fa * cs[j] - fc * sn[j]);
                        c = from_f32<IO>(fa * sn[j] + fc * cs[j]);
                    }
                }
                store_pack<IO, PAIRS>(y + h * yh + e0, v0[i]);
                if (second) store_pack<IO, PAIRS>(y + h * yh + e1, v1[i]);
            }
        }
    }
}

template <typename IO, int PAIRS>
cudaError_t launch_pairs(const RotaryArgs &a) {
    RotaryParams p;
    p.x[0] = a.q; p.x[1] = a.k;
    p.y[0] = a.yq; p.y[1] = a.yk;
    p.heads[0] = a.Hq; p.heads[1] = a.Hk;
    p.freqs = a.freqs;
    p.positions = a.positions;
    p.start = a.start;
    p.T = a.T;
    p.tokens = (long long)a.B * a.T;
    p.d = a.d;
    p.r = a.r;
    p.scale = a.scale;
    p.sign = a.transpose ? -1.f : 1.f;
    p.x_tokens = a.x_tokens;
    p.y_tokens = a.y_tokens;
    const bool in_place = a.yq == a.q && (a.Hk == 0 || a.yk == a.k);
    p.units = a.r / (2 * PAIRS) + (in_place ? 0 : (a.d - a.r + 2 * PAIRS - 1) / (2 * PAIRS));
    // Four threads a token share its heads; more of them where the tokens alone would leave the
    // SMs with less than a few warps each (decoding).
    const int most = a.Hq > a.Hk ? a.Hq : a.Hk;
    p.HS = most < 4 ? most : 4;
    while (p.HS < most && p.tokens * p.units * p.HS < 148ll * 512) p.HS = 2 * p.HS < most ? 2 * p.HS : most;
    const long long blocks = (p.tokens * p.units * p.HS + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    timer_begin(a.stream);
    if (a.interleaved) rotary_kernel<IO, PAIRS, true><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p);
    else rotary_kernel<IO, PAIRS, false><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p);
    timer_end(a.stream);
    note_launches(1);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_io(const RotaryArgs &a) {
    return a.r % 16 == 0 && a.d % 8 == 0 ? launch_pairs<IO, 8>(a) : launch_pairs<IO, 1>(a);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a) {
    return a.dtype == LA_BF16 ? launch_io<__nv_bfloat16>(a) : launch_io<float>(a);
}

}  // namespace la
