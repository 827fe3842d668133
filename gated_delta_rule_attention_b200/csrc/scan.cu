// scan.cu -- the gated linear recurrence with a vector state (la_linear_scan*).
//
// Lesson page "Linear attention and hybrids", section "Memory must forget: decay and gates":
// the decayed memory S_t = a_t S_{t-1} + (input) with one number per channel instead of a
// matrix per head.  Per batch row and channel,
//
//   h_t = a_t h_{t-1} + u_t,     u_t = x_t, or (1 - a_t) x_t with LA_SCAN_BLEND,
//
// and backwards in time, with l_t = dL/dh_t collected from all later outputs,
//
//   l_t = dh_t + a_{t+1} l_{t+1},   dx_t = l_t (or (1 - a_t) l_t),
//   da_t = l_t h_{t-1} (or l_t (h_{t-1} - x_t)),   dh_0 = a_1 l_1.
//
// A run of rows acts on the state in front of it as h -> P h + H (P the product of its
// gates, H its own result from a zero state), and two runs join by
// (P, H) o (P', H') = (P P', P' H + H'), so the time axis is cut and joined again:
//   thread   S consecutive rows of V neighbouring channels, walked one after the other;
//   warp     the 32 / LC threads that hold the same channels join by shuffles;
//   CTA      its 8 warps join through shared memory (one thread a channel);
//   cluster  K CTAs take consecutive tiles of the same channels and exchange (P, H) through
//            distributed shared memory, one cluster barrier a step; every CTA folds all K, so
//            all of them carry the state of the step's last row into the next one.
// Once a thread knows the state in front of its rows it walks them again from it, with the
// plain recurrence, and stores.  Everything is in fp32 and in a fixed order (no atomics, no
// waiting on other clusters): results are the same bits from call to call.
//
// Bound by HBM: 8 (bf16) or 12 (fp32) bytes an element and two or three operations.  Each
// input is read once: a thread's rows arrive by cp.async in its own slots of a ring in shared
// memory, kStages tiles ahead, and stay in registers between the two walks.  The backward
// pass needs h_{t-1}: the forward pass keeps the state in front of every 32nd row
// (`checkpoints`, 1/32 of a fp32 h), from which a tile's rows are walked again on chip, so
// the backward pass too reads each input once.
#include "la_internal.cuh"
#include "ptx.cuh"
#include "tmap.cuh"
#include "vec.cuh"

#include <atomic>
#include <initializer_list>
#include <type_traits>

namespace la {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;

template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Row codes of a packed batch (one int32 a row, from scan_rows_kernel): 0 for a row of no
// sequence, else 4 (sequence + 1) + 2 (its last row) + 1 (its first row).
__device__ __forceinline__ bool row_first(int code) { return code & 1; }
__device__ __forceinline__ bool row_last(int code) { return code & 2; }
__device__ __forceinline__ long long row_seq(int code) { return (code >> 2) - 1; }

struct ScanParams {
    const void *x;
    const float *gate;
    const float *state_in;   // [B or N, C]; nullptr: zeros
    float *state_out;        // [B or N, C]; nullptr: not kept.  May be state_in.
    void *h;                 // nullptr: not kept
    float *ckpt;             // [B, ceil(T / 32), C]; nullptr: not kept
    const int *codes;        // packed: [T rounded up to 32]
    long long T, C;
    int blocks;              // channel blocks of one batch row
    int K;                   // CTAs of a cluster
    int steps;               // tiles each CTA walks
};

struct BackwardParams {
    const void *x, *dh;
    const float *gate, *ckpt, *dstate;   // dstate: nullptr for zeros
    void *dx;
    float *dgate, *dstate0;              // dstate0: nullptr: not kept
    long long T, C;
    int blocks, K, steps;
};

// Shape of a kernel: V channels a thread (one vector load), LC threads side by side, E
// elements a thread.
template <int V_, int LC_, int E_>
struct Shape {
    static constexpr int V = V_, LC = LC_, E = E_;
    static constexpr int S = E / V;                 // rows a thread
    static constexpr int CH = LC * V;               // channels a CTA
    static constexpr int G = kThreads / LC;         // row groups of a CTA
    static constexpr int TT = G * S;                // rows a tile
    static constexpr int SUB = 32 / LC;             // row groups of a warp
};

// One CTA's exchange area in dynamic shared memory, behind the ring.
template <int CH>
struct Exchange {
    // by the step's parity, so that a step's writes never meet the last one's reads:
    float2 warp[2][kWarps][CH];   // (P, H) of each warp, then those of all earlier warps
    int reset[2][kWarps];         // packed: a sequence starts in the warp's rows
    float carry[CH];              // state in front of the tile
    int slot_reset[2][kMaxCluster];
    // followed by float2 slot[2][K][CH]: (P, H) of each rank's tile
};

__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t rank, float a, float b) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t rank, int a) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(to), "r"(a) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <typename IO, typename SH, int STAGES>
constexpr size_t scan_ring_bytes() {
    return SH::V == 1 ? 0 : (size_t)STAGES * kThreads * SH::E * (sizeof(float) + sizeof(IO));
}
template <typename IO, typename SH, int STAGES>
constexpr size_t backward_ring_bytes() {
    return SH::V == 1 ? 0
                      : (size_t)STAGES * kThreads * (SH::E * (sizeof(float) + 2 * sizeof(IO)) + SH::V * sizeof(float));
}
template <typename SH>
size_t exchange_bytes(int K) {
    return sizeof(Exchange<SH::CH>) + (K > 1 ? (size_t)2 * K * SH::CH * sizeof(float2) : 0);
}

// Two CTAs an SM: the ring's bytes in flight of one cover the other's barriers.  Odd channel
// counts (V = 1) have no 4-byte aligned rows for cp.async: their rows are loaded straight into
// registers.
template <typename IO, typename SH, int STAGES, bool BLEND, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(const ScanParams p) {
    constexpr int V = SH::V, LC = SH::LC, S = SH::S, CH = SH::CH, TT = SH::TT, SUB = SH::SUB;
    constexpr bool ASYNC = V > 1;
    using XV = Pack<IO, V>;
    using AV = Pack<float, V>;
    extern __shared__ __align__(16) unsigned char smem[];
    AV *ring_a = reinterpret_cast<AV *>(smem);                               // [STAGES][S][kThreads]
    XV *ring_x = reinterpret_cast<XV *>(ring_a + (ASYNC ? STAGES * S * kThreads : 0));
    auto *ex = reinterpret_cast<Exchange<CH> *>(smem + scan_ring_bytes<IO, SH, STAGES>());
    float2 *slots = reinterpret_cast<float2 *>(ex + 1);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lc = tid % LC, grp = tid / LC;
    const int K = p.K, rank = blockIdx.x % K;
    const long long col = blockIdx.x / K;
    const long long b = col / p.blocks;
    const long long cb = (col % p.blocks) * CH, c0 = cb + lc * V;
    const bool act = c0 < p.C;
    const long long T = p.T, C = p.C;
    const IO *xb = static_cast<const IO *>(p.x) + b * T * C + c0;
    const float *ab = p.gate + b * T * C + c0;
    IO *hb = p.h ? static_cast<IO *>(p.h) + b * T * C + c0 : nullptr;

    auto first_row = [&](int step) { return ((long long)step * K + rank) * TT + (long long)grp * S; };
    auto fetch = [&](int step) {
        if constexpr (ASYNC) {
            const long long t0 = first_row(step);
            AV *sa = ring_a + (step % STAGES) * S * kThreads + tid;
            XV *sx = ring_x + (step % STAGES) * S * kThreads + tid;
            if (act && step < p.steps) {
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (t0 + s < T) {
                        copy_async<sizeof(AV)>(sa + s * kThreads, ab + (t0 + s) * C);
                        copy_async<sizeof(XV)>(sx + s * kThreads, xb + (t0 + s) * C);
                    }
            }
            copy_commit();
        }
    };
    // thread `tid` < CH folds channel cb + tid; its running state
    const bool folds = tid < CH;
    float run = 0.f;
    if (!PACKED && folds && cb + tid < C && p.state_in) run = p.state_in[b * C + cb + tid];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) fetch(i);
    if (K > 1) {   // every CTA of the cluster runs before the first store to its shared memory
        cluster_arrive();
        cluster_wait();
    }

    for (int step = 0; step < p.steps; ++step) {
        const int par = step & 1;
        const long long t0 = first_row(step);
        AV a[S];
        XV x[S];
        int code[PACKED ? S : 1];
        if constexpr (PACKED) {
#pragma unroll
            for (int s = 0; s < S; ++s) code[s] = 0;
            if (t0 < T) {
#pragma unroll
                for (int s = 0; s < S; s += 4) {
                    const int4 c = *reinterpret_cast<const int4 *>(p.codes + t0 + s);
                    code[s] = c.x, code[s + 1] = c.y, code[s + 2] = c.z, code[s + 3] = c.w;
                }
            }
        }
        if constexpr (ASYNC) {
            copy_wait<STAGES - 1>();
            const AV *sa = ring_a + (step % STAGES) * S * kThreads + tid;
            const XV *sx = ring_x + (step % STAGES) * S * kThreads + tid;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                a[s] = sa[s * kThreads];
                x[s] = sx[s * kThreads];
            }
            fetch(step + STAGES);   // into the slots just read, which no other thread touches
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (act && t0 + s < T) {
                    a[s] = *reinterpret_cast<const AV *>(ab + (t0 + s) * C);
                    x[s] = *reinterpret_cast<const XV *>(xb + (t0 + s) * C);
                }
        }
        // rows behind the end, and channels behind the last: a = 1, u = 0 leaves the state
        if (!act || t0 + S > T) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (!act || t0 + s >= T)
#pragma unroll
                    for (int j = 0; j < V; ++j) a[s].v[j] = 1.f, x[s].v[j] = from_f32<IO>(0.f);
        }
        auto input = [&](int s, int j) {
            const float u = to_f32(x[s].v[j]);
            return BLEND ? (1.f - a[s].v[j]) * u : u;
        };
        // the thread's own rows: (P, H), and in a packed batch whether a sequence starts there.
        // A first row starts from its sequence's slot; the row's h replaces its gate for the
        // second walk, because the slot may be overwritten by then.
        float P[V], H[V];
        bool reset = false;
#pragma unroll
        for (int j = 0; j < V; ++j) P[j] = 1.f, H[j] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if constexpr (PACKED) {
                if (code[s] == 0) continue;
                if (row_first(code[s])) {
                    reset = true;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float h0 = (act && p.state_in) ? p.state_in[row_seq(code[s]) * C + c0 + j] : 0.f;
                        H[j] = a[s].v[j] = fmaf(a[s].v[j], h0, input(s, j));
                    }
                    continue;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                H[j] = fmaf(a[s].v[j], H[j], input(s, j));
                P[j] *= a[s].v[j];
            }
        }
        // join the warp's groups: inclusive, then shifted to what lies in front of the thread
        int seen = reset;
#pragma unroll
        for (int off = LC; off < 32; off *= 2) {
            const int before = PACKED ? __shfl_up_sync(~0u, seen, off) : 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float Pb = __shfl_up_sync(~0u, P[j], off), Hb = __shfl_up_sync(~0u, H[j], off);
                if (lane >= off && !(PACKED && seen)) {
                    H[j] = fmaf(P[j], Hb, H[j]);
                    P[j] *= Pb;
                }
            }
            if (PACKED && lane >= off) seen |= before;
        }
        if (lane >= 32 - LC) {
#pragma unroll
            for (int j = 0; j < V; ++j) ex->warp[par][warp][lc * V + j] = make_float2(P[j], H[j]);
            if (PACKED && lane == 31) ex->reset[par][warp] = seen;
        }
        float Pf[V], Hf[V];
        int seenf = 0;
        if (SUB > 1) {
            if (PACKED) seenf = __shfl_up_sync(~0u, seen, LC);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                Pf[j] = __shfl_up_sync(~0u, P[j], LC);
                Hf[j] = __shfl_up_sync(~0u, H[j], LC);
            }
        }
        if (SUB == 1 || lane < LC) {
            seenf = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) Pf[j] = 1.f, Hf[j] = 0.f;
        }
        __syncthreads();
        // join the warps: each slot gets what lies in front of it in the tile
        float Pt = 1.f, Ht = 0.f;
        int rt = 0;
        if (folds) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 q = ex->warp[par][w][tid];
                ex->warp[par][w][tid] = make_float2(Pt, Ht);
                if (PACKED && ex->reset[par][w]) {
                    rt = 1, Pt = q.x, Ht = q.y;
                } else {
                    Ht = fmaf(q.x, Ht, q.y);
                    Pt *= q.x;
                }
            }
        }
        float cin = run;
        if (K > 1) {
            if (folds) {
                const uint32_t at = ptx::smem_u32(slots + ((size_t)par * K + rank) * CH + tid);
                for (int q = 0; q < K; ++q) store_cluster(at, q, Pt, Ht);
                if (PACKED && tid == 0) {
                    const uint32_t ar = ptx::smem_u32(&ex->slot_reset[par][rank]);
                    for (int q = 0; q < K; ++q) store_cluster(ar, q, rt);
                }
            }
            cluster_arrive();
            cluster_wait();
            if (folds) {
                for (int q = 0; q < K; ++q) {
                    if (q == rank) cin = run;
                    const float2 e = slots[((size_t)par * K + q) * CH + tid];
                    run = (PACKED && ex->slot_reset[par][q]) ? e.y : fmaf(e.x, run, e.y);
                }
            }
        } else {
            run = (PACKED && rt) ? Ht : fmaf(Pt, run, Ht);
        }
        if (folds) ex->carry[tid] = cin;
        __syncthreads();
        // the state in front of the thread's rows
        float hv[V];
        bool earlier = false;
        if constexpr (PACKED)
            for (int w = 0; w < warp; ++w) earlier |= ex->reset[par][w] != 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 w = ex->warp[par][warp][lc * V + j];
            const float front = (PACKED && earlier) ? w.y : fmaf(w.x, ex->carry[lc * V + j], w.y);
            hv[j] = (PACKED && seenf) ? Hf[j] : fmaf(Pf[j], front, Hf[j]);
        }
        if (p.ckpt && act && t0 < T && t0 % kScanCheckpoint == 0) {
            AV k;
#pragma unroll
            for (int j = 0; j < V; ++j) k.v[j] = hv[j];
            const long long rows = (T + kScanCheckpoint - 1) / kScanCheckpoint;
            *reinterpret_cast<AV *>(p.ckpt + (b * rows + t0 / kScanCheckpoint) * C + c0) = k;
        }
        if (act) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (t0 + s >= T) break;
                if (PACKED && code[s] == 0) continue;
                XV o;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    hv[j] = (PACKED && row_first(code[s])) ? a[s].v[j] : fmaf(a[s].v[j], hv[j], input(s, j));
                    o.v[j] = from_f32<IO>(hv[j]);
                }
                if (hb) *reinterpret_cast<XV *>(hb + (t0 + s) * C) = o;
                if constexpr (PACKED) {
                    if (row_last(code[s])) {
#pragma unroll
                        for (int j = 0; j < V; ++j) p.state_out[row_seq(code[s]) * C + c0 + j] = hv[j];
                    }
                }
            }
        }
    }
    if constexpr (ASYNC) copy_wait<0>();
    if (!PACKED && rank == 0 && folds && cb + tid < C && p.state_out) p.state_out[b * C + cb + tid] = run;
    if (K > 1) {   // no CTA may leave while another one's store to it is in flight
        cluster_arrive();
        cluster_wait();
    }
}

// The backward pass over dense batches: tiles from the last row to the first.  A run of rows
// acts on m (the next row's a l) as m -> P m + M.
template <typename IO, typename SH, int STAGES, bool BLEND>
__global__ void __launch_bounds__(kThreads, 2) scan_backward_kernel(const BackwardParams p) {
    constexpr int V = SH::V, LC = SH::LC, S = SH::S, CH = SH::CH, TT = SH::TT, SUB = SH::SUB;
    constexpr bool ASYNC = V > 1;
    constexpr int kGroups = kScanCheckpoint / S;   // row groups between two checkpoints
    static_assert(kScanCheckpoint % S == 0 && TT % kScanCheckpoint == 0, "tiles hold whole checkpoint spans");
    using XV = Pack<IO, V>;
    using AV = Pack<float, V>;
    extern __shared__ __align__(16) unsigned char smem[];
    AV *ring_a = reinterpret_cast<AV *>(smem);                        // [STAGES][S][kThreads]
    AV *ring_k = ring_a + (ASYNC ? STAGES * S * kThreads : 0);        // [STAGES][kThreads]
    XV *ring_x = reinterpret_cast<XV *>(ring_k + (ASYNC ? STAGES * kThreads : 0));
    XV *ring_d = ring_x + (ASYNC ? STAGES * S * kThreads : 0);
    auto *ex = reinterpret_cast<Exchange<CH> *>(smem + backward_ring_bytes<IO, SH, STAGES>());
    float2 *slots = reinterpret_cast<float2 *>(ex + 1);
    __shared__ float2 fwd[2][kWarps][CH];   // (P, H) of each warp's rows forwards, then the state in front

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lc = tid % LC, grp = tid / LC;
    const int K = p.K, rank = blockIdx.x % K;
    const long long col = blockIdx.x / K;
    const long long b = col / p.blocks;
    const long long cb = (col % p.blocks) * CH, c0 = cb + lc * V;
    const bool act = c0 < p.C;
    const long long T = p.T, C = p.C;
    const long long rows = (T + kScanCheckpoint - 1) / kScanCheckpoint;
    const long long tiles = (T + TT - 1) / TT;
    const IO *xb = static_cast<const IO *>(p.x) + b * T * C + c0;
    const IO *db = static_cast<const IO *>(p.dh) + b * T * C + c0;
    const float *ab = p.gate + b * T * C + c0;
    const float *kb = p.ckpt + b * rows * C + c0;
    IO *ob = static_cast<IO *>(p.dx) + b * T * C + c0;
    float *gb = p.dgate ? p.dgate + b * T * C + c0 : nullptr;
    // a group at a checkpoint walks forwards from it; the others continue
    const bool kept = grp % kGroups == 0;

    // first row of the thread at a step; negative tiles (before the first row) hold none
    auto first_row = [&](int step) {
        return (tiles - 1 - ((long long)step * K + rank)) * TT + (long long)grp * S;
    };
    auto fetch = [&](int step) {
        if constexpr (ASYNC) {
            const long long t0 = first_row(step);
            const int st = step % STAGES;
            if (act && step < p.steps && t0 >= 0 && t0 < T) {
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (t0 + s < T) {
                        const int at = (st * S + s) * kThreads + tid;
                        copy_async<sizeof(AV)>(ring_a + at, ab + (t0 + s) * C);
                        copy_async<sizeof(XV)>(ring_x + at, xb + (t0 + s) * C);
                        copy_async<sizeof(XV)>(ring_d + at, db + (t0 + s) * C);
                    }
                if (kept) copy_async<sizeof(AV)>(ring_k + st * kThreads + tid, kb + t0 / kScanCheckpoint * C);
            }
            copy_commit();
        }
    };
    const bool folds = tid < CH;
    float run = 0.f;
    if (folds && cb + tid < C && p.dstate) run = p.dstate[b * C + cb + tid];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) fetch(i);
    if (K > 1) {   // every CTA of the cluster runs before the first store to its shared memory
        cluster_arrive();
        cluster_wait();
    }

    for (int step = 0; step < p.steps; ++step) {
        const int par = step & 1;
        const long long t0 = first_row(step);
        const bool live = act && t0 >= 0 && t0 < T;
        AV a[S], k;
        XV x[S], d[S];
        if constexpr (ASYNC) {
            copy_wait<STAGES - 1>();
            const int st = step % STAGES;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int at = (st * S + s) * kThreads + tid;
                a[s] = ring_a[at];
                x[s] = ring_x[at];
                d[s] = ring_d[at];
            }
            k = ring_k[st * kThreads + tid];
            fetch(step + STAGES);
        } else if (live) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (t0 + s < T) {
                    a[s] = *reinterpret_cast<const AV *>(ab + (t0 + s) * C);
                    x[s] = *reinterpret_cast<const XV *>(xb + (t0 + s) * C);
                    d[s] = *reinterpret_cast<const XV *>(db + (t0 + s) * C);
                }
            if (kept) k = *reinterpret_cast<const AV *>(kb + t0 / kScanCheckpoint * C);
        }
        if (!live || t0 + S > T) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (!live || t0 + s >= T)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        a[s].v[j] = 1.f;
                        x[s].v[j] = from_f32<IO>(0.f);
                        d[s].v[j] = from_f32<IO>(0.f);
                    }
        }
        if (!live || !kept) {
#pragma unroll
            for (int j = 0; j < V; ++j) k.v[j] = 0.f;
        }
        auto input = [&](int s, int j) {
            const float u = to_f32(x[s].v[j]);
            return BLEND ? (1.f - a[s].v[j]) * u : u;
        };
        // the thread's rows: P, forwards H (from the checkpoint where it has one), backwards M
        float P[V], H[V], M[V];
#pragma unroll
        for (int j = 0; j < V; ++j) P[j] = 1.f, H[j] = k.v[j], M[j] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                H[j] = fmaf(a[s].v[j], H[j], input(s, j));
                P[j] *= a[s].v[j];
            }
#pragma unroll
        for (int s = S - 1; s >= 0; --s)
#pragma unroll
            for (int j = 0; j < V; ++j) M[j] = a[s].v[j] * (to_f32(d[s].v[j]) + M[j]);
        // join the warp's groups, forwards (a checkpoint ends the reach back) and backwards
        float Pb[V];
#pragma unroll
        for (int j = 0; j < V; ++j) Pb[j] = P[j];
        bool stop = kept;
#pragma unroll
        for (int off = LC; off < 32; off *= 2) {
            const bool stop_before = __shfl_up_sync(~0u, (int)stop, off);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float Pf = __shfl_up_sync(~0u, P[j], off), Hf = __shfl_up_sync(~0u, H[j], off);
                const float Pn = __shfl_down_sync(~0u, Pb[j], off), Mn = __shfl_down_sync(~0u, M[j], off);
                if (lane >= off && !stop) {
                    H[j] = fmaf(P[j], Hf, H[j]);
                    P[j] *= Pf;
                }
                if (lane < 32 - off) {
                    M[j] = fmaf(Pb[j], Mn, M[j]);
                    Pb[j] *= Pn;
                }
            }
            if (lane >= off) stop |= stop_before;
        }
        if (lane >= 32 - LC) {
#pragma unroll
            for (int j = 0; j < V; ++j) fwd[par][warp][lc * V + j] = make_float2(P[j], H[j]);
        }
        if (lane < LC) {
#pragma unroll
            for (int j = 0; j < V; ++j) ex->warp[par][warp][lc * V + j] = make_float2(Pb[j], M[j]);
        }
        if (lane == 31) ex->reset[par][warp] = stop;
        // shifted: what lies in front of (forwards) and behind (backwards) the thread in the warp
        float Pf[V], Hf[V], Pn[V], Mn[V];
        bool stopf = false;
        if (SUB > 1) {
            stopf = __shfl_up_sync(~0u, (int)stop, LC);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                Pf[j] = __shfl_up_sync(~0u, P[j], LC);
                Hf[j] = __shfl_up_sync(~0u, H[j], LC);
                Pn[j] = __shfl_down_sync(~0u, Pb[j], LC);
                Mn[j] = __shfl_down_sync(~0u, M[j], LC);
            }
        }
        if (SUB == 1 || lane < LC) {
            stopf = false;
#pragma unroll
            for (int j = 0; j < V; ++j) Pf[j] = 1.f, Hf[j] = 0.f;
        }
        if (SUB == 1 || lane >= 32 - LC) {
#pragma unroll
            for (int j = 0; j < V; ++j) Pn[j] = 1.f, Mn[j] = 0.f;
        }
        __syncthreads();
        float Pt = 1.f, Mt = 0.f;
        if (folds) {
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                const float2 q = ex->warp[par][w][tid];
                ex->warp[par][w][tid] = make_float2(Pt, Mt);
                Mt = fmaf(q.x, Mt, q.y);
                Pt *= q.x;
            }
        } else if (tid >= kThreads - CH) {   // other threads join forwards
            const int ch = tid - (kThreads - CH);
            float state = 0.f;   // in front of the tile's first row: a checkpoint, in its own group
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 q = fwd[par][w][ch];
                fwd[par][w][ch].y = state;
                state = ex->reset[par][w] ? q.y : fmaf(q.x, state, q.y);
            }
        }
        float cin = run;
        if (K > 1) {
            if (folds) {
                const uint32_t at = ptx::smem_u32(slots + ((size_t)par * K + rank) * CH + tid);
                for (int q = 0; q < K; ++q) store_cluster(at, q, Pt, Mt);
            }
            cluster_arrive();
            cluster_wait();
            if (folds) {
                for (int q = 0; q < K; ++q) {
                    if (q == rank) cin = run;
                    const float2 e = slots[((size_t)par * K + q) * CH + tid];
                    run = fmaf(e.x, run, e.y);
                }
            }
        } else {
            run = fmaf(Pt, run, Mt);
        }
        if (folds) ex->carry[tid] = cin;
        __syncthreads();
        if (live) {
            float hv[S][V], m[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 w = ex->warp[par][warp][lc * V + j];
                m[j] = fmaf(Pn[j], fmaf(w.x, ex->carry[lc * V + j], w.y), Mn[j]);
                const float front = fwd[par][warp][lc * V + j].y;
                float h = kept ? k.v[j] : stopf ? Hf[j] : fmaf(Pf[j], front, Hf[j]);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    hv[s][j] = h;
                    h = fmaf(a[s].v[j], h, input(s, j));
                }
            }
#pragma unroll
            for (int s = S - 1; s >= 0; --s) {
                XV o;
                AV g;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float l = to_f32(d[s].v[j]) + m[j], av = a[s].v[j];
                    o.v[j] = from_f32<IO>(BLEND ? (1.f - av) * l : l);
                    g.v[j] = l * (BLEND ? hv[s][j] - to_f32(x[s].v[j]) : hv[s][j]);
                    m[j] = av * l;
                }
                if (t0 + s < T) {
                    *reinterpret_cast<XV *>(ob + (t0 + s) * C) = o;
                    if (gb) *reinterpret_cast<AV *>(gb + (t0 + s) * C) = g;
                }
            }
        }
    }
    if constexpr (ASYNC) copy_wait<0>();
    if (rank == 0 && folds && cb + tid < C && p.dstate0) p.dstate0[b * C + cb + tid] = run;
    if (K > 1) {
        cluster_arrive();
        cluster_wait();
    }
}

// ------------------------------------------------------------------------------- rows by TMA

// V neighbouring channels of one lane, as one (V = 1) or packed (V = 2) fp32 operand.
template <int V>
struct Lane;
template <>
struct Lane<1> {
    float v;
    static __device__ __forceinline__ Lane all(float x) { return {x}; }
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ void set(int, float x) { v = x; }
    static __device__ __forceinline__ Lane load(const float *p) { return {*p}; }
    static __device__ __forceinline__ Lane load(const __nv_bfloat16 *p) { return {__bfloat162float(*p)}; }
    __device__ __forceinline__ void store(float *p) const { *p = v; }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *p = __float2bfloat16_rn(v); }
};
template <>
struct Lane<2> {
    unsigned long long v;
    static __device__ __forceinline__ Lane make(float a, float b) {
        Lane r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
        return r;
    }
    static __device__ __forceinline__ Lane all(float x) { return make(x, x); }
    __device__ __forceinline__ float2 both() const {
        float2 r;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
        return r;
    }
    __device__ __forceinline__ float get(int j) const { return j ? both().y : both().x; }
    __device__ __forceinline__ void set(int j, float x) {
        const float2 b = both();
        *this = j ? make(b.x, x) : make(x, b.y);
    }
    static __device__ __forceinline__ Lane load(const float *p) {
        const float2 f = *reinterpret_cast<const float2 *>(p);
        return make(f.x, f.y);
    }
    static __device__ __forceinline__ Lane load(const __nv_bfloat16 *p) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);   // bf16 -> fp32: the high half
        return make(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float2 *>(p) = both(); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        const float2 f = both();
        *reinterpret_cast<uint32_t *>(p) = ptx::pack_bf16x2(f.x, f.y);
    }
};
__device__ __forceinline__ Lane<1> fma(Lane<1> a, Lane<1> b, Lane<1> c) { return {fmaf(a.v, b.v, c.v)}; }
__device__ __forceinline__ Lane<1> mul(Lane<1> a, Lane<1> b) { return {a.v * b.v}; }
__device__ __forceinline__ Lane<1> add(Lane<1> a, Lane<1> b) { return {a.v + b.v}; }
__device__ __forceinline__ Lane<2> fma(Lane<2> a, Lane<2> b, Lane<2> c) {
    Lane<2> r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Lane<2> mul(Lane<2> a, Lane<2> b) {
    Lane<2> r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Lane<2> add(Lane<2> a, Lane<2> b) {
    Lane<2> r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
// (1 - a) x with one rounding of the exact x - a x
template <int V>
__device__ __forceinline__ Lane<V> blended(Lane<V> a, Lane<V> x) {
    return fma(mul(a, Lane<V>::all(-1.f)), x, x);
}

// (P, H) of a run of rows, one lane's channels.
template <int V>
struct alignas(8 * V) Run {
    Lane<V> P, H;
};
// To shared memory of CTA `rank` of the cluster; the bytes count towards its barrier `bar` (both
// given by this CTA's own addresses).
__device__ __forceinline__ uint32_t of_rank(uint32_t addr, uint32_t rank) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(addr), "r"(rank));
    return to;
}
__device__ __forceinline__ void send(uint32_t addr, uint32_t bar, uint32_t rank, const Run<1> &r) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                     of_rank(addr, rank)),
                 "f"(r.P.v), "f"(r.H.v), "r"(of_rank(bar, rank))
                 : "memory");
}
__device__ __forceinline__ void send(uint32_t addr, uint32_t bar, uint32_t rank, const Run<2> &r) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(
                     of_rank(addr, rank)),
                 "l"(r.P.v), "l"(r.H.v), "r"(of_rank(bar, rank))
                 : "memory");
}
__device__ __forceinline__ void send(uint32_t addr, uint32_t bar, uint32_t rank, int v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.s32 [%0], %1, [%2];" ::"r"(of_rank(addr, rank)),
                 "r"(v), "r"(of_rank(bar, rank))
                 : "memory");
}

struct TmaScanParams {
    CUtensorMap gate, x;     // [B][T][C], boxes of S rows x 32 V channels
    ScanParams s;
    unsigned *err;
};

// After a wait that ran out: give the copies still in flight 10 ms to land before the block's
// shared memory goes.
__device__ __noinline__ void settle() {
    for (int i = 0; i < 1000; ++i) __nanosleep(10000);
}

// Shape: V channels a lane, E elements a thread; a warp has S rows of 32 V channels.
template <int V_, int E_>
struct TmaShape {
    static constexpr int V = V_, E = E_, S = E / V, CH = 32 * V, TT = kWarps * S;
};

// Shared memory: the ring, [STAGES][kWarps] of (gate rows, x rows); then this.
template <typename SH, int STAGES>
struct TmaExchange {
    Run<SH::V> warp[2][kWarps][32];   // by the step's parity
    uint64_t full[STAGES][kWarps];
    uint64_t met[2];                  // K > 1: the step's runs of all ranks are here
    int reset[2][kWarps];
    int slot_reset[2][kMaxCluster];
    int abort;
    // followed, on 16 bytes, by Run slot[2][K][32]
};
template <typename IO, typename SH>
constexpr uint32_t tma_rows_bytes() { return SH::S * SH::CH * (sizeof(float) + sizeof(IO)); }

// Each warp runs its own pipeline: one lane asks for the boxes of the warp's rows, STAGES steps
// ahead, into a part of the ring that only this warp reads.  All lanes of a warp hold the same
// rows, so rows behind the end, sequence starts and full tiles are decided for the whole warp.
// Every thread folds the eight warps' (P, H) of its channels itself, and with K > 1 the K
// CTAs', so a step has one barrier of the CTA and no thread waits for another's fold.  With K > 1
// the ranks' runs are sent to each other by st.async, whose bytes complete the receiver's
// barrier of the step's parity.  A slot is written again two steps later: its sender has then
// had this CTA's run of the step between, sent after all of this CTA had read the slot.
template <typename IO, typename SH, int STAGES, bool BLEND, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) scan_tma_kernel(const __grid_constant__ TmaScanParams q) {
    constexpr int V = SH::V, S = SH::S, CH = SH::CH, TT = SH::TT;
    constexpr uint32_t kRows = tma_rows_bytes<IO, SH>();
    using L = Lane<V>;
    extern __shared__ __align__(128) unsigned char boxes[];
    auto *ex = reinterpret_cast<TmaExchange<SH, STAGES> *>(boxes + (size_t)STAGES * kWarps * kRows);
    auto *slots = reinterpret_cast<Run<V> *>(boxes + (size_t)STAGES * kWarps * kRows +
                                             (sizeof(TmaExchange<SH, STAGES>) + 15) / 16 * 16);
    const ScanParams &p = q.s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.K, rank = blockIdx.x % K;
    const long long col = blockIdx.x / K;
    const int b = (int)(col / p.blocks);
    const int cb = (int)(col % p.blocks) * CH, c0 = cb + lane * V;
    const bool act = c0 < p.C;
    const long long T = p.T, C = p.C;
    IO *hb = p.h ? static_cast<IO *>(p.h) + b * T * C + c0 : nullptr;

    if (tid < STAGES * kWarps) ptx::mbar_init(&ex->full[0][0] + tid, 1);
    if (tid == 0) {
        ex->abort = 0;
        ptx::mbar_init(&ex->met[0], 1);
        ptx::mbar_init(&ex->met[1], 1);
    }
    ptx::fence_mbar_init();
    if (K > 1) {   // also: every CTA of the cluster runs before the first store to its shared memory
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    auto first_row = [&](int step) { return ((long long)step * K + rank) * TT + warp * S; };
    auto fetch = [&](int step) {   // one lane
        const long long t0 = first_row(step);
        if (step < p.steps && t0 < T) {
            unsigned char *to = boxes + (size_t)(step % STAGES * kWarps + warp) * kRows;
            uint64_t *bar = &ex->full[step % STAGES][warp];
            ptx::mbar_arrive_expect_tx(bar, kRows);
            ptx::tma_load_3d(ptx::smem_u32(to), &q.gate, cb, (int)t0, b, bar);
            ptx::tma_load_3d(ptx::smem_u32(to) + S * CH * sizeof(float), &q.x, cb, (int)t0, b, bar);
        }
    };
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) fetch(i);
    }
    L run = L::all(0.f);
    if (!PACKED && act && p.state_in) run = L::load(p.state_in + b * C + c0);

    for (int step = 0; step < p.steps; ++step) {
        const int par = step & 1;
        const long long t0 = first_row(step);
        L a[S], u[S];
        int code[PACKED ? S : 1];
        if constexpr (PACKED) {
#pragma unroll
            for (int s = 0; s < S; ++s) code[s] = 0;
            if (t0 < T) {
#pragma unroll
                for (int s = 0; s < S; s += 4) {
                    const int4 c = *reinterpret_cast<const int4 *>(p.codes + t0 + s);
                    code[s] = c.x, code[s + 1] = c.y, code[s + 2] = c.z, code[s + 3] = c.w;
                }
            }
        }
        if (t0 < T) {
            ptx::mbar_wait(&ex->full[step % STAGES][warp], (step / STAGES) & 1, &ex->abort, q.err);
            const unsigned char *at = boxes + (size_t)(step % STAGES * kWarps + warp) * kRows;
            const float *sa = reinterpret_cast<const float *>(at) + lane * V;
            const IO *sx = reinterpret_cast<const IO *>(at + S * CH * sizeof(float)) + lane * V;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                a[s] = L::load(sa + s * CH);
                u[s] = L::load(sx + s * CH);
                if (BLEND) u[s] = blended(a[s], u[s]);
            }
        }
        __syncwarp();
        if (lane == 0) fetch(step + STAGES);   // into the part that the warp has just read
        if (t0 + S > T) {   // rows behind the end: a = 1, u = 0 leaves the state
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (t0 + s >= T) a[s] = L::all(1.f), u[s] = L::all(0.f);
        }
        // the warp's own rows: (P, H).  A sequence's first row starts from its slot of the states;
        // the row's h replaces its input for the second walk, when the slot may be overwritten.
        Run<V> own{L::all(1.f), L::all(0.f)};
        bool reset = false;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if constexpr (PACKED) {
                if (code[s] == 0) continue;
                if (row_first(code[s])) {
                    reset = true;
                    if (act && p.state_in)
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            u[s].set(j, fmaf(a[s].get(j), p.state_in[row_seq(code[s]) * C + c0 + j], u[s].get(j)));
                    own.H = u[s];
                    continue;
                }
            }
            own.H = fma(a[s], own.H, u[s]);
            own.P = mul(own.P, a[s]);
        }
        ex->warp[par][warp][lane] = own;
        if (PACKED && lane == 0) ex->reset[par][warp] = reset;
        __syncthreads();
        // the rows of the tile in front of the warp, and the whole tile
        Run<V> front{L::all(1.f), L::all(0.f)}, all = front;
        bool front_reset = false, all_reset = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) front = all, front_reset = all_reset;
            const Run<V> r = ex->warp[par][w][lane];
            if (PACKED && ex->reset[par][w]) {
                all = r, all_reset = true;
            } else {
                all.H = fma(r.P, all.H, r.H);
                all.P = mul(all.P, r.P);
            }
        }
        L in = run;
        if (K > 1) {
            const uint32_t at = ptx::smem_u32(slots + ((size_t)par * K + rank) * 32 + lane);
            const uint32_t bar = ptx::smem_u32(&ex->met[par]);
            for (int to = warp; to < K; to += kWarps) {
                send(at, bar, to, all);
                if (PACKED && lane == 0) send(ptx::smem_u32(&ex->slot_reset[par][rank]), bar, to, (int)all_reset);
            }
            if (tid == 0) ptx::mbar_arrive_expect_tx(&ex->met[par], K * (32 * (int)sizeof(Run<V>) + (PACKED ? 4 : 0)));
            ptx::mbar_wait(&ex->met[par], (step >> 1) & 1, &ex->abort, q.err);
            for (int r = 0; r < K; ++r) {
                if (r == rank) in = run;
                const Run<V> e = slots[((size_t)par * K + r) * 32 + lane];
                run = (PACKED && ex->slot_reset[par][r]) ? e.H : fma(e.P, run, e.H);
            }
        } else {
            run = (PACKED && all_reset) ? all.H : fma(all.P, run, all.H);
        }
        L h = (PACKED && front_reset) ? front.H : fma(front.P, in, front.H);
        if (act && t0 < T) {
            if (p.ckpt && t0 % kScanCheckpoint == 0) {
                const long long rows = (T + kScanCheckpoint - 1) / kScanCheckpoint;
                h.store(p.ckpt + (b * rows + t0 / kScanCheckpoint) * C + c0);
            }
            IO *to = hb + t0 * C;
            auto row = [&](int s) {
                if constexpr (PACKED) {
                    if (code[s] == 0) return;
                    h = row_first(code[s]) ? u[s] : fma(a[s], h, u[s]);
                    if (row_last(code[s])) {
#pragma unroll
                        for (int j = 0; j < V; ++j) p.state_out[row_seq(code[s]) * C + c0 + j] = h.get(j);
                    }
                } else {
                    h = fma(a[s], h, u[s]);
                }
                h.store(to + s * C);
            };
            if (hb) {
                if (t0 + S <= T) {
#pragma unroll
                    for (int s = 0; s < S; ++s) row(s);
                } else {
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        if (t0 + s < T) row(s);
                }
            }
        }
    }
    if (!PACKED && rank == 0 && warp == 0 && act && p.state_out)
#pragma unroll
        for (int j = 0; j < V; ++j) p.state_out[b * C + c0 + j] = run.get(j);
    if (ex->abort) settle();
    if (K > 1) {   // no CTA may leave while another one's store to it is in flight
        cluster_arrive();
        cluster_wait();
    }
}

struct TmaBackwardParams {
    CUtensorMap gate, x, dh;
    BackwardParams b;
    unsigned *err;
};
// Shared memory: the ring, [STAGES][kWarps] of (gate, x, dh rows, a checkpoint row); then this.
template <typename SH, int STAGES>
struct TmaBackwardExchange {
    Run<SH::V> warp[2][kWarps][32];   // (P, H) forwards
    Lane<SH::V> M[2][kWarps][32];
    uint64_t full[STAGES][kWarps];
    uint64_t met[2];
    int abort;
};
template <typename IO, typename SH>
constexpr uint32_t tma_backward_rows_bytes() {
    return SH::S * SH::CH * (sizeof(float) + 2 * sizeof(IO)) + SH::CH * sizeof(float);
}

template <typename IO, typename SH, int STAGES, bool BLEND>
__global__ void __launch_bounds__(kThreads, 2) scan_backward_tma_kernel(const __grid_constant__ TmaBackwardParams q) {
    constexpr int V = SH::V, S = SH::S, CH = SH::CH, TT = SH::TT;
    constexpr int kGroups = kScanCheckpoint / S;   // warps between two checkpoints
    static_assert(kScanCheckpoint % S == 0 && TT % kScanCheckpoint == 0, "tiles hold whole checkpoint spans");
    constexpr uint32_t kRows = tma_backward_rows_bytes<IO, SH>(), kBoxes = kRows - CH * sizeof(float);
    using L = Lane<V>;
    extern __shared__ __align__(128) unsigned char boxes[];
    auto *ex = reinterpret_cast<TmaBackwardExchange<SH, STAGES> *>(boxes + (size_t)STAGES * kWarps * kRows);
    auto *slots = reinterpret_cast<Run<V> *>(boxes + (size_t)STAGES * kWarps * kRows +
                                             (sizeof(TmaBackwardExchange<SH, STAGES>) + 15) / 16 * 16);
    const BackwardParams &p = q.b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.K, rank = blockIdx.x % K;
    const long long col = blockIdx.x / K;
    const int b = (int)(col / p.blocks);
    const int cb = (int)(col % p.blocks) * CH, c0 = cb + lane * V;
    const bool act = c0 < p.C;
    const long long T = p.T, C = p.C;
    const long long tiles = (T + TT - 1) / TT;
    const float *kb = p.ckpt + (b * ((T + kScanCheckpoint - 1) / kScanCheckpoint)) * C + cb;
    const uint32_t kept_bytes = (uint32_t)(C - cb < CH ? C - cb : CH) * sizeof(float);
    IO *ob = static_cast<IO *>(p.dx) + b * T * C + c0;
    float *gb = p.dgate ? p.dgate + b * T * C + c0 : nullptr;
    const bool kept = warp % kGroups == 0;   // the warp's rows start at a checkpoint

    if (tid < STAGES * kWarps) ptx::mbar_init(&ex->full[0][0] + tid, 1);
    if (tid == 0) {
        ex->abort = 0;
        ptx::mbar_init(&ex->met[0], 1);
        ptx::mbar_init(&ex->met[1], 1);
    }
    ptx::fence_mbar_init();
    if (K > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    auto first_row = [&](int step) { return (tiles - 1 - ((long long)step * K + rank)) * TT + warp * S; };
    // A warp's rows may lie behind the last row at the first steps, and in front of row 0 at the
    // last ones: only the loads that were asked for are waited for, and counted for the parity.
    auto live_at = [&](int step) {
        const long long t0 = first_row(step);
        return step < p.steps && t0 >= 0 && t0 < T;
    };
    auto fetch = [&](int step) {   // one lane
        if (live_at(step)) {
            const long long t0 = first_row(step);
            const uint32_t to = ptx::smem_u32(boxes + (size_t)(step % STAGES * kWarps + warp) * kRows);
            uint64_t *bar = &ex->full[step % STAGES][warp];
            ptx::mbar_arrive_expect_tx(bar, kBoxes + (kept ? kept_bytes : 0));
            ptx::tma_load_3d(to, &q.gate, cb, (int)t0, b, bar);
            ptx::tma_load_3d(to + S * CH * sizeof(float), &q.x, cb, (int)t0, b, bar);
            ptx::tma_load_3d(to + S * CH * (sizeof(float) + sizeof(IO)), &q.dh, cb, (int)t0, b, bar);
            if (kept) ptx::bulk_load(to + kBoxes, kb + t0 / kScanCheckpoint * C, kept_bytes, bar);
        }
    };
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) fetch(i);
    }
    uint32_t phases = 0;   // a bit a stage: the parity of its next load
    L run = L::all(0.f);
    if (act && p.dstate)
#pragma unroll
        for (int j = 0; j < V; ++j) run.set(j, p.dstate[b * C + c0 + j]);

    for (int step = 0; step < p.steps; ++step) {
        const int par = step & 1, st = step % STAGES;
        const long long t0 = first_row(step);
        const bool live = live_at(step);
        L a[S], x[S], d[S], k = L::all(0.f);
        if (live) {
            ptx::mbar_wait(&ex->full[st][warp], (phases >> st) & 1, &ex->abort, q.err);
            phases ^= 1u << st;
            const unsigned char *at = boxes + (size_t)(st * kWarps + warp) * kRows;
            const float *sa = reinterpret_cast<const float *>(at) + lane * V;
            const IO *sx = reinterpret_cast<const IO *>(at + S * CH * sizeof(float)) + lane * V;
            const IO *sd = sx + S * CH;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                a[s] = L::load(sa + s * CH);
                x[s] = L::load(sx + s * CH);
                d[s] = L::load(sd + s * CH);
            }
            if (kept && act) k = L::load(reinterpret_cast<const float *>(at + kBoxes) + lane * V);
        }
        __syncwarp();
        if (lane == 0) fetch(step + STAGES);
        if (!live || t0 + S > T) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (!live || t0 + s >= T) a[s] = L::all(1.f), x[s] = L::all(0.f), d[s] = L::all(0.f);
        }
        // the warp's rows: P, forwards H (from the checkpoint where it has one), backwards M
        Run<V> own{L::all(1.f), k};
        L M = L::all(0.f), before[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            own.H = fma(a[s], own.H, BLEND ? blended(a[s], x[s]) : x[s]);
            own.P = mul(own.P, a[s]);
        }
#pragma unroll
        for (int s = S - 1; s >= 0; --s) M = mul(a[s], add(d[s], M));
        ex->warp[par][warp][lane] = own;
        ex->M[par][warp][lane] = M;
        __syncthreads();
        // forwards: the state in front of the warp, from the last checkpoint
        L h = k;
        if (!kept) {
            const int from = warp / kGroups * kGroups;
            h = ex->warp[par][from][lane].H;
            for (int w = from + 1; w < warp; ++w) {
                const Run<V> r = ex->warp[par][w][lane];
                h = fma(r.P, h, r.H);
            }
        }
        // backwards: what the rows of the tile behind the warp do to m, and the whole tile
        Run<V> behind{L::all(1.f), L::all(0.f)}, all = behind;
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            if (w == warp) behind = all;
            const L P = ex->warp[par][w][lane].P;
            all.H = fma(P, all.H, ex->M[par][w][lane]);
            all.P = mul(all.P, P);
        }
        L in = run;
        if (K > 1) {
            const uint32_t at = ptx::smem_u32(slots + ((size_t)par * K + rank) * 32 + lane);
            const uint32_t bar = ptx::smem_u32(&ex->met[par]);
            for (int to = warp; to < K; to += kWarps) send(at, bar, to, all);
            if (tid == 0) ptx::mbar_arrive_expect_tx(&ex->met[par], K * 32 * (int)sizeof(Run<V>));
            ptx::mbar_wait(&ex->met[par], (step >> 1) & 1, &ex->abort, q.err);
            for (int r = 0; r < K; ++r) {
                if (r == rank) in = run;
                const Run<V> e = slots[((size_t)par * K + r) * 32 + lane];
                run = fma(e.P, run, e.H);
            }
        } else {
            run = fma(all.P, run, all.H);
        }
        if (act && live) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                before[s] = h;
                h = fma(a[s], h, BLEND ? blended(a[s], x[s]) : x[s]);
            }
            L m = fma(behind.P, in, behind.H);
            const bool full = t0 + S <= T;
#pragma unroll
            for (int s = S - 1; s >= 0; --s) {
                const L l = add(d[s], m);
                m = mul(a[s], l);
                if (full || t0 + s < T) {
                    (BLEND ? blended(a[s], l) : l).store(ob + (t0 + s) * C);
                    if (gb) {
                        const L g = BLEND ? add(before[s], mul(x[s], L::all(-1.f))) : before[s];
                        mul(l, g).store(gb + (t0 + s) * C);
                    }
                }
            }
        }
    }
    if (rank == 0 && warp == 0 && act && p.dstate0)
#pragma unroll
        for (int j = 0; j < V; ++j) p.dstate0[b * C + c0 + j] = run.get(j);
    if (ex->abort) settle();
    if (K > 1) {   // no CTA may leave while another one's store to it is in flight
        cluster_arrive();
        cluster_wait();
    }
}

// One token: no reuse, every operand once.  Flat over N * C elements, V a thread (the last ones
// singly; V = 1 where a tensor starts off the vectors' boundaries).
template <typename IO, int V, bool BLEND>
__global__ void __launch_bounds__(256)
scan_step_kernel(long long n, const IO *__restrict__ x, const float *__restrict__ gate, float *__restrict__ state,
                 IO *__restrict__ h) {
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * V;
    auto one = [](float a, float s, float u) { return fmaf(a, s, BLEND ? (1.f - a) * u : u); };
    if (i + V <= n) {
        const auto a = load_pack<float, V>(gate + i);
        auto s = load_pack<float, V>(state + i);
        const auto u = load_pack<IO, V>(x + i);
        Pack<IO, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s.v[j] = one(a.v[j], s.v[j], to_f32(u.v[j]));
            o.v[j] = from_f32<IO>(s.v[j]);
        }
        store_pack<float, V>(state + i, s);
        store_pack<IO, V>(h + i, o);
    } else {
        for (long long e = i; e < n; ++e) {
            const float s = one(gate[e], state[e], to_f32(x[e]));
            state[e] = s;
            h[e] = from_f32<IO>(s);
        }
    }
}

// Row codes of a packed batch, checks of its offsets, and the zero state of an empty sequence
// without an initial one.  The first `row_blocks` blocks search the sequence of each row (the
// last s with cu[s] <= t); then one block a sequence.
__global__ void __launch_bounds__(256)
scan_rows_kernel(int T, int padded, int row_blocks, int N, long long C, const int *__restrict__ cu,
                 int *__restrict__ codes, float *__restrict__ zero_state, unsigned *err) {
    if ((int)blockIdx.x < row_blocks) {
        const int t = blockIdx.x * 256 + threadIdx.x;
        if (t >= padded) return;
        int code = 0;
        if (t < T) {
            int lo = 0, hi = N + 1;   // entries [0, lo) are <= t
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (min(max(cu[mid], 0), T) <= t) lo = mid + 1;
                else hi = mid;
            }
            const int s = lo - 1;
            if (s >= 0 && s < N) code = 4 * (s + 1) + (cu[s + 1] == t + 1 ? 2 : 0) + (max(cu[s], 0) == t ? 1 : 0);
        }
        codes[t] = code;
        return;
    }
    const int s = blockIdx.x - row_blocks;
    const int a = cu[s], e = cu[s + 1];
    if (threadIdx.x == 0 && (a < 0 || e > T || e < a) && err) atomicOr(err, (unsigned)kErrBadInput);
    if (zero_state && min(e, T) <= max(a, 0))
        for (long long c = threadIdx.x; c < C; c += 256) zero_state[s * C + c] = 0.f;
}

// ------------------------------------------------------------------------------- host side

// How the columns (batch rows x channel blocks) and the tiles of a call are spread: the
// cluster width whose estimated time is the least.  A CTA alone moves at most `kCtaRate`
// bytes/ns (its ring's bytes over the latency of HBM under load) and all of them together
// `kRate`; clusters that do not fit at once take further waves.
constexpr double kCtaRate = 40.0, kRate = 6500.0;

struct Plan {
    int K = 1;
    double cost = 1e300;
};

template <typename L>   // L: Forward or Backward, one kernel
Plan plan_clusters(long long cols, long long tiles, double tile_bytes) {
    // clusters of 2^i CTAs that run at once, plus one (0: not asked yet); the same on every B200
    static std::atomic<int> known[5];
    constexpr auto kernel = L::kernel;
    Plan best;
    for (int i = 0; i < 5; ++i) {
        const int K = 1 << i;
        if (K > 1 && K >= 2 * tiles) break;
        int fit = known[i].load(std::memory_order_relaxed) - 1;
        if (fit < 0) {
            const size_t smem = L::smem(K);
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
                (K > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)) {
                (void)cudaGetLastError();
                break;
            }
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim = {(unsigned)K, 1, 1};
            cfg.gridDim = dim3(K * 1024);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                n = 0;
            }
            fit = n;
            known[i].store(n + 1, std::memory_order_relaxed);
        }
        if (fit < 1) continue;
        const double waves = (double)((cols + fit - 1) / fit);
        const double active = (double)(cols < fit ? cols : fit) * K;
        const double steps = (double)((tiles + K - 1) / K);
        const double rate = active * kCtaRate < kRate ? kCtaRate : kRate / active;
        const double cost = waves * steps * (tile_bytes / rate + (K > 1 ? 300.0 : 0.0));
        if (cost < best.cost) best.cost = cost, best.K = K;
    }
    return best;
}

template <typename P>
cudaError_t launch_cluster(void (*kernel)(P), const P &p, long long cols, int K, size_t smem, cudaStream_t stream) {
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err == cudaSuccess && K > 8)
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess) return err;
    if (cols * K > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)K, 1, 1};
    cfg.gridDim = dim3((unsigned)(cols * K));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    timer_begin(stream);
    err = cudaLaunchKernelEx(&cfg, kernel, p);
    timer_end(stream);
    note_launches(1);
    return err != cudaSuccess ? err : cudaGetLastError();
}

template <typename IO, typename SH, int STAGES, bool BLEND, bool PACKED>
struct Forward {
    static constexpr auto kernel = scan_kernel<IO, SH, STAGES, BLEND, PACKED>;
    static size_t smem(int K) { return scan_ring_bytes<IO, SH, STAGES>() + exchange_bytes<SH>(K); }
    static long long cols(const ScanArgs &a) { return (long long)a.B * ((a.C + SH::CH - 1) / SH::CH); }
    static long long tiles(const ScanArgs &a) { return ((long long)a.T + SH::TT - 1) / SH::TT; }
    static Plan plan(const ScanArgs &a) {
        return plan_clusters<Forward>(cols(a), tiles(a), (double)kThreads * SH::E * (sizeof(float) + 2 * sizeof(IO)));
    }
    static cudaError_t launch(const ScanArgs &a, int K) {
        ScanParams p;
        p.x = a.x; p.gate = a.gate;
        p.state_in = a.state_in; p.state_out = a.state_out;
        p.h = a.h; p.ckpt = a.ckpt; p.codes = a.codes;
        p.T = a.T; p.C = a.C;
        p.blocks = (int)((a.C + SH::CH - 1) / SH::CH);
        p.K = K;
        p.steps = (int)((tiles(a) + K - 1) / K);
        return launch_cluster<ScanParams>(kernel, p, cols(a), K, smem(K), a.stream);
    }
};

template <typename IO, typename SH, int STAGES, bool BLEND>
struct Backward {
    static constexpr auto kernel = scan_backward_kernel<IO, SH, STAGES, BLEND>;
    static size_t smem(int K) { return backward_ring_bytes<IO, SH, STAGES>() + exchange_bytes<SH>(K); }
    static long long cols(const ScanBackwardArgs &a) { return (long long)a.B * ((a.C + SH::CH - 1) / SH::CH); }
    static long long tiles(const ScanBackwardArgs &a) { return ((long long)a.T + SH::TT - 1) / SH::TT; }
    static Plan plan(const ScanBackwardArgs &a) {
        return plan_clusters<Backward>(cols(a), tiles(a),
                                       (double)kThreads * SH::E * (2 * sizeof(float) + 3 * sizeof(IO)));
    }
    static cudaError_t launch(const ScanBackwardArgs &a, int K) {
        BackwardParams p;
        p.x = a.x; p.dh = a.dh;
        p.gate = a.gate; p.ckpt = a.ckpt; p.dstate = a.dstate;
        p.dx = a.dx; p.dgate = a.dgate; p.dstate0 = a.dstate0;
        p.T = a.T; p.C = a.C;
        p.blocks = (int)((a.C + SH::CH - 1) / SH::CH);
        p.K = K;
        p.steps = (int)((tiles(a) + K - 1) / K);
        return launch_cluster<BackwardParams>(kernel, p, cols(a), K, smem(K), a.stream);
    }
};

// Row tensors as TMA sees them: [B][T][C] in boxes of S rows x CH channels.  False where a row
// does not start on 16 bytes (or a size is beyond a tensor map).
template <typename SH>
bool row_map(CUtensorMap *map, const void *base, size_t elem, long long B, long long T, long long C) {
    return make_tmap_3d(map, base, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                        (uint32_t)elem, C, T, B, C * elem, T * C * elem, SH::CH, SH::S, false);
}

template <typename IO, typename SH, int STAGES, bool BLEND, bool PACKED>
struct ForwardTma {
    static constexpr auto kernel = scan_tma_kernel<IO, SH, STAGES, BLEND, PACKED>;
    static size_t smem(int K) {
        return (size_t)STAGES * kWarps * tma_rows_bytes<IO, SH>() + (sizeof(TmaExchange<SH, STAGES>) + 15) / 16 * 16 +
               (K > 1 ? (size_t)2 * K * 32 * sizeof(Run<SH::V>) : 0);
    }
    static long long cols(const ScanArgs &a) { return (long long)a.B * ((a.C + SH::CH - 1) / SH::CH); }
    static long long tiles(const ScanArgs &a) { return ((long long)a.T + SH::TT - 1) / SH::TT; }
    static Plan plan(const ScanArgs &a) {
        return plan_clusters<ForwardTma>(cols(a), tiles(a), (double)kThreads * SH::E * (sizeof(float) + 2 * sizeof(IO)));
    }
    static cudaError_t launch(const ScanArgs &a, int K) {
        TmaScanParams q;
        if (!row_map<SH>(&q.gate, a.gate, sizeof(float), a.B, a.T, a.C) ||
            !row_map<SH>(&q.x, a.x, sizeof(IO), a.B, a.T, a.C))
            return cudaErrorInvalidValue;
        ScanParams &p = q.s;
        p.x = a.x; p.gate = a.gate;
        p.state_in = a.state_in; p.state_out = a.state_out;
        p.h = a.h; p.ckpt = a.ckpt; p.codes = a.codes;
        p.T = a.T; p.C = a.C;
        p.blocks = (int)((a.C + SH::CH - 1) / SH::CH);
        p.K = K;
        p.steps = (int)((tiles(a) + K - 1) / K);
        q.err = device_error_word();
        return launch_cluster<TmaScanParams>(kernel, q, cols(a), K, smem(K), a.stream);
    }
};

template <typename IO, typename SH, int STAGES, bool BLEND>
struct BackwardTma {
    static constexpr auto kernel = scan_backward_tma_kernel<IO, SH, STAGES, BLEND>;
    static size_t smem(int K) {
        return (size_t)STAGES * kWarps * tma_backward_rows_bytes<IO, SH>() +
               (sizeof(TmaBackwardExchange<SH, STAGES>) + 15) / 16 * 16 +
               (K > 1 ? (size_t)2 * K * 32 * sizeof(Run<SH::V>) : 0);
    }
    static long long cols(const ScanBackwardArgs &a) { return (long long)a.B * ((a.C + SH::CH - 1) / SH::CH); }
    static long long tiles(const ScanBackwardArgs &a) { return ((long long)a.T + SH::TT - 1) / SH::TT; }
    static Plan plan(const ScanBackwardArgs &a) {
        return plan_clusters<BackwardTma>(cols(a), tiles(a),
                                          (double)kThreads * SH::E * (2 * sizeof(float) + 3 * sizeof(IO)));
    }
    static cudaError_t launch(const ScanBackwardArgs &a, int K) {
        TmaBackwardParams q;
        if (!row_map<SH>(&q.gate, a.gate, sizeof(float), a.B, a.T, a.C) ||
            !row_map<SH>(&q.x, a.x, sizeof(IO), a.B, a.T, a.C) || !row_map<SH>(&q.dh, a.dh, sizeof(IO), a.B, a.T, a.C))
            return cudaErrorInvalidValue;
        BackwardParams &p = q.b;
        p.x = a.x; p.dh = a.dh;
        p.gate = a.gate; p.ckpt = a.ckpt; p.dstate = a.dstate;
        p.dx = a.dx; p.dgate = a.dgate; p.dstate0 = a.dstate0;
        p.T = a.T; p.C = a.C;
        p.blocks = (int)((a.C + SH::CH - 1) / SH::CH);
        p.K = K;
        p.steps = (int)((tiles(a) + K - 1) / K);
        q.err = device_error_word();
        return launch_cluster<TmaBackwardParams>(kernel, q, cols(a), K, smem(K), a.stream);
    }
};

// Whether rows can come by TMA: 16-byte rows and starts (and channels that a lane's vectors and
// the checkpoints' bulk copies divide), sizes within a tensor map.
bool tma_rows(long long B, long long T, long long C, size_t elem, std::initializer_list<const void *> in,
              std::initializer_list<const void *> out) {
    if (C * elem % 16 || C * 4 % 16 || T * C * 4 >= (1ll << 40)) return false;
    for (const void *q : in)
        if (reinterpret_cast<uintptr_t>(q) % 16) return false;
    for (const void *q : out)
        if (reinterpret_cast<uintptr_t>(q) % 8) return false;
    return true;
}

// Channels a thread: the widest vectors that the rows' length and the tensors' starts allow.
template <typename IO>
int vector_width(long long C, std::initializer_list<const void *> io, std::initializer_list<const void *> fp32) {
    for (int V = 4; V > 1; V /= 2) {
        bool ok = C % V == 0;
        for (const void *q : io) ok = ok && reinterpret_cast<uintptr_t>(q) % (V * sizeof(IO)) == 0;
        for (const void *q : fp32) ok = ok && reinterpret_cast<uintptr_t>(q) % (V * sizeof(float)) == 0;
        if (ok) return V;
    }
    return 1;
}

// The wide shape, or the narrow one where it gives enough more parallelism.
template <typename Wide, typename Narrow, typename Args>
cudaError_t launch_best(const Args &a) {
    const Plan w = Wide::plan(a), n = Narrow::plan(a);
    return n.cost < 0.9 * w.cost ? Narrow::launch(a, n.K) : Wide::launch(a, w.K);
}

template <typename IO, int V, bool BLEND, bool PACKED>
cudaError_t forward_v(const ScanArgs &a) {
    constexpr int E = sizeof(IO) == 2 && V > 1 ? 32 : 16, STAGES = sizeof(IO) == 2 ? 2 : 3;
    return launch_best<Forward<IO, Shape<V, 16, E>, STAGES, BLEND, PACKED>,
                       Forward<IO, Shape<V, 4, E>, STAGES, BLEND, PACKED>>(a);
}
template <typename IO, int V>
cudaError_t forward_flags(const ScanArgs &a) {
    if (a.codes) return a.blend ? forward_v<IO, V, true, true>(a) : forward_v<IO, V, false, true>(a);
    return a.blend ? forward_v<IO, V, true, false>(a) : forward_v<IO, V, false, false>(a);
}
template <typename IO, bool BLEND, bool PACKED>
cudaError_t forward_tma(const ScanArgs &a) {
    constexpr int E = sizeof(IO) == 2 ? 32 : 16, STAGES = sizeof(IO) == 2 ? 2 : 3;
    return launch_best<ForwardTma<IO, TmaShape<2, E>, STAGES, BLEND, PACKED>,
                       ForwardTma<IO, TmaShape<1, E>, STAGES, BLEND, PACKED>>(a);
}
template <typename IO>
cudaError_t forward_io(const ScanArgs &a) {
    if (tma_rows(a.B, a.T, a.C, sizeof(IO), {a.x, a.gate}, {a.h, a.ckpt, a.state_in, a.state_out})) {
        if (a.codes) return a.blend ? forward_tma<IO, true, true>(a) : forward_tma<IO, false, true>(a);
        return a.blend ? forward_tma<IO, true, false>(a) : forward_tma<IO, false, false>(a);
    }
    const int V = vector_width<IO>(a.C, {a.x, a.h}, {a.gate, a.ckpt});
    return V == 4 ? forward_flags<IO, 4>(a) : V == 2 ? forward_flags<IO, 2>(a) : forward_flags<IO, 1>(a);
}

template <typename IO, int V, bool BLEND>
cudaError_t backward_v(const ScanBackwardArgs &a) {
    constexpr int E = sizeof(IO) == 2 && V > 1 ? 16 : 8, STAGES = sizeof(IO) == 2 ? 2 : 3;
    return launch_best<Backward<IO, Shape<V, 16, E>, STAGES, BLEND>, Backward<IO, Shape<V, 4, E>, STAGES, BLEND>>(a);
}
template <typename IO, bool BLEND>
cudaError_t backward_tma(const ScanBackwardArgs &a) {
    constexpr int STAGES = sizeof(IO) == 2 ? 3 : 2;
    return launch_best<BackwardTma<IO, TmaShape<2, 16>, STAGES, BLEND>, BackwardTma<IO, TmaShape<1, 16>, STAGES, BLEND>>(a);
}
template <typename IO>
cudaError_t backward_io(const ScanBackwardArgs &a) {
    if (tma_rows(a.B, a.T, a.C, sizeof(IO), {a.x, a.gate, a.dh, a.ckpt}, {a.dx, a.dgate}))
        return a.blend ? backward_tma<IO, true>(a) : backward_tma<IO, false>(a);
    const int V = vector_width<IO>(a.C, {a.x, a.dh, a.dx}, {a.gate, a.ckpt, a.dgate});
    if (V == 4) return a.blend ? backward_v<IO, 4, true>(a) : backward_v<IO, 4, false>(a);
    if (V == 2) return a.blend ? backward_v<IO, 2, true>(a) : backward_v<IO, 2, false>(a);
    return a.blend ? backward_v<IO, 1, true>(a) : backward_v<IO, 1, false>(a);
}

}  // namespace

size_t scan_codes_bytes(int T) { return sizeof(int) * (((size_t)T + 31) / 32 * 32); }

cudaError_t launch_scan_rows(const ScanArgs &a, const int *cu, int N, int *codes, float *zero_state) {
    const int padded = (a.T + 31) / 32 * 32, row_blocks = (padded + 255) / 256;
    timer_begin(a.stream);
    scan_rows_kernel<<<(unsigned)row_blocks + (unsigned)N, 256, 0, a.stream>>>(a.T, padded, row_blocks, N, a.C, cu,
                                                                               codes, zero_state, device_error_word());
    timer_end(a.stream);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_scan(const ScanArgs &a) {
    return a.dtype == LA_BF16 ? forward_io<__nv_bfloat16>(a) : forward_io<float>(a);
}

cudaError_t launch_scan_backward(const ScanBackwardArgs &a) {
    return a.dtype == LA_BF16 ? backward_io<__nv_bfloat16>(a) : backward_io<float>(a);
}

cudaError_t launch_scan_step(const ScanArgs &a) {
    const long long n = (long long)a.B * a.C;
    auto go = [&](auto io, auto blend) {
        using IO = decltype(io);
        constexpr bool BLEND = decltype(blend)::value;
        const IO *x = static_cast<const IO *>(a.x);
        IO *h = static_cast<IO *>(a.h);
        if (vector_width<IO>(4, {x, h}, {a.gate, a.state_out}) == 4)
            scan_step_kernel<IO, 4, BLEND><<<(unsigned)((n + 1023) / 1024), 256, 0, a.stream>>>(n, x, a.gate,
                                                                                              a.state_out, h);
        else
            scan_step_kernel<IO, 1, BLEND><<<(unsigned)((n + 255) / 256), 256, 0, a.stream>>>(n, x, a.gate,
                                                                                            a.state_out, h);
    };
    if (n > 256ll * INT32_MAX) return cudaErrorInvalidConfiguration;
    timer_begin(a.stream);
    if (a.dtype == LA_BF16) a.blend ? go(__nv_bfloat16{}, std::true_type{}) : go(__nv_bfloat16{}, std::false_type{});
    else a.blend ? go(float{}, std::true_type{}) : go(float{}, std::false_type{});
    timer_end(a.stream);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace la
