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
#include "scan_util.cuh"
#include "vec.cuh"

#include <initializer_list>
#include <type_traits>

namespace la {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

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

template <typename IO, typename SH, int STAGES, bool BLEND, bool PACKED>
struct Forward {
    static constexpr auto kernel = scan_kernel<IO, SH, STAGES, BLEND, PACKED>;
    static constexpr int kBlock = kThreads, kChannels = SH::CH, kMost = 16;
    static constexpr double kRate = 4000.0;
    static constexpr double kTileBytes = (double)kThreads * SH::E * (sizeof(float) + 2 * sizeof(IO));
    static double step_ns(int K) { return 2200.0 + (K > 1 ? 300.0 : 0.0); }
    static size_t smem(int K) { return scan_ring_bytes<IO, SH, STAGES>() + exchange_bytes<SH>(K); }
    static long long cols(const ScanArgs &a) { return (long long)a.B * ((a.C + SH::CH - 1) / SH::CH); }
    static long long tiles(const ScanArgs &a) { return ((long long)a.T + SH::TT - 1) / SH::TT; }
    static cudaError_t launch(const ScanArgs &a, int K) {
        return launch_cluster<Forward>(scan_params<Forward>(a, K), cols(a), K, a.stream);
    }
};

template <typename IO, typename SH, int STAGES, bool BLEND>
struct Backward {
    static constexpr auto kernel = scan_backward_kernel<IO, SH, STAGES, BLEND>;
    static constexpr int kBlock = kThreads, kChannels = SH::CH, kMost = 16;
    static constexpr double kRate = 4000.0;
    static constexpr double kTileBytes = (double)kThreads * SH::E * (2 * sizeof(float) + 3 * sizeof(IO));
    static double step_ns(int K) { return 2200.0 + (K > 1 ? 300.0 : 0.0); }
    static size_t smem(int K) { return backward_ring_bytes<IO, SH, STAGES>() + exchange_bytes<SH>(K); }
    static long long cols(const ScanBackwardArgs &a) { return (long long)a.B * ((a.C + SH::CH - 1) / SH::CH); }
    static long long tiles(const ScanBackwardArgs &a) { return ((long long)a.T + SH::TT - 1) / SH::TT; }
    static cudaError_t launch(const ScanBackwardArgs &a, int K) {
        return launch_cluster<Backward>(backward_params<Backward>(a, K), cols(a), K, a.stream);
    }
};

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
template <typename IO>
cudaError_t forward_io(const ScanArgs &a) {
    const int V = vector_width<IO>(a.C, {a.x, a.h}, {a.gate, a.ckpt});
    return V == 4 ? forward_flags<IO, 4>(a) : V == 2 ? forward_flags<IO, 2>(a) : forward_flags<IO, 1>(a);
}

template <typename IO, int V, bool BLEND>
cudaError_t backward_v(const ScanBackwardArgs &a) {
    constexpr int E = sizeof(IO) == 2 && V > 1 ? 16 : 8, STAGES = sizeof(IO) == 2 ? 2 : 3;
    return launch_best<Backward<IO, Shape<V, 16, E>, STAGES, BLEND>, Backward<IO, Shape<V, 4, E>, STAGES, BLEND>>(a);
}
template <typename IO>
cudaError_t backward_io(const ScanBackwardArgs &a) {
    const int V = vector_width<IO>(a.C, {a.x, a.dh, a.dx}, {a.gate, a.ckpt, a.dgate});
    if (V == 4) return a.blend ? backward_v<IO, 4, true>(a) : backward_v<IO, 4, false>(a);
    if (V == 2) return a.blend ? backward_v<IO, 2, true>(a) : backward_v<IO, 2, false>(a);
    return a.blend ? backward_v<IO, 1, true>(a) : backward_v<IO, 1, false>(a);
}

}  // namespace

// The codes are read in whole tiles of rows.
constexpr int kCodeRows = 256;
size_t scan_codes_bytes(int T) { return sizeof(int) * (((size_t)T + kCodeRows - 1) / kCodeRows * kCodeRows); }

cudaError_t launch_scan_rows(const ScanArgs &a, const int *cu, int N, int *codes, float *zero_state) {
    const int padded = (a.T + kCodeRows - 1) / kCodeRows * kCodeRows, row_blocks = (padded + 255) / 256;
    timer_begin(a.stream);
    scan_rows_kernel<<<(unsigned)row_blocks + (unsigned)N, 256, 0, a.stream>>>(a.T, padded, row_blocks, N, a.C, cu,
                                                                               codes, zero_state, device_error_word());
    timer_end(a.stream);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_scan(const ScanArgs &a) {
    if (scan_tma_takes(a)) return launch_scan_tma(a);
    return a.dtype == LA_BF16 ? forward_io<__nv_bfloat16>(a) : forward_io<float>(a);
}

cudaError_t launch_scan_backward(const ScanBackwardArgs &a) {
    if (scan_tma_takes(a)) return launch_scan_backward_tma(a);
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
