// linrec.cu -- gated linear recurrence, forward and gradient.
//
//   a_t = sigmoid(f_t),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  y_t = h_t silu(z_t)
//   gradient, backwards in time, mu_t the adjoint of h_{t-1}:
//     lam_t = dy_t silu(z_t) + mu_{t+1},  mu_t = a_t lam_t
//     df_t = lam_t (h_{t-1} - x_t) a_t (1 - a_t),  dx_t = lam_t (1 - a_t),
//     dz_t = dy_t h_t silu'(z_t)
//
// Bound by memory: every channel is a scalar recurrence, about 25 FP32 and 2 to
// 6 MUFU operations per element against 6 to 28 bytes.  The sequence is cut
// into tiles so that few channels still fill the GPU: a span of steps acts on
// the state as h -> P h + q, and spans compose by (P1, q1) o (P2, q2) =
// (P1 P2, P2 q1 + q2).
//
//  * A CTA takes a tile of 8 S steps by 64 channels; warp w takes S consecutive
//    steps, a lane two neighbouring channels, so a warp's access to a step is
//    one row segment of 64 channels.  Inputs come through a ring of shared
//    memory tiles filled with cp.async, so the next tile's loads are in flight
//    while this one waits for its predecessors.
//  * Each warp scans its steps from zero, keeping a_t and b_t in registers;
//    the warps' (P, q) meet in shared memory; tiles chain through a decoupled
//    look-back (Merrill and Garland's single-pass prefix scan): a tile publishes
//    its aggregate, or its inclusive state at once where its predecessor's is
//    already there, and composes backwards to the newest inclusive state.
//    Tiles are handed out in order by a ticket, so a predecessor is always
//    running or done; every wait is bounded (SSM_ERR_TIMEOUT).
//  * Each warp then replays its steps from its entry state and writes y.
// The gradient is the same scan of (a_t, a_t dh_t) in reverse order.  The states
// it needs are not stored but taken again: the forward keeps the state every 64
// steps in fp32, and each tile replays its own steps from there.
//
// Masked steps: a gate of +inf holds the state whatever x is there (b_t = 0 where
// 1 - a_t = 0), a gate of -inf restarts it whatever it was (a_t = 0 drops h, NaN
// and infinities too); their gradients are 0.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "scan_internal.h"

namespace {

using namespace ssm;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCh = 64;         // channels per tile, two per lane
constexpr int kKeep = 64;       // steps between kept states
constexpr int kWalkSteps = 16;  // sequences up to this long take one thread per channel pair

enum : uint32_t { kFlagNone = 0, kFlagAgg = 1, kFlagInc = 2 };

struct alignas(16) LinHeader {
    uint32_t ticket;
    uint32_t status;
    uint32_t pad[62];
};
static_assert(sizeof(LinHeader) == 256, "workspace header is 256 bytes");

struct LinArgs {
    const void* in[4];        // f, x, then forward: z; gradient: dy, z
    long long stride[4];      // elements between steps of each
    const float* h0;          // forward: initial state; gradient: dfinal_state; may be NULL
    float* last;              // forward: final state; gradient: dinitial_state; may be NULL
    const float* first;       // gradient: the forward's initial state, may be NULL
    void* out[3];             // forward: y; gradient: df, dx, dz
    float* keep;              // states entering each 64 steps [ceil(L / 64)][batch][dim]
    LinHeader* head;          // NULL with one tile per sequence
    uint32_t* status;
    uint32_t* flags;          // [tiles][blocks]
    float* agg;               // [tiles][batch][dim][2]
    float* inc;               // [tiles][batch][dim]
    int batch, seqlen, dim;
    int cblocks, blocks, tiles;  // channel blocks, channel blocks x batch, tiles per sequence
    uint32_t spin_limit;
    int drop_first_publish;
    int vec_out;              // dim even: two channels in one store
    int keep_status;          // the status word holds an earlier scan's result to keep
};

// ------------------------------------------------------------- elements

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a = sigmoid(f), om = 1 - a, both to a few ulp: with t = e^-f, a = 1 / (1 + t)
// and om = t / (1 + t).  t stops at 2^126, the largest power whose reciprocal
// is a normal number; there (f < -87) a is taken as exactly 0.
constexpr float kGateZero = 2e-38f;
__device__ __forceinline__ void gate(float f, float& a, float& om) {
    const float t = ex2_approx(min_nan(f * -kLog2e, 126.0f));
    const float r = rcp_approx(1.0f + t);
    om = t * r;
    a = r < kGateZero ? 0.0f : r;
}

// (1 - a) x, 0 where the gate holds the state
__device__ __forceinline__ float input_term(float om, float x) {
    return om == 0.0f ? 0.0f : om * x;
}

// a h + b, b where the gate restarts the state
__device__ __forceinline__ float step(float a, float h, float b) {
    return a == 0.0f ? b : fmaf(a, h, b);
}

template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    __device__ static float2 get(const void* p) {
        const uint32_t w = *static_cast<const uint32_t*>(p);
        return make_float2(bf16lo(w), bf16hi(w));
    }
    __device__ static void put(void* p, float2 v) {
        *static_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
    }
};
template <> struct Pair<float> {
    __device__ static float2 get(const void* p) { return *static_cast<const float2*>(p); }
    __device__ static void put(void* p, float2 v) { *static_cast<float2*>(p) = v; }
};

// two channels of a row in global memory, the second only where it exists
template <typename T>
__device__ __forceinline__ void put2(void* base, size_t i, float2 v, bool both, bool vec) {
    T* p = static_cast<T*>(base) + i;
    if (vec && both) {
        Pair<T>::put(p, v);
    } else {
        p[0] = from_f32<T>(v.x);
        if (both) p[1] = from_f32<T>(v.y);
    }
}

__device__ __forceinline__ float2 load_state2(const float* p, size_t i, bool both) {
    return make_float2(p[i], both ? p[i + 1] : 0.0f);
}

// --------------------------------------------------------------- loading

// BYTES per asynchronous copy (16 or 4), or 0: element loads through registers
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t n) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
                     : "memory");
}

__device__ __forceinline__ void copy_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile of STEPS x 64 channels of one input into shared memory [step][64];
// what lies past the sequence or the channels is filled with zeros.
template <typename T, int STEPS, int BYTES>
__device__ __forceinline__ void load_tile(void* dst, const void* src, long long stride, int b,
                                          int t0, int c0, int seqlen, int dim) {
    constexpr int kUnit = BYTES ? BYTES / (int)sizeof(T) : 1;  // elements per copy
    constexpr int kPerRow = kCh / kUnit;
    const T* base = static_cast<const T*>(src) + (long long)b * seqlen * stride + c0;
#pragma unroll 4
    for (int i = threadIdx.x; i < STEPS * kPerRow; i += kThreads) {
        const int r = i / kPerRow, c = (i % kPerRow) * kUnit;
        const bool in = t0 + r < seqlen && c0 + c < dim;
        const T* p = in ? base + (long long)(t0 + r) * stride + c : static_cast<const T*>(src);
        T* d = static_cast<T*>(dst) + r * kCh + c;
        // a unit lies wholly inside the row or wholly outside: dim is a
        // multiple of it
        if constexpr (BYTES) copy_async<BYTES>(smem_u32(d), p, in ? BYTES : 0);
        else *d = in ? *p : from_f32<T>(0.0f);
    }
}

// ------------------------------------------------------------- look-back

// Warp 0: given the tile's aggregate (P, q) of this lane's two channels, the
// state that enters the tile, from the tiles before it (`seq` counts tiles in
// the order of the scan).  Publishes the aggregate unless the predecessor's
// inclusive state is already there, and the inclusive state unless the tile is
// the last.
__device__ __forceinline__ float2 look_back(const LinArgs& a, int seq, int blk, size_t chan,
                                            bool valid, bool both, float2 P, float2 q) {
    const int lane = threadIdx.x & 31;
    const size_t stride = (size_t)a.batch * a.dim;
    uint32_t* flags = a.flags + blk;
    float2 h = make_float2(0.0f, 0.0f);
    if (seq == 0) {
        if (a.h0 && valid) h = load_state2(a.h0, chan, both);
    } else {
        int j_inc = -1;
        uint32_t f0 = 0;
        if (lane == 0) f0 = ld_acquire_gpu(flags + (size_t)(seq - 1) * a.blocks);
        f0 = __shfl_sync(0xffffffffu, f0, 0);
        bool ok = true;
        if (f0 == kFlagInc) {
            j_inc = seq - 1;
        } else {
            if (valid) {
                float* g = a.agg + ((size_t)seq * stride + chan) * 2;
                __stcg(reinterpret_cast<float2*>(g), make_float2(P.x, q.x));
                if (both) __stcg(reinterpret_cast<float2*>(g) + 1, make_float2(P.y, q.y));
            }
            __syncwarp();
            if (lane == 0) st_release_gpu(flags + (size_t)seq * a.blocks, kFlagAgg);
            int j_hi = seq - 1;
            uint32_t polls = 0, ns = 20;
            while (true) {
                const int j = j_hi - lane;
                uint32_t f = kFlagNone;
                if (j >= 0) f = ld_acquire_gpu(flags + (size_t)j * a.blocks);
                const uint32_t inc_mask = __ballot_sync(0xffffffffu, f == kFlagInc);
                const uint32_t none_mask = __ballot_sync(0xffffffffu, f == kFlagNone);
                const int first = inc_mask ? __ffs(inc_mask) - 1 : 32;
                const uint32_t below = first >= 32 ? 0xffffffffu : ((1u << first) - 1u);
                if ((none_mask & below) == 0) {
                    if (first < 32) { j_inc = j_hi - first; break; }
                    j_hi -= 32;  // 32 aggregates and no inclusive state: further back
                    continue;
                }
                if (++polls >= a.spin_limit) { ok = false; break; }
                __nanosleep(ns);
                ns = ns < 160 ? ns * 2 : 160;
            }
            if (!ok && lane == 0) record_status(a.status, SSM_ERR_TIMEOUT);
        }
        __syncwarp();
        if (ok && valid) {
            const float* s = a.inc + (size_t)j_inc * stride + chan;
            h.x = __ldcg(s);
            if (both) h.y = __ldcg(s + 1);
#pragma unroll 4
            for (int j = j_inc + 1; j < seq; ++j) {
                const float2* g =
                    reinterpret_cast<const float2*>(a.agg + ((size_t)j * stride + chan) * 2);
                const float2 u = __ldcg(g);
                h.x = step(u.x, h.x, u.y);
                if (both) {
                    const float2 w = __ldcg(g + 1);
                    h.y = step(w.x, h.y, w.y);
                }
            }
        }
    }
    const float2 end = make_float2(step(P.x, h.x, q.x), step(P.y, h.y, q.y));
    if (seq == a.tiles - 1) {
        if (a.last && valid) {
            a.last[chan] = end.x;
            if (both) a.last[chan + 1] = end.y;
        }
    } else {
        if (valid) {
            float* s = a.inc + (size_t)seq * stride + chan;
            __stcg(s, end.x);
            if (both) __stcg(s + 1, end.y);
        }
        __syncwarp();
        if (lane == 0 && !(a.drop_first_publish && seq == 0))
            st_release_gpu(flags + (size_t)seq * a.blocks, kFlagInc);
    }
    return h;
}

// ---------------------------------------------------------- tile kernels

// Shared memory of one CTA: the ring of input tiles, the warps' aggregates
// (forward P, q; gradient also the reverse q) and the tile's entry state.
template <typename T, int S, int NIN, int STAGES>
struct LinSmem {
    static constexpr int kTile = kWarps * S * kCh * (int)sizeof(T);
    static constexpr int kStage = NIN * kTile;
};

// GRAD false: inputs f, x[, z], output y.  GRAD true: inputs f, x, dy[, z],
// outputs df, dx[, dz].
template <typename T, typename TO, int S, int STAGES, int BYTES, bool GATED, bool GRAD>
__global__ void __launch_bounds__(kThreads, 2) linrec_tile_kernel(const LinArgs a) {
    constexpr int NIN = (GRAD ? 3 : 2) + (GATED ? 1 : 0);
    constexpr int STEPS = kWarps * S;
    using SM = LinSmem<T, S, NIN, STAGES>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 s_P[kWarps][32], s_q[kWarps][32], s_r[GRAD ? kWarps : 1][32];
    __shared__ float2 s_h[32];
    __shared__ int s_item[STAGES + 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int items = a.blocks * a.tiles;
    int own = blockIdx.x;  // without tickets: blockIdx.x, + gridDim.x, ...

    auto next_item = [&]() -> int {  // thread 0
        if (a.head) return (int)min(atomicAdd(&a.head->ticket, 1u), 0x7fffffffu);
        const int i = own;
        own = own < items ? own + (int)gridDim.x : own;
        return i;
    };
    auto fetch = [&](int item, int stage) {
        if (item < items) {
            const int seq = item / a.blocks, blk = item % a.blocks;
            const int tile = GRAD ? a.tiles - 1 - seq : seq;
            const int b = blk / a.cblocks, c0 = (blk % a.cblocks) * kCh;
#pragma unroll
            for (int i = 0; i < NIN; ++i)
                load_tile<T, STEPS, BYTES>(smem + stage * SM::kStage + i * SM::kTile, a.in[i],
                                           a.stride[i], b, tile * STEPS, c0, a.seqlen, a.dim);
        }
        copy_commit();
    };

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) s_item[i] = next_item();
        // one tile per sequence: no waits, so nothing else writes the status
        if (!a.head && blockIdx.x == 0 && !a.keep_status) *a.status = 0;
    }
    __syncthreads();
    int queue[STAGES];  // this tile and the ones being fetched
#pragma unroll
    for (int i = 0; i < STAGES; ++i) queue[i] = s_item[i];
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(queue[i], i);

    for (int turn = 0; queue[0] < items; ++turn) {
        const int stage = turn % STAGES;
        copy_wait<STAGES - 2>();
        __syncthreads();  // the tile is there; the previous one is done with
        int ahead = 0;
        if (tid == 0) ahead = next_item();  // read back after the next barriers
        fetch(queue[STAGES - 1], (turn + STAGES - 1) % STAGES);

        const int seq = queue[0] / a.blocks, blk = queue[0] % a.blocks;
        const int tile = GRAD ? a.tiles - 1 - seq : seq;
        const int b = blk / a.cblocks, c = (blk % a.cblocks) * kCh + lane * 2;
        const bool valid = c < a.dim, both = c + 1 < a.dim;
        const size_t chan = (size_t)b * a.dim + c;
        const int t0 = tile * STEPS + warp * S;
        const uint8_t* base = smem + stage * SM::kStage;
        auto at = [&](int i, int k) -> const void* {
            return base + i * SM::kTile + ((warp * S + k) * kCh + lane * 2) * (int)sizeof(T);
        };

        // the state entering the tile, for the gradient's replay
        float2 hk = make_float2(0.0f, 0.0f);
        if constexpr (GRAD) {
            if (valid) {
                if (tile * STEPS > 0)
                    hk = load_state2(a.keep + (size_t)(tile * STEPS / kKeep) * a.batch * a.dim,
                                     chan, both);
                else if (a.first)
                    hk = load_state2(a.first, chan, both);
            }
        }

        // ---- the warp's steps from zero
        float2 ga[S], gb[S];  // a_t, and b_t (forward) or 1 - a_t (gradient)
        float2 P = make_float2(1.0f, 1.0f), q = make_float2(0.0f, 0.0f);
        float2 r = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const float2 f = Pair<T>::get(at(0, k)), x = Pair<T>::get(at(1, k));
            float2 om, bt;
            gate(f.x, ga[k].x, om.x);
            gate(f.y, ga[k].y, om.y);
            if (t0 + k >= a.seqlen) {
                ga[k] = make_float2(1.0f, 1.0f);
                om = make_float2(0.0f, 0.0f);
            }
            bt.x = input_term(om.x, x.x);
            bt.y = input_term(om.y, x.y);
            gb[k] = GRAD ? om : bt;
            q.x = step(ga[k].x, q.x, bt.x);
            q.y = step(ga[k].y, q.y, bt.y);
            P.x *= ga[k].x;
            P.y *= ga[k].y;
        }
        // dh_t = dy_t silu(z_t), 0 past the sequence (the tile is zero there)
        auto grad_in = [&](int k) -> float2 {
            float2 d = Pair<T>::get(at(2, k));
            if constexpr (GATED) {
                const float2 z = Pair<T>::get(at(3, k));
                d.x *= silu_f(z.x);
                d.y *= silu_f(z.y);
            }
            return d;
        };
        if constexpr (GRAD) {
#pragma unroll
            for (int k = S - 1; k >= 0; --k) {
                const float2 d = grad_in(k);
                r.x = step(ga[k].x, r.x + d.x, 0.0f);
                r.y = step(ga[k].y, r.y + d.y, 0.0f);
            }
            s_r[warp][lane] = r;
        }
        s_P[warp][lane] = P;
        s_q[warp][lane] = q;
        __syncthreads();

        // ---- across warps and tiles
        if (warp == 0) {
            float2 TP = make_float2(1.0f, 1.0f), tq = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const int w = GRAD ? kWarps - 1 - i : i;
                const float2 p = s_P[w][lane], v = GRAD ? s_r[w][lane] : s_q[w][lane];
                tq.x = step(p.x, tq.x, v.x);
                tq.y = step(p.y, tq.y, v.y);
                TP.x *= p.x;
                TP.y *= p.y;
            }
            s_h[lane] = look_back(a, seq, blk, chan, valid, both, TP, tq);
            if (tid == 0) s_item[STAGES] = ahead;
        }
        __syncthreads();

        if constexpr (!GRAD) {
            float2 h = s_h[lane];
            for (int w = 0; w < warp; ++w) {
                const float2 p = s_P[w][lane], v = s_q[w][lane];
                h.x = step(p.x, h.x, v.x);
                h.y = step(p.y, h.y, v.y);
            }
            if (a.keep && valid && t0 % kKeep == 0 && t0 < a.seqlen) {
                float* s = a.keep + (size_t)(t0 / kKeep) * a.batch * a.dim + chan;
                s[0] = h.x;
                if (both) s[1] = h.y;
            }
            if (a.out[0]) {
                const size_t o = ((size_t)b * a.seqlen + t0) * a.dim + c;
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    h.x = step(ga[k].x, h.x, gb[k].x);
                    h.y = step(ga[k].y, h.y, gb[k].y);
                    float2 y = h;
                    if constexpr (GATED) {
                        const float2 z = Pair<T>::get(at(2, k));
                        y.x *= silu_f(z.x);
                        y.y *= silu_f(z.y);
                    }
                    if (valid && t0 + k < a.seqlen)
                        put2<TO>(a.out[0], o + (size_t)k * a.dim, y, both, a.vec_out);
                }
            }
        } else {
            float2 h = hk, mu = s_h[lane];
            for (int w = 0; w < warp; ++w) {
                const float2 p = s_P[w][lane], v = s_q[w][lane];
                h.x = step(p.x, h.x, v.x);
                h.y = step(p.y, h.y, v.y);
            }
            for (int w = kWarps - 1; w > warp; --w) {
                const float2 p = s_P[w][lane], v = s_r[w][lane];
                mu.x = step(p.x, mu.x, v.x);
                mu.y = step(p.y, mu.y, v.y);
            }
            float2 before[S];  // h_{t-1}
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const float2 x = Pair<T>::get(at(1, k));
                before[k] = h;
                h.x = step(ga[k].x, h.x, input_term(gb[k].x, x.x));
                h.y = step(ga[k].y, h.y, input_term(gb[k].y, x.y));
            }
            const size_t o = ((size_t)b * a.seqlen + t0) * a.dim + c;
#pragma unroll
            for (int k = S - 1; k >= 0; --k) {
                const bool in = valid && t0 + k < a.seqlen;
                const size_t ok = o + (size_t)k * a.dim;
                const float2 x = Pair<T>::get(at(1, k));
                float2 d = Pair<T>::get(at(2, k));
                if constexpr (GATED) {
                    const float2 z = Pair<T>::get(at(3, k));
                    float2 dz;
                    float sg = rcp_approx(1.0f + ex2_approx(z.x * -kLog2e));
                    dz.x = d.x * h.x * sg * fmaf(z.x, 1.0f - sg, 1.0f);
                    d.x *= z.x * sg;
                    sg = rcp_approx(1.0f + ex2_approx(z.y * -kLog2e));
                    dz.y = d.y * h.y * sg * fmaf(z.y, 1.0f - sg, 1.0f);
                    d.y *= z.y * sg;
                    if (in) put2<TO>(a.out[2], ok, dz, both, a.vec_out);
                }
                const float2 lam = make_float2(d.x + mu.x, d.y + mu.y);
                float2 df, dx;
                dx.x = gb[k].x == 0.0f ? 0.0f : lam.x * gb[k].x;
                dx.y = gb[k].y == 0.0f ? 0.0f : lam.y * gb[k].y;
                const float sx = ga[k].x * gb[k].x, sy = ga[k].y * gb[k].y;
                df.x = sx == 0.0f ? 0.0f : lam.x * (before[k].x - x.x) * sx;
                df.y = sy == 0.0f ? 0.0f : lam.y * (before[k].y - x.y) * sy;
                if (in) {
                    put2<TO>(a.out[0], ok, df, both, a.vec_out);
                    put2<TO>(a.out[1], ok, dx, both, a.vec_out);
                }
                mu.x = step(ga[k].x, lam.x, 0.0f);
                mu.y = step(ga[k].y, lam.y, 0.0f);
                h = before[k];
            }
        }
#pragma unroll
        for (int i = 0; i + 1 < STAGES; ++i) queue[i] = queue[i + 1];
        queue[STAGES - 1] = s_item[STAGES];
    }
    copy_wait<0>();
}

// -------------------------------------------------------- short sequences

// One thread walks the steps of two channels: a decode step (one token) is a
// single pass over the states.
template <typename T, typename TO, bool VEC, bool GATED>
__global__ void __launch_bounds__(128) linrec_walk_kernel(const LinArgs a) {
    const int pairs = (a.dim + 1) / 2;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i == 0 && !a.keep_status) *a.status = 0;
    if (i >= (long long)a.batch * pairs) return;
    const int b = (int)(i / pairs), c = (int)(i % pairs) * 2;
    const bool both = c + 1 < a.dim;
    const size_t chan = (size_t)b * a.dim + c;
    auto get = [&](int k, int t) -> float2 {
        const T* p = static_cast<const T*>(a.in[k]) + ((long long)b * a.seqlen + t) * a.stride[k] + c;
        if constexpr (VEC) return Pair<T>::get(p);
        return make_float2(to_f32(p[0]), both ? to_f32(p[1]) : 0.0f);
    };
    float2 h = make_float2(0.0f, 0.0f);
    if (a.h0) h = load_state2(a.h0, chan, both);
    if (a.keep && a.seqlen > 0) {
        a.keep[chan] = h.x;
        if (both) a.keep[chan + 1] = h.y;
    }
#pragma unroll 2
    for (int t = 0; t < a.seqlen; ++t) {
        const float2 f = get(0, t), x = get(1, t);
        float2 g, om, y;
        gate(f.x, g.x, om.x);
        gate(f.y, g.y, om.y);
        h.x = step(g.x, h.x, input_term(om.x, x.x));
        h.y = step(g.y, h.y, input_term(om.y, x.y));
        y = h;
        if constexpr (GATED) {
            const float2 z = get(2, t);
            y.x *= silu_f(z.x);
            y.y *= silu_f(z.y);
        }
        if (a.out[0])
            put2<TO>(a.out[0], ((size_t)b * a.seqlen + t) * a.dim + c, y, both, a.vec_out);
    }
    if (a.last) {
        a.last[chan] = h.x;
        if (both) a.last[chan + 1] = h.y;
    }
}

// ---------------------------------------------------------------- launch

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// Steps of a forward tile by type: 128 of bf16 or 64 of fp32 are 16 KB of one
// input; the gradient keeps three values per step in registers, so 64.
constexpr int kFwdStepsBf16 = 128, kFwdStepsF32 = 64, kBwdSteps = 64;

int tiles_of(int seqlen, int steps) { return (seqlen + steps - 1) / steps; }

// header, flags, aggregates and inclusive states of `tiles` tiles
size_t scan_bytes(int batch, int dim, int tiles) {
    const size_t blocks = (size_t)batch * ((dim + kCh - 1) / kCh);
    return 256 + (tiles > 1 ? round256((size_t)tiles * blocks * 4) +
                                  round256((size_t)tiles * batch * dim * 8) +
                                  round256((size_t)tiles * batch * dim * 4)
                            : 0);
}

bool sizes_ok(int batch, int seqlen, int dim) { return batch >= 0 && seqlen >= 0 && dim >= 0; }

// one int counts the tiles of all blocks, with room for the tickets past the end
bool sizes_fit(int batch, int seqlen, int dim) {
    const double blocks = (double)batch * ((dim + kCh - 1) / kCh);
    return blocks * tiles_of(seqlen, 64) < 2.0e9 && (double)batch * dim < 2.0e9;
}

// Fills in the work area of one scan; returns the bytes it takes.
size_t place(LinArgs& a, uint8_t* ws, int tiles) {
    a.cblocks = (a.dim + kCh - 1) / kCh;
    a.blocks = a.batch * a.cblocks;
    a.tiles = tiles;
    a.status = reinterpret_cast<uint32_t*>(ws) + 1;
    const size_t need = scan_bytes(a.batch, a.dim, tiles);
    if (tiles > 1) {
        a.head = reinterpret_cast<LinHeader*>(ws);
        size_t o = 256;
        a.flags = reinterpret_cast<uint32_t*>(ws + o);
        o += round256((size_t)tiles * a.blocks * 4);
        a.agg = reinterpret_cast<float*>(ws + o);
        o += round256((size_t)tiles * a.batch * a.dim * 8);
        a.inc = reinterpret_cast<float*>(ws + o);
    }
    return need;
}

bool set_smem(const void* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
           cudaSuccess;
}

template <typename T, typename TO, int S, int BYTES, bool GATED, bool GRAD>
bool launch_tile(const LinArgs& a, cudaStream_t s) {
    constexpr int NIN = (GRAD ? 3 : 2) + (GATED ? 1 : 0);
    // the ring fills about half of an SM's shared memory
    constexpr int kTile = LinSmem<T, S, NIN, 1>::kStage;
    constexpr int STAGES = BYTES == 0 ? 2 : kTile * 3 <= 100 * 1024 ? 3 : 2;
    constexpr int smem = STAGES * kTile;
    auto kernel = linrec_tile_kernel<T, TO, S, STAGES, BYTES, GATED, GRAD>;
    if (!set_smem(reinterpret_cast<const void*>(kernel), smem)) return false;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return false;
    const long long items = (long long)a.blocks * a.tiles;
    const unsigned grid = (unsigned)std::min<long long>(items, 2ll * sms);
    if (a.head) {
        // header and flags are neighbours; an earlier scan's status stays
        const size_t flags = round256((size_t)a.tiles * a.blocks * 4);
        if (a.keep_status) {
            if (cudaMemsetAsync(&a.head->ticket, 0, sizeof(uint32_t), s) != cudaSuccess ||
                cudaMemsetAsync(a.flags, 0, flags, s) != cudaSuccess)
                return false;
        } else if (cudaMemsetAsync(a.head, 0, sizeof(LinHeader) + flags, s) != cudaSuccess) {
            return false;
        }
    }
    kernel<<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

template <typename T, typename TO, int S, bool GRAD>
bool launch_by(const LinArgs& a, int bytes, bool gated, cudaStream_t s) {
    if (bytes == 16)
        return gated ? launch_tile<T, TO, S, 16, true, GRAD>(a, s)
                     : launch_tile<T, TO, S, 16, false, GRAD>(a, s);
    if (bytes == 4)
        return gated ? launch_tile<T, TO, S, 4, true, GRAD>(a, s)
                     : launch_tile<T, TO, S, 4, false, GRAD>(a, s);
    if constexpr (sizeof(T) == 2)
        return gated ? launch_tile<T, TO, S, 0, true, GRAD>(a, s)
                     : launch_tile<T, TO, S, 0, false, GRAD>(a, s);
    return false;
}

// The widest copy every row of every input allows: 16 bytes, 4, or elements.
int copy_bytes(const LinArgs& a, int n, size_t es) {
    for (int unit : {16, 4}) {
        bool ok = (size_t)a.dim * es % unit == 0;
        for (int i = 0; i < n; ++i)
            ok = ok && reinterpret_cast<uintptr_t>(a.in[i]) % unit == 0 &&
                 (size_t)a.stride[i] * es % unit == 0;
        if (ok) return unit;
    }
    return 0;
}

template <typename T, typename TO>
bool launch_walk(const LinArgs& a, bool vec, bool gated, cudaStream_t s) {
    const long long n = (long long)a.batch * ((a.dim + 1) / 2);
    const unsigned grid = (unsigned)((n + 127) / 128);
    auto go = [&](auto kernel) { kernel<<<grid, 128, 0, s>>>(a); };
    if (vec) gated ? go(linrec_walk_kernel<T, TO, true, true>)
                   : go(linrec_walk_kernel<T, TO, true, false>);
    else gated ? go(linrec_walk_kernel<T, TO, false, true>)
               : go(linrec_walk_kernel<T, TO, false, false>);
    return cudaGetLastError() == cudaSuccess;
}

template <typename F>
bool by_types(ssm_dtype_t in, ssm_dtype_t out, F&& f) {
    using B = __nv_bfloat16;
    if (in == SSM_F32) return out == SSM_F32 ? f(float{}, float{}) : f(float{}, B{});
    return out == SSM_F32 ? f(B{}, float{}) : f(B{}, B{});
}

// The forward scan (a.out[0] may be NULL: states only).
bool run_forward(LinArgs& a, ssm_dtype_t in, ssm_dtype_t out, bool gated, cudaStream_t s) {
    const size_t es = ssm_host::dtype_size(in);
    const int nin = gated ? 3 : 2;
    return by_types(in, out, [&](auto ti, auto to) -> bool {
        using T = decltype(ti);
        using TO = decltype(to);
        if (a.seqlen <= kWalkSteps) {
            // two channels in one load: 2 * es bytes
            bool vec = a.dim % 2 == 0;
            for (int i = 0; i < nin; ++i)
                vec = vec && reinterpret_cast<uintptr_t>(a.in[i]) % (2 * es) == 0 &&
                      a.stride[i] % 2 == 0;
            return launch_walk<T, TO>(a, vec, gated, s);
        }
        constexpr int S = (sizeof(T) == 2 ? kFwdStepsBf16 : kFwdStepsF32) / kWarps;
        return launch_by<T, TO, S, false>(a, copy_bytes(a, nin, es), gated, s);
    });
}

int fwd_tiles(int seqlen, ssm_dtype_t in) {
    return seqlen <= kWalkSteps ? 1
                                : tiles_of(seqlen, in == SSM_BF16 ? kFwdStepsBf16 : kFwdStepsF32);
}

struct Span { const void* p; size_t n; };

// bytes that `steps` rows of `dim` elements `stride` apart cover
size_t strided_bytes(long long steps, int dim, long long stride, size_t es) {
    return steps > 0 ? ((size_t)(steps - 1) * stride + dim) * es : 0;
}

}  // namespace

extern "C" size_t ssm_linrec_checkpoint_bytes(int batch, int seqlen, int dim) {
    if (!sizes_ok(batch, seqlen, dim)) return 0;
    return (size_t)tiles_of(seqlen, kKeep) * batch * dim * 4;
}

extern "C" size_t ssm_linrec_workspace_bytes(int batch, int seqlen, int dim) {
    if (!sizes_ok(batch, seqlen, dim) || !sizes_fit(batch, seqlen, dim)) return 0;
    return scan_bytes(batch, dim, tiles_of(seqlen, 64));
}

extern "C" size_t ssm_linrec_bwd_workspace_bytes(int batch, int seqlen, int dim) {
    if (!sizes_ok(batch, seqlen, dim) || !sizes_fit(batch, seqlen, dim)) return 0;
    return scan_bytes(batch, dim, tiles_of(seqlen, 64)) +
           round256(ssm_linrec_checkpoint_bytes(batch, seqlen, dim));
}

extern "C" ssm_status_t ssm_linrec_fwd(const void* f, const void* x, const void* z,
                                       long long f_stride, long long x_stride,
                                       long long z_stride, const float* initial_state, void* y,
                                       float* final_state, float* checkpoints, int batch,
                                       int seqlen, int dim, ssm_dtype_t in_dtype,
                                       ssm_dtype_t out_dtype, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    using namespace ssm_host;
    if (!sizes_ok(batch, seqlen, dim)) return SSM_ERR_SHAPE;
    if (f_stride < dim || x_stride < dim || (z && z_stride < dim)) return SSM_ERR_SHAPE;
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return SSM_ERR_DTYPE;
    if (!sizes_fit(batch, seqlen, dim)) return SSM_ERR_UNSUPPORTED;
    const size_t states = (size_t)batch * dim;
    if (states == 0) return SSM_OK;
    if (seqlen > 0 && (!f || !x || !y)) return SSM_ERR_NULL;
    if (!workspace || workspace_bytes < ssm_linrec_workspace_bytes(batch, seqlen, dim))
        return SSM_ERR_WORKSPACE;
    const size_t es = dtype_size(in_dtype);
    for (const void* p : {(const void*)initial_state, (const void*)y, (const void*)final_state,
                          (const void*)checkpoints, (const void*)workspace})
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    for (const void* p : {f, x, z})
        if (reinterpret_cast<uintptr_t>(p) % es) return SSM_ERR_ALIGN;
    const long long steps = (long long)batch * seqlen;
    const Span ins[] = {{f, strided_bytes(steps, dim, f_stride, es)},
                        {x, strided_bytes(steps, dim, x_stride, es)},
                        {z, strided_bytes(steps, dim, z_stride, es)},
                        {initial_state, states * 4}};
    const Span outs[] = {{y, (size_t)steps * dim * dtype_size(out_dtype)},
                         {final_state, states * 4},
                         {checkpoints, ssm_linrec_checkpoint_bytes(batch, seqlen, dim)},
                         {workspace, ssm_linrec_workspace_bytes(batch, seqlen, dim)}};
    for (const Span& o : outs)
        for (const Span& i : ins) {
            // the state may be updated in place
            if (o.p == final_state && i.p == initial_state && final_state == initial_state)
                continue;
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
        }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;

    LinArgs a{};
    a.in[0] = f; a.in[1] = x; a.in[2] = z;
    a.stride[0] = f_stride; a.stride[1] = x_stride; a.stride[2] = z_stride;
    a.h0 = initial_state; a.last = final_state; a.keep = checkpoints; a.out[0] = y;
    a.batch = batch; a.seqlen = seqlen; a.dim = dim;
    a.vec_out = dim % 2 == 0;
    ssm_internal::lookback_setting(&a.spin_limit, &a.drop_first_publish);
    place(a, static_cast<uint8_t*>(workspace), fwd_tiles(seqlen, in_dtype));
    return run_forward(a, in_dtype, out_dtype, z != nullptr, static_cast<cudaStream_t>(stream))
               ? SSM_OK : SSM_ERR_CUDA;
}

extern "C" ssm_status_t ssm_linrec_bwd(const void* f, const void* x, const void* z,
                                       long long f_stride, long long x_stride,
                                       long long z_stride, const float* initial_state,
                                       const void* dy, const float* dfinal_state,
                                       const float* checkpoints, void* df, void* dx, void* dz,
                                       float* dinitial_state, int batch, int seqlen, int dim,
                                       ssm_dtype_t in_dtype, ssm_dtype_t grad_dtype,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ssm_host;
    if (!sizes_ok(batch, seqlen, dim)) return SSM_ERR_SHAPE;
    if (f_stride < dim || x_stride < dim || (z && z_stride < dim)) return SSM_ERR_SHAPE;
    if (!dtype_ok(in_dtype) || !dtype_ok(grad_dtype)) return SSM_ERR_DTYPE;
    if (!sizes_fit(batch, seqlen, dim)) return SSM_ERR_UNSUPPORTED;
    const size_t states = (size_t)batch * dim;
    if (states == 0) return SSM_OK;
    if (seqlen > 0 && (!f || !x || !dy || !df || !dx || (z && !dz))) return SSM_ERR_NULL;
    if (!workspace || workspace_bytes < ssm_linrec_bwd_workspace_bytes(batch, seqlen, dim))
        return SSM_ERR_WORKSPACE;
    const size_t es = dtype_size(in_dtype);
    for (const void* p : {(const void*)initial_state, dy, (const void*)dfinal_state,
                          (const void*)checkpoints, (const void*)df, (const void*)dx,
                          (const void*)dz, (const void*)dinitial_state, (const void*)workspace})
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    for (const void* p : {f, x, z})
        if (reinterpret_cast<uintptr_t>(p) % es) return SSM_ERR_ALIGN;
    const long long steps = (long long)batch * seqlen;
    const size_t gb = (size_t)steps * dim * dtype_size(grad_dtype);
    const size_t kept = ssm_linrec_checkpoint_bytes(batch, seqlen, dim);
    const Span ins[] = {{f, strided_bytes(steps, dim, f_stride, es)},
                        {x, strided_bytes(steps, dim, x_stride, es)},
                        {z, strided_bytes(steps, dim, z_stride, es)},
                        {dy, (size_t)steps * dim * es},
                        {initial_state, states * 4},
                        {dfinal_state, states * 4},
                        {checkpoints, kept}};
    const Span outs[] = {{df, gb}, {dx, gb}, {z ? dz : nullptr, gb},
                         {dinitial_state, states * 4},
                         {workspace, ssm_linrec_bwd_workspace_bytes(batch, seqlen, dim)}};
    for (const Span& o : outs)
        for (const Span& i : ins) {
            if (o.p == dinitial_state && i.p == dfinal_state && dinitial_state == dfinal_state)
                continue;
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
        }
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    LinArgs a{};
    a.in[0] = f; a.in[1] = x;
    a.stride[0] = f_stride; a.stride[1] = x_stride;
    a.batch = batch; a.seqlen = seqlen; a.dim = dim;
    a.vec_out = dim % 2 == 0;
    ssm_internal::lookback_setting(&a.spin_limit, &a.drop_first_publish);
    if (!checkpoints && seqlen > 0) {
        // the forward again, states only
        LinArgs w = a;
        w.h0 = initial_state;
        w.keep = reinterpret_cast<float*>(ws + scan_bytes(batch, dim, tiles_of(seqlen, 64)));
        place(w, ws, fwd_tiles(seqlen, in_dtype));
        if (!run_forward(w, in_dtype, in_dtype, false, s)) return SSM_ERR_CUDA;
        checkpoints = w.keep;
        a.keep_status = 1;
    }
    a.in[2] = dy; a.stride[2] = dim;
    a.in[3] = z; a.stride[3] = z_stride;
    a.h0 = dfinal_state; a.last = dinitial_state; a.first = initial_state;
    a.keep = const_cast<float*>(checkpoints);
    a.out[0] = df; a.out[1] = dx; a.out[2] = dz;
    if (seqlen == 0) {
        if (!dinitial_state || dinitial_state == dfinal_state) return SSM_OK;
        const cudaError_t e =
            dfinal_state ? cudaMemcpyAsync(dinitial_state, dfinal_state, states * 4,
                                           cudaMemcpyDeviceToDevice, s)
                         : cudaMemsetAsync(dinitial_state, 0, states * 4, s);
        return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
    }
    place(a, ws, tiles_of(seqlen, kBwdSteps));
    const bool ok = by_types(in_dtype, grad_dtype, [&](auto ti, auto to) -> bool {
        using T = decltype(ti);
        using TO = decltype(to);
        return launch_by<T, TO, kBwdSteps / kWarps, true>(a, copy_bytes(a, z ? 4 : 3, es),
                                                          z != nullptr, s);
    });
    return ok ? SSM_OK : SSM_ERR_CUDA;
}
