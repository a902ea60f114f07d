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
//  * A CTA takes a tile of 128 steps (gradient, and rows that are not 16-byte
//    aligned: 64) by 64 channels; each of its 8 (bf16) or 16 (fp32) warps takes
//    consecutive steps, a lane two neighbouring channels, so a warp's access to a
//    step is one row segment of 64 channels.  Inputs come through a ring of shared
//    memory tiles, by TMA where every row is 16-byte aligned, else by cp.async in
//    16-byte pieces at each row's own shift, so the next tile's loads are in
//    flight while this one waits for its predecessors; results go back in place
//    and out by TMA, or by their warps.
//  * Each warp scans its steps from zero, keeping a_t and b_t in registers;
//    the warps' (P, q) meet in shared memory; tiles chain through a decoupled
//    look-back (Merrill and Garland's single-pass prefix scan).  The published
//    values are their own flags (a pattern no result has means "not yet"), so a
//    look-back is one round trip through L2 instead of two, and the warps look at
//    the 7 to 15 tiles before theirs at once.
//    The grid is what the GPU holds at once (a cooperative launch) and CTA i
//    takes tiles i, i + grid, ..., so that the tiles in work are always
//    consecutive ones and a predecessor is running or done; every wait is bounded
//    (SSM_ERR_TIMEOUT).  (Tiles drawn from a counter, two ahead for the loads,
//    left gaps of drawn but unstarted tiles that everything behind waited for:
//    786 us against 470 us for 65536 steps of 1536 channels.)
//  * Each warp then replays its steps from its entry state and writes y.
//  * Masked steps (below) cost comparisons at every step, 45 instructions an
//    element in all; a warp whose gates all lie within |f| < 80, where no step can
//    be masked, takes a path without them.
// The gradient is the same scan of (a_t, a_t dh_t) in reverse order.  The states
// it needs are not stored but taken again: the forward keeps the state before every
// 64th step in fp32, and each tile replays its own steps from there.
//
// Masked steps: a gate of +inf holds the state whatever x is there (b_t = 0 where
// 1 - a_t = 0), a gate of -inf restarts it whatever it was (a_t = 0 drops h, NaN
// and infinities too); their gradients are 0.  A span's decay is 0 only where one of its
// gates is.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "scan_internal.h"
#include "tcgen05.cuh"

namespace {

using namespace ssm;

constexpr int kKeep = 64;       // steps between kept states, and of a gradient's tile
constexpr int kCh = 64;         // channels per tile, two per lane
constexpr int kWalkSteps = 16;  // sequences up to this long take one thread per channel pair
constexpr float kFastGate = 80.0f;

struct alignas(16) LinHeader {
    uint32_t unused;
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
    float* keep;              // states entering every 64 steps [ceil(L / 64)][batch][dim]
    uint32_t* status;
    uint32_t* clear;          // the status word, if the tile kernel has to clear it
    ulonglong2* agg;          // [tiles][blocks][32]: (P, q) of two channels
    uint2* inc;               // [tiles][blocks][32]: the state after the tile
    int batch, seqlen, dim;
    int cblocks, blocks, tiles;  // channel blocks, channel blocks x batch, tiles per sequence
    uint32_t cblocks_inv;        // 2^32 / cblocks, rounded up
    uint32_t spin_limit;
    int drop_first_publish;
    int keep_status;          // the status word holds an earlier scan's result to keep
};

struct LinMaps {
    CUtensorMap in[4], out[3];
};

// ------------------------------------------------------------- elements

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a = sigmoid(f) to 2 ulp, and om = 1 - a, by the multi-function unit's approximate power and
// reciprocal (exact forms would cost more than the rest of a step): with t = e^-f, a = 1 /
// (1 + t) and om = t / (1 + t).  t's exponent is rounded once, which is |f| 2^-24 of t and
// of om: 20 ulp at f = 40.  t stops at 2^126, the largest power whose reciprocal is a normal
// number; there (f < -87) a is taken as exactly 0.
//   An a close to 1 is a multiple of 2^-24, so that a channel's memory 1 / (1 - a) is off
// by up to 2^-25 / (1 - a), as in any fp32 recurrence with a gate rounded to fp32: a
// constant gate's states over 65536 steps are within 2e-5 of the definition's largest at
// f = 6, 5e-4 at f = 10 and 1.7e-3 at f = 12 (a serial fp32 loop with correctly rounded
// gates: 1.2e-5, 4e-4 and 4e-4).
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

// a lane's two channels of a state, APART elements apart, the second only where it exists
template <int APART>
__device__ __forceinline__ float2 load_state2(const float* p, size_t i, bool both) {
    return make_float2(p[i], both ? p[i + APART] : 0.0f);
}
template <int APART>
__device__ __forceinline__ void store_state2(float* p, size_t i, float2 v, bool both) {
    p[i] = v.x;
    if (both) p[i + APART] = v.y;
}

// --------------------------------------------------------------- loading

// 16 bytes of which the first n come from memory, the rest are zeros
__device__ __forceinline__ void copy_async(uint32_t dst, uintptr_t src, uint32_t n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}

__device__ __forceinline__ void copy_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows that are not 16-byte aligned: a tile's row is copied from the 16-byte boundary
// before it, in 16-byte pieces (16 bytes with their part of the row are
// always memory of the tensor's own).  From a row to the next its start moves by d, the
// stride's bytes mod 16, against the boundaries; rows lie kShiftedRow + d apart, so that
// pieces stay on boundaries and a step's address is linear in it.  A lane has channels
// lane and lane + 32: neighbours would straddle words.  (4-byte copies took 99 us, element
// loads 324 us for the forward of batch 8, 2048 steps, 1500 and 1501 channels of bf16 with
// a gate; rows kShiftedRow apart and neighbouring channels 88 us; this 82 us.)
template <typename T>
constexpr int kShiftedRow = kCh * (int)sizeof(T) + 16;
template <typename T>
constexpr int kPieces = kShiftedRow<T> / 16;

// where a row's 64 channels start behind the boundary
__device__ __forceinline__ uint32_t shift_of(const void* base, long long at, int es) {
    return (uint32_t)(reinterpret_cast<uintptr_t>(base) + at * es) & 15u;
}

template <typename T, int STEPS, int THREADS>
__device__ __forceinline__ void load_shifted(void* dst, const void* src, long long stride, int b,
                                             int t0, int c0, int seqlen, int dim) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(src) +
                            (((long long)b * seqlen + t0) * stride + c0) * (long long)sizeof(T);
    const uint32_t bytes = min(kCh, dim - c0) * (int)sizeof(T);
    // THREADS / STEPS neighbouring threads to a row, every so many-th piece each
    constexpr int PER = THREADS / STEPS;
    const int r = threadIdx.x / PER, q = threadIdx.x % PER;
    const uintptr_t at = first + r * stride * (long long)sizeof(T);
    const uintptr_t from = at & ~uintptr_t(15);
    // bytes behind the boundary, none past the sequence
    const int end = t0 + r < seqlen ? (int)((uint32_t)(at & 15) + bytes) : 0;
    const uint32_t d = (uint32_t)(stride * (long long)sizeof(T)) & 15;
    const uint32_t to = smem_u32(dst) + r * kShiftedRow<T> + (((uint32_t)(first & 15) + r * d) & ~15u);
#pragma unroll
    for (int j0 = 0; j0 < kPieces<T>; j0 += PER) {
        const int j = j0 + q, n = max(0, min(16, end - j * 16));
        if (j < kPieces<T>)
            copy_async(to + j * 16, n > 0 ? from + j * 16 : reinterpret_cast<uintptr_t>(src) & ~uintptr_t(15), n);
    }
}

// channels lane and lane + 32 of a row
template <typename T>
__device__ __forceinline__ float2 get_shifted(const uint8_t* at) {
    const T* p = reinterpret_cast<const T*>(at);
    return make_float2(to_f32(p[0]), to_f32(p[32]));
}
template <typename T>
__device__ __forceinline__ void put_shifted(uint8_t* at, float2 v) {
    T* p = reinterpret_cast<T*>(at);
    p[0] = from_f32<T>(v.x);
    p[32] = from_f32<T>(v.y);
}

// A warp's `rows` rows (of S) of results out of shared memory (row r in the place of an
// input's row, whose start moved by `d` from `shift`, at its own offset behind the 16-byte
// boundary before its place in memory): whole 16 bytes where they are the row's, else
// element by element.
template <typename T, int S>
__device__ __forceinline__ void send_shifted(const uint8_t* smem, uint32_t shift, uint32_t d,
                                             void* out, size_t first, int dim, int rows,
                                             int channels, int lane) {
    // 32 / S neighbouring lanes to a row: its whole pieces, then the elements before
    // the first and after the last
    constexpr int PER = 32 / S, ES = (int)sizeof(T), kEdge = 16 / ES;
    const int r = lane / PER, q = lane % PER;
    if (r >= rows) return;
    uint8_t* p = reinterpret_cast<uint8_t*>(static_cast<T*>(out) + first + (size_t)r * dim);
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15), end = off + channels * ES;
    p -= off;
    const uint8_t* s = smem + r * kShiftedRow<T> + ((shift + r * d) & ~15u);
#pragma unroll
    for (int j0 = 0; j0 < kPieces<T>; j0 += PER) {
        const int j = (j0 + q) * 16;
        if (j >= off && j + 16 <= end)
            *reinterpret_cast<uint4*>(p + j) = *reinterpret_cast<const uint4*>(s + j);
    }
    // up to kEdge - 1 elements at either end
    const int head = min((off + 15) & ~15, end), tail = max(end & ~15, head);
#pragma unroll
    for (int e0 = 0; e0 < kEdge; e0 += PER) {
        const int e = (e0 + q) * ES;
        if (off + e < head)
            *reinterpret_cast<T*>(p + off + e) = *reinterpret_cast<const T*>(s + off + e);
        if (tail + e < end)
            *reinterpret_cast<T*>(p + tail + e) = *reinterpret_cast<const T*>(s + tail + e);
    }
}

// ------------------------------------------------------------- look-back

// What the work area is filled with before a scan: a NaN pattern no result has
// (results' NaNs are 0x7fffffff), and the status word's "nothing recorded".
constexpr uint32_t kNotYet = 0xffffffffu;

__device__ __forceinline__ uint32_t published(float v) {
    return v != v ? 0x7fffffffu : __float_as_uint(v);
}

__device__ __forceinline__ void put_agg(ulonglong2* p, float2 P, float2 q) {
    const unsigned long long u = (unsigned long long)published(q.x) << 32 | __float_as_uint(P.x);
    const unsigned long long v = (unsigned long long)published(q.y) << 32 | __float_as_uint(P.y);
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(u), "l"(v) : "memory");
}

// (P.x, P.y, q.x, q.y); each channel's pair is one 64-bit access, so a q that is there
// has its P
__device__ __forceinline__ bool get_agg(const ulonglong2* p, float4& r) {
    unsigned long long u, v;
    asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(u), "=l"(v) : "l"(p) : "memory");
    r = make_float4(__uint_as_float((uint32_t)u), __uint_as_float((uint32_t)v),
                    __uint_as_float((uint32_t)(u >> 32)), __uint_as_float((uint32_t)(v >> 32)));
    return (uint32_t)(u >> 32) != kNotYet && (uint32_t)(v >> 32) != kNotYet;
}

__device__ __forceinline__ void put_inc(uint2* p, float2 h) {
    asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(published(h.x)),
                 "r"(published(h.y))
                 : "memory");
}

__device__ __forceinline__ bool get_inc(const uint2* p, float2& h) {
    uint32_t u, v;
    asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(u), "=r"(v) : "l"(p) : "memory");
    h = make_float2(__uint_as_float(u), __uint_as_float(v));
    return u != kNotYet && v != kNotYet;
}

// What the tiles before a tile have published.
template <int WARPS, int PER>
struct Look {
    static constexpr int kTiles = (WARPS - 1) * PER;  // warp 0 has the aggregate to make
    float4 v[kTiles][32];  // of the tile i + 1 before: its aggregate, or its state in x, y
    int state[kTiles];     // whether it is the state
};

// A warp's part of a look-back: waits until each of its tiles has published
// something, or a nearer one its state (every lane publishes, those past the
// channels too).
template <int WARPS, int N>
__device__ __forceinline__ bool look(const LinArgs& a, Look<WARPS, N>& s, int seq, int blk,
                                     int warp, int lane) {
    // (blocks reach past 2^26, of 32 entries each)
    const size_t step = (size_t)a.blocks * 32, at = (size_t)blk * 32 + lane;
    const int first = seq - warp;  // tiles seq - warp, then WARPS - 1 further back
    uint32_t polls = 0;
    bool done[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        done[i] = first - i * (WARPS - 1) < 0;
        if (done[i] && lane == 0) s.state[warp - 1 + i * (WARPS - 1)] = 0;
    }
    while (true) {
        float2 h[N];
        float4 r[N];
        bool inc[N], agg[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            inc[i] = agg[i] = false;
            if (!done[i]) {
                const size_t o = (size_t)(first - i * (WARPS - 1)) * step + at;
                inc[i] = get_inc(a.inc + o, h[i]);
                agg[i] = get_agg(a.agg + o, r[i]);
            }
        }
        bool all = true;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (done[i]) continue;
            const int w = warp - 1 + i * (WARPS - 1);
            if (__all_sync(0xffffffffu, inc[i])) {
                s.v[w][lane] = make_float4(h[i].x, h[i].y, 0.0f, 0.0f);
                if (lane == 0) s.state[w] = 1;
                // nothing further back is needed
                for (int k = i; k < N; ++k) done[k] = true;
            } else if (__all_sync(0xffffffffu, agg[i])) {
                s.v[w][lane] = r[i];
                if (lane == 0) s.state[w] = 0;
                done[i] = true;
            } else {
                all = false;
            }
        }
        if (all) return true;
        if (++polls >= a.spin_limit) return false;
        if (polls > 4) __nanosleep(40);
    }
}

// ---------------------------------------------------- packed pairs of fp32

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The decay of a span of steps, the product of their gates, is 0 only where one of them
// restarts the state.  A product that fell below every number counts as the least one, so
// that a NaN or an infinity outlasts the span as it outlasts each step; a finite state h is
// off by at most 2^-149 |h|.  While it grows, -0 says that a gate was 0.
constexpr float kLeast = 0x1p-149f;
__device__ __forceinline__ float2 longer_span(float2 product, float2 a) {
    const float2 p = mul2(product, a);
    return make_float2(a.x == 0.0f ? -0.0f : p.x, a.y == 0.0f ? -0.0f : p.y);
}
__device__ __forceinline__ float span_decay(float product) {
    return __float_as_int(product) < 0 ? 0.0f : fmaxf(product, kLeast);
}
__device__ __forceinline__ float2 span_decay(float2 product) {
    return make_float2(span_decay(product.x), span_decay(product.y));
}

// sigmoid(v) and the t = e^-v it comes from, for |v| < 80 or where an infinite t
// gives the right 0
__device__ __forceinline__ float2 sigmoid2(float2 v, float2& t) {
    const float2 e = mul2(v, both(-kLog2e));
    t = make_float2(ex2_approx(e.x), ex2_approx(e.y));
    const float2 d = add2(t, both(1.0f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// The arithmetic of a step for two channels.  FAST: gates within |f| < 80.
template <bool FAST>
struct Step {
    __device__ static void gates(float2 f, float2& a, float2& om) {
        if constexpr (FAST) {
            float2 t;
            a = sigmoid2(f, t);
            om = mul2(t, a);
        } else {
            gate(f.x, a.x, om.x);
            gate(f.y, a.y, om.y);
        }
    }
    __device__ static float2 input(float2 om, float2 x) {  // (1 - a) x
        if constexpr (FAST) return mul2(om, x);
        return make_float2(input_term(om.x, x.x), input_term(om.y, x.y));
    }
    __device__ static float2 next(float2 a, float2 h, float2 b) {  // a h + b
        if constexpr (FAST) return fma2(a, h, b);
        return make_float2(step(a.x, h.x, b.x), step(a.y, h.y, b.y));
    }
    __device__ static float2 decay(float2 a, float2 h) {  // a h
        if constexpr (FAST) return mul2(a, h);
        return make_float2(step(a.x, h.x, 0.0f), step(a.y, h.y, 0.0f));
    }
    // lam (h - x) a (1 - a)
    __device__ static float2 dgate(float2 a, float2 om, float2 lam, float2 h, float2 x) {
        const float2 s = mul2(a, om);
        const float2 d = mul2(mul2(lam, fma2(x, both(-1.0f), h)), s);
        if constexpr (FAST) return d;
        return make_float2(s.x == 0.0f ? 0.0f : d.x, s.y == 0.0f ? 0.0f : d.y);
    }
};

// whether every one of a lane's raw gate pairs lies within |f| < 80
template <typename T, int S>
__device__ __forceinline__ bool all_fast(const void* const* rows) {
    if constexpr (sizeof(T) == 2) {
        __nv_bfloat162 m = __habs2(*static_cast<const __nv_bfloat162*>(rows[0]));
#pragma unroll
        for (int k = 1; k < S; ++k)
            m = __hmax2_nan(m, __habs2(*static_cast<const __nv_bfloat162*>(rows[k])));
        return __low2float(m) < kFastGate && __high2float(m) < kFastGate;
    } else {
        bool ok = true;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const float2 f = *static_cast<const float2*>(rows[k]);
            ok = ok && fabsf(f.x) < kFastGate && fabsf(f.y) < kFastGate;
        }
        return ok;
    }
}

// ---------------------------------------------------------- tile kernels

__host__ __device__ constexpr int tile_steps(bool grad, bool tma) {
    return grad || !tma ? kKeep : 2 * kKeep;
}

template <typename T, int NIN, bool GRAD, bool TMA>
struct LinSmem {
    static constexpr int kRow = TMA ? kCh * (int)sizeof(T) : kShiftedRow<T>;
    static constexpr int kTile = tile_steps(GRAD, TMA) * (kRow + (TMA ? 0 : 16));  // of one input
    static constexpr int kStage = NIN * kTile;
};

// GRAD false: inputs f, x[, z], output y.  GRAD true: inputs f, x, dy[, z],
// outputs df, dx[, dz].  TMA: every row 16-byte aligned; else shifted rows.
template <typename T, typename TO, int WARPS, int STAGES, bool TMA, bool GATED, bool GRAD, int MINB>
__global__ void __launch_bounds__(WARPS * 32, MINB)
    linrec_tile_kernel(const __grid_constant__ LinMaps maps, const LinArgs a) {
    constexpr int NIN = (GRAD ? 3 : 2) + (GATED ? 1 : 0);
    constexpr int STEPS = tile_steps(GRAD, TMA), S = STEPS / WARPS;
    // results of the inputs' size take their places in the tile, and leave by TMA or,
    // where rows are shifted, by their warps
    constexpr bool STAGED = sizeof(T) == sizeof(TO), INPLACE = TMA && STAGED;
    using SM = LinSmem<T, NIN, GRAD, TMA>;
    constexpr int APART = TMA ? 1 : 32;  // a lane's channels are neighbours, or not
    extern __shared__ __align__(1024) uint8_t smem[];
    // the warps' (P, q), gradient also the reverse q; each q is replaced by that of
    // all that stands before its warp in the scan's order (for the gradient's q: in
    // time), whose P is beside
    __shared__ float2 s_P[WARPS][32], s_q[WARPS][32], s_r[GRAD ? WARPS : 1][32];
    __shared__ float2 s_preP[WARPS][32], s_timeP[GRAD ? WARPS : 1][32];
    // a gradient's CTAs, two of which share an SM, have no room for more than seven
    using L = Look<WARPS, WARPS == 8 && !GRAD ? 2 : 1>;
    __shared__ L s_look;
    __shared__ uint64_t full[STAGES];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool copies = TMA ? tid == WARPS * 32 - 32 : true;  // the TMA thread, or all

    // a tile of this CTA: its place in the scan and its channel block, moved on by
    // the grid without divisions
    struct At {
        int seq, blk;
    };
    const int dseq = gridDim.x / a.blocks, dblk = gridDim.x % a.blocks;
    auto next = [&](At t) {
        t.seq += dseq;
        t.blk += dblk;
        if (t.blk >= a.blocks) {
            t.blk -= a.blocks;
            ++t.seq;
        }
        return t;
    };
    auto where = [&](At t, int& tile, int& b, int& c0) {
        tile = GRAD ? a.tiles - 1 - t.seq : t.seq;
        b = __umulhi((uint32_t)t.blk, a.cblocks_inv);  // at most one off
        int r = t.blk - b * a.cblocks;
        if (r < 0) {
            --b;
            r += a.cblocks;
        } else if (r >= a.cblocks) {
            ++b;
            r -= a.cblocks;
        }
        c0 = r * kCh;
    };
    auto fetch = [&](At t, int stage) {
        if (t.seq < a.tiles) {
            int tile, b, c0;
            where(t, tile, b, c0);
            uint8_t* dst = smem + stage * SM::kStage;
            if constexpr (TMA) {
                mbar_arrive_expect_tx(&full[stage], SM::kStage);
#pragma unroll
                for (int i = 0; i < NIN; ++i)
                    tma_load_3d(dst + i * SM::kTile, &maps.in[i], &full[stage], c0, tile * STEPS, b);
            } else {
#pragma unroll
                for (int i = 0; i < NIN; ++i)
                    load_shifted<T, STEPS, WARPS * 32>(dst + i * SM::kTile, a.in[i], a.stride[i], b,
                                                       tile * STEPS, c0, a.seqlen, a.dim);
            }
        }
        if constexpr (!TMA) copy_commit();
    };
    // the results of a tile out of `stage`
    auto send = [&](At t, int stage) {
        int tile, b, c0;
        where(t, tile, b, c0);
        uint8_t* src = smem + stage * SM::kStage;
        if constexpr (!GRAD) {
            if (a.out[0]) tma_store_3d(&maps.out[0], src, c0, tile * STEPS, b);
        } else {
            tma_store_3d(&maps.out[0], src, c0, tile * STEPS, b);
            tma_store_3d(&maps.out[1], src + SM::kTile, c0, tile * STEPS, b);
            if constexpr (GATED)
                tma_store_3d(&maps.out[2], src + 3 * SM::kTile, c0, tile * STEPS, b);
        }
        bulk_commit();
    };

    // one tile per sequence: nothing was cleared before the launch, and only a load
    // that never comes, seconds later, writes the status too.  (The tile count and the
    // flag tested here instead of by the host: 142 us against 133 us for 65536 steps of
    // 1536 channels, as the forward kernel uses every register it may have.)
    if constexpr (!TMA)
        if (tid == 0 && a.clear && blockIdx.x == 0) *a.clear = kNotYet;
    if constexpr (TMA) {
        if (tid == 0) {
            for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
            fence_mbar_init();
            if (a.clear && blockIdx.x == 0) *a.clear = kNotYet;
        }
        __syncthreads();
    }
    // tile i + STAGES - 1 of this CTA is fetched during its tile i, once the ring's
    // place, tile i - 1's, has been sent
    At cur{(int)blockIdx.x / a.blocks, (int)blockIdx.x % a.blocks}, ahead = cur, before = cur;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
        if (copies) fetch(ahead, i);
        ahead = next(ahead);
    }

    int turn = 0, stage = 0, last_stage = STAGES - 1;
    uint32_t parity = 0;
    bool ok = true;
    for (; cur.seq < a.tiles; before = cur, cur = next(cur), ++turn) {
        if constexpr (TMA) ok = mbar_wait(&full[stage], parity, nullptr);
        else copy_wait<STAGES - 2>();
        // the tile is there, the previous one is done with
        if (!__syncthreads_and(ok)) {
            if (tid == 0) atomicCAS(a.status, kNotYet, SSM_ERR_TIMEOUT);
            ok = false;
            break;
        }
        if constexpr (INPLACE)
            if (copies && turn > 0) send(before, last_stage);

        const int seq = cur.seq, blk = cur.blk;
        int tile, b, c;
        where(cur, tile, b, c);
        const int c0 = c;
        c += lane * (TMA ? 2 : 1);
        const bool valid = c < a.dim, two = c + APART < a.dim;
        const size_t chan = (size_t)b * a.dim + c;
        const int t0 = tile * STEPS + warp * S;
        // aligned rows: this lane's channels of the warp's first row
        uint8_t* base = smem + stage * SM::kStage +
                        (TMA ? warp * S * SM::kRow + lane * 2 * (int)sizeof(T) : 0);
        const long long row0 = (long long)b * a.seqlen + t0;
        // shifted rows: the same of each input, the distance of its rows, where the warp's
        // first row starts behind its 16-byte boundary, and how far that moves from a row
        // to the next
        uint32_t in_at[NIN], in_row[NIN], sh_in[NIN], d_in[NIN], sh_out[3] = {}, d_out = 0;
        if constexpr (!TMA) {
#pragma unroll
            for (int i = 0; i < NIN; ++i) {
                d_in[i] = (uint32_t)(a.stride[i] * (long long)sizeof(T)) & 15;
                in_row[i] = SM::kRow + d_in[i];
                // of the tile's first row, then of the warp's
                sh_in[i] = shift_of(a.in[i], (row0 - warp * S) * a.stride[i] + c0, sizeof(T)) +
                           warp * S * d_in[i];
                in_at[i] = i * SM::kTile + warp * S * SM::kRow + sh_in[i] + lane * (int)sizeof(T);
            }
#pragma unroll
            for (int i = 0; i < (GRAD ? (GATED ? 3 : 2) : 1); ++i)
                sh_out[i] = shift_of(a.out[i], row0 * a.dim + c0, sizeof(TO));
            d_out = (uint32_t)a.dim * (uint32_t)sizeof(TO) & 15;
        }
        // this lane's two channels of input i at the warp's step k
        auto get = [&](int i, int k) -> float2 {
            if constexpr (TMA) return Pair<T>::get(base + i * SM::kTile + k * SM::kRow);
            else return get_shifted<T>(base + in_at[i] + k * in_row[i]);
        };
        // a result into the place of input i (shifted rows: at its own offset there)
        const size_t o = (size_t)row0 * a.dim + c;
        auto put = [&](int i, int k, int result, float2 v) {
            if constexpr (INPLACE) {
                Pair<TO>::put(base + i * SM::kTile + k * SM::kRow, v);
            } else if constexpr (STAGED) {
                put_shifted<TO>(base + i * SM::kTile + (warp * S + k) * SM::kRow +
                                    ((sh_in[i] + k * d_in[i]) & ~15u) +
                                    ((sh_out[result] + k * d_out) & 15) + lane * (int)sizeof(TO),
                                v);
            } else if (valid && t0 + k < a.seqlen) {
                TO* p = static_cast<TO*>(a.out[result]) + o + (size_t)k * a.dim;
                if constexpr (TMA) {
                    Pair<TO>::put(p, v);
                } else {
                    p[0] = from_f32<TO>(v.x);
                    if (two) p[APART] = from_f32<TO>(v.y);
                }
            }
        };
        auto send_rows = [&](int i, int result) {
            if constexpr (!TMA && STAGED) {
                __syncwarp();
                send_shifted<TO, S>(base + i * SM::kTile + warp * S * SM::kRow, sh_in[i], d_in[i],
                                    a.out[result], o - lane, a.dim, min(S, a.seqlen - t0),
                                    min(kCh, a.dim - c0), lane);
            }
        };

        // the state entering the tile, for the gradient's replay
        float2 hk = make_float2(0.0f, 0.0f);
        if constexpr (GRAD) {
            if (valid) {
                if (tile > 0)
                    hk = load_state2<APART>(a.keep + (size_t)tile * a.batch * a.dim, chan, two);
                else if (a.first)
                    hk = load_state2<APART>(a.first, chan, two);
            }
        }

        float2 ga[S], gb[S];  // a_t, and b_t (forward) or 1 - a_t (gradient)
        // shifted rows: warps whose steps are all past the sequence have nothing to do
        // (aligned rows are zeros there, and the branch costs registers that the kernel
        // does not have: 116 us became 118 us for the gradient of 8 x 2048 x 1536); a warp
        // whose gates all lie within |f| < 80 needs no comparisons
        const bool live = TMA || t0 < a.seqlen;
        bool fast = false;
        if (live) {
            if constexpr (TMA) {
                const void* rows[S];
#pragma unroll
                for (int k = 0; k < S; ++k) rows[k] = base + k * SM::kRow;
                fast = all_fast<T, S>(rows);
            } else {
                fast = true;
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    const float2 f = get(0, k);
                    ga[k] = f;  // read once: the gate takes its place
                    fast = fast && fabsf(f.x) < kFastGate && fabsf(f.y) < kFastGate;
                }
            }
            fast = __all_sync(0xffffffffu, fast && t0 + S <= a.seqlen);
        }

        // ---- the warp's steps from zero
        float2 P = both(1.0f), q = both(0.0f);
        auto scan = [&](auto fast_) {
            constexpr bool F = decltype(fast_)::value;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const float2 x = get(1, k);
                float2 om;
                Step<F>::gates(TMA ? get(0, k) : ga[k], ga[k], om);
                if (!F && t0 + k >= a.seqlen) {
                    ga[k] = both(1.0f);
                    om = both(0.0f);
                }
                const float2 bt = Step<F>::input(om, x);
                gb[k] = GRAD ? om : bt;
                q = Step<F>::next(ga[k], q, bt);
                // (a NaN gate is NaN in q: left out here, so that a restart before it counts)
                P = F ? mul2(P, ga[k])
                      : longer_span(P, make_float2(fminf(ga[k].x, 1.0f), fminf(ga[k].y, 1.0f)));
            }
            P = F ? make_float2(fmaxf(P.x, kLeast), fmaxf(P.y, kLeast)) : span_decay(P);
            if constexpr (GRAD) {
                // mu through the steps: dh_t = dy_t silu(z_t), 0 past the sequence
                // (the tile is zero there)
                float2 r = both(0.0f);
#pragma unroll
                for (int k = S - 1; k >= 0; --k) {
                    float2 d = get(2, k);
                    if constexpr (GATED) {
                        const float2 z = get(3, k);
                        float2 t;
                        d = mul2(d, mul2(z, sigmoid2(z, t)));
                    }
                    r = Step<F>::decay(ga[k], add2(r, d));
                }
                s_r[warp][lane] = r;
            }
        };
        if (fast) scan(std::true_type{});
        else if (live) scan(std::false_type{});
        else if (GRAD) s_r[GRAD ? warp : 0][lane] = both(0.0f);
        s_P[warp][lane] = P;
        s_q[warp][lane] = q;
        __syncthreads();

        if constexpr (TMA) {
            if (copies) {
                if constexpr (INPLACE) bulk_wait_read_all();
                fetch(ahead, last_stage);
            }
        }

        // ---- across warps and tiles: the state (gradient: mu) entering this one
        float2 in = both(0.0f), TP = both(1.0f), tq = both(0.0f);
        const size_t mine = ((size_t)seq * a.blocks + blk) * 32 + lane;
        if (warp == 0) {
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const int w = GRAD ? WARPS - 1 - i : i;
                float2& q_ = GRAD ? s_r[w][lane] : s_q[w][lane];
                const float2 own = q_, p = s_P[w][lane];
                q_ = tq;
                s_preP[w][lane] = TP;
                tq = Step<false>::next(p, tq, own);
                TP = longer_span(TP, p);
            }
            TP = span_decay(TP);
            // the first tile has its state at once, the last one's is nobody's to read
            if (seq > 0 && seq < a.tiles - 1) put_agg(a.agg + mine, TP, tq);
        } else if (GRAD && warp == 1) {
            float2 fP = both(1.0f), fq = both(0.0f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 own = s_q[w][lane], p = s_P[w][lane];
                s_q[w][lane] = fq;
                s_timeP[w][lane] = fP;
                fq = Step<false>::next(p, fq, own);
                fP = longer_span(fP, p);
            }
        }
        // every thread's copies: once the aggregate is out (before it: 84 us for the 82 us
        // above)
        if constexpr (!TMA) fetch(ahead, last_stage);
        if (seq == 0) {
            if (a.h0 && valid) in = load_state2<APART>(a.h0, chan, two);
            __syncthreads();
        } else {
            while (true) {
                const bool found = warp == 0 || look(a, s_look, seq, blk, warp, lane);
                if (!__syncthreads_and(found)) {
                    if (tid == 0) atomicCAS(a.status, kNotYet, SSM_ERR_TIMEOUT);
                    in = both(__int_as_float(0x7fffffff));
                    break;
                }
                int w = 0;
                while (w < L::kTiles && !s_look.state[w]) ++w;
                if (w < L::kTiles) {
                    // from the newest state through the aggregates after it, in
                    // order: the same operations wherever the state was found
                    const float4 h = s_look.v[w][lane];
                    in = make_float2(h.x, h.y);
                    for (--w; w >= 0; --w) {
                        const float4 g = s_look.v[w][lane];
                        in = Step<false>::next(make_float2(g.x, g.y), in, make_float2(g.z, g.w));
                    }
                    break;
                }
                __syncthreads();  // aggregates and no state yet: look again
            }
        }
        if (warp == 0) {
            const float2 end = Step<false>::next(TP, in, tq);
            if (seq < a.tiles - 1) {
                if (!(a.drop_first_publish && seq == 0)) put_inc(a.inc + mine, end);
            } else if (a.last && valid) {
                store_state2<APART>(a.last, chan, end, two);
            }
        }
        in = Step<false>::next(span_decay(s_preP[warp][lane]), in,
                               GRAD ? s_r[warp][lane] : s_q[warp][lane]);

        // ---- the steps again from the warp's entry state
        if constexpr (!GRAD) {
            float2 h = in;
            if (a.keep && warp * S % kKeep == 0 && valid && t0 < a.seqlen) {
                float* s = a.keep + (size_t)(t0 / kKeep) * a.batch * a.dim + chan;
                store_state2<APART>(s, 0, h, two);
            }
            auto replay = [&](auto fast_) {
                constexpr bool F = decltype(fast_)::value;
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    h = Step<F>::next(ga[k], h, gb[k]);
                    float2 y = h;
                    if constexpr (GATED) {
                        const float2 z = get(2, k);
                        float2 t;
                        y = mul2(y, mul2(z, sigmoid2(z, t)));
                    }
                    put(0, k, 0, y);
                }
            };
            if (a.out[0] && live) {
                if (fast) replay(std::true_type{});
                else replay(std::false_type{});
                send_rows(0, 0);
            }
        } else {
            float2 mu = in, h = Step<false>::next(span_decay(s_timeP[warp][lane]), hk, s_q[warp][lane]);
            auto replay = [&](auto fast_) {
                constexpr bool F = decltype(fast_)::value;
                float2 prev[S];  // h_{t-1}
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    prev[k] = h;
                    h = Step<F>::next(ga[k], h, Step<F>::input(gb[k], get(1, k)));
                }
#pragma unroll
                for (int k = S - 1; k >= 0; --k) {
                    const float2 x = get(1, k);
                    float2 d = get(2, k);
                    if constexpr (GATED) {
                        const float2 z = get(3, k);
                        float2 t;
                        const float2 sg = sigmoid2(z, t);
                        const float2 si = mul2(z, sg);
                        // silu' = sg (1 + z (1 - sg)) = sg + si - si sg
                        const float2 ds = fma2(mul2(si, both(-1.0f)), sg, add2(sg, si));
                        const float2 dz = mul2(mul2(d, h), ds);
                        d = mul2(d, si);
                        if constexpr (!TMA) __syncwarp();  // the row is read before it is replaced
                        put(3, k, 2, dz);
                    }
                    const float2 lam = add2(d, mu);
                    const float2 df = Step<F>::dgate(ga[k], gb[k], lam, prev[k], x);
                    const float2 dx = Step<F>::input(gb[k], lam);
                    if constexpr (!TMA && !GATED) __syncwarp();
                    put(0, k, 0, df);
                    put(1, k, 1, dx);
                    mu = Step<F>::decay(ga[k], lam);
                    h = prev[k];
                }
            };
            if (live) {
                if (fast) replay(std::true_type{});
                else replay(std::false_type{});
                send_rows(0, 0);
                send_rows(1, 1);
                if constexpr (GATED) send_rows(3, 2);
            }
        }
        if constexpr (INPLACE) fence_proxy_async_smem();
        ahead = next(ahead);
        last_stage = stage;
        if (++stage == STAGES) {
            stage = 0;
            parity ^= 1;
        }
    }
    if constexpr (INPLACE) {
        __syncthreads();
        if (copies) {
            if (ok && turn > 0) send(before, last_stage);
            bulk_wait_all();
        }
    }
    if constexpr (!TMA) copy_wait<0>();
    // a load that never came: leave what is in flight time to land
    if (!ok)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// -------------------------------------------------------- short sequences

// One thread walks the steps of CPT channels (two where every pair of them is aligned),
// AHEAD steps' loads in flight: eight, and one where there is one, which then fetches less
// code (batch 128, 2560 channels: 2.4 us against 2.6 us).  A decode step (one token) is a
// single pass over the states, and many sequences fill the GPU by themselves.
constexpr int kWalkThreads = 128, kWalkAhead = 8;

template <typename T, int CPT>
__device__ __forceinline__ float2 walk_get(const void* base, long long at) {
    const T* p = static_cast<const T*>(base) + at;
    if constexpr (CPT == 2) return Pair<T>::get(p);
    return make_float2(to_f32(*p), 0.0f);
}

template <typename T, int CPT>
__device__ __forceinline__ void walk_put(void* base, long long at, float2 v) {
    T* p = static_cast<T*>(base) + at;
    if constexpr (CPT == 2) Pair<T>::put(p, v);
    else *p = from_f32<T>(v.x);
}

template <typename T, typename TO, int CPT, int AHEAD, bool GATED>
__global__ void __launch_bounds__(kWalkThreads) linrec_walk_kernel(const LinArgs a) {
    const int per = a.dim / CPT;
    const long long i = (long long)blockIdx.x * kWalkThreads + threadIdx.x;
    // nothing recorded: a gradient's tiles, which may follow, record over that word only
    if (i == 0 && a.status && !a.keep_status) *a.status = kNotYet;
    if (i >= (long long)a.batch * per) return;
    const int b = (int)(i / per), c = (int)(i % per) * CPT;
    const long long chan = (long long)b * a.dim + c, row0 = (long long)b * a.seqlen;
    float2 h = make_float2(0.0f, 0.0f);
    if (a.h0) h = walk_get<float, CPT>(a.h0, chan);
    for (int t0 = 0; t0 < a.seqlen; t0 += AHEAD) {
        float2 f[AHEAD], x[AHEAD], z[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (t0 + k >= a.seqlen) break;
            const long long t = row0 + t0 + k;
            f[k] = walk_get<T, CPT>(a.in[0], t * a.stride[0] + c);
            x[k] = walk_get<T, CPT>(a.in[1], t * a.stride[1] + c);
            if constexpr (GATED) z[k] = walk_get<T, CPT>(a.in[2], t * a.stride[2] + c);
        }
        if (a.keep && t0 % kKeep == 0)
            walk_put<float, CPT>(a.keep, (long long)(t0 / kKeep) * a.batch * a.dim + chan, h);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (t0 + k >= a.seqlen) break;
            float2 g, om, u;
            Step<false>::gates(f[k], g, om);
            h = Step<false>::next(g, h, Step<false>::input(om, x[k]));
            float2 y = h;
            if constexpr (GATED) y = mul2(y, mul2(z[k], sigmoid2(z[k], u)));
            if (a.out[0]) walk_put<TO, CPT>(a.out[0], (row0 + t0 + k) * a.dim + c, y);
        }
    }
    if (a.last) walk_put<float, CPT>(a.last, chan, h);
}

// The gradient of a sequence of up to kWalkSteps steps: forwards keeping each step's
// state, then backwards.
template <typename T, typename TO, int CPT, bool GATED>
__global__ void __launch_bounds__(kWalkThreads) linrec_walk_bwd_kernel(const LinArgs a) {
    const int per = a.dim / CPT;
    const long long i = (long long)blockIdx.x * kWalkThreads + threadIdx.x;
    if (i == 0 && !a.keep_status) *a.status = kNotYet;
    if (i >= (long long)a.batch * per) return;
    const int b = (int)(i / per), c = (int)(i % per) * CPT;
    const long long chan = (long long)b * a.dim + c, row0 = (long long)b * a.seqlen;
    float2 h = make_float2(0.0f, 0.0f), mu = h;
    if (a.first) h = walk_get<float, CPT>(a.first, chan);
    if (a.h0) mu = walk_get<float, CPT>(a.h0, chan);
    float2 prev[kWalkSteps];  // h_{t-1}
#pragma unroll
    for (int k = 0; k < kWalkSteps; ++k) {
        if (k >= a.seqlen) break;
        float2 g, om;
        Step<false>::gates(walk_get<T, CPT>(a.in[0], (row0 + k) * a.stride[0] + c), g, om);
        prev[k] = h;
        h = Step<false>::next(
            g, h, Step<false>::input(om, walk_get<T, CPT>(a.in[1], (row0 + k) * a.stride[1] + c)));
    }
#pragma unroll
    for (int k = kWalkSteps - 1; k >= 0; --k) {
        if (k >= a.seqlen) continue;
        const long long t = row0 + k, at = t * a.dim + c;
        float2 g, om;  // again: the lines are in the cache
        Step<false>::gates(walk_get<T, CPT>(a.in[0], t * a.stride[0] + c), g, om);
        const float2 x = walk_get<T, CPT>(a.in[1], t * a.stride[1] + c);
        float2 d = walk_get<T, CPT>(a.in[2], t * a.stride[2] + c);
        if constexpr (GATED) {
            const float2 z = walk_get<T, CPT>(a.in[3], t * a.stride[3] + c);
            float2 u;
            const float2 sg = sigmoid2(z, u), si = mul2(z, sg);
            const float2 ds = fma2(mul2(si, both(-1.0f)), sg, add2(sg, si));
            walk_put<TO, CPT>(a.out[2], at, mul2(mul2(d, h), ds));
            d = mul2(d, si);
        }
        const float2 lam = add2(d, mu);
        walk_put<TO, CPT>(a.out[0], at, Step<false>::dgate(g, om, lam, prev[k], x));
        walk_put<TO, CPT>(a.out[1], at, Step<false>::input(om, lam));
        mu = Step<false>::decay(g, lam);
        h = prev[k];
    }
    if (a.last) walk_put<float, CPT>(a.last, chan, mu);
}

// ---------------------------------------------------------------- launch

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

constexpr int kMostSteps = 0x7fffffff - 2 * kKeep;

int tiles_of(int seqlen, int steps) { return seqlen / steps + (seqlen % steps != 0); }

// header, aggregates and inclusive states of `tiles` tiles
size_t scan_bytes(int batch, int dim, int tiles) {
    const size_t blocks = (size_t)batch * ((dim + kCh - 1) / kCh);
    return sizeof(LinHeader) + (tiles > 1 ? (size_t)tiles * blocks * 32 * 24 : 0);
}

bool sizes_ok(int batch, int seqlen, int dim) { return batch >= 0 && seqlen >= 0 && dim >= 0; }

// one int counts the tiles of all blocks, one a sequence's steps to the end of its last tile,
// one the channels
bool sizes_fit(int batch, int seqlen, int dim) {
    if (seqlen > kMostSteps || dim > 2000000000) return false;
    const double blocks = (double)batch * ((dim + kCh - 1) / kCh);
    return blocks * tiles_of(seqlen, kKeep) < 2.0e9 && (double)batch * dim < 2.0e9;
}

// Fills in the work area of one scan.
void place(LinArgs& a, uint8_t* ws, int tiles) {
    a.cblocks = (a.dim + kCh - 1) / kCh;
    a.cblocks_inv = (uint32_t)std::min<uint64_t>(0xffffffffu, (uint64_t(1) << 32) / a.cblocks + 1);
    a.blocks = a.batch * a.cblocks;
    a.tiles = tiles;
    if (!ws) return;  // a walked sequence
    a.status = reinterpret_cast<uint32_t*>(ws) + 1;
    a.agg = reinterpret_cast<ulonglong2*>(ws + sizeof(LinHeader));
    a.inc = reinterpret_cast<uint2*>(a.agg + (size_t)tiles * a.blocks * 32);
}

// (batch, seqlen, dim) with rows `stride` elements apart, boxes of a tile
bool make_map(CUtensorMap* map, const void* base, size_t es, long long stride, const LinArgs& a,
              int steps) {
    auto fn = ssm_host::encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.seqlen, (cuuint64_t)a.batch};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * es, (cuuint64_t)stride * es * a.seqlen};
    const cuuint32_t box[3] = {(cuuint32_t)kCh, (cuuint32_t)steps, 1}, one[3] = {1, 1, 1};
    return fn(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
              const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, typename TO, bool TMA, bool GATED, bool GRAD>
bool launch_tile(LinArgs& a, uint8_t* ws, cudaStream_t s) {
    constexpr int NIN = (GRAD ? 3 : 2) + (GATED ? 1 : 0);
    // 16 warps an SM, and as many stages as fit in its shared memory
    constexpr int WARPS = sizeof(T) == 2 ? 8 : 16, MINB = 16 / WARPS;
    constexpr int kStage = LinSmem<T, NIN, GRAD, TMA>::kStage;
    constexpr int STAGES = 96 * 1024 * WARPS / 8 / kStage;
    static_assert(STAGES >= 2, "one tile at work, one coming in");
    constexpr int smem = STAGES * kStage;
    auto kernel = linrec_tile_kernel<T, TO, WARPS, STAGES, TMA, GATED, GRAD, MINB>;
    place(a, ws, tiles_of(a.seqlen, tile_steps(GRAD, TMA)));
    const void* fn = reinterpret_cast<const void*>(kernel);
    static std::atomic<int> cache[ssm_host::kMaxDevices];
    const int slots =
        ssm_host::sm_count() * ssm_host::resident_ctas(fn, WARPS * 32, smem, cache);
    if (slots < 1) return false;
    LinMaps maps{};
    if constexpr (TMA) {
        for (int i = 0; i < NIN; ++i)
            if (!make_map(&maps.in[i], a.in[i], sizeof(T), a.stride[i], a, tile_steps(GRAD, TMA))) return false;
        for (int i = 0; i < 3 && sizeof(T) == sizeof(TO); ++i)
            if (a.out[i] && !make_map(&maps.out[i], a.out[i], sizeof(TO), a.dim, a,
                                       tile_steps(GRAD, TMA)))
                return false;
    }
    const long long items = (long long)a.blocks * a.tiles;
    const unsigned grid = (unsigned)std::min<long long>(items, slots);
    if (a.tiles == 1) {
        a.clear = a.keep_status ? nullptr : a.status;
        kernel<<<grid, WARPS * 32, smem, s>>>(maps, a);
        return cudaGetLastError() == cudaSuccess;
    }
    // header and published values are neighbours; an earlier scan's status stays
    uint8_t* from = reinterpret_cast<uint8_t*>(a.agg) - (a.keep_status ? 0 : sizeof(LinHeader));
    if (cudaMemsetAsync(from, 0xff,
                        (size_t)items * 32 * 24 + (a.keep_status ? 0 : sizeof(LinHeader)),
                        s) != cudaSuccess)
        return false;
    void* args[] = {&maps, &a};
    return cudaLaunchCooperativeKernel(fn, dim3(grid), dim3(WARPS * 32), args, smem, s) ==
           cudaSuccess;
}

// Whether TMA can take the inputs' rows and bring the results' home.
bool rows_aligned(const LinArgs& a, int n, size_t es, size_t out_es) {
    bool ok = a.dim * es % 16 == 0 && a.dim * out_es % 16 == 0;
    for (int i = 0; i < n; ++i)
        ok = ok && reinterpret_cast<uintptr_t>(a.in[i]) % 16 == 0 &&
             (size_t)a.stride[i] * es % 16 == 0;
    return ok;
}

template <typename T, typename TO, bool GRAD>
bool launch_by(LinArgs& a, uint8_t* ws, bool gated, cudaStream_t s) {
    const int nin = (GRAD ? 3 : 2) + (gated ? 1 : 0);
    if (rows_aligned(a, nin, sizeof(T), sizeof(TO)))
        return gated ? launch_tile<T, TO, true, true, GRAD>(a, ws, s)
                     : launch_tile<T, TO, true, false, GRAD>(a, ws, s);
    return gated ? launch_tile<T, TO, false, true, GRAD>(a, ws, s)
                 : launch_tile<T, TO, false, false, GRAD>(a, ws, s);
}

// Sequences of up to kWalkSteps steps, and (forward) of up to twice that where a thread to
// each channel or pair of them gives the GPU enough warps, are walked.  Walk and tiles, us,
// with a gate:
//   channels    bf16: 17 steps   32 steps   48 steps   fp32: 17 steps   32 steps
//   10240             5    6      8    6     12    5         3    8      5    7
//   40960             5   10      9   10     12   10         4   16      5   15
//   81920             6   17      9   17     13   17         5   26      7   26
//   655360           35  123     64  123     93  117        30  184     51  175
// (A tile is mostly empty at these lengths; of unaligned bf16 rows 41041 channels, 32 steps
// take 9 us against 8.  In fp32 the walk stays ahead for longer: 655360 channels, 128 steps
// 191 us against 218 us, 40960 channels 26 us against 21 us; in bf16 it is behind at 64
// steps: 124 us against 106 us.)
constexpr long long kWalkChannels = 65536;

bool walks(int batch, int seqlen, int dim) {
    return seqlen <= kWalkSteps ||
           (seqlen <= 2 * kWalkSteps && (long long)batch * dim >= kWalkChannels);
}

template <typename T, typename TO, bool GRAD>
bool launch_walk(const LinArgs& a, bool gated, cudaStream_t s) {
    // two channels in one access to each input and result
    const int nin = (GRAD ? 3 : 2) + (gated ? 1 : 0);
    bool pairs = a.dim % 2 == 0;
    for (int i = 0; i < nin; ++i)
        pairs = pairs && reinterpret_cast<uintptr_t>(a.in[i]) % (2 * sizeof(T)) == 0 &&
                a.stride[i] % 2 == 0;
    const long long n = (long long)a.batch * (pairs ? a.dim / 2 : a.dim);
    const unsigned grid = (unsigned)((n + kWalkThreads - 1) / kWalkThreads);
    auto go = [&](auto kernel) { kernel<<<grid, kWalkThreads, 0, s>>>(a); };
    if constexpr (GRAD) {
        if (pairs) gated ? go(linrec_walk_bwd_kernel<T, TO, 2, true>)
                         : go(linrec_walk_bwd_kernel<T, TO, 2, false>);
        else gated ? go(linrec_walk_bwd_kernel<T, TO, 1, true>)
                   : go(linrec_walk_bwd_kernel<T, TO, 1, false>);
    } else {
        auto by = [&](auto ahead) {
            constexpr int A = decltype(ahead)::value;
            if (pairs) gated ? go(linrec_walk_kernel<T, TO, 2, A, true>)
                             : go(linrec_walk_kernel<T, TO, 2, A, false>);
            else gated ? go(linrec_walk_kernel<T, TO, 1, A, true>)
                       : go(linrec_walk_kernel<T, TO, 1, A, false>);
        };
        if (a.seqlen == 1) by(std::integral_constant<int, 1>{});
        else by(std::integral_constant<int, kWalkAhead>{});
    }
    return cudaGetLastError() == cudaSuccess;
}

template <typename F>
bool by_types(ssm_dtype_t in, ssm_dtype_t out, F&& f) {
    using B = __nv_bfloat16;
    if (in == SSM_F32) return out == SSM_F32 ? f(float{}, float{}) : f(float{}, B{});
    return out == SSM_F32 ? f(B{}, float{}) : f(B{}, B{});
}

// The forward scan (a.out[0] may be NULL: states only).
bool run_forward(LinArgs& a, uint8_t* ws, ssm_dtype_t in, ssm_dtype_t out, bool gated,
                 cudaStream_t s) {
    return by_types(in, out, [&](auto ti, auto to) -> bool {
        using T = decltype(ti);
        using TO = decltype(to);
        if (walks(a.batch, a.seqlen, a.dim)) return launch_walk<T, TO, false>(a, gated, s);
        return launch_by<T, TO, false>(a, ws, gated, s);
    });
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
    return scan_bytes(batch, dim, tiles_of(seqlen, kKeep));
}

extern "C" size_t ssm_linrec_bwd_workspace_bytes(int batch, int seqlen, int dim) {
    if (!sizes_ok(batch, seqlen, dim) || !sizes_fit(batch, seqlen, dim)) return 0;
    return scan_bytes(batch, dim, tiles_of(seqlen, kKeep)) +
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
    // a walked sequence waits for nothing: it runs without a workspace too
    const bool walked = seqlen <= kWalkSteps && !workspace;
    if (!walked &&
        (!workspace || workspace_bytes < ssm_linrec_workspace_bytes(batch, seqlen, dim)))
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
    ssm_internal::lookback_setting(&a.spin_limit, &a.drop_first_publish);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    place(a, ws, 1);
    return run_forward(a, ws, in_dtype, out_dtype, z != nullptr, static_cast<cudaStream_t>(stream))
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
    ssm_internal::lookback_setting(&a.spin_limit, &a.drop_first_publish);
    if (!checkpoints && seqlen > kWalkSteps) {  // walked ones are short enough to keep them
        // the forward again, states only
        LinArgs w = a;
        w.h0 = initial_state;
        w.keep = reinterpret_cast<float*>(ws + scan_bytes(batch, dim, tiles_of(seqlen, kKeep)));
        place(w, ws, 1);
        if (!run_forward(w, ws, in_dtype, in_dtype, false, s)) return SSM_ERR_CUDA;
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
    place(a, ws, 1);
    const bool ok = by_types(in_dtype, grad_dtype, [&](auto ti, auto to) -> bool {
        using T = decltype(ti);
        using TO = decltype(to);
        if (seqlen <= kWalkSteps) return launch_walk<T, TO, true>(a, z != nullptr, s);
        return launch_by<T, TO, true>(a, ws, z != nullptr, s);
    });
    return ok ? SSM_OK : SSM_ERR_CUDA;
}
