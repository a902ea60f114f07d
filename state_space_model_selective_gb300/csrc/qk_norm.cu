// qk_norm.cu -- RMS norm of every query and key head over its own columns, and
// the rotation by position, in one pass; and the gradient.
//
//   n = x / sqrt(mean(x^2) + eps),  t = n w,
//   (y_a, y_b) = (t_a cos - t_b sin, t_a sin + t_b cos)  for the pairs (a, b) of the
//   first rot columns, at the angle position * inv_freq[pair];  y = t behind them
//   gradient: g = dy turned back, dx = r (g w - n mean(g w n)),
//             dw = sum over tokens and heads of g n
//
// Memory bounds it where the issue slots do not: an arithmetic instruction takes a
// scheduler two cycles here, and a row of 128 bf16 leaves a lane 16 elements.  So two
// floats go to an instruction where that is possible, rows are counted on without
// divisions, and a token's rot / 2 sines and cosines are made once for all its heads: a CTA
// takes a few tokens with all their heads and puts them into shared memory first.
//
// Angles of far positions: position * inv_freq is a phase in turns whose whole part
// does not matter, so inv_freq / 2 pi is taken as a 64-bit binary fraction and
// multiplied by the (whole) position modulo 2^64: the fraction of a turn comes out to
// 2^-52 * position, in four integer instructions.  (An fp32 product is off by 0.06 rad
// at position 10^6; a product in fp64 runs at one 64th of fp32's rate here.)
//
// Layout of the work: a lane holds two 8-element chunks of a row -- chunk p of the
// first and of the second half of the rotated columns, so that both partners of a
// rotation are in one lane -- and a row takes 1 to 16 lanes.  Rotations whose halves
// are no multiples of 8 columns exchange partners through shared memory.
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace {

using namespace ssm;

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;
constexpr int kTable = 1024;      // sines and cosines a CTA holds at a time (pairs x tokens)
constexpr int kHeldTable = 512;   // the same where lanes hold them
constexpr int kFwdCtas = 4;       // of the forward on an SM
constexpr int kBwdCtas = 2;       // of the gradient
constexpr int kBwdMost = 152 * kBwdCtas;  // its CTAs at most, whose sums of dw are joined

// How a row's columns are paired.
enum Pairs {
    kHalves,      // (i, i + rot / 2), rot / 2 a multiple of 8: partners in one lane
    kNeighbours,  // (2 i, 2 i + 1)
    kShared       // (i, i + rot / 2), any rot: partners through shared memory
};

struct QkArgs {
    const void* x[2];          // q, k
    const void* dy[2];         // gradient only
    void* y[2];                // outputs; gradient: dq, dk
    const float* w[2];         // may be NULL (ones)
    long long stride[2];       // of x, elements between tokens
    int heads[2];
    const long long* pos;
    const double* freq;
    float* partial;            // gradient: [gridDim.x][2][dim]
    long long tokens;
    float eps, inv_dim;
    int dim, rot, lanes;       // lanes of a row, a power of two
    int tile;                  // tokens a CTA takes at a time
    int vec[2];                // x's rows are 16-byte aligned
    int join;                  // gradient: dw is wanted
};

// The first column of a lane's two chunks (dim where it has none): lane p's are the pth of
// the first and of the second half, of the rotated columns and then of the others, so that
// neighbouring lanes read and write neighbouring chunks.
template <int MODE>
__device__ __forceinline__ void lane_columns(const QkArgs& a, int p, int& c0, int& c1) {
    const int half = MODE == kHalves ? a.rot / 16 : 0;
    const int rest = a.dim / 8 - 2 * half, near = (rest + 1) / 2;
    if (p < half) {
        c0 = 8 * p;
        c1 = 8 * (p + half);
    } else {
        const int j = p - half;
        c0 = j < near ? 8 * (2 * half + j) : a.dim;
        c1 = near + j < rest ? 8 * (2 * half + near + j) : a.dim;
    }
}

// Two floats to an instruction.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpair(v, a, b);
    return a + b;
}

// 8 consecutive elements as loaded: raw bits, converted when they are used, so that
// loads in flight take few registers.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void load_each(const __nv_bfloat16* p) {
        const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = u[2 * i] | ((uint32_t)u[2 * i + 1] << 16);
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(f2* f) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pair(bf16lo(w[i]), bf16hi(w[i]));
    }
};
template <> struct Raw<float> {
    ulonglong2 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const ulonglong2*>(p));
        b = __ldcs(reinterpret_cast<const ulonglong2*>(p) + 1);
    }
    __device__ __forceinline__ void load_each(const float* p) {
        a = make_ulonglong2(pair(p[0], p[1]), pair(p[2], p[3]));
        b = make_ulonglong2(pair(p[4], p[5]), pair(p[6], p[7]));
    }
    __device__ __forceinline__ void zero() { a = b = make_ulonglong2(0, 0); }
    __device__ __forceinline__ void get(f2* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    }
};

// A lane's two chunks of a row.  A tile's rows are addressed by its base, the same for all
// threads, and 32-bit byte offsets.  FULL: all lanes have both chunks, and rows are aligned.
struct Chunks {
    uint32_t o0, d1;     // the first chunk's offset in the row, and the second's from it
    bool in0, in1;
};
template <bool FULL, typename T>
__device__ __forceinline__ void load_row(Raw<T>& a, Raw<T>& b, const T* base, uint32_t at, const Chunks& c,
                                         bool vec) {
    const T* p0 = reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + (at + c.o0));
    const T* p1 = reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + (at + c.o0 + c.d1));
    if (FULL) {
        a.load(p0);
        b.load(p1);
    } else {
        if (!c.in0) a.zero();
        else if (vec) a.load(p0);
        else a.load_each(p0);
        if (!c.in1) b.zero();
        else if (vec) b.load(p1);
        else b.load_each(p1);
    }
}

__device__ __forceinline__ void store8(float* p, const f2* f) {
    __stcs(reinterpret_cast<ulonglong2*>(p), make_ulonglong2(f[0], f[1]));
    __stcs(reinterpret_cast<ulonglong2*>(p) + 1, make_ulonglong2(f[2], f[3]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f2* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpair(f[i], a, b);
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

template <bool FULL, typename T>
__device__ __forceinline__ void store_row(T* base, uint32_t at, const Chunks& c, const f2* u, const f2* v) {
    char* p = reinterpret_cast<char*>(base);
    if (FULL || c.in0) store8(reinterpret_cast<T*>(p + (at + c.o0)), u);
    if (FULL || c.in1) store8(reinterpret_cast<T*>(p + (at + c.o0 + c.d1)), v);
}

// Sum over the `lanes` lanes of a row (all lanes of the warp take part).
__device__ __forceinline__ float row_sum(float v, int lanes) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
        if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The 64-bit fraction of a turn that one position is worth.
__device__ __forceinline__ unsigned long long turn_of(double freq) {
    const double t = freq * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// Cosines, sines and negative sines of a tile's tokens, each [token][pair]; rot / 2 pairs a
// token, `pitch` floats apart (a multiple of 4).
template <int N> struct Table {
    float cos[N], sin[N], neg[N];
};
__host__ __device__ __forceinline__ int table_pitch(int rot) { return (rot / 2 + 3) / 4 * 4; }
// A thread's pair and its fraction of a turn stay the same for all tiles.
struct Angles {
    unsigned long long turn;
    int pair, first, per;   // threads of the same pair are `per` tokens apart
    __device__ __forceinline__ Angles(const QkArgs& a) {
        const int half = max(a.rot / 2, 1);
        per = kThreads / half;
        pair = threadIdx.x % half;
        first = threadIdx.x / half;
        if (a.rot == 0 || first >= per) first = 1 << 30;  // no part in it
        turn = first < per ? turn_of(a.freq[pair]) : 0;
    }
    template <int N>
    __device__ __forceinline__ void make(const QkArgs& a, long long t0, int n, Table<N>& cs) const {
        const int pitch = table_pitch(a.rot);
        for (int t = first; t < n; t += per) {
            const unsigned long long phase = (unsigned long long)a.pos[t0 + t] * turn;
            // in half turns, -1 to 1
            const float r = (float)(long long)phase * 1.0842021724855044e-19f;  // 2^-63
            float s, c;
            sincospif(r, &s, &c);
            const int at = t * pitch + pair;
            cs.cos[at] = c;
            cs.sin[at] = s;
            cs.neg[at] = -s;
        }
    }
};

// u and v (8 elements each, pairs) turned by the token's angles (BACK: turned back), in
// place.  `c`, `s`, `m`: the token's cosines, sines and their negatives; `buf`: this row's
// floats of shared memory (kShared).
template <int MODE, bool BACK>
__device__ __forceinline__ void turn(const QkArgs& a, const float* c, const float* s, const float* m,
                                     int p, int c0, int c1, f2* u, f2* v, float* buf) {
    const int half = a.rot / 2;
    if constexpr (MODE == kHalves) {
        if (p < a.rot / 16) {
            if (BACK) {
                const float* t = s;
                s = m;
                m = t;
            }
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const ulonglong2 cc = *reinterpret_cast<const ulonglong2*>(c + c0 + 2 * i);
                const ulonglong2 ss = *reinterpret_cast<const ulonglong2*>(s + c0 + 2 * i);
                const ulonglong2 mm = *reinterpret_cast<const ulonglong2*>(m + c0 + 2 * i);
                const f2 ce[2] = {cc.x, cc.y}, se[2] = {ss.x, ss.y}, me[2] = {mm.x, mm.y};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const f2 x = u[i + e], y = v[i + e];
                    u[i + e] = fma2(x, ce[e], mul2(y, me[e]));
                    v[i + e] = fma2(x, se[e], mul2(y, ce[e]));
                }
            }
        }
    } else if constexpr (MODE == kNeighbours) {
        auto both = [&](f2* x, int col) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = (col >> 1) + i;
                if (k < half) {
                    const float co = c[k], si = BACK ? -s[k] : s[k];
                    float e, o;
                    unpair(x[i], e, o);
                    x[i] = ::pair(fmaf(e, co, -o * si), fmaf(e, si, o * co));
                }
            }
        };
        both(u, c0);
        both(v, c1);
    } else {
        __syncwarp();
        if (c0 < a.dim)
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f2*>(buf + c0 + 2 * i) = u[i];
        if (c1 < a.dim)
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f2*>(buf + c1 + 2 * i) = v[i];
        __syncwarp();
        auto each = [&](f2* x, int from) {
            if (from >= a.dim) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float t[2];
                unpair(x[i], t[0], t[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = from + 2 * i + e;
                    if (col >= a.rot) continue;
                    const bool first = col < half;
                    const int k = first ? col : col - half;
                    const float si = BACK ? -s[k] : s[k];
                    const float other = buf[first ? col + half : col - half];
                    t[e] = fmaf(t[e], c[k], first ? -other * si : other * si);
                }
                x[i] = ::pair(t[0], t[1]);
            }
        };
        each(u, c0);
        each(v, c1);
    }
}

// Both weights in shared memory, ones where there is none and for a lane's missing columns.
constexpr int kWeights = kMaxDim + 8;
__device__ __forceinline__ void load_weights(const QkArgs& a, float* w) {
    for (int e = threadIdx.x; e < 2 * kWeights; e += kThreads) {
        const float* p = a.w[e / kWeights];
        const int c = e % kWeights;
        w[e] = p && c < a.dim ? p[c] : 1.0f;
    }
}
__device__ __forceinline__ void weights_of(const float* w, int c0, int c1, f2* u, f2* v) {
    const ulonglong2* p0 = reinterpret_cast<const ulonglong2*>(w + c0);
    const ulonglong2* p1 = reinterpret_cast<const ulonglong2*>(w + c1);
    const ulonglong2 a = p0[0], b = p0[1], c = p1[0], d = p1[1];
    u[0] = a.x; u[1] = a.y; u[2] = b.x; u[3] = b.y;
    v[0] = c.x; v[1] = c.y; v[2] = d.x; v[3] = d.y;
}

// The rows (token, head) of a tile that one group of lanes takes, every `groups`th, and
// where they start in a tensor whose tokens are `stride` elements apart.
struct Walk {
    int t, h, dt, dh, heads;
    uint32_t at, step, wrap;  // bytes; a tile has less than 2^31 of them
    __device__ __forceinline__ Walk(int group, int groups, int n, int dim, long long stride, int size)
        : heads(n) {
        t = group / n;
        h = group - t * n;
        dt = groups / n;
        dh = groups - dt * n;
        at = (uint32_t)(t * stride + h * dim) * size;
        step = (uint32_t)(dt * stride + dh * dim) * size;
        wrap = (uint32_t)(stride - (long long)n * dim) * size;
    }
    __device__ __forceinline__ void next() {
        t += dt;
        h += dh;
        at += step;
        if (h >= heads) {
            h -= heads;
            ++t;
            at += wrap;
        }
    }
};

// Held angles: a lane keeps its pairs' angles in registers while it goes through its part of one
// token's heads.
struct Held {
    f2 c[4], s[4];         // cosines and sines
    bool turned;
    // pairs col .. col + 7 of the token at `at`; BACK: turned back
    template <bool BACK, int N>
    __device__ __forceinline__ void take(const Table<N>& table, int at, int col, bool on) {
        turned = on;
        if (!on) return;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const ulonglong2 cc = *reinterpret_cast<const ulonglong2*>(table.cos + at + col + 2 * i);
            const ulonglong2 ss = *reinterpret_cast<const ulonglong2*>((BACK ? table.neg : table.sin) + at + col + 2 * i);
            c[i] = cc.x; c[i + 1] = cc.y;
            s[i] = ss.x; s[i + 1] = ss.y;
        }
    }
    __device__ __forceinline__ void turn(f2* u, f2* v) const {
        if (turned)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f2 x = u[i], y = v[i];
                u[i] = fma2(x, c[i], mul2(y, s[i] ^ 0x8000000080000000ull));
                v[i] = fma2(x, s[i], mul2(y, c[i]));
            }
    }
};
// The rows that a warp takes with held angles: one token's heads, q's and then k's, a group of
// lanes to each of as many neighbouring heads as it has groups.
constexpr int kHeldTokens = kThreads / 32;   // of a tile, one to a warp
struct Share {
    int group, groups, rows_q, rows;
    __device__ __forceinline__ Share(const QkArgs& a, int lanes) {
        groups = 32 / lanes;
        group = (threadIdx.x & 31) / lanes;
        rows_q = a.heads[0] / groups;
        rows = rows_q + a.heads[1] / groups;
    }
    __device__ __forceinline__ bool starts(int r) const { return r == 0 || r == rows_q; }
    __device__ __forceinline__ int of(int r) const { return r >= rows_q; }  // q or k
};

// A row group's shared memory for kShared.
template <int MODE> constexpr int kBufFloats = MODE == kShared ? kThreads * 16 : 4;

// CTAs walk the tokens, the next tile's sines and cosines made while this one's rows are on their
// way.  FULL: aligned rows of 16, 32, ... 256 columns, without checks.  HELD: as described above.
// 16384 tokens of 32 + 8 heads of 128 bf16 take 64 us, 5.2 TB/s, bound by HBM and 190 instructions a
// warp and 4 rows (not held 68 us, 293; held by three CTAs an SM 68 us; lanes of a warp on four
// tokens, 256 bytes of each at a time, 75 us).
template <typename TI, typename TO, int MODE, bool FULL, bool HELD>
__global__ void __launch_bounds__(kThreads, kFwdCtas) qk_fwd_kernel(const QkArgs a) {
    __shared__ __align__(16) Table<HELD ? kHeldTable : kTable> tables[2];
    __shared__ __align__(16) float weights[2 * kWeights];
    __shared__ __align__(16) float bufs[kBufFloats<MODE>];
    const int lanes = a.lanes, groups = kThreads / lanes;
    const int group = threadIdx.x / lanes, p = threadIdx.x % lanes;
    int c0, c1;
    lane_columns<MODE>(a, p, c0, c1);
    const Chunks in_x{c0 * (uint32_t)sizeof(TI), (c1 - c0) * (uint32_t)sizeof(TI), c0 < a.dim, c1 < a.dim};
    const Chunks in_y{c0 * (uint32_t)sizeof(TO), (c1 - c0) * (uint32_t)sizeof(TO), c0 < a.dim, c1 < a.dim};
    float* buf = MODE == kShared ? bufs + group * (16 * lanes) : nullptr;
    const int pitch = table_pitch(a.rot);
    const long long stride = (long long)gridDim.x * a.tile;
    long long t0 = (long long)blockIdx.x * a.tile;
    const Angles angles(a);
    load_weights(a, weights);
    if (t0 < a.tokens) angles.make(a, t0, (int)min((long long)a.tile, a.tokens - t0), tables[0]);
    // held: the next row is on its way, the next tile's first one too
    const Share share(a, HELD ? lanes : 1);
    Raw<TI> r0, r1;
    const TI* x = nullptr;
    auto ahead = [&](int row, long long t) {
        const int which = share.of(row);
        if (share.starts(row)) x = static_cast<const TI*>(a.x[which]) + t * a.stride[which] + share.group * a.dim;
        else x += share.groups * a.dim;
        load_row<true>(r0, r1, x, 0, in_x, true);
    };
    if (HELD && t0 + (threadIdx.x >> 5) < a.tokens) ahead(0, t0 + (threadIdx.x >> 5));
    __syncthreads();

    for (int k = 0; t0 < a.tokens; t0 += stride, k ^= 1) {
        const int n = (int)min((long long)a.tile, a.tokens - t0);
        const auto& table = tables[k];
        if (t0 + stride < a.tokens)  // the next tile's
            angles.make(a, t0 + stride, (int)min((long long)a.tile, a.tokens - t0 - stride), tables[k ^ 1]);
        if constexpr (HELD) {
            const int t = threadIdx.x >> 5;
            Held held;
            held.template take<false>(table, t * pitch, c0, p < a.rot / 16);
            TO* y = nullptr;
#pragma unroll 1
            for (int row = 0; row < (t < n ? share.rows : 0); ++row, y += share.groups * a.dim) {
                const int which = share.of(row);
                if (share.starts(row))
                    y = static_cast<TO*>(a.y[which]) + ((t0 + t) * a.heads[which] + share.group) * a.dim;
                f2 u[4], v[4], wu[4], wv[4];
                r0.get(u);
                r1.get(v);
                if (row + 1 < share.rows) ahead(row + 1, t0 + t);
                else if (t0 + stride + t < a.tokens) ahead(0, t0 + stride + t);
                f2 s = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) s = fma2(u[i], u[i], fma2(v[i], v[i], s));
                const float r = rsqrtf(fmaf(row_sum(sum2(s), lanes), a.inv_dim, a.eps));
                weights_of(weights + which * kWeights, c0, c1, wu, wv);
                const f2 r2 = pair(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = mul2(u[i], mul2(wu[i], r2));
                    v[i] = mul2(v[i], mul2(wv[i], r2));
                }
                held.turn(u, v);
                store_row<true>(y, 0, in_y, u, v);
            }
        } else
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int heads = a.heads[which];
            if (heads == 0) continue;
            const TI* x = static_cast<const TI*>(a.x[which]) + t0 * a.stride[which];
            TO* y = static_cast<TO*>(a.y[which]) + t0 * heads * a.dim;
            const bool vec = a.vec[which] != 0;
            const int rows = n * heads;
            // rows beyond the last are loaded as zeros and not stored: every lane of a
            // warp takes part in the shuffles
            Raw<TI> r0, r1;
            Walk in(group, groups, heads, a.dim, a.stride[which], sizeof(TI));
            int t = 0, t_next = 0;  // the rows' tokens
            uint32_t out = (uint32_t)(group * a.dim) * sizeof(TO);
            auto fetch = [&]() {
                t_next = min(in.t, n - 1);
                if (in.t < n) {
                    load_row<FULL>(r0, r1, x, in.at, in_x, vec);
                } else {
                    r0.zero();
                    r1.zero();
                }
                in.next();
            };
            fetch();
            for (int row = group; row - group < rows;
                 row += groups, out += (uint32_t)(groups * a.dim) * sizeof(TO)) {
                f2 u[4], v[4], wu[4], wv[4];
                r0.get(u);
                r1.get(v);
                t = t_next;
                if (row - group + groups < rows) fetch();
                f2 s = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) s = fma2(u[i], u[i], fma2(v[i], v[i], s));
                const float r = rsqrtf(fmaf(row_sum(sum2(s), lanes), a.inv_dim, a.eps));
                weights_of(weights + which * kWeights, c0, c1, wu, wv);
                const f2 r2 = pair(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = mul2(u[i], mul2(wu[i], r2));
                    v[i] = mul2(v[i], mul2(wv[i], r2));
                }
                const int at = t * pitch;
                turn<MODE, false>(a, table.cos + at, table.sin + at, table.neg + at, p, c0, c1, u, v, buf);
                if (row < rows) store_row<FULL>(y, out, in_y, u, v);
            }
        }
        __syncthreads();  // this table is read, the next one is made
    }
}

// A row's gradient in place of dy (g, q), already turned back, and its part of dw (none where the
// row is not there, with eps 0 either).
__device__ __forceinline__ void row_gradient(const QkArgs& a, int lanes, bool there, const f2* u, const f2* v,
                                             f2* g, f2* q, f2* wu, f2* wv, f2* sum) {
    f2 s2 = 0, m2 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s2 = fma2(u[i], u[i], fma2(v[i], v[i], s2));
        wu[i] = mul2(wu[i], g[i]);
        wv[i] = mul2(wv[i], q[i]);
        m2 = fma2(wu[i], u[i], fma2(wv[i], v[i], m2));
    }
    const float s = row_sum(sum2(s2), lanes), m = row_sum(sum2(m2), lanes);
    const float r = there ? rsqrtf(fmaf(s, a.inv_dim, a.eps)) : 0.0f;
    const float mr = -m * a.inv_dim * r * r;  // of mean(g w n) r, per x
    const f2 r2 = pair(r, r), mr2 = pair(mr, mr);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum[i] = fma2(g[i], mul2(u[i], r2), sum[i]);
        sum[4 + i] = fma2(q[i], mul2(v[i], r2), sum[4 + i]);
        g[i] = mul2(r2, fma2(mr2, u[i], wu[i]));
        q[i] = mul2(r2, fma2(mr2, v[i], wv[i]));
    }
}

// TI: the type of x and dx, TO: of dy.  16384 tokens of 32 heads of 128 bf16 take 77 us, 5.2 TB/s:
// 284 instructions a warp and 4 rows on two CTAs an SM (not held 99 us, 386; one float to an
// instruction 135 us).
template <typename TI, typename TO, int MODE, bool FULL, bool HELD>
__global__ void __launch_bounds__(kThreads, kBwdCtas) qk_bwd_kernel(const QkArgs a) {
    __shared__ __align__(16) Table<HELD ? kHeldTable : kTable> tables[2];
    __shared__ __align__(16) float weights[2 * kWeights];
    // rows' exchange, then the sums of dw; held: a thread's dw of q and k
    __shared__ __align__(16) float sums[kThreads * 16 * (HELD ? 2 : 1)];
    const int lanes = a.lanes, groups = kThreads / lanes;
    const int group = threadIdx.x / lanes, p = threadIdx.x % lanes;
    int c0, c1;
    lane_columns<MODE>(a, p, c0, c1);
    const Chunks in_x{c0 * (uint32_t)sizeof(TI), (c1 - c0) * (uint32_t)sizeof(TI), c0 < a.dim, c1 < a.dim};
    const Chunks in_y{c0 * (uint32_t)sizeof(TO), (c1 - c0) * (uint32_t)sizeof(TO), c0 < a.dim, c1 < a.dim};
    float* buf = sums + group * (16 * lanes);
    const int pitch = table_pitch(a.rot);
    const long long stride = (long long)gridDim.x * a.tile;
    long long t0 = (long long)blockIdx.x * a.tile;
    const Angles angles(a);
    load_weights(a, weights);
    if (t0 < a.tokens) angles.make(a, t0, (int)min((long long)a.tile, a.tokens - t0), tables[0]);
    // held: the next row is on its way, the next tile's first one too
    const Share share(a, HELD ? lanes : 1);
    Raw<TI> x0, x1;
    Raw<TO> d0, d1;
    const TI* x = nullptr;
    const TO* dy = nullptr;
    auto ahead = [&](int row, long long t) {
        const int which = share.of(row);
        if (share.starts(row)) {
            x = static_cast<const TI*>(a.x[which]) + t * a.stride[which] + share.group * a.dim;
            dy = static_cast<const TO*>(a.dy[which]) + (t * a.heads[which] + share.group) * a.dim;
        } else {
            x += share.groups * a.dim;
            dy += share.groups * a.dim;
        }
        load_row<true>(x0, x1, x, 0, in_x, true);
        load_row<true>(d0, d1, dy, 0, in_y, true);
    };
    if (HELD && t0 + (threadIdx.x >> 5) < a.tokens) ahead(0, t0 + (threadIdx.x >> 5));
    __syncthreads();

    f2 dw[2][8];  // of q and k (held: not in registers all along)
    f2* own = reinterpret_cast<f2*>(sums) + threadIdx.x;  // [2][8], kThreads apart
    if constexpr (HELD)
#pragma unroll
        for (int i = 0; i < 16; ++i) own[i * kThreads] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0;
    for (int k = 0; t0 < a.tokens; t0 += stride, k ^= 1) {
        const int n = (int)min((long long)a.tile, a.tokens - t0);
        const auto& table = tables[k];
        if (t0 + stride < a.tokens)  // the next tile's
            angles.make(a, t0 + stride, (int)min((long long)a.tile, a.tokens - t0 - stride), tables[k ^ 1]);
        if constexpr (HELD) {
            const int t = threadIdx.x >> 5;
            Held held;
            held.template take<true>(table, t * pitch, c0, p < a.rot / 16);
            int row = 0;
#pragma unroll 1
            for (int which = 0; which < (t < n ? 2 : 0); ++which) {
                const int end = which ? share.rows : share.rows_q;
                if (row == end) continue;
                TI* dx = static_cast<TI*>(a.y[which]) + ((t0 + t) * a.heads[which] + share.group) * a.dim;
                f2 sum[8];
                f2* at = own + which * 8 * kThreads;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = at[i * kThreads];
#pragma unroll 1
                for (; row < end; ++row, dx += share.groups * a.dim) {
                    f2 u[4], v[4], g[4], q[4], wu[4], wv[4];
                    x0.get(u);
                    x1.get(v);
                    d0.get(g);
                    d1.get(q);
                    if (row + 1 < share.rows) ahead(row + 1, t0 + t);
                    else if (t0 + stride + t < a.tokens) ahead(0, t0 + stride + t);
                    held.turn(g, q);
                    weights_of(weights + which * kWeights, c0, c1, wu, wv);
                    row_gradient(a, lanes, true, u, v, g, q, wu, wv, sum);
                    store_row<true>(dx, 0, in_x, g, q);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) at[i * kThreads] = sum[i];
            }
        } else {
        auto rows_of = [&](int which, f2* sum) {
            const int heads = a.heads[which];
            if (heads == 0) return;
            const TI* x = static_cast<const TI*>(a.x[which]) + t0 * a.stride[which];
            const TO* dy = static_cast<const TO*>(a.dy[which]) + t0 * heads * a.dim;
            TI* dx = static_cast<TI*>(a.y[which]) + t0 * heads * a.dim;
            const bool vec = a.vec[which] != 0;
            const int rows = n * heads;
            Raw<TI> x0, x1;
            Raw<TO> d0, d1;
            Walk in(group, groups, heads, a.dim, a.stride[which], sizeof(TI));
            int t = 0, t_next = 0;
            uint32_t up = (uint32_t)(group * a.dim) * sizeof(TO), out = (uint32_t)(group * a.dim) * sizeof(TI);
            auto fetch = [&]() {
                t_next = min(in.t, n - 1);
                if (in.t < n) {
                    load_row<FULL>(x0, x1, x, in.at, in_x, vec);
                    load_row<FULL>(d0, d1, dy, up, in_y, true);
                } else {
                    x0.zero(); x1.zero(); d0.zero(); d1.zero();
                }
                in.next();
                up += (uint32_t)(groups * a.dim) * sizeof(TO);
            };
            fetch();
            for (int row = group; row - group < rows;
                 row += groups, out += (uint32_t)(groups * a.dim) * sizeof(TI)) {
                f2 u[4], v[4], g[4], q[4], wu[4], wv[4];
                x0.get(u);
                x1.get(v);
                d0.get(g);
                d1.get(q);
                t = t_next;
                if (row - group + groups < rows) fetch();
                const int at = t * pitch;
                turn<MODE, true>(a, table.cos + at, table.sin + at, table.neg + at, p, c0, c1, g, q, buf);
                weights_of(weights + which * kWeights, c0, c1, wu, wv);
                row_gradient(a, lanes, row < rows, u, v, g, q, wu, wv, sum);
                if (row < rows) store_row<FULL>(dx, out, in_x, g, q);
            }
        };
        rows_of(0, dw[0]);
        rows_of(1, dw[1]);
        }
        __syncthreads();  // this table is read, the next one is made
    }
    if (!a.join) return;
    if constexpr (HELD) {
        // (own words only, before they are written over)
#pragma unroll
        for (int i = 0; i < 16; ++i) dw[i / 8][i % 8] = own[i * kThreads];
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        // the CTA's sum over its groups, in their order
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c0 < a.dim) *reinterpret_cast<f2*>(sums + group * a.dim + c0 + 2 * i) = dw[which][i];
            if (c1 < a.dim) *reinterpret_cast<f2*>(sums + group * a.dim + c1 + 2 * i) = dw[which][4 + i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            float s = 0.0f;
            for (int j = 0; j < groups; ++j) s += sums[j * a.dim + c];
            a.partial[((long long)blockIdx.x * 2 + which) * a.dim + c] = s;
        }
    }
}

// dw of q and k (columns 0 .. 2 dim - 1) from the CTAs' sums: a warp's lanes take 32
// columns, 32 warps every 32nd CTA, joined in their order.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const float* partial, int ctas, int dim,
                                                     float* dwq, float* dwk) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < 2 * dim)
#pragma unroll 8
        for (int j = warp; j < ctas; j += 32) s += partial[(long long)j * 2 * dim + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * dim) {
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) t += part[j][lane];
        float* out = c < dim ? dwq : dwk;
        if (out) out[c < dim ? c : c - dim] = t;
    }
}

// ------------------------------------------------------------------- host

struct Span { const void* p; size_t n; };

size_t strided_bytes(long long rows, long long width, long long stride, size_t es) {
    return rows > 0 ? ((size_t)(rows - 1) * stride + width) * es : 0;
}

bool sizes_ok(long long tokens, int qheads, int kheads, int dim) {
    return tokens >= 0 && qheads >= 0 && kheads >= 0 && dim >= 1;
}

// heads and tokens that an int can count together, heads of 8 to 256 columns
bool sizes_fit(long long tokens, int qheads, int kheads, int dim) {
    return dim % 8 == 0 && dim <= kMaxDim && qheads <= 4096 && kheads <= 4096 &&
           tokens <= (1LL << 40);
}

// Lanes of a row, tokens of a tile.
void plan(QkArgs& a, int mode, long long slots) {
    const int chunks = a.dim / 8;
    const int need = mode == kHalves ? a.rot / 16 + (chunks - a.rot / 8 + 1) / 2 : (chunks + 1) / 2;
    a.lanes = 1;
    while (a.lanes < need) a.lanes *= 2;
    // rows for four rounds of the CTA's groups, no more tokens than the table holds, and
    // few enough that all the CTAs have some
    const int groups = kThreads / a.lanes, heads = std::max(1, a.heads[0] + a.heads[1]);
    long long t = (4 * groups + heads - 1) / heads;
    if (a.rot > 0) t = std::min<long long>(t, kTable / table_pitch(a.rot));
    t = std::min(t, (a.tokens + slots - 1) / slots);
    // what lies between its first and last element fits 31 bits (a single token's heads do)
    t = std::min(t, (1LL << 29) / std::max(1LL, std::max(a.stride[0], a.stride[1])) - 1);
    t = std::min(t, (1LL << 29) / ((long long)heads * a.dim));
    a.tile = (int)std::max(1LL, t);
}

template <typename F>
bool by_types(ssm_dtype_t in, ssm_dtype_t out, F&& f) {
    using B = __nv_bfloat16;
    if (in == SSM_F32) return out == SSM_F32 ? f(float{}, float{}) : f(float{}, B{});
    return out == SSM_F32 ? f(B{}, float{}) : f(B{}, B{});
}

template <typename F>
void by_mode(int mode, F&& f) {
    if (mode == kHalves) f(std::integral_constant<int, kHalves>{});
    else if (mode == kNeighbours) f(std::integral_constant<int, kNeighbours>{});
    else f(std::integral_constant<int, kShared>{});
}

// Rows of 16, 32, ... 256 columns that are aligned: no lane goes without
bool whole(const QkArgs& a) {
    for (int i = 0; i < 2; ++i)
        if (a.heads[i] > 0 && !a.vec[i]) return false;
    return a.dim == 16 * a.lanes;
}

// Whether angles are held: with heads for all of a warp's groups of lanes, and whole tiles for every
// CTA.  With fewer tokens or other heads rows are spread over all lanes instead.
bool hold(QkArgs& a, int mode, long long slots) {
    const int groups = 32 / a.lanes;
    if (mode != kHalves || !whole(a) || a.heads[0] % groups || a.heads[1] % groups ||
        kHeldTokens * table_pitch(a.rot) > kHeldTable || a.tokens < slots * kHeldTokens)
        return false;
    a.tile = kHeldTokens;
    return true;
}

ssm_status_t check_sizes(const QkArgs& a, int interleaved, ssm_dtype_t in, ssm_dtype_t out) {
    using namespace ssm_host;
    if (!sizes_ok(a.tokens, a.heads[0], a.heads[1], a.dim) || a.rot < 0 || a.rot > a.dim ||
        a.rot % 2 || (interleaved != 0 && interleaved != 1))
        return SSM_ERR_SHAPE;
    for (int i = 0; i < 2; ++i)
        if (a.heads[i] > 0 && a.stride[i] < (long long)a.heads[i] * a.dim) return SSM_ERR_SHAPE;
    if (!dtype_ok(in) || !dtype_ok(out)) return SSM_ERR_DTYPE;
    if (!sizes_fit(a.tokens, a.heads[0], a.heads[1], a.dim)) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

int mode_of(const QkArgs& a, int interleaved) {
    return interleaved ? kNeighbours : a.rot % 16 == 0 ? kHalves : kShared;
}

// Fills what the forward and the gradient share and checks the inputs they share.
ssm_status_t shared_args(QkArgs& a, ssm_dtype_t in) {
    using namespace ssm_host;
    for (int i = 0; i < 2; ++i) {
        if (a.heads[i] == 0) continue;
        if (!a.x[i]) return SSM_ERR_NULL;
        if (reinterpret_cast<uintptr_t>(a.x[i]) % dtype_size(in)) return SSM_ERR_ALIGN;
        if (a.w[i] && !aligned16(a.w[i])) return SSM_ERR_ALIGN;
        a.vec[i] = aligned16(a.x[i]) && a.stride[i] * dtype_size(in) % 16 == 0;
    }
    if (a.rot > 0 && (!a.pos || !a.freq)) return SSM_ERR_NULL;
    if (a.rot > 0 && (reinterpret_cast<uintptr_t>(a.pos) % 8 || !aligned16(a.freq)))
        return SSM_ERR_ALIGN;
    a.inv_dim = 1.0f / (float)a.dim;
    return SSM_OK;
}

}  // namespace

extern "C" ssm_status_t ssm_qk_norm_rope_fwd(
    const void* q, const void* k, long long q_stride, long long k_stride, const float* q_weight,
    const float* k_weight, const long long* positions, const double* inv_freq, float eps,
    int rot_dim, int interleaved, void* q_out, void* k_out, long long tokens, int qheads,
    int kheads, int headdim, ssm_dtype_t in_dtype, ssm_dtype_t out_dtype, void* stream) {
    using namespace ssm_host;
    QkArgs a{};
    a.x[0] = q; a.x[1] = k; a.stride[0] = q_stride; a.stride[1] = k_stride;
    a.w[0] = q_weight; a.w[1] = k_weight; a.pos = positions; a.freq = inv_freq;
    a.eps = eps; a.rot = rot_dim; a.tokens = tokens; a.heads[0] = qheads; a.heads[1] = kheads;
    a.dim = headdim; a.y[0] = q_out; a.y[1] = k_out;
    if (ssm_status_t st = check_sizes(a, interleaved, in_dtype, out_dtype)) return st;
    if (tokens == 0 || qheads + kheads == 0) return SSM_OK;
    if (ssm_status_t st = shared_args(a, in_dtype)) return st;
    size_t xb[2], yb[2];
    for (int i = 0; i < 2; ++i) {
        const long long width = (long long)a.heads[i] * headdim;
        xb[i] = width ? strided_bytes(tokens, width, a.stride[i], dtype_size(in_dtype)) : 0;
        yb[i] = (size_t)tokens * width * dtype_size(out_dtype);
        if (width && !a.y[i]) return SSM_ERR_NULL;
        if (width && !aligned16(a.y[i])) return SSM_ERR_ALIGN;
    }
    const Span ins[] = {{q, xb[0]}, {k, xb[1]}, {q_weight, (size_t)headdim * 4},
                        {k_weight, (size_t)headdim * 4},
                        {positions, rot_dim ? (size_t)tokens * 8 : 0},
                        {inv_freq, (size_t)rot_dim * 4}};
    for (const Span& i : ins)
        for (int o = 0; o < 2; ++o)
            if (overlaps(a.y[o], yb[o], i.p, i.n)) return SSM_ERR_ALIAS;
    if (overlaps(q_out, yb[0], k_out, yb[1])) return SSM_ERR_ALIAS;

    const int sms = sm_count();
    if (sms == 0) return SSM_ERR_CUDA;
    const int mode = mode_of(a, interleaved);
    plan(a, mode, (long long)sms * kFwdCtas);
    const bool held = hold(a, mode, (long long)sms * kFwdCtas);
    const unsigned grid =
        (unsigned)std::min<long long>((tokens + a.tile - 1) / a.tile, (long long)sms * kFwdCtas);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    by_types(in_dtype, out_dtype, [&](auto ti, auto to) {
        by_mode(mode, [&](auto m) {
            constexpr int MODE = decltype(m)::value;
            using TI = decltype(ti);
            using TO = decltype(to);
            if constexpr (MODE == kHalves)
                if (held) {
                    qk_fwd_kernel<TI, TO, MODE, true, true><<<grid, kThreads, 0, s>>>(a);
                    return;
                }
            if (whole(a)) qk_fwd_kernel<TI, TO, MODE, true, false><<<grid, kThreads, 0, s>>>(a);
            else qk_fwd_kernel<TI, TO, MODE, false, false><<<grid, kThreads, 0, s>>>(a);
        });
        return true;
    });
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

extern "C" size_t ssm_qk_norm_rope_bwd_workspace_bytes(long long tokens, int qheads, int kheads,
                                                       int headdim) {
    if (!sizes_ok(tokens, qheads, kheads, headdim) || !sizes_fit(tokens, qheads, kheads, headdim))
        return 0;
    return 256 + (size_t)std::min<long long>(tokens, kBwdMost) * 2 * headdim * 4;
}

extern "C" ssm_status_t ssm_qk_norm_rope_bwd(
    const void* dq_out, const void* dk_out, const void* q, const void* k, long long q_stride,
    long long k_stride, const float* q_weight, const float* k_weight, const long long* positions,
    const double* inv_freq, float eps, int rot_dim, int interleaved, void* dq, void* dk,
    float* dq_weight, float* dk_weight, long long tokens, int qheads, int kheads, int headdim,
    ssm_dtype_t in_dtype, ssm_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
    void* stream) {
    using namespace ssm_host;
    QkArgs a{};
    a.x[0] = q; a.x[1] = k; a.stride[0] = q_stride; a.stride[1] = k_stride;
    a.w[0] = q_weight; a.w[1] = k_weight; a.pos = positions; a.freq = inv_freq;
    a.eps = eps; a.rot = rot_dim; a.tokens = tokens; a.heads[0] = qheads; a.heads[1] = kheads;
    a.dim = headdim; a.dy[0] = dq_out; a.dy[1] = dk_out; a.y[0] = dq; a.y[1] = dk;
    a.join = dq_weight || dk_weight;
    if (ssm_status_t st = check_sizes(a, interleaved, in_dtype, out_dtype)) return st;
    float* dws[2] = {dq_weight, dk_weight};
    for (float* d : dws)
        if (d && !aligned16(d)) return SSM_ERR_ALIGN;
    const size_t wb = (size_t)headdim * 4;
    if (overlaps(dq_weight, wb, dk_weight, wb)) return SSM_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0 || qheads + kheads == 0) {
        for (float* d : dws)
            if (d && cudaMemsetAsync(d, 0, wb, s) != cudaSuccess) return SSM_ERR_CUDA;
        return SSM_OK;
    }
    if (ssm_status_t st = shared_args(a, in_dtype)) return st;
    size_t xb[2], yb[2], gb[2];
    for (int i = 0; i < 2; ++i) {
        const long long width = (long long)a.heads[i] * headdim;
        xb[i] = width ? strided_bytes(tokens, width, a.stride[i], dtype_size(in_dtype)) : 0;
        yb[i] = (size_t)tokens * width * dtype_size(out_dtype);
        gb[i] = (size_t)tokens * width * dtype_size(in_dtype);
        if (width && (!a.dy[i] || !a.y[i])) return SSM_ERR_NULL;
        if (width && (!aligned16(a.dy[i]) || !aligned16(a.y[i]))) return SSM_ERR_ALIGN;
    }
    const size_t need = ssm_qk_norm_rope_bwd_workspace_bytes(tokens, qheads, kheads, headdim);
    if (a.join && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
    if (a.join && !aligned16(workspace)) return SSM_ERR_ALIGN;
    const Span ins[] = {{q, xb[0]}, {k, xb[1]}, {dq_out, yb[0]}, {dk_out, yb[1]}, {q_weight, wb},
                        {k_weight, wb}, {positions, rot_dim ? (size_t)tokens * 8 : 0},
                        {inv_freq, (size_t)rot_dim * 4}};
    const Span outs[] = {{dq, gb[0]}, {dk, gb[1]}, {dq_weight, wb}, {dk_weight, wb},
                         {workspace, a.join ? need : 0}};
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;

    const int mode = mode_of(a, interleaved);
    plan(a, mode, kBwdMost);
    const bool held = hold(a, mode, kBwdMost);
    const unsigned grid = (unsigned)std::min<long long>((tokens + a.tile - 1) / a.tile, kBwdMost);
    a.partial = static_cast<float*>(workspace);
    by_types(in_dtype, out_dtype, [&](auto ti, auto to) {
        by_mode(mode, [&](auto m) {
            constexpr int MODE = decltype(m)::value;
            using TI = decltype(ti);
            using TO = decltype(to);
            if constexpr (MODE == kHalves)
                if (held) {
                    qk_bwd_kernel<TI, TO, MODE, true, true><<<grid, kThreads, 0, s>>>(a);
                    return;
                }
            if (whole(a)) qk_bwd_kernel<TI, TO, MODE, true, false><<<grid, kThreads, 0, s>>>(a);
            else qk_bwd_kernel<TI, TO, MODE, false, false><<<grid, kThreads, 0, s>>>(a);
        });
        return true;
    });
    if (a.join)
        qk_dw_kernel<<<(2 * headdim + 31) / 32, 1024, 0, s>>>(a.partial, (int)grid, headdim,
                                                              dq_weight, dk_weight);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}
