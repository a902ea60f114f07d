// gated_delta.cuh -- what the gated delta rule's forward (gated_delta.cu) and gradient
// (gated_delta_bwd.cu) share: the chunked form, the records kept per chunk and head,
// operand tiles and copies.
//
// Per head, with the state S (dstate x headdim here), for chunks of 64 steps that start
// from S0 (G_i = sum of g up to step i, everything inside the chunk):
//   D_ij = exp(G_i - G_j), j <= i;   e_i = exp(G_i);   w_j = exp(G_63 - G_j)
//   A_ij = beta_i (k_i . k_j) D_ij, j < i;   T = (1 + A)^-1;   b = diag(beta)
//   R = V - e K S0                      what each step's value is off the carried state
//   U = T b R                           the steps' updates
//   Y = e Q S0 + P b R,    P = ((Q K^T) D) T
//   S1 = e_63 S0 + H b R,  H = K^T diag(w) T
// P and H depend on q, k and the gates alone, so one kernel makes them for all chunks at
// once, and the chain over the chunks is two products deep: K S0 and H b R.
// b goes with R, not into P and H, for the gradient's sake: theirs with respect to b R is z, of
// which dR = b z and dbeta_i = z_i . E_i, with the steps' errors E = N R, N = b^-1 T b, U = b E.
// No step's small beta is ever rounded beside other steps' larger ones and divided by.
//
// Operands are fp16 under one power of two per tile, chosen from the tile's largest value
// or a bound of it: bf16 inputs are exact in it down to 2^-30 of that, a value as the sum
// of two fp16 (hi + lo) is to 2^-22 or 2^-39 of the bound, where two bf16 leave 2^-17 and cost the
// same products.  (With bf16 the state of 1000 steps was 5e-6 off, 2-norm.)
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace gdn {

using namespace ssm;

constexpr int kC = 64;            // steps of a chunk
constexpr int kPan = 64;          // columns of headdim that one chain takes
constexpr uint32_t kTile = 8192;  // a 64 x 64 fp16 tile: 64 rows of 128 bytes

// The gates of a record: base-2 logarithms of the decay from the chunk's start as the
// sum of two floats, a bit for every step that learns nothing, and what the tiles have to
// be multiplied with.
struct Gates {
    float hi[kC], lo[kC];
    float beta[kC];
    unsigned long long masked;
    float s_k, s_h, s_p, s_n;
    float e_max;   // the largest decay from the chunk's start to a step
    float b_top, b_down;  // a power of two that no beta is above, 1 at least, and its inverse
    // no |H e b|, 64 |P e b| or |N e| is above these, e and b of the column's step: of products with
    // what has decayed (or grown) since the chunk's start
    float h_e, p_e, n_e;
    uint16_t s_q[kC];        // in bf16
    __device__ __forceinline__ float q_factor(int i) const { return __uint_as_float((uint32_t)s_q[i] << 16); }
};
// Q has a factor of its own, s_q, for each step: the same for all that learn, so that dY may enter
// products with P (held without s_q) and Q under s_q; a masked step whose q is larger than theirs (it may
// be padding) has its own and takes none of their bits.
constexpr uint32_t kGateBytes = 1024;
static_assert(sizeof(Gates) <= kGateBytes, "gates fit their place");

// The record of one chunk and head (bytes): gates | panels of K and Q (64 columns of
// dstate: 64 rows each) | H hi | H lo (dstate rows) | P hi | P lo | N.  Tiles are stored as
// they lie in shared memory: rows of 128 bytes whose 16-byte pieces are XORed with (row mod
// 8), so that one bulk copy brings in what the chain needs.
__host__ __device__ constexpr uint32_t h_bytes(int dk) { return (uint32_t)dk * 128u; }
__host__ __device__ constexpr uint32_t kq_bytes(int dk) { return (uint32_t)(dk / 64) * 2 * kTile; }
__host__ __device__ constexpr uint32_t rec_kq(int) { return kGateBytes; }
__host__ __device__ constexpr uint32_t rec_h(int dk) { return kGateBytes + kq_bytes(dk); }
__host__ __device__ constexpr uint32_t rec_p(int dk) { return rec_h(dk) + 2 * h_bytes(dk); }
__host__ __device__ constexpr uint32_t rec_n(int dk) { return rec_p(dk) + 2 * kTile; }
__host__ __device__ constexpr uint32_t rec_bytes(int dk) { return rec_n(dk) + kTile; }
// What training keeps for each chunk, head and 64 columns of headdim, rounded to one fp16:
// R | S0 | factors (forward), z | dY | L | their factors (gradient).  Only dq, dk, dg and dbeta come
// from them.  The forward's factors: of E = N R (the products of the tiles), of S0, of U (from a
// bound), and what takes E to U's.
constexpr uint32_t kFactorBytes = 128;
__host__ __device__ constexpr uint32_t kept_bytes(int dk) { return kTile + h_bytes(dk) + kFactorBytes; }
__host__ __device__ constexpr uint32_t adjoint_bytes(int dk) { return 2 * kTile + h_bytes(dk) + kFactorBytes; }

__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
    return ex2_approx((hi_i - hi_j) + (lo_i - lo_j));
}

// ------------------------------------------------- two floats to an instruction

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
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Decays from steps j .. j + 3 to one whose logarithms are -mh and -ml (both halves of a pair);
// 0 behind `last`.
__device__ __forceinline__ void decays4(const Gates* g, int j, f2 mh, f2 ml, int last, float* d) {
    const ulonglong2 h = *reinterpret_cast<const ulonglong2*>(g->hi + j);
    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(g->lo + j);
    unpair(add2(add2(h.x, mh), add2(l.x, ml)), d[0], d[1]);
    unpair(add2(add2(h.y, mh), add2(l.y, ml)), d[2], d[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = j + e <= last ? ex2_approx(-d[e]) : 0.0f;
}

// ------------------------------------------------------------------ rounding

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// N pairs as hi + lo.
template <int N>
__device__ __forceinline__ void split(const f2* x, uint32_t* hi, uint32_t* lo) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float a, b;
        unpair(x[e], a, b);
        hi[e] = pack_f16(a, b);
        asm("{\n\t.reg .b16 p, q, m;\n\t"
            "mov.b32 {p, q}, %2;\n\t"
            "mov.b16 m, 0xbc00;\n\t"  // -1
            "fma.rn.f32.f16 %0, p, m, %0;\n\t"
            "fma.rn.f32.f16 %1, q, m, %1;\n\t}"
            : "+f"(a), "+f"(b)
            : "r"(hi[e]));
        lo[e] = pack_f16(a, b);
    }
}
template <int N>
__device__ __forceinline__ void round_to(const f2* x, uint32_t* hi) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float a, b;
        unpair(x[e], a, b);
        hi[e] = pack_f16(a, b);
    }
}
template <int N>
__device__ __forceinline__ void scaled(const f2* x, float scale, f2* y) {
    const f2 s = pair(scale, scale);
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = mul2(x[e], s);
}
// 8, 16 or 32 columns of this thread's lane of tensor memory, as pairs.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, f2* v) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pair(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, f2* v) {
    float x[32];
    ssm::tmem_ld32(taddr, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = pair(x[2 * e], x[2 * e + 1]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, f2* v) {
    float x[16];
    ssm::tmem_ld16(taddr, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = pair(x[2 * e], x[2 * e + 1]);
}

// A tile's factor: a power of two that brings `most` (the largest magnitude, or a bound of
// it) to 2^top or less than twice that; `back` undoes it.  Infinities and NaN stay what
// they are, values below 2^-100 count as that.
__device__ __forceinline__ float tile_scale(float most, int top, float& back) {
    const uint32_t e = min(max(__float_as_uint(most) >> 23 & 0xffu, 27u), 254u);
    const uint32_t f = 254u + (uint32_t)top - e;   // 127 + top - (e - 127)
    const uint32_t g = min(f, 253u);
    back = __uint_as_float((254u - g) << 23);
    return __uint_as_float(g << 23);
}
// The inverse of a power of two.
__device__ __forceinline__ float inverse(float v) { return __uint_as_float((254u << 23) - __float_as_uint(v)); }
// A product of a tile's factor with others: it overflows where the tile's values are 0, or so small
// that they count as 0, and must leave them that.
__device__ __forceinline__ float finite_factor(float f) { return fabsf(f) > 1.7e38f ? copysignf(1.7e38f, f) : f; }
constexpr int kTop = 12;    // of a measured maximum
constexpr int kBoundTop = 14;  // of a bound
// The largest stored magnitude of a tile scaled by its maximum.
constexpr float kTopValue = 8192.0f;

// The largest magnitude of N pairs over a warp (NaN aside).
template <int N>
__device__ __forceinline__ float warp_most(const f2* v) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float a, b;
        unpair(v[e], a, b);
        asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(a), "f"(b));
    }
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}
// Infinities become NaN, which largest values do not see: what is not finite does not take
// the others' bits.
template <int N>
__device__ __forceinline__ void drop_infinities(f2* v) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = fma2(v[e], 0, v[e]);
}
template <int N>
__device__ __forceinline__ float warp_most_or_nan(f2* v) {
    float m = warp_most<N>(v);
    if (m == __int_as_float(0x7f800000)) {
        drop_infinities<N>(v);
        m = warp_most<N>(v);
    }
    return m;
}
__device__ __forceinline__ float warp_most(float m) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}
template <int N>
__device__ __forceinline__ float most_of(const float* s) {
    float m = s[0];
#pragma unroll
    for (int e = 1; e < N; ++e) m = fmaxf(m, s[e]);
    return m;
}

// -------------------------------------------------------------------- tiles

// Byte offset of 16-byte piece c of row r of a tile of 128-byte rows.
__device__ __forceinline__ uint32_t piece(int r, int c) {
    return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}
// N columns, 8, 16 or 32.
template <int N>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, f2* v) {
    if constexpr (N == 8) tmem_ld8(taddr, v);
    else if constexpr (N == 16) tmem_ld16(taddr, v);
    else tmem_ld32(taddr, v);
}
// 8 N values (4 N packed pairs) as pieces c0 .. c0 + N - 1 of row r.
template <int N>
__device__ __forceinline__ void put_pieces(uint8_t* tile, int r, int c0, const uint32_t* w) {
#pragma unroll
    for (int c = 0; c < N; ++c)
        *reinterpret_cast<uint4*>(tile + piece(r, c0 + c)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
// 32 values (16 packed pairs) as pieces c0 .. c0 + 3 of row r.
__device__ __forceinline__ void put32(uint8_t* tile, int r, int c0, const uint32_t* w) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(tile + piece(r, c0 + c)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
__device__ __forceinline__ void unpack8_bf16(uint4 w, f2* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = pair(bf16lo(u[e]), bf16hi(u[e]));
}
__device__ __forceinline__ void unpack8_f16(uint4 w, f2* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 h = unpack_f16(u[e]);
        f[e] = pair(h.x, h.y);
    }
}
// The largest finite magnitude of bf16, two at a time.  Magnitudes compare as integers, and
// with the least exponent added infinities and NaN are negative ones: a value that is not
// finite does not take the others' bits.
struct MostBf16 {
    uint32_t m = 0x00800080u;
    __device__ __forceinline__ void see(uint4 w) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            asm("max.s16x2 %0, %0, %1;" : "+r"(m) : "r"((u[e] & 0x7fff7fffu) + 0x00800080u));
    }
    __device__ __forceinline__ float value() const {
        return __uint_as_float((max(m >> 16, m & 0xffffu) - 0x80u) << 16);
    }
};
// 8 pairs to 16 consecutive elements whose address is a multiple of 32 bytes (a whole sector
// of bf16 to a lane).
__device__ __forceinline__ void store16(__nv_bfloat16* p, const f2* o) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float a, b;
        unpair(o[e], a, b);
        w[e] = pack_bf16(a, b);
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// 4 pairs to 8 consecutive elements.
__device__ __forceinline__ void store8(float* p, const f2* o) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(o[0], o[1]);
    *reinterpret_cast<ulonglong2*>(p + 4) = make_ulonglong2(o[2], o[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f2* o) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        unpair(o[e], a, b);
        w[e] = pack_bf16(a, b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// Whether all rows of `cols` bf16 lie at multiples of 32 bytes (tensors start at any of 16).
__device__ __forceinline__ bool rows_of_sectors(const void* base, int cols) {
    return cols % 16 == 0 && (reinterpret_cast<uintptr_t>(base) & 31) == 0;
}
// N pairs as the columns col .. of a row of `cols` whose column col lies at p (cols a multiple
// of 8); `wide`: rows_of_sectors (col is a multiple of 16).
template <int N, typename T>
__device__ __forceinline__ void store_row(T* p, const f2* o, int col, int cols, bool wide) {
    if (sizeof(T) == 2 && wide && N % 8 == 0) {
        if constexpr (sizeof(T) == 2 && N % 8 == 0)
#pragma unroll
            for (int e = 0; e < N; e += 8)
                if (col + 2 * e < cols) store16(p + 2 * e, o + e);
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 4)
            if (col + 2 * e < cols) store8(p + 2 * e, o + e);
    }
}
__device__ __forceinline__ float gate_at(const void* p, long long i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                : static_cast<const float*>(p)[i];
}

// Instruction descriptor, kind::f16 with fp16 operands and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
    mma_bf16(d_tmem, a_desc, b_desc, idesc, accumulate);  // the types are the descriptor's
}

// The same from a whole warp, whose operands are then the same for all its lanes (they need not be
// taken from vector to uniform registers one by one): the lane with `one` set issues it.
__device__ __forceinline__ void mma_f16_warp(int one, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ int elect_one() {
    int one;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, e;\n\t}"
        : "=r"(one));
    return one;
}
// A tile's descriptor moved on by `bytes`: its address is the low word's first bits.  One addition, where
// a descriptor made anew takes five instructions of the one thread that issues all products.
__device__ __forceinline__ uint64_t moved(uint64_t desc, uint32_t bytes) {
    return (desc & 0xffffffff00000000ull) | ((uint32_t)desc + (bytes >> 4));
}
// K-major operand (rows of 64 values along the contraction) of R rows, k-step kk.
template <int R>
__device__ __forceinline__ uint64_t kdesc(uint32_t tile, int kk) {
    return moved(smem_desc_k128(tile), (uint32_t)((kk >> 2) * (R * 128) + (kk & 3) * 32));
}
// MN-major operand (one row of 64 values per step of the contraction), k-step kk;
// further blocks of 64 `lbo` bytes apart.
__device__ __forceinline__ uint64_t mdesc(uint32_t tile, int kk, uint32_t lbo) {
    return moved(smem_desc_mn128(tile, lbo), (uint32_t)kk * 2048u);
}

// `bytes` (a multiple of 16) of global memory to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// `bytes` (a multiple of 16) of shared memory to global memory, in the thread's bulk group.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// One arrival of a warp whose lanes have all come this far.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Looks for what is due in a moment without being put to sleep first (a woken thread is
// some 200 cycles late, of the 3000 that a chunk takes).
__device__ __forceinline__ bool mbar_look(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = smem_u32(bar);
    for (int i = 0; i < 256; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        if (done) return true;
    }
    return false;
}
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, uint32_t* status) {
    return mbar_look(bar, parity) || mbar_wait(bar, parity, status);
}
// A wait that a whole warp takes together, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
    if (__all_sync(0xffffffffu, mbar_look(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

// Largest values that warps tell one another while products run, without a barrier: a word
// of shared memory each, its last byte the chunk it belongs to, rounded up to the others (it
// only enters bounds).  A word is written and read as a whole.
__device__ __forceinline__ void post_most(uint32_t* slot, float most, int chunk) {
    *reinterpret_cast<volatile uint32_t*>(slot) =
        (__float_as_uint(most) & 0xffffff00u) | ((uint32_t)(chunk + 1) & 0xffu);
}
// The largest of 4 N words once they all belong to `chunk`; false when that takes too long.
template <int N>
__device__ __forceinline__ bool read_most(const uint32_t* slots, int chunk, float& most, uint32_t* status) {
    const uint32_t tag = (uint32_t)(chunk + 1) & 0xffu, addr = smem_u32(slots);
    for (uint32_t tries = 0; tries < (1u << 26); ++tries) {
        uint32_t off = 0, m = 0;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint32_t w[4];
            asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(addr + 16 * n)
                         : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                off |= w[e] ^ tag;
                m = max(m, w[e]);
            }
        }
        if (__all_sync(0xffffffffu, (off & 0xffu) == 0)) {
            most = __uint_as_float(m | 0xffu);
            return true;
        }
    }
    record_status(status, SSM_ERR_TIMEOUT);
    return false;
}

// Registers move from the warps that load and multiply to the NW that compute: a kernel of 12
// warps has 168 a thread at launch, 64512 in all; then 8 warps have 224 and 4 have 56.  One of 20
// has 96, 61440 in all; then 16 have 104 and 4 have 64.
template <int NW>
__device__ __forceinline__ void take_registers() {
    if constexpr (NW == 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
}
template <int NW>
__device__ __forceinline__ void give_registers() {
    if constexpr (NW == 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}
constexpr int kSplitThreads = 384;

struct Dims {
    int batch, seqlen, heads, groups, dk, dv;
    int chunks, pans;   // ceil(seqlen / 64), ceil(dv / 64)
};

}  // namespace gdn

namespace gdn_host {

// (batch, seqlen, heads, dim) bf16 whose tokens are `step` elements apart, as a 4-D map
// {dim, heads, seqlen, batch} with boxes of 64 columns of one head and 64 steps (128-byte
// swizzle, zeros past any end).
inline bool make_map(CUtensorMap* map, const void* base, int batch, int seqlen, int heads, int dim,
                     long long step) {
    ssm_host::EncodeTiledFn fn = ssm_host::encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)seqlen,
                                (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)dim * 2, (cuuint64_t)step * 2,
                                   (cuuint64_t)step * 2 * seqlen};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)gdn::kC, 1};
    const cuuint32_t estride[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
              estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sizes as the entry points check them.
inline bool sizes_ok(int batch, int seqlen, int heads, int groups, int dk, int dv) {
    return batch >= 0 && seqlen >= 0 && heads >= 0 && groups >= 0 && dk >= 1 && dv >= 1 &&
           (groups == 0 ? heads == 0 : heads > 0 && heads % groups == 0);
}
inline bool sizes_fit(int batch, int seqlen, int heads, int dk, int dv) {
    return dk % 8 == 0 && dv % 8 == 0 && dk <= 128 && dv <= 256 && seqlen < (1 << 30) &&
           (long long)batch * heads * ((seqlen + 63LL) / 64) < (1LL << 30) &&
           (long long)batch * heads < (1LL << 30) / 4;
}
inline int dk_tile(int dk) { return dk <= 64 ? 64 : 128; }
inline size_t chunk_count(int batch, int seqlen, int heads) {
    return (size_t)batch * heads * (((size_t)seqlen + gdn::kC - 1) / gdn::kC);
}
// A word for each record, and one more
inline size_t flags_bytes(int batch, int seqlen, int heads) {
    return ((chunk_count(batch, seqlen, heads) + 1) * 4 + 1023) / 1024 * 1024;
}
inline size_t records_bytes(int batch, int seqlen, int heads, int dk) {
    return chunk_count(batch, seqlen, heads) * gdn::rec_bytes(dk_tile(dk));
}
inline size_t keep_bytes(int batch, int seqlen, int heads, int dk, int dv) {
    return chunk_count(batch, seqlen, heads) * ((dv + 63) / 64) * gdn::kept_bytes(dk_tile(dk));
}

inline size_t adjoints_bytes(int batch, int seqlen, int heads, int dk, int dv) {
    return chunk_count(batch, seqlen, heads) * ((dv + 63) / 64) * gdn::adjoint_bytes(dk_tile(dk));
}

struct Span { const void* p; size_t n; };

inline size_t strided_bytes(long long steps, long long width, long long stride, size_t es) {
    return steps > 0 ? ((size_t)(steps - 1) * stride + width) * es : 0;
}

}  // namespace gdn_host

namespace gdn_internal {

// The chunked forward over bf16 q, k, v: records and, where y, final_state or kept are
// given, the chain.  y may be NULL (kept states only).  Arguments are checked by the caller.
struct Forward {
    const void *q, *k, *v;
    long long q_step, k_step, v_step;
    const void *g, *beta;
    ssm_dtype_t gate_dtype;
    const float* initial_state;
    void* y;
    ssm_dtype_t out_dtype;
    float* final_state;
    uint8_t* records;
    uint8_t* kept;       // NULL: nothing is kept
    uint32_t* status;
    uint32_t* flags;     // flags_bytes, or NULL
    int batch, seqlen, heads, groups, dk, dv;
};
ssm_status_t chunked_forward(const Forward& f, cudaStream_t stream);

}  // namespace gdn_internal
