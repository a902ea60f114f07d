// gated_delta.cu -- the gated delta rule, forward: S = exp(g) S; u = beta (v - S k);
// S += u k^T; y = S q.
//
// Three kernels:
//  * walk: the steps as they are defined, for a few tokens (one: a decode step).  Bound by
//    reading and writing the states.
//  * records: P, H and the gates of every chunk of 64 steps (gated_delta.cuh), all chunks at
//    once: three products on the tensor cores around the inverse of a unit triangle in fp32.
//  * chain: the chunks of one head and 64 columns of headdim in order.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "gated_delta.cuh"

namespace {

using namespace gdn;

// ------------------------------------------------------------------- walk

constexpr int kWalkThreads = 128;
constexpr int kWalkRows = 8;       // rows of the state (of headdim) a warp holds
constexpr int kWalkSteps = 16;     // longest bf16 sequence that is walked

struct WalkArgs {
    const void *q, *k, *v, *g, *beta;
    long long q_step, k_step, v_step;
    const float* h0;
    float* last;
    void* y;
    int batch, seqlen, heads, groups, dk, dv, gates_bf16;
};

__device__ __forceinline__ float gate_at(const void* p, long long i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

// A warp holds kWalkRows rows of one head's state, 8 lanes to a row, 4 rows at a time:
// lane s of a row has the columns 4 (8 j + s) .. + 3, so that a load is 128 contiguous
// bytes a row and a dot product takes 3 shuffles.  NJ = ceil(dstate / 32).
template <typename T, typename TO, int NJ>
__global__ void __launch_bounds__(kWalkThreads) walk_kernel(const WalkArgs a) {
    constexpr int SETS = kWalkRows / 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7;
    const int per_head = (a.dv + kWalkRows - 1) / kWalkRows;
    const long long item = (long long)blockIdx.x * (kWalkThreads / 32) + warp;
    const long long bh = item / per_head;
    if (bh >= (long long)a.batch * a.heads) return;
    const int row0 = (int)(item % per_head) * kWalkRows + (lane >> 3);
    const int b = (int)(bh / a.heads), h = (int)(bh % a.heads);
    const int group = h / (a.heads / a.groups);

    float4 S[SETS][NJ];
#pragma unroll
    for (int s = 0; s < SETS; ++s)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = 4 * (8 * j + sub), row = row0 + 4 * s;
            S[s][j] = a.h0 && c < a.dk && row < a.dv
                          ? __ldcs(reinterpret_cast<const float4*>(a.h0 + (bh * a.dv + row) * a.dk + c))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    const T* q = static_cast<const T*>(a.q) + (long long)b * a.seqlen * a.q_step + group * a.dk;
    const T* k = static_cast<const T*>(a.k) + (long long)b * a.seqlen * a.k_step + group * a.dk;
    const T* v = static_cast<const T*>(a.v) + (long long)b * a.seqlen * a.v_step + h * a.dv;
    TO* y = static_cast<TO*>(a.y) + (long long)b * a.seqlen * a.heads * a.dv + h * a.dv;
    const long long gate0 = (long long)b * a.seqlen * a.heads + h;

    for (int t = 0; t < a.seqlen; ++t) {
        const float decay = ex2_approx(gate_at(a.g, gate0 + (long long)t * a.heads, a.gates_bf16) * kLog2e);
        const float beta = gate_at(a.beta, gate0 + (long long)t * a.heads, a.gates_bf16);
        float4 kv[NJ], qv[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = 4 * (8 * j + sub);
            qv[j] = kv[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < a.dk) {
                qv[j] = load4(q + t * a.q_step + c);
                if (beta != 0.0f) kv[j] = load4(k + t * a.k_step + c);
            }
        }
#pragma unroll
        for (int s = 0; s < SETS; ++s) {
            const int row = row0 + 4 * s;
            float sk = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float* e = reinterpret_cast<float*>(&S[s][j]);
                const float* kk = reinterpret_cast<const float*>(&kv[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a decay of 0 starts the state anew, whatever it was
                    e[i] = decay == 0.0f ? 0.0f : e[i] * decay;
                    sk = fmaf(e[i], kk[i], sk);
                }
            }
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) sk += __shfl_xor_sync(0xffffffffu, sk, o);
            // a beta of 0 is a mask: neither k nor v is looked at
            const float u = beta != 0.0f && row < a.dv
                                ? beta * (to_f32(v[t * a.v_step + row]) - sk) : 0.0f;
            float out = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float* e = reinterpret_cast<float*>(&S[s][j]);
                const float* kk = reinterpret_cast<const float*>(&kv[j]);
                const float* qq = reinterpret_cast<const float*>(&qv[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[i] = fmaf(u, kk[i], e[i]);
                    out = fmaf(e[i], qq[i], out);
                }
            }
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
            if (sub == 0 && row < a.dv) y[(long long)t * a.heads * a.dv + row] = from_f32<TO>(out);
        }
    }
    if (!a.last) return;
#pragma unroll
    for (int s = 0; s < SETS; ++s)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = 4 * (8 * j + sub), row = row0 + 4 * s;
            if (c < a.dk && row < a.dv)
                __stcs(reinterpret_cast<float4*>(a.last + (bh * a.dv + row) * a.dk + c), S[s][j]);
        }
}

// ---------------------------------------------------------------- records

constexpr int kRecThreads = 256;
constexpr int kPitch = 68;  // floats between the rows of the triangle

template <int DK> struct RecSmem {
    static constexpr uint32_t kq = 0;                    // panels of [K 64 rows | Q 64 rows]
    static constexpr uint32_t p_hi = (DK / 64) * 2 * kTile;
    static constexpr uint32_t p_lo = p_hi + kTile;
    static constexpr uint32_t t_hi = p_lo + kTile;       // T', rows i, columns j
    static constexpr uint32_t t_lo = t_hi + kTile;
    static constexpr uint32_t w_hi = t_lo + kTile;       // diag(w) T'
    static constexpr uint32_t w_lo = w_hi + kTile;
    static constexpr uint32_t tri = w_lo + kTile;        // A, then T (fp32)
    static constexpr uint32_t misc = tri + kC * kPitch * 4;
    static constexpr uint32_t bytes = misc + 1024;
};

struct RecArgs {
    const void *g, *beta;
    uint8_t* records;
    uint32_t* status;
    Dims d;
    int gates_bf16;
    int keep_t;      // T' is wanted (training)
};

// T = (1 + A)^-1 in place, A strictly lower 64 x 64 (zeros above).  The four 16 x 16
// blocks on the diagonal by substitution, a thread to a column, then blocks joined in
// pairs: the lower left of [[X, 0], [L, Z]]^-1 is -Z^-1 L X^-1.  `tmp`: 32 x 36 floats.
__device__ __forceinline__ void invert_unit_lower(float* m, float* tmp, int tid) {
    if (tid < 64) {
        const int b = (tid >> 4) * 16, c = tid & 15;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s = r == c ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < r; ++j) s = fmaf(-m[(b + r) * kPitch + b + j], x[j], s);
            x[r] = s;
        }
        __syncwarp();  // a block's columns are read and written by one half warp
#pragma unroll
        for (int r = 0; r < 16; ++r) m[(b + r) * kPitch + b + c] = x[r];
    }
    __syncthreads();
    // joins of 16: blocks (1, 0) and (3, 2); two elements to a thread
    {
        const int pair = tid >> 7, r = (tid >> 3) & 15, c = (tid & 7) * 2;
        const float* L = m + (pair * 32 + 16) * kPitch + pair * 32;
        const float* X = m + pair * 32 * kPitch + pair * 32;
        const float* Z = X + 16 * kPitch + 16;
        float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float l = L[r * kPitch + j];
            a0 = fmaf(l, X[j * kPitch + c], a0);
            a1 = fmaf(l, X[j * kPitch + c + 1], a1);
        }
        float* t = tmp + (pair * 16 + r) * 36 + c;
        t[0] = a0;
        t[1] = a1;
        __syncthreads();
        a0 = a1 = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float z = Z[r * kPitch + j];
            a0 = fmaf(-z, tmp[(pair * 16 + j) * 36 + c], a0);
            a1 = fmaf(-z, tmp[(pair * 16 + j) * 36 + c + 1], a1);
        }
        float* o = m + (pair * 32 + 16 + r) * kPitch + pair * 32 + c;
        o[0] = a0;
        o[1] = a1;
    }
    __syncthreads();
    // join of 32: four elements to a thread
    {
        const int r = tid >> 3, c = (tid & 7) * 4;
        const float* L = m + 32 * kPitch;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
            const float l = L[r * kPitch + j];
            const float4 x = *reinterpret_cast<const float4*>(m + j * kPitch + c);
            s.x = fmaf(l, x.x, s.x); s.y = fmaf(l, x.y, s.y);
            s.z = fmaf(l, x.z, s.z); s.w = fmaf(l, x.w, s.w);
        }
        *reinterpret_cast<float4*>(tmp + r * 36 + c) = s;
        __syncthreads();
        s = make_float4(0.f, 0.f, 0.f, 0.f);
        const float* Z = m + 32 * kPitch + 32;
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
            const float z = -Z[r * kPitch + j];
            const float4 x = *reinterpret_cast<const float4*>(tmp + j * 36 + c);
            s.x = fmaf(z, x.x, s.x); s.y = fmaf(z, x.y, s.y);
            s.z = fmaf(z, x.z, s.z); s.w = fmaf(z, x.w, s.w);
        }
        *reinterpret_cast<float4*>(m + (32 + r) * kPitch + c) = s;
    }
    __syncthreads();
}

template <int DK>
__global__ void __launch_bounds__(kRecThreads, 2)
    records_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const RecArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using M = RecSmem<DK>;
    constexpr int NP = DK / 64;
    constexpr uint32_t kTmX = 0, kTmH = 64, kTmP = 128, kTmCols = 256;
    const uint32_t sb = smem_u32(smem);
    float* tri = reinterpret_cast<float*>(smem + M::tri);
    float* tmp = reinterpret_cast<float*>(smem + M::t_hi);  // before T' is written there
    float* s_hi = reinterpret_cast<float*>(smem + M::misc);
    float* s_lo = s_hi + kC;
    float* s_beta = s_lo + kC;
    long long* s_sum = reinterpret_cast<long long*>(s_beta + kC);
    uint32_t* s_flags = reinterpret_cast<uint32_t*>(s_sum + 1);  // masked, NaN (two words each)
    uint64_t* bar_in = reinterpret_cast<uint64_t*>(s_flags + 4);
    uint64_t* bar_mma = bar_in + 1;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar_mma + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
    const long long ch = blockIdx.x;
    const int c = (int)(ch % a.d.chunks);
    const long long bh = ch / a.d.chunks;
    const int b = (int)(bh / a.d.heads), h = (int)(bh % a.d.heads);
    const int group = h / (a.d.heads / a.d.groups), t0 = c * kC;
    uint8_t* rec = a.records + ch * rec_bytes(DK);

    if (warp == 0) tmem_alloc(s_tmem, kTmCols);
    if (tid == 0) {
        mbar_init(bar_in, 1);
        mbar_init(bar_mma, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar_in, NP * 2 * kTile);
        for (int p = 0; p < NP; ++p) {
            tma_load_4d(smem + M::kq + p * 2 * kTile, &tm_k, bar_in, 64 * p, group, t0, b);
            tma_load_4d(smem + M::kq + p * 2 * kTile + kTile, &tm_q, bar_in, 64 * p, group, t0, b);
        }
    }
    // the gates: base-2 logarithms summed as integers of 2^-32, so that differences of far
    // sums are as exact as near ones (a decay of 2^-300 and less is 0 all the same)
    long long sum = 0;
    if (tid < kC) {
        const int t = t0 + tid;
        const long long at = ((long long)b * a.d.seqlen + t) * a.d.heads + h;
        const bool in = t < a.d.seqlen;
        const float g = in ? gate_at(a.g, at, a.gates_bf16) : 0.0f;
        const float beta = in ? gate_at(a.beta, at, a.gates_bf16) : 0.0f;
        s_beta[tid] = beta;
        const float g2 = fminf(fmaxf(g * kLog2e, -300.0f), 300.0f);
        sum = __float2ll_rn(g2 * 4294967296.0f);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        const uint32_t off = __ballot_sync(0xffffffffu, beta == 0.0f);
        const uint32_t bad = __ballot_sync(0xffffffffu, isnan(g));
        if (lane == 0) {
            s_flags[warp] = off;
            s_flags[2 + warp] = bad;
        }
        if (tid == 31) *s_sum = sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    const unsigned long long masked = (unsigned long long)s_flags[1] << 32 | s_flags[0];
    if (tid < kC) {
        if (warp == 1) sum += *s_sum;
        const unsigned long long bad = (unsigned long long)s_flags[3] << 32 | s_flags[2];
        float hi = (float)sum;
        const float lo = (float)(sum - (long long)hi) * 2.3283064365386963e-10f;  // 2^-32
        hi *= 2.3283064365386963e-10f;
        if (bad & (~0ull >> (63 - tid))) hi = __int_as_float(0x7fc00000);
        s_hi[tid] = hi;
        s_lo[tid] = lo;
        Gates* gates = reinterpret_cast<Gates*>(rec + hp_bytes(DK) + kTile);
        gates->hi[tid] = hi;
        gates->lo[tid] = lo;
        if (tid == 0) gates->masked = masked;
    }
    bool ok = warp_wait(bar_in, 0, a.status);
    if (masked) {  // steps that learn nothing: their keys are not looked at
        if (ok)
            for (int e = tid; e < NP * kC * 8; e += kRecThreads) {
                const int r = (e >> 3) & 63;
                if (masked >> r & 1)
                    *reinterpret_cast<uint4*>(smem + M::kq + (e >> 9) * 2 * kTile + r * 128 +
                                              (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
        fence_proxy_async_smem();
    }
    ok = __syncthreads_and(ok);

    // ---- [K; Q] K^T
    if (tid == 0 && ok) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
            mma_bf16(tmem + kTmX, kdesc<128>(sb + M::kq, kk), kdesc<128>(sb + M::kq, kk),
                     idesc_bf16_f32(128, 64), kk > 0);
        mma_commit(bar_mma);
    }
    ok = __syncthreads_and(ok && warp_wait(bar_mma, 0, a.status));
    tc_fence_after();
    {
        float x[32];
        tmem_ld32(t_lane + kTmX + 32 * part, x);
        tmem_wait_ld();
        const int i = row & 63;
        const bool is_q = row >= kC;
        const float hi = s_hi[i], lo = s_lo[i], beta = is_q ? 1.0f : s_beta[i];
        const int last = is_q ? i : i - 1;  // of the columns that count
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int j = 32 * part + e;
            x[e] = j <= last ? beta * x[e] * decay(hi, lo, s_hi[j], s_lo[j]) : 0.0f;
        }
        if (is_q) {
            put32_split(smem + M::p_hi, smem + M::p_lo, i, 4 * part, x);
        } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(tri + i * kPitch + 32 * part + e) =
                    make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
    }
    __syncthreads();
    invert_unit_lower(tri, tmp, tid);

    // ---- T' and diag(w) T' as operands: row i = tid / 4, 16 columns
    {
        const int i = tid >> 2, j0 = (tid & 3) * 16;
        const float w = decay(s_hi[kC - 1], s_lo[kC - 1], s_hi[i], s_lo[i]);
        uint32_t th[8], tl[8], wh[8], wl[8];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const int j = j0 + e;
            const float x = tri[i * kPitch + j] * s_beta[j];
            const float y = tri[i * kPitch + j + 1] * s_beta[j + 1];
            split2(x, y, th[e >> 1], tl[e >> 1]);
            split2(w * x, w * y, wh[e >> 1], wl[e >> 1]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t off = piece(i, (j0 >> 3) + s);
            const uint4 hi4 = make_uint4(th[4 * s], th[4 * s + 1], th[4 * s + 2], th[4 * s + 3]);
            *reinterpret_cast<uint4*>(smem + M::t_hi + off) = hi4;
            *reinterpret_cast<uint4*>(smem + M::t_lo + off) =
                make_uint4(tl[4 * s], tl[4 * s + 1], tl[4 * s + 2], tl[4 * s + 3]);
            *reinterpret_cast<uint4*>(smem + M::w_hi + off) =
                make_uint4(wh[4 * s], wh[4 * s + 1], wh[4 * s + 2], wh[4 * s + 3]);
            *reinterpret_cast<uint4*>(smem + M::w_lo + off) =
                make_uint4(wl[4 * s], wl[4 * s + 1], wl[4 * s + 2], wl[4 * s + 3]);
            if (a.keep_t) *reinterpret_cast<uint4*>(rec + hp_bytes(DK) + off) = hi4;
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();

    // ---- H = K^T diag(w) T' (rows of dstate) and P T' (rows 64 to 127: the tile of 128
    // rows starts one tile early, its first half is not read)
    if (tid == 0 && ok) {
        tc_fence_after();
        constexpr uint32_t idH = idesc_bf16_f32(128, 64) | kIdescAMN | kIdescBMN;
        constexpr uint32_t idP = idesc_bf16_f32(128, 64) | kIdescBMN;
        // of 64 columns of dstate the second block of rows is not read either
        constexpr uint32_t lbo = NP > 1 ? 2 * kTile : kTile;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            mma_bf16(tmem + kTmH, mdesc(sb + M::kq, kk, lbo), mdesc(sb + M::w_hi, kk, kTile), idH, kk > 0);
            mma_bf16(tmem + kTmH, mdesc(sb + M::kq, kk, lbo), mdesc(sb + M::w_lo, kk, kTile), idH, 1);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ph = kdesc<128>(sb + M::p_hi - kTile, kk);
            const uint64_t pl = kdesc<128>(sb + M::p_lo - kTile, kk);
            mma_bf16(tmem + kTmP, ph, mdesc(sb + M::t_hi, kk, kTile), idP, kk > 0);
            mma_bf16(tmem + kTmP, ph, mdesc(sb + M::t_lo, kk, kTile), idP, 1);
            mma_bf16(tmem + kTmP, pl, mdesc(sb + M::t_hi, kk, kTile), idP, 1);
        }
        mma_commit(bar_mma);
    }
    ok = ok && warp_wait(bar_mma, 1, a.status);
    tc_fence_after();
    if (ok) {
        float x[32];
        if (row < DK) {
            tmem_ld32(t_lane + kTmH + 32 * part, x);
            tmem_wait_ld();
            put32_split(rec, rec + h_bytes(DK), row, 4 * part, x);
        }
        if (row >= kC) {
            tmem_ld32(t_lane + kTmP + 32 * part, x);
            tmem_wait_ld();
            put32_split(rec + 2 * h_bytes(DK), rec + 2 * h_bytes(DK) + kTile, row - kC, 4 * part, x);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kTmCols);
}

// ------------------------------------------------------------------ chain

constexpr int kChainThreads = 288;  // 8 warps on rows, one that loads and multiplies

template <int DK> struct ChainSmem {
    static constexpr uint32_t kq = 0;                              // of a stage
    static constexpr uint32_t hp = (DK / 64) * 2 * kTile;
    static constexpr uint32_t stage = hp + hp_bytes(DK);
    static constexpr uint32_t s_hi = 2 * stage;                    // S0, rows of dstate
    static constexpr uint32_t s_lo = s_hi + h_bytes(DK);
    static constexpr uint32_t r_hi = s_lo + h_bytes(DK);           // R, rows of steps
    static constexpr uint32_t r_lo = r_hi + kTile;
    static constexpr uint32_t misc = r_lo + kTile;
    static constexpr uint32_t bytes = misc + 128;
};

struct ChainArgs {
    const __nv_bfloat16* v;
    const uint8_t* records;
    uint8_t* kept;
    const float* h0;
    float* last;
    void* y;
    uint32_t* status;
    Dims d;
    long long v_step;
};

// One head and 64 columns of headdim, chunk after chunk.  Rows of products are lanes of
// tensor memory: of K S0 and Q S0 the steps (0 to 63 and 64 to 127), of H R the state's
// rows, of P R the steps (64 to 127).  Two warpgroups take 32 columns each.  The state stays
// in registers (a row of dstate to a lane) and goes through shared memory as the sum of
// two bf16 each chunk, as R does.
template <int DK, typename TO>
__global__ void __launch_bounds__(kChainThreads, 1)
    chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const ChainArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using M = ChainSmem<DK>;
    constexpr int NP = DK / 64;
    constexpr uint32_t kTmX = 0, kTmH = 64, kTmY = 128, kTmCols = 256;
    const uint32_t sb = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + M::misc);  // a stage has come in
    uint64_t* bar_x = full + 2;   // [K; Q] S0 done
    uint64_t* bar_h = full + 3;   // H R done
    uint64_t* bar_y = full + 4;   // P R done: the stage and R are free
    uint64_t* bar_s = full + 5;   // S0 is in shared memory
    uint64_t* bar_r = full + 6;   // R is
    uint64_t* bar_o = full + 7;   // P R has been read
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + 8);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pan = blockIdx.x % a.d.pans;
    const long long bh = blockIdx.x / a.d.pans;
    const int b = (int)(bh / a.d.heads), h = (int)(bh % a.d.heads);
    const int nc = a.d.chunks;
    const uint8_t* rec0 = a.records + bh * nc * rec_bytes(DK);

    if (warp == 8) tmem_alloc(s_tmem, kTmCols);
    if (tid == 0) {
        mbar_init(full, 1);
        mbar_init(full + 1, 1);
        mbar_init(bar_x, 1);
        mbar_init(bar_h, 1);
        mbar_init(bar_y, 1);
        mbar_init(bar_s, 8);
        mbar_init(bar_r, 4);
        mbar_init(bar_o, 4);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 8) {
        if (lane == 0) {
            const int group = h / (a.d.heads / a.d.groups);
            int loads = 0;
            auto load = [&](int c) {
                uint8_t* st = smem + (c & 1) * M::stage;
                uint64_t* bar = full + (c & 1);
                mbar_arrive_expect_tx(bar, M::stage);
                for (int p = 0; p < NP; ++p) {
                    tma_load_4d(st + M::kq + p * 2 * kTile, &tm_k, bar, 64 * p, group, c * kC, b);
                    tma_load_4d(st + M::kq + p * 2 * kTile + kTile, &tm_q, bar, 64 * p, group, c * kC, b);
                }
                bulk_load(st + M::hp, rec0 + (long long)c * rec_bytes(DK), hp_bytes(DK), bar);
                ++loads;
            };
            load(0);
            if (nc > 1) load(1);
            constexpr uint32_t id = idesc_bf16_f32(128, 64) | kIdescBMN;
            int waited = 0;
            for (int c = 0; c < nc; ++c) {
                const uint32_t ph = c & 1, st = sb + (c & 1) * M::stage;
                if (!mbar_wait(full + (c & 1), (c >> 1) & 1, a.status)) break;
                ++waited;
                if (!mbar_wait(bar_s, ph, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk) {
                    mma_bf16(tmem + kTmX, kdesc<128>(st + M::kq, kk), mdesc(sb + M::s_hi, kk, kTile), id, kk > 0);
                    mma_bf16(tmem + kTmX, kdesc<128>(st + M::kq, kk), mdesc(sb + M::s_lo, kk, kTile), id, 1);
                }
                mma_commit(bar_x);
                if (!mbar_wait(bar_r, ph, a.status)) break;
                tc_fence_after();
                const uint32_t hh = st + M::hp, hl = hh + h_bytes(DK), pp = hl + h_bytes(DK);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16(tmem + kTmH, kdesc<DK>(hh, kk), mdesc(sb + M::r_hi, kk, kTile), id, kk > 0);
                    mma_bf16(tmem + kTmH, kdesc<DK>(hh, kk), mdesc(sb + M::r_lo, kk, kTile), id, 1);
                    mma_bf16(tmem + kTmH, kdesc<DK>(hl, kk), mdesc(sb + M::r_hi, kk, kTile), id, 1);
                }
                mma_commit(bar_h);
                if (c > 0 && !mbar_wait(bar_o, ph ^ 1, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16(tmem + kTmY, kdesc<128>(pp - kTile, kk), mdesc(sb + M::r_hi, kk, kTile), id, kk > 0);
                    mma_bf16(tmem + kTmY, kdesc<128>(pp - kTile, kk), mdesc(sb + M::r_lo, kk, kTile), id, 1);
                    mma_bf16(tmem + kTmY, kdesc<128>(pp, kk), mdesc(sb + M::r_hi, kk, kTile), id, 1);
                }
                mma_commit(bar_y);
                if (c + 2 < nc) {
                    if (!mbar_wait(bar_y, ph, a.status)) break;
                    load(c + 2);
                }
            }
            // never leave with a load still landing
            for (; waited < loads; ++waited)
                (void)mbar_wait(full + (waited & 1), (waited >> 1) & 1, a.status);
        }
    } else {
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + 32 * part;
        const int col0 = pan * kPan + 32 * part;      // first column of headdim
        const bool on_k = row < kC;                   // of [K; Q] S0
        const int i = row & 63;
        float S[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
            S[e] = a.h0 && row < a.d.dk && col0 + e < a.d.dv
                       ? a.h0[(bh * a.d.dv + col0 + e) * a.d.dk + row] : 0.0f;
        // S0 of chunk c as an operand, and kept
        auto put_state = [&](int c) {
            if (row < DK) {
                put32_split(smem + M::s_hi, smem + M::s_lo, row, 4 * part, S);
                if (a.kept)
                    put32(a.kept + ((bh * nc + c) * a.d.pans + pan) * kept_bytes(DK) + kTile, row,
                          4 * part, S);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(bar_s);
        };
        put_state(0);
        // what a chunk's rows take from global memory, read one chunk ahead
        uint4 v[4];
        float e_row = 0.0f, e_end = 0.0f;
        bool off = true;
        auto fetch = [&](int c) {
            const Gates* g = reinterpret_cast<const Gates*>(rec0 + (long long)c * rec_bytes(DK) +
                                                            hp_bytes(DK) + kTile);
            e_row = ex2_approx(g->hi[i] + g->lo[i]);
            e_end = ex2_approx(g->hi[kC - 1] + g->lo[kC - 1]);
            off = g->masked >> i & 1;
            const long long t = (long long)b * a.d.seqlen + c * kC + i;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                v[p] = on_k && !off && col0 + 8 * p < a.d.dv
                           ? *reinterpret_cast<const uint4*>(a.v + t * a.v_step + (long long)h * a.d.dv +
                                                             col0 + 8 * p)
                           : make_uint4(0, 0, 0, 0);
        };
        fetch(0);
        for (int c = 0; c < nc; ++c) {
            const uint32_t ph = c & 1;
            const float er = e_row, ee = e_end;
            float x[32];
            if (!warp_wait(bar_x, ph, a.status)) break;
            tc_fence_after();
            tmem_ld32(t_lane + kTmX, x);
            tmem_wait_ld();
            if (on_k) {
                // (the products that read R before are done: bar_x follows them)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    float vv[8];
                    unpack8(v[p], vv);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float carried = er == 0.0f ? 0.0f : er * x[8 * p + e];
                        x[8 * p + e] = off ? 0.0f : vv[e] - carried;
                    }
                }
                put32_split(smem + M::r_hi, smem + M::r_lo, i, 4 * part, x);
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(bar_r);
                if (a.kept)
                    put32(a.kept + ((bh * nc + c) * a.d.pans + pan) * kept_bytes(DK), i, 4 * part, x);
            }
            if (c + 1 < nc) fetch(c + 1);
            float z[32];
            if (!warp_wait(bar_h, ph, a.status)) break;
            tc_fence_after();
            tmem_ld32(t_lane + kTmH, z);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) S[e] = ee == 0.0f ? z[e] : fmaf(ee, S[e], z[e]);
            if (c + 1 < nc) put_state(c + 1);
            if (!on_k) {
                if (!warp_wait(bar_y, ph, a.status)) break;
                tc_fence_after();
                tmem_ld32(t_lane + kTmY, z);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(bar_o);
                const int t = c * kC + i;
                if (a.y && t < a.d.seqlen) {
                    TO* y = static_cast<TO*>(a.y) +
                            (((long long)b * a.d.seqlen + t) * a.d.heads + h) * a.d.dv + col0;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        if (col0 + 8 * p >= a.d.dv) break;
                        float o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = er == 0.0f ? z[8 * p + e] : fmaf(er, x[8 * p + e], z[8 * p + e]);
                        if constexpr (sizeof(TO) == 4) {
                            *reinterpret_cast<float4*>(y + 8 * p) = make_float4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<float4*>(y + 8 * p + 4) = make_float4(o[4], o[5], o[6], o[7]);
                        } else {
                            *reinterpret_cast<uint4*>(y + 8 * p) =
                                make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                           pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                        }
                    }
                }
            }
        }
        if (a.last && row < a.d.dk)
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (col0 + e < a.d.dv) a.last[(bh * a.d.dv + col0 + e) * a.d.dk + row] = S[e];
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, kTmCols);
}

// ------------------------------------------------------------------- host

template <typename K>
bool allow_smem(K kernel, uint32_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
           cudaSuccess;
}

template <int DK>
ssm_status_t run_chunked(const gdn_internal::Forward& f, cudaStream_t s) {
    CUtensorMap mq, mk;
    if (!gdn_host::make_map(&mq, f.q, f.batch, f.seqlen, f.groups, f.dk, f.q_step) ||
        !gdn_host::make_map(&mk, f.k, f.batch, f.seqlen, f.groups, f.dk, f.k_step))
        return SSM_ERR_CUDA;
    Dims d{f.batch, f.seqlen, f.heads, f.groups, f.dk, f.dv, (f.seqlen + kC - 1) / kC,
           (f.dv + kPan - 1) / kPan};
    RecArgs r{};
    r.g = f.g; r.beta = f.beta; r.records = f.records; r.status = f.status; r.d = d;
    r.gates_bf16 = f.gate_dtype == SSM_BF16;
    r.keep_t = f.kept != nullptr;
    const unsigned chs = (unsigned)((long long)f.batch * f.heads * d.chunks);
    if (!allow_smem(records_kernel<DK>, RecSmem<DK>::bytes)) return SSM_ERR_CUDA;
    records_kernel<DK><<<chs, kRecThreads, RecSmem<DK>::bytes, s>>>(mq, mk, r);
    ChainArgs a{};
    a.v = static_cast<const __nv_bfloat16*>(f.v); a.records = f.records; a.kept = f.kept;
    a.h0 = f.initial_state; a.last = f.final_state; a.y = f.y; a.status = f.status; a.d = d;
    a.v_step = f.v_step;
    const unsigned grid = (unsigned)((long long)f.batch * f.heads * d.pans);
    auto go = [&](auto kernel) {
        if (!allow_smem(kernel, ChainSmem<DK>::bytes)) return false;
        kernel<<<grid, kChainThreads, ChainSmem<DK>::bytes, s>>>(mq, mk, a);
        return true;
    };
    if (!(f.out_dtype == SSM_F32 ? go(chain_kernel<DK, float>) : go(chain_kernel<DK, __nv_bfloat16>)))
        return SSM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

ssm_status_t run_walk(const WalkArgs& a, ssm_dtype_t in, ssm_dtype_t out, cudaStream_t s) {
    const long long items = (long long)a.batch * a.heads * ((a.dv + kWalkRows - 1) / kWalkRows);
    const unsigned grid = (unsigned)((items + kWalkThreads / 32 - 1) / (kWalkThreads / 32));
    auto go = [&](auto ti, auto to) {
        using T = decltype(ti);
        using TO = decltype(to);
        if (a.dk <= 32) walk_kernel<T, TO, 1><<<grid, kWalkThreads, 0, s>>>(a);
        else if (a.dk <= 64) walk_kernel<T, TO, 2><<<grid, kWalkThreads, 0, s>>>(a);
        else walk_kernel<T, TO, 4><<<grid, kWalkThreads, 0, s>>>(a);
    };
    using B = __nv_bfloat16;
    if (in == SSM_F32) out == SSM_F32 ? go(float{}, float{}) : go(float{}, B{});
    else out == SSM_F32 ? go(B{}, float{}) : go(B{}, B{});
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

// fp32 sequences, and bf16 ones of a few tokens from which nothing is kept
bool walks(int seqlen, ssm_dtype_t in, bool keep) {
    return in == SSM_F32 || (seqlen <= kWalkSteps && !keep);
}

}  // namespace

namespace gdn_internal {

ssm_status_t chunked_forward(const Forward& f, cudaStream_t s) {
    return gdn_host::dk_tile(f.dk) == 64 ? run_chunked<64>(f, s) : run_chunked<128>(f, s);
}

}  // namespace gdn_internal

extern "C" size_t ssm_gated_delta_checkpoint_bytes(int batch, int seqlen, int nheads, int dstate,
                                                   int headdim) {
    using namespace gdn_host;
    if (!sizes_ok(batch, seqlen, nheads, nheads, dstate, headdim) ||
        !sizes_fit(batch, seqlen, nheads, dstate, headdim))
        return 0;
    return records_bytes(batch, seqlen, nheads, dstate) +
           keep_bytes(batch, seqlen, nheads, dstate, headdim);
}

extern "C" size_t ssm_gated_delta_workspace_bytes(int batch, int seqlen, int nheads, int dstate,
                                                  int headdim) {
    using namespace gdn_host;
    if (!sizes_ok(batch, seqlen, nheads, nheads, dstate, headdim) ||
        !sizes_fit(batch, seqlen, nheads, dstate, headdim))
        return 0;
    return 1024 + records_bytes(batch, seqlen, nheads, dstate);
}

extern "C" ssm_status_t ssm_gated_delta_fwd(
    const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
    long long v_stride, const void* g, const void* beta, const float* initial_state, void* y,
    float* final_state, void* checkpoints, int batch, int seqlen, int nheads, int ngroups,
    int dstate, int headdim, ssm_dtype_t in_dtype, ssm_dtype_t gate_dtype, ssm_dtype_t out_dtype,
    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ssm_host;
    using gdn_host::Span;
    using gdn_host::strided_bytes;
    if (!gdn_host::sizes_ok(batch, seqlen, nheads, ngroups, dstate, headdim)) return SSM_ERR_SHAPE;
    const long long qw = (long long)ngroups * dstate, vw = (long long)nheads * headdim;
    if (q_stride < qw || k_stride < qw || v_stride < vw) return SSM_ERR_SHAPE;
    if (!dtype_ok(in_dtype) || !dtype_ok(gate_dtype) || !dtype_ok(out_dtype)) return SSM_ERR_DTYPE;
    if (!gdn_host::sizes_fit(batch, seqlen, nheads, dstate, headdim) ||
        (checkpoints && in_dtype != SSM_BF16))
        return SSM_ERR_UNSUPPORTED;
    if (batch == 0 || nheads == 0) return SSM_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t sb = (size_t)batch * nheads * headdim * dstate * 4, es = dtype_size(in_dtype);
    const long long steps = (long long)batch * seqlen;
    const bool walk = walks(seqlen, in_dtype, checkpoints != nullptr);
    const size_t cb = checkpoints ? ssm_gated_delta_checkpoint_bytes(batch, seqlen, nheads, dstate, headdim) : 0;
    const size_t wb = walk || seqlen == 0 ? 0
                      : checkpoints ? 1024
                                    : ssm_gated_delta_workspace_bytes(batch, seqlen, nheads, dstate, headdim);
    if (seqlen > 0 && (!q || !k || !v || !g || !beta || !y)) return SSM_ERR_NULL;
    if (wb && (!workspace || workspace_bytes < wb)) return SSM_ERR_WORKSPACE;
    for (const void* p : {q, k, v, (const void*)initial_state, (const void*)y,
                          (const void*)final_state, (const void*)checkpoints, (const void*)workspace})
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    for (long long st : {q_stride, k_stride, v_stride})
        if (seqlen > 0 && st * es % 16) return SSM_ERR_ALIGN;
    const size_t gs = dtype_size(gate_dtype);
    for (const void* p : {g, beta})
        if (reinterpret_cast<uintptr_t>(p) % gs) return SSM_ERR_ALIGN;
    const size_t gb = (size_t)steps * nheads * gs;
    const Span ins[] = {{q, strided_bytes(steps, qw, q_stride, es)},
                        {k, strided_bytes(steps, qw, k_stride, es)},
                        {v, strided_bytes(steps, vw, v_stride, es)},
                        {g, gb}, {beta, gb}, {initial_state, sb}};
    const Span outs[] = {{y, (size_t)steps * vw * dtype_size(out_dtype)},
                         {final_state, sb}, {checkpoints, cb}, {workspace, wb}};
    for (const Span& o : outs)
        for (const Span& i : ins) {
            // the state may be updated in place: each is read before it is written
            if (o.p == final_state && i.p == initial_state && final_state == initial_state) continue;
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
        }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;
    if (seqlen == 0) {
        if (!final_state || final_state == initial_state) return SSM_OK;
        const cudaError_t e = initial_state ? cudaMemcpyAsync(final_state, initial_state, sb,
                                                              cudaMemcpyDeviceToDevice, s)
                                            : cudaMemsetAsync(final_state, 0, sb, s);
        return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
    }
    if (walk) {
        WalkArgs a{q, k, v, g, beta, q_stride, k_stride, v_stride, initial_state, final_state, y,
                   batch, seqlen, nheads, ngroups, dstate, headdim, gate_dtype == SSM_BF16};
        return run_walk(a, in_dtype, out_dtype, s);
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (cudaMemsetAsync(ws, 0, 8, s) != cudaSuccess) return SSM_ERR_CUDA;
    gdn_internal::Forward f{};
    f.q = q; f.k = k; f.v = v; f.q_step = q_stride; f.k_step = k_stride; f.v_step = v_stride;
    f.g = g; f.beta = beta; f.gate_dtype = gate_dtype; f.initial_state = initial_state;
    f.y = y; f.out_dtype = out_dtype; f.final_state = final_state;
    f.status = reinterpret_cast<uint32_t*>(ws) + 1;
    f.batch = batch; f.seqlen = seqlen; f.heads = nheads; f.groups = ngroups; f.dk = dstate; f.dv = headdim;
    f.records = checkpoints ? static_cast<uint8_t*>(checkpoints) : ws + 1024;
    f.kept = checkpoints ? f.records + gdn_host::records_bytes(batch, seqlen, nheads, dstate) : nullptr;
    return gdn_internal::chunked_forward(f, s);
}
