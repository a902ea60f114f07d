// gated_delta.cu -- the gated delta rule, forward: S = exp(g) S; u = beta (v - S k);
// S += u k^T; y = S q.
//
// Four kernels:
//  * walk: the steps as they are defined, for a few tokens (one: a decode step).  Bound by
//    reading and writing the states.
//  * records: P, H and the gates of every chunk of 64 steps (gated_delta.cuh), all chunks at
//    once: three products on the tensor cores around the inverse of a unit triangle in fp32.
//  * chain: the chunks of one head and 64 (or 32) columns of headdim in order.
//  * both: records and chains at once, where chains are few.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "gated_delta.cuh"
#include "scan_internal.h"

namespace {

using namespace gdn;

// ------------------------------------------------------------------- walk

constexpr int kWalkThreads = 128;
constexpr int kWalkRows = 8;       // rows of the state (of headdim) a warp holds
// The longest bf16 sequence that is walked.  A step costs the same again, a chunk costs what it
// costs however few of its steps there are; inputs not in the caches, at headdim = dstate = 128,
// 8, 10 and 12 steps walked, and in chunks: 128 x 32 heads 467, 569, 653 and 533 us; 32 x 32 heads
// 137, 160, 186 and 155 us; 8 x 16 heads 29, 35, 39 and 39 us.  Smaller states could be walked
// for longer (32 x 32 heads of 64 x 64, 16 steps: 68 and 87 us).
constexpr int kWalkSteps = 10;

struct WalkArgs {
    const void *q, *k, *v, *g, *beta;
    long long q_step, k_step, v_step;
    const float* h0;
    float* last;
    void* y;
    int batch, seqlen, heads, groups, dk, dv, gates_bf16;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

// A warp holds kWalkRows rows of one head's state, 8 lanes to a row, 4 rows at a time:
// lane s of a row has the columns 4 (8 j + s) .. + 3, so that a load is 128 contiguous
// bytes a row and a dot product takes 3 shuffles.  NJ = ceil(dstate / 32).  Bound by reading
// and writing the state: one token of 256 x 32 heads of 128 x 64 92 us, 5.8 TB/s (with 4 rows
// to a warp 104 us).
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
    static constexpr uint32_t t_hi = kq_bytes(DK);       // T, rows i, columns j
    static constexpr uint32_t t_lo = t_hi + kTile;
    static constexpr uint32_t w_hi = t_lo + kTile;       // diag(w) T
    static constexpr uint32_t w_lo = w_hi + kTile;
    static constexpr uint32_t p_hi = w_lo + kTile;       // (Q K^T) D
    static constexpr uint32_t p_lo = p_hi + kTile;
    static constexpr uint32_t n = p_lo + kTile;          // b^-1 T b
    static constexpr uint32_t gates = n + kTile;         // as the record has them
    static constexpr uint32_t misc = gates + kGateBytes;
    static constexpr uint32_t bytes = misc + 1536;
    // A, then T (fp32), in the place of T's and its w's first tile; H and P leave from there too
    static constexpr uint32_t tri = t_hi;
    static constexpr uint32_t tmp = w_lo;
};

struct RecArgs {
    const void *g, *beta;
    uint8_t* records;
    uint32_t* status;
    uint32_t* flags;  // of chunks and heads whose records are in memory, or NULL
    Dims d;
    unsigned count;   // of chunks and heads
    int gates_bf16;
    int keep_n;       // N is wanted (training)
    int drop_first;   // (a test's) the first record is not told
};

template <int V> struct Vec;
template <> struct Vec<1> { using T = float; };
template <> struct Vec<2> { using T = float2; };
template <> struct Vec<4> { using T = float4; };

// Joins pairs of inverted blocks of N rows: the lower left of [[X, 0], [L, Z]]^-1 is
// -Z^-1 L X^-1.  In two steps, the first product through `tmp` (rows of 36 floats).  Warps
// take four columns of the first, then four rows of the second, so that what is zero in
// the triangles is left out by whole warps.
template <int N>
__device__ __forceinline__ void join_blocks(float* m, float* tmp, int warp, int lane) {
    constexpr int V = N / 8, W = N / 4;  // columns to a lane, warps to a pair
    using T = typename Vec<V>::T;
    const int w = warp % W, at = (warp / W) * 2 * N;
    const float* X = m + at * kPitch + at;
    const float* L = X + N * kPitch;
    float* t = tmp + (warp / W) * N * 36;
    auto add = [](float* s, const float* left, const float* right, int pitch) {
        const float4 l = *reinterpret_cast<const float4*>(left);
        const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const T x = *reinterpret_cast<const T*>(right + e * pitch);
            const float* xv = reinterpret_cast<const float*>(&x);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = fmaf(lv[e], xv[v], s[v]);
        }
    };
    {
        float s[V] = {};
        const int r = lane % N, c = 4 * w + (lane / N) * V;
#pragma unroll 2
        for (int j = 4 * w; j < N; j += 4) add(s, L + r * kPitch + j, X + j * kPitch + c, kPitch);
        *reinterpret_cast<T*>(t + r * 36 + c) = *reinterpret_cast<const T*>(s);
    }
    named_bar_sync(1, kRecThreads);
    {
        float s[V] = {};
        const int r = 4 * w + lane / 8, c = (lane % 8) * V;
#pragma unroll 2
        for (int j = 0; j <= 4 * w; j += 4) add(s, L + N + r * kPitch + j, t + j * 36 + c, 36);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = -s[v];
        *reinterpret_cast<T*>(m + (at + N + r) * kPitch + at + c) = *reinterpret_cast<const T*>(s);
    }
    named_bar_sync(1, kRecThreads);
}

// T = (1 + A)^-1 in place, A strictly lower 64 x 64 (zeros above).  The eight 8 x 8
// blocks on the diagonal by substitution, a thread to a column, then blocks joined in
// pairs three times.  `tmp`: 32 x 36 floats.  In fp32: what is lost here no later product
// gives back.
__device__ __forceinline__ void invert_unit_lower(float* m, float* tmp, int tid) {
    if (tid < 64) {
        const int b = (tid >> 3) * 8, c = tid & 7;
        const float* base = m + b * kPitch + b;
        float x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float s = r == c ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < r; j += 4) {
                const float4 l = *reinterpret_cast<const float4*>(base + r * kPitch + j);
                s = fmaf(-l.x, x[j], s);
                if (j + 1 < r) s = fmaf(-l.y, x[j + 1], s);
                if (j + 2 < r) s = fmaf(-l.z, x[j + 2], s);
                if (j + 3 < r) s = fmaf(-l.w, x[j + 3], s);
            }
            x[r] = s;
        }
        __syncwarp();  // a block's columns are read and written by one quarter of a warp
#pragma unroll
        for (int r = 0; r < 8; ++r) m[(b + r) * kPitch + b + c] = x[r];
    }
    named_bar_sync(1, kRecThreads);
    join_blocks<8>(m, tmp, tid >> 5, tid & 31);
    join_blocks<16>(m, tmp, tid >> 5, tid & 31);
    join_blocks<32>(m, tmp, tid >> 5, tid & 31);
}

// The beta of a row of the triangle: N divides the row by it, so that it must not be too small for
// the row to be held.  A smaller one is taken for this, which changes T by as much and N not at
// all (masked rows are 0 in either).
__device__ __forceinline__ float row_beta(float b) {
    constexpr float least = 8.673617379884035e-19f;  // 2^-60
    return fabsf(b) < least ? copysignf(least, b) : b;
}

// Bound by the issue of some 15400 warp instructions a chunk and head (16700 with N): 4096 of them at
// dstate 128 take 125 us (137 us), two CTAs' phases filling each other's waits.
//
// CTAs walk the chunks and heads, two CTAs to an SM; the next chunk's K and Q come in while
// this one's H and P leave.
//
// The work of eight warps: the items `first`, first + step, ...  With flags they are told one
// by one, and go through the chunks of all heads side by side.
template <int DK, bool FLAGS>
__device__ __forceinline__ void make_records(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                             const RecArgs& a, uint8_t* smem, uint32_t tmem,
                                             unsigned first, unsigned step) {
    using M = RecSmem<DK>;
    constexpr int NP = DK / 64;
    // tensor memory: [K; Q] K^T, then H (hi and lo columns); P (hi and lo columns)
    constexpr uint32_t kTmX = 0, kTmH = 0, kTmP = 128;
    const uint32_t sb = smem_u32(smem);
    float* tri = reinterpret_cast<float*>(smem + M::tri);
    float* tmp = reinterpret_cast<float*>(smem + M::tmp);
    Gates* gates = reinterpret_cast<Gates*>(smem + M::gates);
    float* s_beta = reinterpret_cast<float*>(smem + M::misc);
    float* s_dec = s_beta + kC;                                   // [32]: decays to step 31
    float* s_inv = s_dec + 32;                                    // [64]: inverse ones from 0 or 32
    float* s_span = s_inv + kC;                                   // [2]: their largest logarithm
    float* s_most = s_span + 4;                                   // [4][8]
    long long* s_sum = reinterpret_cast<long long*>(s_most + 32);
    uint32_t* s_flags = reinterpret_cast<uint32_t*>(s_sum + 1);   // masked, NaN, growing: two words each
    uint64_t* bar_in = reinterpret_cast<uint64_t*>(s_flags + 6);
    uint64_t* bar_mma = bar_in + 1;
    float* s_e = reinterpret_cast<float*>(smem + M::misc + 1024);  // [64]: decays from the chunk's start; [3][8]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane, i = row & 63;
    const bool is_q = row >= kC;

    const unsigned chunks = a.d.chunks, heads = a.d.heads, ratio = heads / a.d.groups;
    const unsigned all_heads = heads * a.d.batch;
    auto chunk_of = [&](unsigned item) {
        return FLAGS ? (item % all_heads) * chunks + item / all_heads : item;
    };
    auto load = [&](unsigned ch) {  // K and Q of a chunk (one thread)
        const unsigned bh = ch / chunks, b = bh / heads;
        const int t0 = (int)(ch - bh * chunks) * kC, group = (int)((bh - b * heads) / ratio);
        mbar_arrive_expect_tx(bar_in, kq_bytes(DK));
        for (int p = 0; p < NP; ++p) {
            tma_load_4d(smem + M::kq + p * 2 * kTile, &tm_k, bar_in, 64 * p, group, t0, b);
            tma_load_4d(smem + M::kq + p * 2 * kTile + kTile, &tm_q, bar_in, 64 * p, group, t0, b);
        }
    };
    float g = 0.0f, beta = 0.0f;  // of step tid, one chunk ahead
    auto fetch = [&](unsigned ch) {
        if (tid >= kC) return;
        const unsigned bh = ch / chunks, b = bh / heads;
        const int t = (int)(ch - bh * chunks) * kC + tid;
        const long long at = ((long long)b * a.d.seqlen + t) * heads + (bh - b * heads);
        const bool in = t < a.d.seqlen;
        g = in ? gate_at(a.g, at, a.gates_bf16) : 0.0f;
        beta = in ? gate_at(a.beta, at, a.gates_bf16) : 0.0f;
    };
    if (first < a.count) fetch(chunk_of(first));
    if (tid == 0) {
        mbar_init(bar_in, 1);
        mbar_init(bar_mma, 1);
        fence_mbar_init();
        if (first < a.count) load(chunk_of(first));
    }
    named_bar_sync(1, kRecThreads);
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    bool ok = true;
    bool landing = false;  // (thread 0) a load is on its way
    uint32_t mma_phase = 0, in_phase = 0;

    // (thread 0) what went out before is in memory: told to the chains
    auto tell = [&](unsigned ch) {
        bulk_wait_all();
        asm volatile("fence.proxy.async;" ::: "memory");
        if (!(a.drop_first && ch == 0)) st_release_gpu(a.flags + ch, 1u);
    };
    unsigned before = 0;
    for (unsigned item = first; item < a.count && ok; item += step) {
        const unsigned ch = chunk_of(item);
        uint8_t* rec = a.records + (size_t)ch * rec_bytes(DK);
        const bool more = step < a.count - item;
        // ---- the gates: base-2 logarithms summed as integers of 2^-32, so that differences
        // of far sums are as exact as near ones (a decay of 2^-300 and less is 0 all the same)
        long long sum = 0;
        if (tid < kC) {
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
            const uint32_t grows = __ballot_sync(0xffffffffu, !(g <= 0.0f));
            if (lane == 0) {
                s_flags[warp] = off;
                s_flags[2 + warp] = bad;
                s_flags[4 + warp] = grows;
            }
            if (tid == 31) *s_sum = sum;
        }
        if (tid == 0) bulk_wait_read_all();  // the last chunk's stores have left shared memory
        named_bar_sync(1, kRecThreads);
        const unsigned long long masked = (unsigned long long)s_flags[1] << 32 | s_flags[0];
        const bool grows = s_flags[4] | s_flags[5];
        if (tid < kC) {
            if (warp == 1) sum += *s_sum;
            const unsigned long long bad = (unsigned long long)s_flags[3] << 32 | s_flags[2];
            float hi = (float)sum;
            const float lo = (float)(sum - (long long)hi) * 2.3283064365386963e-10f;  // 2^-32
            hi *= 2.3283064365386963e-10f;
            if (bad & (~0ull >> (63 - tid))) hi = __int_as_float(0x7fc00000);
            gates->hi[tid] = hi;
            gates->lo[tid] = lo;
            if (tid == 0) gates->masked = masked;
            gates->beta[tid] = beta;
            const float e = ex2_approx(hi + lo);
            s_e[tid] = e;
            // (a beta that is not finite spoils its chunk whatever it is held under)
            const float m = warp_most(e), mb = warp_most(fabsf(beta) < 1e38f ? fabsf(beta) : 0.0f);
            if (lane == 0) {
                s_most[8 + warp] = m;
                s_most[16 + warp] = mb;
            }
        }
        if (more) fetch(chunk_of(item + step));

        // ---- K and Q to fp16, in place.  Steps that learn nothing: their keys are not looked at
        ok = warp_wait(bar_in, in_phase, a.status);
        in_phase ^= 1;
        landing = false;
        uint4 raw[NP * 4];
        MostBf16 seen, seen_q[2];  // K, and two steps of Q (8 lanes to a step)
        const int r0 = tid >> 3;   // this thread's steps are r0 and r0 + 32
#pragma unroll
        for (int e = 0; e < NP * 4; ++e) {
            raw[e] = *reinterpret_cast<const uint4*>(smem + M::kq + (tid + kRecThreads * e) * 16);
            if (e & 2) {
                seen_q[e & 1].see(raw[e]);
            } else {
                if (masked >> (r0 + 32 * (e & 1)) & 1) raw[e] = make_uint4(0, 0, 0, 0);
                seen.see(raw[e]);
            }
        }
        float most = warp_most(seen.value()), most_q = 0.0f;
        // the steps whose q a common factor is for: those that learn, or all if none does
        const unsigned long long apart = ~masked == 0 ? 0 : masked;
        float own_q[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float m = seen_q[n].value();
            if (apart >> (r0 + 32 * n) & 1) {
                own_q[n] = m;
            } else {
                own_q[n] = 0.0f;
                most_q = fmaxf(most_q, m);
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) own_q[n] = fmaxf(own_q[n], __shfl_xor_sync(0xffffffffu, own_q[n], o));
        }
        most_q = warp_most(most_q);
        if (lane == 0) {
            s_most[warp] = most;
            s_most[24 + warp] = most_q;
        }
        ok = named_bar_and(1, kRecThreads, ok);
        float s_k, s_q[2], q_scale[2];
        most = most_of<8>(s_most);
        const float k_scale = tile_scale(most, kTop, s_k);
        most_q = most_of<8>(s_most + 24);
        if (most == 0.0f) most = 1.0f;
        // (dY and the gradient's W enter products under it, beside rows under the keys': not below a
        // 2^10th of theirs.  For a q that is next to nothing beside the keys, 2^-24, theirs does)
        if (most_q > most * 5.9604645e-8f) most = fmaxf(most_q, most * 0.0009765625f);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            q_scale[n] = tile_scale(fmaxf(most, own_q[n]), kTop, s_q[n]);
            if ((tid & 7) == 0) gates->s_q[r0 + 32 * n] = (uint16_t)(__float_as_uint(s_q[n]) >> 16);
        }
#pragma unroll
        for (int e = 0; e < NP * 4; ++e) {
            f2 x[4];
            uint32_t w[4];
            unpack8_bf16(raw[e], x);
            scaled<4>(x, e & 2 ? q_scale[e & 1] : k_scale, x);
            round_to<4>(x, w);
            *reinterpret_cast<uint4*>(smem + M::kq + (tid + kRecThreads * e) * 16) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (tid < 32) s_dec[tid] = decay(gates->hi[31], gates->lo[31], gates->hi[tid], gates->lo[tid]);
        if (tid < kC) {
            const float d = (gates->hi[tid & 32] - gates->hi[tid]) + (gates->lo[tid & 32] - gates->lo[tid]);
            s_inv[tid] = ex2_approx(d);
            const float span = warp_most(fabsf(d));  // (NaN is above all)
            if (lane == 0) s_span[warp] = span;
        }
        if (tid == 0) {
            gates->s_k = s_k;
            gates->e_max = fmaxf(s_most[8], s_most[9]);
            const float b = fmaxf(fmaxf(s_most[16], s_most[17]), 1.0f);
            const uint32_t top = (__float_as_uint(b) + 0x7fffffu) & 0xff800000u;
            gates->b_top = __uint_as_float(top);
            gates->b_down = inverse(gates->b_top);
        }
        fence_proxy_async_smem();
        named_bar_sync(1, kRecThreads);

        // ---- [K; Q] K^T
        if (tid == 0 && ok) {
            if (FLAGS && item != first) tell(before);
            before = ch;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk)
                mma_f16(tmem + kTmX, kdesc<128>(sb + M::kq, kk), kdesc<128>(sb + M::kq, kk),
                        idesc_f16(128, 64), kk > 0);
            mma_commit(bar_mma);
            bulk_store(rec + rec_kq(DK), smem + M::kq, kq_bytes(DK));
            bulk_commit();
        }
        ok = warp_wait(bar_mma, mma_phase, a.status) && ok;
        mma_phase ^= 1;
        tc_fence_after();
        f2 x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0;
        // rows 0 to 31 have nothing in columns 32 to 63
        const bool any = !(part == 1 && (quarter & 1) == 0);
        if (ok && any) {
            tmem_ld32(t_lane + kTmX + 32 * part, x);
            tmem_wait_ld();
            const float hi = gates->hi[i], lo = gates->lo[i];
            const float f = is_q ? s_k : s_k * s_k * row_beta(s_beta[i]);
            const int j0 = 32 * part;
            const int last = is_q ? i : i - 1;  // of the columns that count
            if (part == 0 && (quarter & 1) && !grows) {
                // rows behind 32, columns before it: the decay from step 31 to the row times
                // that from the column to step 31, neither above 1
                const float e_i = f * decay(hi, lo, gates->hi[31], gates->lo[31]);
                const f2 e2 = pair(e_i, e_i);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 d4 = *reinterpret_cast<const float4*>(s_dec + 2 * e);
                    x[e] = mul2(x[e], mul2(e2, pair(d4.x, d4.y)));
                    x[e + 1] = mul2(x[e + 1], mul2(e2, pair(d4.z, d4.w)));
                }
            } else if ((quarter & 1) == part && s_span[part] < 60.0f) {
                // a block on the diagonal whose decay fp32 holds: from its first step to the
                // row, and inversely to the column
                const float e_i = f * decay(hi, lo, gates->hi[j0], gates->lo[j0]);
                const f2 e2 = pair(e_i, e_i);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const int j = j0 + 2 * e;
                    const float4 d4 = *reinterpret_cast<const float4*>(s_inv + j);
                    float a0, a1, a2, a3;
                    unpair(mul2(x[e], mul2(e2, pair(d4.x, d4.y))), a0, a1);
                    unpair(mul2(x[e + 1], mul2(e2, pair(d4.z, d4.w))), a2, a3);
                    x[e] = pair(j <= last ? a0 : 0.0f, j + 1 <= last ? a1 : 0.0f);
                    x[e + 1] = pair(j + 2 <= last ? a2 : 0.0f, j + 3 <= last ? a3 : 0.0f);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const int j = j0 + 2 * e;
                    float d[4];
                    decays4(gates, j, pair(-hi, -hi), pair(-lo, -lo), last, d);
                    // (columns past the row may hold a q that is not finite)
                    float a0, a1, a2, a3;
                    unpair(x[e], a0, a1);
                    unpair(x[e + 1], a2, a3);
                    x[e] = pair(j <= last ? a0 * (f * d[0]) : 0.0f, j + 1 <= last ? a1 * (f * d[1]) : 0.0f);
                    x[e + 1] = pair(j + 2 <= last ? a2 * (f * d[2]) : 0.0f, j + 3 <= last ? a3 * (f * d[3]) : 0.0f);
                }
            }
        }
        most = warp_most_or_nan<16>(x);
        if (lane == 0 && is_q) s_most[(quarter & 1) * 2 + part] = most;
        if (!is_q)
#pragma unroll
            for (int e = 0; e < 16; e += 2)
                *reinterpret_cast<ulonglong2*>(tri + i * kPitch + 32 * part + 2 * e) =
                    make_ulonglong2(x[e], x[e + 1]);
        tc_fence_before();
        ok = named_bar_and(1, kRecThreads, ok);
        float s_p;  // of the operand (Q K^T) D
        const float p_scale = tile_scale(most_of<4>(s_most), kTop, s_p);
        uint32_t hw[16], lw[16];
        if (is_q) {
            scaled<16>(x, p_scale, x);
            split<16>(x, hw, lw);
            put32(smem + M::p_hi, i, 4 * part, hw);
            put32(smem + M::p_lo, i, 4 * part, lw);
        }
        invert_unit_lower(tri, tmp, tid);

        // ---- T and diag(w) T as operands, N to be kept: row r = tid / 4, 16 columns
        float s_t, s_w;
        {
            const int r = tid >> 2, j0 = (tid & 3) * 16;
            const float w = decay(gates->hi[kC - 1], gates->lo[kC - 1], gates->hi[r], gates->lo[r]);
            f2 t[8], wt[8], nt[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const ulonglong2 m2 = *reinterpret_cast<const ulonglong2*>(tri + r * kPitch + j0 + 2 * e);
                t[e] = m2.x;
                t[e + 1] = m2.y;
            }
            scaled<8>(t, w, wt);
            const float mt = warp_most<8>(t), mw = warp_most<8>(wt);
            if (lane == 0) {
                s_most[warp] = mt;
                s_most[8 + warp] = mw;
            }
            if (a.keep_n) {
                const float inv = 1.0f / row_beta(s_beta[r]);
                const f2 inv2 = pair(inv, inv);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(s_beta + j0 + 2 * e);
                    nt[e] = mul2(t[e], mul2(inv2, b2.x));
                    nt[e + 1] = mul2(t[e + 1], mul2(inv2, b2.y));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {  // the diagonal is 1
                    float n0, n1;
                    unpair(nt[e], n0, n1);
                    nt[e] = pair(j0 + 2 * e == r ? 1.0f : n0, j0 + 2 * e + 1 == r ? 1.0f : n1);
                }
                const float mn = warp_most<8>(nt);
                if (lane == 0) s_most[16 + warp] = mn;
            }
            named_bar_sync(1, kRecThreads);  // (the triangle has been read)
            const float t_scale = tile_scale(most_of<8>(s_most), kTop, s_t);
            const float w_scale = tile_scale(most_of<8>(s_most + 8), kTop, s_w);
            uint32_t th[8], tl[8], wh[8], wl[8];
            scaled<8>(t, t_scale, t);
            scaled<8>(wt, w_scale, wt);
            split<8>(t, th, tl);
            split<8>(wt, wh, wl);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t off = piece(r, (j0 >> 3) + s);
                auto put = [&](uint32_t tile, const uint32_t* v) {
                    *reinterpret_cast<uint4*>(smem + tile + off) =
                        make_uint4(v[4 * s], v[4 * s + 1], v[4 * s + 2], v[4 * s + 3]);
                };
                put(M::t_hi, th);
                put(M::t_lo, tl);
                put(M::w_hi, wh);
                put(M::w_lo, wl);
            }
            if (a.keep_n) {
                float s_n;
                scaled<8>(nt, tile_scale(most_of<8>(s_most + 16), kTop, s_n), nt);
                round_to<8>(nt, th);
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    *reinterpret_cast<uint4*>(smem + M::n + piece(r, (j0 >> 3) + s)) =
                        make_uint4(th[4 * s], th[4 * s + 1], th[4 * s + 2], th[4 * s + 3]);
                if (tid == 0) gates->s_n = s_n;
            }
        }
        fence_proxy_async_smem();
        named_bar_sync(1, kRecThreads);

        // ---- H = K^T diag(w) T (rows of dstate) and P T (rows 64 to 127: the tile of 128
        // rows starts one tile early, its first half is not read); columns 64 to 127: the
        // right operand's lo part
        if (tid == 0 && ok) {
            tc_fence_after();
            constexpr uint32_t idH = idesc_f16(128, 128) | kIdescAMN | kIdescBMN;
            constexpr uint32_t idP = idesc_f16(128, 128) | kIdescBMN;
            constexpr uint32_t idP64 = idesc_f16(128, 64) | kIdescBMN;
            // of 64 columns of dstate the second block of rows is not read either
            constexpr uint32_t lbo = NP > 1 ? 2 * kTile : kTile;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f16(tmem + kTmH, mdesc(sb + M::kq, kk, lbo), mdesc(sb + M::w_hi, kk, kTile), idH, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f16(tmem + kTmP, kdesc<128>(sb + M::p_hi - kTile, kk), mdesc(sb + M::t_hi, kk, kTile),
                        idP, kk > 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f16(tmem + kTmP, kdesc<128>(sb + M::p_lo - kTile, kk), mdesc(sb + M::t_hi, kk, kTile),
                        idP64, 1);
            mma_commit(bar_mma);
            if (a.keep_n) {
                bulk_store(rec + rec_n(DK), smem + M::n, kTile);
                bulk_commit();
            }
        }
        ok = warp_wait(bar_mma, mma_phase, a.status) && ok;
        mma_phase ^= 1;
        tc_fence_after();
        if (tid == 0 && ok) {
            bulk_wait_read_all();   // K, Q and N have left
            if (more) load(chunk_of(item + step));
            landing = more;
        }
        auto both = [&](uint32_t at, f2* v) {  // columns of the hi and the lo part
#pragma unroll
            for (int e0 = 0; e0 < 16; e0 += 8) {
                f2 y[8];
                tmem_ld16(t_lane + at + 2 * e0, v + e0);
                tmem_ld16(t_lane + at + 64 + 2 * e0, y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e0 + e] = add2(v[e0 + e], y[e]);
            }
        };
        // (P is read once more for its operand: with both parts of it and of H a thread has no
        // registers to keep it)
        f2 px[16], hx[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) hx[e] = px[e] = 0;
        if (ok && is_q) both(kTmP + 32 * part, px);
        const float mp = warp_most<16>(px);
        if (ok && row < DK) both(kTmH + 32 * part, hx);
        const float mh = warp_most<16>(hx);
        if (lane == 0) {
            s_most[warp] = mh;
            s_most[8 + warp] = mp;
        }
        tc_fence_before();
        ok = named_bar_and(1, kRecThreads, ok);
        if (!ok) break;
        float s_h2, s_p2;
        const float h_scale = tile_scale(most_of<8>(s_most), kTop, s_h2);
        const float p2_scale = tile_scale(most_of<8>(s_most + 8), kTop, s_p2);
        if (row < DK) {
            scaled<16>(hx, h_scale, hx);
            split<16>(hx, hw, lw);
            put32(smem + M::t_hi, row, 4 * part, hw);
            put32(smem + M::t_hi + h_bytes(DK), row, 4 * part, lw);
        }
        if (is_q) {
            both(kTmP + 32 * part, px);
            scaled<16>(px, p2_scale, px);
            split<16>(px, hw, lw);
            put32(smem + M::p_hi, i, 4 * part, hw);
            put32(smem + M::p_lo, i, 4 * part, lw);
        }
        tc_fence_before();
        if (tid == 0) {
            gates->s_h = s_h2 * s_k * s_w;
            gates->s_p = s_p2 * s_p * s_t;
            gates->h_e = kTopValue * gates->s_h * gates->b_top;  // (without growth a step's decay is 1 at most)
            gates->p_e = kC * kTopValue * gates->s_p * gates->b_top;
            gates->n_e = kTopValue * gates->s_n;
        }
        if (grows) {  // from the operands' hi parts as they lie there, a thread's own
            auto most_e = [&](uint32_t tile, int r, int c0, int n, bool in) {
                float m = 0.0f;
#pragma unroll 1
                for (int c = c0; in && c < c0 + n; ++c) {
                    f2 y[4];
                    unpack8_f16(*reinterpret_cast<const uint4*>(smem + tile + piece(r, c)), y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a0, a1;
                        unpair(mul2(y[e], *reinterpret_cast<const f2*>(s_e + 8 * c + 2 * e)), a0, a1);
                        m = fmaxf(m, fmaxf(fabsf(a0), fabsf(a1)));
                    }
                }
                return warp_most(m);
            };
            const float me[3] = {most_e(M::t_hi, row, 4 * part, 4, row < DK), most_e(M::p_hi, i, 4 * part, 4, is_q),
                                 most_e(M::n, tid >> 2, (tid & 3) * 2, 2, a.keep_n)};
            if (lane == 0)
                for (int n = 0; n < 3; ++n) s_e[kC + 8 * n + warp] = me[n];
            named_bar_sync(1, kRecThreads);
            if (tid == 0) {
                // (an operand's rounding is 2^-11)
                gates->h_e = 1.001f * most_of<8>(s_e + kC) * gates->s_h * gates->b_top;
                gates->p_e = kC * 1.001f * most_of<8>(s_e + kC + 8) * gates->s_p * gates->b_top;
                gates->n_e = 1.001f * most_of<8>(s_e + kC + 16) * gates->s_n;
            }
        }
        fence_proxy_async_smem();
        named_bar_sync(1, kRecThreads);
        if (tid == 0) {
            bulk_store(rec, smem + M::gates, kGateBytes);
            bulk_store(rec + rec_h(DK), smem + M::t_hi, 2 * h_bytes(DK));
            bulk_store(rec + rec_p(DK), smem + M::p_hi, 2 * kTile);
            bulk_commit();
        }
    }
    if (tid == 0) {
        bulk_wait_all();
        if (FLAGS && ok && first < a.count) tell(before);
        if (landing) (void)mbar_wait(bar_in, in_phase, a.status);  // never leave with one landing
    }
}

// The eight warps' tensor memory, allocated and given back around `work`.
template <uint32_t COLS, typename F>
__device__ __forceinline__ void with_tmem(uint32_t* place, int warp, F&& work) {
    if ((threadIdx.x >> 5) == warp) tmem_alloc(place, COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *place;
    work(tmem);
    tc_fence_before();
    __syncthreads();
    if ((threadIdx.x >> 5) == warp) tmem_dealloc(tmem, COLS);
}

template <int DK>
__global__ void __launch_bounds__(kRecThreads, 2)
    records_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const RecArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    with_tmem<256>(reinterpret_cast<uint32_t*>(smem + RecSmem<DK>::bytes - 8), 0, [&](uint32_t tmem) {
        make_records<DK, false>(tm_q, tm_k, a, smem, tmem, blockIdx.x, gridDim.x);
    });
}

// ------------------------------------------------------------------ chain

// Warps on rows (16 for 64 columns of headdim, 4 % faster than 8; 8 for 32), one that
// multiplies, one that loads (a copy takes its issuer some 100 cycles, and a chunk has a dozen),
// one that looks for records, one idle
template <int PW> constexpr int kRowWarps = PW / 4;
template <int PW> constexpr int kChainThreads = 32 * (kRowWarps<PW> + 4);

// PW: columns of headdim a CTA takes (64, or 32 where heads are few).
template <int DK, int PW> struct ChainSmem {
    // a stage (two in turn): gates, panels of K (twice: 128 rows), v (64 columns), panels of Q,
    // P hi | lo
    static constexpr uint32_t k = kGateBytes;
    static constexpr uint32_t v = k + kq_bytes(DK);
    static constexpr uint32_t q = v + kTile;
    static constexpr uint32_t p = q + kq_bytes(DK) / 2;
    static constexpr uint32_t stage = p + 2 * kTile;
    // one H hi | lo: the next comes in between its product and the next but one's
    static constexpr uint32_t h = 2 * stage;
    // S0, rows of dstate, and b R, rows of steps: hi and lo tiles, or both in a tile's row
    static constexpr uint32_t s = h + 2 * h_bytes(DK);
    static constexpr uint32_t s_bytes = (PW / 32) * h_bytes(DK);
    static constexpr uint32_t r = s + s_bytes;
    static constexpr uint32_t r_bytes = (PW / 32) * kTile;
    static constexpr uint32_t misc = r + r_bytes;
    static constexpr uint32_t bytes = misc + 512;
    static_assert(bytes <= 227 * 1024, "shared memory");
};

struct ChainArgs {
    const uint8_t* records;
    uint8_t* kept;
    const float* h0;
    float* last;
    void* y;
    uint32_t* status;
    const uint32_t* flags;  // of records that are being made meanwhile, or NULL
    uint32_t spin_limit;    // looks at one of them before giving up
    Dims d;       // pans: panels of PW columns
};

// One head and PW columns of headdim, chunk after chunk.  Rows of products are lanes of
// tensor memory: of K S0 the steps, twice over, so that all warps share the work on R (a
// warp only reaches its quarter of the lanes); of H b R the state's rows; of Q S0 and P b R the
// steps in lanes 64 to 127.  The state stays in registers (a row of dstate to a lane, 16
// columns) and goes through shared memory as hi + lo each chunk, as b R does.  Right
// operands are [hi | lo] side by side, 2 PW columns to an instruction: at 64 columns an
// instruction is bound by reading its 4 KB of A (55 cycles against 64 for twice the columns).
//
// A chunk of 64 columns takes some 2.6 us (128 heads of 128 x 128, 32 chunks, 256 CTAs: 169 us with what
// training keeps), of 32 columns 1.65 us: instructions of the five passes through registers, their
// fetch (straight code that two warps of a scheduler share), the products' issue and their latency,
// one after the other.
//
// The factors of S and R have to be known before they are written, and a reduction over
// the CTA there would lie on the chain.  So they come from bounds: |R| <= |V| + e |K|_1 |S|,
// |S1| <= e_63 |S| + |b| (|H|_1 |V| + |H e|_1 |K|_1 |S|), with the measured maxima of V and S,
// found while products run.  A bound 2^20 too large would still leave 20 bits.
template <int DK, int PW, typename TO, bool FLAGS>
__device__ __forceinline__ void run_chain(const CUtensorMap& tm_v, const ChainArgs& a, uint8_t* smem,
                                          uint32_t tmem, unsigned index) {
    using M = ChainSmem<DK, PW>;
    constexpr int NP = DK / 64;
    constexpr int NW = kRowWarps<PW>;             // warps on rows
    constexpr int PARTS = NW / 4;                 // of the columns
    constexpr int SC = PW / PARTS, RC = SC / 2;   // columns of S and of R to a thread
    constexpr int kMosts = NW + NW / 2;           // largest values of a chunk
    // tensor memory, hi and lo columns each: K S0, H b R, Q S0, P b R
    constexpr uint32_t kTmX = 0, kTmH = 128, kTmQ = 256, kTmY = 384;
    const uint32_t sb = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + M::misc);  // a stage has come in
    uint64_t* full_h = full + 2;  // H has
    uint64_t* bar_x = full + 3;   // K S0 done
    uint64_t* bar_h = full + 4;   // H b R done
    uint64_t* bar_y = full + 5;   // Q S0 and P b R done: the stage and b R are free
    uint64_t* bar_s = full + 6;   // S0 is in shared memory
    uint64_t* bar_r = full + 7;   // b R is
    uint64_t* bar_o = full + 8;   // Q S0 and P b R have been read
    uint32_t* s_most = reinterpret_cast<uint32_t*>(full + 10);  // [2 chunks][NW warps of S0, NW / 2 of V]
    float* s_first = reinterpret_cast<float*>(s_most + 2 * kMosts);  // [NW]: of the first S0
    uint32_t* s_made = reinterpret_cast<uint32_t*>(s_first + NW);  // records known to be in memory
    uint32_t* s_stop = s_made + 1;  // the chunk whose record never came: all leave when it is due
    constexpr uint32_t kNotMade = 0xffffffffu;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pan = index % a.d.pans;
    const long long bh = index / a.d.pans;
    const int b = (int)(bh / a.d.heads), h = (int)(bh % a.d.heads);
    const int nc = a.d.chunks;

    if (tid == 0) {
        for (int n = 0; n < 6; ++n) mbar_init(full + n, n == 2 ? 2 : 1);
        mbar_init(bar_s, NW);
        mbar_init(bar_r, NW);
        mbar_init(bar_o, NW / 2);
        for (int n = 0; n < 2 * kMosts; ++n) s_most[n] = 0;
        *s_made = 0;
        *s_stop = kNotMade;
        fence_mbar_init();
    }
    __syncthreads();

    if (warp >= NW) {
        give_registers<NW>();
        // Products are issued by one thread.  With 32 columns they are so short that its instructions
        // are what they wait for: there the warp makes the operands together (8192 steps of 16 heads
        // 274 us -> 255 us); with 64, where the votes of its waits cost more, the thread by itself.
        constexpr bool kWarp = PW == 32;
        if (warp == NW && (kWarp || lane == 0)) {
            const int one = kWarp ? elect_one() : 1;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return kWarp ? warp_wait(bar, parity, a.status) : mbar_poll(bar, parity, a.status);
            };
            auto multiply = [&](uint32_t d, uint64_t left, uint64_t right, uint32_t id, uint32_t add) {
                if constexpr (kWarp) mma_f16_warp(one, d, left, right, id, add);
                else mma_f16(d, left, right, id, add);
            };
            auto kept_of = [&](int c) {
                return a.kept + ((bh * nc + c) * a.d.pans + pan) * kept_bytes(DK);
            };
            // right operands: S0 and b R with both parts, or b R's hi part alone
            constexpr uint32_t id2 = idesc_f16(128, 2 * PW) | kIdescBMN;
            constexpr uint32_t id1 = idesc_f16(128, 64) | kIdescBMN;
            for (int c = 0; c < nc; ++c) {
                const uint32_t ph = c & 1, st = sb + (c & 1) * M::stage;
                if (!wait(full + (c & 1), (c >> 1) & 1)) break;
                if (FLAGS && *s_stop == (uint32_t)c) break;
                if (!wait(bar_s, ph)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    multiply(tmem + kTmX, kdesc<128>(st + M::k, kk), mdesc(sb + M::s, kk, h_bytes(DK)),
                             id2, kk > 0);
                if (one) mma_commit(bar_x);
                if (PW == 64 && a.kept) {  // S0's hi part is what training keeps
                    bulk_store(kept_of(c) + kTile, smem + M::s, h_bytes(DK));
                    bulk_commit();
                }
                if (c > 0 && !wait(bar_o, ph ^ 1)) break;
                tc_fence_after();
                // Q in rows 64 to 127: its tiles of 128 rows start one tile early
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    multiply(tmem + kTmQ, kdesc<64>(st + M::q - kTile, kk), mdesc(sb + M::s, kk, h_bytes(DK)),
                             id2, kk > 0);
                if (!wait(full_h, ph)) break;
                if (!wait(bar_r, ph)) break;
                tc_fence_after();
                if (PW == 64 && a.kept) {
                    bulk_wait_read_all();  // S0's place is written when H b R is done
                    // R is in the place of V
                    bulk_store(kept_of(c), smem + (c & 1) * M::stage + M::v, kTile);
                    bulk_commit();
                }
                const uint32_t hh = sb + M::h, hl = hh + h_bytes(DK), pp = st + M::p;
                // (of 64 rows of H the 64 behind them are not read)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    multiply(tmem + kTmH, kdesc<DK>(hh, kk), mdesc(sb + M::r, kk, kTile), id2, kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    multiply(tmem + kTmH, kdesc<DK>(hl, kk), mdesc(sb + M::r, kk, kTile), id1, 1);
                if (one) mma_commit(bar_h);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    multiply(tmem + kTmY, kdesc<128>(pp - kTile, kk), mdesc(sb + M::r, kk, kTile), id2, kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    multiply(tmem + kTmY, kdesc<128>(pp, kk), mdesc(sb + M::r, kk, kTile), id1, 1);
                if (PW == 64 && a.kept) bulk_wait_read_all();  // the stage is loaded again
                if (one) mma_commit(bar_y);
            }
            if (one) bulk_wait_all();
        } else if (warp == NW + 1 && lane == 0) {
            const uint8_t* rec0 = a.records + bh * nc * rec_bytes(DK);
            int loads = 0, h_loads = 0;
            // a record that is being made at the same time: false when that takes too long
            auto made = [&](int c) {
                if constexpr (FLAGS) {
                    const uint32_t addr = smem_u32(s_made);
                    for (uint32_t tries = 0; tries < (1u << 27); ++tries) {
                        uint32_t n;
                        asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(n) : "r"(addr) : "memory");
                        if (n == kNotMade) return false;
                        if (n > (uint32_t)c) return true;
                    }
                    record_status(a.status, SSM_ERR_TIMEOUT);
                    return false;
                }
                return true;
            };
            auto load = [&](int c) {
                uint8_t* st = smem + (c & 1) * M::stage;
                uint64_t* bar = full + (c & 1);
                if (FLAGS && !made(c)) {
                    *s_stop = (uint32_t)c;
                    mbar_arrive(bar);
                    return false;
                }
                const uint8_t* rec = rec0 + (long long)c * rec_bytes(DK);
                mbar_arrive_expect_tx(bar, M::stage);
                bulk_load(st, rec, kGateBytes, bar);
                for (int p = 0; p < NP; ++p) {
                    const uint8_t* kq = rec + rec_kq(DK) + p * 2 * kTile;
                    bulk_load(st + M::k + p * 2 * kTile, kq, kTile, bar);
                    bulk_load(st + M::k + p * 2 * kTile + kTile, kq, kTile, bar);
                    bulk_load(st + M::q + p * kTile, kq + kTile, kTile, bar);
                }
                tma_load_4d(st + M::v, &tm_v, bar, pan * PW, h, c * kC, b);
                bulk_load(st + M::p, rec + rec_p(DK), 2 * kTile, bar);
                ++loads;
                return true;
            };
            auto load_h = [&](int c) {
                mbar_arrive_expect_tx(full_h, 2 * h_bytes(DK));
                bulk_load(smem + M::h, rec0 + (long long)c * rec_bytes(DK) + rec_h(DK), 2 * h_bytes(DK), full_h);
                ++h_loads;
            };
            // H counts as in once the chunk before is known to be done too, so that no barrier
            // is ever a whole turn ahead of this thread
            bool here = load(0);
            if (here) {
                load_h(0);
                mbar_arrive(full_h);
                if (nc > 1) here = load(1);
            }
            for (int c = 0; c + 1 < nc && here; ++c) {
                if (!mbar_wait(bar_h, c & 1, a.status)) break;
                load_h(c + 1);
                if (!mbar_wait(bar_y, c & 1, a.status)) break;
                mbar_arrive(full_h);
                if (c + 2 < nc) here = load(c + 2);
            }
            // never leave with a load still landing
            for (int c = max(0, loads - 2); c < loads; ++c)
                (void)mbar_wait(full + (c & 1), (c >> 1) & 1, a.status);
            if (h_loads > 0) (void)mbar_wait(full_h, (h_loads - 1) & 1, a.status);
        } else if (FLAGS && warp == NW + 2 && lane == 0) {
            // Looks for records that are being made, ahead of the loads: a look takes most of a
            // microsecond
            const uint32_t addr = smem_u32(s_made);
            for (int c = 0; c < nc; ++c) {
                uint32_t tries = 0;
                while (ld_acquire_gpu(a.flags + bh * nc + c) == 0 && ++tries < a.spin_limit) {}
                const bool there = tries < a.spin_limit;
                if (!there) record_status(a.status, SSM_ERR_TIMEOUT);
                asm volatile("fence.proxy.async;" ::: "memory");
                asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(addr),
                             "r"(there ? (uint32_t)c + 1 : kNotMade)
                             : "memory");
                if (!there) break;
            }
        }
    } else {
        take_registers<NW>();
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const bool upper = row >= kC;                 // these rows write y
        const int i = row & 63;                       // the row's step
        const int col0 = pan * PW + SC * part;        // first column of S and y
        const int rc = RC * (2 * part + (upper ? 1 : 0));  // first column of R, in the panel
        // pieces of a row's hi and lo part
        constexpr uint32_t lo_s = PW == 64 ? h_bytes(DK) : 0, lo_r = PW == 64 ? kTile : 0;
        constexpr int lo_c = PW == 64 ? 0 : 4;
        f2 S[SC / 2];      // times its operand's factor; s_s undoes it
        float s_s = 0.0f;
        // what a chunk's rows take from its gates, read before the stage can be refilled
        float f_k = 0.0f, f_q = 0.0f, e_end = 0.0f, k_bound = 0.0f, h_bound = 0.0f, s_h = 0.0f, s_p = 0.0f, b_part = 0.0f,
              b_top = 1.0f;
        bool off = true;
        // the gates of chunk c, and the largest values of its V (upper warps)
        auto gates_of = [&](int c) {
            const bool in = warp_wait(full + (c & 1), (c >> 1) & 1, a.status) &&
                            !(FLAGS && *s_stop == (uint32_t)c);
            const Gates* g = reinterpret_cast<const Gates*>(smem + (c & 1) * M::stage);
            const float e_row = ex2_approx(g->hi[i] + g->lo[i]);
            f_k = e_row * g->s_k;
            f_q = e_row * g->q_factor(i);
            e_end = ex2_approx(g->hi[kC - 1] + g->lo[kC - 1]);
            off = g->masked >> i & 1;
            s_h = g->s_h;
            s_p = g->s_p * g->q_factor(i);
            b_part = g->beta[i] * g->b_down;
            b_top = g->b_top;
            // of |K|_1 over a row, in units of the largest S; of what H takes from that
            k_bound = (DK * kTopValue) * g->s_k;
            h_bound = kC * g->h_e * k_bound;
            k_bound *= fmaxf(g->e_max, 1.0f);
            if (upper) {
                MostBf16 seen;
                const uint8_t* tile = smem + (c & 1) * M::stage + M::v;
#pragma unroll
                for (int p = 0; p < SC / 8; ++p)
                    seen.see(*reinterpret_cast<const uint4*>(tile + piece(i, (SC / 8) * part + p)));
                const float v = warp_most(off ? 0.0f : seen.value());
                if (lane == 0) post_most(s_most + kMosts * (c & 1) + NW + (quarter & 1) * PARTS + part, v, c);
            }
            return in;
        };
        auto factors_of = [&](int c) {
            return reinterpret_cast<float*>(a.kept + ((bh * nc + c) * a.d.pans + pan) * kept_bytes(DK) +
                                            kTile + h_bytes(DK));
        };
        // S0 of chunk c as an operand, and its largest values
        auto put_state = [&](int c) {
            uint32_t hw[SC / 2], lw[SC / 2];
            if (row < DK) {
                split<SC / 2>(S, hw, lw);
                put_pieces<SC / 8>(smem + M::s, row, (SC / 8) * part, hw);
                put_pieces<SC / 8>(smem + M::s + lo_s, row, (SC / 8) * part + lo_c, lw);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(bar_s);
            const float m = warp_most<SC / 2>(S) * s_s;
            if (lane == 0) post_most(s_most + kMosts * (c & 1) + warp, m, c);
            if (PW == 64 && a.kept && tid == 0) factors_of(c)[1] = s_s;
        };
        bool ok = gates_of(0);
        {   // the first chunk: its largest values are measured.  A state that the first step
            // starts anew is not looked at
            const Gates* g = reinterpret_cast<const Gates*>(smem);
            const bool given = a.h0 && row < a.d.dk && ex2_approx(g->hi[0] + g->lo[0]) != 0.0f;
#pragma unroll
            for (int e = 0; e < SC / 2; ++e) {
                const float* at = a.h0 + (bh * a.d.dv + col0 + 2 * e) * a.d.dk + row;
                // (columns come in eights)
                const bool in = given && col0 + 2 * e < a.d.dv;
                S[e] = pair(in ? at[0] : 0.0f, in ? at[a.d.dk] : 0.0f);
            }
            drop_infinities<SC / 2>(S);
            const float m = warp_most<SC / 2>(S);
            if (lane == 0) s_first[warp] = m;
            named_bar_sync(1, 32 * NW);
            scaled<SC / 2>(S, tile_scale(most_of<NW>(s_first), kBoundTop, s_s), S);
            if (ok) put_state(0);
        }
        for (int c = 0; c < nc && ok; ++c) {
            const uint32_t ph = c & 1;
            const float fs = f_k * s_s, fq = f_q * s_s, ee = e_end, sp = s_p, sh = s_h;
            float s_max, v_max;
            ok = read_most<NW / 4>(s_most + kMosts * ph, c, s_max, a.status) &&
                 read_most<NW / 8>(s_most + kMosts * ph + NW, c, v_max, a.status);
            if (!ok) break;
            const float r_bound = fmaf(k_bound, s_max, v_max);
            float s_r, s_next;   // of R, and of the next S
            const float r_scale = tile_scale(r_bound, kBoundTop, s_r);
            const float s_br = s_r * b_top;
            // |H|_1 over a row is at most 64 times its largest value
            const float next = tile_scale(fmaf(h_bound + ee, s_max, kC * 2 * kTopValue * sh * b_top * v_max),
                                          kBoundTop, s_next);
            // ---- R, times its factor, and b R, times b_top less
            {
                uint8_t* tile = smem + (c & 1) * M::stage + M::v;
                f2 v[RC / 2];
#pragma unroll
                for (int p = 0; p < RC / 8; ++p) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    // a masked step's value is not looked at (its row of K is 0)
                    if (!off) w = *reinterpret_cast<const uint4*>(tile + piece(i, rc / 8 + p));
                    unpack8_bf16(w, v + 4 * p);
                }
                scaled<RC / 2>(v, r_scale, v);
                const f2 f = pair(-fs * r_scale, -fs * r_scale);
                f2 x[RC / 2], y[RC / 2];
                ok = warp_wait(bar_x, ph, a.status);
                if (!ok) break;
                tc_fence_after();
                tmem_cols<RC>(t_lane + kTmX + rc, x);
                tmem_cols<RC>(t_lane + kTmX + PW + rc, y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < RC / 2; ++e) x[e] = fma2(f, add2(x[e], y[e]), v[e]);
                uint32_t hw[RC / 2], lw[RC / 2];
                if (PW == 64 && a.kept) {  // V is done with: its largest values are known
                    round_to<RC / 2>(x, hw);
                    put_pieces<RC / 8>(tile, i, rc / 8, hw);
                }
                scaled<RC / 2>(x, b_part, x);
                // (the products that read b R before are done: bar_x follows them)
                split<RC / 2>(x, hw, lw);
                put_pieces<RC / 8>(smem + M::r, i, rc / 8, hw);
                put_pieces<RC / 8>(smem + M::r + lo_r, i, rc / 8 + lo_c, lw);
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(bar_r);
                if (PW == 64 && a.kept && tid == 0) {
                    const Gates* g = reinterpret_cast<const Gates*>(smem + (c & 1) * M::stage);
                    float s_u;
                    (void)tile_scale(kC * b_top * fmaf(kTopValue * g->s_n, v_max, g->n_e * (DK * kTopValue * g->s_k) * s_max),
                                     kBoundTop, s_u);
                    float* f = factors_of(c);
                    f[0] = s_r * g->s_n;
                    f[2] = s_u;
                    f[3] = f[0] * inverse(s_u);
                }
            }
            // ---- the state, times its next factor; the next chunk's gates meanwhile
            scaled<SC / 2>(S, ee * s_s * next, S);
            const float added = sh * s_br * next;
            if (c + 1 < nc) ok = gates_of(c + 1);
            ok = warp_wait(bar_h, ph, a.status) && ok;
            if (!ok) break;
            tc_fence_after();
            if (DK == 128 || !upper) {  // (with 64 rows, what is in the other lanes is no state)
                f2 z[SC / 2], y[SC / 2];
                tmem_cols<SC>(t_lane + kTmH + SC * part, z);
                tmem_cols<SC>(t_lane + kTmH + PW + SC * part, y);
                tmem_wait_ld();
                const f2 a2 = pair(added, added);
#pragma unroll
                for (int e = 0; e < SC / 2; ++e) S[e] = fma2(a2, add2(z[e], y[e]), S[e]);
            }
            s_s = s_next;
            if (c + 1 < nc) put_state(c + 1);
            if (!upper) continue;
            // ---- y
            ok = warp_wait(bar_y, ph, a.status);
            if (!ok) break;
            tc_fence_after();
            f2 x[SC / 2], z[SC / 2];
            tmem_cols<SC>(t_lane + kTmQ + SC * part, x);
            tmem_cols<SC>(t_lane + kTmY + SC * part, z);
            tmem_wait_ld();
            f2 w[SC / 2];
            tmem_cols<SC>(t_lane + kTmQ + PW + SC * part, w);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < SC / 2; ++e) x[e] = add2(x[e], w[e]);
            tmem_cols<SC>(t_lane + kTmY + PW + SC * part, w);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < SC / 2; ++e) z[e] = add2(z[e], w[e]);
            tc_fence_before();
            warp_arrive(bar_o);
            const int t = c * kC + i;
            if (a.y && t < a.d.seqlen) {
                TO* y = static_cast<TO*>(a.y) +
                        (((long long)b * a.d.seqlen + t) * a.d.heads + h) * a.d.dv + col0;
                const f2 f = pair(sp * s_br, sp * s_br), q = pair(fq, fq);
#pragma unroll
                for (int e = 0; e < SC / 2; ++e) x[e] = fma2(q, x[e], mul2(f, z[e]));
                store_row<SC / 2>(y, x, col0, a.d.dv, rows_of_sectors(a.y, a.d.dv));
            }
        }
        if (a.last && row < a.d.dk)
#pragma unroll
            for (int e = 0; e < SC / 2; ++e)
                if (col0 + 2 * e < a.d.dv) {
                    float v0, v1;
                    unpair(S[e], v0, v1);
                    float* at = a.last + (bh * a.d.dv + col0 + 2 * e) * a.d.dk + row;
                    at[0] = v0 * s_s;
                    at[a.d.dk] = v1 * s_s;
                }
    }
}

template <int DK, int PW, typename TO>
__global__ void __launch_bounds__(kChainThreads<PW>, 1)
    chain_kernel(const __grid_constant__ CUtensorMap tm_v, const ChainArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t bytes = ChainSmem<DK, PW>::bytes;
    with_tmem<512>(reinterpret_cast<uint32_t*>(smem + bytes - 8), kRowWarps<PW>, [&](uint32_t tmem) {
        run_chain<DK, PW, TO, false>(tm_v, a, smem, tmem, blockIdx.x);
    });
}

// Records and chains at once, for chains so few that they leave SMs idle: CTAs take numbers,
// the first `makers` make records, chunk by chunk of all heads, and tell the others, which
// follow.  A chain only waits for CTAs with lower numbers, which have started and wait for
// nothing.
template <int DK, typename TO>
__global__ void __launch_bounds__(kChainThreads<32>, 1)
    both_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const RecArgs r, const ChainArgs a,
                uint32_t* ticket, unsigned makers) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t bytes = ChainSmem<DK, 32>::bytes;
    static_assert(RecSmem<DK>::bytes <= bytes, "records' place");
    uint32_t* place = reinterpret_cast<uint32_t*>(smem + bytes - 8);
    if (threadIdx.x == 0) place[1] = atomicAdd(ticket, 1u);
    with_tmem<512>(place, 8, [&](uint32_t tmem) {
        const unsigned number = place[1];
        if (number >= makers) {
            run_chain<DK, 32, TO, true>(tm_v, a, smem, tmem, number - makers);
        } else if (threadIdx.x < kRecThreads) {
            take_registers<8>();
            make_records<DK, true>(tm_q, tm_k, r, smem, tmem, number, makers);
        } else {
            give_registers<8>();
        }
    });
}

// ------------------------------------------------------------------- host

template <typename K>
bool allow_smem(K kernel, uint32_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
           cudaSuccess;
}

template <int DK>
ssm_status_t run_chunked(const gdn_internal::Forward& f, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!gdn_host::make_map(&mq, f.q, f.batch, f.seqlen, f.groups, f.dk, f.q_step) ||
        !gdn_host::make_map(&mk, f.k, f.batch, f.seqlen, f.groups, f.dk, f.k_step) ||
        !gdn_host::make_map(&mv, f.v, f.batch, f.seqlen, f.heads, f.dv, f.v_step))
        return SSM_ERR_CUDA;
    const int sms = ssm_host::sm_count();
    if (sms == 0) return SSM_ERR_CUDA;
    Dims d{f.batch, f.seqlen, f.heads, f.groups, f.dk, f.dv, (f.seqlen + kC - 1) / kC,
           (f.dv + kPan - 1) / kPan};
    RecArgs r{};
    r.g = f.g; r.beta = f.beta; r.records = f.records; r.status = f.status; r.d = d;
    r.gates_bf16 = f.gate_dtype == SSM_BF16;
    r.keep_n = f.kept != nullptr;
    r.count = (unsigned)((long long)f.batch * f.heads * d.chunks);
    ChainArgs a{};
    a.records = f.records; a.kept = f.kept; a.h0 = f.initial_state; a.last = f.final_state;
    a.y = f.y; a.status = f.status; a.d = d;
    // Panels of 32 columns take 0.65 of the time of 64 a chunk (1.65 and 2.6 us), on twice the CTAs (one
    // to an SM): for heads so few that these run at once where the wider ones would leave SMs idle
    const long long bh = (long long)f.batch * f.heads;
    const long long wide = bh * d.pans, narrow = bh * ((f.dv + 31) / 32);
    const bool half = !f.kept && 7 * ((narrow + sms - 1) / sms) < 10 * ((wide + sms - 1) / sms);
    if (half) a.d.pans = (f.dv + 31) / 32;
    // Where these leave SMs idle, the records may be made on those meanwhile.  That costs some 9 us and
    // 0.13 us for each chunk of a chain (its records come one by one), and saves the records' own
    // launch, 0.03 us for each chunk and head; four SMs to a head keep up with its chains.  One
    // after the other and at once, headdim 128: 8192 steps, 1 head 222 and 240 us, 8 heads 257 and
    // 248 us, 18 heads (4.4 SMs to each) 294 and 255 us, 20 heads (3.6) 301 and 308 to 330 us; 2048 steps,
    // 16 heads 89 and 89 us; 512 steps, 16 heads 40 and 49 us.
    const long long makers = sms - narrow;
    if (half && f.flags && makers >= 4 * bh && r.count > 300u + 5u * d.chunks) {
        if (cudaMemsetAsync(f.flags, 0, (r.count + 1) * 4ull, s) != cudaSuccess) return SSM_ERR_CUDA;
        r.flags = f.flags + 1;
        a.flags = f.flags + 1;
        ssm_internal::lookback_setting(&a.spin_limit, &r.drop_first);
        auto both = [&](auto to) {
            using TO = decltype(to);
            constexpr uint32_t bytes = ChainSmem<DK, 32>::bytes;
            if (!allow_smem(both_kernel<DK, TO>, bytes)) return false;
            both_kernel<DK, TO><<<(unsigned)sms, kChainThreads<32>, bytes, s>>>(mq, mk, mv, r, a, f.flags,
                                                                         (unsigned)makers);
            return true;
        };
        if (!(f.out_dtype == SSM_F32 ? both(float{}) : both(__nv_bfloat16{}))) return SSM_ERR_CUDA;
        return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
    }
    if (!allow_smem(records_kernel<DK>, RecSmem<DK>::bytes)) return SSM_ERR_CUDA;
    records_kernel<DK><<<std::min<unsigned>(r.count, 2 * sms), kRecThreads, RecSmem<DK>::bytes, s>>>(mq, mk, r);
    const unsigned grid = (unsigned)(half ? narrow : wide);
    auto go = [&](auto pw, auto to) {
        constexpr int PW = decltype(pw)::value;
        using TO = decltype(to);
        constexpr uint32_t bytes = ChainSmem<DK, PW>::bytes;
        if (!allow_smem(chain_kernel<DK, PW, TO>, bytes)) return false;
        chain_kernel<DK, PW, TO><<<grid, kChainThreads<PW>, bytes, s>>>(mv, a);
        return true;
    };
    auto by_out = [&](auto pw) {
        return f.out_dtype == SSM_F32 ? go(pw, float{}) : go(pw, __nv_bfloat16{});
    };
    if (!(half ? by_out(std::integral_constant<int, 32>{}) : by_out(std::integral_constant<int, 64>{})))
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

extern "C" int ssm_gated_delta_walked_steps(void) { return kWalkSteps; }

extern "C" size_t ssm_gated_delta_workspace_bytes(int batch, int seqlen, int nheads, int dstate,
                                                  int headdim) {
    using namespace gdn_host;
    if (!sizes_ok(batch, seqlen, nheads, nheads, dstate, headdim) ||
        !sizes_fit(batch, seqlen, nheads, dstate, headdim))
        return 0;
    return 1024 + flags_bytes(batch, seqlen, nheads) + records_bytes(batch, seqlen, nheads, dstate);
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
    f.flags = checkpoints ? nullptr : reinterpret_cast<uint32_t*>(ws + 1024);
    f.records = checkpoints ? static_cast<uint8_t*>(checkpoints)
                            : ws + 1024 + gdn_host::flags_bytes(batch, seqlen, nheads);
    f.kept = checkpoints ? f.records + gdn_host::records_bytes(batch, seqlen, nheads, dstate) : nullptr;
    return gdn_internal::chunked_forward(f, s);
}
