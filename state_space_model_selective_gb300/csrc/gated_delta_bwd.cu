// gated_delta_bwd.cu -- the gradient of the gated delta rule, from what the forward kept
// (gated_delta.cuh has the chunked form and its names).
//
// With L the adjoint of the state behind a chunk, per chunk, backwards:
//   dR = P^T dY + H^T L                 (also V's gradient)
//   L0 = e_63 L + Q^T (e dY) - K^T (e dR)
// is a chain two products deep again (chain_bwd_kernel, one head and 64 columns of headdim
// a CTA).  With dR and L kept, everything else is one kernel over all chunks at once:
//   U = T' R;  F = [dR; dY] S0^T;  F2 = U L^T;  [dA'; dP'] = [-dR; dY] U^T
//   dKK = dA' D (j < i),  dQK = dP' D (j <= i)          (beta cancels in dA A: dR = beta T^T dU)
//   dQ = dQK K + e F_q;   dK = dKK K + dKK^T K + dQK^T Q - e F_k + w F2
//   dbeta_i = (dR_i . R_i + sum_j dKK_ij KK_ij) / beta_i
//   dg_t = sum_{i >= t} (sums of row i less sums of column i of M + e_i (q_i F_q,i - k_i F_k,i))
//          + sum_{j < t} w_j k_j F2_j + e_63 <L, S0>,   M = dKK KK + dQK QK
#include <algorithm>
#include <cstring>

#include "gated_delta.cuh"

namespace {

using namespace gdn;

__device__ __forceinline__ float gate_at(const void* p, long long i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void put_gate(void* p, long long i, int bf16, float v) {
    if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ void store8(float* p, const float* o) {
    *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* o) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                              pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
}

// ------------------------------------------------------------------ chain

constexpr int kChainThreads = 288;

template <int DK> struct ChainSmem {
    static constexpr uint32_t k_bytes = (DK / 64) * kTile;
    // a stage: K panels, H hi | lo
    static constexpr uint32_t stage = k_bytes + 2 * h_bytes(DK);
    static constexpr uint32_t q = 2 * stage;
    static constexpr uint32_t p = q + k_bytes;               // P hi | lo, dY
    static constexpr uint32_t dy = p + 2 * kTile;
    static constexpr uint32_t l_hi = dy + kTile;             // L, rows of dstate
    static constexpr uint32_t l_lo = l_hi + h_bytes(DK);
    static constexpr uint32_t o_hi = l_lo + h_bytes(DK);     // e dY, rows of steps
    static constexpr uint32_t o_lo = o_hi + kTile;
    static constexpr uint32_t r_hi = o_lo + kTile;           // -e dR
    static constexpr uint32_t r_lo = r_hi + kTile;
    static constexpr uint32_t xch = r_lo + kTile;            // 64 x 64 fp32, columns first
    static constexpr uint32_t misc = xch + 64 * 64 * 4;
    static constexpr uint32_t bytes = misc + 128;
};

struct ChainArgs {
    const __nv_bfloat16* dy;
    const uint8_t* records;
    uint8_t* kept;          // dR | L
    const float* dlast;
    float* dh0;
    void* dv;
    uint32_t* status;
    Dims d;
};

// Products with a hi and a lo operand on the left put both into the 128 rows of one
// instruction: rows 64 to 127 of dR's tensor memory are its lo part, added through shared
// memory.
template <int DK, typename TG>
__global__ void __launch_bounds__(kChainThreads, 1)
    chain_bwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_dy, const ChainArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using M = ChainSmem<DK>;
    constexpr int NP = DK / 64;
    constexpr uint32_t kTmR = 0, kTmL = 64, kTmCols = 128;
    const uint32_t sb = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + M::misc);  // K and H of a stage
    uint64_t* full_q = full + 2;
    uint64_t* full_p = full + 3;   // P and dY
    uint64_t* bar_x = full + 4;    // dR done
    uint64_t* bar_l = full + 5;    // L0's products done
    uint64_t* bar_s = full + 6;    // L is in shared memory
    uint64_t* bar_o = full + 7;    // e dY is
    uint64_t* bar_r = full + 8;    // -e dR is
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + 9);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pan = blockIdx.x % a.d.pans;
    const long long bh = blockIdx.x / a.d.pans;
    const int b = (int)(bh / a.d.heads), h = (int)(bh % a.d.heads);
    const int nc = a.d.chunks;
    const uint8_t* rec0 = a.records + bh * nc * rec_bytes(DK);

    if (warp == 8) tmem_alloc(s_tmem, kTmCols);
    if (tid == 0) {
        for (int i = 0; i < 6; ++i) mbar_init(full + i, 1);
        mbar_init(bar_s, 8);
        mbar_init(bar_o, 4);
        mbar_init(bar_r, 4);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 8) {
        if (lane == 0) {
            const int group = h / (a.d.heads / a.d.groups);
            int kh_loads = 0, q_loads = 0, p_loads = 0;
            auto load_kh = [&](int it) {
                const int c = nc - 1 - it;
                uint8_t* st = smem + (it & 1) * M::stage;
                mbar_arrive_expect_tx(full + (it & 1), M::stage);
                for (int p = 0; p < NP; ++p)
                    tma_load_4d(st + p * kTile, &tm_k, full + (it & 1), 64 * p, group, c * kC, b);
                bulk_load(st + M::k_bytes, rec0 + (long long)c * rec_bytes(DK), 2 * h_bytes(DK),
                          full + (it & 1));
                ++kh_loads;
            };
            auto load_q = [&](int it) {
                mbar_arrive_expect_tx(full_q, M::k_bytes);
                for (int p = 0; p < NP; ++p)
                    tma_load_4d(smem + M::q + p * kTile, &tm_q, full_q, 64 * p, group,
                                (nc - 1 - it) * kC, b);
                ++q_loads;
            };
            auto load_p = [&](int it) {
                const int c = nc - 1 - it;
                mbar_arrive_expect_tx(full_p, 3 * kTile);
                bulk_load(smem + M::p, rec0 + (long long)c * rec_bytes(DK) + 2 * h_bytes(DK),
                          2 * kTile, full_p);
                tma_load_4d(smem + M::dy, &tm_dy, full_p, pan * kPan, h, c * kC, b);
                ++p_loads;
            };
            load_p(0);
            load_kh(0);
            load_q(0);
            if (nc > 1) load_kh(1);
            int kh_seen = 0, q_seen = 0, p_seen = 0;
            constexpr uint32_t id = idesc_bf16_f32(128, 64) | kIdescAMN | kIdescBMN;
            // (of 64 columns of dstate the second block of rows is not read)
            constexpr uint32_t lbo = kTile;
            for (int it = 0; it < nc; ++it) {
                const uint32_t ph = it & 1, st = sb + (it & 1) * M::stage;
                if (!mbar_wait(full_p, ph, a.status)) break;
                ++p_seen;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16(tmem + kTmR, mdesc(sb + M::p, kk, kTile), mdesc(sb + M::dy, kk, kTile),
                             id, kk > 0);
                if (!mbar_wait(full + (it & 1), (it >> 1) & 1, a.status)) break;
                ++kh_seen;
                if (!mbar_wait(bar_s, ph, a.status)) break;
                tc_fence_after();
                const uint32_t hh = st + M::k_bytes;
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk) {
                    mma_bf16(tmem + kTmR, mdesc(hh, kk, h_bytes(DK)), mdesc(sb + M::l_hi, kk, kTile), id, 1);
                    mma_bf16(tmem + kTmR, mdesc(hh, kk, h_bytes(DK)), mdesc(sb + M::l_lo, kk, kTile), id, 1);
                }
                mma_commit(bar_x);
                if (!mbar_wait(full_q, ph, a.status)) break;
                ++q_seen;
                if (!mbar_wait(bar_o, ph, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16(tmem + kTmL, mdesc(sb + M::q, kk, lbo), mdesc(sb + M::o_hi, kk, kTile), id, kk > 0);
                    mma_bf16(tmem + kTmL, mdesc(sb + M::q, kk, lbo), mdesc(sb + M::o_lo, kk, kTile), id, 1);
                }
                if (it + 1 < nc) {
                    if (!mbar_wait(bar_x, ph, a.status)) break;
                    load_p(it + 1);
                }
                if (!mbar_wait(bar_r, ph, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16(tmem + kTmL, mdesc(st, kk, lbo), mdesc(sb + M::r_hi, kk, kTile), id, 1);
                    mma_bf16(tmem + kTmL, mdesc(st, kk, lbo), mdesc(sb + M::r_lo, kk, kTile), id, 1);
                }
                mma_commit(bar_l);
                if (it + 1 < nc) {
                    if (!mbar_wait(bar_l, ph, a.status)) break;
                    load_q(it + 1);
                    if (it + 2 < nc) load_kh(it + 2);
                }
            }
            // never leave with a load still landing
            for (; kh_seen < kh_loads; ++kh_seen)
                (void)mbar_wait(full + (kh_seen & 1), (kh_seen >> 1) & 1, a.status);
            if (q_seen < q_loads) (void)mbar_wait(full_q, q_seen & 1, a.status);
            if (p_seen < p_loads) (void)mbar_wait(full_p, p_seen & 1, a.status);
        }
    } else {
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + 32 * part;
        const int col0 = pan * kPan + 32 * part;
        const bool upper = row >= kC;   // these rows make e dY
        const int i = row & 63;
        float* xch = reinterpret_cast<float*>(smem + M::xch) + 32 * part * 64 + i;
        float L[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
            L[e] = a.dlast && row < a.d.dk && col0 + e < a.d.dv
                       ? a.dlast[(bh * a.d.dv + col0 + e) * a.d.dk + row] : 0.0f;
        auto put_state = [&](int c) {
            if (row < DK) {
                put32_split(smem + M::l_hi, smem + M::l_lo, row, 4 * part, L);
                put32(a.kept + ((bh * nc + c) * a.d.pans + pan) * kept_bytes(DK) + kTile, row,
                      4 * part, L);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(bar_s);
        };
        uint4 dy[4];
        float e_row = 0.0f, e_end = 0.0f;
        bool off = true;
        auto fetch = [&](int c) {
            const Gates* g = reinterpret_cast<const Gates*>(rec0 + (long long)c * rec_bytes(DK) +
                                                            hp_bytes(DK) + kTile);
            e_row = ex2_approx(g->hi[i] + g->lo[i]);
            e_end = ex2_approx(g->hi[kC - 1] + g->lo[kC - 1]);
            off = g->masked >> i & 1;
            const int t = c * kC + i;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                dy[p] = upper && t < a.d.seqlen && col0 + 8 * p < a.d.dv
                            ? *reinterpret_cast<const uint4*>(
                                  a.dy + (((long long)b * a.d.seqlen + t) * a.d.heads + h) * a.d.dv +
                                  col0 + 8 * p)
                            : make_uint4(0, 0, 0, 0);
        };
        put_state(nc - 1);
        fetch(nc - 1);
        bool ok = true;  // the same for all lanes of a warp
        for (int it = 0; it < nc; ++it) {
            const int c = nc - 1 - it;
            const uint32_t ph = it & 1;
            const float er = e_row, ee = e_end;
            const bool masked = off;
            float x[32];
            if (upper) {  // (the products that read e dY before are done: bar_l follows them)
#pragma unroll
                for (int p = 0; p < 4; ++p) unpack8(dy[p], x + 8 * p);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] *= er;
                put32_split(smem + M::o_hi, smem + M::o_lo, i, 4 * part, x);
                fence_proxy_async_smem();
                warp_arrive(bar_o);
            }
            if (c > 0) fetch(c - 1);
            ok = ok && warp_wait(bar_x, ph, a.status);
            tc_fence_after();
            if (ok) {
                tmem_ld32(t_lane + kTmR, x);
                tmem_wait_ld();
                if (upper)
#pragma unroll
                    for (int e = 0; e < 32; ++e) xch[64 * e] = x[e];
            }
            tc_fence_before();
            if (!named_bar_and(1, 256, ok)) break;  // all eight warps leave together
            if (!upper) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] += xch[64 * e];
                const int t = c * kC + i;
                if (t < a.d.seqlen) {
                    TG* dv = static_cast<TG*>(a.dv) +
                             (((long long)b * a.d.seqlen + t) * a.d.heads + h) * a.d.dv + col0;
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (col0 + 8 * p < a.d.dv) store8(dv + 8 * p, x + 8 * p);
                }
                put32(a.kept + ((bh * nc + c) * a.d.pans + pan) * kept_bytes(DK), i, 4 * part, x);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] *= -er;
                put32_split(smem + M::r_hi, smem + M::r_lo, i, 4 * part, x);
                if (masked && part < NP) {
                    // a masked step's key is not looked at: its dR is 0, but 0 NaN is not
                    (void)mbar_wait(full + (it & 1), (it >> 1) & 1, a.status);
#pragma unroll
                    for (int p = 0; p < 8; ++p)
                        *reinterpret_cast<uint4*>(smem + (it & 1) * M::stage + part * kTile + i * 128 +
                                                  16 * p) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                warp_arrive(bar_r);
            }
            float z[32];
            ok = warp_wait(bar_l, ph, a.status);
            tc_fence_after();
            if (ok) {
                tmem_ld32(t_lane + kTmL, z);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) L[e] = ee == 0.0f ? z[e] : fmaf(ee, L[e], z[e]);
                if (c > 0) put_state(c - 1);
            }
        }
        if (a.dh0 && row < a.d.dk)
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (col0 + e < a.d.dv) a.dh0[(bh * a.d.dv + col0 + e) * a.d.dk + row] = L[e];
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, kTmCols);
}

// ------------------------------------------------------------------ grads

constexpr int kGradThreads = 256;

template <int DK> struct GradSmem {
    static constexpr uint32_t kq = 0;                        // panels of [K | Q]
    static constexpr uint32_t rdo = 0;                       // of a stage: dR, dY
    static constexpr uint32_t s0 = 2 * kTile;
    static constexpr uint32_t l = s0 + h_bytes(DK);
    static constexpr uint32_t t = l + h_bytes(DK);           // T', then R
    static constexpr uint32_t r = t + kTile;
    static constexpr uint32_t stage = r + kTile;
    static constexpr uint32_t stages = (DK / 64) * 2 * kTile;
    static constexpr uint32_t u = stages + 2 * stage;        // U, then W (rows 64 to 127 of
    static constexpr uint32_t w = u + kTile;                 // U's operand are not read)
    static constexpr uint32_t sums = w + 3 * kTile;          // floats (W^T's second block reads
                                                             // one tile past W)
    static constexpr uint32_t n_sums = 128 * 2 + 4 * 64 + 64 * 2 + 64 * 2 + 8 + 64 * 2 + 64;
    static constexpr uint32_t misc = sums + n_sums * 4;
    static constexpr uint32_t bytes = misc + 128;
};

struct GradArgs {
    const uint8_t* records;
    const uint8_t* kept;     // R | S0
    const uint8_t* adjoint;  // dR | L
    const void *g, *beta;
    void *dq, *dk, *dg, *dbeta;
    uint32_t* status;
    Dims d;
    int gates_bf16;
};

// 8 products of a row's 16-byte pieces of two tiles, summed.
__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
    float x[8], y[8], s = 0.0f;
    unpack8(a, x);
    unpack8(b, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
    return s;
}

template <int DK, typename TG>
__global__ void __launch_bounds__(kGradThreads, 1)
    grads_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_dy, const GradArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using M = GradSmem<DK>;
    constexpr int NP = DK / 64, CW = DK / 2;  // columns of dstate a thread holds
    // tensor memory: F, F2; [dA'; dP'], [K; Q] K^T and U until W is made, then W K and W^T [K; Q]
    constexpr uint32_t kTmF = 0, kTmF2 = 128, kTmA = 256, kTmX = 320, kTmU = 384, kTmW = 384,
                       kTmV = 256, kTmCols = 512;
    const uint32_t sb = smem_u32(smem);
    float* s_row = reinterpret_cast<float*>(smem + M::sums);  // [128][2]
    float* s_col = s_row + 256;                               // [4][64]
    float* s_dec = s_col + 256;                               // [64][2]
    float* s_db = s_dec + 128;                                // [64][2]
    float* s_c = s_db + 128;                                  // [8]
    float* s_hi = s_c + 8;
    float* s_lo = s_hi + 64;
    float* s_scan = s_lo + 64;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + M::misc);
    uint64_t* bar_kq = full + 2;
    uint64_t* bar_u = full + 3;
    uint64_t* bar_f = full + 4;
    uint64_t* bar_w = full + 5;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + 6);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
    const bool is_q = row >= kC;
    const int i = row & 63;
    const int nc = a.d.chunks, ratio = a.d.heads / a.d.groups;
    const int c = blockIdx.x % nc;
    const int bg = blockIdx.x / nc, b = bg / a.d.groups, group = bg % a.d.groups;
    const int t0 = c * kC;
    const int steps = ratio * a.d.pans;
    auto chunk_of = [&](int n) {  // index of the chunk and head of step n
        return ((long long)b * a.d.heads + group * ratio + n / a.d.pans) * nc + c;
    };

    if (warp == 0) tmem_alloc(s_tmem, kTmCols);
    int loads = 0;
    auto load = [&](int n) {
        uint8_t* st = smem + M::stages + (n & 1) * M::stage;
        uint64_t* bar = full + (n & 1);
        const long long ch = chunk_of(n), at = (ch * a.d.pans + n % a.d.pans) * kept_bytes(DK);
        mbar_arrive_expect_tx(bar, M::stage);
        bulk_load(st + M::rdo, a.adjoint + at, kTile, bar);
        tma_load_4d(st + M::rdo + kTile, &tm_dy, bar, (n % a.d.pans) * kPan,
                    group * ratio + n / a.d.pans, t0, b);
        bulk_load(st + M::s0, a.kept + at + kTile, h_bytes(DK), bar);
        bulk_load(st + M::l, a.adjoint + at + kTile, h_bytes(DK), bar);
        bulk_load(st + M::t, a.records + ch * rec_bytes(DK) + hp_bytes(DK), kTile, bar);
        bulk_load(st + M::r, a.kept + at, kTile, bar);
        ++loads;
    };
    if (tid == 0) {
        for (int n = 0; n < 6; ++n) mbar_init(full + n, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar_kq, NP * 2 * kTile);
        for (int p = 0; p < NP; ++p) {
            tma_load_4d(smem + M::kq + p * 2 * kTile, &tm_k, bar_kq, 64 * p, group, t0, b);
            tma_load_4d(smem + M::kq + p * 2 * kTile + kTile, &tm_q, bar_kq, 64 * p, group, t0, b);
        }
        load(0);
        if (steps > 1) load(1);
    }
    // keys that no head of the group looks at
    unsigned long long unseen = ~0ull;
    for (int n = 0; n < steps; n += a.d.pans)
        unseen &= reinterpret_cast<const Gates*>(a.records + chunk_of(n) * rec_bytes(DK) +
                                                 hp_bytes(DK) + kTile)->masked;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    bool ok = warp_wait(bar_kq, 0, a.status);
    if (unseen) {
        if (ok)
            for (int e = tid; e < NP * kC * 8; e += kGradThreads) {
                const int r = (e >> 3) & 63;
                if (unseen >> r & 1)
                    *reinterpret_cast<uint4*>(smem + M::kq + (e >> 9) * 2 * kTile + r * 128 +
                                              (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
        fence_proxy_async_smem();
    }
    ok = __syncthreads_and(ok);

    float acc[CW];  // of dK (rows 0 to 63) or dQ
#pragma unroll
    for (int e = 0; e < CW; ++e) acc[e] = 0.0f;
    float hi_i = 0.0f, lo_i = 0.0f, beta_sum = 0.0f, ls = 0.0f;
    bool off = false;

    for (int n = 0; n < steps && ok; ++n) {
        const int p = n % a.d.pans, h = group * ratio + n / a.d.pans;
        const uint32_t st = sb + M::stages + (n & 1) * M::stage;
        const uint8_t* sg = smem + M::stages + (n & 1) * M::stage;
        const long long ch = chunk_of(n);
        const Gates* gates = reinterpret_cast<const Gates*>(a.records + ch * rec_bytes(DK) +
                                                            hp_bytes(DK) + kTile);
        if (p == 0) {  // a head begins
            hi_i = gates->hi[i];
            lo_i = gates->lo[i];
            off = gates->masked >> i & 1;
            if (tid < kC) {
                s_hi[tid] = hi_i;
                s_lo[tid] = lo_i;
            }
            beta_sum = ls = 0.0f;
        }
        // ---- U = T' R, and with a head's first columns [K; Q] K^T
        if (tid == 0) {
            const bool in = mbar_wait(full + (n & 1), (n >> 1) & 1, a.status);
            tc_fence_after();
            if (in) {
                if (p == 0)
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        mma_bf16(tmem + kTmX, kdesc<128>(sb + M::kq, kk), kdesc<128>(sb + M::kq, kk),
                                 idesc_bf16_f32(128, 64), kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16(tmem + kTmU, kdesc<128>(st + M::t, kk), mdesc(st + M::r, kk, kTile),
                             idesc_bf16_f32(128, 64) | kIdescBMN, kk > 0);
                mma_commit(bar_u);
            }
        }
        ok = warp_wait(full + (n & 1), (n >> 1) & 1, a.status);
        // sums over this panel's columns: dR . R, and L . S0
        if (ok) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t off4 = piece(row, 4 * part + q);
                if (!is_q)
                    beta_sum += dot8(*reinterpret_cast<const uint4*>(sg + M::rdo + off4),
                                     *reinterpret_cast<const uint4*>(sg + M::r + off4));
                if (row < DK)
                    ls += dot8(*reinterpret_cast<const uint4*>(sg + M::s0 + off4),
                               *reinterpret_cast<const uint4*>(sg + M::l + off4));
            }
        }
        ok = ok && warp_wait(bar_u, n & 1, a.status);
        tc_fence_after();
        if (ok && !is_q) {
            float x[32];
            tmem_ld32(t_lane + kTmU + 32 * part, x);
            tmem_wait_ld();
            put32(smem + M::u, i, 4 * part, x);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t id64 = idesc_bf16_f32(128, 64), idk = idesc_bf16_f32(128, DK);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t more = p > 0 || kk > 0;
                mma_bf16(tmem + kTmA, kdesc<128>(st + M::rdo, kk), kdesc<64>(sb + M::u, kk), id64, more);
                mma_bf16(tmem + kTmF, kdesc<128>(st + M::rdo, kk), kdesc<DK>(st + M::s0, kk), idk, more);
                mma_bf16(tmem + kTmF2, kdesc<128>(sb + M::u, kk), kdesc<DK>(st + M::l, kk), idk, more);
            }
            mma_commit(bar_f);
        }
        ok = warp_wait(bar_f, n & 1, a.status);
        tc_fence_after();
        if (tid == 0 && ok && n + 2 < steps) load(n + 2);
        ok = __syncthreads_and(ok);
        if (!ok || p + 1 < a.d.pans) continue;

        // ---- the head's last columns are in: W = [dKK; dQK], and its sums with [KK; QK]
        float rsum = 0.0f;
        {
            float x[32], m[32];
            tmem_ld32(t_lane + kTmA + 32 * part, x);
            tmem_ld32(t_lane + kTmX + 32 * part, m);
            tmem_wait_ld();
            const int last = is_q ? i : i - 1;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const int j = 32 * part + e;
                x[e] = j <= last ? (is_q ? x[e] : -x[e]) * decay(hi_i, lo_i, s_hi[j], s_lo[j]) : 0.0f;
                m[e] = j <= last ? m[e] * x[e] : 0.0f;
                rsum += m[e];
            }
            put32(smem + M::w, row, 4 * part, x);
            // sums over the warp's 32 rows: lane l ends with column l
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
                for (int k = 0; k < o; ++k) {
                    const bool up = lane & o;
                    const float send = up ? m[k] : m[k + o];
                    m[k] = (up ? m[k + o] : m[k]) + __shfl_xor_sync(0xffffffffu, send, o);
                }
            s_col[quarter * 64 + 32 * part + lane] = m[0];
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t idW = idesc_bf16_f32(128, DK) | kIdescBMN;
            constexpr uint32_t idV = idesc_bf16_f32(128, DK) | kIdescAMN | kIdescBMN;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_bf16(tmem + kTmW, kdesc<128>(sb + M::w, kk), mdesc(sb + M::kq, kk, 2 * kTile), idW, kk > 0);
            // (rows 64 to 127 of W^T [K; Q] are not read)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16(tmem + kTmV, mdesc(sb + M::w, kk, kTile), mdesc(sb + M::kq, kk, 2 * kTile), idV, kk > 0);
            mma_commit(bar_w);
        }
        // ---- the state's parts
        const float er = ex2_approx(hi_i + lo_i);
        const float wr = decay(s_hi[kC - 1], s_lo[kC - 1], hi_i, lo_i);
        float into = 0.0f, outof = 0.0f;
#pragma unroll
        for (int b8 = 0; b8 < CW; b8 += 16) {
            const int c0 = CW * part + b8;
            float f[16], f2[16], x[16];
            tmem_ld16(t_lane + kTmF + c0, f);
            if (!is_q) tmem_ld16(t_lane + kTmF2 + c0, f2);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 2; ++q)
                unpack8(*reinterpret_cast<const uint4*>(
                            smem + M::kq + (c0 >> 6) * 2 * kTile + piece(row, ((c0 & 63) >> 3) + q)),
                        x + 8 * q);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                into = fmaf(x[e], f[e], into);
                acc[b8 + e] = fmaf(is_q ? er : -er, f[e], acc[b8 + e]);
                if (!is_q) {
                    outof = fmaf(x[e], f2[e], outof);
                    acc[b8 + e] = fmaf(wr, f2[e], acc[b8 + e]);
                }
            }
        }
        s_row[2 * row + part] = rsum + (is_q ? er * into : -er * into);
        if (!is_q) {
            s_dec[2 * i + part] = wr * outof;
            s_db[2 * i + part] = beta_sum + rsum;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        if (lane == 0) s_c[warp] = ls;
        __syncthreads();
        // ---- the gates
        if (tid < kC) {
            const int t = t0 + i;
            const long long at = ((long long)b * a.d.seqlen + t) * a.d.heads + h;
            float up = s_row[2 * i] + s_row[2 * i + 1] + s_row[128 + 2 * i] + s_row[129 + 2 * i];
            for (int q = 0; q < 4; ++q) up -= s_col[q * 64 + i];
            float down = s_dec[2 * i] + s_dec[2 * i + 1];
            const float own = down;
            // sums of `up` from here on, of `down` before here
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_down_sync(0xffffffffu, up, o);
                const float d = __shfl_up_sync(0xffffffffu, down, o);
                if (lane + o < 32) up += u;
                if (lane >= o) down += d;
            }
            if (tid == 32) s_scan[0] = up;
            if (tid == 31) s_scan[1] = down;
            named_bar_sync(2, 64);
            if (warp == 0) up += s_scan[0];
            if (warp == 1) down += s_scan[1];
            float all = 0.0f;
            for (int q = 0; q < 8; ++q) all += s_c[q];
            if (t < a.d.seqlen) {
                const float e_end = ex2_approx(s_hi[kC - 1] + s_lo[kC - 1]);
                // a gate of -inf cuts the past off: its gradient is 0
                const bool cut = ex2_approx(gate_at(a.g, at, a.gates_bf16) * kLog2e) == 0.0f;
                put_gate(a.dg, at, a.gates_bf16, cut ? 0.0f : up + (down - own) + e_end * all);
                put_gate(a.dbeta, at, a.gates_bf16,
                         off ? 0.0f : (s_db[2 * i] + s_db[2 * i + 1]) / gate_at(a.beta, at, a.gates_bf16));
            }
        }
        // ---- the products with W
        ok = warp_wait(bar_w, (n / a.d.pans) & 1, a.status);
        tc_fence_after();
        if (ok) {
#pragma unroll
            for (int b8 = 0; b8 < CW; b8 += 16) {
                const int c0 = CW * part + b8;
                float f[16], f2[16];
                tmem_ld16(t_lane + kTmW + c0, f);
                if (!is_q) tmem_ld16(t_lane + kTmV + c0, f2);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[b8 + e] += is_q ? f[e] : f[e] + f2[e];
            }
        }
        tc_fence_before();
        ok = __syncthreads_and(ok);  // sums and tensor memory are free for the next head
    }
    if (ok && t0 + i < a.d.seqlen) {
        TG* out = static_cast<TG*>(is_q ? a.dq : a.dk) +
                  (((long long)b * a.d.seqlen + t0 + i) * a.d.groups + group) * a.d.dk + CW * part;
#pragma unroll
        for (int e = 0; e < CW; e += 8)
            if (CW * part + e < a.d.dk) store8(out + e, acc + e);
    }
    if (tid == 0 && !ok) {  // never leave with a load still landing
        if (loads > 0) (void)mbar_wait(full + ((loads - 1) & 1), ((loads - 1) >> 1) & 1, a.status);
        if (loads > 1) (void)mbar_wait(full + (loads & 1), ((loads - 2) >> 1) & 1, a.status);
        (void)mbar_wait(bar_kq, 0, a.status);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kTmCols);
}

// ------------------------------------------------------------------- host

template <typename K>
bool allow_smem(K kernel, uint32_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
           cudaSuccess;
}

struct Backward {
    const void *q, *k, *dy;
    long long q_step, k_step;
    ChainArgs chain;
    GradArgs grads;
};

template <int DK, typename TG>
ssm_status_t run_backward(const Backward& w, cudaStream_t s) {
    const Dims& d = w.chain.d;
    CUtensorMap mq, mk, my;
    if (!gdn_host::make_map(&mq, w.q, d.batch, d.seqlen, d.groups, d.dk, w.q_step) ||
        !gdn_host::make_map(&mk, w.k, d.batch, d.seqlen, d.groups, d.dk, w.k_step) ||
        !gdn_host::make_map(&my, w.dy, d.batch, d.seqlen, d.heads, d.dv, (long long)d.heads * d.dv))
        return SSM_ERR_CUDA;
    if (!allow_smem(chain_bwd_kernel<DK, TG>, ChainSmem<DK>::bytes) ||
        !allow_smem(grads_kernel<DK, TG>, GradSmem<DK>::bytes))
        return SSM_ERR_CUDA;
    chain_bwd_kernel<DK, TG><<<(unsigned)((long long)d.batch * d.heads * d.pans), kChainThreads,
                               ChainSmem<DK>::bytes, s>>>(mq, mk, my, w.chain);
    grads_kernel<DK, TG><<<(unsigned)((long long)d.batch * d.groups * d.chunks), kGradThreads,
                           GradSmem<DK>::bytes, s>>>(mq, mk, my, w.grads);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

}  // namespace

extern "C" size_t ssm_gated_delta_bwd_workspace_bytes(int batch, int seqlen, int nheads, int dstate,
                                                      int headdim) {
    using namespace gdn_host;
    if (!sizes_ok(batch, seqlen, nheads, nheads, dstate, headdim) ||
        !sizes_fit(batch, seqlen, nheads, dstate, headdim))
        return 0;
    return 1024 + keep_bytes(batch, seqlen, nheads, dstate, headdim);
}

extern "C" ssm_status_t ssm_gated_delta_bwd(
    const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
    long long v_stride, const void* g, const void* beta, const float* initial_state, const void* dy,
    const float* dfinal_state, const void* checkpoints, void* dq, void* dk, void* dv, void* dg,
    void* dbeta, float* dinitial_state, int batch, int seqlen, int nheads, int ngroups, int dstate,
    int headdim, ssm_dtype_t in_dtype, ssm_dtype_t gate_dtype, ssm_dtype_t grad_dtype,
    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ssm_host;
    using gdn_host::Span;
    using gdn_host::strided_bytes;
    if (!gdn_host::sizes_ok(batch, seqlen, nheads, ngroups, dstate, headdim)) return SSM_ERR_SHAPE;
    const long long qw = (long long)ngroups * dstate, vw = (long long)nheads * headdim;
    if (q_stride < qw || k_stride < qw || v_stride < vw) return SSM_ERR_SHAPE;
    if (!dtype_ok(in_dtype) || !dtype_ok(gate_dtype) || !dtype_ok(grad_dtype)) return SSM_ERR_DTYPE;
    if (!gdn_host::sizes_fit(batch, seqlen, nheads, dstate, headdim) || in_dtype != SSM_BF16)
        return SSM_ERR_UNSUPPORTED;
    if (batch == 0 || nheads == 0) return SSM_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t sb = (size_t)batch * nheads * headdim * dstate * 4, es = dtype_size(in_dtype);
    const long long steps = (long long)batch * seqlen;
    if (seqlen > 0 && (!q || !k || !v || !g || !beta || !dy || !dq || !dk || !dv || !dg || !dbeta))
        return SSM_ERR_NULL;
    const size_t kb = ssm_gated_delta_checkpoint_bytes(batch, seqlen, nheads, dstate, headdim);
    const size_t own = ssm_gated_delta_bwd_workspace_bytes(batch, seqlen, nheads, dstate, headdim);
    const size_t wb = seqlen == 0 ? 0 : own + (checkpoints ? 0 : kb);
    if (wb && (!workspace || workspace_bytes < wb)) return SSM_ERR_WORKSPACE;
    for (const void* p : {q, k, v, (const void*)initial_state, dy, (const void*)dfinal_state, checkpoints,
                          (const void*)dq, (const void*)dk, (const void*)dv,
                          (const void*)dinitial_state, (const void*)workspace})
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    for (long long st : {q_stride, k_stride, v_stride})
        if (seqlen > 0 && st * es % 16) return SSM_ERR_ALIGN;
    const size_t gs = dtype_size(gate_dtype);
    for (const void* p : {g, beta, (const void*)dg, (const void*)dbeta})
        if (reinterpret_cast<uintptr_t>(p) % gs) return SSM_ERR_ALIGN;
    const size_t gb = (size_t)steps * nheads * gs, ge = dtype_size(grad_dtype);
    const Span ins[] = {{q, strided_bytes(steps, qw, q_stride, es)},
                        {k, strided_bytes(steps, qw, k_stride, es)},
                        {v, strided_bytes(steps, vw, v_stride, es)},
                        {g, gb}, {beta, gb}, {initial_state, sb}, {dy, (size_t)steps * vw * es},
                        {dfinal_state, sb}, {checkpoints, checkpoints ? kb : 0}};
    const Span outs[] = {{dq, (size_t)steps * qw * ge}, {dk, (size_t)steps * qw * ge},
                         {dv, (size_t)steps * vw * ge}, {dg, gb}, {dbeta, gb},
                         {dinitial_state, sb}, {workspace, wb}};
    for (const Span& o : outs)
        for (const Span& i : ins) {
            if (o.p == dinitial_state && i.p == dfinal_state && dinitial_state == dfinal_state) continue;
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
        }
    for (int i = 0; i < 7; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;
    if (seqlen == 0) {
        if (!dinitial_state || dinitial_state == dfinal_state) return SSM_OK;
        const cudaError_t e = dfinal_state ? cudaMemcpyAsync(dinitial_state, dfinal_state, sb,
                                                             cudaMemcpyDeviceToDevice, s)
                                           : cudaMemsetAsync(dinitial_state, 0, sb, s);
        return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (cudaMemsetAsync(ws, 0, 8, s) != cudaSuccess) return SSM_ERR_CUDA;
    uint32_t* status = reinterpret_cast<uint32_t*>(ws) + 1;
    const uint8_t* records = static_cast<const uint8_t*>(checkpoints);
    const size_t rb = gdn_host::records_bytes(batch, seqlen, nheads, dstate);
    if (!checkpoints) {  // the forward again, without y
        gdn_internal::Forward f{};
        f.q = q; f.k = k; f.v = v; f.q_step = q_stride; f.k_step = k_stride; f.v_step = v_stride;
        f.g = g; f.beta = beta; f.gate_dtype = gate_dtype; f.initial_state = initial_state;
        f.out_dtype = SSM_BF16; f.status = status;
        f.batch = batch; f.seqlen = seqlen; f.heads = nheads; f.groups = ngroups; f.dk = dstate; f.dv = headdim;
        f.records = ws + own;
        f.kept = f.records + rb;
        if (ssm_status_t st = gdn_internal::chunked_forward(f, s)) return st;
        records = f.records;
    }
    Backward w{};
    w.q = q; w.k = k; w.dy = dy; w.q_step = q_stride; w.k_step = k_stride;
    const Dims d{batch, seqlen, nheads, ngroups, dstate, headdim, (seqlen + kC - 1) / kC,
                 (headdim + kPan - 1) / kPan};
    w.chain.dy = static_cast<const __nv_bfloat16*>(dy);
    w.chain.records = records;
    w.chain.kept = ws + 1024;
    w.chain.dlast = dfinal_state; w.chain.dh0 = dinitial_state; w.chain.dv = dv;
    w.chain.status = status; w.chain.d = d;
    w.grads.records = records; w.grads.kept = records + rb; w.grads.adjoint = ws + 1024;
    w.grads.g = g; w.grads.beta = beta;
    w.grads.dq = dq; w.grads.dk = dk; w.grads.dg = dg; w.grads.dbeta = dbeta;
    w.grads.status = status; w.grads.d = d; w.grads.gates_bf16 = gate_dtype == SSM_BF16;
    const bool small = gdn_host::dk_tile(dstate) == 64;
    if (grad_dtype == SSM_F32) return small ? run_backward<64, float>(w, s) : run_backward<128, float>(w, s);
    return small ? run_backward<64, __nv_bfloat16>(w, s) : run_backward<128, __nv_bfloat16>(w, s);
}
