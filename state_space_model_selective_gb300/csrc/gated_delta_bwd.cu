// gated_delta_bwd.cu -- the gradient of the gated delta rule, from what the forward kept
// (gated_delta.cuh has the chunked form and its names).
//
// With L the adjoint of the state behind a chunk, per chunk, backwards:
//   z = P^T dY + H^T L,  dR = b z       (dR is also V's gradient)
//   L0 = e_63 L + Q^T (e dY) - K^T (e dR)
// is a chain two products deep again (chain_bwd_kernel, one head and 64 columns of headdim
// a CTA).  With z and L kept, everything else is one kernel over all chunks at once:
//   E = N R;  U = b E;  F = [dR; dY] S0^T;  F2 = U L^T;  [dA'; dP'] = [-dR; dY] U^T
//   dKK = dA' D (j < i),  dQK = dP' D (j <= i)          (beta cancels in dA A: dR = b T^T dU)
//   dQ = dQK K + e F_q;   dK = dKK K + dKK^T K + dQK^T Q - e F_k + w F2
//   dbeta_i = z_i . E_i
// z is the operand of F and dA'; b enters their rows afterwards.
//   dg_t = sum_{i >= t} dG_i + sum_{j < t} w_j k_j . F2_j + e_63 <L, S0>   (grads_kernel)
#include <algorithm>
#include <cstring>

#include "gated_delta.cuh"

namespace {

using namespace gdn;

__device__ __forceinline__ void put_gate(void* p, long long i, int bf16, float v) {
    if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
}
// ------------------------------------------------------------------ chain

constexpr int kRowWarps = 16;
constexpr int kChainThreads = 32 * (kRowWarps + 4);

template <int DK> struct ChainSmem {
    static constexpr uint32_t k_bytes = (DK / 64) * kTile;
    // a stage: gates, K panels, H hi | lo
    static constexpr uint32_t k = kGateBytes;
    static constexpr uint32_t h = k + k_bytes;
    static constexpr uint32_t stage = h + 2 * h_bytes(DK);
    static constexpr uint32_t q = 2 * stage;
    static constexpr uint32_t p = q + k_bytes;               // P hi | lo
    static constexpr uint32_t l_hi = p + 2 * kTile;          // L, rows of dstate
    static constexpr uint32_t l_lo = l_hi + h_bytes(DK);
    static constexpr uint32_t dy = l_lo + h_bytes(DK);       // dY, rows of steps
    static constexpr uint32_t o_hi = dy + kTile;             // e dY
    static constexpr uint32_t o_lo = o_hi + kTile;
    static constexpr uint32_t r_hi = o_lo + kTile;           // -e dR
    static constexpr uint32_t r_lo = r_hi + kTile;
    static constexpr uint32_t z = r_lo + kTile;              // z, on its way out
    static constexpr uint32_t xch = z + kTile;               // 64 x 64 fp32, columns first
    static constexpr uint32_t misc = xch + 64 * 64 * 4;
    static constexpr uint32_t bytes = misc + 512;
};

struct ChainArgs {
    const __nv_bfloat16* dy;
    const uint8_t* records;
    uint8_t* kept;          // z | dY | L
    const float* dlast;
    float* dh0;
    void* dv;
    uint32_t* status;
    Dims d;
};

// One head and 64 columns of headdim, backwards; laid out as the forward's chain.  H^T L and
// P^T dY have 64 rows, so both parts of the left operand go into the 128 rows of one
// instruction: rows 64 to 127 are their lo part, added through shared memory.  The warps on
// those rows also make dY and e dY of the chunk before, while the others work on z.  The
// factors come from bounds as the forward's do, with the largest values of L and dY measured.
// Bound as the forward's chain: 8 x 16 heads of 128 x 128, 32 chunks, 200 us, 3.1 us a chunk (3 % more
// with 8 warps on rows).
template <int DK, typename TG>
__global__ void __launch_bounds__(kChainThreads, 1)
    chain_bwd_kernel(const ChainArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using M = ChainSmem<DK>;
    constexpr int NP = DK / 64;
    constexpr int kMosts = kRowWarps + kRowWarps / 2;  // largest values of a chunk
    // tensor memory: P^T dY; hi and lo columns of H^T L, of Q^T e dY and of -K^T e dR
    constexpr uint32_t kTmP = 0, kTmX = 64, kTmQ = 192, kTmK = 320, kTmCols = 512;
    const uint32_t sb = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + M::misc);  // gates, K and H of a stage
    uint64_t* full_q = full + 2;
    uint64_t* full_p = full + 3;
    uint64_t* bar_x = full + 4;    // P^T dY and H^T L done
    uint64_t* bar_q = full + 5;    // Q^T e dY done
    uint64_t* bar_l = full + 6;    // K^T e dR done
    uint64_t* bar_s = full + 7;    // L is in shared memory
    uint64_t* bar_o = full + 8;    // dY and e dY are
    uint64_t* bar_r = full + 9;    // -e dR is
    uint64_t* bar_z = full + 10;   // z is
    uint32_t* s_most = reinterpret_cast<uint32_t*>(full + 12);  // [2 chunks][16 warps of L, 8 of dY]
    float* s_first = reinterpret_cast<float*>(s_most + 2 * kMosts);  // [16]: of the first L
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_first + kRowWarps);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pan = blockIdx.x % a.d.pans;
    const long long bh = blockIdx.x / a.d.pans;
    const int b = (int)(bh / a.d.heads), h = (int)(bh % a.d.heads);
    const int nc = a.d.chunks;
    const uint8_t* rec0 = a.records + bh * nc * rec_bytes(DK);

    if (warp == kRowWarps) tmem_alloc(s_tmem, kTmCols);
    if (tid == 0) {
        for (int i = 0; i < 7; ++i) mbar_init(full + i, i == 2 ? 2 : 1);
        mbar_init(bar_s, kRowWarps);
        mbar_init(bar_o, kRowWarps / 2);
        mbar_init(bar_r, kRowWarps / 2);
        mbar_init(bar_z, kRowWarps / 2);
        for (int n = 0; n < 2 * kMosts; ++n) s_most[n] = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp >= kRowWarps) {
        give_registers<kRowWarps>();
        if (warp == kRowWarps && lane == 0) {
            auto kept_of = [&](int it) {
                return a.kept + ((bh * nc + nc - 1 - it) * a.d.pans + pan) * adjoint_bytes(DK);
            };
            constexpr uint32_t id = idesc_f16(128, 128) | kIdescAMN | kIdescBMN;
            constexpr uint32_t id64 = idesc_f16(128, 64) | kIdescAMN | kIdescBMN;
            for (int it = 0; it < nc; ++it) {
                const uint32_t ph = it & 1, st = sb + (it & 1) * M::stage;
                bulk_wait_read_all();  // z's place is written again when H^T L is done
                if (!mbar_poll(full_p, ph, a.status)) break;
                if (!mbar_poll(bar_o, ph, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16(tmem + kTmP, mdesc(sb + M::p, kk, kTile), mdesc(sb + M::dy, kk, kTile),
                            id64, kk > 0);
                if (!mbar_poll(full + (it & 1), (it >> 1) & 1, a.status)) break;
                if (!mbar_poll(bar_s, ph, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    mma_f16(tmem + kTmX, mdesc(st + M::h, kk, h_bytes(DK)),
                            mdesc(sb + M::l_hi, kk, h_bytes(DK)), id, kk > 0);
                mma_commit(bar_x);
                // dY and L's hi part are kept as they are
                bulk_store(kept_of(it) + kTile, smem + M::dy, kTile);
                bulk_store(kept_of(it) + 2 * kTile, smem + M::l_hi, h_bytes(DK));
                bulk_commit();
                if (!mbar_poll(full_q, ph, a.status)) break;
                tc_fence_after();
                // (of 64 columns of dstate the second block of rows is not read)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16(tmem + kTmQ, mdesc(sb + M::q, kk, kTile), mdesc(sb + M::o_hi, kk, kTile), id, kk > 0);
                bulk_wait_read_all();  // dY's place is written when this is done, L's later
                mma_commit(bar_q);
                if (!mbar_poll(bar_r, ph, a.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16(tmem + kTmK, mdesc(st + M::k, kk, kTile), mdesc(sb + M::r_hi, kk, kTile), id, kk > 0);
                mma_commit(bar_l);
                if (!mbar_poll(bar_z, ph, a.status)) break;
                bulk_store(kept_of(it), smem + M::z, kTile);
                bulk_commit();
            }
            bulk_wait_all();
        } else if (warp == kRowWarps + 1 && lane == 0) {
            int kh_loads = 0, q_loads = 0, p_loads = 0;
            auto rec_of = [&](int it) { return rec0 + (long long)(nc - 1 - it) * rec_bytes(DK); };
            auto load_kh = [&](int it) {
                uint8_t* st = smem + (it & 1) * M::stage;
                uint64_t* bar = full + (it & 1);
                mbar_arrive_expect_tx(bar, M::stage);
                bulk_load(st, rec_of(it), kGateBytes, bar);
                for (int p = 0; p < NP; ++p)
                    bulk_load(st + M::k + p * kTile, rec_of(it) + rec_kq(DK) + p * 2 * kTile, kTile, bar);
                bulk_load(st + M::h, rec_of(it) + rec_h(DK), 2 * h_bytes(DK), bar);
                ++kh_loads;
            };
            auto load_q = [&](int it) {
                mbar_arrive_expect_tx(full_q, M::k_bytes);
                for (int p = 0; p < NP; ++p)
                    bulk_load(smem + M::q + p * kTile, rec_of(it) + rec_kq(DK) + p * 2 * kTile + kTile,
                              kTile, full_q);
                ++q_loads;
            };
            auto load_p = [&](int it) {
                mbar_arrive_expect_tx(full_p, 2 * kTile);
                bulk_load(smem + M::p, rec_of(it) + rec_p(DK), 2 * kTile, full_p);
                ++p_loads;
            };
            // Q counts as in once the chunk before is known to be done too, so that no barrier
            // is ever a whole turn ahead of this thread
            load_kh(0);
            load_p(0);
            load_q(0);
            mbar_arrive(full_q);
            if (nc > 1) load_kh(1);
            for (int it = 0; it + 1 < nc; ++it) {
                if (!mbar_wait(bar_q, it & 1, a.status)) break;  // (it follows bar_x)
                load_p(it + 1);
                load_q(it + 1);
                if (!mbar_wait(bar_l, it & 1, a.status)) break;
                mbar_arrive(full_q);
                if (it + 2 < nc) load_kh(it + 2);
            }
            // never leave with a load still landing
            for (int it = max(0, kh_loads - 2); it < kh_loads; ++it)
                (void)mbar_wait(full + (it & 1), (it >> 1) & 1, a.status);
            (void)mbar_wait(full_q, (q_loads - 1) & 1, a.status);
            (void)mbar_wait(full_p, (p_loads - 1) & 1, a.status);
        }
    } else {
        take_registers<kRowWarps>();
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + 16 * part;
        const int col0 = pan * kPan + 16 * part;
        const bool upper = row >= kC;   // these rows make dY and e dY
        const int i = row & 63;
        f2* xch = reinterpret_cast<f2*>(smem + M::xch) + 8 * part * 64 + i;
        f2 L[8];          // times its operand's factor; s_l undoes it
        float s_l = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float* at = a.dlast + (bh * a.d.dv + col0 + 2 * e) * a.d.dk + row;
            // (columns come in eights)
            const bool in = a.dlast && row < a.d.dk && col0 + 2 * e < a.d.dv;
            L[e] = pair(in ? at[0] : 0.0f, in ? at[a.d.dk] : 0.0f);
        }
        auto factors_of = [&](int c) {
            return reinterpret_cast<float*>(a.kept + ((bh * nc + c) * a.d.pans + pan) * adjoint_bytes(DK) +
                                            2 * kTile + h_bytes(DK));
        };
        // what a chunk's rows take from its gates, read before the stage can be refilled
        float e_row = 0.0f, e_end = 0.0f, e_max = 1.0f, s_k = 0.0f, s_h = 0.0f, s_p = 0.0f, h_e = 0.0f,
              p_e = 0.0f, own = 0.0f;  // own: of dY's rows Q's factor, of z's beta
        auto gates_of = [&](int it) {
            const bool in = warp_wait(full + (it & 1), (it >> 1) & 1, a.status);
            const Gates* g = reinterpret_cast<const Gates*>(smem + (it & 1) * M::stage);
            e_row = ex2_approx(g->hi[i] + g->lo[i]);
            e_end = ex2_approx(g->hi[kC - 1] + g->lo[kC - 1]);
            e_max = fmaxf(g->e_max, 1.0f);
            s_k = g->s_k;
            s_h = g->s_h;
            s_p = g->s_p;
            own = upper ? g->q_factor(i) : g->beta[i];
            h_e = g->h_e;
            p_e = g->p_e;
            return in;
        };
        auto put_state = [&](int it) {
            uint32_t hw[8], lw[8];
            if (row < DK) {
                split<8>(L, hw, lw);
                put_pieces<2>(smem + M::l_hi, row, 2 * part, hw);
                put_pieces<2>(smem + M::l_lo, row, 2 * part, lw);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(bar_s);
            const float m = warp_most<8>(L) * s_l;
            if (lane == 0) post_most(s_most + kMosts * (it & 1) + warp, m, it);
            if (tid == 0) factors_of(nc - 1 - it)[2] = s_l;
        };
        uint4 dy[2];
        auto fetch = [&](int c) {
            const int t = c * kC + i;
#pragma unroll
            for (int p = 0; p < 2; ++p)
                dy[p] = upper && t < a.d.seqlen && col0 + 8 * p < a.d.dv
                            ? *reinterpret_cast<const uint4*>(
                                  a.dy + (((long long)b * a.d.seqlen + t) * a.d.heads + h) * a.d.dv +
                                  col0 + 8 * p)
                            : make_uint4(0, 0, 0, 0);
        };
        // (upper warps) dY and e dY, times Q's factors, of step `it` as operands, dY kept
        auto put_dy = [&](int it, float e, float sq) {
            f2 x[8], y[8];
            MostBf16 seen;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                seen.see(dy[p]);
                unpack8_bf16(dy[p], x + 4 * p);
            }
            const float m = warp_most(seen.value() * sq);
            uint32_t* most = s_most + kMosts * (it & 1) + kRowWarps;
            if (lane == 0) post_most(most + (quarter & 1) * 4 + part, m, it);
            float all = 0.0f;
            const bool told = read_most<2>(most, it, all, a.status);
            float s_dy, s_o;
            uint32_t hw[8], lw[8];
            scaled<8>(x, finite_factor(sq * tile_scale(all, kTop, s_dy)), y);
            round_to<8>(y, hw);
            put_pieces<2>(smem + M::dy, i, 2 * part, hw);
            if (tid == 64) factors_of(nc - 1 - it)[1] = s_dy;
            scaled<8>(x, finite_factor(e * finite_factor(sq * tile_scale(all * e_max, kBoundTop, s_o))), x);
            split<8>(x, hw, lw);
            put_pieces<2>(smem + M::o_hi, i, 2 * part, hw);
            put_pieces<2>(smem + M::o_lo, i, 2 * part, lw);
            fence_proxy_async_smem();
            warp_arrive(bar_o);
            return told;
        };
        {   // the last chunk: its largest values are measured
            drop_infinities<8>(L);
            const float m = warp_most<8>(L);
            if (lane == 0) s_first[warp] = m;
            named_bar_sync(1, 32 * kRowWarps);
            scaled<8>(L, tile_scale(most_of<kRowWarps>(s_first), kBoundTop, s_l), L);
            put_state(0);
        }
        bool ok = gates_of(0);  // the same for all lanes of a warp
        fetch(nc - 1);
        if (upper) ok = put_dy(0, e_row, own) && ok;
        for (int it = 0; it < nc; ++it) {
            const int c = nc - 1 - it;
            const uint32_t ph = it & 1;
            const float er = e_row, ee = e_end, em = e_max, sk = s_k, sh = s_h, sp = s_p, br = own;
            if (c > 0) fetch(c - 1);
            f2 x[8];
            // bounds: of L and dY (times Q's factors) measured, of z, e dR and the next L from them
            float l_max = 0.0f, dy_max = 0.0f;
            ok = ok && read_most<4>(s_most + kMosts * ph, it, l_max, a.status) &&
                 read_most<2>(s_most + kMosts * ph + kRowWarps, it, dy_max, a.status);
            const float z_bound = kC * kTopValue * sp * 2.0f * dy_max + DK * kTopValue * sh * 2.0f * l_max;
            const float edr_bound = p_e * dy_max + h_e * (DK * l_max);
            float s_od, s_dyd, s_z, s_g, s_next;
            (void)tile_scale(dy_max * em, kBoundTop, s_od);  // (put_dy's factors)
            (void)tile_scale(dy_max, kTop, s_dyd);
            const float z_scale = tile_scale(z_bound, kBoundTop, s_z);
            const float g_scale = tile_scale(edr_bound, kBoundTop, s_g);
            const float next = tile_scale(fmaf(ee, l_max, kC * kTopValue * 2.0f *
                                                              (em * dy_max + sk * edr_bound)), kBoundTop, s_next);
            ok = ok && warp_wait(bar_x, ph, a.status);
            tc_fence_after();
            if (ok) {
                const f2 fp = pair(sp * s_dyd, sp * s_dyd), fx = pair(sh * s_l, sh * s_l);
                f2 z[8];
                tmem_ld16(t_lane + kTmP, x);
                tmem_ld16(t_lane + kTmX, z);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = fma2(fp, x[e], mul2(fx, z[e]));
                if (upper) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) xch[64 * e] = x[e];
                } else {
                    tmem_ld16(t_lane + kTmX + 64, z);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = fma2(fx, z[e], x[e]);
                }
            }
            tc_fence_before();
            if (!named_bar_and(1, 32 * kRowWarps, ok)) break;  // all warps on rows leave together
            if (!upper) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = add2(x[e], xch[64 * e]);
                uint32_t hw[8], lw[8];
                f2 y[8];
                scaled<8>(x, -finite_factor(er * br * g_scale), y);
                split<8>(y, hw, lw);
                put_pieces<2>(smem + M::r_hi, i, 2 * part, hw);
                put_pieces<2>(smem + M::r_lo, i, 2 * part, lw);
                fence_proxy_async_smem();
                warp_arrive(bar_r);
                scaled<8>(x, z_scale, y);
                round_to<8>(y, hw);
                put_pieces<2>(smem + M::z, i, 2 * part, hw);
                fence_proxy_async_smem();
                warp_arrive(bar_z);
                if (tid == 0) factors_of(c)[0] = s_z;
                scaled<8>(x, br, x);
                const int t = c * kC + i;
                if (t < a.d.seqlen) {
                    TG* dv = static_cast<TG*>(a.dv) +
                             (((long long)b * a.d.seqlen + t) * a.d.heads + h) * a.d.dv + col0;
                    store_row<8>(dv, x, col0, a.d.dv, rows_of_sectors(a.dv, a.d.dv));
                }
            }
            // ---- L0 = e_63 L + Q^T e dY - K^T e dR
            scaled<8>(L, ee * s_l * next, L);
            s_l = s_next;
            auto add = [&](uint32_t at, float factor) {
                // (with 64 rows, what is in the other lanes is no adjoint)
                if (DK == 64 && upper) return;
                const f2 f = pair(factor, factor);
                f2 z[8], y[8];
                tmem_ld16(t_lane + at, z);
                tmem_ld16(t_lane + at + 64, y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) L[e] = fma2(f, add2(z[e], y[e]), L[e]);
            };
            ok = warp_wait(bar_q, ph, a.status);
            tc_fence_after();
            if (ok) add(kTmQ, s_od * next);
            if (c > 0) {
                ok = gates_of(it + 1) && ok;
                // (the products that read dY and e dY are done: bar_q follows them)
                if (upper) ok = put_dy(it + 1, e_row, own) && ok;
            }
            ok = ok && warp_wait(bar_l, ph, a.status);
            tc_fence_after();
            if (ok) {
                add(kTmK, sk * s_g * next);
                if (c > 0) put_state(it + 1);
            }
        }
        if (a.dh0 && row < a.d.dk)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col0 + 2 * e < a.d.dv) {
                    float v0, v1;
                    unpair(L[e], v0, v1);
                    float* at = a.dh0 + (bh * a.d.dv + col0 + 2 * e) * a.d.dk + row;
                    at[0] = v0 * s_l;
                    at[a.d.dk] = v1 * s_l;
                }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kRowWarps) tmem_dealloc(tmem, kTmCols);
}

// ------------------------------------------------------------------ grads

// 8 warps on rows, one that loads, one that multiplies, two for the gates' gradients
constexpr int kGradThreads = kSplitThreads;
constexpr int kMaxPans = 4;

template <int DK> struct GradSmem {
    // of a head (two in turn): gates, panels of [K | Q], N (64 rows; the 64 behind them in its
    // operand are not read)
    static constexpr uint32_t kq = kGateBytes;
    static constexpr uint32_t nn = kq + kq_bytes(DK);
    static constexpr uint32_t head = nn + kTile;
    // of a head's 64 columns of headdim (two in turn): R, S0, then [z; dY], L
    static constexpr uint32_t r = 0;
    static constexpr uint32_t s0 = kTile;
    static constexpr uint32_t zdy = s0 + h_bytes(DK);
    static constexpr uint32_t l = zdy + 2 * kTile;
    static constexpr uint32_t stage = l + h_bytes(DK);
    static constexpr uint32_t stages = 2 * head;
    static constexpr uint32_t u = stages + 2 * stage;   // U, then W (rows 64 to 127 of U's
    static constexpr uint32_t w = u + kTile;            // operand are not read)
    static constexpr uint32_t sums = w + 2 * kTile;     // (W^T's second block, not read either)
    static constexpr uint32_t misc = sums + 4608;
    static constexpr uint32_t factors = misc + 256;     // [2 heads][4 panels][8] floats
    static constexpr uint32_t bytes = w + 3 * kTile;
    static_assert(factors + 256 <= bytes, "sums fit behind W");
};

struct GradArgs {
    const uint8_t* records;
    const uint8_t* kept;     // R | S0
    const uint8_t* adjoint;  // z | dY | L
    const void* g;
    void *dq, *dk, *dg, *dbeta;
    uint32_t* status;
    Dims d;
    unsigned count;          // of chunks and groups
    int splits, per;         // CTAs that share an item's heads (a cluster), and heads of one
    int gates_bf16;
    int fresh;               // there was no initial state
};

__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpair(v, a, b);
    return a + b;
}
// Products of a row's 16-byte pieces of two tiles, added to `s`.
__device__ __forceinline__ f2 dot8(uint4 a, uint4 b, f2 s) {
    f2 x[4], y[4];
    unpack8_f16(a, x);
    unpack8_f16(b, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fma2(x[e], y[e], s);
    return s;
}

// The exponent of a power of two, and back (0 for what is too small).
__device__ __forceinline__ int exponent(float v) { return (int)(__float_as_uint(v) >> 23) - 127; }
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)max(e + 127, 0) << 23); }
// U's products with L and those with z and dY have one U, whose factor follows L's: columns
// of headdim with this much less in L than others (with nothing, where no later step read
// them) are left out of F2, so that their U never loses bits (2^7 or so at most, on fp16's
// 2^-14 to 2^15).  Products below 2^kNone in all columns count as 0.
constexpr int kFar = -16, kNone = -110;

// All threads of a cluster's CTAs meet here, what they wrote to shared memory is seen.
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_address(uint32_t own, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(own), "r"(rank));
    return r;
}
__device__ __forceinline__ f2 cluster_load(uint32_t at) {
    f2 v;
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}

// What the warps on rows leave for those of a head's gates.
struct Sums {
    float dot[2 * kC][2];  // of what counts from step t on
    float end[kC][2];      // before step t
    float db[kC][2];
    float ls[8];           // <L, S0>
};

// The largest product of U's and L's factors over the panels of a head.
__device__ __forceinline__ int largest_ul(const float* fac, int pans) {
    int e = kNone;
    for (int p = 0; p < pans; ++p) e = max(e, exponent(fac[8 * p + 2]) + exponent(fac[8 * p + 6]));
    return e;
}

// CTAs walk the chunks and groups of heads; one warp brings in what comes next, one issues the
// products, E's of the next columns ahead of time.  Rows of products are lanes: steps as k
// rows (0 to 63) and as q rows (64 to 127).  All wait for one another by mbarriers, so that no
// step of one warp holds up the others' (242 us for 8 x 2048 steps of 16 heads when the warps on
// rows met at barriers and did the rest themselves, 217 us now).
//
// The gates' gradients need no sums over D's rows and columns: scaling k_i as it reads by
// e^{G_i}, as it writes by e^{-G_i} and q_i by e^{G_i} is what G does, so with dk split into
// what comes from reading (dKK K - e F_k) and from writing (dKK^T K + dQK^T Q + w F2)
//   dG_i = q_i . dq_i + k_i . dk_read,i - k_i . dk_write,i
// where the parts of w F2 also belong to the chunk's end: they count before step t instead
// of from it on.
template <int DK, typename TG>
__global__ void __launch_bounds__(kGradThreads, 1) grads_kernel(const GradArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using M = GradSmem<DK>;
    constexpr int CP = DK / 4;  // pairs of columns of dstate a thread holds
    // tensor memory: F, then W K; F2; [dA'; dP'], then W^T [K; Q]; E
    constexpr uint32_t kTmF = 0, kTmW = 0, kTmF2 = 128, kTmA = 256, kTmV = 256, kTmE = 384,
                       kTmCols = 512;
    const uint32_t sb = smem_u32(smem);
    Sums* sums = reinterpret_cast<Sums*>(smem + M::sums);             // [2 heads]
    uint32_t* s_most = reinterpret_cast<uint32_t*>(sums + 2);         // [2 heads][8 warps]: of W
    float* s_scan = reinterpret_cast<float*>(s_most + 16);            // [2]
    static_assert(2 * sizeof(Sums) + 72 <= M::misc - M::sums, "sums fit");
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + M::misc);  // [2] columns are in
    uint64_t* empty = full + 2;                                    // [2] and have been read
    uint64_t* full_h = full + 4;                                   // [2] a head is in
    uint64_t* empty_h = full + 6;                                  // [2]
    uint64_t* dots_in = full + 8;                                  // [2] a head's sums are there
    uint64_t* dots_out = full + 10;                                // [2]
    uint64_t* bar_e = full + 12;   // products done: E; F; A and F2; W's two
    uint64_t* bar_f = full + 13;
    uint64_t* bar_a = full + 14;
    uint64_t* bar_w = full + 15;
    uint64_t* u_in = full + 16;    // U is in shared memory, the last A has been read
    uint64_t* f_out = full + 17;   // F has been read
    uint64_t* w_in = full + 18;    // W is in shared memory
    uint64_t* w_out = full + 19;   // W's products and F2 have been read
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + 20);
    float* factors = reinterpret_cast<float*>(smem + M::factors);  // E, S0, U, E's to U's, z, dY, L

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned nc = a.d.chunks, groups = a.d.groups;
    const int ratio = a.d.heads / a.d.groups, pans = a.d.pans;
    // this CTA's items, and its heads of them
    const unsigned first = blockIdx.x / a.splits, step = gridDim.x / a.splits, rank = blockIdx.x % a.splits;
    const int head_lo = (int)rank * a.per, mine = min(a.per, ratio - head_lo);

    if (warp == 8) tmem_alloc(s_tmem, kTmCols);
    if (tid == 0) {
        for (int n = 0; n < 2; ++n) {
            mbar_init(full + n, 1);
            mbar_init(empty + n, 8);
            mbar_init(full_h + n, 1);
            mbar_init(empty_h + n, 10);
            mbar_init(dots_in + n, 8);
            mbar_init(dots_out + n, 2);
        }
        for (int n = 12; n < 16; ++n) mbar_init(full + n, 1);
        for (int n = 16; n < 20; ++n) mbar_init(full + n, 8);
        for (int n = 0; n < 16; ++n) s_most[n] = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp >= 8) {
        give_registers<8>();
        if (warp == 8 && lane == 0) {
            int n = 0, hn = 0;  // columns and heads loaded
            bool ok = true;
            for (unsigned item = first; item < a.count && ok; item += step) {
                const unsigned bg = item / nc, c = item - bg * nc;
                const unsigned b = bg / groups, head0 = b * a.d.heads + (bg - b * groups) * ratio + head_lo;
                for (int hh = 0; hh < mine && ok; ++hh, ++hn) {
                    const size_t ch = (size_t)(head0 + hh) * nc + c;
                    if (hn >= 2) ok = mbar_wait(empty_h + (hn & 1), ((hn >> 1) - 1) & 1, a.status);
                    if (!ok) break;
                    uint8_t* hd = smem + (hn & 1) * M::head;
                    uint64_t* bh = full_h + (hn & 1);
                    const uint8_t* rec = a.records + ch * rec_bytes(DK);
                    const uint8_t* kept0 = a.kept + ch * pans * kept_bytes(DK);
                    const uint8_t* adj0 = a.adjoint + ch * pans * adjoint_bytes(DK);
                    mbar_arrive_expect_tx(bh, M::head + 32 * pans);
                    bulk_load(hd, rec, kGateBytes + kq_bytes(DK), bh);
                    bulk_load(hd + M::nn, rec + rec_n(DK), kTile, bh);
                    for (int p = 0; p < pans; ++p) {
                        float* f = factors + 8 * (kMaxPans * (hn & 1) + p);
                        bulk_load(f, kept0 + p * kept_bytes(DK) + kTile + h_bytes(DK), 16, bh);
                        bulk_load(f + 4, adj0 + p * adjoint_bytes(DK) + 2 * kTile + h_bytes(DK), 16, bh);
                    }
                    for (int p = 0; p < pans; ++p, ++n) {
                        if (n >= 2) ok = mbar_wait(empty + (n & 1), ((n >> 1) - 1) & 1, a.status);
                        if (!ok) break;
                        uint8_t* st = smem + M::stages + (n & 1) * M::stage;
                        uint64_t* bar = full + (n & 1);
                        mbar_arrive_expect_tx(bar, M::stage);
                        bulk_load(st + M::r, kept0 + p * kept_bytes(DK), kTile + h_bytes(DK), bar);
                        bulk_load(st + M::zdy, adj0 + p * adjoint_bytes(DK), 2 * kTile + h_bytes(DK), bar);
                    }
                }
            }
            // never leave with a load still landing
            for (int k = max(0, n - 2); k < n; ++k) (void)mbar_wait(full + (k & 1), (k >> 1) & 1, a.status);
            for (int k = max(0, hn - 2); k < hn; ++k)
                (void)mbar_wait(full_h + (k & 1), (k >> 1) & 1, a.status);
        } else if (warp == 9) {
            const int one = elect_one();
            constexpr uint32_t id64 = idesc_f16(128, 64), idk = idesc_f16(128, DK);
            constexpr uint32_t idW = idesc_f16(128, DK) | kIdescBMN;
            constexpr uint32_t idV = idesc_f16(128, DK) | kIdescAMN | kIdescBMN;
            // E = N R
            auto multiply_e = [&](int n, int hn) {
                if (!warp_wait(full + (n & 1), (n >> 1) & 1, a.status)) return false;
                const uint32_t st = sb + M::stages + (n & 1) * M::stage, hd = sb + (hn & 1) * M::head;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16_warp(one, tmem + kTmE, kdesc<128>(hd + M::nn, kk), mdesc(st + M::r, kk, kTile), id64 | kIdescBMN,
                            kk > 0);
                if (one) mma_commit(bar_e);
                return true;
            };
            // F = [z; dY] S0^T, of columns that are in
            auto multiply_f = [&](int n) {
                const uint32_t st = sb + M::stages + (n & 1) * M::stage;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16_warp(one, tmem + kTmF, kdesc<128>(st + M::zdy, kk), kdesc<DK>(st + M::s0, kk), idk, kk > 0);
                if (one) mma_commit(bar_f);
                return true;
            };
            const int heads = first < a.count ? (int)((a.count - 1 - first) / step + 1) * mine : 0;
            bool ok = heads > 0 && warp_wait(full_h, 0, a.status) && multiply_e(0, 0) && multiply_f(0);
            for (int hn = 0, n = 0; hn < heads && ok; ++hn) {
                const float* fac = factors + 8 * kMaxPans * (hn & 1);
                const uint32_t hd = sb + (hn & 1) * M::head;
                const int e_ul = largest_ul(fac, pans);
                bool begun = false;  // F2
                for (int p = 0; p < pans && ok; ++p, ++n) {
                    const uint32_t st = sb + M::stages + (n & 1) * M::stage;
                    const bool near = exponent(fac[8 * p + 2]) + exponent(fac[8 * p + 6]) - e_ul >= kFar || e_ul == kNone;
                    ok = warp_wait(u_in, n & 1, a.status);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16_warp(one, tmem + kTmA, kdesc<128>(st + M::zdy, kk), kdesc<64>(sb + M::u, kk), id64, kk > 0);
                    if (near) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16_warp(one, tmem + kTmF2, kdesc<128>(sb + M::u, kk), kdesc<DK>(st + M::l, kk), idk,
                                    begun || kk > 0);
                        begun = true;
                    }
                    if (one) mma_commit(bar_a);
                    if (p + 1 < pans)
                        ok = multiply_e(n + 1, hn) && warp_wait(f_out, n & 1, a.status) && multiply_f(n + 1);
                }
                ok = ok && warp_wait(w_in, hn & 1, a.status);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16_warp(one, tmem + kTmW, kdesc<128>(sb + M::w, kk), mdesc(hd + M::kq, kk, 2 * kTile), idW, kk > 0);
                // (rows 64 to 127 of W^T [K; Q] are not read)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_f16_warp(one, tmem + kTmV, mdesc(sb + M::w, kk, kTile), mdesc(hd + M::kq, kk, 2 * kTile), idV, kk > 0);
                if (one) mma_commit(bar_w);
                if (hn + 1 < heads)
                    ok = warp_wait(full_h + ((hn + 1) & 1), ((hn + 1) >> 1) & 1, a.status) &&
                         multiply_e(n, hn + 1) && warp_wait(w_out, hn & 1, a.status) && multiply_f(n);
            }
        } else if (warp >= 10) {
            // ---- the gates: step i
            const int i = tid - 10 * 32;
            int hn = 0;
            bool ok = true;
            for (unsigned item = first; item < a.count && ok; item += step) {
                const unsigned bg = item / nc;
                const int t = (int)(item - bg * nc) * kC + i;
                const int b = (int)(bg / groups), group = (int)(bg - b * groups);
                const bool in = t < a.d.seqlen;
                for (int hh = 0; hh < mine && ok; ++hh, ++hn) {
                    const long long at = ((long long)b * a.d.seqlen + t) * a.d.heads + group * ratio + head_lo + hh;
                    const float g = in ? gate_at(a.g, at, a.gates_bf16) : 0.0f;
                    const Gates* gates = reinterpret_cast<const Gates*>(smem + (hn & 1) * M::head);
                    const Sums& s = sums[hn & 1];
                    ok = warp_wait(full_h + (hn & 1), (hn >> 1) & 1, a.status) &&
                         warp_wait(dots_in + (hn & 1), (hn >> 1) & 1, a.status);
                    ok = named_bar_and(2, 64, ok);
                    if (!ok) break;
                    float up = s.dot[i][0] + s.dot[i][1] + s.dot[kC + i][0] + s.dot[kC + i][1];
                    float down = s.end[i][0] + s.end[i][1];
                    const float self = down, db = s.db[i][0] + s.db[i][1];
                    float all = 0.0f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) all += s.ls[q];
                    const float e_end = ex2_approx(gates->hi[kC - 1] + gates->lo[kC - 1]);
                    const bool off = gates->masked >> i & 1;
                    // sums of `up` from here on, of `down` before here
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float u = __shfl_down_sync(0xffffffffu, up, o);
                        const float d = __shfl_up_sync(0xffffffffu, down, o);
                        if (lane + o < 32) up += u;
                        if (lane >= o) down += d;
                    }
                    if (i == 32) s_scan[0] = up;
                    if (i == 31) s_scan[1] = down;
                    warp_arrive(dots_out + (hn & 1));
                    warp_arrive(empty_h + (hn & 1));
                    named_bar_sync(2, 64);
                    if (warp == 10) up += s_scan[0];
                    else down += s_scan[1];
                    if (in) {
                        // a gate of -inf cuts the past off, and a first one without a state has
                        // none: their gradients are 0
                        const bool cut = ex2_approx(g * kLog2e) == 0.0f || (t == 0 && a.fresh);
                        put_gate(a.dg, at, a.gates_bf16, cut ? 0.0f : up + (down - self) + e_end * all);
                        put_gate(a.dbeta, at, a.gates_bf16, off ? 0.0f : db);
                    }
                }
            }
        }
        if (a.splits > 1) {  // (as the warps on rows do)
            __syncwarp();
            cluster_meet();
            cluster_meet();
        }
    } else {
        take_registers<8>();
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const bool is_q = row >= kC;
        const int i = row & 63, col0 = (DK / 2) * part;  // first column of dstate
        int n = 0, hn = 0;
        bool ok = true;
        for (unsigned item = first; item < a.count && ok; item += step) {
            const unsigned bg = item / nc;
            const int c = (int)(item - bg * nc), t0 = c * kC;
            const int b = (int)(bg / groups), group = (int)(bg - b * groups);
            f2 acc[CP];  // of dK (rows 0 to 63) or dQ, summed over heads
#pragma unroll
            for (int e = 0; e < CP; ++e) acc[e] = 0;
            for (int hh = 0; hh < mine; ++hh, ++hn) {
                const uint32_t hd = sb + (hn & 1) * M::head;
                const uint8_t* hg = smem + (hn & 1) * M::head;
                const Gates* gates = reinterpret_cast<const Gates*>(hg);
                const float* fac = factors + 8 * kMaxPans * (hn & 1);
                bool here = warp_wait(full_h + (hn & 1), (hn >> 1) & 1, a.status);
                // dY's rows are kept times Q's factors (powers of two): what undoes it
                const float inv_q = inverse(gates->q_factor(i));
                // of this row in F and in A: as a q row for dY, as a k row for -dR = -b z
                const float er = ex2_approx(gates->hi[i] + gates->lo[i]);
                const float f_row = is_q ? er * inv_q : -er * gates->beta[i];
                const float a_row = is_q ? 1.0f : -gates->beta[i] * gates->s_k;
                // a step's row of K or Q, columns col0 + 16 n .. + 15
                auto own_row = [&](int n16, f2* v) {
                    const int c0 = col0 + 16 * n16;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        unpack8_f16(*reinterpret_cast<const uint4*>(
                                        hg + M::kq + (c0 >> 6) * 2 * kTile + piece(row, ((c0 & 63) >> 3) + q)),
                                    v + 4 * q);
                };
                // Products of U and L are summed over the panels where they are: U's factor is
                // chosen so that all have the same, the largest of theirs
                const int e_ul = largest_ul(fac, pans);
                // what the other heads have left in the sums does not belong to this one's dot
                float before = 0.0f;
                if (hh > 0) {
                    f2 d = 0;
#pragma unroll
                    for (int n16 = 0; n16 < CP / 8; ++n16) {
                        f2 v[8];
                        own_row(n16, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) d = fma2(v[e], acc[8 * n16 + e], d);
                    }
                    before = sum2(d);
                }
                f2 own[16];  // of [dA'; dP']
#pragma unroll
                for (int e = 0; e < 16; ++e) own[e] = 0;
                float beta_sum = 0.0f, ls = 0.0f;
                for (int p = 0; p < pans; ++p, ++n) {
                    const uint8_t* sg = smem + M::stages + (n & 1) * M::stage;
                    const float s_s = fac[8 * p + 1], s_row = fac[8 * p + (is_q ? 5 : 4)], s_l = fac[8 * p + 6];
                    here = warp_wait(full + (n & 1), (n >> 1) & 1, a.status) && here;
                    const int below = max(exponent(fac[8 * p + 2]) + exponent(s_l) - e_ul, kFar);
                    f2 e_row[16];
                    if (!is_q) {
                        here = warp_wait(bar_e, n & 1, a.status) && here;
                        tc_fence_after();
                        f2 x[16];
                        uint32_t hw[16];
                        tmem_ld32(t_lane + kTmE + 32 * part, e_row);
                        tmem_wait_ld();
                        scaled<16>(e_row, fac[8 * p + 3] * power(below) * gates->beta[i], x);
                        round_to<16>(x, hw);
                        put32(smem + M::u, i, 4 * part, hw);
                        fence_proxy_async_smem();
                        tc_fence_before();
                    } else {
                        tc_fence_before();
                    }
                    if (here) warp_arrive(u_in);
                    // sums over these columns: z . E, and L . S0
                    {
                        f2 ze = 0, dl = 0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t at = piece(row, 4 * part + q);
                            if (!is_q) {
                                f2 z[4];
                                unpack8_f16(*reinterpret_cast<const uint4*>(sg + M::zdy + at), z);
#pragma unroll
                                for (int e = 0; e < 4; ++e) ze = fma2(z[e], e_row[4 * q + e], ze);
                            }
                            if (row < DK)
                                dl = dot8(*reinterpret_cast<const uint4*>(sg + M::s0 + at),
                                          *reinterpret_cast<const uint4*>(sg + M::l + at), dl);
                        }
                        beta_sum = fmaf(s_row * fac[8 * p], sum2(ze), beta_sum);
                        ls = fmaf(s_s * s_l, sum2(dl), ls);
                    }
                    ok = here && warp_wait(bar_f, n & 1, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    {
                        const float f1 = f_row * s_row * s_s;
                        const f2 f1p = pair(f1, f1);
#pragma unroll
                        for (int e0 = 0; e0 < CP; e0 += 16) {
                            f2 f[16];
                            tmem_ld32(t_lane + kTmF + col0 + 2 * e0, f);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) acc[e0 + e] = fma2(f1p, f[e], acc[e0 + e]);
                        }
                        tc_fence_before();
                        warp_arrive(f_out);
                    }
                    ok = warp_wait(bar_a, n & 1, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    {
                        const float fa = a_row * s_row * (fac[8 * p + 2] * power(-below));
                        const f2 fap = pair(fa, fa);
                        f2 x[16];
                        tmem_ld32(t_lane + kTmA + 32 * part, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) own[e] = fma2(fap, x[e], own[e]);
                    }
                    warp_arrive(empty + (n & 1));  // these columns have been read
                }
                if (!ok) break;

                // ---- W = [dKK; dQK], rows times K's and Q's factors: as W^T [K; Q] needs them
                {
                    const float hi = -gates->hi[i], lo = -gates->lo[i];
                    const f2 mh = pair(hi, hi), ml = pair(lo, lo);
                    const int last = is_q ? i : i - 1;
                    if (part == 1 && (quarter & 1) == 0) {  // rows to 31, columns from 32
#pragma unroll
                        for (int e = 0; e < 16; ++e) own[e] = 0;
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const int j = 32 * part + 2 * e;
                            float d[4];
                            decays4(gates, j, mh, ml, last, d);
                            own[e] = mul2(own[e], pair(d[0], d[1]));
                            own[e + 1] = mul2(own[e + 1], pair(d[2], d[3]));
                        }
                    }
                    const float most = warp_most_or_nan<16>(own);
                    if (lane == 0) post_most(s_most + 8 * (hn & 1) + warp, most, hn);
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
                float s_w, w_most;
                ok = read_most<2>(s_most + 8 * (hn & 1), hn, w_most, a.status);
                if (!ok) break;
                scaled<16>(own, tile_scale(w_most, kTop, s_w), own);
                {
                    uint32_t hw[16];
                    round_to<16>(own, hw);
                    put32(smem + M::w, row, 4 * part, hw);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(w_in);
                Sums& s = sums[hn & 1];
                ok = (hn < 2 || warp_wait(dots_out + (hn & 1), ((hn >> 1) - 1) & 1, a.status)) &&
                     warp_wait(bar_w, hn & 1, a.status);
                if (!ok) break;
                tc_fence_after();
                {
                    const float wr = decay(gates->hi[kC - 1], gates->lo[kC - 1], gates->hi[i], gates->lo[i]);
                    const float f1 = is_q ? s_w * (gates->s_k * inv_q) : s_w;
                    const float g2 = e_ul > kNone ? wr * power(min(e_ul, 127)) : 0.0f;
                    const f2 f1p = pair(f1, f1), g2p = pair(g2, g2);
                    f2 whole = 0, end = 0, write = 0;  // dots with this row
#pragma unroll
                    for (int n16 = 0; n16 < CP / 8; ++n16) {
                        f2 v[8], f[8];
                        tmem_ld16(t_lane + kTmW + col0 + 16 * n16, f);
                        own_row(n16, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[8 * n16 + e] = fma2(f1p, f[e], acc[8 * n16 + e]);
                        if (!is_q) {
                            tmem_ld16(t_lane + kTmV + col0 + 16 * n16, f);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                write = fma2(v[e], f[e], write);
                                acc[8 * n16 + e] = fma2(f1p, f[e], acc[8 * n16 + e]);
                            }
                            tmem_ld16(t_lane + kTmF2 + col0 + 16 * n16, f);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                end = fma2(v[e], f[e], end);
                                acc[8 * n16 + e] = fma2(g2p, f[e], acc[8 * n16 + e]);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) whole = fma2(v[e], acc[8 * n16 + e], whole);
                    }
                    const float s_row = is_q ? gates->q_factor(i) : gates->s_k;
                    const float own_dot = s_row * (sum2(whole) - before);
                    const float wv = s_row * f1 * sum2(write), we = s_row * g2 * sum2(end);
                    s.dot[row][part] = is_q ? own_dot : own_dot - 2.0f * wv - we;
                    if (!is_q) {
                        s.end[i][part] = we;
                        s.db[i][part] = beta_sum;
                    }
                    if (lane == 0) s.ls[warp] = ls;
                }
                tc_fence_before();
                warp_arrive(w_out);
                warp_arrive(dots_in + (hn & 1));
                warp_arrive(empty_h + (hn & 1));
            }
            // With few items the CTAs of a cluster have some heads each of one, the only one they
            // have: the first adds the others' sums to its own, from where the columns were (all
            // of them have been read)
            if (a.splits > 1) {
                f2* left = reinterpret_cast<f2*>(smem + M::stages) + tid;
                static_assert(CP * 256 * 8 <= 2 * M::stage, "sums fit");
                named_bar_sync(1, 256);  // no warp on rows reads columns any more
                if (rank > 0)
#pragma unroll
                    for (int e = 0; e < CP; ++e) left[e * 256] = acc[e];
                cluster_meet();
                if (rank == 0)
                    for (int r = 1; r < a.splits; ++r) {
                        const uint32_t there = cluster_address(smem_u32(left), r);
#pragma unroll
                        for (int e = 0; e < CP; ++e) acc[e] = add2(acc[e], cluster_load(there + e * 256 * 8));
                    }
                cluster_meet();  // (the others' memory has been read)
                if (rank > 0) break;
            }
            if (ok && t0 + i < a.d.seqlen) {
                void* base = is_q ? a.dq : a.dk;
                TG* out = static_cast<TG*>(base) +
                          (((long long)b * a.d.seqlen + t0 + i) * a.d.groups + group) * a.d.dk + col0;
                store_row<CP>(out, acc, col0, a.d.dk, rows_of_sectors(base, a.d.dk));
            }
        }
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

template <int DK, typename TG>
ssm_status_t run_backward(const ChainArgs& chain, GradArgs grads, cudaStream_t s) {
    const Dims& d = chain.d;
    const int sms = ssm_host::sm_count();
    if (sms == 0 || !allow_smem(chain_bwd_kernel<DK, TG>, ChainSmem<DK>::bytes) ||
        !allow_smem(grads_kernel<DK, TG>, GradSmem<DK>::bytes))
        return SSM_ERR_CUDA;
    chain_bwd_kernel<DK, TG><<<(unsigned)((long long)d.batch * d.heads * d.pans), kChainThreads,
                               ChainSmem<DK>::bytes, s>>>(chain);
    grads.count = (unsigned)((long long)d.batch * d.groups * d.chunks);
    // CTAs walk the items with all their heads, or up to 8 share one item's (each then has just the
    // one): whichever takes fewer rounds of heads, with half a head's time for the start and the
    // sum.  (The whole gradient, unshared and shared: one chunk of 21 heads 144 and 44 us, 8 chunks of
    // 24 heads in 3 groups 75 and 46 us.)
    const int ratio = d.heads / d.groups;
    auto rounds = [&](long long ctas) { return (ctas + sms - 1) / sms; };
    long long best = rounds(grads.count) * ratio * 2;
    grads.per = ratio;
    for (int n = 2; n <= std::min(ratio, 8); ++n) {
        const int per = (ratio + n - 1) / n, used = (ratio + per - 1) / per;
        const long long cost = rounds((long long)grads.count * used) * (per * 2 + 1);
        if (cost < best) {
            best = cost;
            grads.per = per;
        }
    }
    grads.splits = (ratio + grads.per - 1) / grads.per;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(grads.splits > 1 ? grads.count * grads.splits : std::min<unsigned>(grads.count, sms));
    config.blockDim = dim3(kGradThreads);
    config.dynamicSmemBytes = GradSmem<DK>::bytes;
    config.stream = s;
    cudaLaunchAttribute cluster[1];
    cluster[0].id = cudaLaunchAttributeClusterDimension;
    cluster[0].val.clusterDim = {(unsigned)grads.splits, 1, 1};
    config.attrs = cluster;
    config.numAttrs = grads.splits > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&config, grads_kernel<DK, TG>, grads) != cudaSuccess) return SSM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

}  // namespace

extern "C" size_t ssm_gated_delta_bwd_workspace_bytes(int batch, int seqlen, int nheads, int dstate,
                                                      int headdim) {
    using namespace gdn_host;
    if (!sizes_ok(batch, seqlen, nheads, nheads, dstate, headdim) ||
        !sizes_fit(batch, seqlen, nheads, dstate, headdim))
        return 0;
    return 1024 + adjoints_bytes(batch, seqlen, nheads, dstate, headdim);
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
    const Dims d{batch, seqlen, nheads, ngroups, dstate, headdim, (seqlen + kC - 1) / kC,
                 (headdim + kPan - 1) / kPan};
    ChainArgs c{};
    c.dy = static_cast<const __nv_bfloat16*>(dy);
    c.records = records; c.kept = ws + 1024; c.dlast = dfinal_state; c.dh0 = dinitial_state;
    c.dv = dv; c.status = status; c.d = d;
    GradArgs w{};
    w.records = records; w.kept = records + rb; w.adjoint = ws + 1024; w.g = g;
    w.dq = dq; w.dk = dk; w.dg = dg; w.dbeta = dbeta; w.status = status; w.d = d;
    w.gates_bf16 = gate_dtype == SSM_BF16;
    w.fresh = !initial_state;
    const bool small = gdn_host::dk_tile(dstate) == 64;
    if (grad_dtype == SSM_F32) return small ? run_backward<64, float>(c, w, s) : run_backward<128, float>(c, w, s);
    return small ? run_backward<64, __nv_bfloat16>(c, w, s) : run_backward<128, __nv_bfloat16>(c, w, s);
}
