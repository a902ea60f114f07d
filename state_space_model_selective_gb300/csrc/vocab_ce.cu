// vocab_ce.cu -- softmax cross entropy of the logits h W^T over a large
// vocabulary, without the logits in memory: loss, and gradient.
//
//   l = h W^T,  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_t,target
//   P_tv = (exp(l_tv - lse_t) - [v = target_t]) dloss_t
//   dh = P W,  dW = P^T h
//
// The logits are sums of the tensor cores' fp32 accumulators, which truncate instead of
// rounding: lse and loss are 0.4 to 1.2e-6 off (2-norm, dim 1536 to 2048), against 1e-7 for
// sums that round.  Two accumulators of half the depth would halve that, but there is room
// for two, and the second one is what the epilogue of the tile before runs beside.
//
// Bound by the tensor cores: 2 tokens dim vocab multiply-adds a product, one
// product for the loss and three for the gradient (the logits are computed
// again, since the softmax needs the whole row's lse first).
//
// All four products run in one tcgen05 pipeline.  A cluster of two CTAs computes
// 256 x 256 tiles (cta_group::2: each CTA holds 128 rows of A, 128 of B and the
// 128 x 256 half of the accumulator that belongs to its rows of A), because a
// pair loads 32 KB per CTA for what a single CTA's 128 x 256 tile needs 48 KB
// for, and the loads go through L2.  Per CTA: one thread issues TMA loads into
// a ring of six 64-deep stages, one thread of the first CTA issues the MMAs, and
// eight warps empty the accumulators, of which there are two, so that a tile's
// epilogue runs under the next tile's products.
//  * logits, K-major h and W: the epilogue keeps each row's maximum and sum of
//    exponentials of its 128 columns (fp32, base 2), and the target's logit; a
//    small kernel joins them.
//  * gradient, for a piece of the vocabulary at a time: the logits again, with
//    P / max |dloss| as the epilogue, rounded to bf16, which the tensor cores'
//    operands have to be, then dh += P W and dW = P^T h in one launch, where W, h
//    and P are read as MN-major operands.  The rounding is at most 2^-9 of each
//    value and independent from value to value, so the products' sums keep it
//    below 2^-9 (in an fp32 result too: a second bf16 term of P would cost both
//    products again); without the division by the largest dloss the targets' entries
//    of a mean loss, which outweigh the rest, would all be off by the same
//    rounding of 1 / n (0.25 % of the gradients at 1986 tokens, against 0.17 % for
//    rounding the result to bf16).  The factor comes back in fp32 in dW's
//    epilogue and dh's last sum.
// The sum over pieces and over splits of one piece's vocabulary is kept in fp32
// and taken in a fixed order: runs are bit-equal.
#include <algorithm>

#include "tcgen05.cuh"

namespace {

using namespace ssm;

constexpr int kTile = 256;               // rows and columns of a pair's tile
constexpr int kHalf = 128;               // rows of A and of B one CTA holds
constexpr int kDepth = 64;               // K of one stage: 128 bytes of bf16
constexpr int kStages = 6;
constexpr uint32_t kBox = 64 * 128;      // a 64 x 64 box of bf16
constexpr uint32_t kOperand = 2 * kBox;  // 128 x 64
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr int kEpiWarps = 8;
constexpr uint32_t kOutBox = 32 * 128;   // a warp's 32 rows by 128 bytes on their way out
constexpr uint32_t kSmemBytes = kStages * kStageBytes + kEpiWarps * kOutBox + 1024;
constexpr int kThreads = (kEpiWarps + 2) * 32;  // + TMA warp, MMA warp
constexpr uint32_t kTmemCols = 512;             // two accumulators of 256 columns
constexpr int kEpilogue = 6;  // stages in whose time a tile's epilogue runs (2 us)
constexpr int kGroupM = 32;  // token tiles whose h stays in L2 while W passes

enum Mode { kLoss, kProb, kGrad };

struct CeHeader {
    uint32_t unused;
    uint32_t status;
    float scale;  // gradient: max |dloss| of the tokens that count
    uint32_t pad[61];
};
static_assert(sizeof(CeHeader) == 256, "workspace header is 256 bytes");

struct CeArgs {
    int tokens, dim, vocab;
    uint32_t* status;
    const long long* targets;
    // loss
    uint32_t* failed;    // [CTAs]: whether a wait ran out
    float2* parts;       // [2 * vocab tiles][tokens]: maximum (base 2), sum
    float* target_logit; // [tokens]
    // gradient
    const float* lse;
    const float* dloss;
    const float* scale;  // in the header
    __nv_bfloat16* P;    // [tokens][ld], columns v0 .. v0 + width of the vocabulary
    int ld, v0, width;   // width: what is left of the vocabulary, at most ld
    float* dh_parts;     // [splits][tokens][dim]
    int first_piece, splits, split_depth;  // stages of one split's K
    void* dW;
    int dw_bf16;
};

// ------------------------------------------------- pairs of CTAs (cta_group::2)

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// the address of the first CTA's copy of a shared variable
__device__ __forceinline__ uint32_t first_cta(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void arrive_remote(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
                 : "memory");
}

// mbar_wait, acquiring what the other CTA's arrivals released
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint32_t* status) {
    const uint32_t addr = smem_u32(bar);
    for (uint32_t i = 0; i < kMbarSpinLimit; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity), "r"(1000u)
            : "memory");
        if (done) return true;
    }
    record_status(status, SSM_ERR_TIMEOUT);
    return false;
}

// a box into this CTA's shared memory, its bytes counted on the first CTA's barrier
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                         int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
        "bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// arrive on both CTAs' copies of `bar` once the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// ------------------------------------------------------------------ work

// One tile of one product: operand origins, K range, and what it is for.
struct Item {
    bool dw;         // kGrad: dW's tile, else dh's
    int m0, n0;      // rows and columns of the result
    int k0, depth;   // first K, stages
    int split;
};

// The pair's items, in order.  Loss and P: tiles round-robin, token tiles fastest
// within groups of kGroupM, so that W passes once per group.  Gradient: dh's
// (few, deep) tiles round-robin first; the pairs that have one less of them take
// dW tiles for that time, then all take the rest in turn, so that at any time
// the pairs work on neighbouring tiles and share them in L2.
template <Mode MODE>
struct Schedule {
    int pairs, pair;
    int mt, nt;                  // tiles of tokens, and of vocabulary (kGrad: of dim)
    int n_dh, n_dw, dh_depth, dw_depth;
    int own_dh, free_pairs, early, n_early;

    __device__ Schedule(const CeArgs& a, int pairs_, int pair_) : pairs(pairs_), pair(pair_) {
        mt = (a.tokens + kTile - 1) / kTile;
        if constexpr (MODE == kGrad) {
            nt = (a.dim + kTile - 1) / kTile;
            n_dh = mt * nt * a.splits;
            n_dw = (a.width + kTile - 1) / kTile * nt;
            dh_depth = a.split_depth;
            dw_depth = (a.tokens + kDepth - 1) / kDepth;
            const int rest = n_dh % pairs;
            own_dh = n_dh / pairs + (pair < rest ? 1 : 0);
            free_pairs = rest ? pairs - rest : 0;
            // dW tiles in the time of one of dh: a tile takes its products' time or its
            // epilogue's
            const int dw_cost = max(dw_depth, kEpilogue);
            early = (max(dh_depth, kEpilogue) + dw_cost / 2) / dw_cost;
            n_early = (int)min((long long)n_dw, (long long)early * free_pairs);
        } else {
            nt = ((MODE == kProb ? a.width : a.vocab) + kTile - 1) / kTile;
        }
    }

    __device__ bool get(const CeArgs& a, int i, Item& w) const {
        if constexpr (MODE != kGrad) {
            const long long t = (long long)i * pairs + pair;
            if (t >= (long long)mt * nt) return false;
            const int group = (int)(t / ((long long)kGroupM * nt));
            const int gm = min(kGroupM, mt - group * kGroupM);
            const int r = (int)(t - (long long)group * kGroupM * nt);
            w.m0 = (group * kGroupM + r % gm) * kTile;
            w.n0 = r / gm * kTile;
            w.k0 = 0;
            w.depth = (a.dim + kDepth - 1) / kDepth;
            w.dw = false;
            w.split = 0;
            return true;
        } else {
            if (i < own_dh) {
                const int t = i * pairs + pair;
                w.dw = false;
                w.split = t / (mt * nt);
                const int r = t % (mt * nt);
                w.m0 = r / nt * kTile;
                w.n0 = r % nt * kTile;
                const int all = (a.width + kDepth - 1) / kDepth;
                w.k0 = w.split * dh_depth * kDepth;
                w.depth = min(dh_depth, all - w.split * dh_depth);
                return true;
            }
            i -= own_dh;
            int t;
            const bool is_free = free_pairs && pair >= pairs - free_pairs;
            if (is_free) {
                const int me = pair - (pairs - free_pairs);
                const int mine = (n_early - me + free_pairs - 1) / free_pairs;
                if (i < mine) {
                    t = i * free_pairs + me;
                } else {
                    t = n_early + (i - mine) * pairs + pair;
                }
            } else {
                t = n_early + i * pairs + pair;
            }
            if (t >= n_dw) return false;
            w.dw = true;
            w.split = 0;
            w.m0 = t / nt * kTile;
            w.n0 = t % nt * kTile;
            w.k0 = 0;
            w.depth = dw_depth;
            return true;
        }
    }
};

// -------------------------------------------------------------- epilogues

// maximum and sum of 2^(l - maximum) of a row's columns so far, base 2
struct RowSum {
    float m, s;
    __device__ void add(const float* v, int n) {
        float cm = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < n) cm = fmaxf(cm, v[j]);
        cm = fmaxf(m, cm * kLog2e);
        const float base = cm == -INFINITY ? 0.0f : cm;
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < n) t += ex2_approx(fmaf(v[j], kLog2e, -base));
        s = fmaf(s, ex2_approx(m - base), t);
        m = cm;
    }
};

// v[at], as 32 selections: indexed, the array would live in local memory, written
// for every tile
__device__ __forceinline__ float pick(const float* v, int at) {
    float l = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.eq.s32 p, %1, %2;\n\t"
            "selp.f32 %0, %3, %0, p;\n\t}"
            : "+f"(l)
            : "r"(at), "r"(j), "f"(v[j]));
    return l;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A warp's 32 rows (one to a lane) go out 128 bytes of each at a time: into shared
// memory in the 128-byte swizzle (16-byte pieces XORed with row mod 8), from there by
// TMA, which clips them at the tensor's end.  (Rows written by their lanes, 16 bytes at
// 32 places at a time, made loss and gradient of 8 tokens take 446 us, against 242 us.)
struct OutBox {
    uint32_t smem;  // the warp's 4 KB
    int lane;

    __device__ void ready() const {  // the last box has been read out
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
    }
    __device__ void put(int piece, uint4 w) const {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         smem + lane * 128 + ((piece ^ (lane & 7)) << 4)),
                     "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                     : "memory");
    }
    __device__ void put_bf16(int piece0, const float* v) const {  // 32 values
#pragma unroll
        for (int j = 0; j < 4; ++j)
            put(piece0 + j, make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]),
                                       pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                                       pack_bf16(v[8 * j + 4], v[8 * j + 5]),
                                       pack_bf16(v[8 * j + 6], v[8 * j + 7])));
    }
    __device__ void put_f32(const float* v) const {  // 32 values
#pragma unroll
        for (int j = 0; j < 8; ++j)
            put(j, make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                              __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
    }
    __device__ void send(const CUtensorMap* map, int c0, int c1) const {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                    reinterpret_cast<uint64_t>(map)),
                "r"(smem), "r"(c0), "r"(c1)
                : "memory");
            bulk_commit();
        }
    }
    // ADD: onto what is there, in fp32
    template <bool ADD>
    __device__ void send3(const CUtensorMap* map, int c0, int c1, int c2) const {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if constexpr (ADD)
                asm volatile(
                    "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group "
                    "[%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                    "r"(smem), "r"(c0), "r"(c1), "r"(c2)
                    : "memory");
            else
                asm volatile(
                    "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group "
                    "[%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                    "r"(smem), "r"(c0), "r"(c1), "r"(c2)
                    : "memory");
            bulk_commit();
        }
    }
};

// The half (128 columns) of one row of an accumulator that this thread empties:
// taddr is its first column, row0 the warp's first row in the result, c0 the first
// column.  `release` is called once the accumulator has been read.  (The TMEM loads
// are warp-wide: lanes that took different branches meet before.)
template <Mode MODE, typename F>
__device__ __forceinline__ void epilogue(const CeArgs& a, const Item& w, uint32_t taddr, int row0,
                                         int c0, const OutBox& out, const CUtensorMap* map_dh,
                                         const CUtensorMap* map_out, F&& release) {
    const int row = row0 + out.lane;
    if constexpr (MODE == kLoss) {
        float v[32];
        const bool in = row < a.tokens;
        const long long target = in ? a.targets[row] : -1;
        RowSum sum{-INFINITY, 0.0f};
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
            __syncwarp();
            tmem_ld32(taddr + c, v);
            tmem_wait_ld();
            if (c + 32 == kHalf) release();
            const int col = c0 + c;
            if (col + 32 <= a.vocab) sum.add(v, 32);
            else if (col < a.vocab) sum.add(v, a.vocab - col);
            const long long at = target - col;
            if (at >= 0 && at < 32 && target < a.vocab) a.target_logit[row] = pick(v, (int)at);
        }
        if (in) a.parts[(size_t)(c0 / kHalf) * a.tokens + row] = make_float2(sum.m, sum.s);
    } else if constexpr (MODE == kProb) {
        float v[32];
        const bool in = row < a.tokens;
        const long long target = in ? a.targets[row] : -1;
        const bool counts = target >= 0 && target < a.vocab;
        const float g = counts ? __fdiv_rn(a.dloss[row], *a.scale) : 0.0f;
        const float lse2 = in ? a.lse[row] * kLog2e : 0.0f;
        // the target's column in the piece, -1 where it is in none of it
        const long long rel = target - a.v0;
        const int tcol = counts && rel >= 0 && rel < a.width ? (int)rel : -1;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
            __syncwarp();
            tmem_ld32(taddr + c, v);
            tmem_wait_ld();
            if (c + 32 == kHalf) release();
            const int col = c0 + c;  // within the piece
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                float p = ex2_approx(fmaf(v[j], kLog2e, -lse2));
                if (tcol == col + j) p -= 1.0f;
                v[j] = p * g;
            }
            // a token without loss takes nothing, whatever its logits are
            if (!counts) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.0f;
            }
            if ((c & 32) == 0) out.ready();
            out.put_bf16((c & 32) / 8, v);
            if ((c & 32) && col - 32 < a.width && row0 < a.tokens)
                out.send(map_out, col - 32, row0);
        }
    } else {
        float v[32];
        const float scale = *a.scale;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
            __syncwarp();
            tmem_ld32(taddr + c, v);
            tmem_wait_ld();
            if (c + 32 == kHalf) release();
            const int col = c0 + c;
            if (w.dw) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= scale;
                if (a.dw_bf16) {
                    if ((c & 32) == 0) out.ready();
                    out.put_bf16((c & 32) / 8, v);
                    if ((c & 32) && col - 32 < a.dim && row0 < a.width)
                        out.send(map_out, col - 32, a.v0 + row0);
                } else {
                    out.ready();
                    out.put_f32(v);
                    if (col < a.dim && row0 < a.width) out.send(map_out, col, a.v0 + row0);
                }
            } else {
                out.ready();
                out.put_f32(v);
                if (col < a.dim && row0 < a.tokens) {
                    if (a.first_piece) out.send3<false>(map_dh, col, row0, w.split);
                    else out.send3<true>(map_dh, col, row0, w.split);
                }
            }
        }
    }
}

// ----------------------------------------------------------------- kernel

// Tensor maps of h (tokens x dim), W (vocab x dim) and P (tokens x ld): boxes of 64
// of K by a CTA's 128 rows (loss and P), or 64 x 64 (gradient).
template <Mode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ce_kernel(const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_W,
              const __grid_constant__ CUtensorMap tm_P, const __grid_constant__ CUtensorMap tm_dh,
              const __grid_constant__ CUtensorMap tm_out, const CeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t s_tmem, s_failed;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        s_failed = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&s_tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Schedule<MODE> sched(a, gridDim.x / 2, blockIdx.x / 2);
    bool ok = true;

    if (warp == kEpiWarps) {
        // ---- loads: this CTA's half of A and of B
        if (lane == 0) {
            uint32_t n = 0;  // stages filled
            Item w;
            for (int i = 0; ok && sched.get(a, i, w); ++i) {
                const int am = w.m0 + (int)rank * kHalf, bn = w.n0 + (int)rank * kHalf;
                for (int kb = 0; kb < w.depth; ++kb, ++n) {
                    const uint32_t s = n % kStages;
                    if (!mbar_wait(&empty[s], ((n / kStages) & 1) ^ 1, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = first_cta(&full[s]);
                    const uint32_t A = smem + s * kStageBytes, B = A + kOperand;
                    const int k = w.k0 + kb * kDepth;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
                    if constexpr (MODE != kGrad) {
                        load_box(A, &tm_h, bar, k, am);
                        load_box(B, &tm_W, bar, k, a.v0 + bn);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (w.dw) {
                                load_box(A + j * kBox, &tm_P, bar, am + 64 * j, k);
                                load_box(B + j * kBox, &tm_h, bar, bn + 64 * j, k);
                            } else {
                                load_box(A + j * kBox, &tm_P, bar, k, am + 64 * j);
                                load_box(B + j * kBox, &tm_W, bar, bn + 64 * j, a.v0 + k);
                            }
                        }
                    }
                }
            }
            // the MMAs' arrivals on this CTA's barriers are all in before it ends
            for (uint32_t q = n > kStages ? n - kStages : 0; ok && q < n; ++q)
                ok = mbar_wait(&empty[q % kStages], (q / kStages) & 1, a.status);
        }
    } else if (warp == kEpiWarps + 1) {
        // ---- products, issued by the first CTA for both
        if (lane == 0 && rank == 0) {
            uint32_t n = 0;
            Item w;
            for (int i = 0; ok && sched.get(a, i, w); ++i) {
                const uint32_t d = tmem + (i & 1) * kTile;
                const bool a_mn = MODE == kGrad && w.dw, b_mn = MODE == kGrad;
                const uint32_t idesc = idesc_bf16_f32(kTile, kTile) | (a_mn ? kIdescAMN : 0) |
                                       (b_mn ? kIdescBMN : 0);
                ok = wait_cluster(&acc_empty[i & 1], ((i >> 1) & 1) ^ 1, a.status);
                tc_fence_after();
                for (int kb = 0; ok && kb < w.depth; ++kb, ++n) {
                    const uint32_t s = n % kStages;
                    ok = wait_cluster(&full[s], (n / kStages) & 1, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t A = smem + s * kStageBytes, B = A + kOperand;
                    // 16 of K: 32 bytes within a K-major row, 16 rows of an MN-major tile
                    const uint64_t da = a_mn ? smem_desc_mn128(A, kBox) : smem_desc_k128(A);
                    const uint64_t db = b_mn ? smem_desc_mn128(B, kBox) : smem_desc_k128(B);
                    const uint32_t sa = a_mn ? 2048u >> 4 : 32u >> 4, sb = b_mn ? 2048u >> 4 : 32u >> 4;
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k)
                        mma_pair(d, da + k * sa, db + k * sb, idesc, (uint32_t)(kb | k));
                    commit_pair(&empty[s]);
                }
                if (ok) commit_pair(&acc_full[i & 1]);
            }
        }
    } else {
        // ---- epilogue: warp w of a quarter's two empties lanes 32 (w % 4) .. and
        // the columns of its half
        const int quarter = warp & 3, half = warp >> 2;
        const OutBox out{smem + kStages * kStageBytes + warp * kOutBox, lane};
        Item w;
        for (int i = 0; sched.get(a, i, w); ++i) {
            // every lane waits: each then acquires by itself
            ok = mbar_wait(&acc_full[i & 1], (i >> 1) & 1, a.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (i & 1) * kTile +
                                   half * kHalf;
            epilogue<MODE>(a, w, taddr, w.m0 + (int)rank * kHalf + quarter * 32,
                           w.n0 + half * kHalf, out, &tm_dh, &tm_out, [&] {
                               tc_fence_before();
                               __syncwarp();
                               if (lane == 0) arrive_remote(first_cta(&acc_empty[i & 1]));
                           });
        }
        if (MODE != kLoss && lane == 0) bulk_wait_all();
    }
    // a wait ran out: leave the copies in flight time to land before the shared
    // memory goes
    if (!ok) {
        s_failed = 1;
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (MODE == kLoss && threadIdx.x == 0) a.failed[blockIdx.x] = s_failed;
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
}

// ------------------------------------------------------------- few tokens

// Up to 64 tokens the loss is bound by reading W once, and the pair's 256 rows of
// tokens would be mostly empty (8 tokens of dim 1536, vocabulary 50280: 49 us with
// them, 31 us here; a read of W at the card's copy rate: 23 us).  Here the vocabulary
// is the MMA's rows and the tokens its columns: each CTA takes one contiguous,
// evenly cut range of the vocabulary in 128-row tiles (the last one as many rows as
// are left, in boxes of 64 and 16, so that no CTA reads more than 15 rows beyond its
// share; all of it in boxes of 16 was bound by one thread's issue of nine loads a
// stage: 37 us), and keeps each row's and token's running maximum and sum in registers until its
// range is through.
constexpr int kFewTokens = 64;
constexpr uint32_t kFewW = 128 * 128;            // a stage's W
constexpr int kFewThreads = 192;                 // 4 epilogue warps, TMA, MMA

template <int N>
__host__ __device__ constexpr uint32_t few_stage() { return kFewW + N * 128; }

template <int N>
__host__ __device__ constexpr int few_stages() { return 216 * 1024 / few_stage<N>(); }

// PROB: the epilogue is P instead (bf16, a token's 32 neighbouring columns to a warp's
// store).
template <int N, bool PROB>
__global__ void __launch_bounds__(kFewThreads, 1)
    ce_few_kernel(const __grid_constant__ CUtensorMap tm_h,
                  const __grid_constant__ CUtensorMap tm_W128,
                  const __grid_constant__ CUtensorMap tm_W64,
                  const __grid_constant__ CUtensorMap tm_W16, const CeArgs a, int share) {
    constexpr uint32_t kFewStages = few_stages<N>();
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kFewStages], empty[kFewStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t s_tmem, s_failed;
    __shared__ int s_target[N];
    __shared__ float2 s_join[4][N];  // PROB: of [0], a token's lse (base 2) and dloss / scale
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = (int)min((long long)blockIdx.x * share, (long long)a.vocab);
    const int r1 = (int)min((long long)r0 + share, (long long)a.vocab);
    const int ntiles = (r1 - r0 + 127) / 128, depth = (a.dim + kDepth - 1) / kDepth;
    constexpr uint32_t kCols = 2 * N < 32 ? 32 : 2 * N;

    // the n-th stage's loads: tile t's depths from kb on
    uint32_t n = 0;
    int t = 0, kb = 0;
    auto load_next = [&] {
        const uint32_t s = n % kFewStages;
        const int row = r0 + t * 128, rows = min(128, (r1 - row + 15) / 16 * 16);
        uint8_t* W = smem_raw + (smem - smem_u32(smem_raw)) + s * few_stage<N>();
        mbar_arrive_expect_tx(&full[s], (rows + N) * 128);
        if (rows == 128) {
            tma_load_2d(W, &tm_W128, &full[s], kb * kDepth, row);
        } else {
            int j = 0;
            if (rows >= 64) {
                tma_load_2d(W, &tm_W64, &full[s], kb * kDepth, row);
                j = 64;
            }
            for (; j < rows; j += 16)
                tma_load_2d(W + j * 128, &tm_W16, &full[s], kb * kDepth, row + j);
        }
        tma_load_2d(W + kFewW, &tm_h, &full[s], kb * kDepth, 0);
        ++n;
        if (++kb == depth) {
            kb = 0;
            ++t;
        }
    };
    if (warp == 4 && lane == 0) {
        s_failed = 0;
        for (uint32_t i = 0; i < kFewStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        fence_mbar_init();
        // the ring's first filling does not wait for the other warps' preparations (with
        // the join's reads all at its start: 33 us became 31 us)
        while (t < ntiles && n < kFewStages) load_next();
    }
    for (int i = tid; i < N; i += kFewThreads) {
        const long long t = i < a.tokens ? a.targets[i] : -1;
        s_target[i] = t >= r0 && t < r1 ? (int)t : -1;
        if constexpr (PROB) {
            const bool counts = t >= 0 && t < a.vocab;
            s_join[0][i] = counts ? make_float2(a.lse[i] * kLog2e, __fdiv_rn(a.dloss[i], *a.scale))
                                  : make_float2(0.0f, 0.0f);
            s_join[1][i].x = counts ? 1.0f : 0.0f;
        }
    }
    if (warp == 0) tmem_alloc(&s_tmem, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;

    // the join may take its place beside this kernel's CTAs
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 4) {
        if (lane == 0) {
            while (t < ntiles) {
                ok = mbar_wait(&empty[n % kFewStages], ((n / kFewStages) & 1) ^ 1, nullptr);
                if (!ok) break;
                load_next();
            }
            for (uint32_t q = n > kFewStages ? n - kFewStages : 0; ok && q < n; ++q)
                ok = mbar_wait(&empty[q % kFewStages], (q / kFewStages) & 1, nullptr);
        }
    } else if (warp == 5) {
        if (lane == 0) {
            uint32_t n = 0;
            for (int t = 0; ok && t < ntiles; ++t) {
                ok = mbar_wait(&acc_empty[t & 1], ((t >> 1) & 1) ^ 1, nullptr);
                tc_fence_after();
                for (int kb = 0; ok && kb < depth; ++kb, ++n) {
                    const uint32_t s = n % kFewStages;
                    ok = mbar_wait(&full[s], (n / kFewStages) & 1, nullptr);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t W = smem + s * few_stage<N>();
                    const uint64_t da = smem_desc_k128(W), db = smem_desc_k128(W + kFewW);
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k)
                        mma_bf16(tmem + (t & 1) * N, da + 2 * k, db + 2 * k, idesc_bf16_f32(128, N),
                                 (uint32_t)(kb | k));
                    mma_commit(&empty[s]);
                }
                if (ok) mma_commit(&acc_full[t & 1]);
            }
        }
    } else {
        // rows' running maxima and sums, base 2, by token
        float m[N], sum[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            m[j] = -INFINITY;
            sum[j] = 0.0f;
        }
        for (int t = 0; t < ntiles; ++t) {
            ok = mbar_wait(&acc_full[t & 1], (t >> 1) & 1, nullptr);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const int row = r0 + t * 128 + warp * 32 + lane;
            float v[N];
#pragma unroll
            for (int c = 0; c < N; c += 16)
                tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + (t & 1) * N + c, v + c);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[t & 1]);
            if constexpr (PROB) {
                if (row < r1) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        if (j >= a.tokens) break;
                        const float2 g = s_join[0][j];
                        float p = ex2_approx(fmaf(v[j], kLog2e, -g.x));
                        if (s_target[j] == row) p -= 1.0f;
                        // a token without loss takes nothing, whatever its logits are
                        p = s_join[1][j].x != 0.0f ? p * g.y : 0.0f;
                        a.P[(size_t)j * a.ld + row] = __float2bfloat16_rn(p);
                    }
                }
            } else if (row < r1) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (s_target[j] == row) a.target_logit[j] = v[j];
                    const float l = v[j] * kLog2e, n = fmaxf(m[j], l);
                    // n is -inf only where every logit so far is
                    const float base = n == -INFINITY ? 0.0f : n;
                    sum[j] = fmaf(sum[j], ex2_approx(m[j] - base), ex2_approx(l - base));
                    m[j] = n;
                }
            }
        }
        // over the warp's rows, then the four warps
#pragma unroll
        for (int j = 0; j < (PROB ? 0 : N); ++j) {
            float mx = m[j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            float sj = sum[j] * ex2_approx(m[j] - (mx == -INFINITY ? 0.0f : mx));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sj += __shfl_xor_sync(0xffffffffu, sj, o);
            if (lane == 0) s_join[warp][j] = make_float2(mx, sj);
        }
    }
    if (!ok) {
        s_failed = 1;
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!PROB && tid < a.tokens) {
        float mx = -INFINITY, sj = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, s_join[w][tid].x);
        const float base = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            sj = fmaf(s_join[w][tid].y, ex2_approx(s_join[w][tid].x - base), sj);
        a.parts[(size_t)blockIdx.x * a.tokens + tid] = make_float2(mx, sj);
    }
    if (tid == 0) {
        if (!PROB) a.failed[blockIdx.x] = s_failed;
        else if (s_failed) record_status(a.status, SSM_ERR_TIMEOUT);
    }
    if (warp == 0) tmem_dealloc(tmem, kCols);
}

// Joins the column halves' maxima and sums: a CTA takes 8 rows, 128 threads to a row
// every 128th part, eight reads ahead; then warp w joins the 128 of row w.  (Threads
// that waited for each read took 30 us for 8 tokens' 394 parts, 32 rows to a CTA 22 us
// for 300 tokens' 1000.)  The first CTA also tells the status, from what the loss
// kernel's CTAs left.
constexpr int kJoinRows = 8, kJoinLanes = 128;

__global__ void __launch_bounds__(1024) ce_join_kernel(const float2* parts, int nparts,
                                                       const float* target_logit,
                                                       const long long* targets, int tokens,
                                                       int vocab, float* loss, float* lse,
                                                       const uint32_t* failed, int nctas,
                                                       uint32_t* status) {
    __shared__ float2 sh[kJoinLanes][kJoinRows + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = threadIdx.x % kJoinRows, q = threadIdx.x / kJoinRows;
    const int row = blockIdx.x * kJoinRows + r;
    // what a row's warp needs at the end is read here, so that reads wait only once
    const int mine = blockIdx.x * kJoinRows + warp;
    const bool last = warp < kJoinRows && lane == 0 && mine < tokens;
    const long long at = last ? targets[mine] : -1;
    // launched beside the loss kernel's end: wait for all it wrote
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float logit = at >= 0 && at < vocab ? target_logit[mine] : 0.0f;
    uint32_t f = 0;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < nctas; i += 1024) f |= failed[i];
    float m = -INFINITY, s = 0.0f;
    auto join = [&](float2 p) {
        const float n = fmaxf(m, p.x), base = n == -INFINITY ? 0.0f : n;
        s = s * ex2_approx(m - base) + p.y * ex2_approx(p.x - base);
        m = n;
    };
    if (row < tokens) {
        for (int i = q; i < nparts; i += 8 * kJoinLanes) {
            float2 p[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                p[k] = i + kJoinLanes * k < nparts
                           ? parts[(size_t)(i + kJoinLanes * k) * tokens + row]
                           : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) join(p[k]);
        }
    }
    sh[q][r] = make_float2(m, s);
    f = __syncthreads_or((int)f);
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = f ? SSM_ERR_TIMEOUT : SSM_OK;
    if (warp < kJoinRows) {
        m = -INFINITY;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kJoinLanes / 32; ++k) join(sh[lane + 32 * k][warp]);
        float mx = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float t = s * ex2_approx(m - (mx == -INFINITY ? 0.0f : mx));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (last) {
            const float l = fmaf(mx, 0.6931471805599453f, logf(t));
            lse[mine] = l;
            loss[mine] = at < 0 ? 0.0f : at < vocab ? l - logit : NAN;
        }
    }
}

// header of a gradient: max |dloss| over the tokens that count (1 where that is
// no usable factor: 0, infinite or NaN)
__global__ void __launch_bounds__(1024) ce_scale_kernel(const float* dloss,
                                                        const long long* targets, int tokens,
                                                        int vocab, CeHeader* head) {
    __shared__ float sh[32];
    float m = 0.0f;
    for (int i = threadIdx.x; i < tokens; i += 1024) {
        const long long t = targets[i];
        if (t >= 0 && t < vocab) m = fmaxf(m, fabsf(dloss[i]));
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = sh[threadIdx.x];
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (threadIdx.x == 0) {
            head->scale = m > 1e-30f && m < 1e30f ? m : 1.0f;
            head->status = 0;
        }
    }
}

// dh = the factor times the sum of the splits' parts, in order
template <typename T>
__global__ void __launch_bounds__(256) ce_dh_kernel(const float* parts, int splits, size_t n,
                                                    const float* scale, T* dh) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    float4 t = *reinterpret_cast<const float4*>(parts + i);
    for (int k = 1; k < splits; ++k) {
        const float4 p = *reinterpret_cast<const float4*>(parts + k * n + i);
        t.x += p.x; t.y += p.y; t.z += p.z; t.w += p.w;
    }
    const float f = *scale;
    t.x *= f; t.y *= f; t.z *= f; t.w *= f;
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(dh + i) = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
    else
        *reinterpret_cast<float4*>(dh + i) = t;
}

// ------------------------------------------------------------------- host

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
int tiles(int n) { return (n + kTile - 1) / kTile; }

// GB300 has 76 pairs of SMs; the plan may not depend on the device, since the
// workspace size follows from it.
constexpr int kPairs = 76;

// The gradient's pieces: P takes tokens x piece bf16, at most 256 MB (which
// spreads the launches' ends over enough work) but at least 4096 columns.
constexpr size_t kPieceElements = size_t(1) << 27;

struct Plan {
    int piece;   // columns of one piece, a multiple of 256
    int splits;  // of a piece's vocabulary in dh
};

Plan plan_grad(int tokens, int dim, int vocab) {
    Plan p;
    const size_t fit = std::max<size_t>(kPieceElements / std::max(tokens, 1) / kTile * kTile, 4096);
    const int pieces = (int)(((size_t)vocab + fit - 1) / fit);
    p.piece = tiles((vocab + pieces - 1) / pieces) * kTile;
    // dh's tiles are as deep as the piece is wide: split them until they fit
    // under an even share of the launch's work
    const long long nt = tiles(dim), dh = tiles(tokens) * nt, dw = tiles(p.piece) * nt;
    const long long dh_depth = p.piece / kDepth;
    const long long dw_cost = std::max((tokens + kDepth - 1) / kDepth, kEpilogue);
    const long long share = (dh * dh_depth + dw * dw_cost + kPairs - 1) / kPairs;
    p.splits = 1;
    while (p.splits < 32 &&
           (dh * p.splits + kPairs - 1) / kPairs * ((dh_depth + p.splits - 1) / p.splits) >
               share + share / 8)
        ++p.splits;
    return p;
}

// (all three are counted in ints, whole tiles, pieces and CTAs' shares too)
constexpr int kMost = 1 << 30;
bool sizes_fit(int tokens, int dim, int vocab) {
    return dim % 8 == 0 && tokens <= kMost && dim <= kMost && vocab <= kMost &&
           (double)tokens * vocab / (kTile * kTile) < 1e9;
}

constexpr int kMaxCtas = 1024;  // room for their flags
int grid_ctas() { return 2 * std::min(std::max(1, ssm_host::sm_count() / 2), kMaxCtas / 2); }

template <Mode MODE>
bool launch(const CUtensorMap& h, const CUtensorMap& W, const CUtensorMap& P,
            const CUtensorMap& dh, const CUtensorMap& out, const CeArgs& a, cudaStream_t s) {
    auto kernel = ce_kernel<MODE>;
    static std::atomic<int> cache[ssm_host::kMaxDevices];
    if (ssm_host::resident_ctas(reinterpret_cast<const void*>(kernel), kThreads, kSmemBytes, cache) <
        1)
        return false;
    kernel<<<grid_ctas(), kThreads, kSmemBytes, s>>>(h, W, P, dh, out, a);
    return cudaGetLastError() == cudaSuccess;
}

// the vocabulary of one CTA of the few-token kernel, whole boxes of 16 rows
int few_share(int vocab) { return ((vocab + grid_ctas() - 1) / grid_ctas() + 15) / 16 * 16; }

template <int N, bool PROB>
bool launch_few_as(const CUtensorMap& h, const CUtensorMap* W, const CeArgs& a, cudaStream_t s) {
    auto kernel = ce_few_kernel<N, PROB>;
    constexpr int smem = few_stages<N>() * few_stage<N>() + 1024;
    static std::atomic<int> cache[ssm_host::kMaxDevices];
    if (ssm_host::resident_ctas(reinterpret_cast<const void*>(kernel), kFewThreads, smem, cache) < 1)
        return false;
    kernel<<<grid_ctas(), kFewThreads, smem, s>>>(h, W[0], W[1], W[2], a, few_share(a.vocab));
    return cudaGetLastError() == cudaSuccess;
}

// columns of the few-token kernel
int few_cols(int tokens) { return tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64; }

// W: its maps of 128, 64 and 16 rows
template <bool PROB>
bool launch_few(const CUtensorMap& h, const CUtensorMap* W, const CeArgs& a, cudaStream_t s) {
    const int cols = few_cols(a.tokens);
    return cols == 16   ? launch_few_as<16, PROB>(h, W, a, s)
           : cols == 32 ? launch_few_as<32, PROB>(h, W, a, s)
                        : launch_few_as<64, PROB>(h, W, a, s);
}

bool few_maps(CUtensorMap* mh, CUtensorMap* mw, const void* h, const void* W, int tokens, int dim,
              int vocab) {
    using ssm_host::make_tmap_2d;
    return make_tmap_2d(mh, h, SSM_BF16, tokens, dim, few_cols(tokens), 64) &&
           make_tmap_2d(&mw[0], W, SSM_BF16, vocab, dim, kHalf, 64) &&
           make_tmap_2d(&mw[1], W, SSM_BF16, vocab, dim, 64, 64) &&
           make_tmap_2d(&mw[2], W, SSM_BF16, vocab, dim, 16, 64);
}

// P, (tokens, width) with rows ld apart: past its width it reads as 0, whatever the
// rows hold there
bool make_p_map(CUtensorMap* map, const CeArgs& a, int box_rows) {
    auto fn = ssm_host::encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)a.width, (cuuint64_t)a.tokens};
    const cuuint64_t strides[1] = {(cuuint64_t)a.ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.P, dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// dh's fp32 sums, (splits, tokens, dim): clipped at each split's tokens
bool make_parts_map(CUtensorMap* map, const float* base, int dim, int tokens, int splits) {
    auto fn = ssm_host::encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)tokens, (cuuint64_t)splits};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 4, (cuuint64_t)dim * 4 * tokens};
    const cuuint32_t box[3] = {32, 32, 1}, one[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(base), dims, strides, box,
              one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

struct Span { const void* p; size_t n; };

}  // namespace

extern "C" size_t ssm_vocab_ce_workspace_bytes(int tokens, int dim, int vocab) {
    if (tokens < 0 || dim < 1 || vocab < 1 || !sizes_fit(tokens, dim, vocab)) return 0;
    return 256 + kMaxCtas * 4 + round256((size_t)tokens * 4) +
           round256((size_t)std::max(2 * tiles(vocab), tokens <= kFewTokens ? kMaxCtas : 0) * tokens *
                    8);
}

extern "C" size_t ssm_vocab_ce_bwd_workspace_bytes(int tokens, int dim, int vocab) {
    if (tokens < 0 || dim < 1 || vocab < 1 || !sizes_fit(tokens, dim, vocab)) return 0;
    const Plan p = plan_grad(tokens, dim, vocab);
    return 256 + round256((size_t)tokens * p.piece * 2) +
           round256((size_t)p.splits * tokens * dim * 4);
}

static ssm_status_t ce_check(int tokens, int dim, int vocab) {
    if (tokens < 0 || dim < 1 || vocab < 1) return SSM_ERR_SHAPE;
    return sizes_fit(tokens, dim, vocab) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

extern "C" ssm_status_t ssm_vocab_ce_fwd(const void* h, const void* W, const long long* targets,
                                         float* loss, float* lse, int tokens, int dim, int vocab,
                                         ssm_dtype_t in_dtype, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    using namespace ssm_host;
    if (ssm_status_t st = ce_check(tokens, dim, vocab)) return st;
    if (!dtype_ok(in_dtype)) return SSM_ERR_DTYPE;
    if (in_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    if (tokens == 0) return SSM_OK;
    if (!h || !W || !targets || !loss || !lse) return SSM_ERR_NULL;
    const size_t need = ssm_vocab_ce_workspace_bytes(tokens, dim, vocab);
    if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
    for (const void* p : {h, W, (const void*)targets, (const void*)loss, (const void*)lse,
                          (const void*)workspace})
        if (!aligned16(p)) return SSM_ERR_ALIGN;
    const Span ins[] = {{h, (size_t)tokens * dim * 2}, {W, (size_t)vocab * dim * 2},
                        {targets, (size_t)tokens * 8}};
    const Span outs[] = {{loss, (size_t)tokens * 4}, {lse, (size_t)tokens * 4}, {workspace, need}};
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;

    const bool few = tokens <= kFewTokens;
    CUtensorMap mh, mw[3];
    if (few ? !few_maps(&mh, mw, h, W, tokens, dim, vocab)
            : !make_tmap_2d(&mh, h, SSM_BF16, tokens, dim, kHalf, 64) ||
                  !make_tmap_2d(&mw[0], W, SSM_BF16, vocab, dim, kHalf, 64))
        return SSM_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CeArgs a{};
    a.tokens = tokens; a.dim = dim; a.vocab = vocab; a.targets = targets;
    a.failed = reinterpret_cast<uint32_t*>(ws + 256);
    a.target_logit = reinterpret_cast<float*>(ws + 256 + kMaxCtas * 4);
    a.parts = reinterpret_cast<float2*>(ws + 256 + kMaxCtas * 4 + round256((size_t)tokens * 4));
    const bool ok = few ? launch_few<false>(mh, mw, a, s)
                        : launch<kLoss>(mh, mw[0], mh, mh, mh, a, s);
    if (!ok) return SSM_ERR_CUDA;
    // launched as the loss kernel's CTAs end, which saves the gap between the two
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((tokens + kJoinRows - 1) / kJoinRows);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(
        &cfg, ce_join_kernel, (const float2*)a.parts, few ? grid_ctas() : 2 * tiles(vocab),
        (const float*)a.target_logit, targets, tokens, vocab, loss, lse, (const uint32_t*)a.failed,
        grid_ctas(), &reinterpret_cast<CeHeader*>(ws)->status);
    return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

extern "C" ssm_status_t ssm_vocab_ce_bwd(const void* h, const void* W, const long long* targets,
                                         const float* lse, const float* dloss, void* dh, void* dW,
                                         int tokens, int dim, int vocab, ssm_dtype_t in_dtype,
                                         ssm_dtype_t grad_dtype, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    using namespace ssm_host;
    if (ssm_status_t st = ce_check(tokens, dim, vocab)) return st;
    if (!dtype_ok(in_dtype) || !dtype_ok(grad_dtype)) return SSM_ERR_DTYPE;
    if (in_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    const size_t ge = dtype_size(grad_dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!dW || (tokens > 0 && (!h || !W || !targets || !lse || !dloss || !dh))) return SSM_ERR_NULL;
    if (!aligned16(dW)) return SSM_ERR_ALIGN;
    if (tokens == 0)
        return cudaMemsetAsync(dW, 0, (size_t)vocab * dim * ge, s) == cudaSuccess ? SSM_OK
                                                                                  : SSM_ERR_CUDA;
    const size_t need = ssm_vocab_ce_bwd_workspace_bytes(tokens, dim, vocab);
    if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
    for (const void* p : {h, W, (const void*)targets, (const void*)lse, (const void*)dloss,
                          (const void*)dh, (const void*)workspace})
        if (!aligned16(p)) return SSM_ERR_ALIGN;
    const Span ins[] = {{h, (size_t)tokens * dim * 2}, {W, (size_t)vocab * dim * 2},
                        {targets, (size_t)tokens * 8}, {lse, (size_t)tokens * 4},
                        {dloss, (size_t)tokens * 4}};
    const Span outs[] = {{dh, (size_t)tokens * dim * ge}, {dW, (size_t)vocab * dim * ge},
                         {workspace, need}};
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;

    const Plan plan = plan_grad(tokens, dim, vocab);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    CeArgs a{};
    a.tokens = tokens; a.dim = dim; a.vocab = vocab; a.targets = targets;
    a.status = &reinterpret_cast<CeHeader*>(ws)->status;
    a.lse = lse; a.dloss = dloss; a.dW = dW; a.dw_bf16 = grad_dtype == SSM_BF16;
    a.P = reinterpret_cast<__nv_bfloat16*>(ws + 256);
    a.ld = plan.piece;
    a.dh_parts = reinterpret_cast<float*>(ws + 256 + round256((size_t)tokens * plan.piece * 2));
    // products of the gradient: boxes of 64 x 64; of the logits: as the forward; what
    // the epilogues write: boxes of 32 rows by 128 bytes
    const bool few = tokens <= kFewTokens && plan.piece >= vocab;
    CUtensorMap mh, mw, mp, mdh, mdw, mpo, lh, lw[3];
    if (!make_tmap_2d(&mh, h, SSM_BF16, tokens, dim, 64, 64) ||
        !make_tmap_2d(&mw, W, SSM_BF16, vocab, dim, 64, 64) ||
        !make_tmap_2d(&mdw, dW, grad_dtype, vocab, dim, 32, 128 / (int)ge) ||
        !make_parts_map(&mdh, a.dh_parts, dim, tokens, plan.splits))
        return SSM_ERR_CUDA;
    if (few ? !few_maps(&lh, lw, h, W, tokens, dim, vocab)
            : !make_tmap_2d(&lh, h, SSM_BF16, tokens, dim, kHalf, 64) ||
                  !make_tmap_2d(&lw[0], W, SSM_BF16, vocab, dim, kHalf, 64))
        return SSM_ERR_CUDA;
    CeHeader* head = reinterpret_cast<CeHeader*>(ws);
    a.scale = &head->scale;
    ce_scale_kernel<<<1, 1024, 0, s>>>(dloss, targets, tokens, vocab, head);
    // a split is the same number of stages in every piece, so that the narrower
    // last piece uses the first splits only
    a.split_depth = (plan.piece / kDepth + plan.splits - 1) / plan.splits;
    const int first_depth = (std::min(plan.piece, vocab) + kDepth - 1) / kDepth;
    const int used = (first_depth + a.split_depth - 1) / a.split_depth;
    for (int v0 = 0; v0 < vocab; v0 += plan.piece) {
        a.v0 = v0;
        a.width = std::min(plan.piece, vocab - v0);
        a.first_piece = v0 == 0;
        const int depth = (a.width + kDepth - 1) / kDepth;
        a.splits = (depth + a.split_depth - 1) / a.split_depth;
        if (!make_p_map(&mp, a, 64) || !make_p_map(&mpo, a, 32) ||
            !(few ? launch_few<true>(lh, lw, a, s)
                  : launch<kProb>(lh, lw[0], mp, mdh, mpo, a, s)) ||
            !launch<kGrad>(mh, mw, mp, mdh, mdw, a, s))
            return SSM_ERR_CUDA;
    }
    const size_t n = (size_t)tokens * dim;
    const unsigned grid = (unsigned)((n / 4 + 255) / 256);
    if (grad_dtype == SSM_BF16)
        ce_dh_kernel<<<grid, 256, 0, s>>>(a.dh_parts, used, n, a.scale,
                                          static_cast<__nv_bfloat16*>(dh));
    else
        ce_dh_kernel<<<grid, 256, 0, s>>>(a.dh_parts, used, n, a.scale,
                                          static_cast<float*>(dh));
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}
