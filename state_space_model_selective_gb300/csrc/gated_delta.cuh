// gated_delta.cuh -- what the gated delta rule's forward (gated_delta.cu) and gradient
// (gated_delta_bwd.cu) share: the chunked form, the records kept per chunk and head,
// operand tiles and copies.
//
// Per head, with the state S (dstate x headdim here), for chunks of 64 steps that start
// from S0 (G_i = sum of g up to step i, everything inside the chunk):
//   D_ij = exp(G_i - G_j), j <= i;   e_i = exp(G_i);   w_j = exp(G_63 - G_j)
//   A_ij = beta_i (k_i . k_j) D_ij, j < i;   T = (1 + A)^-1;   T' = T diag(beta)
//   R = V - e K S0                      what each step's value is off the carried state
//   U = T' R                            the steps' updates
//   Y = e Q S0 + P R,    P = ((Q K^T) D) T'
//   S1 = e_63 S0 + H R,  H = K^T diag(w) T'
// P and H depend on q, k and the gates alone, so one kernel makes them for all chunks at
// once, and the chain over the chunks is two products deep: K S0 and H R.
#pragma once

#include "common.cuh"
#include "tcgen05.cuh"

namespace gdn {

using namespace ssm;

constexpr int kC = 64;          // steps of a chunk
constexpr int kPan = 64;        // columns of headdim that one chain takes
constexpr uint32_t kTile = 8192;  // a 64 x 64 bf16 tile: 64 rows of 128 bytes

// The record of one chunk and head (bytes): H hi | H lo (dstate rows each) | P hi |
// P lo | T' | the gates.  Tiles are stored as they lie in shared memory: rows of 128
// bytes whose 16-byte pieces are XORed with (row mod 8), so that one bulk copy
// brings H and P in.  hi + lo: a value as the sum of two bf16, 2^-17 of it off.
constexpr uint32_t kGateBytes = 1024;
__host__ __device__ constexpr uint32_t h_bytes(int dk) { return (uint32_t)dk * 128u; }
__host__ __device__ constexpr uint32_t hp_bytes(int dk) { return 2 * h_bytes(dk) + 2 * kTile; }
__host__ __device__ constexpr uint32_t rec_bytes(int dk) {
    return hp_bytes(dk) + kTile + kGateBytes;
}
// What training keeps for each chunk, head and 64 columns of headdim: R | S0 (forward),
// dR | dS1 (gradient), rounded to bf16: only products whose results are rounded to bf16
// themselves read them.
__host__ __device__ constexpr uint32_t kept_bytes(int dk) { return kTile + h_bytes(dk); }

// The gates of a record: base-2 logarithms of the decay from the chunk's start as the
// sum of two floats, and a bit for every step that learns nothing.
struct Gates {
    float hi[kC], lo[kC];
    unsigned long long masked;
};
static_assert(sizeof(Gates) <= kGateBytes, "gates fit their place");

__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
    return ex2_approx((hi_i - hi_j) + (lo_i - lo_j));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// (a, b) = hi + lo, each a pair of bf16.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hp, uint32_t& lp) {
    hp = pack_bf16(a, b);
    lp = pack_bf16(a - bf16lo(hp), b - bf16hi(hp));
}

// Byte offset of 16-byte piece c of row r of a tile of 128-byte rows.
__device__ __forceinline__ uint32_t piece(int r, int c) {
    return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}

// 32 values as the 4 pieces c0 .. c0 + 3 of row r, split into a hi and a lo tile.
__device__ __forceinline__ void put32_split(uint8_t* hi, uint8_t* lo, int r, int c0, const float* v) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(v[8 * c + 2 * e], v[8 * c + 2 * e + 1], h[e], l[e]);
        const uint32_t off = piece(r, c0 + c);
        *reinterpret_cast<uint4*>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}
// The same, rounded to one tile.
__device__ __forceinline__ void put32(uint8_t* tile, int r, int c0, const float* v) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(tile + piece(r, c0 + c)) =
            make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                       pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]));
}
__device__ __forceinline__ void unpack8(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16lo(u[e]);
        f[2 * e + 1] = bf16hi(u[e]);
    }
}

// K-major operand (rows of 64 bf16 along the contraction) of R rows, k-step kk.
template <int R>
__device__ __forceinline__ uint64_t kdesc(uint32_t tile, int kk) {
    return smem_desc_k128(tile + (uint32_t)((kk >> 2) * (R * 128) + (kk & 3) * 32));
}
// MN-major operand (one row of 64 bf16 per step of the contraction), k-step kk;
// further blocks of 64 `lbo` bytes apart.
__device__ __forceinline__ uint64_t mdesc(uint32_t tile, int kk, uint32_t lbo) {
    return smem_desc_mn128(tile + (uint32_t)kk * 2048u, lbo);
}

// `bytes` (a multiple of 16) of global memory to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// One arrival of a warp whose lanes have all come this far.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// A wait that a whole warp takes together, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

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
           (groups == 0 ? heads == 0 : heads % groups == 0);
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
inline size_t records_bytes(int batch, int seqlen, int heads, int dk) {
    return chunk_count(batch, seqlen, heads) * gdn::rec_bytes(dk_tile(dk));
}
inline size_t keep_bytes(int batch, int seqlen, int heads, int dk, int dv) {
    return chunk_count(batch, seqlen, heads) * ((dv + 63) / 64) * gdn::kept_bytes(dk_tile(dk));
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
    int batch, seqlen, heads, groups, dk, dv;
};
ssm_status_t chunked_forward(const Forward& f, cudaStream_t stream);

}  // namespace gdn_internal
