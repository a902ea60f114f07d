// norm.cu -- RMS norm with the residual's addition: forward, forward with an
// 8-bit output and scales, and gradient.
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   8-bit: amax over each group of a row's y, scale = amax / 448,
//          q = e4m3(y * 448 / amax)
//   gradient at the kept s: n = s r, g = dy w,
//          ds = r (g - n mean(g n)) + dsum,   dw = sum over rows of dy n
//
// Bound by memory: about ten FP32 operations per element against 6 to 20
// bytes, so the row is read once into registers, reduced, and written once.
//
// Layout of the work: a warp owns blocks of 256 consecutive elements of a row
// (block k of warp w starts at 256 (w + k warps)), so that a quantisation group
// of up to 256 elements never leaves a warp.  Where rows are 16-byte aligned
// (dim a multiple of 8) a lane holds 8 consecutive elements, moved with 16-byte
// accesses; else lane l holds elements l, 32 + l, ... of the block, so that the
// element-wise accesses of a warp are contiguous.  Rows of up to 256 elements
// take one warp each, several to a CTA; longer rows take one CTA of up to
// 32 warps of one block or 16 of four.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "common.cuh"

namespace {

using namespace ssm;

constexpr int kBlock = 256;      // elements of a row one warp owns at a time
constexpr int kMaxDim = 16384;   // 16 warps of 4 blocks
constexpr float kE4m3Max = 448.0f;
constexpr int kBwdThreads = 640;
constexpr int kFwdThreads = 1024;  // of the forward on an SM at a time

struct NormArgs {
    const void* x;         // forward: x; gradient: the kept sum
    const void* residual;  // forward: may be NULL; gradient: dsum, may be NULL
    const float* weight;
    const void* dy;        // gradient only
    void* y;               // forward: y or q; gradient: dx
    void* sum;             // forward: the sum, may be NULL; gradient: dresidual, may be NULL
    float* scales;         // 8-bit only
    float* partial;        // gradient only: [gridDim.x][dim] sums of dy n
    float eps, inv_dim;
    long long rows;
    int dim;
    int warps_per_row, rows_per_cta;
    int group, ngroups;    // 8-bit only; group 0 = the whole row
};

// The 8 elements a lane holds of block `blk` of a row, as they come from memory:
// loaded a row ahead of their use.  Elements past `dim` read as 0.
template <typename T, bool VEC>
struct Raw {
    static constexpr int kWords = VEC ? (int)sizeof(T) / 2 : 8;
    using Word = std::conditional_t<VEC, uint4, float>;
    Word w[kWords];

    __device__ void load(const T* p, int blk, int lane, int dim) {
        if constexpr (VEC) {
            const int i = blk * kBlock + lane * 8;
#pragma unroll
            for (int j = 0; j < kWords; ++j)
                w[j] = i < dim ? __ldcs(reinterpret_cast<const uint4*>(p + i) + j)
                               : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = blk * kBlock + j * 32 + lane;
                w[j] = i < dim ? to_f32(p[i]) : 0.0f;
            }
        }
    }
    __device__ float get(int j) const {  // j a constant
        if constexpr (!VEC) return w[j];
        else if constexpr (sizeof(T) == 2) {
            const uint32_t u = (j >> 1) == 0 ? w[0].x : (j >> 1) == 1 ? w[0].y
                             : (j >> 1) == 2 ? w[0].z : w[0].w;
            return j & 1 ? bf16hi(u) : bf16lo(u);
        } else {
            const uint4& q = w[j >> 2];
            return __uint_as_float((j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w);
        }
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int blk, int lane, int dim, const float* v) {
    if constexpr (VEC) {
        const int i = blk * kBlock + lane * 8;
        if (i >= dim) return;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(p + i) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7]));
        } else {
            *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(p + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = blk * kBlock + j * 32 + lane;
            if (i < dim) p[i] = from_f32<T>(v[j]);
        }
    }
}

// weight, read by every row: cached
template <bool VEC>
__device__ __forceinline__ void load_weight(const float* p, int blk, int lane, int dim, float* v) {
    if constexpr (VEC) {
        const int i = blk * kBlock + lane * 8;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (i < dim) {
            a = __ldg(reinterpret_cast<const float4*>(p + i));
            b = __ldg(reinterpret_cast<const float4*>(p + i + 4));
        }
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = blk * kBlock + j * 32 + lane;
            v[j] = i < dim ? __ldg(p + i) : 0.0f;
        }
    }
}

// two e4m3 values, round to nearest even, magnitudes above 448 to 448
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// max over the `width` consecutive lanes (a power of two) this lane is among
__device__ __forceinline__ float lanes_max(float v, int width) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o < width) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// amax -> 448 / amax, the factor q takes, within 2 ulp (an exact division costs as
// much as the rest of the quantisation).  0 for a group of zeros, and for one whose
// amax is infinite or NaN, where the factor leaves NaN in the places it came from;
// kept finite so that a zero beside denormals stays zero.
__device__ __forceinline__ float quant_factor(float amax) {
    return amax > 0.0f ? fminf(kE4m3Max * rcp_approx(amax), FLT_MAX) : 0.0f;
}

__device__ __forceinline__ float quant_scale(float amax) { return amax * (1.0f / kE4m3Max); }

enum Out { kPlain, kE4m3 };

// The 8-bit output of a row: v is its y.
template <int NV, bool VEC>
__device__ __forceinline__ void quantise(const NormArgs& a, long long row, float (*v)[8], int wr,
                                         int lane, int warp, float* red) {
    uint8_t* q = static_cast<uint8_t*>(a.y) + (size_t)row * a.dim;
    float* scales = a.scales + (size_t)row * a.ngroups;
    float row_amax = 0.0f;
    if (a.group == 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) row_amax = max_nan(row_amax, fabsf(v[k][j]));
        row_amax = lanes_max(row_amax, 32);
        if (a.warps_per_row > 1) {
            if (lane == 0) red[warp] = row_amax;
            __syncthreads();
            row_amax = lanes_max(lane < a.warps_per_row ? red[lane] : 0.0f, 32);
        }
        if (wr == 0 && lane == 0) scales[0] = quant_scale(row_amax);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int blk = wr + k * a.warps_per_row;
        float amax[8];  // VEC: one group per lane, in amax[0]
        if (a.group == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) amax[j] = row_amax;
        } else if constexpr (VEC) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[k][j]));
            const int width = a.group >> 3;
            amax[0] = lanes_max(m, width);
            const int i = blk * kBlock + lane * 8;
            if ((lane & (width - 1)) == 0 && i < a.dim)
                scales[i / a.group] = quant_scale(amax[0]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) amax[j] = lanes_max(fabsf(v[k][j]), 32);
            // a group is group / 32 consecutive rows of 32 lanes
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                if (o * 32 < a.group) {
                    float t[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) t[j] = max_nan(amax[j], amax[j ^ o]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) amax[j] = t[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = blk * kBlock + j * 32;
                if (lane == 0 && i % a.group == 0 && i < a.dim)
                    scales[i / a.group] = quant_scale(amax[j]);
            }
        }
        if constexpr (VEC) {
            const float f = quant_factor(amax[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] *= f;
            const int i = blk * kBlock + lane * 8;
            if (i < a.dim)
                *reinterpret_cast<uint2*>(q + i) =
                    make_uint2(e4m3x2(v[k][0], v[k][1]) | e4m3x2(v[k][2], v[k][3]) << 16,
                               e4m3x2(v[k][4], v[k][5]) | e4m3x2(v[k][6], v[k][7]) << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = blk * kBlock + j * 32 + lane;
                if (i < a.dim)
                    q[i] = (uint8_t)e4m3x2(v[k][j] * quant_factor(amax[j]), 0.0f);
            }
        }
    }
}

// ------------------------------------------------------------- forward

// A CTA (with one warp to a row: each warp) walks rows, the next row's loads in
// flight while this one is reduced and written: one row to a CTA, and CTAs that
// come and go, left the memory idle during each CTA's reductions (4.7 TB/s at
// 16384 rows of 2048 with an 8-bit output, against @Q8@ TB/s).
template <typename TX, typename TR, typename TY, int NV, bool VEC, Out OUT>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[2][2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wr = warp % a.warps_per_row;  // the warp within its row
    const bool has_res = a.residual != nullptr;
    long long row = (long long)blockIdx.x * a.rows_per_cta + warp / a.warps_per_row;
    const long long step = (long long)gridDim.x * a.rows_per_cta;

    Raw<TX, VEC> x[NV];
    Raw<TR, VEC> res[NV];
    auto load = [&](long long r) {
        const size_t base = (size_t)r * a.dim;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int blk = wr + k * a.warps_per_row;
            x[k].load(static_cast<const TX*>(a.x) + base, blk, lane, a.dim);
            if (has_res) res[k].load(static_cast<const TR*>(a.residual) + base, blk, lane, a.dim);
        }
    };
    if (row < a.rows) load(row);
    float w1[8];  // the weight, kept where a lane has one block of it
    if constexpr (NV == 1) load_weight<VEC>(a.weight, wr, lane, a.dim, w1);
    // `row` is the same in a CTA, or the warps do not meet
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        const size_t base = (size_t)row * a.dim;
        float v[NV][8];
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[k][j] = x[k].get(j);
                if (has_res) v[k][j] += res[k].get(j);
            }
        if (row + step < a.rows) load(row + step);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int blk = wr + k * a.warps_per_row;
            if (a.sum) store8<VEC>(static_cast<TR*>(a.sum) + base, blk, lane, a.dim, v[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[k][j], v[k][j], ss);
        }
        ss = warp_sum(ss);
        if (a.warps_per_row > 1) {
            // two buffers: a warp may write the next row's sums while another still
            // reads this row's
            if (lane == 0) red[0][turn][warp] = ss;
            __syncthreads();
            ss = warp_sum(lane < a.warps_per_row ? red[0][turn][lane] : 0.0f);
        }
        const float r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));

#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int blk = wr + k * a.warps_per_row;
            float w[8];
            if constexpr (NV > 1) load_weight<VEC>(a.weight, blk, lane, a.dim, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * r * (NV > 1 ? w[j] : w1[j]);
            if constexpr (OUT == kPlain)
                store8<VEC>(static_cast<TY*>(a.y) + base, blk, lane, a.dim, v[k]);
        }
        if constexpr (OUT == kE4m3) quantise<NV, VEC>(a, row, v, wr, lane, warp, red[1][turn]);
    }
}

// ------------------------------------------------------------ gradient

// CTAs walk rows as the forward's do, each thread keeping the weight's gradient of
// its columns in registers; norm_dw_kernel adds the CTAs' sums in order.  AHEAD:
// the next row's loads are in flight while this one is reduced (three inputs of
// two blocks a warp are as much as the registers hold).
template <typename TX, typename TR, typename TY, int NV, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormArgs a) {
    __shared__ float2 red[2][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool has_add = a.residual != nullptr;
    float dw[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.0f;
    Raw<TR, VEC> rs[NV], radd[NV];
    Raw<TY, VEC> rdy[NV];
    auto load = [&](long long r) {
        const size_t base = (size_t)r * a.dim;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int blk = warp + k * a.warps_per_row;
            rs[k].load(static_cast<const TR*>(a.x) + base, blk, lane, a.dim);
            rdy[k].load(static_cast<const TY*>(a.dy) + base, blk, lane, a.dim);
            if (has_add) radd[k].load(static_cast<const TR*>(a.residual) + base, blk, lane, a.dim);
        }
    };
    int turn = 0;
    if (AHEAD && blockIdx.x < a.rows) load(blockIdx.x);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const size_t base = (size_t)row * a.dim;
        if constexpr (!AHEAD) load(row);
        Raw<TR, VEC> s[NV], add[NV];
        Raw<TY, VEC> dy[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            s[k] = rs[k];
            dy[k] = rdy[k];
            if (has_add) add[k] = radd[k];
        }
        if (AHEAD && row + gridDim.x < a.rows) load(row + gridDim.x);
        float ss = 0.0f, sg = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[8];
            load_weight<VEC>(a.weight, warp + k * a.warps_per_row, lane, a.dim, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(s[k].get(j), s[k].get(j), ss);
                sg = fmaf(s[k].get(j), dy[k].get(j) * w[j], sg);
            }
        }
        ss = warp_sum(ss);
        sg = warp_sum(sg);
        if (a.warps_per_row > 1) {
            if (lane == 0) red[turn][warp] = make_float2(ss, sg);
            __syncthreads();
            const float2 t = lane < a.warps_per_row ? red[turn][lane] : make_float2(0.f, 0.f);
            ss = warp_sum(t.x);
            sg = warp_sum(t.y);
        }
        const float r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
        const float c = sg * a.inv_dim * r * r;  // mean(g n) r, so that n mean(g n) = s c
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int blk = warp + k * a.warps_per_row;
            float w[8], d[8];
            load_weight<VEC>(a.weight, blk, lane, a.dim, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sj = s[k].get(j), g = dy[k].get(j);
                d[j] = r * fmaf(-sj, c, g * w[j]);
                if (has_add) d[j] += add[k].get(j);
                dw[k][j] = fmaf(g, sj * r, dw[k][j]);
            }
            if (a.y) store8<VEC>(static_cast<TX*>(a.y) + base, blk, lane, a.dim, d);
            if (a.sum) store8<VEC>(static_cast<TR*>(a.sum) + base, blk, lane, a.dim, d);
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
        store8<VEC>(a.partial + (size_t)blockIdx.x * a.dim, warp + k * a.warps_per_row, lane,
                    a.dim, dw[k]);
}

// dw[c] = sum of the CTAs' partial[i][c] in a fixed order: 8 warps take every
// eighth partial row, then warp 0 adds the 8 sums.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* partial, int parts, int dim,
                                                      float* dw) {
    __shared__ float acc[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (c < dim) {
        int i = warp;
        for (; i + 56 < parts; i += 64) {  // eight loads at a time
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = partial[(size_t)(i + 8 * k) * dim + c];
#pragma unroll
            for (int k = 0; k < 8; ++k) t += v[k];
        }
        for (; i < parts; i += 8) t += partial[(size_t)i * dim + c];
    }
    acc[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < dim) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += acc[i][lane];
        dw[c] = t;
    }
}

// -------------------------------------------------------------- launch

// The most CTAs a gradient takes: their sums of dw are written and read once more.
// (The workspace's size follows from it, so it does not depend on the device.)
constexpr int kBwdCtas = 152 * 4;

template <typename F>
bool by_types(ssm_dtype_t x, ssm_dtype_t r, ssm_dtype_t y, F&& f) {
    using B = __nv_bfloat16;
    if (x == SSM_F32 && r == SSM_F32 && y == SSM_F32) f(float{}, float{}, float{});
    else if (x == SSM_F32 && r == SSM_F32 && y == SSM_BF16) f(float{}, float{}, B{});
    else if (x == SSM_BF16 && r == SSM_F32 && y == SSM_F32) f(B{}, float{}, float{});
    else if (x == SSM_BF16 && r == SSM_F32 && y == SSM_BF16) f(B{}, float{}, B{});
    else if (x == SSM_BF16 && r == SSM_BF16 && y == SSM_F32) f(B{}, B{}, float{});
    else if (x == SSM_BF16 && r == SSM_BF16 && y == SSM_BF16) f(B{}, B{}, B{});
    else return false;
    return true;
}

// blocks of 256 elements -> warps of a row, with NV blocks to a warp
int row_warps(int dim, int nv) { return ((dim + kBlock - 1) / kBlock + nv - 1) / nv; }

struct Span { const void* p; size_t n; };

}  // namespace

static ssm_status_t norm_check_sizes(int rows, int dim, ssm_dtype_t in, ssm_dtype_t res) {
    using namespace ssm_host;
    if (rows < 0 || dim < 1) return SSM_ERR_SHAPE;
    if (!dtype_ok(in) || !dtype_ok(res)) return SSM_ERR_DTYPE;
    if (dim > kMaxDim || (in == SSM_F32 && res == SSM_BF16)) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

static ssm_status_t norm_fwd(const void* x, const void* residual, const float* weight, float eps,
                             int group, void* y, float* scales, void* sum, int rows, int dim,
                             ssm_dtype_t in, ssm_dtype_t res, ssm_dtype_t out, bool e4m3,
                             void* stream) {
    using namespace ssm_host;
    if (ssm_status_t st = norm_check_sizes(rows, dim, in, res)) return st;
    if (!e4m3 && !dtype_ok(out)) return SSM_ERR_DTYPE;
    if (e4m3 && group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
        return group < 0 ? SSM_ERR_SHAPE : SSM_ERR_UNSUPPORTED;
    if (rows == 0) return SSM_OK;
    if (!x || !weight || !y || (e4m3 && !scales)) return SSM_ERR_NULL;
    for (const void* p : {x, residual, (const void*)weight, (const void*)y, (const void*)scales,
                          (const void*)sum})
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    const size_t n = (size_t)rows * dim;
    const int ngroups = !e4m3 ? 0 : group == 0 ? 1 : (dim + group - 1) / group;
    const Span ins[] = {{x, n * dtype_size(in)}, {residual, n * dtype_size(res)},
                        {weight, (size_t)dim * 4}};
    const Span outs[] = {{y, n * (e4m3 ? 1 : dtype_size(out))},
                         {sum, n * dtype_size(res)},
                         {scales, (size_t)rows * ngroups * 4}};
    for (const Span& o : outs)
        for (const Span& i : ins) {
            // the sum may take the residual's place: every element is read by
            // the thread that writes it
            if (o.p == sum && i.p == residual && sum == residual) continue;
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
        }
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;

    NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.sum = sum; a.scales = scales;
    a.eps = eps; a.inv_dim = 1.0f / (float)dim; a.rows = rows; a.dim = dim;
    a.group = group; a.ngroups = ngroups;
    const int nv = dim <= 32 * kBlock ? 1 : 4, warps = row_warps(dim, nv);
    a.warps_per_row = warps;
    a.rows_per_cta = warps == 1 ? 4 : 1;
    const int threads = 32 * warps * a.rows_per_cta;
    // as many CTAs as are resident: @THREADS@ threads to an SM
    const int resident = ssm_host::sm_count() * std::max(1, kFwdThreads / threads);
    const unsigned grid = (unsigned)std::min<long long>(
        ((long long)rows + a.rows_per_cta - 1) / a.rows_per_cta, resident);
    if (grid == 0) return SSM_ERR_CUDA;
    const bool vec = dim % 8 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    by_types(in, res, e4m3 ? SSM_F32 : out, [&](auto tx, auto tr, auto ty) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        using TY = decltype(ty);
        auto go = [&](auto kernel) { kernel<<<grid, threads, 0, s>>>(a); };
        if constexpr (sizeof(TY) == 4) {
            if (e4m3) {
                if (nv == 1) vec ? go(norm_fwd_kernel<TX, TR, TY, 1, true, kE4m3>)
                                 : go(norm_fwd_kernel<TX, TR, TY, 1, false, kE4m3>);
                else vec ? go(norm_fwd_kernel<TX, TR, TY, 4, true, kE4m3>)
                         : go(norm_fwd_kernel<TX, TR, TY, 4, false, kE4m3>);
                return;
            }
        }
        if (nv == 1) vec ? go(norm_fwd_kernel<TX, TR, TY, 1, true, kPlain>)
                         : go(norm_fwd_kernel<TX, TR, TY, 1, false, kPlain>);
        else vec ? go(norm_fwd_kernel<TX, TR, TY, 4, true, kPlain>)
                 : go(norm_fwd_kernel<TX, TR, TY, 4, false, kPlain>);
    });
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

extern "C" ssm_status_t ssm_add_rmsnorm_fwd(const void* x, const void* residual,
                                            const float* weight, float eps, void* y,
                                            void* sum_out, int rows, int dim,
                                            ssm_dtype_t in_dtype, ssm_dtype_t res_dtype,
                                            ssm_dtype_t out_dtype, void* stream) {
    return norm_fwd(x, residual, weight, eps, 0, y, nullptr, sum_out, rows, dim, in_dtype,
                    res_dtype, out_dtype, false, stream);
}

extern "C" ssm_status_t ssm_add_rmsnorm_e4m3_fwd(const void* x, const void* residual,
                                                 const float* weight, float eps, int group,
                                                 void* q, float* scales, void* sum_out, int rows,
                                                 int dim, ssm_dtype_t in_dtype,
                                                 ssm_dtype_t res_dtype, void* stream) {
    return norm_fwd(x, residual, weight, eps, group, q, scales, sum_out, rows, dim, in_dtype,
                    res_dtype, SSM_F32, true, stream);
}

extern "C" size_t ssm_add_rmsnorm_bwd_workspace_bytes(int rows, int dim) {
    if (rows < 0 || dim < 1 || dim > kMaxDim) return 0;
    return 256 + (size_t)std::min(rows, kBwdCtas) * dim * 4;
}

extern "C" ssm_status_t ssm_add_rmsnorm_bwd(const void* sum, const float* weight, float eps,
                                            const void* dy, const void* dsum, void* dx,
                                            void* dresidual, float* dweight, int rows, int dim,
                                            ssm_dtype_t in_dtype, ssm_dtype_t res_dtype,
                                            ssm_dtype_t dy_dtype, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    using namespace ssm_host;
    if (ssm_status_t st = norm_check_sizes(rows, dim, in_dtype, res_dtype)) return st;
    if (!dtype_ok(dy_dtype)) return SSM_ERR_DTYPE;
    if (!dweight || (rows > 0 && (!sum || !weight || !dy || (!dx && !dresidual))))
        return SSM_ERR_NULL;
    for (const void* p : {sum, (const void*)weight, dy, dsum, (const void*)dx,
                          (const void*)dresidual, (const void*)dweight, (const void*)workspace})
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    if (rows > 0 &&
        (!workspace || workspace_bytes < ssm_add_rmsnorm_bwd_workspace_bytes(rows, dim)))
        return SSM_ERR_WORKSPACE;
    const size_t n = (size_t)rows * dim;
    const Span ins[] = {{sum, n * dtype_size(res_dtype)}, {weight, (size_t)dim * 4},
                        {dy, n * dtype_size(dy_dtype)}, {dsum, n * dtype_size(res_dtype)}};
    const Span outs[] = {{dx, n * dtype_size(in_dtype)}, {dresidual, n * dtype_size(res_dtype)},
                         {dweight, (size_t)dim * 4}, {workspace, rows ? workspace_bytes : 0}};
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (overlaps(o.p, o.n, i.p, i.n)) return SSM_ERR_ALIAS;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return SSM_ERR_ALIAS;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0)
        return cudaMemsetAsync(dweight, 0, (size_t)dim * 4, s) == cudaSuccess ? SSM_OK
                                                                              : SSM_ERR_CUDA;
    NormArgs a{};
    a.x = sum; a.residual = dsum; a.weight = weight; a.dy = dy; a.y = dx; a.sum = dresidual;
    a.partial = static_cast<float*>(workspace);
    a.eps = eps; a.inv_dim = 1.0f / (float)dim; a.rows = rows; a.dim = dim;
    const int nv = dim <= 16 * kBlock ? 1 : dim <= 32 * kBlock ? 2 : 4;
    const int warps = row_warps(dim, nv);
    a.warps_per_row = warps;
    a.rows_per_cta = 1;
    const unsigned grid = (unsigned)std::min(
        rows, std::min(kBwdCtas, ssm_host::sm_count() * std::max(1, kBwdThreads / (32 * warps))));
    if (grid == 0) return SSM_ERR_CUDA;
    const bool vec = dim % 8 == 0;
    by_types(in_dtype, res_dtype, dy_dtype, [&](auto tx, auto tr, auto ty) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        using TY = decltype(ty);
        auto go = [&](auto kernel) { kernel<<<grid, 32u * warps, 0, s>>>(a); };
        if (nv == 1) vec ? go(norm_bwd_kernel<TX, TR, TY, 1, true, true>)
                         : go(norm_bwd_kernel<TX, TR, TY, 1, false, true>);
        else if (nv == 2) vec ? go(norm_bwd_kernel<TX, TR, TY, 2, true, true>)
                              : go(norm_bwd_kernel<TX, TR, TY, 2, false, true>);
        else vec ? go(norm_bwd_kernel<TX, TR, TY, 4, true, false>)
                 : go(norm_bwd_kernel<TX, TR, TY, 4, false, false>);
    });
    norm_dw_kernel<<<(dim + 31) / 32, 256, 0, s>>>(a.partial, (int)grid, dim, dweight);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}
