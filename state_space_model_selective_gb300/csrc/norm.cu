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
// Layout of the work: a lane holds 8 neighbouring elements, a warp 32 such chunks, so
// that a quantisation group of up to 256 elements never leaves a warp.  Rows of up
// to 64 (128) elements take 8 (16) lanes each, rows of up to 256 one warp, longer rows
// one CTA of up to 32 warps with one chunk a lane or 17 with four.  CTAs (with one
// warp or less to a row: their warps) walk rows, the next row's loads in flight while
// this one is reduced and written: one row to a CTA, and CTAs that come and go, left
// the memory idle during each CTA's reductions (461 us against 394 us for forward and
// gradient of 16384 rows of 5120, bf16 with an fp32 residual).
//
// Widths that are no multiple of 8: chunks are cut at multiples of 8 of the tensor's
// flat index, where every type is 16-byte aligned, so that a row's first and last
// chunk may be shared with its neighbours; only those are written element by element.
// A row's shift against the chunks is row * dim mod 8, and CTAs step by multiples of 8
// rows, so a lane's columns, and with them its weights and its sum of dw, stay the
// same.  (Element-wise accesses took 34.8 us for 10000 rows of 1001, bf16 with 8-bit
// output, against 19.5 us.)  These rows are further from their bytes than the others (19.5
// us for 10.4 us of them), and where a lane holds two or four of their pieces, or four of any
// row's in the gradient, registers spill: forward and gradient of 4096 bf16 rows with an
// fp32 residual take 163 us at 8192 columns, 312 us at 8191 and 278 us at 12288 (119, 119 and
// 178 us of bytes).
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace {

using namespace ssm;

constexpr int kMaxDim = 16384;
constexpr float kE4m3Max = 448.0f;
constexpr int kFwdThreads = 1024;  // of the forward on an SM at a time
constexpr int kBwdThreads = 640;   // of the gradient, bound by registers
constexpr int kMaxGroups = kMaxDim / 32;
constexpr int kSmallWarps = 8;     // of a CTA whose warps take rows by themselves

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
    int warps_per_row;     // 1: a warp takes 32 / lanes rows at a time
    int lanes;             // of a row's first warp: 8, 16 or 32
    int rows_per_cta;
    int group, ngroups;    // 8-bit only; group 0 = the whole row
};

// ------------------------------------------------------------------ chunks

// A lane's 8 elements of a row, i0 .. i0 + 7; those outside 0 .. dim - 1 are a
// neighbouring row's.
struct Chunk {
    int i0;
    bool any, full;
};

template <bool ALIGNED>
__device__ __forceinline__ Chunk chunk_at(int c, int shift, int dim, bool valid) {
    Chunk k;
    k.i0 = 8 * c - (ALIGNED ? 0 : shift);
    k.any = valid && k.i0 < dim;
    k.full = k.any && (ALIGNED || (k.i0 >= 0 && k.i0 + 8 <= dim));
    return k;
}

// 16 bytes read once, or zeros.  Volatile, so that the compiler leaves the next row's
// loads before this row's barrier instead of moving them to where they save registers
// (a few percent of forward and gradient of 16384 rows of 5120).
__device__ __forceinline__ uint4 load16(const void* p, bool in) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)in)
        : "memory");
    return v;
}

// The 8 elements as they come from memory: loaded a row ahead of their use.
template <typename T, bool ALIGNED>
struct Raw {
    static constexpr int kWords = (int)sizeof(T) / 2;
    uint4 w[kWords];

    // `at`: the chunk's first element in the tensor of `total` elements, a multiple of 8
    __device__ void load(const void* base, long long at, long long total, bool any) {
        const T* p = static_cast<const T*>(base) + at;
        const bool whole = any && (ALIGNED || at + 8 <= total);
#pragma unroll
        for (int j = 0; j < kWords; ++j)
            w[j] = load16(reinterpret_cast<const uint4*>(p) + j, whole);
        if (!ALIGNED && any && !whole) {  // the tensor's last elements
            uint32_t u[4 * kWords] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (at + j >= total) continue;
                if constexpr (sizeof(T) == 2)
                    u[j >> 1] |= (uint32_t)__bfloat16_as_ushort(p[j]) << (16 * (j & 1));
                else
                    u[j] = __float_as_uint(p[j]);
            }
#pragma unroll
            for (int j = 0; j < kWords; ++j)
                w[j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
        }
    }
    __device__ float get(int j) const {  // j a constant
        if constexpr (sizeof(T) == 2) {
            const uint32_t u = (j >> 1) == 0 ? w[0].x : (j >> 1) == 1 ? w[0].y
                             : (j >> 1) == 2 ? w[0].z : w[0].w;
            return j & 1 ? bf16hi(u) : bf16lo(u);
        } else {
            const uint4& q = w[j >> 2];
            return __uint_as_float((j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w);
        }
    }
    // zeros in the places of the neighbouring rows
    __device__ void mask(const Chunk& k, int dim) {
        if constexpr (!ALIGNED) {
            if (k.any && !k.full) {
                uint32_t u[4 * kWords] = {w[0].x, w[0].y, w[0].z, w[0].w};
                if constexpr (kWords == 2) {
                    u[4] = w[1].x; u[5] = w[1].y; u[6] = w[1].z; u[7] = w[1].w;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (k.i0 + j >= 0 && k.i0 + j < dim) continue;
                    if constexpr (sizeof(T) == 2) u[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
                    else u[j] = 0;
                }
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    w[j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
            }
        }
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store8(void* base, long long at, const Chunk& k, int dim,
                                       const float* v) {
    T* p = static_cast<T*>(base) + at;
    if (k.full) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(p) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7]));
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else if (!ALIGNED && k.any) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k.i0 + j >= 0 && k.i0 + j < dim) p[j] = from_f32<T>(v[j]);
    }
}

template <bool ALIGNED>
__device__ __forceinline__ void load_weight(const float* p, const Chunk& k, int dim, float* v) {
    if (ALIGNED) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (k.any) {
            a = __ldg(reinterpret_cast<const float4*>(p + k.i0));
            b = __ldg(reinterpret_cast<const float4*>(p + k.i0 + 4));
        }
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = k.any && k.i0 + j >= 0 && k.i0 + j < dim ? __ldg(p + k.i0 + j) : 0.0f;
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

// over the `width` consecutive lanes (a power of two) this lane is among
__device__ __forceinline__ float lanes_sum(float v, int width) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o < width) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float lanes_max(float v, int width) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o < width) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// 448 / amax, the factor q takes, within 2 ulp (an exact division costs as much as the rest
// of the quantisation) for an amax within 2^-100 .. 2^100.
__device__ __forceinline__ float quant_factor(float amax) { return kE4m3Max * rcp_approx(amax); }

// Whether amax is outside of that, where it or the factor may have no normal reciprocal: one
// comparison of the bits, which zeros, infinities and NaN fail too.
__device__ __forceinline__ bool quant_far(float amax) {
    constexpr uint32_t kLow = 0x0d800000u, kHigh = 0x71800000u;
    return __float_as_uint(amax) - kLow > kHigh - kLow;
}

// The power of two by which such a group comes nearer before it is quantised.
__device__ __forceinline__ float quant_nearer(float amax) {
    return !quant_far(amax) ? 1.0f : amax < 1.0f ? 0x1p64f : 0x1p-64f;
}

__device__ __forceinline__ float quant_scale(float amax) { return amax * (1.0f / kE4m3Max); }

enum Out { kPlain, kE4m3 };

// The 8-bit output of a row: v is its y (0 in the neighbouring rows' places).
template <int NV, bool ALIGNED, bool SMALL>
__device__ __forceinline__ void quantise(const NormArgs& a, long long row, float (*v)[8],
                                         const Chunk* ks, int lane, int warp, int wr, float* red,
                                         uint32_t* s_amax) {
    const long long base = row * a.dim;
    uint8_t* q = static_cast<uint8_t*>(a.y);
    constexpr bool small = SMALL;
    const int lanes = SMALL ? a.lanes : 32;
    float amax_of[NV][2];  // of the chunk's group, and of the next one's where it spans two
    int cut[NV];           // first element of that
    if (a.group == 0) {
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(v[k][j]));
        amax = lanes_max(amax, lanes);
        if (!small) {
            if (lane == 0) red[warp] = amax;
            __syncthreads();
            amax = lanes_max(lane < a.warps_per_row ? red[lane] : 0.0f, 32);
        }
        if (wr == 0 && (lane & (lanes - 1)) == 0 && row < a.rows) a.scales[row] = quant_scale(amax);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            amax_of[k][0] = amax_of[k][1] = amax;
            cut[k] = 8;
        }
    } else if constexpr (ALIGNED) {
        const int width = min(a.group >> 3, lanes);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(v[k][j]));
            amax = lanes_max(amax, width);
            if ((lane & (width - 1)) == 0 && ks[k].any)
                a.scales[row * a.ngroups + ks[k].i0 / a.group] = quant_scale(amax);
            amax_of[k][0] = amax_of[k][1] = amax;
            cut[k] = 8;
        }
    } else {
        // groups are cut in the row, chunks in the tensor: the maxima meet in shared
        // memory (magnitudes are ordered as their bits are, NaN above all)
        const int sub = small ? (threadIdx.x / lanes) * 8 : 0;
        const int me = small ? lane & (lanes - 1) : (int)threadIdx.x;
        const int all = small ? lanes : (int)blockDim.x;
        auto sync = [&] {
            if (small) __syncwarp();
            else __syncthreads();
        };
        for (int g = me; g < a.ngroups; g += all) s_amax[sub + g] = 0;
        sync();
        int first[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            first[k] = max(ks[k].i0, 0) / a.group;
            cut[k] = min(8, (first[k] + 1) * a.group - ks[k].i0);
            if (ks[k].any) {
                float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j < cut[k]) m0 = max_nan(m0, fabsf(v[k][j]));
                    else m1 = max_nan(m1, fabsf(v[k][j]));
                }
                atomicMax(&s_amax[sub + first[k]], __float_as_uint(m0));
                if (cut[k] < 8 && first[k] + 1 < a.ngroups)
                    atomicMax(&s_amax[sub + first[k] + 1], __float_as_uint(m1));
            }
        }
        sync();
        if (row < a.rows)
            for (int g = me; g < a.ngroups; g += all)
                a.scales[row * a.ngroups + g] = quant_scale(__uint_as_float(s_amax[sub + g]));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            amax_of[k][0] = amax_of[k][1] = 1.0f;
            if (ks[k].any) {
                amax_of[k][0] = __uint_as_float(s_amax[sub + first[k]]);
                if (cut[k] < 8 && first[k] + 1 < a.ngroups)
                    amax_of[k][1] = __uint_as_float(s_amax[sub + first[k] + 1]);
            }
        }
        sync();  // before the next row's zeros
    }
    bool far = false;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        far = far || quant_far(amax_of[k][0]) || (!ALIGNED && quant_far(amax_of[k][1]));
    if (__builtin_expect(far, 0)) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[k][j] *= quant_nearer(ALIGNED || j < cut[k] ? amax_of[k][0] : amax_of[k][1]);
            // factor 0 for a group of zeros, and for one whose amax is infinite or NaN, where
            // it leaves NaN in the places that came from
#pragma unroll
            for (int i = 0; i < 2; ++i)
                amax_of[k][i] = amax_of[k][i] > 0.0f ? amax_of[k][i] * quant_nearer(amax_of[k][i])
                                                     : INFINITY;
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const float f0 = quant_factor(amax_of[k][0]);
        const float f1 = ALIGNED ? f0 : quant_factor(amax_of[k][1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] *= ALIGNED || j < cut[k] ? f0 : f1;
        const uint2 w = make_uint2(e4m3x2(v[k][0], v[k][1]) | e4m3x2(v[k][2], v[k][3]) << 16,
                                   e4m3x2(v[k][4], v[k][5]) | e4m3x2(v[k][6], v[k][7]) << 16);
        uint8_t* p = q + base + ks[k].i0;
        if (ks[k].full) {
            *reinterpret_cast<uint2*>(p) = w;
        } else if (!ALIGNED && ks[k].any) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (ks[k].i0 + j >= 0 && ks[k].i0 + j < a.dim)
                    p[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
        }
    }
}

// ------------------------------------------------------------- forward

// SMALL: a row takes one warp or less.
template <typename TX, typename TR, typename TY, int NV, bool ALIGNED, bool SMALL, Out OUT>
__global__ void __launch_bounds__(SMALL ? 256 : !ALIGNED ? 544 : NV == 1 ? 1024 : 512)
    norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[2][2][32];
    __shared__ uint32_t s_amax[OUT == kE4m3 && !ALIGNED ? kMaxGroups : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr bool small = SMALL;
    const int lanes = SMALL ? a.lanes : 32;
    const int wr = small ? 0 : warp;  // the warp within its row
    const int c = small ? lane & (lanes - 1) : warp * 32 + lane;
    const bool has_res = a.residual != nullptr;
    const long long total = a.rows * a.dim, step = (long long)gridDim.x * a.rows_per_cta;
    // the warp's first row, and this lane's
    long long first = (long long)blockIdx.x * a.rows_per_cta + (small ? warp * (32 / lanes) : 0);
    const int sub = small ? lane / lanes : 0;
    const int shift = (int)((first + sub) * a.dim & 7);

    Chunk ks[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k)
        ks[k] = chunk_at<ALIGNED>(c + k * 32 * a.warps_per_row, shift, a.dim, true);
    Raw<TX, ALIGNED> x[NV];
    Raw<TR, ALIGNED> res[NV];
    auto load = [&](long long row) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long at = row * a.dim + ks[k].i0;
            const bool any = ks[k].any && (!SMALL || row < a.rows);
            x[k].load(a.x, at, total, any);
            if (has_res) res[k].load(a.residual, at, total, any);
        }
    };
    if (first < a.rows) load(first + sub);
    float w1[8];  // the weight, kept where a lane has one chunk
    if constexpr (NV == 1) load_weight<ALIGNED>(a.weight, ks[0], a.dim, w1);
    // `first` is the same in a CTA, or its warps do not meet
    for (int turn = 0; first < a.rows; first += step, turn ^= 1) {
        const long long row = first + sub;
        Chunk now[NV];
        float v[NV][8];
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            now[k] = ks[k];
            if constexpr (SMALL) {  // the warp's other rows may be past the last one
                now[k].any = ks[k].any && row < a.rows;
                now[k].full = ks[k].full && row < a.rows;
            }
            x[k].mask(now[k], a.dim);
            if (has_res) res[k].mask(now[k], a.dim);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[k][j] = x[k].get(j);
                if (has_res) v[k][j] += res[k].get(j);
            }
        }
        if (first + step < a.rows) load(row + step);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (a.sum) store8<TR, ALIGNED>(a.sum, row * a.dim + now[k].i0, now[k], a.dim, v[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[k][j], v[k][j], ss);
        }
        ss = lanes_sum(ss, lanes);
        if (!small) {
            // two buffers: a warp may write the next row's sums while another still
            // reads this row's
            if (lane == 0) red[0][turn][warp] = ss;
            __syncthreads();
            ss = lanes_sum(lane < a.warps_per_row ? red[0][turn][lane] : 0.0f, 32);
        }
        const float r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));

#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[8];
            if constexpr (NV > 1) load_weight<ALIGNED>(a.weight, ks[k], a.dim, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * r * (NV > 1 ? w[j] : w1[j]);
            if constexpr (OUT == kPlain)
                store8<TY, ALIGNED>(a.y, row * a.dim + now[k].i0, now[k], a.dim, v[k]);
        }
        if constexpr (OUT == kE4m3)
            quantise<NV, ALIGNED, SMALL>(a, row, v, now, lane, warp, wr, red[1][turn], s_amax);
    }
}

// ------------------------------------------------------------ gradient

// CTAs walk rows as the forward's do, each lane keeping the weight's gradient of its
// columns in registers; norm_dw_kernel adds the CTAs' sums in order.  AHEAD: the next
// row's loads are in flight while this one is reduced (three inputs of two chunks a
// lane are as much as the registers hold).
template <typename TX, typename TR, typename TY, int NV, bool ALIGNED, bool SMALL, bool AHEAD>
__global__ void __launch_bounds__(SMALL ? 256 : ALIGNED ? 512 : 544)
    norm_bwd_kernel(const NormArgs a) {
    __shared__ float2 red[2][32];
    __shared__ float s_dw[SMALL ? 256 : 1];  // of a CTA whose warps take rows by themselves
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr bool small = SMALL;
    const int lanes = SMALL ? a.lanes : 32;
    const int c = small ? lane & (lanes - 1) : warp * 32 + lane;
    const bool has_add = a.residual != nullptr;
    const long long total = a.rows * a.dim, step = (long long)gridDim.x * a.rows_per_cta;
    long long first = (long long)blockIdx.x * a.rows_per_cta + (small ? warp * (32 / lanes) : 0);
    const int sub = small ? lane / lanes : 0;
    const int shift = (int)((first + sub) * a.dim & 7);
    Chunk ks[NV];
    float dw[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        ks[k] = chunk_at<ALIGNED>(c + k * 32 * a.warps_per_row, shift, a.dim, true);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.0f;
    }
    float w1[8];  // the weight, kept where a lane has one chunk
    if constexpr (NV == 1) load_weight<ALIGNED>(a.weight, ks[0], a.dim, w1);
    struct In {
        Raw<TR, ALIGNED> s[NV], add[NV];
        Raw<TY, ALIGNED> dy[NV];
    };
    auto load = [&](In& in, long long row) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long at = row * a.dim + ks[k].i0;
            const bool any = ks[k].any && (!SMALL || row < a.rows);
            in.s[k].load(a.x, at, total, any);
            in.dy[k].load(a.dy, at, total, any);
            if (has_add) in.add[k].load(a.residual, at, total, any);
        }
    };
    int turn = 0;
    // the row `first`, held in `in`; the next one's loads into `ahead`
    auto row_of = [&](In& in, In& ahead) {
        const long long row = first + sub;
        Chunk now[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            now[k] = ks[k];
            if constexpr (SMALL) {
                now[k].any = ks[k].any && row < a.rows;
                now[k].full = ks[k].full && row < a.rows;
            }
        }
        if constexpr (!AHEAD) load(in, row);
        else if (first + step < a.rows) load(ahead, row + step);
        float ss = 0.0f, sg = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[8];
            in.s[k].mask(now[k], a.dim);
            in.dy[k].mask(now[k], a.dim);
            if constexpr (NV > 1) load_weight<ALIGNED>(a.weight, ks[k], a.dim, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sj = in.s[k].get(j);
                ss = fmaf(sj, sj, ss);
                sg = fmaf(sj, in.dy[k].get(j) * (NV > 1 ? w[j] : w1[j]), sg);
            }
        }
        ss = lanes_sum(ss, lanes);
        sg = lanes_sum(sg, lanes);
        if (!small) {
            if (lane == 0) red[turn][warp] = make_float2(ss, sg);
            __syncthreads();
            const float2 t = lane < a.warps_per_row ? red[turn][lane] : make_float2(0.f, 0.f);
            ss = lanes_sum(t.x, 32);
            sg = lanes_sum(t.y, 32);
        }
        // a row past the last one is zeros: with eps 0 its r would be infinite and reach dw
        const float r = !SMALL || row < a.rows ? rsqrtf(fmaf(ss, a.inv_dim, a.eps)) : 0.0f;
        const float c_ = sg * a.inv_dim * r * r;  // mean(g n) r, so that n mean(g n) = s c
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long at = row * a.dim + now[k].i0;
            float w[8], d[8];
            if constexpr (NV > 1) load_weight<ALIGNED>(a.weight, ks[k], a.dim, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sj = in.s[k].get(j), g = in.dy[k].get(j);
                d[j] = r * fmaf(-sj, c_, g * (NV > 1 ? w[j] : w1[j]));
                if (has_add) d[j] += in.add[k].get(j);
                dw[k][j] = fmaf(g, sj * r, dw[k][j]);
            }
            if (a.y) store8<TX, ALIGNED>(a.y, at, now[k], a.dim, d);
            if (a.sum) store8<TR, ALIGNED>(a.sum, at, now[k], a.dim, d);
        }
        first += step;
        turn ^= 1;
    };
    // One chunk a lane: two sets of inputs in turn, so that none is copied.  With two
    // chunks the two unrolled rows spill (419 us against 377 us for forward and
    // gradient of 16384 rows of 5120).
    In in0, in1;
    if (AHEAD && first < a.rows) load(in0, first + sub);
    while (first < a.rows) {
        if constexpr (AHEAD && NV == 1) {
            row_of(in0, in1);
            if (first >= a.rows) break;
            row_of(in1, in0);
        } else {
            in1 = in0;
            row_of(in1, in0);
        }
    }
    float* out = a.partial + (size_t)blockIdx.x * a.dim;
    if constexpr (SMALL) {
        // the rows' lane groups one after another, so that the order is fixed
        for (int i = threadIdx.x; i < a.dim; i += blockDim.x) s_dw[i] = 0.0f;
        for (int g = 0; g < a.rows_per_cta; ++g) {
            __syncthreads();
            if ((int)threadIdx.x / lanes == g && ks[0].any) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (ks[0].i0 + j >= 0 && ks[0].i0 + j < a.dim) s_dw[ks[0].i0 + j] += dw[0][j];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.dim; i += blockDim.x) out[i] = s_dw[i];
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (ks[k].any && ks[k].i0 + j >= 0 && ks[k].i0 + j < a.dim)
                    out[ks[k].i0 + j] = dw[k][j];
    }
}

// dw[c] = sum of the CTAs' partial[i][c] in a fixed order: each warp takes every 32nd
// partial row, ten of them (a GB300's grid) in flight, then warp 0 adds the warps' sums.
constexpr int kDwWarps = 32, kDwAhead = 10;

__global__ void __launch_bounds__(kDwWarps * 32) norm_dw_kernel(const float* partial, int parts,
                                                               int dim, float* dw) {
    __shared__ float acc[kDwWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (c < dim) {
        for (int i = warp; i < parts; i += kDwWarps * kDwAhead) {
            float v[kDwAhead];
#pragma unroll
            for (int k = 0; k < kDwAhead; ++k)
                v[k] = i + kDwWarps * k < parts ? partial[(size_t)(i + kDwWarps * k) * dim + c] : 0.0f;
#pragma unroll
            for (int k = 0; k < kDwAhead; ++k) t += v[k];
        }
    }
    acc[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < dim) {
#pragma unroll
        for (int i = 1; i < kDwWarps; ++i) t += acc[i][lane];
        dw[c] = t;
    }
}

// -------------------------------------------------------------- launch

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

// Chunks of a row: at a shift it reaches into one more.
int row_chunks(int dim) { return (dim + 7) / 8 + (dim % 8 ? 1 : 0); }

// Lanes and warps of a row with nv chunks to a lane.
void row_plan(int dim, int nv, int* lanes, int* warps) {
    const int n = row_chunks(dim);
    *lanes = n <= 8 ? 8 : n <= 16 ? 16 : 32;
    *warps = (n + 32 * nv - 1) / (32 * nv);
}

// The gradient's chunks per lane, its CTA and the most CTAs: their sums of dw are
// written and read once more.  (The workspace's size follows from it, so it does not
// depend on the device: a GB300 has 152 SMs.)
struct BwdPlan {
    int nv, lanes, warps, rows_per_cta, threads, most;
};

BwdPlan bwd_plan(int dim) {
    BwdPlan p;
    const int n = row_chunks(dim);
    p.nv = n <= 512 ? 1 : n <= 1024 ? 2 : 4;  // up to 16 (17) warps
    row_plan(dim, p.nv, &p.lanes, &p.warps);
    const bool small = p.warps == 1 && p.nv == 1;
    p.rows_per_cta = small ? kSmallWarps * (32 / p.lanes) : 1;
    p.threads = 32 * (small ? kSmallWarps : p.warps);
    p.most = 152 * std::max(1, kBwdThreads / p.threads);
    return p;
}

// CTAs step by multiples of 8 rows, so that a lane's columns stay the same
unsigned whole_grid(long long rows, int rows_per_cta, long long most, bool aligned) {
    long long g = std::min((rows + rows_per_cta - 1) / rows_per_cta, most);
    if (!aligned) g = std::max<long long>(8, g / 8 * 8);
    return (unsigned)g;
}

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
    const bool vec = dim % 8 == 0;
    // one chunk a lane up to 32 warps, or the 17 that unaligned rows' registers allow
    const int nv = row_chunks(dim) <= (vec ? 1024 : 544) ? 1 : 4;
    int warps;
    row_plan(dim, nv, &a.lanes, &warps);
    a.warps_per_row = warps;
    const bool small = warps == 1;
    a.rows_per_cta = small ? kSmallWarps * (32 / a.lanes) : 1;
    const int threads = 32 * (small ? kSmallWarps : warps);
    const int sms = ssm_host::sm_count();
    if (sms == 0) return SSM_ERR_CUDA;
    const unsigned grid =
        whole_grid(rows, a.rows_per_cta, (long long)sms * std::max(1, kFwdThreads / threads), vec);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    by_types(in, res, e4m3 ? SSM_F32 : out, [&](auto tx, auto tr, auto ty) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        using TY = decltype(ty);
        auto go = [&](auto kernel) { kernel<<<grid, threads, 0, s>>>(a); };
        auto pick = [&](auto out) {
            constexpr Out O = decltype(out)::value;
            if (small) vec ? go(norm_fwd_kernel<TX, TR, TY, 1, true, true, O>)
                           : go(norm_fwd_kernel<TX, TR, TY, 1, false, true, O>);
            else if (nv == 1) vec ? go(norm_fwd_kernel<TX, TR, TY, 1, true, false, O>)
                                  : go(norm_fwd_kernel<TX, TR, TY, 1, false, false, O>);
            else vec ? go(norm_fwd_kernel<TX, TR, TY, 4, true, false, O>)
                     : go(norm_fwd_kernel<TX, TR, TY, 4, false, false, O>);
        };
        if constexpr (sizeof(TY) == 4) {
            if (e4m3) {
                pick(std::integral_constant<Out, kE4m3>{});
                return;
            }
        }
        pick(std::integral_constant<Out, kPlain>{});
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
    const BwdPlan p = bwd_plan(dim);
    return 256 + (size_t)whole_grid(rows, p.rows_per_cta, p.most, dim % 8 == 0) * dim * 4;
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
    const BwdPlan p = bwd_plan(dim);
    a.lanes = p.lanes;
    a.warps_per_row = p.warps;
    a.rows_per_cta = p.rows_per_cta;
    const bool vec = dim % 8 == 0;
    const int sms = ssm_host::sm_count();
    if (sms == 0) return SSM_ERR_CUDA;
    const unsigned grid = whole_grid(
        rows, p.rows_per_cta, std::min(p.most, sms * std::max(1, kBwdThreads / p.threads)), vec);
    by_types(in_dtype, res_dtype, dy_dtype, [&](auto tx, auto tr, auto ty) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        using TY = decltype(ty);
        auto go = [&](auto kernel) { kernel<<<grid, p.threads, 0, s>>>(a); };
        if (p.rows_per_cta > 1) vec ? go(norm_bwd_kernel<TX, TR, TY, 1, true, true, true>)
                                    : go(norm_bwd_kernel<TX, TR, TY, 1, false, true, true>);
        else if (p.nv == 1) vec ? go(norm_bwd_kernel<TX, TR, TY, 1, true, false, true>)
                                : go(norm_bwd_kernel<TX, TR, TY, 1, false, false, true>);
        else if (p.nv == 2) vec ? go(norm_bwd_kernel<TX, TR, TY, 2, true, false, true>)
                                : go(norm_bwd_kernel<TX, TR, TY, 2, false, false, true>);
        else vec ? go(norm_bwd_kernel<TX, TR, TY, 4, true, false, false>)
                 : go(norm_bwd_kernel<TX, TR, TY, 4, false, false, false>);
    });
    norm_dw_kernel<<<(dim + 31) / 32, kDwWarps * 32, 0, s>>>(a.partial, (int)grid, dim, dweight);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}
