// Rows and weights to e4m3 codes with a float32 scale per 128 columns (of one row, or of 128
// rows), and SwiGLU with such an output (moe_quantize_fp8, moe_swiglu_fp8; declared in
// include/moe_grouped.h).
//
//     a = max(largest |v| of the block, 2^-100);  scale = a / 448;  code = e4m3(v * (448 / a))
//
// Each value is read once and held in registers between the maximum and the codes.  HBM bounds it: 32768 x
// 7168 bf16 rows 114 us, 0.92 of the copy rate, as weights 116 us; SwiGLU of 32768 x 2048 58 us, 0.86, the
// instructions close behind (the schedulers issue in 80% of the cycles).  With live_rows every block reads the
// word, 1 to 2 us (32768 x 2048 59 us), and the blocks of rows that are not taken cost their launch alone: 34 us with
// half of the rows live, 9.5 with none.
#include <cuda_fp8.h>

#include <type_traits>

#include "../../include/moe_grouped.h"
#include "block_common.cuh"

namespace moe {
namespace {

struct QuantArgs {
    const void *x;
    const int32_t *live;      // NULL: all rows
    uint8_t *codes;
    float *scales;
    int64_t stride, R;        // of x in elements; rows of all matrices
    int rows, cols, piece;    // of a matrix; pieces of a row
    int row_blocks;           // BLOCK: blocks of 128 rows in a matrix
};

// 8 columns as they lie in memory, and as floats.  EVEN: they start on a 16-byte boundary.
template <typename T>
struct Raw {
    static constexpr int kVecs = sizeof(T) / 2;
    uint4 v[kVecs];
    template <bool EVEN> __device__ __forceinline__ void load(const T *p) {
        if constexpr (EVEN) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else if constexpr (sizeof(T) == 4) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
            v[0] = make_uint4(w[0], w[1], w[2], w[3]);
            v[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            const uint16_t *w = reinterpret_cast<const uint16_t *>(p);
            v[0] = make_uint4(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16, w[4] | (uint32_t)w[5] << 16,
                              w[6] | (uint32_t)w[7] << 16);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
        if constexpr (sizeof(T) == 4) {
            f[0] = __uint_as_float(v[0].x); f[1] = __uint_as_float(v[0].y);
            f[2] = __uint_as_float(v[0].z); f[3] = __uint_as_float(v[0].w);
            f[4] = __uint_as_float(v[1].x); f[5] = __uint_as_float(v[1].y);
            f[6] = __uint_as_float(v[1].z); f[7] = __uint_as_float(v[1].w);
        } else {
            f[0] = lo_f32(v[0].x); f[1] = hi_f32(v[0].x); f[2] = lo_f32(v[0].y); f[3] = hi_f32(v[0].y);
            f[4] = lo_f32(v[0].z); f[5] = hi_f32(v[0].z); f[6] = lo_f32(v[0].w); f[7] = hi_f32(v[0].w);
        }
    }
};

__device__ __forceinline__ float largest(const float (&f)[8]) {
    float m = 0.f;   // (fmaxf passes over what is not a number)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
    return m;
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(f[2 * j], inv), __fmul_rn(f[2 * j + 1], inv)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// g / (1 + exp(-g)).  The exponential is the hardware's power of two of the rounded product
// t = -g log2(e), times 1 + (what the rounding of t left out) ln 2: without that factor its error
// would grow with |g|.  Both are taken of g held within 88.71: from there on t and its remainder are no
// longer a product and a small rest of it, while e at 88.71, 2^127.98, has a reciprocal below the
// normal numbers, which the instruction gives as 0.  So silu is 0 for finite g below -87.3 (1 / (1 + exp(-g))
// is below 2^-126 there, and silu is above -2^-119), NaN at -infinity as in the formula, and g from 88.71 on.
// The remainder's part is added to 1 + e: added to e first it lengthens the chain (32768 x 2048 59.4 us for
// 57.9).  (The hardware's forms that keep numbers below the normal ones take several instructions each; with
// them 87 us.)
__device__ __forceinline__ float silu(float g) {
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f, kEnd = 88.71f;
    constexpr float kLog2eRest = 1.4426950408889634 - (double)kLog2e;   // of the constant's own rounding
    const float h = fminf(fmaxf(g, -kEnd), kEnd), t = -h * kLog2e;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    const float rest = fmaf(-h, kLog2eRest, fmaf(-h, kLog2e, -t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, rest * kLn2, 1.f + e)));
    return g * r;
}

constexpr int kQuantThreads = 256;
constexpr int kQuantUnits = 2;   // runs of 8 columns of a thread

// A warp takes one piece of a row, 16 lanes to a block of 128 columns.
template <typename T, bool EVEN, bool SWIGLU>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(QuantArgs a) {
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = i / a.piece;
    if (row >= a.R || (a.live && row >= *a.live)) return;
    const int c0 = ((int)(i - row * a.piece) * 32 * kQuantUnits + (threadIdx.x & 31)) * 8;
    const T *x = static_cast<const T *>(a.x) + row * a.stride;
    Raw<T> raw[kQuantUnits], raw_up[SWIGLU ? kQuantUnits : 1];
#pragma unroll
    for (int u = 0; u < kQuantUnits; ++u) {
        const int c = c0 + 256 * u;
        if (c < a.cols) {
            raw[u].template load<EVEN>(x + c);
            if (SWIGLU) raw_up[SWIGLU ? u : 0].template load<EVEN>(x + a.cols + c);
        } else {
            raw[u].zero();
            raw_up[SWIGLU ? u : 0].zero();
        }
    }
    float f[kQuantUnits][8], m[kQuantUnits];
#pragma unroll
    for (int u = 0; u < kQuantUnits; ++u) {
        raw[u].floats(f[u]);
        if (SWIGLU) {
            float up[8];
            raw_up[SWIGLU ? u : 0].floats(up);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[u][j] = silu(f[u][j]) * up[j];
        }
        m[u] = largest(f[u]);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m[u] = fmaxf(m[u], __shfl_xor_sync(kAllLanes, m[u], o));
        m[u] = fmaxf(m[u], 0x1p-100f);
    }
    // The two blocks' four quotients by one division: lanes 0 and 1 of every 16 have the factors, 2 and
    // 3 the scales.
    static_assert(kQuantUnits == 2, "four quotients");
    const int lane = threadIdx.x & 15;
    const float mine = lane & 1 ? m[1] : m[0];
    const float q = __fdiv_rn(lane & 2 ? mine : 448.f, lane & 2 ? 448.f : mine);
#pragma unroll
    for (int u = 0; u < kQuantUnits; ++u) {
        const int c = c0 + 256 * u;
        const float inv = __shfl_sync(kAllLanes, q, u, 16);
        if (c >= a.cols) continue;
        *reinterpret_cast<uint2 *>(a.codes + row * a.cols + c) = codes8(f[u], inv);
        if (lane == 2 + u) a.scales[row * (a.cols >> 7) + (c >> 7)] = q;
    }
}

// A block takes 128 rows of 128 columns: 16 threads to a row, 16 rows at a time.
// (Four blocks to an SM, 64 registers to a thread: some of the values that are held between the maximum and the
// codes go through local memory, 104 to 120 bytes a thread.)
template <typename T, bool EVEN>
__global__ void __launch_bounds__(256, 4) quantize_blocks_kernel(QuantArgs a) {
    __shared__ float red[8];
    pdl_wait();
    const int cb = a.cols >> 7;
    const int64_t i = blockIdx.x, block = i / cb, matrix = block / a.row_blocks;
    const int b = (int)(i - block * cb), r0 = (int)(block - matrix * a.row_blocks) * 128 + (threadIdx.x >> 4);
    const int c = b * 128 + (threadIdx.x & 15) * 8;
    Raw<T> raw[8];
    float f[8], m = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        if (r0 + 16 * u < a.rows)
            raw[u].template load<EVEN>(static_cast<const T *>(a.x) + (matrix * a.rows + r0 + 16 * u) * a.stride + c);
        else raw[u].zero();
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        raw[u].floats(f);
        m = fmaxf(m, largest(f));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    m = fmaxf(m, 0x1p-100f);
    const float inv = __fdiv_rn(448.f, m);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        raw[u].floats(f);
        if (r0 + 16 * u < a.rows)
            *reinterpret_cast<uint2 *>(a.codes + (matrix * a.rows + r0 + 16 * u) * a.cols + c) = codes8(f, inv);
    }
    if (threadIdx.x == 0) a.scales[block * cb + b] = __fdiv_rn(m, 448.f);
}

int quantize(const moe_quantize *q, const void *x, const int32_t *live, uint8_t *codes, float *scales, bool swiglu,
             cudaStream_t s) {
    if (!q || q->num_rows < 0 || q->cols < 1 || q->matrices < 1 || bad_dtype(q->x_dtype) ||
        (q->block_rows != 1 && (q->block_rows != 128 || swiglu)))
        return MOE_ERR_INVALID_ARGUMENT;
    if (live && (q->block_rows != 1 || q->matrices != 1)) return MOE_ERR_INVALID_ARGUMENT;
    if (q->cols % 128) return MOE_ERR_HIDDEN_ALIGNMENT;
    if (q->cols > MOE_MAX_HIDDEN) return MOE_ERR_LIMIT;
    const int64_t width = (int64_t)q->cols * (swiglu ? 2 : 1), stride = q->x_stride ? q->x_stride : width;
    if (stride < width) return MOE_ERR_INVALID_ARGUMENT;
    const int64_t R = (int64_t)q->matrices * q->num_rows, b = (int64_t)dtype_bytes(q->x_dtype);
    if (R > 0 && (!x || !codes || !scales)) return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(x, b) || !is_aligned(live, 4) || !is_aligned(codes, 16) || !is_aligned(scales, 4))
        return MOE_ERR_MISALIGNED;
    const int rc = check_device();
    if (rc != MOE_OK) return rc;
    if (R == 0) return MOE_OK;
    const bool even = is_aligned(x, 16) && stride * b % 16 == 0;
    QuantArgs a{x, live, codes, scales, stride, R, q->num_rows, q->cols, 0, 0};
    int64_t blocks;
    if (q->block_rows == 128) {
        a.row_blocks = (q->num_rows + 127) / 128;
        blocks = (int64_t)q->matrices * a.row_blocks * (q->cols / 128);
    } else {
        constexpr int piece = 256 * kQuantUnits;
        a.piece = (q->cols + piece - 1) / piece;
        blocks = (R * a.piece + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    }
    if (blocks >= ((int64_t)1 << 31)) return MOE_ERR_LIMIT;
    auto run = [&](auto t, auto ev) {
        using T = decltype(t);
        constexpr bool E = decltype(ev)::value;
        auto *kernel = q->block_rows == 128 ? quantize_blocks_kernel<T, E>
                       : swiglu             ? quantize_rows_kernel<T, E, true>
                                            : quantize_rows_kernel<T, E, false>;
        return status_of(launch_pdl(kernel, dim3((unsigned)blocks), dim3(kQuantThreads), 0, s, a));
    };
    const bool f32 = q->x_dtype == MOE_DTYPE_FP32;
    if (even) return f32 ? run(float{}, std::true_type{}) : run(__nv_bfloat16{}, std::true_type{});
    return f32 ? run(float{}, std::false_type{}) : run(__nv_bfloat16{}, std::false_type{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_quantize_fp8(const moe_quantize *q, const void *x_dev, const int32_t *live_rows_dev,
                                uint8_t *codes_dev, float *scales_dev, void *stream) {
    return quantize(q, x_dev, live_rows_dev, codes_dev, scales_dev, false, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_swiglu_fp8(const moe_quantize *q, const void *gate_up_dev, const int32_t *live_rows_dev,
                              uint8_t *codes_dev, float *scales_dev, void *stream) {
    return quantize(q, gate_up_dev, live_rows_dev, codes_dev, scales_dev, true, static_cast<cudaStream_t>(stream));
}
