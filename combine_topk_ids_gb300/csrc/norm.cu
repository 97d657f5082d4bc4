// Residual addition and root-mean-square norm in front of the expert layer, and its gradient
// (moe_add_rmsnorm, moe_add_rmsnorm_backward; declared in include/moe_block.h).
//
// Forward, one row of H columns:  h = x + r;  rstd = 1/sqrt(sum(h^2)/H + eps);
// y = h*rstd*w, stored as bf16, as e4m3 codes with a scale per 128 columns, or both.
// A row is read once and held in registers between the sum of squares and the scaling, so
// the call moves what it has to: x, r in; h, y out.  HBM bounds it.
#include <cuda_fp8.h>

#include "block_common.cuh"

namespace moe {
namespace {

constexpr int kMaxParts = 304;   // row blocks that write a partial dweight (two per SM)

struct NormArgs {
    const void *x, *res, *w;
    void *sum, *out;
    uint8_t *q;
    float *scales, *rstd;
    int64_t xs, rs, ss, os;   // row strides in elements
    int T, H;
    float eps;
    unsigned shift_mask;      // 15: chunks follow the 16-byte boundaries of x's rows; 0: columns
};

// Columns [i, i + 8) of a row, in the row's own type.  load() issues one 16-byte load (two for
// float32) where they all exist and the address allows it, and nothing else, so that a
// thread's loads are under way together; floats() fetches what load() could not: the columns
// of [0, H) one by one, 0 outside.
template <bool F32>
struct Raw8 {
    uint4 v[F32 ? 2 : 1];

    static __device__ __forceinline__ bool whole(const void *row, int i, int H) {
        return i >= 0 && i + 8 <= H && ((reinterpret_cast<uintptr_t>(row) + (int64_t)i * (F32 ? 4 : 2)) & 15) == 0;
    }
    __device__ __forceinline__ void load(const void *row, int i, int H) {
        if (whole(row, i, H)) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + (int64_t)i * (F32 ? 4 : 2));
            v[0] = p[0];
            if (F32) v[F32 ? 1 : 0] = p[1];
        }
    }
    __device__ __forceinline__ void floats(const void *row, int i, int H, float (&f)[8]) const {
        if (F32) {
            const uint4 &a = v[0], &b = v[F32 ? 1 : 0];
            f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
            f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
        } else {
            const uint4 &a = v[0];
            f[0] = lo_f32(a.x); f[1] = hi_f32(a.x); f[2] = lo_f32(a.y); f[3] = hi_f32(a.y);
            f[4] = lo_f32(a.z); f[5] = hi_f32(a.z); f[6] = lo_f32(a.w); f[7] = hi_f32(a.w);
        }
        if (!whole(row, i, H)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[j] = 0.f;
                if (i + j >= 0 && i + j < H)
                    f[j] = F32 ? static_cast<const float *>(row)[i + j]
                               : __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[i + j]);
            }
        }
    }
};

template <bool F32>
__device__ __forceinline__ void store8(void *row, int i, int H, const float (&f)[8]) {
    if (Raw8<F32>::whole(row, i, H)) {
        if (F32) {
            float *p = static_cast<float *>(row) + i;
            *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(row) + i) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j >= 0 && i + j < H) {
                if (F32) static_cast<float *>(row)[i + j] = f[j];
                else static_cast<__nv_bfloat16 *>(row)[i + j] = __float2bfloat16_rn(f[j]);
            }
    }
}

// Sum over the threads of one row (blockDim.x of them), the same bits in each.
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    float *mine = red + threadIdx.y * nw;
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < nw; ++i) v += mine[i];
    return v;
}

// e4m3 codes of 8 columns of a 128-column block that 16 lanes hold.  All lanes call it.
__device__ __forceinline__ uint2 quant8(const float (&y)[8], float &scale) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, o));
    const float a = fmaxf(m, 0x1p-100f);
    scale = __fdiv_rn(a, 448.0f);
    const float inv = __fdiv_rn(448.0f, a);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[2 * j], inv), __fmul_rn(y[2 * j + 1], inv)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// blockDim.x threads per row, VPT chunks of 8 columns each, blockDim.y rows per block.
// Chunk c covers columns [8c - s, 8c - s + 8), where s is the number of elements by which
// the row of x starts behind a 16-byte boundary: packed rows of an odd length start at any
// offset, and the chunks then still lie on 16-byte boundaries, the row's ends apart.
template <int VPT, int MAXT, bool R32, bool W32>
__global__ void __launch_bounds__(MAXT) add_rmsnorm_kernel(NormArgs a) {
    __shared__ float red[32];
    pdl_begin();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < a.T;   // rows past the end take part in the block's barrier only
    const int H = live ? a.H : 0;
    const int64_t tr = live ? t : 0;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + tr * a.xs;
    const char *res = a.res ? static_cast<const char *>(a.res) + tr * a.rs * (R32 ? 4 : 2) : nullptr;
    const int s = (int)((reinterpret_cast<uintptr_t>(x) & a.shift_mask) >> 1);
    Raw8<false> rx[VPT];
    Raw8<R32> rr[VPT];
    Raw8<W32> rw[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = 8 * (int)(threadIdx.x + v * blockDim.x) - s;
        rx[v].load(x, i, H);
        if (res) rr[v].load(res, i, H);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) rw[v].load(a.w, 8 * (int)(threadIdx.x + v * blockDim.x) - s, H);
    float h[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = 8 * (int)(threadIdx.x + v * blockDim.x) - s;
        rx[v].floats(x, i, H, h[v]);
        if (res) {
            float r[8];
            rr[v].floats(res, i, H, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[v][j] += r[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[v][j], h[v][j], ss);
    }
    ss = row_sum(ss, red);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)a.H) + a.eps));
    if (live && threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = 8 * (int)(threadIdx.x + v * blockDim.x) - s;
        if (a.sum) store8<R32>(static_cast<char *>(a.sum) + tr * a.ss * (R32 ? 4 : 2), i, H, h[v]);
        float w[8];
        rw[v].floats(a.w, i, H, w);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[v][j] * rstd * w[j];
        if (a.out) store8<false>(static_cast<__nv_bfloat16 *>(a.out) + tr * a.os, i, H, y);
        if (a.q) {
            float sc;
            const uint2 c = quant8(y, sc);
            if (i < H) {
                *reinterpret_cast<uint2 *>(a.q + tr * a.H + i) = c;
                if ((i & 127) == 0) a.scales[tr * (a.H >> 7) + (i >> 7)] = sc;
            }
        }
    }
}

struct NormBackArgs {
    const void *dout, *h, *w, *dsum;
    void *dx;
    const float *rstd;
    float *part;              // [gridDim.x][H]
    int64_t ds, hs, ss, os;   // row strides in elements
    int T, H;
};

// Each block takes every gridDim.x-th group of blockDim.y rows and keeps its columns' sums of
// dout * xhat in registers; they leave as one row of `part`.
template <int VPT, int MAXT, bool R32, bool W32>
__global__ void __launch_bounds__(MAXT) add_rmsnorm_backward_kernel(NormBackArgs a) {
    __shared__ float red[32];
    extern __shared__ float cols[];   // [H] when blockDim.y > 1
    pdl_begin();
    float dw[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[v][j] = 0.f;
    Raw8<W32> rw[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) rw[v].load(a.w, 8 * (int)(threadIdx.x + v * blockDim.x), a.H);
    Raw8<false> rg[VPT];
    Raw8<R32> rh[VPT], rs[VPT];
    float rstd = 0.f;
    // row t's inputs under way, while the row before it is computed
    auto fetch = [&](int64_t t) {
        const int H = t < a.T ? a.H : 0;
        const int64_t tr = t < a.T ? t : 0;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = 8 * (int)(threadIdx.x + v * blockDim.x);
            rg[v].load(static_cast<const __nv_bfloat16 *>(a.dout) + tr * a.ds, i, H);
            rh[v].load(static_cast<const char *>(a.h) + tr * a.hs * (R32 ? 4 : 2), i, H);
            if (a.dsum) rs[v].load(static_cast<const char *>(a.dsum) + tr * a.ss * (R32 ? 4 : 2), i, H);
        }
        rstd = t < a.T ? a.rstd[t] : 0.f;
    };
    const int64_t groups = ((int64_t)a.T + blockDim.y - 1) / blockDim.y;
    fetch((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
    for (int64_t gr = blockIdx.x; gr < groups; gr += gridDim.x) {
        const int64_t t = gr * blockDim.y + threadIdx.y;
        const int H = t < a.T ? a.H : 0;
        const int64_t tr = t < a.T ? t : 0;
        const float rt = rstd;
        float g[VPT][8], xh[VPT][8];
        float along = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = 8 * (int)(threadIdx.x + v * blockDim.x);
            float w[8];
            rg[v].floats(static_cast<const __nv_bfloat16 *>(a.dout) + tr * a.ds, i, H, g[v]);
            rh[v].floats(static_cast<const char *>(a.h) + tr * a.hs * (R32 ? 4 : 2), i, H, xh[v]);
            rw[v].floats(a.w, i, H, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[v][j] *= rt;
                dw[v][j] = fmaf(g[v][j], xh[v][j], dw[v][j]);
                g[v][j] *= w[j];
                along = fmaf(g[v][j], xh[v][j], along);
            }
        }
        along = row_sum(along, red) / (float)a.H;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[v][j] = rt * (g[v][j] - xh[v][j] * along);
            if (a.dsum) {
                float d[8];
                rs[v].floats(static_cast<const char *>(a.dsum) + tr * a.ss * (R32 ? 4 : 2),
                             8 * (int)(threadIdx.x + v * blockDim.x), H, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[v][j] += d[j];
            }
        }
        fetch((gr + gridDim.x) * blockDim.y + threadIdx.y);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            store8<R32>(static_cast<char *>(a.dx) + tr * a.os * (R32 ? 4 : 2), 8 * (int)(threadIdx.x + v * blockDim.x),
                        H, g[v]);
        __syncthreads();   // before the next rows write red
    }
    float *part = a.part + (int64_t)blockIdx.x * a.H;
    if (blockDim.y == 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) store8<true>(part, 8 * (int)(threadIdx.x + v * blockDim.x), a.H, dw[v]);
        return;
    }
    for (int y = 0; y < (int)blockDim.y; ++y) {   // the rows' sums in a fixed order
        if ((int)threadIdx.y == y) {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 8 * (int)(threadIdx.x + v * blockDim.x) + j;
                    if (i < a.H) cols[i] = (y ? cols[i] : 0.f) + dw[v][j];
                }
        }
        __syncthreads();
    }
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < a.H; i += blockDim.x * blockDim.y) part[i] = cols[i];
}

// dweight = sum of the partial rows: 32 columns per block, row r of `part` on thread row r % 32.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float *part, float *dw, int parts, int H) {
    __shared__ float tile[32][33];
    pdl_begin();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (c < H)
        for (int r = threadIdx.y; r < parts; r += 32) v += part[(int64_t)r * H + c];
    tile[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || c >= H) return;
    v = 0.f;
    for (int r = 0; r < 32; ++r) v += tile[r][threadIdx.x];
    dw[c] = v;
}

struct NormShape {
    int vpt, threads, rows;   // chunks per thread, threads per row, rows per block
};

// Chunks of 8 columns spread over whole warps: 2 per thread up to 4096 columns, 4 up to 8192,
// 8 above; short rows share a block of about 256 threads.
NormShape norm_shape(int64_t chunks) {
    NormShape n;
    n.vpt = chunks <= 512 ? 2 : chunks <= 1024 ? 4 : 8;
    n.threads = (int)((chunks + 32 * n.vpt - 1) / (32 * n.vpt)) * 32;
    n.rows = n.threads >= 256 ? 1 : 256 / n.threads;
    return n;
}

// The gradient holds more for each column (the column's sum, a second input): 2 chunks per
// thread up to 8192 columns, 4 up to 16384, 8 above.
NormShape norm_back_shape(int64_t chunks) {
    NormShape n;
    n.vpt = chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
    n.threads = (int)((chunks + 32 * n.vpt - 1) / (32 * n.vpt)) * 32;
    n.rows = n.threads >= 256 ? 1 : 256 / n.threads;
    return n;
}

int check_norm(const moe_norm *n) {
    if (!n) return MOE_ERR_INVALID_ARGUMENT;
    if (n->num_tokens < 0 || n->hidden < 1 || bad_dtype(n->residual_dtype) || bad_dtype(n->weight_dtype) ||
        !(n->eps >= 0.f))
        return MOE_ERR_INVALID_ARGUMENT;
    for (int64_t s : {n->x_stride, n->residual_stride, n->sum_stride, n->out_stride})
        if (s != 0 && s < n->hidden) return MOE_ERR_INVALID_ARGUMENT;
    return n->hidden > MOE_MAX_HIDDEN ? MOE_ERR_LIMIT : MOE_OK;
}

int64_t stride_of(const moe_norm *n, int64_t s) { return s ? s : n->hidden; }

int backward_blocks(const moe_norm *n, const NormShape &sh) {
    const int64_t groups = ((int64_t)n->num_tokens + sh.rows - 1) / sh.rows;
    return (int)(groups < kMaxParts ? groups : kMaxParts);
}

template <int VPT, int MAXT>
struct Shape {
    static constexpr int vpt = VPT, maxt = MAXT;
};

template <bool BACK, typename F>
cudaError_t with_shape(const NormShape &sh, bool r32, bool w32, F &&f) {
    auto types = [&](auto v) {
        if (r32) return w32 ? f(v, std::true_type{}, std::true_type{}) : f(v, std::true_type{}, std::false_type{});
        return w32 ? f(v, std::false_type{}, std::true_type{}) : f(v, std::false_type{}, std::false_type{});
    };
    constexpr int wide = BACK ? 512 : 256;   // threads a row takes at most below the largest shape
    if (sh.vpt == 2) return sh.threads <= 256 ? types(Shape<2, 256>{}) : types(Shape<2, wide>{});
    if (sh.vpt == 4) return types(Shape<4, wide>{});
    if (!BACK && sh.threads <= 256) return types(Shape<8, 256>{});
    return types(Shape<8, 1024>{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_add_rmsnorm(const moe_norm *n, const void *x_dev, const void *residual_dev, const void *weight_dev,
                    void *sum_dev, void *out_dev, void *out_fp8_dev, float *scales_dev, float *rstd_dev,
                    void *stream) {
    int rc = check_norm(n);
    if (rc != MOE_OK) return rc;
    if (n->num_tokens > 0 && (!x_dev || !weight_dev || (!out_dev && !out_fp8_dev) || !out_fp8_dev != !scales_dev))
        return MOE_ERR_INVALID_ARGUMENT;
    if (out_fp8_dev && n->hidden % 128 != 0) return MOE_ERR_HIDDEN_ALIGNMENT;
    if (!is_aligned(x_dev, 2) || !is_aligned(residual_dev, dtype_bytes(n->residual_dtype)) ||
        !is_aligned(weight_dev, dtype_bytes(n->weight_dtype)) || !is_aligned(out_dev, 2) ||
        !is_aligned(sum_dev, dtype_bytes(n->residual_dtype)) || !is_aligned(out_fp8_dev, 16) ||
        !is_aligned(scales_dev, 4) || !is_aligned(rstd_dev, 4))
        return MOE_ERR_MISALIGNED;
    if ((rc = check_device()) != MOE_OK) return rc;
    if (n->num_tokens == 0) return MOE_OK;
    NormArgs a{x_dev, residual_dev, weight_dev, sum_dev, out_dev, static_cast<uint8_t *>(out_fp8_dev),
               scales_dev, rstd_dev, stride_of(n, n->x_stride), stride_of(n, n->residual_stride),
               stride_of(n, n->sum_stride), stride_of(n, n->out_stride), n->num_tokens, n->hidden, n->eps, 0};
    // rows that may start off a 16-byte boundary need up to 7 columns of room before the first
    // (not where that is one chunk more than a block holds, nor with codes, whose blocks are fixed)
    const bool even = out_fp8_dev || (is_aligned(x_dev, 16) && a.xs % 8 == 0) || n->hidden > MOE_MAX_HIDDEN - 8;
    a.shift_mask = even ? 0 : 15;
    const NormShape sh = norm_shape(((int64_t)n->hidden + (even ? 0 : 7) + 7) / 8);
    const dim3 grid((unsigned)(((int64_t)a.T + sh.rows - 1) / sh.rows)), block(sh.threads, sh.rows);
    return status_of(with_shape<false>(sh, n->residual_dtype == MOE_DTYPE_FP32, n->weight_dtype == MOE_DTYPE_FP32,
                                [&](auto v, auto r32, auto w32) {
                                    return launch_pdl(add_rmsnorm_kernel<decltype(v)::vpt, decltype(v)::maxt,
                                                                         decltype(r32)::value, decltype(w32)::value>,
                                                      grid, block, 0, static_cast<cudaStream_t>(stream), a);
                                }));
}

int moe_add_rmsnorm_workspace_size(const moe_norm *n, size_t *bytes) {
    int rc = check_norm(n);
    if (rc != MOE_OK) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
    *bytes = (size_t)kMaxParts * (size_t)n->hidden * 4;
    return MOE_OK;
}

int moe_add_rmsnorm_backward(const moe_norm *n, const void *dout_dev, const void *h_dev, const void *weight_dev,
                             const float *rstd_dev, const void *dsum_dev, void *dx_dev, float *dweight_dev,
                             void *workspace_dev, size_t workspace_bytes, void *stream) {
    size_t need = 0;
    int rc = moe_add_rmsnorm_workspace_size(n, &need);
    if (rc != MOE_OK) return rc;
    if (!dweight_dev || !workspace_dev ||
        (n->num_tokens > 0 && (!dout_dev || !h_dev || !weight_dev || !rstd_dev || !dx_dev)))
        return MOE_ERR_INVALID_ARGUMENT;
    const size_t rb = dtype_bytes(n->residual_dtype);
    if (!is_aligned(dout_dev, 2) || !is_aligned(h_dev, rb) || !is_aligned(weight_dev, dtype_bytes(n->weight_dtype)) ||
        !is_aligned(rstd_dev, 4) || !is_aligned(dsum_dev, rb) || !is_aligned(dx_dev, rb) ||
        !is_aligned(dweight_dev, 4) || !is_aligned(workspace_dev, 256))
        return MOE_ERR_MISALIGNED;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if ((rc = check_device()) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const NormShape sh = norm_back_shape(((int64_t)n->hidden + 7) / 8);
    const int blocks = backward_blocks(n, sh);
    float *part = static_cast<float *>(workspace_dev);
    if (blocks > 0) {
        NormBackArgs a{dout_dev, h_dev, weight_dev, dsum_dev, dx_dev, rstd_dev, part, stride_of(n, n->x_stride),
                       stride_of(n, n->residual_stride), stride_of(n, n->sum_stride),
                       stride_of(n, n->out_stride), n->num_tokens, n->hidden};
        const size_t smem = sh.rows > 1 ? (size_t)n->hidden * 4 : 0;   // at most 8 KB: rows > 1 below 2048 columns
        const cudaError_t e = with_shape<true>(
            sh, n->residual_dtype == MOE_DTYPE_FP32, n->weight_dtype == MOE_DTYPE_FP32,
            [&](auto v, auto r32, auto w32) {
                return launch_pdl(add_rmsnorm_backward_kernel<decltype(v)::vpt, decltype(v)::maxt,
                                                              decltype(r32)::value, decltype(w32)::value>,
                                  dim3(blocks), dim3(sh.threads, sh.rows), smem, s, a);
            });
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return status_of(launch_pdl(sum_parts_kernel, dim3((n->hidden + 31) / 32), dim3(32, 32), 0, s,
                                (const float *)part, dweight_dev, blocks, (int)n->hidden));
}

}  // extern "C"
