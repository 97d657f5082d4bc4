// Residual addition and root-mean-square norm in front of the expert layer (moe_add_rmsnorm;
// declared in include/moe_block.h).
//
// One row of H columns:  h = x + r;  rstd = 1/sqrt(sum(h^2)/H + eps);  y = h*rstd*w, stored as
// bf16, as e4m3 codes with a scale per 128 columns, or both.
// A row is read once and held in registers between the sum of squares and the scaling, so the
// call moves what it has to: x, r in; h, y out.  HBM bounds it.  Measured: 32768 rows of 7168
// columns to bf16 and e4m3 (2.12 GB) 330 us, 6.4 TB/s, 0.96 of the measured peak (a block per
// row without the next row under way: 355 us); to bf16 alone 296 us (0.95), with a float32 stream
// 454 us (0.93); one row of 7168 3.3 us.
// 4999 rows of 2047 columns (81.9 MB), off 16-byte boundaries, 22 us (0.55): no unit is full.  8
// blocks of 160 threads fit an SM (48 registers), the schedulers issue in 66% of the active
// cycles, the load pipe is busy in 57%, and the longest stall is for loads: latency and
// instructions share the time.  Above 16384 columns a block of 1024 threads has 64 registers for 64
// columns a thread and keeps a part of the row in local memory: 1000 rows of 20000 112 us (0.21).
#include <cuda_fp8.h>

#include "norm.cuh"

namespace moe {
namespace {

struct NormArgs {
    const void *x, *res, *w;
    void *sum, *out;
    uint8_t *q;
    float *scales, *rstd;
    int64_t xs, rs, ss, os;   // row strides in elements
    int T, H;
    float eps;
    int shift;                // ODD: chunks follow the 16-byte boundaries of x's rows
};

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

// blockDim.x threads per row, VPT chunks of 8 columns each, blockDim.y rows per block; a block
// takes every gridDim.x-th group of rows, and the next row's inputs are under way while one is
// computed.
// ODD: some rows are off 16-byte boundaries (packed rows of an odd length start at any offset).
// Chunk c then covers columns [8c - s, 8c - s + 8), where s is the number of elements by which
// the row of x starts behind a boundary: x, and what lies as x does, is still read and written
// 16 bytes at a time, the row's ends apart.  (A block then takes one group: what the next row's
// inputs would hold of registers gives more blocks instead.)
template <int VPT, int MAXT, bool R32, bool W32, bool ODD>
__global__ void __launch_bounds__(MAXT, MAXT > 256 ? 1 : 8 / VPT < 3 ? 8 / VPT : ODD ? 5 : 2) add_rmsnorm_kernel(NormArgs a) {
    __shared__ float red[2][32];
    pdl_begin();
    const int64_t groups = ((int64_t)a.T + blockDim.y - 1) / blockDim.y, step = (int64_t)gridDim.x * blockDim.y;
    int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    Raw8<false, ODD> rx[VPT];
    Raw8<R32, ODD> rr[VPT];
    Raw8<W32, ODD> rw[ODD ? 1 : VPT];
    auto x = [&](int64_t t) { return static_cast<const __nv_bfloat16 *>(a.x) + (t < a.T ? t : 0) * a.xs; };
    auto res = [&](int64_t t) { return static_cast<const char *>(a.res) + (t < a.T ? t : 0) * a.rs * (R32 ? 4 : 2); };
    auto columns = [&](int64_t t) { return t < a.T ? a.H : 0; };   // rows past the end have none
    auto column = [&](int64_t t, int v) {
        return 8 * (int)(threadIdx.x + v * blockDim.x) - (ODD && a.shift ? (int)((reinterpret_cast<uintptr_t>(x(t)) & 15) >> 1) : 0);
    };
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            rx[v].load(x(t), column(t, v), columns(t));
            if (a.res) rr[v].load(res(t), column(t, v), columns(t));
        }
    };
    if (!ODD)
#pragma unroll
        for (int v = 0; v < VPT; ++v) rw[v].load(a.w, column(t, v), a.H);
    if (!ODD) fetch(t);
    int turn = 0;
    for (int64_t gr = blockIdx.x; gr < groups; gr += gridDim.x, t += step) {
        const int H = columns(t);
        const int64_t tr = t < a.T ? t : 0;
        float h[VPT][8];
        float ss = 0.f;
        if (ODD) fetch(t);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            rx[v].floats(x(t), column(t, v), H, h[v]);
            if (a.res) {
                float r[8];
                rr[v].floats(res(t), column(t, v), H, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[v][j] += r[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(h[v][j], h[v][j], ss);
        }
        if (!ODD) fetch(t + step);   // (sum and out may lie over residual and x: their next rows are other rows)
        ss = row_sum(ss, red[turn]);   // (two turns: the last row's sums are read until the next barrier)
        turn ^= 1;
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)a.H) + a.eps));
        if (t < a.T && threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = column(t, v);
            if (a.sum) store8<R32, ODD>(static_cast<char *>(a.sum) + tr * a.ss * (R32 ? 4 : 2), i, H, h[v]);
            float w[8];
            if (ODD) rw[0].load(a.w, i, H);
            rw[ODD ? 0 : v].floats(a.w, i, H, w);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = h[v][j] * rstd * w[j];
            if (a.out) store8<false, ODD>(static_cast<__nv_bfloat16 *>(a.out) + tr * a.os, i, H, y);
            if (a.q) {   // (a.shift is 0 then)
                float sc;
                const uint2 c = quant8(y, sc);
                if (i < H) {
                    *reinterpret_cast<uint2 *>(a.q + tr * a.H + i) = c;
                    if ((i & 127) == 0) a.scales[tr * (a.H >> 7) + (i >> 7)] = sc;
                }
            }
        }
        if (ODD) break;
    }
}

// 2 chunks of 8 columns per thread up to 4096 columns, 4 up to 8192, 8 above.
NormShape norm_shape(int64_t chunks) { return spread(chunks, chunks <= 512 ? 2 : chunks <= 1024 ? 4 : 8); }

template <typename F>
cudaError_t with_shape(const NormShape &sh, bool r32, bool w32, bool odd, F &&f) {
    if (sh.vpt == 2) return with_types(Shape<2, 256>{}, r32, w32, odd, f);
    if (sh.vpt == 4) return with_types(Shape<4, 256>{}, r32, w32, odd, f);
    if (sh.threads <= 256) return with_types(Shape<8, 256>{}, r32, w32, odd, f);
    return with_types(Shape<8, 1024>{}, r32, w32, odd, f);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_add_rmsnorm(const moe_norm *n, const void *x_dev, const void *residual_dev, const void *weight_dev,
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
    const size_t rb = dtype_bytes(n->residual_dtype);
    const bool odd = n->hidden % 8 || !is_aligned(weight_dev, 16) || !even_rows(x_dev, a.xs, 2) ||
                     !even_rows(residual_dev, a.rs, rb) || !even_rows(sum_dev, a.ss, rb) || !even_rows(out_dev, a.os, 2);
    // Rows of x off a boundary need up to 7 columns of room before the first (not where that is
    // one chunk more than a block holds, nor with codes, whose blocks are fixed).
    a.shift = !even_rows(x_dev, a.xs, 2) && !out_fp8_dev && n->hidden <= MOE_MAX_HIDDEN - 8;
    const NormShape sh = norm_shape(((int64_t)n->hidden + (a.shift ? 7 : 0) + 7) / 8);
    const int64_t groups = ((int64_t)a.T + sh.rows - 1) / sh.rows;
    return status_of(with_shape(
        sh, n->residual_dtype == MOE_DTYPE_FP32, n->weight_dtype == MOE_DTYPE_FP32, odd,
        [&](auto v, auto r32, auto w32, auto odd) {
            constexpr auto kernel = add_rmsnorm_kernel<decltype(v)::vpt, decltype(v)::maxt, decltype(r32)::value,
                                                       decltype(w32)::value, decltype(odd)::value>;
            const int64_t most = decltype(odd)::value ? groups : resident_blocks<kernel>(sh.threads * sh.rows);
            return launch_pdl(kernel, dim3((unsigned)(groups < most ? groups : most)), dim3(sh.threads, sh.rows), 0,
                              static_cast<cudaStream_t>(stream), a);
        }));
}
