// The routed experts' SwiGLU FFN of a decode batch with 4-bit weights (moe_forward_w4), the
// weights' one-time order (moe_prepare_weights_w4) and their quantisation (moe_quantize_w4);
// declared in include/moe_block.h.
//
//     out[t] = sum_j w[t, j] * W2_e (silu(Wg_e x[t]) * (Wu_e x[t])),   W = (code - 8) * scale
//
// A decode batch has few rows for each expert, so the time is that of reading the picked
// experts' codes once.  They feed warp-level matrix instructions (16 weight rows x 16 inputs
// x 8 batch rows, bf16 with float32 sums) straight from global memory: the prepared order
// gives each lane the 32 weights of its matrix fragments for 64 inputs in one 16-byte load,
// 512 contiguous bytes for the warp.  Codes become bf16 integers without rounding; the sums
// over a group of inputs are multiplied by its scale in float32.
#include "block_common.cuh"

namespace moe {
namespace {

constexpr int kW4Warps = 8;
constexpr int kAhead = 8;      // 16-byte weight loads that a lane has under way

struct W4Plan {
    int64_t T, H, E, k, I, P, G;
    size_t head, rows, act, y, total;   // workspace offsets
};

// head: [0] number of picked experts, then their ids [E] and the starts of their rows [E + 1]
struct W4Args {
    const uint16_t *x;
    const void *ids;
    const float *weights;
    const uint4 *w1, *w2;
    const uint16_t *s1, *s2;
    uint16_t *out, *act;        // act [P][2][I]: bf16 pair (high, low) of the activation
    float *y;                   // [P][H]
    int32_t *status, *head, *rows;
    int T, H, E, k, I, P, ids64;
};

__device__ __forceinline__ int load_id(const W4Args &a, int64_t p) {
    const int64_t v = a.ids64 ? static_cast<const int64_t *>(a.ids)[p] : static_cast<const int32_t *>(a.ids)[p];
    return v >= 0 && v < a.E ? (int)v : v == -1 ? -1 : -2;
}

// One block: the picks of each expert, the experts that have any.  The order of an expert's
// rows is left open; every row's result is its own column of the products.
__global__ void __launch_bounds__(1024) w4_group_kernel(W4Args a) {
    __shared__ int32_t count[MOE_MAX_EXPERTS], sums[64];
    __shared__ int32_t bad;
    pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < MOE_MAX_EXPERTS; e += 1024) count[e] = 0;
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int64_t p = tid; p < a.P; p += 1024) {
        const int e = load_id(a, p);
        if (e >= 0) atomicAdd(&count[e], 1);
        if (e == -2) bad = 1;
    }
    __syncthreads();
    // exclusive sums over the experts, two per thread: rows, and experts with rows
    const int e0 = 2 * tid;
    const int c0 = count[e0], c1 = count[e0 + 1];
    int rows = c0 + c1, used = (c0 > 0) + (c1 > 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int r = __shfl_up_sync(kAllLanes, rows, o), u = __shfl_up_sync(kAllLanes, used, o);
        if (lane >= o) {
            rows += r;
            used += u;
        }
    }
    if (lane == 31) {
        sums[warp] = rows;
        sums[32 + warp] = used;
    }
    __syncthreads();
    int rbase = 0, ubase = 0;
    for (int w = 0; w < warp; ++w) {
        rbase += sums[w];
        ubase += sums[32 + w];
    }
    int r = rbase + rows - c0 - c1, u = ubase + used - (c0 > 0) - (c1 > 0);
    int32_t *ids = a.head + 1, *starts = a.head + 1 + a.E;
    if (c0 > 0) {
        ids[u] = e0;
        starts[u++] = r;
    }
    count[e0] = r;
    r += c0;
    if (c1 > 0) {
        ids[u] = e0 + 1;
        starts[u++] = r;
    }
    count[e0 + 1] = r;
    r += c1;
    if (tid == 1023) {
        a.head[0] = u;
        starts[u] = r;
        *a.status = bad ? MOE_STATUS_BAD_EXPERT_ID : 0;
    }
    __syncthreads();
    for (int64_t p = tid; p < a.P; p += 1024) {
        const int e = load_id(a, p);
        if (e >= 0) a.rows[atomicAdd(&count[e], 1)] = (int)p;
    }
}

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight codes (nibble i + 4j: element j of fragment register i) to four bf16 pairs of
// code - 8: a code in the low mantissa bits of 128 is 128 + code, and 136 is taken off again.
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t (&a)[4]) {
    const __nv_bfloat162 off = __float2bfloat162_rn(136.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), off);
        a[i] = *reinterpret_cast<const uint32_t *>(&d);
    }
}

// acc[n][.] = one tile of 16 weight rows times NT blocks of 8 columns, over K inputs.
//   w       the tile's prepared codes, at this lane's 16 bytes of the first 64 inputs
//   sc      the tile's prepared scales, at this lane's first pair (rows g, g + 8)
//   col[n]  this lane's column (lane / 4 of block n) of inputs, or NULL (a column of zeros)
template <int NT, int G>
__device__ __forceinline__ void w4_tile(const uint4 *w, const uint16_t *sc, const uint16_t *const (&col)[NT], int K,
                                        float (&acc)[NT][4]) {
    constexpr int kPairs = 128 / G;   // scale pairs per 128 inputs
    const int q = threadIdx.x & 3;
    const int chunks = K / 64;
    uint4 buf[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        buf[i] = i < chunks ? ld_stream(w + (int64_t)i * 32) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    for (int c0 = 0; c0 < chunks; c0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; u += 2) {
            if (c0 + u < chunks) {   // chunks is even: 128 inputs at a time
                uint32_t pairs[kPairs];
#pragma unroll
                for (int i = 0; i < kPairs; ++i)
                    pairs[i] = __ldg(reinterpret_cast<const uint32_t *>(sc) + (int64_t)(c0 + u) / 2 * 8 * kPairs + i);
                float part[NT][4];
#pragma unroll
                for (int step = 0; step < 8; step += 2) {   // 32 inputs: two matrix steps
                    const uint4 v = buf[u + step / 4];
                    uint4 b[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        b[n] = col[n] ? __ldg(reinterpret_cast<const uint4 *>(col[n] + (c0 + u) * 64 + step * 16 + q * 8))
                                      : make_uint4(0, 0, 0, 0);
                    if (step * 16 % G == 0) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
                    }
                    uint32_t f[4];
                    unpack_codes(step % 4 == 0 ? v.x : v.z, f);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_bf16(part[n], f, b[n].x, b[n].y);
                    unpack_codes(step % 4 == 0 ? v.y : v.w, f);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_bf16(part[n], f, b[n].z, b[n].w);
                    if ((step + 2) * 16 % G == 0) {
                        const uint32_t p = pairs[step * 16 / G];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            acc[n][0] = fmaf(lo_f32(p), part[n][0], acc[n][0]);
                            acc[n][1] = fmaf(lo_f32(p), part[n][1], acc[n][1]);
                            acc[n][2] = fmaf(hi_f32(p), part[n][2], acc[n][2]);
                            acc[n][3] = fmaf(hi_f32(p), part[n][3], acc[n][3]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (c0 + u + i + kAhead < chunks) buf[u + i] = ld_stream(w + (int64_t)(c0 + u + i + kAhead) * 32);
            }
        }
    }
}

__device__ __forceinline__ float silu(float v) { return __fdiv_rn(v, 1.0f + expf(-v)); }

// Gate and up rows i0 .. i0 + 7 of one expert (they share a tile: rows 0..7 and 8..15) for up
// to 8 NT of its picks.
template <int NT, int G>
__device__ __forceinline__ void w4_up(const W4Args &a, int64_t tile, int i0, const int32_t *rows, int n) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint16_t *col[NT];
#pragma unroll
    for (int b = 0; b < NT; ++b) {
        const int c = 8 * b + g;
        col[b] = c < n ? a.x + (int64_t)(rows[c] / a.k) * a.H : nullptr;
    }
    float acc[NT][4];
    w4_tile<NT, G>(a.w1 + tile * (a.H / 64) * 32 + lane, a.s1 + (tile * (a.H / G) * 8 + g * (128 / G)) * 2, col, a.H, acc);
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = 8 * b + 2 * q + j;
            if (c >= n) continue;
            const float h = silu(acc[b][j]) * acc[b][2 + j];
            const __nv_bfloat16 hi = __float2bfloat16_rn(h);
            const float back = __bfloat162float(hi);
            const __nv_bfloat16 lo = __float2bfloat16_rn(isinf(back) ? 0.f : h - back);
            uint16_t *o = a.act + (int64_t)rows[c] * 2 * a.I + i0 + g;
            o[0] = __bfloat16_as_ushort(hi);
            o[a.I] = __bfloat16_as_ushort(lo);
        }
}

// Output rows h0 .. h0 + 15 for up to 4 NT picks: columns 2r and 2r + 1 are the high and the
// low part of pick r's activation, whose products are added at the end.
template <int NT, int G>
__device__ __forceinline__ void w4_down(const W4Args &a, int64_t tile, int h0, const int32_t *rows, int n) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint16_t *col[NT];
#pragma unroll
    for (int b = 0; b < NT; ++b) {
        const int c = 8 * b + g;
        col[b] = c / 2 < n ? a.act + ((int64_t)rows[c / 2] * 2 + (c & 1)) * a.I : nullptr;
    }
    float acc[NT][4];
    w4_tile<NT, G>(a.w2 + tile * (a.I / 64) * 32 + lane, a.s2 + (tile * (a.I / G) * 8 + g * (128 / G)) * 2, col, a.I, acc);
#pragma unroll
    for (int b = 0; b < NT; ++b) {
        const int r = 4 * b + q;
        if (r >= n) continue;
        float *o = a.y + (int64_t)rows[r] * a.H + h0 + g;
        o[0] = acc[b][0] + acc[b][1];
        o[8] = acc[b][2] + acc[b][3];
    }
}

// UP: the first product and the activation; else the second product.  A warp takes a tile of
// one expert at a time; the warps of a block take neighbouring tiles and so share inputs.
template <bool UP, int G>
__global__ void __launch_bounds__(kW4Warps * 32, 2) w4_product_kernel(W4Args a) {
    pdl_begin();
    const int tiles = UP ? a.I / 8 : a.H / 16;
    const int64_t units = (int64_t)a.head[0] * tiles;
    const int32_t *ids = a.head + 1, *starts = a.head + 1 + a.E;
    const int64_t stride = (int64_t)gridDim.x * kW4Warps;
    for (int64_t u = (int64_t)blockIdx.x * kW4Warps + (threadIdx.x >> 5); u < units; u += stride) {
        const int which = (int)(u / tiles), i = (int)(u - (int64_t)which * tiles);
        const int64_t tile = (int64_t)ids[which] * tiles + i;
        const int begin = starts[which], end = starts[which + 1];
        const int per = UP ? 1 : 2;   // columns per row
        for (int r = begin; r < end;) {
            const int left = end - r;
            if (left * per <= 8) {
                if (UP) w4_up<1, G>(a, tile, 8 * i, a.rows + r, left);
                else w4_down<1, G>(a, tile, 16 * i, a.rows + r, left);
                break;
            }
            const int n = min(left, 16 / per);
            if (UP) w4_up<2, G>(a, tile, 8 * i, a.rows + r, n);
            else w4_down<2, G>(a, tile, 16 * i, a.rows + r, n);
            r += n;
        }
    }
}

// out[t] = sum over the picks, in their order, of weight * y; eight columns per thread.
__global__ void __launch_bounds__(256) w4_combine_kernel(W4Args a) {
    pdl_begin();
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = v / (a.H / 8);
    const int c = (int)(v - t * (a.H / 8)) * 8;
    if (t >= a.T) return;
    float o[8] = {};
    for (int j = 0; j < a.k; ++j) {
        const int64_t p = t * a.k + j;
        if (load_id(a, p) < 0) continue;
        const float w = a.weights[p];
        const float4 *y = reinterpret_cast<const float4 *>(a.y + p * a.H + c);
        const float4 y0 = y[0], y1 = y[1];
        o[0] = fmaf(w, y0.x, o[0]); o[1] = fmaf(w, y0.y, o[1]); o[2] = fmaf(w, y0.z, o[2]); o[3] = fmaf(w, y0.w, o[3]);
        o[4] = fmaf(w, y1.x, o[4]); o[5] = fmaf(w, y1.y, o[5]); o[6] = fmaf(w, y1.z, o[6]); o[7] = fmaf(w, y1.w, o[7]);
    }
    *reinterpret_cast<uint4 *>(a.out + t * a.H + c) =
        make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
}

// Prepared order.  A tile is 16 weight rows: half = rows / 2 > 0 pairs rows i0 .. i0 + 7 with
// rows half + i0 .. (gate and up of w1), half == 0 takes 16 consecutive rows.  For 64 inputs
// from k0 on, lane (g, q) of a tile holds rows g and g + 8, inputs k0 + 8q .. + 7 and
// k0 + 32 + 8q .. + 7: word s (matrix step s) has nibble i + 4j = element j of fragment
// register i, where registers 0, 2 are row g and 1, 3 row g + 8, and registers 2, 3 the next
// two inputs.  One thread per lane and 64 inputs.
__global__ void __launch_bounds__(256) w4_order_codes_kernel(const uint8_t *codes, uint4 *out, int64_t n, int rows,
                                                             int K, int half) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n) return;
    const int lane = (int)(v & 31), g = lane >> 2, q = lane & 3;
    const int64_t c = v >> 5;
    const int chunk = (int)(c % (K / 64));
    const int64_t tile = c / (K / 64);
    const int64_t e = tile / (rows / 16);
    const int i = (int)(tile - e * (rows / 16));
    const int64_t r0 = e * rows + (half ? 8 * i : 16 * i) + g, r1 = r0 + (half ? half : 8);
    uint32_t word[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t k = chunk * 64 + 32 * h + 8 * q;
        const uint32_t a = *reinterpret_cast<const uint32_t *>(codes + (r0 * K + k) / 2);
        const uint32_t b = *reinterpret_cast<const uint32_t *>(codes + (r1 * K + k) / 2);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t x = a >> (16 * s), y = b >> (16 * s);   // four inputs of either row
            word[2 * h + s] = (x & 0xf) | (y & 0xf) << 4 | (x >> 8 & 0xf) << 8 | (y >> 8 & 0xf) << 12 |
                              (x >> 4 & 0xf) << 16 | (y >> 4 & 0xf) << 20 | (x >> 12 & 0xf) << 24 |
                              (y >> 12 & 0xf) << 28;
        }
    }
    out[v] = make_uint4(word[0], word[1], word[2], word[3]);
}

// Scales in the order [tile][128 inputs][g][group][rows g, g + 8]; one thread per pair.
__global__ void __launch_bounds__(256) w4_order_scales_kernel(const uint16_t *scales, uint32_t *out, int64_t n,
                                                              int rows, int K, int half, int G) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n) return;
    const int per = 128 / G;
    const int j = (int)(v % per), g = (int)(v / per % 8);
    const int64_t c = v / (8 * per);
    const int block = (int)(c % (K / 128));
    const int64_t tile = c / (K / 128);
    const int64_t e = tile / (rows / 16);
    const int i = (int)(tile - e * (rows / 16));
    const int64_t r0 = e * rows + (half ? 8 * i : 16 * i) + g, r1 = r0 + (half ? half : 8);
    const int64_t at = (int64_t)block * per + j;
    out[v] = scales[r0 * (K / G) + at] | (uint32_t)scales[r1 * (K / G) + at] << 16;
}

// One thread per group.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const uint16_t *w, uint8_t *codes, uint16_t *scales,
                                                          int64_t n, int G) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n) return;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(w + v * G);
    float m = 0.f;
    for (int i = 0; i < G / 2; ++i) m = fmaxf(m, fmaxf(fabsf(lo_f32(src[i])), fabsf(hi_f32(src[i]))));
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(m, 7.0f));
    const float s = __bfloat162float(sb);
    scales[v] = __bfloat16_as_ushort(sb);
    auto code = [&](float f) { return s > 0.f ? 8 + (int)fminf(fmaxf(rintf(__fdiv_rn(f, s)), -8.f), 7.f) : 8; };
    for (int i = 0; i < G / 2; ++i)
        codes[v * (G / 2) + i] = (uint8_t)(code(lo_f32(src[i])) | code(hi_f32(src[i])) << 4);
}

int make_w4_plan(const moe_w4_geom *g, W4Plan *p) {
    if (!g || g->num_tokens < 0 || g->hidden < 1 || g->num_experts < 1 || g->intermediate < 1 ||
        (g->group != 32 && g->group != 64 && g->group != 128))
        return MOE_ERR_INVALID_ARGUMENT;
    if (g->top_k < 1 || g->top_k > MOE_MAX_TOPK) return MOE_ERR_TOPK;
    if (g->hidden % 128 != 0) return MOE_ERR_HIDDEN_ALIGNMENT;
    if (g->intermediate % 128 != 0) return MOE_ERR_INTERMEDIATE_ALIGNMENT;
    if (g->num_experts > MOE_MAX_EXPERTS || g->hidden > MOE_MAX_HIDDEN) return MOE_ERR_LIMIT;
    p->T = g->num_tokens; p->H = g->hidden; p->E = g->num_experts; p->k = g->top_k; p->I = g->intermediate;
    p->G = g->group; p->P = p->T * p->k;
    if (p->P >= ((int64_t)1 << 31) || 2 * p->I >= ((int64_t)1 << 31)) return MOE_ERR_LIMIT;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = (off + bytes + 255) / 256 * 256;
        return o;
    };
    p->head = take(4 * (2 * p->E + 2));
    p->rows = take(4 * p->P);
    p->act = take(4 * p->P * p->I);
    p->y = take(4 * p->P * p->H);
    p->total = off;
    return MOE_OK;
}

unsigned blocks256(int64_t n) { return (unsigned)((n + 255) / 256); }

cudaError_t order_matrix(const uint8_t *codes, const void *scales, uint8_t *out, void *out_scales, int64_t E,
                         int64_t rows, int64_t K, int half, int G, cudaStream_t s) {
    const int64_t lanes = E * (rows / 16) * (K / 64) * 32, pairs = E * (rows / 16) * (K / G) * 8;
    if ((lanes + 255) / 256 >= ((int64_t)1 << 31) || (pairs + 255) / 256 >= ((int64_t)1 << 31))
        return cudaErrorInvalidValue;
    w4_order_codes_kernel<<<blocks256(lanes), 256, 0, s>>>(codes, reinterpret_cast<uint4 *>(out), lanes, (int)rows,
                                                           (int)K, half);
    w4_order_scales_kernel<<<blocks256(pairs), 256, 0, s>>>(static_cast<const uint16_t *>(scales),
                                                            static_cast<uint32_t *>(out_scales), pairs, (int)rows,
                                                            (int)K, half, G);
    return cudaGetLastError();
}

template <bool UP>
cudaError_t launch_product(const W4Args &a, int64_t G, int64_t most_units, cudaStream_t s) {
    int64_t blocks = (most_units + kW4Warps - 1) / kW4Warps;
    const int64_t most = 2 * (int64_t)num_sms();
    if (blocks > most) blocks = most;
    const dim3 grid((unsigned)blocks), block(kW4Warps * 32);
    if (G == 32) return launch_pdl(w4_product_kernel<UP, 32>, grid, block, 0, s, a);
    if (G == 64) return launch_pdl(w4_product_kernel<UP, 64>, grid, block, 0, s, a);
    return launch_pdl(w4_product_kernel<UP, 128>, grid, block, 0, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_quantize_w4(int64_t rows, int64_t cols, int32_t group, const void *w_dev, uint8_t *codes_dev,
                    void *scales_dev, void *stream) {
    if (rows < 0 || cols < 1 || (group != 32 && group != 64 && group != 128) || cols % group != 0 ||
        rows > ((int64_t)1 << 62) / cols)
        return MOE_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!w_dev || !codes_dev || !scales_dev)) return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(w_dev, 4) || !is_aligned(scales_dev, 2)) return MOE_ERR_MISALIGNED;
    const int64_t n = rows * (cols / group);
    if ((n + 255) / 256 >= ((int64_t)1 << 31)) return MOE_ERR_LIMIT;
    const int rc = check_device();
    if (rc != MOE_OK || n == 0) return rc;
    w4_quantize_kernel<<<blocks256(n), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint16_t *>(w_dev), codes_dev, static_cast<uint16_t *>(scales_dev), n, group);
    return status_of(cudaGetLastError());
}

int moe_prepare_weights_w4(const moe_w4_geom *g, const uint8_t *w1_codes_dev, const void *w1_scales_dev,
                           const uint8_t *w2_codes_dev, const void *w2_scales_dev, uint8_t *w1_prepared_dev,
                           void *w1_scales_prepared_dev, uint8_t *w2_prepared_dev, void *w2_scales_prepared_dev,
                           void *stream) {
    W4Plan p;
    int rc = make_w4_plan(g, &p);
    if (rc != MOE_OK) return rc;
    for (const void *v : {(const void *)w1_codes_dev, w1_scales_dev, (const void *)w2_codes_dev, w2_scales_dev,
                          (const void *)w1_prepared_dev, (const void *)w1_scales_prepared_dev,
                          (const void *)w2_prepared_dev, (const void *)w2_scales_prepared_dev}) {
        if (!v) return MOE_ERR_INVALID_ARGUMENT;
        if (!is_aligned(v, 16)) return MOE_ERR_MISALIGNED;
    }
    if (w1_codes_dev == w1_prepared_dev || w2_codes_dev == w2_prepared_dev ||
        w1_scales_dev == w1_scales_prepared_dev || w2_scales_dev == w2_scales_prepared_dev)
        return MOE_ERR_INVALID_ARGUMENT;
    if ((rc = check_device()) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = order_matrix(w1_codes_dev, w1_scales_dev, w1_prepared_dev, w1_scales_prepared_dev, p.E, 2 * p.I,
                                 p.H, (int)p.I, (int)p.G, s);
    if (e == cudaSuccess)
        e = order_matrix(w2_codes_dev, w2_scales_dev, w2_prepared_dev, w2_scales_prepared_dev, p.E, p.H, p.I, 0,
                         (int)p.G, s);
    return status_of(e);
}

int moe_forward_w4_workspace_size(const moe_w4_geom *g, size_t *bytes) {
    W4Plan p;
    const int rc = make_w4_plan(g, &p);
    if (rc != MOE_OK) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
    *bytes = p.total;
    return MOE_OK;
}

int moe_forward_w4(const moe_w4_geom *g, const void *x_dev, const void *topk_ids_dev, int ids_dtype,
                   const float *topk_weights_dev, const uint8_t *w1_prepared_dev,
                   const void *w1_scales_prepared_dev, const uint8_t *w2_prepared_dev,
                   const void *w2_scales_prepared_dev, void *out_dev, int32_t *status_dev, void *workspace_dev,
                   size_t workspace_bytes, void *stream) {
    W4Plan p;
    int rc = make_w4_plan(g, &p);
    if (rc != MOE_OK) return rc;
    if (ids_dtype != MOE_IDS_INT32 && ids_dtype != MOE_IDS_INT64) return MOE_ERR_IDS_DTYPE;
    if (!w1_prepared_dev || !w1_scales_prepared_dev || !w2_prepared_dev || !w2_scales_prepared_dev || !status_dev ||
        !workspace_dev || (p.T > 0 && (!x_dev || !topk_ids_dev || !topk_weights_dev || !out_dev)))
        return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(workspace_dev, 256) || !is_aligned(x_dev, 16) || !is_aligned(out_dev, 16) ||
        !is_aligned(w1_prepared_dev, 16) || !is_aligned(w2_prepared_dev, 16) ||
        !is_aligned(w1_scales_prepared_dev, 16) || !is_aligned(w2_scales_prepared_dev, 16) ||
        !is_aligned(topk_ids_dev, ids_dtype == MOE_IDS_INT64 ? 8 : 4) || !is_aligned(topk_weights_dev, 4) ||
        !is_aligned(status_dev, 4))
        return MOE_ERR_MISALIGNED;
    if (workspace_bytes < p.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if ((rc = check_device()) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace_dev);
    W4Args a{static_cast<const uint16_t *>(x_dev), topk_ids_dev, topk_weights_dev,
             reinterpret_cast<const uint4 *>(w1_prepared_dev), reinterpret_cast<const uint4 *>(w2_prepared_dev),
             static_cast<const uint16_t *>(w1_scales_prepared_dev),
             static_cast<const uint16_t *>(w2_scales_prepared_dev), static_cast<uint16_t *>(out_dev),
             reinterpret_cast<uint16_t *>(ws + p.act), reinterpret_cast<float *>(ws + p.y), status_dev,
             reinterpret_cast<int32_t *>(ws + p.head), reinterpret_cast<int32_t *>(ws + p.rows), (int)p.T, (int)p.H,
             (int)p.E, (int)p.k, (int)p.I, (int)p.P, ids_dtype == MOE_IDS_INT64};
    cudaError_t e = launch_pdl(w4_group_kernel, dim3(1), dim3(1024), 0, s, a);
    if (e == cudaSuccess && p.T > 0) {
        const int64_t used = p.P < p.E ? p.P : p.E;   // experts that can have picks
        e = launch_product<true>(a, p.G, used * (p.I / 8), s);
        if (e == cudaSuccess) e = launch_product<false>(a, p.G, used * (p.H / 16), s);
        if (e == cudaSuccess)
            e = launch_pdl(w4_combine_kernel, dim3(blocks256(p.T * (p.H / 8))), dim3(256), 0, s, a);
    }
    return status_of(e);
}

}  // extern "C"
