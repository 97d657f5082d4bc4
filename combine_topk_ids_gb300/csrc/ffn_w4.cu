// The routed experts' SwiGLU FFN of a decode batch with 4-bit weights (moe_forward_w4), the
// weights' one-time order (moe_prepare_weights_w4) and their quantisation (moe_quantize_w4);
// declared in include/moe_block.h.
//
//     out[t] = sum_j w[t, j] * W2_e (silu(Wg_e x[t]) * (Wu_e x[t])),   W = (code - 8) * scale
//
// A decode batch has few rows for each expert, so the time is that of reading the picked
// experts' codes once.  They feed warp-level matrix instructions (16 weight rows x 16 inputs
// x 8 batch rows, bf16 with float32 sums): a tcgen05 tile of 128 rows would be nearly empty,
// and its operands would have to be unpacked into shared memory first.  Codes become bf16
// integers without rounding; the sums over a group of inputs are multiplied by its scale in
// float32.  A block takes eight tiles of 16 weight rows; for 128 inputs at a time one warp
// copies their codes and scales (contiguous in the prepared order) and the batch rows' inputs
// to a ring of stages in shared memory, and four warps compute two tiles each.
#include "block_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int kW4Tiles = 8;    // tiles of 16 weight rows that a block takes at a time
constexpr int kW4Warps = 4;    // computing warps, two tiles each; one more warp copies
constexpr int kW4Threads = (kW4Warps + 1) * 32;
constexpr int kW4Blocks = 4;   // blocks on an SM
constexpr int kW4Cols = 16;    // columns of inputs at a time

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

// c (+)= a b; ZERO: the sum starts here.
template <bool ZERO>
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (ZERO)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One matrix step of 16 inputs for NT blocks of columns: eight codes (nibble i + 4j: element j
// of fragment register i) times b.  A code in the low mantissa bits of 128 is the bf16 number
// 128 + code; 136 is taken off again, exactly.
template <bool ZERO, int NT>
__device__ __forceinline__ void w4_step(float (&part)[NT][4], uint32_t w, const uint32_t (&b0)[NT],
                                        const uint32_t (&b1)[NT]) {
    uint32_t f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v;   // (w >> 4i) & 0x000f000f | 0x43004300
        asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w >> (4 * i)), "r"(0x000f000fu), "r"(0x43004300u));
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), __float2bfloat162_rn(136.f));
        f[i] = *reinterpret_cast<const uint32_t *>(&d);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) mma_bf16<ZERO>(part[n], f, b0[n], b1[n]);
}

// What a block works on at a time: kW4Tiles tiles of one expert for up to 16 columns of its
// picks (PER columns a pick).  Walks the units (expert, tiles) of the call from block to block.
template <int PER>
struct W4Item {
    int64_t u, group;
    int i, begin, end;   // group of tiles within the expert; the picks a.rows[begin .. end) still to do

    __device__ __forceinline__ int picks() const { return min(end - begin, kW4Cols / PER); }
    __device__ __forceinline__ bool start(const W4Args &a, int groups, int64_t units) {
        if (u >= units) return false;
        const int which = (int)(u / groups);
        const int32_t *ids = a.head + 1, *starts = a.head + 1 + a.E;
        i = (int)(u - (int64_t)which * groups);
        group = (int64_t)ids[which] * groups + i;
        begin = starts[which];
        end = starts[which + 1];
        return true;
    }
    __device__ __forceinline__ bool advance(const W4Args &a, int groups, int64_t units) {
        begin += picks();
        if (begin < end) return true;
        u += gridDim.x;
        return start(a, groups, units);
    }
};

// A stage holds 128 inputs: the tiles' codes and scales, and the columns' inputs.  The columns
// lie 64 bytes more apart than they are long, so that the eight lanes of a shared-memory phase
// (two columns, four 16-byte pieces) fall on different banks.
template <int G>
struct W4Stage {
    static constexpr int kPairs = 128 / G;   // scale pairs (rows g, g + 8) per 128 inputs
    static constexpr int kCodes = kW4Tiles * 1024, kScales = kW4Tiles * 32 * kPairs, kColumn = 256 + 64;
    static constexpr int kBytes = kCodes + kScales + kW4Cols * kColumn;
    static constexpr int kStages = G == 32 ? 3 : 4;   // what fits four blocks of an SM
};

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// One stage for the warp's two tiles: acc[t][n][.] += tile t times column block n.
template <int NT, int G>
__device__ __forceinline__ void w4_compute(const uint8_t *stage, int warp, float (&acc)[2][NT][4]) {
    using S = W4Stage<G>;
    constexpr int kPairs = S::kPairs;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint4 *w = reinterpret_cast<const uint4 *>(stage) + warp * 2 * 64 + lane;
    const uint32_t *sc = reinterpret_cast<const uint32_t *>(stage + S::kCodes) + (warp * 2 * 8 + g) * kPairs;
    const uint8_t *x = stage + S::kCodes + S::kScales + g * S::kColumn + q * 16;
    float part[2][NT][4];
    uint4 v[2];
#pragma unroll
    for (int h = 0; h < 4; ++h) {   // 32 inputs: two matrix steps
        uint32_t b0[NT], b1[NT], b2[NT], b3[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 b = *reinterpret_cast<const uint4 *>(x + n * 8 * S::kColumn + h * 64);
            b0[n] = b.x; b1[n] = b.y; b2[n] = b.z; b3[n] = b.w;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (h % 2 == 0) v[t] = w[t * 64 + h / 2 * 32];
            if (h * 32 % G == 0) w4_step<true, NT>(part[t], h % 2 ? v[t].z : v[t].x, b0, b1);
            else w4_step<false, NT>(part[t], h % 2 ? v[t].z : v[t].x, b0, b1);
            w4_step<false, NT>(part[t], h % 2 ? v[t].w : v[t].y, b2, b3);
            if ((h + 1) * 32 % G == 0) {
                const uint32_t p = sc[t * 8 * kPairs + h * 32 / G];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[t][n][0] = fmaf(lo_f32(p), part[t][n][0], acc[t][n][0]);
                    acc[t][n][1] = fmaf(lo_f32(p), part[t][n][1], acc[t][n][1]);
                    acc[t][n][2] = fmaf(hi_f32(p), part[t][n][2], acc[t][n][2]);
                    acc[t][n][3] = fmaf(hi_f32(p), part[t][n][3], acc[t][n][3]);
                }
            }
        }
    }
}

__device__ __forceinline__ float silu(float v) { return __fdiv_rn(v, 1.0f + expf(-v)); }

// First product: a tile is rows i0 .. i0 + 7 of the gate and of the up matrix (its rows 0..7
// and 8..15), so a lane holds both factors of its activations.
template <int NT>
__device__ __forceinline__ void w4_store_act(const W4Args &a, int i0, const int32_t *rows, int n,
                                             const float (&acc)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
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

// Second product: columns 2r and 2r + 1 are the high and the low part of pick r's activation,
// whose products are added here.
template <int NT>
__device__ __forceinline__ void w4_store_y(const W4Args &a, int h0, const int32_t *rows, int n,
                                           const float (&acc)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int b = 0; b < NT; ++b) {
        const int r = 4 * b + q;
        if (r >= n) continue;
        float *o = a.y + (int64_t)rows[r] * a.H + h0 + g;
        o[0] = acc[b][0] + acc[b][1];
        o[8] = acc[b][2] + acc[b][3];
    }
}

// UP: the first product and the activation; else the second product.
template <bool UP, int G>
__global__ void __launch_bounds__(kW4Threads, kW4Blocks) w4_product_kernel(W4Args a) {
    using S = W4Stage<G>;
    extern __shared__ __align__(128) uint8_t stages[];   // [kStages][kBytes]
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_u32(full + i), 1);
            mbar_init(smem_u32(empty + i), kW4Warps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_begin();
    const int K = UP ? a.H : a.I, blocks = K / 128;
    const int groups = (UP ? a.I / 8 : a.H / 16) / kW4Tiles;
    const int64_t units = (int64_t)a.head[0] * groups;
    constexpr int kPer = UP ? 1 : 2;
    W4Item<kPer> it;
    it.u = blockIdx.x;
    if (!it.start(a, groups, units)) return;
    int stage = 0;
    uint32_t phase = 0;
    auto next_stage = [&] {
        if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1;
        }
    };

    if (warp == kW4Warps) {   // the copying warp: lanes 0..15 a column each, 16 codes, 17 scales
        int put = 0;
        bool ok = true;
        do {
            const int n = it.picks() * kPer;
            const char *src = nullptr;
            uint32_t bytes = 0, off = 0;
            int step = 0;
            if (lane < n) {
                const int64_t p = a.rows[it.begin + lane / kPer];
                src = reinterpret_cast<const char *>(UP ? a.x + p / a.k * a.H : a.act + (p * 2 + (lane & 1)) * a.I);
                bytes = step = 256;
                off = S::kCodes + S::kScales + lane * S::kColumn;
            } else if (lane == 16) {
                src = reinterpret_cast<const char *>(UP ? a.w1 : a.w2) + it.group * blocks * S::kCodes;
                bytes = step = S::kCodes;
            } else if (lane == 17) {
                src = reinterpret_cast<const char *>(UP ? a.s1 : a.s2) + it.group * blocks * S::kScales;
                bytes = step = S::kScales;
                off = S::kCodes;
            }
            for (int b = 0; b < blocks; ++b) {
                ok = mbar_wait(smem_u32(empty + stage), phase ^ 1, &abort_flag, a.status);
                ok = __all_sync(kAllLanes, ok);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(smem_u32(full + stage), S::kCodes + S::kScales + n * 256);
                __syncwarp();
                if (bytes) bulk_copy(smem_u32(stages) + stage * S::kBytes + off, src, bytes, smem_u32(full + stage));
                src += step;
                ++put;
                next_stage();
            }
        } while (ok && it.advance(a, groups, units));
        if (!ok) {
            // gave up: the copies under way may not outlive the block, so each stage's gets one
            // more bounded wait (the status word already holds MOE_STATUS_TIMEOUT)
            for (int i = max(0, put - S::kStages); i < put; ++i) {
                const unsigned long long t0 = globaltimer();
                while (!mbar_try_wait(smem_u32(full + i % S::kStages), i / S::kStages & 1) &&
                       globaltimer() - t0 < kWaitLimitNs) {}
            }
        }
        return;
    }

    do {
        const int32_t *rows = a.rows + it.begin;
        const int n = it.picks();
        const int first = (it.i * kW4Tiles + warp * 2) * (UP ? 8 : 16);   // of the warp's first tile
        auto run = [&](auto blocks_of_columns) {
            constexpr int NT = decltype(blocks_of_columns)::value;
            float acc[2][NT][4] = {};
            for (int b = 0; b < blocks; ++b) {
                const bool in = mbar_wait(smem_u32(full + stage), phase, &abort_flag, a.status);
                if (!__all_sync(kAllLanes, in)) return false;
                w4_compute<NT, G>(stages + stage * S::kBytes, warp, acc);
                __syncwarp();   // every lane has read the stage
                if (lane == 0) mbar_arrive(smem_u32(empty + stage));
                next_stage();
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (UP) w4_store_act<NT>(a, first + 8 * t, rows, n, acc[t]);
                else w4_store_y<NT>(a, first + 16 * t, rows, n, acc[t]);
            }
            return true;
        };
        if (!(n * kPer <= 8 ? run(std::integral_constant<int, 1>{}) : run(std::integral_constant<int, 2>{}))) return;
    } while (it.advance(a, groups, units));
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
// two inputs.  The order is [8 tiles][128 inputs][tile][64 inputs][lane]; one thread per lane
// and 64 inputs.
__global__ void __launch_bounds__(256) w4_order_codes_kernel(const uint8_t *codes, uint4 *out, int64_t n, int rows,
                                                             int K, int half) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n) return;
    const int lane = (int)(v & 31), g = lane >> 2, q = lane & 3;
    const int64_t c = v / (64 * kW4Tiles);   // [8 tiles][128 inputs]
    const int chunk = (int)(c % (K / 128)) * 2 + (int)(v >> 5 & 1);
    const int64_t tile = c / (K / 128) * kW4Tiles + (v >> 6) % kW4Tiles;
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

// Scales in the order [8 tiles][128 inputs][tile][g][group][rows g, g + 8]; one thread per pair.
__global__ void __launch_bounds__(256) w4_order_scales_kernel(const uint16_t *scales, uint32_t *out, int64_t n,
                                                              int rows, int K, int half, int G) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n) return;
    const int per = 128 / G;
    const int j = (int)(v % per), g = (int)(v / per % 8);
    const int64_t c = v / (8 * per * kW4Tiles);
    const int block = (int)(c % (K / 128));
    const int64_t tile = c / (K / 128) * kW4Tiles + v / (8 * per) % kW4Tiles;
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

template <bool UP, int G>
cudaError_t launch_product_of(const W4Args &a, unsigned blocks, cudaStream_t s) {
    constexpr int smem = W4Stage<G>::kStages * W4Stage<G>::kBytes;
    static std::once_flag once[64];   // per device
    static cudaError_t set[64];
    const int dev = device_ordinal();
    if (dev < 0) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(w4_product_kernel<UP, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    return launch_pdl(w4_product_kernel<UP, G>, dim3(blocks), dim3(kW4Threads), smem, s, a);
}

template <bool UP>
cudaError_t launch_product(const W4Args &a, int64_t G, int64_t most_units, cudaStream_t s) {
    const int64_t most = kW4Blocks * (int64_t)num_sms();
    const unsigned blocks = (unsigned)(most_units < most ? most_units : most);
    if (G == 32) return launch_product_of<UP, 32>(a, blocks, s);
    if (G == 64) return launch_product_of<UP, 64>(a, blocks, s);
    return launch_product_of<UP, 128>(a, blocks, s);
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
        e = launch_product<true>(a, p.G, used * (p.I / 8 / kW4Tiles), s);
        if (e == cudaSuccess) e = launch_product<false>(a, p.G, used * (p.H / 16 / kW4Tiles), s);
        if (e == cudaSuccess)
            e = launch_pdl(w4_combine_kernel, dim3(blocks256(p.T * (p.H / 8))), dim3(256), 0, s, a);
    }
    return status_of(e);
}

}  // extern "C"
