// Products of e4m3 rows and e4m3 weights with a scale per 128 columns and per 128 x 128 block
// (moe_product_fp8; declared in include/moe_grouped.h):
//
//     out[m, n] = sum over blocks b of  sa[m, b] * sb[g, n / 128, b] * (a[m, b] . b[g, n, b])
//
// A block of 128 inner columns is one k-step of the tensor cores: its sum (four K = 32 products of
// tcgen05.mma kind::f8f6f4, exact products added in float32 in tensor memory) is scaled as a whole
// and added to float32 registers, the "promotion" of the partial sum.
//
// product_fp8_kernel computes tiles of 128 output columns and NT rows.  The weights are the M side of
// the products and the rows the N side, so that few rows cost few columns of tensor memory: a lane
// has one output column, a register one row.  192 threads:
//   warp 0      fills a ring of stages (128 x 128 weights, NT x 128 rows) with TMA
//   warp 1      issues the products, each k-step into the next of several buffers in tensor memory
//   warps 2-5   promotion; the scales' products of the next eight k-steps lie in shared memory
// Where the tiles are fewer than the SMs, `split` blocks of a cluster share a tile's k-steps and add
// their sums up through distributed shared memory, in the blocks' order.
#include <cuda_bf16.h>

#include "../../include/moe_grouped.h"
#include "block_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int kBK = 128;            // inner columns (bytes) of a k-step
constexpr int kTileN = 128;         // output columns of a tile: one block of the weights' scales
constexpr int kThreads = 192;
constexpr int kScaleSteps = 8;      // k-steps of one table of scales

struct ProductArgs {
    const float *sa, *sb;
    const int32_t *offsets;     // NULL: one matrix
    void *out;
    int32_t *status;            // NULL: none
    int64_t out_stride;
    int M, N, kb;               // kb: k-steps
    int G, nblk;                // weight matrices (1 without offsets), tiles across the columns
    int split;                  // blocks of a cluster that share a tile
    int out_bf16;
};

// First row of group g, between 0 and M whatever the offsets hold.
__device__ __forceinline__ int row_of(const ProductArgs &a, int g) {
    if (!a.offsets) return g ? a.M : 0;
    return min(max(__ldg(a.offsets + g), 0), a.M);
}

// prefix[g] = tiles of `rows` rows in the groups before g, g <= G.  All threads of the block.
__device__ __forceinline__ void count_tiles(const ProductArgs &a, int rows, int *prefix, int *wsum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int g0 = 0; g0 < a.G; g0 += blockDim.x) {
        const int g = g0 + threadIdx.x;
        const int n = g < a.G ? (max(row_of(a, g + 1) - row_of(a, g), 0) + rows - 1) / rows : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAllLanes, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int ahead = carry;
        for (int w = 0; w < warps; ++w) {
            ahead += w < warp ? wsum[w] : 0;
            carry += wsum[w];
        }
        if (g < a.G) prefix[g] = ahead + incl - n;
        __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.G] = carry;
    __syncthreads();
}

struct Tile {
    int g, m0, rows, nb;   // group, first row, rows that count, tile across the columns
};

// Tiles of a group follow one another, those of the same weights first.
template <int ROWS>
__device__ __forceinline__ Tile tile_of(const ProductArgs &a, const int *prefix, int64_t i) {
    const int q = (int)(i / a.nblk);
    int lo = 0, hi = a.G - 1;   // the largest g with prefix[g] <= q
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    const int local = (int)(i - (int64_t)prefix[lo] * a.nblk), mt = prefix[lo + 1] - prefix[lo];
    Tile t;
    t.g = lo;
    t.nb = local / mt;
    const int begin = row_of(a, lo), end = row_of(a, lo + 1);
    t.m0 = begin + (local - t.nb * mt) * ROWS;
    t.rows = min(ROWS, end - t.m0);
    return t;
}

// Instruction descriptor of kind::f8f6f4: float32 sums (bits 4-5), e4m3 operands (0), both K-major,
// N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t f8_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 lanes x 16 columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// A float in the shared memory of block `rank` of the cluster, at this block's address `addr`.
__device__ __forceinline__ float peer_float(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

__device__ __forceinline__ void store_out(const ProductArgs &a, int64_t m, int n, float v) {
    if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.out)[m * a.out_stride + n] = __float2bfloat16_rn(v);
    else static_cast<float *>(a.out)[m * a.out_stride + n] = v;
}

// Shared memory of a tile of NT rows.
template <int NT> struct Narrow {
    static constexpr int kWeights = kTileN * kBK, kRows = NT * kBK, kStage = kWeights + kRows;
    static constexpr int kStages = 196 * 1024 / kStage < 10 ? 196 * 1024 / kStage : 10;
    static constexpr int kBuffers = 512 / NT < 8 ? 512 / NT : 8;   // partial sums in tensor memory
    static constexpr int kColumns = kBuffers * NT;                 // (a power of two, 32 at least)
    static constexpr int kTable = kScaleSteps * NT * 4;
    static constexpr int kBytes = 1024 + kStages * kStage + 2 * kTable + 512;
    static_assert(kStages * kStage >= NT * kTileN * 4, "the ring holds a split tile's sums");
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    product_fp8_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_weights,
                       ProductArgs a) {
    using S = Narrow<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float *table = reinterpret_cast<float *>(smem + S::kStages * S::kStage);   // [2][kScaleSteps][NT]
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(table) + 2 * S::kTable);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S::kStages + 2 * S::kBuffers);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int32_t *no_status = reinterpret_cast<int32_t *>(tmem_slot + 2);
    int *wsum = reinterpret_cast<int *>(tmem_slot + 3);                        // [6]
    int *prefix = reinterpret_cast<int *>(bars) + 512 / 4;                     // [G + 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S::kStages;
    const uint32_t pfull0 = empty0 + 8 * S::kStages, pempty0 = pfull0 + 8 * S::kBuffers;
    int32_t *status = a.status ? a.status : no_status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < S::kBuffers; ++b) {
            mbar_init(pfull0 + 8 * b, 1);
            mbar_init(pempty0 + 8 * b, 4);   // one arrival of each promoting warp
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_rows)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_weights)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(S::kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    count_tiles(a, NT, prefix, wsum);
    const int64_t total = (int64_t)prefix[a.G] * a.nblk;
    // the k-steps of this block, and its cluster's tiles
    const int rank = a.split > 1 ? (int)cluster_rank() : 0;
    const int k0 = (int)((int64_t)a.kb * rank / a.split), k1 = (int)((int64_t)a.kb * (rank + 1) / a.split);
    const int64_t first = blockIdx.x / a.split, step = gridDim.x / a.split;
    float acc[NT];
    Tile mine{};

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t i = first; i < total && ok; i += step) {
                const Tile t = tile_of<NT>(a, prefix, i);
                for (int k = k0; k < k1; ++k) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, status)) { ok = false; break; }
                    const uint32_t fb = full0 + 8 * stage, at = smem_u32(smem + stage * S::kStage);
                    mbar_expect_tx(fb, S::kStage);
                    tma_load_2d(at, &tm_weights, k * kBK, t.g * a.N + t.nb * kTileN, fb);
                    tma_load_2d(at + S::kWeights, &tm_rows, k * kBK, t.m0, fb);
                    if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true;
            constexpr uint32_t idesc = f8_idesc(kTileN, NT);
            for (int64_t i = first; i < total && ok; i += step) {
                for (int k = k0; k < k1; ++k) {
                    if (!mbar_wait(pempty0 + 8 * buf, bphase ^ 1, abort_flag, status)) { ok = false; break; }
                    if (!mbar_wait(full0 + 8 * stage, phase, abort_flag, status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t w0 = smem_u32(smem + stage * S::kStage), r0 = w0 + S::kWeights;
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)
                        mma_f8(tmem_base + buf * NT, sw128_desc(w0 + kk * 32), sw128_desc(r0 + kk * 32), idesc, kk != 0);
                    mma_commit(empty0 + 8 * stage);
                    mma_commit(pfull0 + 8 * buf);
                    if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                    if (++buf == S::kBuffers) { buf = 0; bphase ^= 1; }
                }
            }
        }
    } else {
        const int thread = threadIdx.x - 64, quad = warp & 3, col = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        int buf = 0, turn = 0;
        uint32_t bphase = 0;
        bool ok = true;
        // (Where a wait has given up the loops go on to their end without waiting: the four warps
        // meet at the tables' barriers as often as ever.)
        for (int64_t i = first; i < total; i += step) {
            const Tile t = tile_of<NT>(a, prefix, i);
            mine = t;
#pragma unroll
            for (int c = 0; c < NT; ++c) acc[c] = 0.f;
            // Scales of eight k-steps: thread -> row thread / 8 (and every 16th after it), k-step
            // thread % 8.  Fetched while the eight before them are promoted.
            constexpr int kEach = NT / 16;
            float next[kEach];
            const float *sb = a.sb + ((int64_t)t.g * a.nblk + t.nb) * a.kb;
            auto fetch = [&](int k) {
                k += thread & 7;
                const float b = k < k1 ? __ldg(sb + k) : 0.f;
#pragma unroll
                for (int r = 0; r < kEach; ++r) {
                    const int row = (thread >> 3) + 16 * r;
                    next[r] = k < k1 && row < t.rows ? b * __ldg(a.sa + (int64_t)(t.m0 + row) * a.kb + k) : 0.f;
                }
            };
            fetch(k0);
            for (int k = k0; k < k1; k += kScaleSteps) {
                float *tab = table + turn * (kScaleSteps * NT);
                turn ^= 1;   // (two tables: all warps are past the one before the last barrier)
#pragma unroll
                for (int r = 0; r < kEach; ++r) tab[(thread & 7) * NT + (thread >> 3) + 16 * r] = next[r];
                asm volatile("bar.sync 1, 128;" ::: "memory");
                fetch(k + kScaleSteps);
                const int n = min(kScaleSteps, k1 - k);
                for (int q = 0; q < n && ok; ++q) {
                    if (!mbar_wait(pfull0 + 8 * buf, bphase, abort_flag, status)) { ok = false; break; }
                    tc_fence_after();
                    const float4 *sc = reinterpret_cast<const float4 *>(tab + q * NT);
#pragma unroll
                    for (int c0 = 0; c0 < NT; c0 += 16) {
                        uint32_t v[16];
                        tmem_ld16(tmem_base + buf * NT + c0 + lanes, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 s = sc[(c0 + c) / 4];
                            acc[c0 + c] = fmaf(__uint_as_float(v[c]), s.x, acc[c0 + c]);
                            acc[c0 + c + 1] = fmaf(__uint_as_float(v[c + 1]), s.y, acc[c0 + c + 1]);
                            acc[c0 + c + 2] = fmaf(__uint_as_float(v[c + 2]), s.z, acc[c0 + c + 2]);
                            acc[c0 + c + 3] = fmaf(__uint_as_float(v[c + 3]), s.w, acc[c0 + c + 3]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pempty0 + 8 * buf);
                    if (++buf == S::kBuffers) { buf = 0; bphase ^= 1; }
                }
            }
            const int n = t.nb * kTileN + col;
            if (a.split == 1 && n < a.N && ok) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    if (c < t.rows) store_out(a, t.m0 + c, n, acc[c]);
            }
        }
    }
    __syncthreads();
    if (*abort_flag) {
        // copies and products in flight get time to land before the memory is released
        const unsigned long long t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {}
    }
    if (a.split > 1 && first < total) {   // (a cluster has one tile then: the ring is free)
        float *sums = reinterpret_cast<float *>(smem);   // [NT][kTileN]
        if (warp >= 2) {
            const int col = (warp & 3) * 32 + lane;
#pragma unroll
            for (int c = 0; c < NT; ++c) sums[c * kTileN + col] = acc[c];
        }
        cluster_sync();
        if (warp >= 2) {
            const int col = (warp & 3) * 32 + lane, n = mine.nb * kTileN + col;
            for (int c = rank; c < mine.rows; c += a.split) {
                float v = 0.f;
                for (int r = 0; r < a.split; ++r) v += peer_float(smem_u32(sums + c * kTileN + col), r);
                if (n < a.N) store_out(a, mine.m0 + c, n, v);
            }
        }
        cluster_sync();   // no block leaves while its sums are read
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(S::kColumns)
                     : "memory");
    }
}

// ------------------------------------------------------------------------------------ host

// A 2-D map of e4m3 codes: `rows` rows of `cols` bytes, `stride` bytes apart, boxes of 128 bytes.
bool make_codes_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t stride, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride};
    cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's shared memory, allowed once on each device (with that device current).
struct PerDevice {
    std::once_flag once[64];
    cudaError_t error[64];
    template <typename K> cudaError_t set(K kernel, int smem) {
        const int d = device_ordinal();
        if (d < 0) return cudaErrorInvalidDevice;
        std::call_once(once[d], [&] {
            error[d] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        });
        return error[d];
    }
};

struct Operands {
    const uint8_t *a, *b;
    int64_t a_stride, K;
};

template <int NT>
int launch_narrow(ProductArgs &p, const Operands &o, cudaStream_t s) {
    using S = Narrow<NT>;
    CUtensorMap rows, weights;
    if (!make_codes_map(&rows, o.a, p.M, o.K, o.a_stride, NT) ||
        !make_codes_map(&weights, o.b, (int64_t)p.G * p.N, o.K, o.K, kTileN))
        return MOE_ERR_CUDA;
    auto kernel = product_fp8_kernel<NT>;
    const int smem = S::kBytes + (p.G + 1) * 4;
    static PerDevice devices;
    const cudaError_t e = devices.set(kernel, S::kBytes + (MOE_MAX_EXPERTS + 1) * 4);
    if (e != cudaSuccess) return status_of(e);
    // tiles there can be: each group may have one that is not full
    const int64_t most = ((int64_t)p.M / NT + (p.G < p.M ? p.G : p.M)) * p.nblk;
    const int sms = num_sms();
    p.split = 1;
    while (p.split < 8 && most * p.split * 2 <= sms && p.kb / (p.split * 2) >= 4) p.split *= 2;
    const int64_t grid = p.split > 1 ? most * p.split : (most < sms ? most : sms);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return status_of(cudaLaunchKernelEx(&cfg, kernel, rows, weights, p));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_product_fp8(const moe_product *p, const uint8_t *a_dev, const float *a_scales_dev,
                               const uint8_t *b_dev, const float *b_scales_dev, const int32_t *offsets_dev,
                               void *out_dev, int32_t *status_dev, void *stream) {
    if (!p || p->num_rows < 0 || p->n < 1 || p->k < 1 || p->groups < 0 || bad_dtype(p->out_dtype))
        return MOE_ERR_INVALID_ARGUMENT;
    if (p->k % 128) return MOE_ERR_HIDDEN_ALIGNMENT;
    if (p->k > MOE_MAX_HIDDEN || p->n > MOE_MAX_HIDDEN || p->groups > MOE_MAX_EXPERTS) return MOE_ERR_LIMIT;
    const int64_t a_stride = p->a_stride ? p->a_stride : p->k, out_stride = p->out_stride ? p->out_stride : p->n;
    if (a_stride < p->k || out_stride < p->n || !p->groups != !offsets_dev) return MOE_ERR_INVALID_ARGUMENT;
    if (p->num_rows > 0 && (!a_dev || !a_scales_dev || !b_dev || !b_scales_dev || !out_dev))
        return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(a_dev, 16) || a_stride % 16 || !is_aligned(b_dev, 16) || !is_aligned(a_scales_dev, 4) ||
        !is_aligned(b_scales_dev, 4) || !is_aligned(offsets_dev, 4) || !is_aligned(status_dev, 4) ||
        !is_aligned(out_dev, dtype_bytes(p->out_dtype)))
        return MOE_ERR_MISALIGNED;
    if (a_stride >= ((int64_t)1 << 40)) return MOE_ERR_LIMIT;   // (what a tensor map holds)
    const int rc = check_device();
    if (rc != MOE_OK) return rc;
    if (p->num_rows == 0) return MOE_OK;
    ProductArgs args{a_scales_dev, b_scales_dev, offsets_dev, out_dev, status_dev, out_stride, p->num_rows, p->n,
                     p->k / kBK, p->groups ? p->groups : 1, (p->n + kTileN - 1) / kTileN, 1,
                     p->out_dtype == MOE_DTYPE_BF16};
    const Operands o{a_dev, b_dev, a_stride, p->k};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t mean = ((int64_t)args.M + args.G - 1) / args.G;
    if (mean <= 12) return launch_narrow<16>(args, o, s);
    if (mean <= 24) return launch_narrow<32>(args, o, s);
    if (mean <= 64) return launch_narrow<64>(args, o, s);
    return launch_narrow<128>(args, o, s);
}
