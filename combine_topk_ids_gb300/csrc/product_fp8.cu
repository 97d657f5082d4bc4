// Products of e4m3 rows and e4m3 weights with a scale per 128 columns and per 128 x 128 block
// (moe_product_fp8; declared in include/moe_grouped.h):
//
//     out[m, n] = sum over blocks b of  sa[m, b] * sb[g, n / 128, b] * (a[m, b] . b[g, n, b])
//
// Bounds.  Few rows: the weights' bytes (HBM; 512 rows over 256 matrices of 4096 x 7168, 206 of them
// with a row, 787 us, 7.7 TB/s), below some 50 MB of them the launch and the latency of one short wave of tiles
// (one row by 4096 x 7168 7.8 us, 4.3 of them the bytes).  64 to 2048 rows: SMs without a tile, or with one when others
// have two (512 x 4096 x 7168 34 us: 64 wide tiles, each through all k-steps).  Many rows: the promotion, and
// close behind it the operands' way into the ring (32768 x 4096 x 7168 688 us in bursts, 2.8 PFLOP/s, and 778, 2.5, in a
// loop of seconds, where the clock falls to 1.65 to 1.75 GHz; in bursts the products alone 424 us, with
// their operands 592, with the promotion and no operands 640; the tensor cores are busy in half of the
// cycles).
//
// A block of 128 inner columns is one k-step of the tensor cores: its sum (four K = 32 products of
// tcgen05.mma kind::f8f6f4, exact products added in float32 in tensor memory) is scaled as a whole
// and added to float32 registers, the "promotion" of the partial sum.
//
// product_fp8_kernel computes tiles of 128 output columns and NT rows.  The weights are the M side of
// the products and the rows the N side, so that few rows cost few columns of tensor memory: a lane
// has one output column, a register one row.  256 threads:
//   warp 0      fills a ring of stages (128 x 128 weights, NT x 128 rows) with TMA
//   warps 1, 6  issue the products, one the even k-steps and one the odd ones, each k-step into the next
//               of several buffers in tensor memory.  (One thread's waits and issues for all of them take
//               longer than the products.)
//   warps 2-5   promotion
//   warp 7      puts the scales' products of the next eight k-steps into shared memory: a promoting warp
//               that had loads of its own under way would wait for them with its tensor-memory loads
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
constexpr int kThreads = 256;
constexpr int kScaleSteps = 8;      // k-steps of one table of scales
constexpr int kMaxSplit = 8;        // blocks that share a tile (the portable size of a cluster)

struct ProductArgs {
    const float *sa, *sb;
    const int32_t *offsets;     // NULL: one matrix
    void *out;
    int32_t *status;            // NULL: none
    int64_t out_stride;
    int M, N, kb;               // kb: k-steps
    int G, nblk;                // weight matrices (1 without offsets), tiles across the columns
    int split;                  // blocks of a cluster that share a tile
    int most_rows;              // row tiles there can be
    int panel;                  // wide tiles: tiles across the columns of a panel
    int out_bf16;
    int out_fours;              // four neighbouring columns of out can be stored at once
    int out_map;                // wide tiles: out has a tensor map (rows on 16-byte boundaries)
};

// First row of group g, between 0 and M whatever the offsets hold.  (Offsets and scales are read by plain loads, not
// through the read-only path: that asks for memory which does not change while the kernel runs, and this one is
// launched while the kernel that writes them does.  The times are the same.)
__device__ __forceinline__ int row_of(const ProductArgs &a, int g) {
    if (!a.offsets) return g ? a.M : 0;
    return min(max(a.offsets[g], 0), a.M);
}

// prefix[g] = tiles of `rows` rows in the groups before g, g <= G; the number of tiles.  All threads of the
// block.  Sums stop at 2^30 - 1, above what ascending offsets can come to (most_rows): offsets that do not
// ascend and pass it get no tile.
__device__ __forceinline__ int count_tiles(const ProductArgs &a, int rows, int *prefix, int *wsum) {
    constexpr int kStop = (1 << 30) - 1;
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            prefix[0] = 0;
            prefix[1] = a.most_rows;
        }
        __syncthreads();
        return a.most_rows * a.nblk;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int g0 = 0; g0 < a.G; g0 += blockDim.x) {
        const int g = g0 + threadIdx.x;
        const int n = g < a.G ? (int)(((int64_t)max(row_of(a, g + 1) - row_of(a, g), 0) + rows - 1) / rows) : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAllLanes, incl, o);
            if (lane >= o) incl = min(incl + v, kStop);
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int ahead = carry;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) ahead = min(ahead + wsum[w], kStop);
            carry = min(carry + wsum[w], kStop);
        }
        if (g < a.G) prefix[g] = min(ahead + incl, kStop) - n;
        __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.G] = carry;
    __syncthreads();
    return carry <= a.most_rows ? carry * a.nblk : 0;
}

struct Tile {
    int g, m0, rows, nb;   // group, first row, rows that count, tile across the columns
};

// Tiles of a group follow one another, those of the same weights first.
template <int ROWS>
__device__ __forceinline__ Tile tile_of(const ProductArgs &a, const int *prefix, int i) {
    const int q = i / a.nblk;
    int lo = 0, hi = a.G - 1;   // the largest g with prefix[g] <= q
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    const int local = i - prefix[lo] * a.nblk, mt = prefix[lo + 1] - prefix[lo];
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
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }

// Waits for this thread's tensor-memory loads, the last of which filled v.
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}


// d += v * s for two columns.  Volatile, as the loads and waits are: left to itself the compiler puts the
// additions where a load has arrived behind the next load's wait, and nothing overlaps (32768 x 4096 x
// 7168 by the wide tiles, without operand loads: 658 us for 608).
__device__ __forceinline__ void add2(float2 &d, uint32_t v0, uint32_t v1, float s0, float s1) {
    asm volatile(
        "{\n\t.reg .b64 v, s, d;\n\t"
        "mov.b64 v, {%2, %3};\n\t"
        "mov.b64 s, {%4, %5};\n\t"
        "mov.b64 d, {%0, %1};\n\t"
        "fma.rn.f32x2 d, v, s, d;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d.x), "+f"(d.y)
        : "r"(v0), "r"(v1), "f"(s0), "f"(s1));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The address of `addr` in block `rank` of the cluster, and four floats there.
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    return remote;
}
__device__ __forceinline__ float4 peer_load(uint32_t remote) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

__device__ __forceinline__ void store_out(const ProductArgs &a, int64_t m, int n, float v) {
    if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.out)[m * a.out_stride + n] = __float2bfloat16_rn(v);
    else static_cast<float *>(a.out)[m * a.out_stride + n] = v;
}

// Shared memory of a tile of NT rows.
template <int NT> struct Narrow {
    static constexpr int kWeights = kTileN * kBK, kRows = NT * kBK, kStage = kWeights + kRows;
    // (even, as the buffers: each stage and buffer always goes to the same issuing thread)
    static constexpr int kStages = NT == 16 ? 10 : NT == 128 ? 6 : 8;
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
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S::kStages + 2 * S::kBuffers + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int32_t *no_status = reinterpret_cast<int32_t *>(tmem_slot + 2);
    int *wsum = reinterpret_cast<int *>(tmem_slot + 3);                        // [8]
    Tile *mine_s = reinterpret_cast<Tile *>(wsum + 8);
    int *prefix = reinterpret_cast<int *>(bars) + 512 / 4;                     // [G + 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S::kStages;
    const uint32_t pfull0 = empty0 + 8 * S::kStages, pempty0 = pfull0 + 8 * S::kBuffers;
    const uint32_t sfull0 = pempty0 + 8 * S::kBuffers, sempty0 = sfull0 + 16;
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
        for (int b = 0; b < 2; ++b) {
            mbar_init(sfull0 + 8 * b, 1);
            mbar_init(sempty0 + 8 * b, 4);
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
    const int total = count_tiles(a, NT, prefix, wsum);
    // the k-steps of this block, and its cluster's tiles
    const int rank = a.split > 1 ? (int)cluster_rank() : 0;
    const int k0 = (int)((int64_t)a.kb * rank / a.split), k1 = (int)((int64_t)a.kb * (rank + 1) / a.split);
    const int first = blockIdx.x / a.split, step = gridDim.x / a.split;
    float2 acc[NT / 2];   // rows 2c and 2c + 1 of the lane's column
    Tile mine{};

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = first; i < total && ok; i += step) {
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
    } else if (warp == 1 || warp == 6) {
        if (lane == 0) {
            const int odd = warp == 6;
            int stage = odd, buf = odd;
            uint32_t phase = 0, bphase = 0;
            constexpr uint32_t idesc = f8_idesc(kTileN, NT);
            const int steps = first < total ? (total - first + step - 1) / step * (k1 - k0) : 0;
            for (int it = odd; it < steps; it += 2) {
                if (!mbar_wait(full0 + 8 * stage, phase, abort_flag, status)) break;
                if (!mbar_wait(pempty0 + 8 * buf, bphase ^ 1, abort_flag, status)) break;
                tc_fence_after();
                const uint32_t w0 = smem_u32(smem + stage * S::kStage), r0 = w0 + S::kWeights;
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk)
                    mma_f8(tmem_base + buf * NT, sw128_desc(w0 + kk * 32), sw128_desc(r0 + kk * 32), idesc, kk != 0);
                mma_commit(empty0 + 8 * stage);
                mma_commit(pfull0 + 8 * buf);
                if ((stage += 2) >= S::kStages) { stage = odd; phase ^= 1; }
                if ((buf += 2) >= S::kBuffers) { buf = odd; bphase ^= 1; }
            }
        }
    } else if (warp == 7) {
        // lane: k-step lane % 8, rows lane / 8 and every fourth behind it; what is fetched waits in registers
        // for its table to be free
        uint32_t turn = 0;
        bool ok = true;
        for (int i = first; i < total && ok; i += step) {
            const Tile t = tile_of<NT>(a, prefix, i);
            const float *sa = a.sa + (int64_t)(t.m0 + (lane >> 3)) * a.kb + (lane & 7);
            const float *sb = a.sb + ((int64_t)t.g * a.nblk + t.nb) * a.kb + (lane & 7);
            for (int k = k0; k < k1; k += kScaleSteps, ++turn) {
                float *tab = table + (turn & 1) * (kScaleSteps * NT);   // [8][NT]
                const bool in = k + (lane & 7) < k1;
                const float w = in ? sb[k] : 0.f;
                float r[NT / 4];
#pragma unroll
                for (int j = 0; j < NT / 4; ++j)
                    r[j] = in && 4 * j + (lane >> 3) < t.rows ? sa[(int64_t)(4 * j) * a.kb + k] : 0.f;
                if (!mbar_wait(sempty0 + 8 * (turn & 1), ((turn >> 1) & 1) ^ 1, abort_flag, status)) { ok = false; break; }
#pragma unroll
                for (int j = 0; j < NT / 4; ++j) tab[(lane & 7) * NT + 4 * j + (lane >> 3)] = w * r[j];
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull0 + 8 * (turn & 1));
            }
        }
    } else {
        const int quad = warp & 3, col = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        int buf = 0;
        uint32_t bphase = 0, turn = 0;
        bool ok = true;
        for (int i = first; i < total && ok; i += step) {
            const Tile t = tile_of<NT>(a, prefix, i);
            mine = t;
#pragma unroll
            for (int c = 0; c < NT / 2; ++c) acc[c] = make_float2(0.f, 0.f);
            for (int k = k0; k < k1 && ok; k += kScaleSteps, ++turn) {
                const float *tab = table + (turn & 1) * (kScaleSteps * NT);
                if (!mbar_wait(sfull0 + 8 * (turn & 1), (turn >> 1) & 1, abort_flag, status)) { ok = false; break; }
                const int n = min(kScaleSteps, k1 - k);
                for (int q = 0; q < n && ok; ++q) {
                    if (!mbar_wait(pfull0 + 8 * buf, bphase, abort_flag, status)) { ok = false; break; }
                    tc_fence_after();
                    const float4 *sc = reinterpret_cast<const float4 *>(tab + q * NT);
                    const uint32_t from = tmem_base + buf * NT + lanes;
                    constexpr int C = NT < 32 ? NT : 32, kLoads = NT / C;   // the next C rows are on their way
                    uint32_t v[2][C];                                        // while C are added
                    tmem_ld(from, v[0]);
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) {
                        tmem_wait(v[j & 1]);
                        if (j + 1 < kLoads) tmem_ld(from + C * (j + 1), v[(j + 1) & 1]);
                        else {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(pempty0 + 8 * buf);
                        }
#pragma unroll
                        for (int c = 0; c < C / 4; ++c) {
                            const float4 s = sc[j * (C / 4) + c];
                            const uint32_t *x = v[j & 1] + 4 * c;
                            add2(acc[j * (C / 2) + 2 * c], x[0], x[1], s.x, s.y);
                            add2(acc[j * (C / 2) + 2 * c + 1], x[2], x[3], s.z, s.w);
                        }
                    }
                    if (++buf == S::kBuffers) { buf = 0; bphase ^= 1; }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty0 + 8 * (turn & 1));
            }
            const int n = t.nb * kTileN + col;
            if (a.split == 1 && n < a.N && ok) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    if (c < t.rows) store_out(a, t.m0 + c, n, c & 1 ? acc[c / 2].y : acc[c / 2].x);
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
        const bool promotes = warp >= 2 && warp < 6;
        if (promotes) {
            const int col = (warp & 3) * 32 + lane;
#pragma unroll
            for (int c = 0; c < NT; ++c) sums[c * kTileN + col] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
            if (warp == 2 && lane == 0) *mine_s = mine;
        }
        cluster_sync();
        // Row by row of the tile, which the cluster's blocks take in turn; four columns to a lane.
        const Tile t = *mine_s;
        const int n = t.nb * kTileN + 4 * lane;
        uint32_t from[kMaxSplit];
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r)
            if (r < a.split) from[r] = peer_address(smem_u32(sums) + 16 * lane, r);
        const int warps = kThreads / 32, stride = a.split * warps;
        for (int c = rank + a.split * warp; c < t.rows; c += 2 * stride) {
            float4 v[2][kMaxSplit];                      // two rows under way
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    if (r < a.split && c + u * stride < t.rows) v[u][r] = peer_load(from[r] + (c + u * stride) * kTileN * 4);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t m = t.m0 + c + u * stride;
                if (c + u * stride >= t.rows) continue;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    if (r < a.split) {
                        s.x += v[u][r].x; s.y += v[u][r].y; s.z += v[u][r].z; s.w += v[u][r].w;
                    }
                if (n + 4 <= a.N && a.out_fours) {
                    if (a.out_bf16)
                        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + m * a.out_stride + n) =
                            make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
                    else *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + m * a.out_stride + n) = s;
                } else {
                    if (n < a.N) store_out(a, m, n, s.x);
                    if (n + 1 < a.N) store_out(a, m, n + 1, s.y);
                    if (n + 2 < a.N) store_out(a, m, n + 2, s.z);
                    if (n + 3 < a.N) store_out(a, m, n + 3, s.w);
                }
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

// ------------------------------------------------------------------------------ many rows

// Tiles of 128 rows and 256 columns.  Here the rows are the M side: a lane has
// one row, a register one column, and a k-step's scale is one number to a thread.  384 threads:
//   warp 0       TMA producer
//   warps 1, 2   issue the products (2: tensor memory)
//   warp 3       puts the scales of the next eight k-steps into shared memory: a promoting warp that had
//                loads of its own under way would wait for them with its tensor-memory loads
//   warps 4-11   promotion: warp % 4 gives the rows, warps 4-7 and 8-11 the two blocks of 128 columns
// A k-step's 128 x 256 sums take half of the tensor memory; the products fill one half while the other
// is promoted.  The promotion has 256 cycles of additions for the 512 of the products, and as many of
// loads; what it loses it loses between them: what a warp does besides them lies behind a load that is
// under way (776 us where the scales' part lay in front of it).
constexpr int kWideThreads = 384;
constexpr int kWideN = 256;
constexpr int kWideLaunchRegs = 168, kWideControlRegs = 72, kWidePromoteRegs = 216;
static_assert(128 * kWideControlRegs + 256 * kWidePromoteRegs <= kWideThreads * kWideLaunchRegs, "register split");

struct Wide {
    static constexpr int kRows = 128;                                 // of a tile
    static constexpr int kA = kRows * kBK, kB = kWideN * kBK, kStage = kA + kB, kStages = 3;
    // Two barriers to a stage, in turn: a filling is then always waited for by the same one of the two
    // issuing threads.  With one, a thread could come before the other's filling of the stage were
    // complete and take the filling before that for its own.
    static constexpr int kFull = 2 * kStages;
    static constexpr int kOut = 32 * 256;                             // a warp's way out: 32 rows of 256 bytes
    // scales of eight k-steps: one to a row, and one to each half of the columns; two such tables
    static constexpr int kTable = (128 + 2) * kScaleSteps * 4;
    static constexpr int kTiles = 8;   // tiles whose place the producer has told the promoting warps (it is six ahead at most)
    static constexpr int kBytes = 1024 + kStages * kStage + 8 * kOut + 2 * kTable + 512;
};

// acc (columns 2i and 2i + 1 of BASE + ..) += c * v
template <int BASE>
__device__ __forceinline__ void add32(float2 (&acc)[64], const uint32_t (&v)[32], float c) {
#pragma unroll
    for (int i = 0; i < 16; ++i) add2(acc[BASE / 2 + i], v[2 * i], v[2 * i + 1], c, c);
}

// The tiles of a group run through panels of columns whose weights (32 MB at most) stay in the L2, row
// tile by row tile: the rows are then read once for each panel, and the weights once.
__device__ __forceinline__ Tile wide_tile(const ProductArgs &a, const int *prefix, int i) {
    const int q = i / a.nblk;
    int lo = 0, hi = a.G - 1;   // the largest g with prefix[g] <= q
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    const int mt = prefix[lo + 1] - prefix[lo], local = i - prefix[lo] * a.nblk;
    const int panel = a.panel == a.nblk ? 0 : local / (a.panel * mt), in = local - panel * a.panel * mt;
    const int wide = min(a.panel, a.nblk - panel * a.panel), m = in / wide;
    const int begin = row_of(a, lo), end = row_of(a, lo + 1);
    Tile t;
    t.g = lo;
    t.nb = panel * a.panel + in - m * wide;
    t.m0 = begin + m * Wide::kRows;
    t.rows = min(Wide::kRows, end - t.m0);
    return t;
}

__global__ void __launch_bounds__(kWideThreads, 1)
    product_fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_weights,
                            const __grid_constant__ CUtensorMap tm_out, ProductArgs a) {
    using S = Wide;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *out_s = smem + S::kStages * S::kStage;
    float *tables = reinterpret_cast<float *>(out_s + 8 * S::kOut);
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(tables) + 2 * S::kTable);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::kFull + S::kStages + 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int32_t *no_status = reinterpret_cast<int32_t *>(tmem_slot + 2);
    int *wsum = reinterpret_cast<int *>(tmem_slot + 3);                    // [12]
    Tile *tiles = reinterpret_cast<Tile *>(wsum + 12);                     // [kTiles]
    int *prefix = reinterpret_cast<int *>(bars) + 512 / 4;                 // [G + 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S::kFull;
    const uint32_t pfull0 = empty0 + 8 * S::kStages, pempty0 = pfull0 + 16, sfull0 = pfull0 + 32, sempty0 = pfull0 + 48;
    int32_t *status = a.status ? a.status : no_status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kFull; ++s) mbar_init(full0 + 8 * s, 1);
        for (int s = 0; s < S::kStages; ++s) mbar_init(empty0 + 8 * s, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(pfull0 + 8 * b, 1);
            mbar_init(pempty0 + 8 * b, 8);   // one arrival of each promoting warp
            mbar_init(sfull0 + 8 * b, 1);
            mbar_init(sempty0 + 8 * b, 8);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_rows)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_weights)) : "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    const int total = count_tiles(a, S::kRows, prefix, wsum);
    const int first = blockIdx.x, step = gridDim.x;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideControlRegs));
        if (warp == 0 && lane == 0) {
            int stage = 0, place = 0;
            uint32_t phase = 0, nth = 0;
            bool ok = true;
            for (int i = first; i < total && ok; i += step) {
                // (the promoting warps see it with the sums of the tile's first k-step; they are done with
                // the tile eight before: its sums are out of the tensor memory, and the ring and that hold
                // five k-steps)
                const Tile t = tiles[nth++ % S::kTiles] = wide_tile(a, prefix, i);
                for (int k = 0; k < a.kb; ++k) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, status)) { ok = false; break; }
                    const uint32_t fb = full0 + 8 * place, at = smem_u32(smem + stage * S::kStage);
                    mbar_expect_tx(fb, S::kStage);
                    tma_load_2d(at, &tm_rows, k * kBK, t.m0, fb);
                    tma_load_2d(at + S::kA, &tm_weights, k * kBK, t.g * a.N + t.nb * kWideN, fb);
                    if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                    if (++place == S::kFull) place = 0;
                }
            }
        } else if ((warp == 1 || warp == 2) && lane == 0) {
            // Every other k-step of this block, which always goes to the same half of the tensor memory.
            // (One thread's waits and issues for all of them take longer than the products.)
            const uint32_t buf = warp - 1;
            constexpr uint32_t idesc = f8_idesc(S::kRows, kWideN);
            const uint32_t steps = first < total ? (uint32_t)((total - first + step - 1) / step) * a.kb : 0;
            int place = buf;   // it % kFull
            uint32_t phase = 0;
            for (uint32_t it = buf; it < steps; it += 2) {
                if (!mbar_wait(full0 + 8 * place, phase, abort_flag, status)) break;
                if (!mbar_wait(pempty0 + 8 * buf, ((it >> 1) & 1) ^ 1, abort_flag, status)) break;
                tc_fence_after();
                const int stage = place % S::kStages;
                const uint32_t a0 = smem_u32(smem + stage * S::kStage), b0 = a0 + S::kA;
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk)
                    mma_f8(tmem_base + buf * kWideN, sw128_desc(a0 + kk * 32), sw128_desc(b0 + kk * 32), idesc, kk != 0);
                mma_commit(empty0 + 8 * stage);
                mma_commit(pfull0 + 8 * buf);
                place += 2;
                if (place >= S::kFull) { place -= S::kFull; phase ^= 1; }
            }
        } else if (warp == 3) {
            // lane: k-step lane % 8, rows lane / 8 and every fourth behind it, eight at a time
            const int scale_blocks = (a.N + 127) / 128;
            uint32_t turn = 0;
            bool ok = true;
            for (int i = first; i < total && ok; i += step) {
                const Tile t = wide_tile(a, prefix, i);
                const int rows = t.rows;
                const float *sa = a.sa + (int64_t)(t.m0 + (lane >> 3)) * a.kb + (lane & 7);
                const float *sb = a.sb + ((int64_t)t.g * scale_blocks + min(2 * t.nb + (lane >> 3), scale_blocks - 1)) * a.kb + (lane & 7);
                for (int k = 0; k < a.kb; k += kScaleSteps, ++turn) {
                    const uint32_t b = turn & 1;
                    float *tab = tables + b * (S::kTable / 4);   // [128][8], then [2][8]
                    const bool in = k + (lane & 7) < a.kb;
                    const float w = in && lane < 16 ? sb[k] : 0.f;
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        float r[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int at = 4 * (8 * h + j);
                            r[j] = in && at + (lane >> 3) < rows ? sa[(int64_t)at * a.kb + k] : 0.f;
                        }
                        if (h == 0 && !mbar_wait(sempty0 + 8 * b, ((turn >> 1) & 1) ^ 1, abort_flag, status)) { ok = false; break; }
#pragma unroll
                        for (int j = 0; j < 8; ++j) tab[(4 * (8 * h + j) + (lane >> 3)) * kScaleSteps + (lane & 7)] = r[j];
                    }
                    if (!ok) break;
                    if (lane < 16) tab[kScaleSteps * 128 + lane] = w;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sfull0 + 8 * b);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWidePromoteRegs));
        const int quad = warp & 3, half = (warp - 4) >> 2, row = quad * 32 + lane;
        const uint32_t lanes = ((uint32_t)(quad * 32) << 16) + 128 * half;
        uint8_t *way_out = out_s + (warp - 4) * S::kOut;
        uint32_t it = 0, turn = 0;
        float4 sa, sb;        // the next four k-steps' scales, read ahead: shared memory, busy with the
                              // products' operands, answers late
        auto scales = [&](int q) {
            const float4 *tab = reinterpret_cast<const float4 *>(tables + (turn & 1) * (S::kTable / 4));
            sa = tab[2 * row + q];
            sb = tab[2 * (128 + half) + q];
        };
        bool ok = first >= total || mbar_wait(sfull0, 0, abort_flag, status);
        scales(0);
        uint32_t nth = 0;
        for (int i = first; i < total; i += step) {
            float2 acc[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] = make_float2(0.f, 0.f);
            float s[4];
#pragma unroll 2
            for (int k = 0; k < a.kb; ++k) {
                const uint32_t buf = it & 1, from = tmem_base + buf * kWideN + lanes;
                if (!mbar_wait(pfull0 + 8 * buf, (it >> 1) & 1, abort_flag, status)) { ok = false; break; }
                tc_fence_after();
                ++it;
                // the next 32 columns are on their way while 32 are added; the buffer is free as soon as
                // the last are in registers
                uint32_t u[32], v[32];
                tmem_ld(from, u);
                const int q = k & 3;
                if (q == 0) {
                    s[0] = sa.x * sb.x; s[1] = sa.y * sb.y; s[2] = sa.z * sb.z; s[3] = sa.w * sb.w;
                    if (k & 4 || k + 4 >= a.kb) {     // the table's last four
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sempty0 + 8 * (turn & 1));
                        ++turn;
                        if (k + 4 < a.kb || i + step < total)
                            if (!mbar_wait(sfull0 + 8 * (turn & 1), (turn >> 1) & 1, abort_flag, status)) { ok = false; break; }
                        scales(0);                    // (behind the last of all: not used)
                    } else scales(1);
                }
                const float c = q < 2 ? (q ? s[1] : s[0]) : q == 2 ? s[2] : s[3];
                tmem_wait(u);
                tmem_ld(from + 32, v);
                add32<0>(acc, u, c);
                tmem_wait(v);
                tmem_ld(from + 64, u);
                add32<32>(acc, v, c);
                tmem_wait(u);
                tmem_ld(from + 96, v);
                add32<64>(acc, u, c);
                tmem_wait(v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pempty0 + 8 * buf);
                add32<96>(acc, v, c);
            }
            if (!ok) break;
            const Tile done = tiles[nth++ % S::kTiles];
            // Out: the warp's 32 rows of 128 columns, 256 bytes of each row at a time through shared memory:
            // two boxes of 32 rows x 128 bytes, which leave as TMA stores where all rows count
            const int n0 = done.nb * kWideN + 128 * half, cols = min(128, a.N - n0);
            const int m = done.m0 + quad * 32;                 // the warp's first row
            const int valid = min(32, done.rows - quad * 32);  // and how many count
            // (16-byte part c of a box's row r lies at place c ^ (r & 7), the swizzle of the tensor map)
            uint32_t mine = smem_u32(way_out) + lane * 128, swizzle = (lane & 7) << 4;
            // (made here: the compiler would keep all sixteen addresses through the k-steps, which have no
            // register to spare)
            asm volatile("" : "+r"(mine), "+r"(swizzle));
            auto put = [&](int c, uint4 v) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + (c >> 3) * 4096 + (((c & 7) << 4) ^ swizzle)),
                             "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
            };
            auto room = [&] {
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
            };
            auto leave = [&](int c0, int n, int size) {        // columns [c0, c0 + n) of `size` bytes each
                if (a.out_map && valid == 32) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (x * 128 < n * size)
                                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                                 reinterpret_cast<uint64_t>(&tm_out)), "r"(n0 + c0 + x * 128 / size), "r"(m),
                                             "r"(smem_u32(way_out + x * 4096))
                                             : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    return;
                }
                __syncwarp();
                uint8_t *to = static_cast<uint8_t *>(a.out) + ((int64_t)m * a.out_stride + n0 + c0) * size;
                if (a.out_map && n * size % 16 == 0) {         // two rows at a time, 16 bytes to a lane
                    const int at = (lane & 15) * 16;
                    if (at < n * size)
#pragma unroll 4
                        for (int r = lane >> 4; r < valid; r += 2)
                            *reinterpret_cast<uint4 *>(to + r * a.out_stride * size + at) = *reinterpret_cast<const uint4 *>(
                                way_out + (at >> 7) * 4096 + r * 128 + ((at & 127) ^ ((r & 7) << 4)));
                    __syncwarp();
                    return;
                }
                const bool word = !(((uint32_t)reinterpret_cast<uintptr_t>(a.out) | (uint32_t)(a.out_stride * size) |
                                     (uint32_t)(n * size)) & 3);   // four bytes to a lane
                for (int r = 0; r < valid; ++r)
                    for (int at = lane * (word ? 4 : size); at < n * size; at += word ? 128 : 32 * size) {
                        const uint8_t *from = way_out + (at >> 7) * 4096 + r * 128 + ((at & 127) ^ ((r & 7) << 4));
                        uint8_t *there = to + r * a.out_stride * size + at;
                        if (word) *reinterpret_cast<uint32_t *>(there) = *reinterpret_cast<const uint32_t *>(from);
                        else *reinterpret_cast<uint16_t *>(there) = *reinterpret_cast<const uint16_t *>(from);
                    }
                __syncwarp();
            };
            if (a.out_bf16) {
                room();
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float2 *x = acc + 4 * c;
                    put(c, make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                                      pack_bf16(x[3].x, x[3].y)));
                }
                leave(0, cols, 2);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    room();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 x = acc[32 * h + 2 * c], y = acc[32 * h + 2 * c + 1];
                        put(c, make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y)));
                    }
                    leave(64 * h, min(64, cols - 64 * h), 4);
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    if (*abort_flag) {
        const unsigned long long t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {}
    }
    if (warp == 2) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
    }
}

// ------------------------------------------------------------------------------------ host

// A 2-D map of `rows` rows of `cols` elements, `stride` bytes apart, in boxes of 128 bytes.
bool make_rows_map(CUtensorMap *m, const void *base, CUtensorMapDataType type, int size, int64_t rows, int64_t cols,
                   int64_t stride, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride};
    cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_codes_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t stride, int box_rows) {
    return make_rows_map(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, cols, stride, box_rows);
}

// Clusters of `cluster` blocks (1: none), after the kernel before it in the stream.
template <typename K, typename... Args>
int launch_clusters(K kernel, int64_t grid, int cluster, int threads, int smem, cudaStream_t s, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return status_of(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Row tiles there can be: each of several groups may have one that is not full.
int64_t most_tiles(const ProductArgs &p, int rows) {
    if (!p.offsets) return ((int64_t)p.M + rows - 1) / rows;
    return (int64_t)p.M / rows + (p.G < p.M ? p.G : p.M);
}

struct Operands {
    const uint8_t *a, *b;
    int64_t a_stride, K;
};

template <int NT>
int launch_narrow(ProductArgs p, const Operands &o, cudaStream_t s) {
    using S = Narrow<NT>;
    CUtensorMap rows, weights;
    if (!make_codes_map(&rows, o.a, p.M, o.K, o.a_stride, NT) ||
        !make_codes_map(&weights, o.b, (int64_t)p.G * p.N, o.K, o.K, kTileN))
        return MOE_ERR_CUDA;
    auto kernel = product_fp8_kernel<NT>;
    const int smem = S::kBytes + (p.G + 1) * 4;
    static PerDevice devices;
    const cudaError_t e = devices.set(kernel, S::kBytes + (MOE_MAX_EXPERTS + 1) * 4,
                                      [](int) { return cudaSuccess; });
    if (e != cudaSuccess) return status_of(e);
    p.most_rows = (int)most_tiles(p, NT);
    const int64_t most = (int64_t)p.most_rows * p.nblk;
    if (most >= ((int64_t)1 << 31)) return MOE_ERR_LIMIT;
    const int sms = num_sms();
    const int64_t grid = p.split > 1 ? most * p.split : (most < sms ? most : sms);
    return launch_clusters(kernel, grid, p.split, kThreads, smem, s, rows, weights, p);
}

int launch_wide(ProductArgs p, const Operands &o, cudaStream_t s) {
    using S = Wide;
    CUtensorMap rows, weights;
    if (!make_codes_map(&rows, o.a, p.M, o.K, o.a_stride, S::kRows) ||
        !make_codes_map(&weights, o.b, (int64_t)p.G * p.N, o.K, o.K, kWideN))
        return MOE_ERR_CUDA;
    const int size = p.out_bf16 ? 2 : 4;
    CUtensorMap out = rows;      // (not looked at without out_map)
    p.out_map = is_aligned(p.out, 16) && p.out_stride * size % 16 == 0 && p.out_stride * size < ((int64_t)1 << 40);
    if (p.out_map && !make_rows_map(&out, p.out, p.out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                                    size, p.M, p.N, p.out_stride * size, 32))
        return MOE_ERR_CUDA;
    auto kernel = product_fp8_wide_kernel;
    static PerDevice devices;
    const cudaError_t e = devices.set(kernel, S::kBytes + (MOE_MAX_EXPERTS + 1) * 4, [&](int) {
        // setmaxnreg.inc waits for registers that the launch has to have: never launch a build whose
        // count makes the split too large
        cudaFuncAttributes fa{};
        const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e == cudaSuccess && fa.numRegs * kWideThreads < 128 * kWideControlRegs + 256 * kWidePromoteRegs)
            return cudaErrorInvalidConfiguration;
        return e;
    });
    if (e != cudaSuccess) return status_of(e);
    p.nblk = (p.N + kWideN - 1) / kWideN;
    const int64_t panel = ((int64_t)32 << 20) / (kWideN * o.K);
    p.panel = panel < 1 ? 1 : panel < p.nblk ? (int)panel : p.nblk;
    p.most_rows = (int)most_tiles(p, S::kRows);
    const int64_t most = (int64_t)p.most_rows * p.nblk;
    if (most >= ((int64_t)1 << 31)) return MOE_ERR_LIMIT;
    const int64_t grid = most < num_sms() ? most : num_sms();
    return launch_clusters(kernel, grid, 1, kWideThreads, S::kBytes + (p.G + 1) * 4, s, rows, weights, out, p);
}

struct Choice {
    int rows, split;   // rows of a tile (0: the wide tiles), blocks that share one
};

// The tiles with the least estimated time.  A tile's k-steps take `step` ns each (measured: a narrow
// tile's operands at 80 to 90 GB/s for an SM up to 64 rows, its promotion at 128; a wide tile's promotion),
// what comes before and after them about 1 us (wide: 1.5), sharing a tile 1 to 2 us more (among 8 blocks
// up to 3).  Several groups' weights come from HBM, 16 KB (wide: 32) for a k-step, and a group of r rows is
// taken for r / rows + 1/2 row tiles, as the rows of groups of different sizes come to.
// Measured, us, by tiles of 16, 32, 64 and 128 rows (with the split that the rule gives them) and wide ones; the
// rule takes the least of each line, or what is within 0.2% of it:
//     rows x n x k             1 x 4096 x 7168    7.6   8.4  10.6  14.9   29.4
//                             64 x 4096 x 7168   14.6  11.7  10.1  12.9   30.7
//                            128 x 4096 x 7168   25.6  16.1  14.5  14.3   33.6
//                            512 x 4096 x 7168   80.5  52.6  39.6  34.5   33.4
//                            777 x 1003 x 1408   11.1  10.3   9.0  11.6   16.8
//     256 groups, 8 rows each, 4096 x 7168        1061  1077  1085  1503   1135
//                16 rows                          1129  1095  1097  1514   1143
//                32 rows                          1547  1179  1134  1538   1155
//                64 rows                          2769  1678  1442  1711   1213
Choice choose_tiles(const ProductArgs &p) {
    static const struct { int rows, n, step, around; } kTiles[] = {
        {16, kTileN, 200, 1000}, {32, kTileN, 230, 1000}, {64, kTileN, 320, 1000}, {128, kTileN, 550, 1000}, {0, kWideN, 500, 1500}};
    const int64_t sms = num_sms();
    Choice best{16, 1};
    int64_t least = INT64_MAX;
    for (const auto &t : kTiles) {
        const int rows = t.rows ? t.rows : Wide::kRows;
        const int64_t blocks = (p.N + t.n - 1) / t.n, most = most_tiles(p, rows) * blocks;
        int64_t tiles = most;
        int step = t.step;
        if (p.offsets) {
            const int64_t groups = p.G < p.M ? p.G : p.M, halves = 2 * (int64_t)p.M / rows + groups;
            tiles = (halves > 2 * groups ? halves : 2 * groups) * blocks / 2;
            const int weights = t.rows ? 370 : 800;
            step = step > weights ? step : weights;
        }
        for (int split = 1; split <= (t.rows ? kMaxSplit : 1); split *= 2) {
            if (split > 1 && (most * split > sms || p.kb < 4 * split)) break;
            const int64_t waves = (tiles * split + sms - 1) / sms;
            const int64_t ns = waves * ((p.kb + split - 1) / split * (int64_t)step + t.around) +
                               (split > 1 ? 1000 + 8 * rows : 0) + (split == 8 ? 25 * rows : 0);
            if (ns < least) {
                least = ns;
                best = {t.rows, split};
            }
        }
    }
    return best;
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
                     p->k / kBK, p->groups ? p->groups : 1, (p->n + kTileN - 1) / kTileN, 1, 0, 1,
                     p->out_dtype == MOE_DTYPE_BF16, 0, 0};
    const size_t four = 4 * dtype_bytes(p->out_dtype);
    args.out_fours = is_aligned(out_dev, four) && out_stride % 4 == 0;
    const Operands o{a_dev, b_dev, a_stride, p->k};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Choice c = choose_tiles(args);
    args.split = c.split;
    switch (c.rows) {
    case 16: return launch_narrow<16>(args, o, s);
    case 32: return launch_narrow<32>(args, o, s);
    case 64: return launch_narrow<64>(args, o, s);
    case 128: return launch_narrow<128>(args, o, s);
    default: return launch_wide(args, o, s);
    }
}
