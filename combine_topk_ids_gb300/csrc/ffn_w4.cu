// The routed experts' SwiGLU FFN of a decode batch with 4-bit weights (moe_forward_w4), the
// weights' one-time order (moe_prepare_weights_w4) and their quantisation (moe_quantize_w4);
// declared in include/moe_block.h.
//
//     out[t] = sum_j w[t, j] * W2_e (silu(Wg_e x[t]) * (Wu_e x[t])),   W = (code - 8) * scale
//
// A decode batch has few rows for each expert, so the time is that of reading the picked
// experts' codes once, and what the kernels may spend on a code is little: at the HBM's rate
// an SM has 22 cycles for the 1024 codes of 16 weight rows x 64 inputs, and its four
// schedulers 88 instructions.  So
//   - warp-level matrix instructions (16 weight rows x 16 inputs x 8 batch rows) take the
//     codes almost as they are stored: the f16 numbers whose low bits are n and 16 n are
//     n * 2^-24 and n * 2^-20, so a mask over a word of eight codes gives two matrix elements,
//     and five instructions all eight.  (A tcgen05 tile's other side would be nearly empty,
//     and its codes would have to pass through shared memory again.)
//   - the 8 that a code is above its weight comes off through the sums of the inputs, where
//     the matrix sum starts;
//   - the inputs are f16 too: 64 of them at a time are divided by a power of two that brings
//     the largest to 2^14 .. 2^15 (W4Inputs).  f16 holds the eight bits of x exactly
//     (while the 64 lie within 2^32 of each other; below that, to 2^-39 of the largest); the
//     activation is rounded to its eleven, eight times finer than out's own rounding.
// Products are exact, sums float32.  A block takes eight tiles of 16 weight rows; for 256
// inputs at a time one warp copies their codes and scales (contiguous in the prepared order)
// and the picks' inputs to a ring of stages in shared memory, and eight warps compute: two
// groups of four, two tiles a warp, take turns at the stages and add up at the end.  (A unit
// then has two warps on each scheduler even where there are fewer units than room for them.)
//
// Measured (hidden 7168, 256 experts, top-8, intermediate 2048, a scale per 128): 64 tokens
// (5.05 GB of picked experts) 820 us, 6.2 TB/s, 0.92 of the measured HBM peak; one token (182 MB)
// 48 us, 0.57: its 256 units of the first product are 1.7 to an SM, and the SMs that have two set
// the time.  16 tokens, hidden 4096, 8 experts, top-2, intermediate 14336, a scale per 64 (741 MB):
// 132 us, 0.84.  The instructions (51 for 1024 codes) and the HBM are close to each other at the
// first: the same products on bf16 fragments took 100 and 1350 us, on e4m3 ones, whose warp-level
// instruction GB300 emulates, 2150 us.
#include <cuda_fp16.h>

#include "block_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int kW4Tiles = 8;    // tiles of 16 weight rows that a block takes at a time
constexpr int kW4Warps = 4;    // computing warps of a group, two tiles each
constexpr int kW4Threads = (2 * kW4Warps + 1) * 32;   // two groups, and one more warp that copies
constexpr int kW4Blocks = 2;   // blocks on an SM
constexpr int kW4Picks = 8;    // picks of one expert taken together
constexpr int kW4FewPicks = 1024;   // up to which every block counts its pick's place itself

// What goes with 64 f16 inputs of one row.  e: the power of two that they are to be multiplied
// with; sum: theirs, of either 32, times -8 * 2^-24.
struct __align__(16) W4Tail {
    float e, sum[2], pad;
};

// 128 inputs of the row at `place` of the picks' order by expert, as a stage holds them.  The
// inputs of eight rows from anywhere on lie on the banks that the eight lanes of a
// shared-memory phase (two rows, four 16-byte pieces) want: 64 bytes past a multiple of 128
// apart.  The tails of every other row take different slots.
struct __align__(16) W4Inputs {
    uint16_t v[128];
    W4Tail tail[4];
    static __host__ __device__ __forceinline__ int slot(int place, int half) { return ((place >> 1) + 2 * half) & 3; }
};
static_assert(sizeof(W4Inputs) == 320, "W4Inputs");

struct W4Plan {
    int64_t T, H, E, k, I, P, G;
    size_t head, entries, picks, x, act, y, total;   // workspace offsets
};

// One run of up to kW4Picks picks of one expert.  An expert's runs follow each other; they work
// through the same weights at the same time (W4Item).
struct __align__(16) W4Entry {
    int32_t expert, first, runs, begin, end, pad[3];   // the expert's first entry and their number; its places
};
static_assert(sizeof(W4Entry) == 32, "W4Item reads the first four at once");

struct W4Args {
    const uint16_t *x;
    const void *ids;
    const float *weights;
    const uint8_t *w1, *w2;
    const uint8_t *s1, *s2;
    uint16_t *out;
    W4Inputs *xq, *act;         // [H / 128][P], [I / 128][P]: by place
    float *y;                   // [P][H]
    int32_t *status, *entries_used, *picks, *places;   // picks: by place; places: by pick
    W4Entry *entries;
    int T, H, E, k, I, P, ids64, placed;
};

__device__ __forceinline__ int load_id(const W4Args &a, int64_t p) {
    const int64_t v = a.ids64 ? static_cast<const int64_t *>(a.ids)[p] : static_cast<const int32_t *>(a.ids)[p];
    return v >= 0 && v < a.E ? (int)v : v == -1 ? -1 : -2;
}

// 1 / e and e for the largest magnitude m of 64 inputs.
__device__ __forceinline__ void power_scale(float m, float &down, float &e) {
    const int b = min(max((int)(__float_as_uint(m) >> 23), 15), 254);   // m >= 0
    down = __uint_as_float((uint32_t)(268 - b) << 23);
    e = __uint_as_float((uint32_t)(b - 14) << 23);
}

// The place of pick p of expert e in the order by expert and pick: the valid picks before it.
// All threads of the block call it.
__device__ __forceinline__ int place_of(const W4Args &a, int p, int e) {
    int before = 0;
    for (int i = 0; i < a.P; i += 1024) {
        const int o = i + (int)threadIdx.x < a.P ? load_id(a, i + threadIdx.x) : -1;
        before += __syncthreads_count(o >= 0 && (o < e || (o == e && i + (int)threadIdx.x < p)));
    }
    return before;
}

// The f16 inputs of pick p: a warp to each 128 of them, half a warp to each 64.
__device__ __forceinline__ void w4_inputs_of_x(const W4Args &a, int p) {
    const int lane = threadIdx.x & 31;
    const int e = load_id(a, p);
    if (e < 0) return;
    const int place = a.placed ? a.places[p] : place_of(a, p, e);
    for (int b = threadIdx.x >> 5; b < a.H / 128; b += 32) {
        const uint2 in = reinterpret_cast<const uint2 *>(a.x + (int64_t)(p / a.k) * a.H + b * 128)[lane];
        float m = fmaxf(fmaxf(fabsf(lo_f32(in.x)), fabsf(hi_f32(in.x))), fmaxf(fabsf(lo_f32(in.y)), fabsf(hi_f32(in.y))));
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, o));
        float down, scale;
        power_scale(m, down, scale);
        const __half2 h0 = __floats2half2_rn(lo_f32(in.x) * down, hi_f32(in.x) * down);
        const __half2 h1 = __floats2half2_rn(lo_f32(in.y) * down, hi_f32(in.y) * down);
        float sum = (__low2float(h0) + __high2float(h0)) + (__low2float(h1) + __high2float(h1));
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
        W4Inputs &r = a.xq[(int64_t)b * a.P + place];
        reinterpret_cast<__half2 *>(r.v)[2 * lane] = h0;
        reinterpret_cast<__half2 *>(r.v)[2 * lane + 1] = h1;
        W4Tail &tail = r.tail[W4Inputs::slot(place, lane / 16)];
        if (lane % 8 == 0) tail.sum[lane / 8 % 2] = sum * -0x1p-21f;
        if (lane % 16 == 0) tail.e = scale;
    }
}

// Block 0 orders the picks by expert and lists the entries.  The others prepare x, counting
// their pick's place themselves where there are few picks: one launch less; for many,
// w4_inputs_kernel does it with the places that block 0 left (`placed`).
__global__ void __launch_bounds__(1024) w4_group_kernel(W4Args a) {
    __shared__ int32_t count[MOE_MAX_EXPERTS], sums[64];
    __shared__ int32_t bad;
    pdl_begin();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x > 0) {
        w4_inputs_of_x(a, blockIdx.x - 1);
        return;
    }
    for (int e = tid; e < MOE_MAX_EXPERTS; e += 1024) count[e] = 0;
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int64_t p = tid; p < a.P; p += 1024) {
        const int e = load_id(a, p);
        if (e >= 0) atomicAdd(&count[e], 1);
        if (e == -2) bad = 1;
    }
    __syncthreads();
    // exclusive sums over the experts, two per thread: picks, and entries
    const int c[2] = {count[2 * tid], count[2 * tid + 1]};
    const int n[2] = {(c[0] + kW4Picks - 1) / kW4Picks, (c[1] + kW4Picks - 1) / kW4Picks};
    int picks = c[0] + c[1], runs = n[0] + n[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int r = __shfl_up_sync(kAllLanes, picks, o), u = __shfl_up_sync(kAllLanes, runs, o);
        if (lane >= o) {
            picks += r;
            runs += u;
        }
    }
    if (lane == 31) {
        sums[warp] = picks;
        sums[32 + warp] = runs;
    }
    __syncthreads();
    int r = picks - c[0] - c[1], u = runs - n[0] - n[1];
    for (int w = 0; w < warp; ++w) {
        r += sums[w];
        u += sums[32 + w];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        for (int i = 0; i < n[j]; ++i)
            a.entries[u + i] = W4Entry{2 * tid + j, u, n[j], r + i * kW4Picks, r + min((i + 1) * kW4Picks, c[j]), {}};
        count[2 * tid + j] = r;
        r += c[j];
        u += n[j];
    }
    if (tid == 1023) {
        *a.entries_used = u;
        *a.status = bad ? MOE_STATUS_BAD_EXPERT_ID : 0;
    }
    __syncthreads();
    // places in pick order: 32 picks at a time, warp after warp
    for (int64_t p0 = 0; p0 < a.P; p0 += 1024) {
        const int64_t p = p0 + tid;
        const int e = p < a.P ? load_id(a, p) : -1;
        const unsigned same = __match_any_sync(kAllLanes, e);
        const int first = __ffs(same) - 1;
        const int warps = (int)min((a.P - p0 + 31) / 32, (int64_t)32);
        for (int w = 0; w < warps; ++w) {
            if (warp == w) {
                int base = 0;
                if (e >= 0 && lane == first) {
                    base = count[e];
                    count[e] = base + __popc(same);
                }
                base = __shfl_sync(kAllLanes, base, first);
                if (e >= 0) {
                    const int place = base + __popc(same & ((1u << lane) - 1));
                    a.picks[place] = (int)p;
                    a.places[p] = place;
                }
            }
            __syncthreads();
        }
    }
}

__global__ void __launch_bounds__(1024) w4_inputs_kernel(W4Args a) {
    pdl_begin();
    w4_inputs_of_x(a, blockIdx.x);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                        float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// What a block works on at a time: kW4Tiles tiles of weight rows for one entry's picks.  The
// units (entry, tiles) of the call go from block to block; an expert's entries take the same
// tiles in neighbouring blocks, so that its weights come from memory once.
struct W4Item {
    int64_t group;       // of tiles, in the matrix
    int i, begin, n;     // of tiles, in the expert; the picks a.picks[begin .. begin + n)

    // EARLY: before the dependency wait, past the L1.
    template <bool EARLY = false>
    __device__ __forceinline__ bool load(const W4Args &a, int64_t u, int groups, int64_t units) {
        if (u >= units) return false;
        auto get = [](const int4 *p) { return EARLY ? __ldcg(p) : *p; };
        const int entry = units < ((int64_t)1 << 31) ? (int)u / groups : (int)(u / groups);
        const int4 *e = reinterpret_cast<const int4 *>(a.entries + entry);
        int4 x = get(e);            // expert, first, runs, begin
        int4 y = get(e + 1);        // end
        i = (int)(u - (int64_t)entry * groups);
        if (x.z > 1) {
            const int local = (int)(u - (int64_t)x.y * groups);   // in the expert's entries
            i = local / x.z;
            e = reinterpret_cast<const int4 *>(a.entries + x.y + (local - i * x.z));
            x = get(e);
            y = get(e + 1);
        }
        group = (int64_t)x.x * groups + i;
        begin = x.w;
        n = y.x - begin;
        return true;
    }
};

// A stage holds 256 inputs, the last of a unit 128 where their number is odd: the tiles' codes,
// then their scales, then the rows, 128 inputs after the other.
template <int G>
struct W4Stage {
    static constexpr int kPairs = 128 / G;   // scale pairs (rows g, g + 8) per 128 inputs
    static constexpr int kCodes = kW4Tiles * 1024, kScales = kW4Tiles * 32 * kPairs;   // of 128 inputs
    static constexpr int kRows = kW4Picks * (int)sizeof(W4Inputs);
    static constexpr int kBytes = 2 * (kCodes + kScales + kRows);
    // An even number: a slot's stages then all go to the same group of warps, which so waits for a
    // slot's next filling only after it has used the last one (a barrier tells no more than
    // two fillings apart).  7 KB are left to other arrays.
    static constexpr int kStages = (227 * 1024 / kW4Blocks - 8 * 1024) / kBytes / 2 * 2;
    static_assert(kStages >= 4, "stages");
};

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 128 inputs for the warp's two tiles: acc[t] += tile t times the picks.  codes, scales, x: this
// lane's in the stage; tails[j]: the first 64 inputs' tail of pick 2q + j (the second 64 inputs'
// lies two slots on: the slots are 64 bytes from a multiple of 64 on).
template <int G>
__device__ __forceinline__ void w4_compute(const uint4 *w, const uint32_t *sc, const uint4 *x, const uint8_t *base,
                                           const int (&tails)[2], float (&acc)[2][4]) {
    constexpr int kPairs = W4Stage<G>::kPairs;
    float s0[2], s1[2];   // scales of rows g, g + 8
#pragma unroll
    for (int c = 0; c < 2; ++c) {   // 64 inputs
        const uint4 b[2] = {x[c * 8], x[c * 8 + 4]};
        W4Tail tail[2];             // of this lane's columns of sums
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float4 *>(&tail[j]) = *reinterpret_cast<const float4 *>(base + (tails[j] ^ (c * 2 * (int)sizeof(W4Tail))));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint4 v = w[t * 64 + c * 32];
            float part[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {   // 16 inputs, a matrix step
                const uint32_t w0 = s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w, w1 = w0 >> 8;
                const uint32_t f[4] = {w0 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x000f000fu, w1 & 0x00f000f0u};
                const uint32_t b0 = s % 2 ? b[s / 2].z : b[s / 2].x, b1 = s % 2 ? b[s / 2].w : b[s / 2].y;
                if (s == 0 || (s == 2 && G == 32)) {   // the sum starts at -8 times the inputs' sum
                    const float z0 = G == 32 ? tail[0].sum[s / 2] : tail[0].sum[0] + tail[0].sum[1];
                    const float z1 = G == 32 ? tail[1].sum[s / 2] : tail[1].sum[0] + tail[1].sum[1];
                    mma_f16(part, f, b0, b1, z0, z1, 16.f * z0, 16.f * z1);
                } else {
                    mma_f16(part, f, b0, b1, part[0], part[1], part[2], part[3]);
                }
                if (s == 3 || (s == 1 && G == 32)) {   // the end of a scale's group or of the 64 inputs
                    if (c == 0 || G < 128) {
                        const uint32_t sp = sc[t * 8 * kPairs + (c * 64 + s * 16) / G];
                        s0[t] = lo_f32(sp);
                        s1[t] = hi_f32(sp);
                    }
                    acc[t][0] = fmaf(s0[t] * tail[0].e, part[0], acc[t][0]);
                    acc[t][1] = fmaf(s0[t] * tail[1].e, part[1], acc[t][1]);
                    acc[t][2] = fmaf(s1[t] * tail[0].e, part[2], acc[t][2]);
                    acc[t][3] = fmaf(s1[t] * tail[1].e, part[3], acc[t][3]);
                }
            }
        }
    }
}

__device__ __forceinline__ float silu(float v) { return __fdiv_rn(v, 1.0f + expf(-v)); }

// Named barriers of the computing warps: the first group's own, "sums written", "sums read".
enum { kBarFirst = 1, kBarWritten = 2, kBarRead = 3 };
template <int THREADS>
__device__ __forceinline__ void bar_sync(int bar) { asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(THREADS) : "memory"); }
template <int THREADS>
__device__ __forceinline__ void bar_arrive(int bar) { asm volatile("bar.arrive %0, %1;" ::"r"(bar), "n"(THREADS) : "memory"); }

// UP: the first product and the activation; else the second product.
template <bool UP, int G>
__global__ void __launch_bounds__(kW4Threads, kW4Blocks) w4_product_kernel(W4Args a) {
    using S = W4Stage<G>;
    extern __shared__ __align__(128) uint8_t stages[];   // [kStages][kBytes]
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages];
    __shared__ __align__(16) uint16_t acts[8][64];
    __shared__ float top[kW4Warps][8], sums[kW4Warps][8], scale[8];
    __shared__ float others[2 * 4][kW4Warps * 32];   // the second group's sums
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
    // The first product lets the second one start as blocks of it end: that one's copying warp
    // then fetches weights, which depend on the grouping alone, before it waits for the activation.
    if (UP) pdl_begin();
    pdl_trigger();
    const int blocks = (UP ? a.H : a.I) / 128, steps = (blocks + 1) / 2;   // 128 inputs, and stages, of a unit
    const int groups = (UP ? a.I / 8 : a.H / 16) / kW4Tiles;
    const int entries = __ldcg(a.entries_used);
    const int64_t units = (int64_t)entries * groups;
    W4Item it;

    if (warp == 2 * kW4Warps) {   // the copying warp: lane 0 the codes, 1 the scales, 2 and 3 the rows
        int put = 0, stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        bool have = it.load<!UP>(a, blockIdx.x, groups, units);
        for (int64_t u = blockIdx.x; ok && have; u += gridDim.x, have = it.load(a, u, groups, units)) {
            const uint8_t *src;
            uint32_t bytes, off;   // of 128 inputs
            int64_t step;          // from one stage's source to the next
            if (lane == 0) {
                src = (UP ? a.w1 : a.w2) + it.group * blocks * S::kCodes;
                bytes = S::kCodes;
                step = 2 * S::kCodes;
                off = 0;
            } else if (lane == 1) {
                src = (UP ? a.s1 : a.s2) + it.group * blocks * S::kScales;
                bytes = S::kScales;
                step = 2 * S::kScales;
                off = 2 * S::kCodes;
            } else {   // the rows of either 128 inputs
                src = reinterpret_cast<const uint8_t *>((UP ? a.xq : a.act) + (lane == 3 ? (int64_t)a.P : 0) + it.begin);
                bytes = it.n * (uint32_t)sizeof(W4Inputs);
                step = 2 * (int64_t)a.P * sizeof(W4Inputs);
                off = 2 * (S::kCodes + S::kScales) + (lane == 3 ? S::kRows : 0);
            }
            int ahead = 0;   // stages of this unit whose weights are under way already
            if (!UP && put == 0) {
                for (; ahead < min(steps, S::kStages); ++ahead) {
                    const uint32_t bar = smem_u32(full + ahead), two = 2 * ahead + 1 < blocks ? 2 : 1;
                    if (lane == 0) mbar_expect_tx(bar, two * (S::kCodes + S::kScales + it.n * (uint32_t)sizeof(W4Inputs)));
                    __syncwarp();
                    if (lane < 2)
                        bulk_copy(smem_u32(stages) + ahead * S::kBytes + off, src + ahead * step, two * bytes, bar);
                }
                pdl_begin();
            }
            for (int b = 0; b < steps; ++b) {
                ok = mbar_wait(smem_u32(empty + stage), phase ^ 1, &abort_flag, a.status);
                ok = __all_sync(kAllLanes, ok);
                if (!ok) break;
                const uint32_t bar = smem_u32(full + stage), two = 2 * b + 1 < blocks ? 2 : 1;
                if (b >= ahead) {
                    if (lane == 0)
                        mbar_expect_tx(bar, two * (S::kCodes + S::kScales + it.n * (uint32_t)sizeof(W4Inputs)));
                    __syncwarp();
                }
                if (lane < 2 + two && (lane >= 2 || b >= ahead))
                    bulk_copy(smem_u32(stages) + stage * S::kBytes + off, src, lane < 2 ? two * bytes : bytes, bar);
                src += step;
                ++put;
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!UP && put == 0) pdl_begin();   // no unit: the kernel still ends after the one before
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

    // A warp whose wait ran out (the status word then holds MOE_STATUS_TIMEOUT) goes on through
    // the units without waiting or computing: the others may stand at a barrier.
    if (!UP) pdl_begin();
    const int g = lane >> 2, q = lane & 3, group = warp / kW4Warps, w = warp % kW4Warps;
    bool ok = true, written = false;
    int put = 0;   // stages of the units so far
    for (int64_t u = blockIdx.x; it.load(a, u, groups, units); u += gridDim.x) {
        float acc[2][4] = {};
        int tails[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            tails[j] = (2 * q + j) * (int)sizeof(W4Inputs) + (int)offsetof(W4Inputs, tail) +
                       W4Inputs::slot(it.begin + 2 * q + j, 0) * (int)sizeof(W4Tail);
        const int first = group ^ (put & 1);   // the group takes the slots of its own parity
        int stage = (put + first) % S::kStages;
        uint32_t phase = (put + first) / S::kStages & 1;
        for (int b = first; b < steps && ok; b += 2) {
            ok = mbar_wait(smem_u32(full + stage), phase, &abort_flag, a.status);
            ok = __all_sync(kAllLanes, ok);
            if (!ok) break;
            const uint8_t *at = stages + stage * S::kBytes;
            const uint4 *codes = reinterpret_cast<const uint4 *>(at) + w * 2 * 64 + lane;
            const uint32_t *sc = reinterpret_cast<const uint32_t *>(at + 2 * S::kCodes) + (w * 2 * 8 + g) * S::kPairs;
            const uint8_t *rows = at + 2 * (S::kCodes + S::kScales);
            const uint4 *x = reinterpret_cast<const uint4 *>(rows + g * sizeof(W4Inputs)) + q;
            w4_compute<G>(codes, sc, x, rows, tails, acc);
            if (2 * b + 1 < blocks)
                w4_compute<G>(codes + S::kCodes / 16, sc + S::kScales / 4, x + S::kRows / 16, rows + S::kRows, tails, acc);
            __syncwarp();   // every lane has read the stage
            if (lane == 0) mbar_arrive(smem_u32(empty + stage));
            stage += 2;
            if (stage >= S::kStages) {
                stage -= S::kStages;
                phase ^= 1;
            }
        }
        put += steps;
        // the even stages' sum plus the odd stages' (or the other way round, which is the same)
        if (group == 1) {
            if (written) bar_sync<kW4Warps * 64>(kBarRead);
            written = true;
#pragma unroll
            for (int i = 0; i < 2 * 4; ++i) others[i][threadIdx.x - kW4Warps * 32] = acc[i / 4][i % 4];
            bar_arrive<kW4Warps * 64>(kBarWritten);
            continue;
        }
        bar_sync<kW4Warps * 64>(kBarWritten);
#pragma unroll
        for (int i = 0; i < 2 * 4; ++i) acc[i / 4][i % 4] += others[i][threadIdx.x];
        bar_arrive<kW4Warps * 64>(kBarRead);
        // the codes' 2^-24 (rows 0..7 of a tile) and 2^-20 (rows 8..15)
        if constexpr (UP) {
            // Rows 0..7 of a tile are gate rows, 8..15 the same up rows: a lane has both factors
            // of inputs 16 w + 8t + g of the unit's 64, of picks 2q and 2q + 1.
            float h[2][2];   // [tile][pick]
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) h[t][j] = silu(acc[t][j] * 0x1p24f) * (acc[t][2 + j] * 0x1p20f);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float m = fmaxf(fabsf(h[0][j]), fabsf(h[1][j]));
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, o));
                if (g == 0) top[w][2 * q + j] = m;
            }
            bar_sync<kW4Warps * 32>(kBarFirst);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = 2 * q + j;
                float down, e;
                power_scale(fmaxf(fmaxf(top[0][c], top[1][c]), fmaxf(top[2][c], top[3][c])), down, e);
                const __half2 v = __floats2half2_rn(h[0][j] * down, h[1][j] * down);
                acts[c][16 * w + g] = __half_as_ushort(__low2half(v));
                acts[c][16 * w + 8 + g] = __half_as_ushort(__high2half(v));
                float sum = __low2float(v) + __high2float(v);
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
                if (g == 0) sums[w][c] = sum;
                if (g == 0 && w == 0) scale[c] = e;
            }
            bar_sync<kW4Warps * 32>(kBarFirst);
            const int c = threadIdx.x >> 3, v = threadIdx.x & 7;   // pick, 8 of its 64 inputs
            if (c < it.n) {
                const int place = it.begin + c;
                W4Inputs &o = a.act[(int64_t)(it.i >> 1) * a.P + place];
                reinterpret_cast<uint4 *>(o.v)[(it.i & 1) * 8 + v] = reinterpret_cast<const uint4 *>(acts[c])[v];
                if (v == 0)
                    *reinterpret_cast<float4 *>(&o.tail[W4Inputs::slot(place, it.i & 1)]) =
                        make_float4(scale[c], (sums[0][c] + sums[1][c]) * -0x1p-21f, (sums[2][c] + sums[3][c]) * -0x1p-21f, 0.f);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = 2 * q + j;
                if (c >= it.n) continue;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float *o = a.y + (int64_t)a.picks[it.begin + c] * a.H + (it.i * kW4Tiles + w * 2 + t) * 16 + g;
                    o[0] = acc[t][j] * 0x1p24f;
                    o[8] = acc[t][2 + j] * 0x1p20f;
                }
            }
        }
    }
    if (written) bar_sync<kW4Warps * 64>(kBarRead);
}

// out[t] = sum over the picks, in their order, of weight * y; a block to 1024 columns of a token.
__global__ void __launch_bounds__(128) w4_combine_kernel(W4Args a) {
    pdl_begin();
    const int64_t t = blockIdx.x;
    const int c = blockIdx.y * 1024 + threadIdx.x * 8;
    if (c >= a.H) return;
    float o[8] = {};
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {   // (a masked pick's y and weight are read, in bounds, and not used)
        const int64_t p = t * a.k + j;
        const bool used = load_id(a, p) >= 0;
        const float w = a.weights[p];
        const float4 *y = reinterpret_cast<const float4 *>(a.y + p * a.H + c);
        const float4 y0 = y[0], y1 = y[1];
        if (used) {
            o[0] = fmaf(w, y0.x, o[0]); o[1] = fmaf(w, y0.y, o[1]); o[2] = fmaf(w, y0.z, o[2]); o[3] = fmaf(w, y0.w, o[3]);
            o[4] = fmaf(w, y1.x, o[4]); o[5] = fmaf(w, y1.y, o[5]); o[6] = fmaf(w, y1.z, o[6]); o[7] = fmaf(w, y1.w, o[7]);
        }
    }
    *reinterpret_cast<uint4 *>(a.out + t * a.H + c) =
        make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
}

// Prepared order.  A tile is 16 weight rows: half = rows / 2 > 0 pairs rows i0 .. i0 + 7 with
// rows half + i0 .. (gate and up of w1), half == 0 takes 16 consecutive rows.  For 64 inputs
// from k0 on, lane (g, q) of a tile holds rows g and g + 8 of inputs k0 + 32h + 8q .. + 7, h =
// 0, 1: word 2h + s has inputs 4s .. 4s + 3 of these in its bytes 0, 2, 1, 3, row g's code in a
// byte's low half and row g + 8's in its high one.  The order is [8 tiles][128 inputs][tile][64 inputs][lane];
// one thread per lane and 64 inputs.
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

// One thread per group.  A group that holds an infinity or NaN has no scale: it gets NaN, so that
// its weights are NaN, and code 8.  (Done once for a model's weights, and not tuned: 939 M weights,
// a scale per 128, 5.1 ms against 0.35 for their bytes; neighbouring threads read 256 bytes apart.)
__global__ void __launch_bounds__(256) w4_quantize_kernel(const uint16_t *w, uint8_t *codes, uint16_t *scales,
                                                          int64_t n, int G) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n) return;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(w + v * G);
    float m = 0.f;
    bool finite = true;
    for (int i = 0; i < G / 2; ++i) {
        const float a = fabsf(lo_f32(src[i])), b = fabsf(hi_f32(src[i]));
        finite = finite && a < __builtin_huge_valf() && b < __builtin_huge_valf();
        m = fmaxf(m, fmaxf(a, b));
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(finite ? __fdiv_rn(m, 7.0f) : __builtin_nanf(""));
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
    p->head = take(4);
    p->entries = take(sizeof(W4Entry) * (p->P < p->E ? p->P : p->E) + sizeof(W4Entry) * (p->P / kW4Picks));
    p->picks = take(8 * p->P);
    p->x = take(sizeof(W4Inputs) * p->P * (p->H / 128));
    p->act = take(sizeof(W4Inputs) * p->P * (p->I / 128));
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
cudaError_t launch_product_of(const W4Args &a, int64_t units, cudaStream_t s) {
    constexpr int smem = W4Stage<G>::kStages * W4Stage<G>::kBytes;
    static std::once_flag once[64];   // per device
    static cudaError_t set[64];
    const int dev = device_ordinal();
    if (dev < 0) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(w4_product_kernel<UP, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    const int64_t most = kW4Blocks * (int64_t)num_sms();
    return launch_pdl(w4_product_kernel<UP, G>, dim3((unsigned)(units < most ? units : most)), dim3(kW4Threads), smem,
                      s, a);
}

template <bool UP>
cudaError_t launch_product(const W4Args &a, int64_t G, int64_t units, cudaStream_t s) {
    if (G == 32) return launch_product_of<UP, 32>(a, units, s);
    if (G == 64) return launch_product_of<UP, 64>(a, units, s);
    return launch_product_of<UP, 128>(a, units, s);
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
    W4Args a{};
    a.x = static_cast<const uint16_t *>(x_dev);
    a.ids = topk_ids_dev;
    a.weights = topk_weights_dev;
    a.w1 = w1_prepared_dev;
    a.w2 = w2_prepared_dev;
    a.s1 = static_cast<const uint8_t *>(w1_scales_prepared_dev);
    a.s2 = static_cast<const uint8_t *>(w2_scales_prepared_dev);
    a.out = static_cast<uint16_t *>(out_dev);
    a.xq = reinterpret_cast<W4Inputs *>(ws + p.x);
    a.act = reinterpret_cast<W4Inputs *>(ws + p.act);
    a.y = reinterpret_cast<float *>(ws + p.y);
    a.status = status_dev;
    a.entries_used = reinterpret_cast<int32_t *>(ws + p.head);
    a.picks = reinterpret_cast<int32_t *>(ws + p.picks);
    a.places = a.picks + p.P;
    a.entries = reinterpret_cast<W4Entry *>(ws + p.entries);
    a.T = (int)p.T; a.H = (int)p.H; a.E = (int)p.E; a.k = (int)p.k; a.I = (int)p.I; a.P = (int)p.P;
    a.ids64 = ids_dtype == MOE_IDS_INT64;
    a.placed = p.P > kW4FewPicks;
    cudaError_t e = launch_pdl(w4_group_kernel, dim3((unsigned)(1 + (a.placed ? 0 : p.P))), dim3(1024), 0, s, a);
    if (e == cudaSuccess && a.placed) e = launch_pdl(w4_inputs_kernel, dim3((unsigned)p.P), dim3(1024), 0, s, a);
    if (e == cudaSuccess && p.T > 0) {
        const int64_t entries = (p.P < p.E ? p.P : p.E) + p.P / kW4Picks;   // at most
        e = launch_product<true>(a, p.G, entries * (p.I / 8 / kW4Tiles), s);
        if (e == cudaSuccess) e = launch_product<false>(a, p.G, entries * (p.H / 16 / kW4Tiles), s);
        if (e == cudaSuccess)
            e = launch_pdl(w4_combine_kernel, dim3((unsigned)p.T, (unsigned)((p.H + 1023) / 1024)), dim3(128), 0, s, a);
    }
    return status_of(e);
}

}  // extern "C"
