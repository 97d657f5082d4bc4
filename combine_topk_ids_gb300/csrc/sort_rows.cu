// A batch's picks in expert order (moe_sort_picks), its rows gathered into that order and summed
// back (moe_sort_rows, moe_unsort_rows), and their gradients; declared in include/moe_grouped.h.
//
// Picks (t, j) are ordered by (expert, t, j).  A pick's row is
//     the picks of smaller experts + the earlier picks of its own expert,
// both counts, so no atomic decides a position.
//
// The rows' kernels read and write each row once; HBM bounds them where rows are on 16-byte boundaries
// (measured, of the copy rate: 32768 tokens of 7168 columns, top-8, in order with the order itself, bf16
// 641 us, 0.98, e4m3 340 us, 0.95; back 587 us; the gradient of 8192 of them 311 us, 0.95).
#include "../../include/moe_grouped.h"
#include "block_common.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------------------ order of picks

struct SortArgs {
    const void *ids;
    int ids64, E, nb;
    int64_t P, chunk;         // picks, and picks of a block (a multiple of 32 for each warp)
    int32_t *offsets, *position, *source, *status;
    int32_t *hist;            // [nb][E] picks of each block and expert, then [nb] bad ids
};

constexpr int kHeld = 4;                    // picks of a lane that stay in registers
constexpr int kLeastRun = 64;              // picks of a warp, before there is another warp's counts to add
constexpr int kMaxSortBlocks = 152;
constexpr int kMaxSortCounts = 152 * 256;   // nb * E: every block reads all of them

// Most warps of a block of sort_assign_kernel, and the most that its table of a row for each (and two more) takes.
constexpr int sort_warps(int E) { return E <= 1024 ? 32 : 16; }
constexpr int kMostTable = (2 + sort_warps(MOE_MAX_EXPERTS)) * MOE_MAX_EXPERTS * 4;
static_assert(kMostTable >= (2 + sort_warps(1024)) * 1024 * 4, "the most experts take the largest table");

// Expert of pick i, -1 where it is masked or dropped.
__device__ __forceinline__ int expert_of(const SortArgs &a, int64_t i, bool &bad) {
    const long long v = a.ids64 ? static_cast<const long long *>(a.ids)[i] : static_cast<const int *>(a.ids)[i];
    if (v >= 0 && v < a.E) return (int)v;
    bad |= v != -1;
    return -1;
}

__global__ void __launch_bounds__(512) sort_count_kernel(SortArgs a) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t p0 = a.chunk * blockIdx.x, p1 = min(p0 + a.chunk, a.P);
    bool bad = false;
#pragma unroll 4
    for (int64_t i = p0 + threadIdx.x; i < p1; i += blockDim.x) {
        const int e = expert_of(a, i, bad);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    bad = __syncthreads_or(bad);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * a.E + e] = hist[e];
    if (threadIdx.x == 0) a.hist[(int64_t)a.nb * a.E + blockIdx.x] = bad;
}

// Up to 1024 picks one block does it all.  Above, blocks of up to 512 picks (more where that would take over
// 152 blocks, or counts over kMaxSortCounts) count theirs first, and then each reads the counts of all.
// Measured with 256 experts, us: 512 picks 3.7, 1024 6.2 (in two kernels 6.6), 2048 6.5 (one block 8.6),
// 4096 7.0 (13), 32768 7.7, 262144 13.6.
//
// Each warp owns a contiguous run of the block's picks: it counts the run by expert, the counts
// become the first position of its run in each expert, and then it ranks the run 32 at a time.
__global__ void __launch_bounds__(1024) sort_assign_kernel(SortArgs a) {
    extern __shared__ int sm[];
    __shared__ int wsum[32];
    const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t p0 = min(a.chunk * blockIdx.x, a.P), p1 = min(p0 + a.chunk, a.P);
    int64_t run = ((p1 - p0 + warps - 1) / warps + 31) / 32 * 32;
    if (run < kLeastRun) run = kLeastRun;
    const int used = run ? (int)((p1 - p0 + run - 1) / run) : 0;   // warps with a run
    const int64_t w0 = min(p0 + warp * run, p1), w1 = min(w0 + run, p1);
    int *total = sm, *before = sm + E, *cur = sm + 2 * E;          // cur [used][E]
    for (int i = threadIdx.x; i < (2 + used) * E; i += blockDim.x) sm[i] = 0;
    pdl_wait();   // (for the counts, and for the ids)
    __syncthreads();
    bool bad = false;
    // the experts of a run of up to 128 picks stay in registers
    const bool held = run <= 32 * kHeld;
    int mine[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        const int64_t i = w0 + 32 * h + lane;
        mine[h] = held && i < w1 ? expert_of(a, i, bad) : -1;
    }
    auto each = [&](auto &&f) {   // f(pick, its expert or -1), 32 at a time
        if (held) {
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (w0 + 32 * h < w1) f(w0 + 32 * h + lane, mine[h]);
        } else
            for (int64_t i0 = w0; i0 < w1; i0 += 32)
                f(i0 + lane, i0 + lane < w1 ? expert_of(a, i0 + lane, bad) : -1);
    };
    each([&](int64_t, int e) {
        const unsigned peers = __match_any_sync(kAllLanes, e);
        if (e >= 0 && lane == __ffs(peers) - 1) cur[warp * E + e] += __popc(peers);
        __syncwarp();
    });
    if (a.nb > 1) {   // counts of all blocks, and of those before this one
        const int wide = (E + 31) / 32 * 32, slices = max(1, (int)blockDim.x / wide);
        for (int i = threadIdx.x; i < slices * wide; i += blockDim.x) {
            const int e = i % wide;
            if (e >= E) continue;
            int all = 0, first = 0;
#pragma unroll 8
            for (int b = i / wide; b < a.nb; b += slices) {
                const int n = a.hist[(int64_t)b * E + e];
                all += n;
                first += b < (int)blockIdx.x ? n : 0;
            }
            atomicAdd(&total[e], all);   // (integers: any order gives the same)
            atomicAdd(&before[e], first);
        }
        bad = false;
        if (blockIdx.x == 0)
            for (int b = threadIdx.x; b < a.nb; b += blockDim.x) bad |= a.hist[(int64_t)a.nb * E + b] != 0;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) *a.status = bad ? MOE_STATUS_BAD_EXPERT_ID : 0;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int n = 0;
        if (e < E) {
            if (a.nb > 1) n = total[e];
            else
#pragma unroll 8
                for (int w = 0; w < used; ++w) n += cur[w * E + e];
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAllLanes, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int ahead = carry, block_sum = 0;
        for (int w = 0; w < warps; ++w) {
            ahead += w < warp ? wsum[w] : 0;
            block_sum += wsum[w];
        }
        if (e < E) {
            const int first = ahead + incl - n;
            if (blockIdx.x == 0) a.offsets[e] = first;
            int at = first + before[e];
            for (int w = 0; w < used; w += 8) {   // (eight at a time: their loads do not wait for the stores)
                int c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = w + i < used ? cur[(w + i) * E + e] : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (w + i < used) cur[(w + i) * E + e] = at;
                    at += c[i];
                }
            }
        }
        carry += block_sum;
        __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = carry;
    const unsigned below = (1u << lane) - 1u;
    each([&](int64_t i, int e) {
        const unsigned peers = __match_any_sync(kAllLanes, e);
        const int at = e >= 0 ? cur[warp * E + e] + __popc(peers & below) : -1;
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) cur[warp * E + e] += __popc(peers);
        __syncwarp();
        if (i < w1) {
            a.position[i] = at;
            if (a.source) {
                if (at >= 0) a.source[at] = (int)i;
                if (i >= carry) a.source[i] = -1;   // behind the last row
            }
        }
    });
}

int sort_blocks(const moe_sort &g) {
    const int64_t P = (int64_t)g.num_tokens * g.top_k;
    if (P <= 1024) return 1;
    int64_t nb = (P + 511) / 512;
    if (nb > kMaxSortBlocks) nb = kMaxSortBlocks;
    if (nb * g.num_experts > kMaxSortCounts) nb = kMaxSortCounts / g.num_experts;
    return (int)nb;
}

int check_sort(const moe_sort *g) {
    if (!g || g->num_tokens < 0 || g->num_experts < 1) return MOE_ERR_INVALID_ARGUMENT;
    if (g->top_k < 1 || g->top_k > MOE_MAX_TOPK) return MOE_ERR_TOPK;
    if (g->num_experts > MOE_MAX_EXPERTS || (int64_t)g->num_tokens * g->top_k > ((int64_t)1 << 31) - 1024)
        return MOE_ERR_LIMIT;
    return MOE_OK;
}

size_t sort_bytes(const moe_sort &g) { return ((size_t)sort_blocks(g) * (g.num_experts + 1) * 4 + 15) / 16 * 16; }

// ------------------------------------------------------------------------------------- rows

// N elements of a row as floats; N > 1: at an address that is a multiple of their size together.
template <typename T, int N> struct Pack;
template <int N> struct Pack<float, N> {
    float v[N];
    __device__ __forceinline__ void load(const float *p) {
        if constexpr (N == 4) {
            const float4 r = *reinterpret_cast<const float4 *>(p);
            v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
        } else v[0] = *p;
    }
    __device__ __forceinline__ float at(int i) const { return v[i]; }
    __device__ __forceinline__ static void store(float *p, const float (&f)[N]) {
        if constexpr (N == 4) *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        else *p = f[0];
    }
};
template <int N> struct Pack<__nv_bfloat16, N> {
    static constexpr int kWords = N > 1 ? N / 2 : 1;
    uint32_t v[kWords];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        if constexpr (N == 8) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p);
            v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
        } else if constexpr (N == 4) {
            const uint2 r = *reinterpret_cast<const uint2 *>(p);
            v[0] = r.x; v[1] = r.y;
        } else v[0] = *reinterpret_cast<const uint16_t *>(p);
    }
    __device__ __forceinline__ float at(int i) const { return i & 1 ? hi_f32(v[i / 2]) : lo_f32(v[i / 2]); }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, const float (&f)[N]) {
        if constexpr (N == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                       pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        else if constexpr (N == 4)
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
        else *p = __float2bfloat16_rn(f[0]);
    }
};

struct CopyArgs {
    const char *x;
    char *rows;
    const float *xs;
    float *rs;
    const int32_t *position;
    int64_t xstride, rstride;   // bytes
    int T, k, num_rows;
    int words;                  // accesses of a row (of the kernel's word)
    int scales;                 // scales of a row
    int nchunk, nchunk_all;     // pieces of a row, and with its scales
};

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
template <typename W> constexpr int kCopyWords = sizeof(W) == 16 ? 4 : 8;   // accesses of a lane in a piece

// A warp copies one piece of a token's row (or of its scales) to the rows of its picks: the row is read
// once, and a lane's four stores of a pick do not wait for one another.
template <typename W>
__device__ __forceinline__ void copy_piece(const CopyArgs &a, const W *src, char *dst, int64_t stride, int words,
                                           int piece, int64_t t) {
    constexpr int U = kCopyWords<W>;
    const int lane = threadIdx.x & 31, c0 = piece * 32 * U + lane;
    const int32_t *pos = a.position + t * a.k;
    const int mine = lane < a.k ? pos[lane] : -1;
    W v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (c0 + 32 * u < words) v[u] = src[c0 + 32 * u];
    for (int j = 0; j < a.k; ++j) {
        const int p = __shfl_sync(kAllLanes, mine, j);
        if (p < 0 || p >= a.num_rows) continue;
        W *d = reinterpret_cast<W *>(dst + p * stride);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < words) d[c0 + 32 * u] = v[u];
    }
}

template <typename W>
__global__ void __launch_bounds__(kRowThreads) sort_rows_kernel(CopyArgs a) {
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    const int64_t t = i / a.nchunk_all;
    const int piece = (int)(i - t * a.nchunk_all);
    if (t >= a.T) return;
    if (piece < a.nchunk)
        copy_piece(a, reinterpret_cast<const W *>(a.x + t * a.xstride), a.rows, a.rstride, a.words, piece, t);
    else
        copy_piece(a, a.xs + t * a.scales, reinterpret_cast<char *>(a.rs), (int64_t)a.scales * 4, a.scales,
                   piece - a.nchunk, t);
}

// Rows of up to 16 words: LANES lanes to a token (and its scales, at most as many).  A warp to a piece
// would leave most lanes without work, and its picks' stores would follow one another.
template <typename W, int LANES>
__global__ void __launch_bounds__(kRowThreads) sort_short_rows_kernel(CopyArgs a) {
    pdl_wait();
    const int64_t t = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) / LANES;
    const int lane = threadIdx.x % LANES;
    if (t >= a.T) return;
    const bool word = lane < a.words, scale = lane < a.scales;
    W v;
    float s;
    if (word) v = reinterpret_cast<const W *>(a.x + t * a.xstride)[lane];
    if (scale) s = a.xs[t * a.scales + lane];
    const int32_t *pos = a.position + t * a.k;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
        const int p = pos[j];
        if (p < 0 || p >= a.num_rows) continue;
        if (word) reinterpret_cast<W *>(a.rows + p * a.rstride)[lane] = v;
        if (scale) a.rs[(int64_t)p * a.scales + lane] = s;
    }
}

struct SumArgs {
    const void *rows;
    const float *w;             // NULL: 1
    const int32_t *position;
    void *out;
    int64_t rstride, ostride;   // elements
    int T, k, H, num_rows, nchunk;
};

constexpr int kSumPicks = 4;    // picks whose loads are under way together

template <int N> constexpr int kSumUnits = N == 1 ? 8 : 2;

// A warp sums one piece of a token's row over its picks, in their order.  Rows off 16-byte boundaries go
// column by column, eight of a lane under way for each of four picks (16381 x 2047 bf16, top-4, 76 us,
// 0.66 of the copy rate; four columns 85).  Pairs of bf16 were slower: 142 us as words or halves by
// address, 105 as aligned words and a shuffle.
template <typename R, typename O, int N>
__global__ void __launch_bounds__(kRowThreads) unsort_rows_kernel(SumArgs a) {
    constexpr int U = kSumUnits<N>;
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = i / a.nchunk;
    if (t >= a.T) return;
    const int c0 = ((int)(i - t * a.nchunk) * 32 * U + lane) * N;   // column of this lane's first element
    int pos = -1;
    float wt = 1.f;
    if (lane < a.k) {
        pos = a.position[t * a.k + lane];
        if (pos >= a.num_rows) pos = -1;
        if (a.w) wt = a.w[t * a.k + lane];
    }
    const R *rows = static_cast<const R *>(a.rows);
    float acc[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < N; ++n) acc[u][n] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += kSumPicks) {
        Pack<R, N> v[kSumPicks][U];
#pragma unroll
        for (int q = 0; q < kSumPicks; ++q) {
            const int p = __shfl_sync(kAllLanes, pos, (j0 + q) & 31);
            if (j0 + q < a.k && p >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + 32 * N * u < a.H) v[q][u].load(rows + p * a.rstride + c0 + 32 * N * u);
        }
#pragma unroll
        for (int q = 0; q < kSumPicks; ++q) {
            const int p = __shfl_sync(kAllLanes, pos, (j0 + q) & 31);
            const float w = __shfl_sync(kAllLanes, wt, (j0 + q) & 31);
            if (j0 + q < a.k && p >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + 32 * N * u < a.H)
#pragma unroll
                        for (int n = 0; n < N; ++n) acc[u][n] = fmaf(w, v[q][u].at(n), acc[u][n]);
        }
    }
    O *out = static_cast<O *>(a.out) + t * a.ostride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + 32 * N * u;
        if (c < a.H) Pack<O, N>::store(out + c, acc[u]);
    }
}

struct BackArgs {
    const void *dout, *rows;    // rows is NULL without dw
    const float *w;             // NULL: 1
    const int32_t *position;
    void *drows;                // NULL: not written
    float *dw;                  // NULL: not written
    int64_t ostride, rstride, dstride;
    int T, k, H, num_rows;
};

template <int N> constexpr int kBackUnits = N == 1 ? 8 : 1;   // accesses of a thread and row under way

// blockDim.x threads to a token, blockDim.y tokens to a block; P picks share a reading of dout.  A warp to
// a token where there are tokens enough: 16381 x 2048 bf16, top-4, 86 us (0.95 of the copy rate; a block to
// a token 168).  Rows off 16-byte boundaries column by column, eight of a lane under way for each pick, at
// fixed distances from one address (x 2047 118 us, 0.69: latency, with the schedulers issuing in 42% of
// the cycles and DRAM at 57%; at distances that hang on the block's size 160, one column 186).
template <typename R, typename O, int N, int P>
__global__ void __launch_bounds__(256, N == 1 ? 3 : 0) unsort_rows_backward_kernel(BackArgs a) {
    constexpr int U = kBackUnits<N>;
    __shared__ float red[8][P];
    pdl_wait();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < a.T;
    const O *dout = static_cast<const O *>(a.dout) + t * a.ostride;
    const R *rows = static_cast<const R *>(a.rows);
    R *drows = static_cast<R *>(a.drows);
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    const int warp = threadIdx.y * nw + (threadIdx.x >> 5);
    for (int j0 = 0; j0 < a.k; j0 += P) {
        int p[P];
        float w[P], dot[P];
#pragma unroll
        for (int q = 0; q < P; ++q) {
            p[q] = live && j0 + q < a.k ? a.position[t * a.k + j0 + q] : -1;
            if (p[q] >= a.num_rows) p[q] = -1;
            w[q] = p[q] >= 0 && a.w ? a.w[t * a.k + j0 + q] : 1.f;
            dot[q] = 0.f;
        }
        for (int c0 = ((threadIdx.x >> 5) * 32 * U + lane) * N; live && c0 < a.H; c0 += blockDim.x * N * U) {
            Pack<O, N> d[U];
            Pack<R, N> v[P][U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + 32 * N * u;
                if (c < a.H) d[u].load(dout + c);
            }
            if (a.dw) {
#pragma unroll
                for (int q = 0; q < P; ++q)
                    if (p[q] >= 0)
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int c = c0 + 32 * N * u;
                            if (c < a.H) v[q][u].load(rows + p[q] * a.rstride + c);
                        }
            }
            if (a.drows) {
#pragma unroll
                for (int q = 0; q < P; ++q)
                    if (p[q] >= 0)
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int c = c0 + 32 * N * u;
                            float g[N];
#pragma unroll
                            for (int n = 0; n < N; ++n) g[n] = w[q] * d[u].at(n);
                            if (c < a.H) Pack<R, N>::store(drows + p[q] * a.dstride + c, g);
                        }
            }
            if (a.dw) {
#pragma unroll
                for (int q = 0; q < P; ++q)
                    if (p[q] >= 0)
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (c0 + 32 * N * u < a.H)
#pragma unroll
                                for (int n = 0; n < N; ++n) dot[q] = fmaf(d[u].at(n), v[q][u].at(n), dot[q]);
            }
        }
        if (!a.dw) continue;
#pragma unroll
        for (int q = 0; q < P; ++q) dot[q] = warp_sum(dot[q]);
        if (nw == 1) {
#pragma unroll
            for (int q = 0; q < P; ++q)
                if (live && lane == q && j0 + q < a.k) a.dw[t * a.k + j0 + q] = dot[q];
            continue;
        }
        if (lane == 0)
#pragma unroll
            for (int q = 0; q < P; ++q) red[warp][q] = dot[q];
        __syncthreads();
        if (live && (int)threadIdx.x < P && j0 + (int)threadIdx.x < a.k) {
            float s = 0.f;
            for (int i = 0; i < nw; ++i) s += red[threadIdx.y * nw + i][threadIdx.x];
            a.dw[t * a.k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------ host

int64_t packed(int64_t stride, int64_t width) { return stride ? stride : width; }

int check_rows(const moe_rows *g) {
    if (!g || g->num_tokens < 0 || g->num_rows < 0 || g->hidden < 1) return MOE_ERR_INVALID_ARGUMENT;
    if (g->top_k < 1 || g->top_k > MOE_MAX_TOPK) return MOE_ERR_TOPK;
    if (g->hidden > MOE_MAX_HIDDEN) return MOE_ERR_LIMIT;
    for (int64_t s : {g->rows_stride, g->drows_stride, g->tokens_stride})
        if (s && s < g->hidden) return MOE_ERR_INVALID_ARGUMENT;
    return MOE_OK;
}

// Whether every row starts at a multiple of `bytes`.
bool rows_on(const void *p, int64_t stride, int64_t elem, size_t bytes) {
    return !p || (is_aligned(p, bytes) && stride * elem % (int64_t)bytes == 0);
}

int64_t blocks_of(int64_t warps) { return (warps + kRowWarps - 1) / kRowWarps; }

// f(R, O, N): the element types of the sorted rows and of the tokens' rows, and the elements of
// one access: 16 bytes of the wider type where every row and its length allow it, else one.
template <typename F>
int with_row_types(int32_t rows_dtype, int32_t tokens_dtype, bool even, F &&f) {
    using B = __nv_bfloat16;
    constexpr auto one = std::integral_constant<int, 1>{};
    constexpr auto four = std::integral_constant<int, 4>{};
    constexpr auto eight = std::integral_constant<int, 8>{};
    const bool r32 = rows_dtype == MOE_DTYPE_FP32, o32 = tokens_dtype == MOE_DTYPE_FP32;
    if (!r32 && !o32) return even ? f(B{}, B{}, eight) : f(B{}, B{}, one);
    if (!r32) return even ? f(B{}, float{}, four) : f(B{}, float{}, one);
    if (!o32) return even ? f(float{}, B{}, four) : f(float{}, B{}, one);
    return even ? f(float{}, float{}, four) : f(float{}, float{}, one);
}

int launch_unsort(const moe_rows *g, const void *rows, const float *weights, const int32_t *position, void *out,
                  int32_t tokens_dtype, cudaStream_t s) {
    const int64_t rb = dtype_bytes(g->rows_dtype), ob = dtype_bytes(tokens_dtype);
    SumArgs a{rows, weights, position, out, packed(g->rows_stride, g->hidden), packed(g->tokens_stride, g->hidden),
              g->num_tokens, g->top_k, g->hidden, g->num_rows, 0};
    const int n = rb == 2 && ob == 2 ? 8 : 4;
    const bool even = g->hidden % n == 0 && rows_on(rows, a.rstride, rb, n * rb) && rows_on(out, a.ostride, ob, n * ob);
    return with_row_types(g->rows_dtype, tokens_dtype, even, [&](auto r, auto o, auto width) {
        constexpr int N = decltype(width)::value;
        constexpr int piece = 32 * N * kSumUnits<N>;
        a.nchunk = (a.H + piece - 1) / piece;
        const int64_t blocks = blocks_of((int64_t)a.T * a.nchunk);
        if (blocks >= ((int64_t)1 << 31)) return (int)MOE_ERR_LIMIT;
        return status_of(launch_pdl(unsort_rows_kernel<decltype(r), decltype(o), N>, dim3((unsigned)blocks),
                                    dim3(kRowThreads), 0, s, a));
    });
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_sort_picks_workspace_size(const moe_sort *g, size_t *bytes) {
    const int rc = check_sort(g);
    if (rc != MOE_OK) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
    *bytes = sort_bytes(*g);
    return MOE_OK;
}

extern "C" int moe_sort_picks(const moe_sort *g, const void *topk_ids_dev, int ids_dtype, int32_t *offsets_dev,
                              int32_t *position_dev, int32_t *source_dev, int32_t *status_dev, void *workspace_dev,
                              size_t workspace_bytes, void *stream) {
    int rc = check_sort(g);
    if (rc != MOE_OK) return rc;
    if (ids_dtype != MOE_IDS_INT32 && ids_dtype != MOE_IDS_INT64) return MOE_ERR_IDS_DTYPE;
    if (!offsets_dev || !workspace_dev || (g->num_tokens > 0 && (!topk_ids_dev || !position_dev)))
        return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(topk_ids_dev, ids_dtype == MOE_IDS_INT64 ? 8 : 4) || !is_aligned(offsets_dev, 4) ||
        !is_aligned(position_dev, 4) || !is_aligned(source_dev, 4) || !is_aligned(status_dev, 4) ||
        !is_aligned(workspace_dev, 16))
        return MOE_ERR_MISALIGNED;
    if (workspace_bytes < sort_bytes(*g)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if ((rc = check_device()) != MOE_OK) return rc;
    SortArgs a{};
    a.ids = topk_ids_dev;
    a.ids64 = ids_dtype == MOE_IDS_INT64;
    a.E = g->num_experts;
    a.P = (int64_t)g->num_tokens * g->top_k;
    a.nb = sort_blocks(*g);
    a.chunk = ((a.P + a.nb - 1) / a.nb + 31) / 32 * 32;
    a.offsets = offsets_dev; a.position = position_dev; a.source = source_dev; a.status = status_dev;
    a.hist = static_cast<int32_t *>(workspace_dev);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    static PerDevice devices;
    cudaError_t e = devices.set(sort_assign_kernel, kMostTable, [](int) { return cudaSuccess; });
    if (e != cudaSuccess) return status_of(e);
    if (a.nb > 1 &&
        (e = launch_pdl(sort_count_kernel, dim3(a.nb), dim3(512), (size_t)a.E * 4, s, a)) != cudaSuccess)
        return status_of(e);
    // one table row for each warp with picks.  All warps read the blocks' counts.
    const int warps = sort_warps(a.E);
    const int64_t need = (a.chunk + kLeastRun - 1) / kLeastRun;
    const int rows = need < warps ? (int)need : warps, threads = a.nb > 1 || rows > 8 ? 32 * warps : 256;
    const size_t smem = (size_t)(2 + rows) * a.E * 4;
    return status_of(launch_pdl(sort_assign_kernel, dim3(a.nb), dim3(threads), smem, s, a));
}

extern "C" int moe_sort_rows(const moe_rows *g, const void *x_dev, const float *x_scales_dev,
                             const int32_t *position_dev, void *rows_dev, float *rows_scales_dev, void *stream) {
    int rc = check_rows(g);
    if (rc != MOE_OK) return rc;
    const bool codes = g->rows_dtype == MOE_DTYPE_E4M3;
    if (!codes && bad_dtype(g->rows_dtype)) return MOE_ERR_INVALID_ARGUMENT;
    const bool none = g->num_tokens == 0 || g->num_rows == 0;   // (an empty matrix has no address)
    if (codes ? !none && (!x_scales_dev || !rows_scales_dev) : x_scales_dev || rows_scales_dev)
        return MOE_ERR_INVALID_ARGUMENT;
    if (codes && g->hidden % 128) return MOE_ERR_HIDDEN_ALIGNMENT;
    const int64_t b = codes ? 1 : (int64_t)dtype_bytes(g->rows_dtype);
    CopyArgs a{};
    a.xstride = packed(g->tokens_stride, g->hidden) * b;
    a.rstride = packed(g->rows_stride, g->hidden) * b;
    if (codes && (a.xstride != g->hidden || a.rstride != g->hidden)) return MOE_ERR_INVALID_ARGUMENT;
    if (!none && (!x_dev || !position_dev || !rows_dev)) return MOE_ERR_INVALID_ARGUMENT;
    const size_t unit = codes ? 16 : (size_t)b;
    if (!is_aligned(x_dev, unit) || !is_aligned(rows_dev, unit) || !is_aligned(x_scales_dev, 4) ||
        !is_aligned(rows_scales_dev, 4) || !is_aligned(position_dev, 4))
        return MOE_ERR_MISALIGNED;
    if ((rc = check_device()) != MOE_OK) return rc;
    if (none) return MOE_OK;
    a.x = static_cast<const char *>(x_dev);
    a.rows = static_cast<char *>(rows_dev);
    a.xs = x_scales_dev; a.rs = rows_scales_dev;
    a.position = position_dev;
    a.T = g->num_tokens; a.k = g->top_k; a.num_rows = g->num_rows;
    a.scales = codes ? g->hidden / 128 : 0;
    const bool even = g->hidden * b % 16 == 0 && rows_on(x_dev, a.xstride, 1, 16) && rows_on(rows_dev, a.rstride, 1, 16);
    const int64_t word = even ? 16 : b;
    a.words = (int)(g->hidden * b / word);
    const int piece = 32 * (word == 16 ? kCopyWords<uint4> : kCopyWords<uint32_t>);
    a.nchunk = (a.words + piece - 1) / piece;
    a.nchunk_all = a.nchunk + (a.scales + 32 * kCopyWords<float> - 1) / (32 * kCopyWords<float>);
    const bool brief = a.words <= 16;
    const int lanes = a.words <= 4 ? 4 : a.words <= 8 ? 8 : 16;
    const int64_t blocks = brief ? ((int64_t)a.T * lanes + kRowThreads - 1) / kRowThreads
                                 : blocks_of((int64_t)a.T * a.nchunk_all);
    if (blocks >= ((int64_t)1 << 31)) return MOE_ERR_LIMIT;
    auto launch = [&](auto w) {
        using W = decltype(w);
        if (brief) {
            auto *kernel = lanes == 4 ? sort_short_rows_kernel<W, 4> : lanes == 8 ? sort_short_rows_kernel<W, 8>
                                                                                 : sort_short_rows_kernel<W, 16>;
            return status_of(launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRowThreads), 0,
                                        static_cast<cudaStream_t>(stream), a));
        }
        return status_of(launch_pdl(sort_rows_kernel<decltype(w)>, dim3((unsigned)blocks), dim3(kRowThreads), 0,
                                    static_cast<cudaStream_t>(stream), a));
    };
    return word == 16 ? launch(uint4{}) : word == 4 ? launch(uint32_t{}) : launch(uint16_t{});
}

extern "C" int moe_unsort_rows(const moe_rows *g, const void *rows_dev, const float *weights_dev,
                               const int32_t *position_dev, void *out_dev, void *stream) {
    int rc = check_rows(g);
    if (rc != MOE_OK) return rc;
    if (bad_dtype(g->rows_dtype) || bad_dtype(g->tokens_dtype)) return MOE_ERR_INVALID_ARGUMENT;
    if (g->num_tokens > 0 && ((!rows_dev && g->num_rows > 0) || !position_dev || !out_dev))
        return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(rows_dev, dtype_bytes(g->rows_dtype)) || !is_aligned(out_dev, dtype_bytes(g->tokens_dtype)) ||
        !is_aligned(weights_dev, 4) || !is_aligned(position_dev, 4))
        return MOE_ERR_MISALIGNED;
    if ((rc = check_device()) != MOE_OK) return rc;
    if (g->num_tokens == 0) return MOE_OK;
    return launch_unsort(g, rows_dev, weights_dev, position_dev, out_dev, g->tokens_dtype,
                         static_cast<cudaStream_t>(stream));
}

extern "C" int moe_sort_rows_backward(const moe_rows *g, const void *drows_dev, const int32_t *position_dev,
                                      void *dx_dev, void *stream) {
    if (!g) return MOE_ERR_INVALID_ARGUMENT;
    moe_rows like = *g;
    like.tokens_dtype = g->rows_dtype;
    return moe_unsort_rows(&like, drows_dev, nullptr, position_dev, dx_dev, stream);
}

extern "C" int moe_unsort_rows_backward(const moe_rows *g, const void *dout_dev, const void *rows_dev,
                                        const float *weights_dev, const int32_t *position_dev, void *drows_dev,
                                        float *dweights_dev, void *stream) {
    int rc = check_rows(g);
    if (rc != MOE_OK) return rc;
    if (bad_dtype(g->rows_dtype) || bad_dtype(g->tokens_dtype) || (g->num_rows > 0 && !drows_dev && !dweights_dev))
        return MOE_ERR_INVALID_ARGUMENT;
    if (g->num_tokens > 0 && (!dout_dev || !position_dev || (dweights_dev && g->num_rows > 0 && !rows_dev)))
        return MOE_ERR_INVALID_ARGUMENT;
    const int64_t rb = dtype_bytes(g->rows_dtype), ob = dtype_bytes(g->tokens_dtype);
    if (!is_aligned(dout_dev, ob) || !is_aligned(rows_dev, rb) || !is_aligned(drows_dev, rb) ||
        !is_aligned(weights_dev, 4) || !is_aligned(dweights_dev, 4) || !is_aligned(position_dev, 4))
        return MOE_ERR_MISALIGNED;
    if ((rc = check_device()) != MOE_OK) return rc;
    if (g->num_tokens == 0 || (!drows_dev && !dweights_dev)) return MOE_OK;
    BackArgs a{dout_dev, rows_dev, weights_dev, position_dev, drows_dev, dweights_dev,
               packed(g->tokens_stride, g->hidden), packed(g->rows_stride, g->hidden),
               packed(g->drows_stride, g->hidden), g->num_tokens, g->top_k, g->hidden, g->num_rows};
    const int n = rb == 2 && ob == 2 ? 8 : 4;
    const bool even = g->hidden % n == 0 && rows_on(dout_dev, a.ostride, ob, n * ob) &&
                      rows_on(dweights_dev ? rows_dev : nullptr, a.rstride, rb, n * rb) &&
                      rows_on(drows_dev, a.dstride, rb, n * rb);
    return with_row_types(g->rows_dtype, g->tokens_dtype, even, [&](auto r, auto o, auto width) {
        constexpr int N = decltype(width)::value;
        // Threads for a token: all its accesses at once, up to a block, as long as the tokens alone are
        // too few warps for the SMs; a warp to a token meets no barrier.
        const int64_t turn = (int64_t)N * kBackUnits<N> * 32, most = ((int64_t)a.H + turn - 1) / turn;
        const int64_t wanted = ((int64_t)num_sms() * 24 + a.T - 1) / a.T;
        int warps = 1;
        while (warps < 8 && warps < most && warps < wanted) warps *= 2;
        const int tokens = 8 / warps;
        const int64_t blocks = ((int64_t)a.T + tokens - 1) / tokens;
        auto launch = [&](auto *kernel) {
            return status_of(launch_pdl(kernel, dim3((unsigned)blocks), dim3(32 * warps, tokens), 0,
                                        static_cast<cudaStream_t>(stream), a));
        };
        using R = decltype(r);
        using O = decltype(o);
        // single columns four picks at a time for any k: eight picks leave registers for four columns only
        // (8192 x 2047, top-8, 165 us; as here 132)
        if constexpr (N == 1) return launch(unsort_rows_backward_kernel<R, O, N, 4>);
        else return a.k <= 4 ? launch(unsort_rows_backward_kernel<R, O, N, 4>) : launch(unsort_rows_backward_kernel<R, O, N, 8>);
    });
}
