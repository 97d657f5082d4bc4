// The gradient of the residual addition and RMS norm (moe_add_rmsnorm_backward; declared in
// include/moe_block.h).
//
// With g = dout * w and xhat = h * rstd, one row:
//     dx = rstd * (g - xhat * mean(g * xhat)) + dsum;     dw += dout * xhat
// dout, h and dsum are read once, dx is written once; the columns' sums stay in registers over a
// block's rows and are added up by a second kernel in a fixed order.  HBM bounds it, if enough
// rows are under way: measured on 8192 rows of 4096 columns (268 MB) 45 us, 5.9 TB/s, 0.89 of the
// measured peak (5 us of it the second kernel), with two rows ahead in shared memory; 51 us with
// one ahead in registers, 59 us with that one's loads issued after the barrier.  Rows of 5120 67 us
// (0.75: 122 to 128 registers leave one block of more than 256 threads on an SM), of 7168 82 us
// (0.86), of 8192 88 us (0.91).  A float32 stream, with one row ahead, 101 us at 4096 columns (0.70).
// Above 16384 columns (float32: 8192) a thread's columns do not fit its registers, and local memory
// sets the time: 1000 rows of 20000 257 us (0.09), 2000 of 12000 in float32 167 us (0.30).
#include <type_traits>

#include "norm.cuh"

namespace moe {
namespace {

constexpr int kMaxParts = 304;   // row blocks that write a partial dweight (two per SM; a multiple of 8, for ODD)

struct NormBackArgs {
    const void *dout, *h, *w, *dsum;
    void *dx;
    const float *rstd;
    float *part;              // [gridDim.x][H]
    int64_t ds, hs, ss, os;   // row strides in elements
    int T, H;
    int shift;                // ODD: chunks follow the 16-byte boundaries of dout's rows
};

// How columns [i, i + 8) of a row lie: not in the row at all, all of them and on a 16-byte
// boundary, some of them and on one, or off the boundaries (then they are taken one by one).
// Rows 8 apart lie alike, whatever their stride.
enum Lie { kAbsent, kWhole, kPartial, kOff };
__device__ __forceinline__ int lie_of(const void *row, int i, int H, int size) {
    if (i >= H || i <= -8) return kAbsent;
    if (((reinterpret_cast<uintptr_t>(row) + (int64_t)i * size) & 15) != 0) return kOff;
    return i >= 0 && i + 8 <= H ? kWhole : kPartial;
}

// A row matrix's first byte and the one after its last: 16 bytes that begin in one row and end in
// the next may be read together.
struct Room {
    const char *begin, *end;
};
__device__ __forceinline__ Room room_of(const void *p, int64_t rows, int64_t stride, int H, int size) {
    const char *c = static_cast<const char *>(p);
    return Room{c, c + ((rows - 1) * stride + H) * size};
}

// Columns [i, i + 8) of a row that may lie in any way.  load() issues 16-byte loads, so that a
// thread's loads are under way together; what cannot be loaded so (rows that lie otherwise than
// the chunks, the matrix's own ends) it fetches column by column.  floats() gives 0 outside the
// row.
template <bool F32>
struct Any8 {
    static constexpr int kSize = F32 ? 4 : 2, kVecs = F32 ? 2 : 1;
    uint4 v[kVecs];

    static __device__ __forceinline__ bool loads(const void *row, int i, int lie, Room room) {
        if (lie != kPartial) return lie == kWhole;
        const char *p = static_cast<const char *>(row) + (int64_t)i * kSize;
        return p >= room.begin && p + 8 * kSize <= room.end;
    }
    __device__ __forceinline__ void load(const void *row, int i, int H, int lie, Room room) {
        if (loads(row, i, lie, room)) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + (int64_t)i * kSize);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) v[k] = p[k];
        } else if (lie != kAbsent) {
            gather(row, i, H);
        }
    }
    __device__ __forceinline__ void gather(const void *row, int i, int H) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) v[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = i; j < i + 8; ++j) {   // the next column comes in at the top
            const bool in = j >= 0 && j < H;
            if (F32) {
                v[0] = make_uint4(v[0].y, v[0].z, v[0].w, v[kVecs - 1].x);
                v[kVecs - 1] = make_uint4(v[kVecs - 1].y, v[kVecs - 1].z, v[kVecs - 1].w,
                                          in ? static_cast<const uint32_t *>(row)[j] : 0u);
            } else {
                const uint32_t c = in ? static_cast<const uint16_t *>(row)[j] : 0u;
                v[0] = make_uint4(__funnelshift_r(v[0].x, v[0].y, 16), __funnelshift_r(v[0].y, v[0].z, 16),
                                  __funnelshift_r(v[0].z, v[0].w, 16), v[0].w >> 16 | c << 16);
            }
        }
    }
    __device__ __forceinline__ void floats(int i, int H, int lie, float (&f)[8]) const {
        Raw8<F32, false> raw;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) raw.v[k] = lie == kAbsent ? make_uint4(0, 0, 0, 0) : v[k];
        raw.floats(nullptr, 0, 0, f);
        if (lie == kPartial)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i + j < 0 || i + j >= H) f[j] = 0.f;
    }
};

// Columns [i, i + 8) of a row on 16-byte boundaries; i and H are multiples of 8.
template <bool F32>
struct Even8 {
    Raw8<F32, false> raw;
    __device__ __forceinline__ void load(const void *row, int i, int H, int = 0, Room = {}) { raw.load(row, i, H); }
    __device__ __forceinline__ void floats(float (&f)[8]) const { raw.floats(nullptr, 0, 0, f); }
    __device__ __forceinline__ void floats(int, int, int, float (&f)[8]) const { floats(f); }
};

// Weights of columns [i, i + 8), read once by a kernel whose rows may lie in any way.
template <bool F32>
struct Single8 {
    float f[8];

    __device__ __forceinline__ void load(const void *w, int i, int H) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = 0.f;
            if (i + j >= 0 && i + j < H)
                f[j] = F32 ? static_cast<const float *>(w)[i + j]
                           : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i + j]);
        }
    }
    __device__ __forceinline__ void floats(float (&o)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = f[j];
    }
};

template <bool F32, bool ODD>
struct Row {
    using Part = std::conditional_t<ODD, Any8<F32>, Even8<F32>>;
    using Weights = std::conditional_t<ODD, Single8<F32>, Even8<F32>>;
};

// Columns [i, i + 8) of a row, those of them in [0, H): 16 bytes at once where they lie so, else
// one by one.
template <bool F32, bool ODD>
__device__ __forceinline__ void store_part(void *row, int i, int H, int lie, const float (&f)[8]) {
    if (ODD ? lie == kAbsent || H == 0 : i >= H) return;
    if (!ODD || lie == kWhole) {
        store8<F32, false>(row, i, H, f);
    } else if (F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j >= 0 && i + j < H) static_cast<float *>(row)[i + j] = f[j];
    } else {   // (a loop, for short code: the next column goes out at the bottom)
        uint4 v = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
#pragma unroll 1
        for (int j = i; j < i + 8; ++j) {
            if (j >= 0 && j < H) static_cast<uint16_t *>(row)[j] = (uint16_t)v.x;
            v = make_uint4(__funnelshift_r(v.x, v.y, 16), __funnelshift_r(v.y, v.z, 16), __funnelshift_r(v.z, v.w, 16), v.w >> 16);
        }
    }
}

// Rows that a thread has under way in shared memory, where a block's fit (up to 16384 columns of
// bf16, 8192 of float32): its own columns alone, so that no barrier is needed.  2000 rows of 12000
// columns 59 us, 92 with the next row in registers, which then spill.
template <int VPT, bool R32>
struct Ring {
    static constexpr bool kUsed = VPT == 2 || (VPT == 4 && !R32);
    static constexpr int kStages = R32 || VPT == 4 ? 2 : 3;
    static constexpr int kHalf = R32 ? 2 : 1;                  // 16-byte pieces of 8 columns of h, dsum
    static constexpr int kPieces = VPT * (1 + 2 * kHalf);      // of a row, for a thread
    static size_t bytes(int threads) { return kUsed ? (size_t)kStages * kPieces * threads * 16 : 0; }
};

__device__ __forceinline__ void copy_16(uint4 *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}

// Each block takes every gridDim.x-th group of blockDim.y rows and keeps its columns' sums of
// dout * xhat in registers; they leave as one row of `part`.  The next rows' inputs are under way
// (Ring; else the next row's, in registers) while one is computed.  ODD: rows off 16-byte
// boundaries.  Chunk c covers columns [8c - s, 8c - s + 8), where s is the number of elements by
// which the row of dout starts behind a boundary, so that what lies as dout does is read and
// written 16 bytes at a time; a thread's rows are a multiple of 8 apart and so lie alike, and
// what is where is found out once.  (With aligned windows around columns of the row, moved into
// place, and no ring: 4096 rows of 4097 columns 109 us against 71, 3000 of 7999 103 against 69,
// 12000 of 1001 50 against 38.)
template <int VPT, int MAXT, bool R32, bool W32, bool ODD>
__global__ void __launch_bounds__(MAXT, 1) add_rmsnorm_backward_kernel(NormBackArgs a) {
    using R = Ring<VPT, R32>;
    __shared__ float red[2][32];
    extern __shared__ __align__(16) uint4 dynamic[];   // the ring, then [H] floats when blockDim.y > 1
    const int threads = blockDim.x * blockDim.y;
    float *cols = reinterpret_cast<float *>(dynamic + (R::kUsed ? R::kStages * R::kPieces * threads : 0));
    uint4 *mine = dynamic + threadIdx.y * blockDim.x + threadIdx.x;   // piece p of stage s: [(s * kPieces + p) * threads]
    pdl_begin();
    pdl_trigger();
    float dw[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[v][j] = 0.f;
    typename Row<W32, ODD>::Weights rw[VPT];
    typename Row<false, ODD>::Part rg[VPT];
    typename Row<R32, ODD>::Part rh[VPT], rs[VPT];
    auto dout = [&](int64_t t) { return static_cast<const __nv_bfloat16 *>(a.dout) + (t < a.T ? t : 0) * a.ds; };
    auto h = [&](int64_t t) { return static_cast<const char *>(a.h) + (t < a.T ? t : 0) * a.hs * (R32 ? 4 : 2); };
    auto dsum = [&](int64_t t) { return static_cast<const char *>(a.dsum) + (t < a.T ? t : 0) * a.ss * (R32 ? 4 : 2); };
    auto dx = [&](int64_t t) { return static_cast<char *>(a.dx) + (t < a.T ? t : 0) * a.os * (R32 ? 4 : 2); };
    auto columns = [&](int64_t t) { return t < a.T ? a.H : 0; };   // rows past the end have none
    const int64_t groups = ((int64_t)a.T + blockDim.y - 1) / blockDim.y, step = (int64_t)gridDim.x * blockDim.y;
    int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int first = 8 * (int)threadIdx.x - (ODD && a.shift ? (int)((reinterpret_cast<uintptr_t>(dout(t)) & 15) >> 1) : 0);
    auto column = [&](int v) { return first + 8 * v * (int)blockDim.x; };
    const Room groom = room_of(a.dout, a.T, a.ds, a.H, 2), hroom = room_of(a.h, a.T, a.hs, a.H, R32 ? 4 : 2),
               sroom = room_of(a.dsum, a.T, a.ss, a.H, R32 ? 4 : 2);
    int lies[VPT];   // ODD: of dout, h, dsum and dx
    if (ODD)
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = column(v), H = columns(t);
            lies[v] = lie_of(dout(t), i, H, 2) | lie_of(h(t), i, H, R32 ? 4 : 2) << 2 |
                      lie_of(dsum(t), i, H, R32 ? 4 : 2) << 4 | lie_of(dx(t), i, H, R32 ? 4 : 2) << 6;
        }
    auto lie = [&](int64_t t, int v, int k) { return ODD && t < a.T ? lies[v] >> 2 * k & 3 : kAbsent; };
#pragma unroll
    for (int v = 0; v < VPT; ++v) rw[v].load(a.w, column(v), a.H);
    // Ring: the pieces of dout, h, dsum of chunk v are v, VPT + kHalf v, VPT + kHalf (VPT + v)
    auto copy_row = [&](int64_t t, int stage) {
        uint4 *to = mine + stage * R::kPieces * threads;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = column(v);
            constexpr int size = R32 ? 4 : 2;
            if (ODD ? Any8<false>::loads(dout(t), i, lie(t, v, 0), groom) : i < columns(t)) copy_16(to + v * threads, dout(t) + i);
            const bool with_h = ODD ? Any8<R32>::loads(h(t), i, lie(t, v, 1), hroom) : i < columns(t);
            const bool with_sum = a.dsum && (ODD ? Any8<R32>::loads(dsum(t), i, lie(t, v, 2), sroom) : i < columns(t));
#pragma unroll
            for (int k = 0; k < R::kHalf; ++k) {
                if (with_h) copy_16(to + (VPT + R::kHalf * v + k) * threads, h(t) + (int64_t)i * size + 16 * k);
                if (with_sum) copy_16(to + (VPT + R::kHalf * (VPT + v) + k) * threads, dsum(t) + (int64_t)i * size + 16 * k);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](auto &part, const void *matrix_row, int64_t t, int i, int lie, Room room, const uint4 *from) {
        if constexpr (ODD) {
#pragma unroll
            for (int k = 0; k < part.kVecs; ++k) part.v[k] = from[k * threads];
            if (lie != kAbsent && !part.loads(matrix_row, i, lie, room)) part.gather(matrix_row, i, columns(t));   // not copied
        } else {
#pragma unroll
            for (int k = 0; k < part.raw.kVecs; ++k) part.raw.v[k] = i < columns(t) ? from[k * threads] : make_uint4(0, 0, 0, 0);
        }
    };
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            rg[v].load(dout(t), column(v), columns(t), lie(t, v, 0), groom);
            rh[v].load(h(t), column(v), columns(t), lie(t, v, 1), hroom);
        }
    };
    auto fetch_dsum = [&](int64_t t) {
        if (a.dsum)
#pragma unroll
            for (int v = 0; v < VPT; ++v) rs[v].load(dsum(t), column(v), columns(t), lie(t, v, 2), sroom);
    };
    if constexpr (R::kUsed) {
        for (int s = 0; s < R::kStages - 1; ++s) copy_row(t + s * step, s);
    } else {
        fetch(t);
        fetch_dsum(t);
    }
    float rstd = t < a.T ? a.rstd[t] : 0.f;
    int turn = 0, stage = 0;
    for (int64_t gr = blockIdx.x; gr < groups; gr += gridDim.x, t += step) {
        const uint4 *row = mine + stage * R::kPieces * threads;
        if constexpr (R::kUsed) {
            copy_row(t + (R::kStages - 1) * step, stage == 0 ? R::kStages - 1 : stage - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 1) : "memory");
            stage = stage + 1 == R::kStages ? 0 : stage + 1;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                take(rg[v], dout(t), t, column(v), lie(t, v, 0), groom, row + v * threads);
                take(rh[v], h(t), t, column(v), lie(t, v, 1), hroom, row + (VPT + R::kHalf * v) * threads);
            }
        }
        const float rt = rstd;
        float g[VPT][8], xh[VPT][8];
        float along = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float w[8];
            rg[v].floats(column(v), columns(t), lie(t, v, 0), g[v]);
            rh[v].floats(column(v), columns(t), lie(t, v, 1), xh[v]);
            rw[v].floats(w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[v][j] *= rt;
                dw[v][j] = fmaf(g[v][j], xh[v][j], dw[v][j]);
                g[v][j] *= w[j];
                along = fmaf(g[v][j], xh[v][j], along);
            }
        }
        if constexpr (!R::kUsed) fetch(t + step);
        rstd = t + step < a.T ? a.rstd[t + step] : 0.f;
        along = row_sum(along, red[turn]) / (float)a.H;   // (two turns: the last row's sums are read until the next barrier)
        turn ^= 1;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[v][j] = rt * (g[v][j] - xh[v][j] * along);
            if (a.dsum) {
                float d[8];
                if constexpr (R::kUsed)
                    take(rs[v], dsum(t), t, column(v), lie(t, v, 2), sroom, row + (VPT + R::kHalf * (VPT + v)) * threads);
                rs[v].floats(column(v), columns(t), lie(t, v, 2), d);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[v][j] += d[j];
            }
        }
        // (dx may be dsum: this row's is read by now, and the others are other rows)
        if constexpr (!R::kUsed) fetch_dsum(t + step);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            store_part<R32, ODD>(dx(t), column(v), columns(t), lie(t, v, 3), g[v]);
    }
    __syncthreads();
    float *part = a.part + (int64_t)blockIdx.x * a.H;
    if (blockDim.y == 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) store_part<true, ODD>(part, column(v), a.H, kOff, dw[v]);
        return;
    }
    for (int y = 0; y < (int)blockDim.y; ++y) {   // the rows' sums in a fixed order
        if ((int)threadIdx.y == y) {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = column(v) + j;
                    if (i >= 0 && i < a.H) cols[i] = (y ? cols[i] : 0.f) + dw[v][j];
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

// The gradient holds more for each column (the column's sum, a second input): 2 chunks per
// thread up to 8192 columns, 4 up to 16384, 8 above.  (8192 rows of 5120 columns 67 us with 2 chunks,
// 91 with 4; of 8192 columns 88 and 116.)
NormShape norm_back_shape(int64_t chunks) { return spread(chunks, chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8); }

int backward_blocks(const moe_norm *n, const NormShape &sh) {
    const int64_t groups = ((int64_t)n->num_tokens + sh.rows - 1) / sh.rows;
    return (int)(groups < kMaxParts ? groups : kMaxParts);
}

template <typename F>
cudaError_t with_shape(const NormShape &sh, bool r32, bool w32, bool odd, F &&f) {
    if (sh.vpt == 2) return with_types(Shape<2, 512>{}, r32, w32, odd, f);
    if (sh.vpt == 4) return with_types(Shape<4, 512>{}, r32, w32, odd, f);
    return with_types(Shape<8, 1024>{}, r32, w32, odd, f);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

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
    // Up to 7 columns of room before the first, as in the norm.  Where dout alone is off the
    // boundaries, it is the one that is fetched column by column: h, dsum and dx lie alike (4096
    // rows of 4096, dout's stride 4097: 161 us with chunks by dout, three quarters of it fetched).
    const bool shift = !even_rows(dout_dev, stride_of(n, n->x_stride), 2) &&
                       !even_rows(h_dev, stride_of(n, n->residual_stride), rb) && n->hidden <= MOE_MAX_HIDDEN - 8;
    const NormShape sh = norm_back_shape(((int64_t)n->hidden + (shift ? 7 : 0) + 7) / 8);
    const int blocks = backward_blocks(n, sh);
    float *part = static_cast<float *>(workspace_dev);
    if (blocks > 0) {
        NormBackArgs a{dout_dev, h_dev, weight_dev, dsum_dev, dx_dev, rstd_dev, part, stride_of(n, n->x_stride),
                       stride_of(n, n->residual_stride), stride_of(n, n->sum_stride),
                       stride_of(n, n->out_stride), n->num_tokens, n->hidden, shift};
        const bool odd = n->hidden % 8 || !is_aligned(weight_dev, 16) || !even_rows(dout_dev, a.ds, 2) ||
                         !even_rows(h_dev, a.hs, rb) || !even_rows(dsum_dev, a.ss, rb) || !even_rows(dx_dev, a.os, rb);
        const cudaError_t e = with_shape(
            sh, n->residual_dtype == MOE_DTYPE_FP32, n->weight_dtype == MOE_DTYPE_FP32, odd,
            [&](auto v, auto r32, auto w32, auto odd) {
                using S = decltype(v);
                constexpr auto kernel = add_rmsnorm_backward_kernel<S::vpt, S::maxt, decltype(r32)::value,
                                                                    decltype(w32)::value, decltype(odd)::value>;
                using R = Ring<S::vpt, decltype(r32)::value>;
                const size_t cols = sh.rows > 1 ? (size_t)n->hidden * 4 : 0;   // at most 8 KB: rows > 1 up to 2048 columns
                const cudaError_t set = allow_smem<kernel>(R::bytes(S::maxt) + 8192);
                if (set != cudaSuccess) return set;
                return launch_pdl(kernel, dim3(blocks), dim3(sh.threads, sh.rows), R::bytes(sh.threads * sh.rows) + cols, s, a);
            });
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return status_of(launch_pdl(sum_parts_kernel, dim3((n->hidden + 31) / 32), dim3(32, 32), 0, s,
                                (const float *)part, dweight_dev, blocks, (int)n->hidden));
}

}  // extern "C"
