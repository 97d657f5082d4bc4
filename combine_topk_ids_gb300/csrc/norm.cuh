// What the norm (norm.cu) and its gradient (norm_backward.cu) share: rows that are read and
// written eight columns at a time, sums over a row, argument checks.
#pragma once

#include <mutex>

#include "block_common.cuh"

namespace moe {
namespace {

// Columns [i, i + 8) of a row, in the row's own type.  load() issues 16-byte loads and nothing
// else, so that a thread's loads are under way together; floats() makes numbers of them, 0
// outside [0, H).
// ODD: the row may start anywhere and be of any length (else everything is on 16-byte
// boundaries, and i is a multiple of 8).  What load() cannot fetch, floats() reads one by one.
template <bool F32, bool ODD>
struct Raw8 {
    static constexpr int kSize = F32 ? 4 : 2, kVecs = F32 ? 2 : 1;
    uint4 v[kVecs];

    // Columns by which column i lies behind a 16-byte boundary.
    static __device__ __forceinline__ int behind(const void *row, int i) {
        return ODD ? (int)((reinterpret_cast<uintptr_t>(row) + (int64_t)i * kSize) & 15) / kSize : 0;
    }
    static __device__ __forceinline__ bool loads(const void *row, int i, int H) {
        return ODD ? i >= 0 && i + 8 <= H && behind(row, i) == 0 : i < H;
    }
    __device__ __forceinline__ void load(const void *row, int i, int H) {
        if (!ODD)
#pragma unroll
            for (int k = 0; k < kVecs; ++k) v[k] = make_uint4(0, 0, 0, 0);
        if (loads(row, i, H)) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + (int64_t)i * kSize);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) v[k] = p[k];
        }
    }
    __device__ __forceinline__ void floats(const void *row, int i, int H, float (&f)[8]) const {
        uint32_t w[4 * kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            w[4 * k] = v[k].x; w[4 * k + 1] = v[k].y; w[4 * k + 2] = v[k].z; w[4 * k + 3] = v[k].w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = F32 ? __uint_as_float(w[F32 ? j : 0]) : j & 1 ? hi_f32(w[j / 2]) : lo_f32(w[j / 2]);
        if (ODD && !loads(row, i, H)) {
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

// Columns [i, i + 8) of a row, those of them in [0, H): 16 bytes at once where the address allows
// it, else bf16 columns in pairs where theirs does.
template <bool F32, bool ODD>
__device__ __forceinline__ void store8(void *row, int i, int H, const float (&f)[8]) {
    if (!ODD && i >= H) return;
    const bool all = !ODD || (i >= 0 && i + 8 <= H);
    const int r = Raw8<F32, ODD>::behind(row, i);
    if (all && r == 0) {
        if (F32) {
            float *p = static_cast<float *>(row) + i;
            *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(row) + i) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
    } else if (!F32 && all) {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(row) + i;
        if (r & 1) {
            p[0] = __float2bfloat16_rn(f[0]);
#pragma unroll
            for (int j = 1; j < 7; j += 2) *reinterpret_cast<uint32_t *>(p + j) = pack_bf16(f[j], f[j + 1]);
            p[7] = __float2bfloat16_rn(f[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j += 2) *reinterpret_cast<uint32_t *>(p + j) = pack_bf16(f[j], f[j + 1]);
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

struct NormShape {
    int vpt, threads, rows;   // chunks per thread, threads per row, rows per block
};

// Chunks of 8 columns, vpt to a thread, over whole warps; short rows share a block of about 256
// threads.
inline NormShape spread(int64_t chunks, int vpt) {
    NormShape n;
    n.vpt = vpt;
    n.threads = (int)((chunks + 32 * vpt - 1) / (32 * vpt)) * 32;
    n.rows = n.threads >= 256 ? 1 : 256 / n.threads;
    return n;
}

inline int check_norm(const moe_norm *n) {
    if (!n) return MOE_ERR_INVALID_ARGUMENT;
    if (n->num_tokens < 0 || n->hidden < 1 || bad_dtype(n->residual_dtype) || bad_dtype(n->weight_dtype) ||
        !(n->eps >= 0.f))
        return MOE_ERR_INVALID_ARGUMENT;
    for (int64_t s : {n->x_stride, n->residual_stride, n->sum_stride, n->out_stride})
        if (s != 0 && s < n->hidden) return MOE_ERR_INVALID_ARGUMENT;
    return n->hidden > MOE_MAX_HIDDEN ? MOE_ERR_LIMIT : MOE_OK;
}

inline int64_t stride_of(const moe_norm *n, int64_t s) { return s ? s : n->hidden; }

// Calls f with a shape and the types as compile-time constants.
template <int VPT, int MAXT>
struct Shape {
    static constexpr int vpt = VPT, maxt = MAXT;
};

template <typename V, typename F>
cudaError_t with_types(V v, bool r32, bool w32, bool odd, F &&f) {
    auto weights = [&](auto r) {
        auto rows = [&](auto w) { return odd ? f(v, r, w, std::true_type{}) : f(v, r, w, std::false_type{}); };
        return w32 ? rows(std::true_type{}) : rows(std::false_type{});
    };
    return r32 ? weights(std::true_type{}) : weights(std::false_type{});
}

// Blocks of a kernel that are on the device at once, by its registers (looked up once).
template <auto KERNEL>
int64_t resident_blocks(int threads) {
    static const int regs = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, KERNEL) == cudaSuccess && at.numRegs > 0 ? (at.numRegs + 7) / 8 * 8 : 255;
    }();
    const int blocks = 65536 / (regs * threads);
    return (int64_t)num_sms() * (blocks < 1 ? 1 : blocks > 2048 / threads ? 2048 / threads : blocks);
}

// Lets a kernel have `most` bytes of dynamic shared memory (set once for each device).
template <auto KERNEL>
cudaError_t allow_smem(size_t most) {
    static std::once_flag once[64];
    static cudaError_t set[64];
    const int dev = device_ordinal();
    if (dev < 0) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    });
    return set[dev];
}

// Whether a row matrix (or NULL) lies on 16-byte boundaries throughout.
inline bool even_rows(const void *p, int64_t stride, size_t size) {
    return !p || (is_aligned(p, 16) && stride * (int64_t)size % 16 == 0);
}

}  // namespace
}  // namespace moe
