// Router in front of the expert layer: expert ids and routing weights from the gate's logits
// (moe_route_topk), and the logits' gradient (moe_route_topk_backward); declared in
// include/moe_block.h.
//
// One warp per token; lane l holds the EPL consecutive experts from l * EPL on, so that the
// lowest lane with a value holds its lowest expert.  Keys are compared as 32-bit integers
// whose order is that of the floats; 0 is "absent".
#include "block_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;   // tokens per block

struct RouterArgs {
    const void *logits;
    const float *bias;
    void *ids;
    float *weights;          // backward: dweights
    void *dlogits;
    int64_t stride;          // of logits, in elements
    int T, E, k, sigmoid, groups, top_groups, pair, renorm, f32, ids64, by_logit;
    float scale;
};

// Order-preserving image of a float; 0 for -infinity and NaN ("absent").  -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return v > -__int_as_float(0x7f800000) ? o : 0u;
}
__device__ __forceinline__ float of_key(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Logit of expert e as float32, -infinity beyond the last expert and for NaN; +infinity
// counts as the largest finite value.
__device__ __forceinline__ float load_logit(const RouterArgs &a, int64_t t, int e) {
    const float none = -__int_as_float(0x7f800000);
    if (e >= a.E) return none;
    const float v = a.f32 ? static_cast<const float *>(a.logits)[t * a.stride + e]
                          : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[t * a.stride + e]);
    return v != v ? none : fminf(v, 3.402823466e38f);
}

__device__ __forceinline__ float sigmoid(float v) { return __fdiv_rn(1.0f, 1.0f + expf(-v)); }

// Scores of a lane's experts.  Softmax over the whole row, with the row's maximum taken out
// before the exponential; a row with no expert has all scores 0.
template <int EPL>
__device__ __forceinline__ void score_row(const RouterArgs &a, const float (&l)[EPL], float (&s)[EPL]) {
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = sigmoid(l[j]);
        return;
    }
    float m = -3.402823466e38f;   // the lowest finite value is a logit like any other
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, o));
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        s[j] = expf(l[j] - m);
        z += s[j];
    }
    z = fmaxf(warp_sum(z), 1e-38f);
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] = __fdiv_rn(s[j], z);
}

template <int EPL>
__global__ void __launch_bounds__(kWarps * 32) route_topk_kernel(RouterArgs a) {
    extern __shared__ uint32_t shared_keys[];   // [kWarps][E] with groups
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    float l[EPL], s[EPL];
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = load_logit(a, t, lane * EPL + j);
    score_row<EPL>(a, l, s);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane * EPL + j;
        const float b = a.bias && e < a.E ? a.bias[e] : 0.f;
        key[j] = key_of(a.by_logit ? l[j] : __fadd_rn(s[j], b));
        if (key_of(l[j]) == 0) key[j] = 0;
    }

    if (a.groups > 1) {   // lane g takes group g's score and its rank among the groups
        uint32_t *keys = shared_keys + warp * a.E;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane * EPL + j < a.E) keys[lane * EPL + j] = key[j];
        __syncwarp();
        const int size = a.E / a.groups;
        uint32_t score = 0;
        if (lane < a.groups) {
            uint32_t first = 0, second = 0;
            for (int i = 0; i < size; ++i) {
                const uint32_t v = keys[lane * size + i];
                second = max(second, min(first, v));
                first = max(first, v);
            }
            score = a.pair && second != 0 ? key_of(__fadd_rn(of_key(first), of_key(second))) : first;
        }
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const uint32_t other = __shfl_sync(kAllLanes, score, g);
            rank += other > score || (other == score && g < lane);
        }
        const uint32_t kept = __ballot_sync(kAllLanes, lane < a.groups && rank < a.top_groups);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane * EPL + j < a.E && !((kept >> ((lane * EPL + j) / size)) & 1)) key[j] = 0;
    }

    // k times the largest key; lane j keeps pick j
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) best = max(best, key[j]);
    int id = -1;
    float w = 0.f;
    for (int i = 0; i < a.k; ++i) {
        const uint32_t top = __reduce_max_sync(kAllLanes, best);
        if (top == 0) break;
        const int owner = __ffs(__ballot_sync(kAllLanes, best == top)) - 1;
        int at = -1;
        float sc = 0.f;
        if (lane == owner) {
            best = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                if (at < 0 && key[j] == top) {
                    at = lane * EPL + j;
                    sc = s[j];
                    key[j] = 0;
                }
                best = max(best, key[j]);
            }
        }
        at = __shfl_sync(kAllLanes, at, owner);
        sc = __shfl_sync(kAllLanes, sc, owner);
        if (lane == i) {
            id = at;
            w = sc;
        }
    }
    if (a.renorm) w = __fdiv_rn(w, fmaxf(warp_sum(w), 1e-38f));
    if (lane < a.k) {
        const int64_t o = t * a.k + lane;
        if (a.ids64) static_cast<int64_t *>(a.ids)[o] = id;
        else static_cast<int32_t *>(a.ids)[o] = id;
        a.weights[o] = w * a.scale;
    }
}

// With p the picked scores, z their sum and g = scale * dweights:
//   ds = g, or (g - sum(g p)/z)/z where renormalised (0 outside the picks);
//   dlogit = ds s (1 - s) for the sigmoid, s (ds - sum(ds s)) for the softmax.
template <int EPL>
__global__ void __launch_bounds__(kWarps * 32) route_topk_backward_kernel(RouterArgs a) {
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    float l[EPL], s[EPL], d[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        l[j] = load_logit(a, t, lane * EPL + j);
        d[j] = 0.f;
    }
    score_row<EPL>(a, l, s);
    int id = -1;
    float g = 0.f;
    if (lane < a.k) {
        const int64_t o = t * a.k + lane;
        const int64_t v = a.ids64 ? static_cast<const int64_t *>(a.ids)[o] : static_cast<const int32_t *>(a.ids)[o];
        if (v >= 0 && v < a.E) {
            id = (int)v;
            g = a.weights[o] * a.scale;
        }
    }
    if (a.renorm) {
        float p = 0.f;   // the score of this lane's pick
        for (int i = 0; i < a.k; ++i) {
            const int e = __shfl_sync(kAllLanes, id, i);
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (e == lane * EPL + j) v = s[j];
            v = e >= 0 ? __shfl_sync(kAllLanes, v, e / EPL) : 0.f;
            if (lane == i) p = v;
        }
        const float z = fmaxf(warp_sum(p), 1e-38f);
        const float along = __fdiv_rn(warp_sum(g * p), z);
        g = id >= 0 ? __fdiv_rn(g - along, z) : 0.f;
    }
    for (int i = 0; i < a.k; ++i) {
        const int e = __shfl_sync(kAllLanes, id, i);
        const float v = __shfl_sync(kAllLanes, g, i);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (e == lane * EPL + j) d[j] += v;
    }
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) d[j] = d[j] * s[j] * (1.0f - s[j]);
    } else {
        float along = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) along = fmaf(d[j], s[j], along);
        along = warp_sum(along);
#pragma unroll
        for (int j = 0; j < EPL; ++j) d[j] = s[j] * (d[j] - along);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane * EPL + j;
        if (e >= a.E) continue;
        if (a.f32) static_cast<float *>(a.dlogits)[t * a.E + e] = d[j];
        else static_cast<__nv_bfloat16 *>(a.dlogits)[t * a.E + e] = __float2bfloat16_rn(d[j]);
    }
}

int check_router(const moe_router *r, int32_t num_tokens, int ids_dtype) {
    if (!r || num_tokens < 0 || r->num_experts < 1 || r->groups < 1 || r->top_groups < 1 ||
        r->top_groups > r->groups || r->num_experts % r->groups != 0 || r->score < 0 || r->score > 1 ||
        r->group_score < 0 || r->group_score > 1 || bad_dtype(r->logits_dtype) ||
        (r->logits_stride != 0 && r->logits_stride < r->num_experts))
        return MOE_ERR_INVALID_ARGUMENT;
    if (r->num_experts > MOE_MAX_EXPERTS || r->groups > MOE_MAX_GROUPS) return MOE_ERR_LIMIT;
    if (r->top_k < 1 || r->top_k > MOE_MAX_TOPK || r->top_k > r->num_experts / r->groups * r->top_groups)
        return MOE_ERR_TOPK;
    if (ids_dtype != MOE_IDS_INT32 && ids_dtype != MOE_IDS_INT64) return MOE_ERR_IDS_DTYPE;
    return MOE_OK;
}

RouterArgs router_args(const moe_router *r, int32_t T, const void *logits, const float *bias, const void *ids,
                       int ids_dtype, const float *weights, void *dlogits) {
    RouterArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.ids = const_cast<void *>(ids);
    a.weights = const_cast<float *>(weights);
    a.dlogits = dlogits;
    a.stride = r->logits_stride ? r->logits_stride : r->num_experts;
    a.T = T;
    a.E = r->num_experts;
    a.k = r->top_k;
    a.sigmoid = r->score == MOE_SCORE_SIGMOID;
    a.groups = r->groups;
    a.top_groups = r->top_groups;
    a.pair = r->group_score == MOE_GROUP_TOP2;
    a.renorm = r->renormalize != 0;
    a.f32 = r->logits_dtype == MOE_DTYPE_FP32;
    a.ids64 = ids_dtype == MOE_IDS_INT64;
    a.by_logit = !bias && (r->groups == 1 || !a.pair);
    a.scale = r->scale;
    return a;
}

// Calls f with the number of experts per lane as a compile-time power of two.
template <typename F>
cudaError_t with_epl(int E, F &&f) {
    if (E <= 32) return f(std::integral_constant<int, 1>{});
    if (E <= 64) return f(std::integral_constant<int, 2>{});
    if (E <= 128) return f(std::integral_constant<int, 4>{});
    if (E <= 256) return f(std::integral_constant<int, 8>{});
    if (E <= 512) return f(std::integral_constant<int, 16>{});
    if (E <= 1024) return f(std::integral_constant<int, 32>{});
    return f(std::integral_constant<int, 64>{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_route_topk(const moe_router *r, int32_t num_tokens, const void *logits_dev, const float *bias_dev,
                   void *topk_ids_dev, int ids_dtype, float *topk_weights_dev, void *stream) {
    int rc = check_router(r, num_tokens, ids_dtype);
    if (rc != MOE_OK) return rc;
    if (num_tokens > 0 && (!logits_dev || !topk_ids_dev || !topk_weights_dev)) return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(logits_dev, dtype_bytes(r->logits_dtype)) || !is_aligned(bias_dev, 4) ||
        !is_aligned(topk_ids_dev, ids_dtype == MOE_IDS_INT64 ? 8 : 4) || !is_aligned(topk_weights_dev, 4))
        return MOE_ERR_MISALIGNED;
    if ((rc = check_device()) != MOE_OK) return rc;
    if (num_tokens == 0) return MOE_OK;
    const RouterArgs a = router_args(r, num_tokens, logits_dev, bias_dev, topk_ids_dev, ids_dtype,
                                     topk_weights_dev, nullptr);
    const size_t smem = a.groups > 1 ? (size_t)kWarps * a.E * 4 : 0;   // at most 32 KB
    return status_of(with_epl(a.E, [&](auto epl) {
        return launch_pdl(route_topk_kernel<decltype(epl)::value>, dim3((a.T + kWarps - 1) / kWarps),
                          dim3(kWarps * 32), smem, static_cast<cudaStream_t>(stream), a);
    }));
}

int moe_route_topk_backward(const moe_router *r, int32_t num_tokens, const void *logits_dev,
                            const void *topk_ids_dev, int ids_dtype, const float *dweights_dev,
                            void *dlogits_dev, void *stream) {
    int rc = check_router(r, num_tokens, ids_dtype);
    if (rc != MOE_OK) return rc;
    if (num_tokens > 0 && (!logits_dev || !topk_ids_dev || !dweights_dev || !dlogits_dev))
        return MOE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(logits_dev, dtype_bytes(r->logits_dtype)) || !is_aligned(dlogits_dev, dtype_bytes(r->logits_dtype)) ||
        !is_aligned(topk_ids_dev, ids_dtype == MOE_IDS_INT64 ? 8 : 4) || !is_aligned(dweights_dev, 4))
        return MOE_ERR_MISALIGNED;
    if ((rc = check_device()) != MOE_OK) return rc;
    if (num_tokens == 0) return MOE_OK;
    const RouterArgs a = router_args(r, num_tokens, logits_dev, nullptr, topk_ids_dev, ids_dtype, dweights_dev,
                                     dlogits_dev);
    return status_of(with_epl(a.E, [&](auto epl) {
        return launch_pdl(route_topk_backward_kernel<decltype(epl)::value>, dim3((a.T + kWarps - 1) / kWarps),
                          dim3(kWarps * 32), 0, static_cast<cudaStream_t>(stream), a);
    }));
}

}  // extern "C"
