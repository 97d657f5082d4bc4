// Router in front of the expert layer: expert ids and routing weights from the gate's logits
// (moe_route_topk), and the logits' gradient (moe_route_topk_backward); declared in
// include/moe_block.h.
//
// One warp per token; lane l holds the EPL consecutive experts from l * EPL on, so that the
// lowest lane with a value holds its lowest expert.  An absent expert's key is -infinity.
//
// The logits are read once and little is written, but a token's selection takes a few hundred
// instructions for E = 256: the instruction issue bounds large batches, the launch small ones.
// So the k largest keys are not taken out one by one: the k-th largest of the lanes' maxima is
// a bound that few keys reach (about 11 for k = 8 of 256); these are put together in shared
// memory and ranked against each other, one to a lane.
//
// Measured, 256 experts, sigmoid, bias, 4 of 8 groups by pairs, k = 8: 64 tokens 2.6 us, 32768
// tokens (37 MB) 21 us: 0.26 of HBM, the schedulers issue in 86% of the cycles (taking the k
// largest out one by one: 65 us).  16381 tokens of 128 experts, softmax, k = 4: 6.7 us; 32768 of 8
// experts, k = 2: 10.6 us, since a token takes a warp however few its experts are.  The gradient at
// 32768 x 256 (70 MB): 13.6 us, 0.77 of HBM (sigmoid 12.0, renormalised 14.2); the loads' latency,
// once for each token's warp, is the rest.
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
    int lanes_per_group, group_shift;   // where a group is a power of two of whole lanes, else 0; its exponent
    float scale;
};

constexpr float kNone = -__builtin_huge_valf();   // the key of an absent expert
constexpr float kMost = 3.402823466e38f;

// An integer that orders as the float does (-0 as +0), and back.
__device__ __forceinline__ int order_of(float v) {
    const int i = __float_as_int(v + 0.0f);
    return i ^ (i >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float of_order(int i) { return __int_as_float(i ^ (i >> 31 & 0x7fffffff)); }

// A lane's EPL values of a row, `fill` beyond the last one.  VEC: four at a time; the lanes'
// experts then all exist or none of them does.
template <int EPL, bool VEC>
__device__ __forceinline__ void load_values(const void *row, bool f32, int first, int E, float fill, float (&l)[EPL]) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = fill;
    if (VEC) {
        if (first < E) {
            if (f32) {
                const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + first);
#pragma unroll
                for (int j = 0; j + 4 <= EPL; j += 4) {
                    const float4 v = p[j / 4];
                    l[j] = v.x; l[j + 1] = v.y; l[j + 2] = v.z; l[j + 3] = v.w;
                }
            } else {
                const uint2 *p = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + first);
#pragma unroll
                for (int j = 0; j + 4 <= EPL; j += 4) {
                    const uint2 v = p[j / 4];
                    l[j] = lo_f32(v.x); l[j + 1] = hi_f32(v.x); l[j + 2] = lo_f32(v.y); l[j + 3] = hi_f32(v.y);
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (first + j < E)
                l[j] = f32 ? static_cast<const float *>(row)[first + j]
                           : __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[first + j]);
    }
}

// -infinity for NaN; +infinity counts as the largest finite value.
__device__ __forceinline__ float clean(float v) { return fmaxf(fminf(v != v ? kNone : v, kMost), kNone); }

__device__ __forceinline__ const void *logits_row(const RouterArgs &a, int64_t t) {
    return static_cast<const char *>(a.logits) + t * a.stride * (a.f32 ? 4 : 2);
}
__device__ __forceinline__ float logit(const RouterArgs &a, int64_t t, int e) {
    const void *row = logits_row(a, t);
    return clean(a.f32 ? static_cast<const float *>(row)[e] : __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]));
}

// e^v as 2^(v log2 e) with the hardware's power of two: relative error 2^-22, and |v| 2^-23 at
// most for the roundings of the product and of log2 e.
__device__ __forceinline__ float exp_of(float v) {
    float p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(v * 1.4426950408889634f));
    return p;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + e^-v).
__device__ __forceinline__ float sigmoid(float v) { return reciprocal(1.0f + exp_of(-v)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAllLanes, v, o));
    return v;
}
template <int EPL>
__device__ __forceinline__ float row_max(const float (&l)[EPL]) {
    float m = -kMost;   // the lowest finite value is a logit like any other
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, l[j]);
    return warp_max(m);
}

// What the gradient keeps of a lane's experts.  Softmax: the scores, over the whole row, with its
// maximum taken out before the exponential, and undivided where the picks' own sum takes the
// row's out again; a row with no expert has all scores 0.  Sigmoid: u = e^-logit, at most the
// largest finite number, from which s = 1 / (1 + u), and 1 - s = u s with all its digits where s
// is next to 1.
template <int EPL>
__device__ __forceinline__ void score_row(const RouterArgs &a, const float (&l)[EPL], float (&s)[EPL]) {
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = fminf(exp_of(-l[j]), kMost);
        return;
    }
    const float m = row_max<EPL>(l);
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        s[j] = exp_of(l[j] - m);
        z += s[j];
    }
    if (a.renorm) return;
    z = __fdiv_rn(1.0f, fmaxf(warp_sum(z), 1e-38f));
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] *= z;
}

// v joins a group's two largest keys.
__device__ __forceinline__ void join(float v, float &first, float &second) {
    second = fmaxf(second, fminf(first, v));
    first = fmaxf(first, v);
}

// Takes the keys of experts outside the top_groups best groups out.
template <int EPL>
__device__ __forceinline__ void keep_groups(const RouterArgs &a, int lane, float (&key)[EPL], float *keys) {
    float first = kNone, second = kNone;
    if (a.lanes_per_group > 0) {      // whole lanes, a power of two of them: exchanges among these
#pragma unroll
        for (int j = 0; j < EPL; ++j) join(key[j], first, second);
        for (int o = 1; o < a.lanes_per_group; o <<= 1) {
            const float f = __shfl_xor_sync(kAllLanes, first, o), s = __shfl_xor_sync(kAllLanes, second, o);
            second = fmaxf(fmaxf(second, s), fminf(first, f));
            first = fmaxf(first, f);
        }
        // a group's lanes share out the comparisons with the groups
        const float score = a.pair && second > kNone ? first + second : first;
        const int per = a.lanes_per_group, mine = lane >> a.group_shift;
        int rank = 0;
        for (int g = lane & (per - 1); g < a.groups + (lane & (per - 1)); g += per) {
            const float other = __shfl_sync(kAllLanes, score, (g << a.group_shift) & 31);
            rank += g < a.groups && (other > score || (other == score && g < mine));
        }
        for (int o = 1; o < per; o <<= 1) rank += __shfl_xor_sync(kAllLanes, rank, o);
        if (rank >= a.top_groups)
#pragma unroll
            for (int j = 0; j < EPL; ++j) key[j] = kNone;
        return;
    }
    // any other size: through shared memory, a lane to each group
    const int size = a.E / a.groups;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        if (lane * EPL + j < a.E) keys[lane * EPL + j] = key[j];
    __syncwarp();
    if (lane < a.groups)
        for (int i = 0; i < size; ++i) join(keys[lane * size + i], first, second);
    __syncwarp();
    const float score = a.pair && second > kNone ? first + second : first;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
        const float other = __shfl_sync(kAllLanes, score, g);
        rank += other > score || (other == score && g < lane);
    }
    const uint32_t kept = __ballot_sync(kAllLanes, lane < a.groups && rank < a.top_groups);
    int g = lane * EPL / size, rest = lane * EPL - g * size;   // of the lane's first expert
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        if (!((kept >> (g & 31)) & 1)) key[j] = kNone;
        if (++rest == size) {
            rest = 0;
            ++g;
        }
    }
}

// A token's room in shared memory: the keys (keep_groups), or 32 candidates (key and expert).
__host__ __device__ constexpr int room_of(int E) { return (E > 64 ? E : 64) + 3 & ~3; }

template <int EPL, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) route_topk_kernel(RouterArgs a) {
    extern __shared__ __align__(16) float rooms[];   // [kWarps][room_of(E)]
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    float *room = rooms + warp * room_of(a.E);
    float key[EPL];
    load_values<EPL, VEC>(logits_row(a, t), a.f32, lane * EPL, a.E, kNone, key);
    // m, z: what a softmax score is made with, exp(logit - m) / z
    float m = 0.f, z = 1.f;
    if (!a.sigmoid || a.by_logit) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = clean(key[j]);
    }
    if (!a.sigmoid) {
        m = row_max<EPL>(key);
        if (!a.renorm || !a.by_logit) {   // the picks' own sum takes z out again
            z = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) z += exp_of(key[j] - m);
            z = __fdiv_rn(1.0f, fmaxf(warp_sum(z), 1e-38f));
        }
    }
    if (!a.by_logit) {
        float b[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) b[j] = 0.f;
        if (a.bias) load_values<EPL, VEC>(a.bias, true, lane * EPL, a.E, 0.f, b);
        // 0 times the logit is not a number for an absent expert, and what is not, for whatever
        // reason, is no key
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const float l = fminf(key[j], kMost);
                key[j] = fmaxf(fmaf(l, 0.f, __fadd_rn(sigmoid(key[j]), b[j])), kNone);
            }
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                key[j] = fmaxf(fmaf(key[j], 0.f, __fadd_rn(exp_of(key[j] - m) * z, b[j])), kNone);
        }
    }
    if (a.groups > 1) keep_groups<EPL>(a, lane, key, room);

    // the bound: the k-th largest of the lanes' maxima; the lowest number if there are fewer
    float best = kNone;
#pragma unroll
    for (int j = 0; j < EPL; ++j) best = fmaxf(best, key[j]);
    const int none = order_of(kNone);
    int rest = order_of(best), top = none;
    for (int i = 0; i < a.k; ++i) {
        top = __reduce_max_sync(kAllLanes, rest);
        if (rest == top) rest = none;   // all of its lanes: the bound only gets lower
    }
    const float bound = fmaxf(of_order(top), -kMost);
    int count = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) count += key[j] >= bound;
    int at = count;   // candidates up to this lane's last
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAllLanes, at, o);
        if (lane >= o) at += v;
    }
    const int n = __shfl_sync(kAllLanes, at, 31);
    int id = -1, rank = lane;
    if (n <= 32) {
        // in the experts' order into shared memory; a lane's candidate comes behind those with a
        // larger key, and behind equal ones before it
        float *slot = room + (at - count);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (key[j] >= bound) {
                slot[0] = key[j];
                slot[32] = __int_as_float(lane * EPL + j);
                ++slot;
            }
        if (lane >= n) room[lane] = kNone;   // (room up to 32: lanes without a candidate)
        __syncwarp();
        if (lane < n) id = __float_as_int(room[32 + lane]);
        // up to 16: lane c and lane 16 + c compare candidate c with every other four
        const bool half = n <= 16;
        const int c = half ? lane & 15 : lane, skip = half ? 8 : 4;
        const float mine = room[c];
        int before = 0;
        for (int i = half ? lane >> 4 << 2 : 0; i < n; i += skip) {
            const float4 o = *reinterpret_cast<const float4 *>(room + i);
            before += o.x > mine || (o.x == mine && i < c);
            before += o.y > mine || (o.y == mine && i + 1 < c);
            before += o.z > mine || (o.z == mine && i + 2 < c);
            before += o.w > mine || (o.w == mine && i + 3 < c);
        }
        const int rest = __shfl_xor_sync(kAllLanes, before, 16);
        if (half) before += rest;
        rank = lane < n ? before : lane;   // (lanes without a candidate keep the places from n on)
    } else {   // many equal keys, or k near the number of lanes: one by one, pick i to lane i
        for (int i = 0; i < a.k; ++i) {
            const float top = of_order(__reduce_max_sync(kAllLanes, order_of(best)));
            if (top == kNone) break;
            const int owner = __ffs(__ballot_sync(kAllLanes, best == top)) - 1;
            int which = -1;
            if (lane == owner) {
                best = kNone;
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    if (which < 0 && key[j] == top) {
                        which = lane * EPL + j;
                        key[j] = kNone;
                    }
                    best = fmaxf(best, key[j]);
                }
            }
            which = __shfl_sync(kAllLanes, which, owner);
            if (lane == i) id = which;
        }
    }
    float w = 0.f;
    if (rank < a.k && id >= 0) {   // the pick's score, from its logit
        const float l = logit(a, t, id);
        w = a.sigmoid ? sigmoid(l) : exp_of(l - m);
        // The softmax's own sum would only be taken out again, and what it makes of small scores
        // lies below float32's normal numbers.
        if (!a.sigmoid && !a.renorm) w *= z;
    }
    if (a.renorm) w = __fdividef(w, fmaxf(warp_sum(w), 1e-38f));   // (the sum is 0 or at least 2^-126)
    if (rank < a.k) {
        const int64_t o = t * a.k + rank;
        if (a.ids64) static_cast<int64_t *>(a.ids)[o] = id;
        else static_cast<int32_t *>(a.ids)[o] = id;
        a.weights[o] = w * a.scale;
    }
}

// With s the scores, g = scale * dweights, and q = s / (the picks' sum of s) the picks' shares:
//   sigmoid   dlogit = s (1 - s) g at the picks, or where renormalised q (1 - s) (g - sum(g q));
//   softmax   s (d - sum(d s)) with d = g at the picks and 0 elsewhere, or where renormalised
//             q (g - sum(g q)) at the picks: the softmax's own sum takes no part.
// The shares are formed first, 0 where the sum is 0: nothing is divided by a sum that may be as
// small as a score.
template <int EPL, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) route_topk_backward_kernel(RouterArgs a) {
    extern __shared__ __align__(16) float rooms[];   // [kWarps][32 * EPL]
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    float *room = rooms + warp * 32 * EPL;
    float l[EPL], s[EPL], d[EPL];
    load_values<EPL, VEC>(logits_row(a, t), a.f32, lane * EPL, a.E, kNone, l);
    int64_t v = -1;
    float g = 0.f;
    if (lane < a.k) {   // (all the loads are under way together)
        const int64_t o = t * a.k + lane;
        v = a.ids64 ? static_cast<const int64_t *>(a.ids)[o] : static_cast<const int32_t *>(a.ids)[o];
        g = a.weights[o] * a.scale;
    }
    const int id = v >= 0 && v < a.E ? (int)v : -1;
    if (id < 0) g = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = clean(l[j]);
    score_row<EPL>(a, l, s);
    if (a.renorm) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) room[lane * EPL + j] = a.sigmoid ? reciprocal(1.0f + s[j]) : s[j];
        __syncwarp();
        const float p = id >= 0 ? room[id] : 0.f;   // the score of this lane's pick
        __syncwarp();
        const float z = warp_sum(p);
        const float q = p * __fdiv_rn(1.0f, z > 0.f ? z : 1.0f);   // (scores are 0 or at least 2^-126: finite)
        if (!(p > 0.f)) g = 0.f;   // (an absent expert's weight's gradient may be anything)
        g = q * (g - warp_sum(g * q));
    }
    // the picks' gradients to the experts' lanes; picks of one expert add up in their order
#pragma unroll
    for (int j = 0; j < EPL; ++j) room[lane * EPL + j] = 0.f;
    __syncwarp();
    const unsigned same = __match_any_sync(kAllLanes, id);
    if (__all_sync(kAllLanes, id < 0 || __popc(same) == 1)) {
        if (id >= 0) room[id] = g;
    } else {
        for (int i = 0; i < a.k; ++i) {
            if (lane == i && id >= 0) room[id] += g;
            __syncwarp();
        }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < EPL; ++j) d[j] = room[lane * EPL + j];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float r = reciprocal(1.0f + s[j]);
            d[j] *= s[j] * r;
            if (!a.renorm) d[j] = r > 0.f ? d[j] * r : 0.f;   // (absent experts as above)
        }
    } else if (!a.renorm) {
        float along = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            d[j] = s[j] > 0.f ? d[j] * s[j] : 0.f;
            along += d[j];
        }
        along = warp_sum(along);
#pragma unroll
        for (int j = 0; j < EPL; ++j) d[j] = fmaf(-along, s[j], d[j]);
    }
    const int first = lane * EPL;
    if (VEC) {
        if (first >= a.E) return;
        if (a.f32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.dlogits) + t * a.E + first);
#pragma unroll
            for (int j = 0; j + 4 <= EPL; j += 4) o[j / 4] = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
        } else {
            uint2 *o = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dlogits) + t * a.E + first);
#pragma unroll
            for (int j = 0; j + 4 <= EPL; j += 4) o[j / 4] = make_uint2(pack_bf16(d[j], d[j + 1]), pack_bf16(d[j + 2], d[j + 3]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = first + j;
            if (e >= a.E) continue;
            if (a.f32) static_cast<float *>(a.dlogits)[t * a.E + e] = d[j];
            else static_cast<__nv_bfloat16 *>(a.dlogits)[t * a.E + e] = __float2bfloat16_rn(d[j]);
        }
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
    int epl = 1;
    while (32 * epl < a.E) epl *= 2;
    const int size = a.E / a.groups, lanes = size / epl;
    a.lanes_per_group = size % epl == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    while (1 << a.group_shift < a.lanes_per_group) ++a.group_shift;
    return a;
}

// Calls f with the number of experts per lane as a compile-time power of two, and whether the
// lanes' experts can be read (and, for the gradient, written) together: four of them aligned,
// and every lane's all there or none.
template <typename F>
cudaError_t with_epl(const RouterArgs &a, F &&f) {
    const size_t b = a.f32 ? 16 : 8;
    auto vec = [&](auto epl) {
        constexpr int n = decltype(epl)::value;
        if constexpr (n >= 4) {
            if (a.E % n == 0 && a.stride % 4 == 0 && is_aligned(a.logits, b) && is_aligned(a.dlogits, b) && is_aligned(a.bias, 16))
                return f(epl, std::true_type{});
        }
        return f(epl, std::false_type{});
    };
    if (a.E <= 32) return vec(std::integral_constant<int, 1>{});
    if (a.E <= 64) return vec(std::integral_constant<int, 2>{});
    if (a.E <= 128) return vec(std::integral_constant<int, 4>{});
    if (a.E <= 256) return vec(std::integral_constant<int, 8>{});
    if (a.E <= 512) return vec(std::integral_constant<int, 16>{});
    if (a.E <= 1024) return vec(std::integral_constant<int, 32>{});
    return vec(std::integral_constant<int, 64>{});
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
    const size_t smem = (size_t)kWarps * room_of(a.E) * 4;   // at most 32 KB
    return status_of(with_epl(a, [&](auto epl, auto vec) {
        return launch_pdl(route_topk_kernel<decltype(epl)::value, decltype(vec)::value>,
                          dim3((a.T - 1) / kWarps + 1), dim3(kWarps * 32), smem,
                          static_cast<cudaStream_t>(stream), a);
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
    return status_of(with_epl(a, [&](auto epl, auto vec) {
        constexpr int n = decltype(epl)::value;
        return launch_pdl(route_topk_backward_kernel<n, decltype(vec)::value>, dim3((a.T - 1) / kWarps + 1),
                          dim3(kWarps * 32), (size_t)kWarps * 32 * n * 4, static_cast<cudaStream_t>(stream), a);
    }));
}

}  // extern "C"
