// route.hip -- routing of tokens to experts, and its gradient, for gfx950.
//
// Forward, per token (pomoai.com "DeepSeek-V3", MoE section: sigmoid scores, 8 of 256 experts
// from 4 of 8 groups, a balance bias that enters the selection only, weights renormalised
// over the selected experts and scaled):
//     s_i = 1 / (1 + exp(-x_i))   or   exp(x_i - max x) / sum exp(x - max x)
//     c_i = s_i + b_i
//     the topk_groups groups of the largest value (the sum of a group's two largest c, or its
//     largest) stay; the top_k largest c among them are the token's experts, largest first
//     w_j = scale * s_j / sum of the selected s   (or scale * s_j)
// Equal values rank by the lower index, so the result is one function of the inputs. To keep
// it so, s has a stated value: expf, additions and divisions rounded to nearest in fp32, the
// softmax's denominator summed in fp64 and rounded once (its value then does not depend on
// the order of the sum, up to about 2^-45).
#include <fp8q.h>

#include "device_common.h"
#include "launch.h"

namespace fp8q {
namespace {

constexpr int kWaves = 4;   // waves per workgroup, each with its own tokens

struct RouteArgs {
    const void *logits;
    const float *bias;
    float *weights;
    int32_t *experts;
    int64_t T;
    int E, k;
    int groups, topk_groups, per;   // per: experts per group
    int lane_shift;                 // log2 of the lanes that share a group
    int group_top2, renormalize;
    float scale;
};

// Order-preserving integer key of a float: a > b as floats is key(a) > key(b) as unsigned.
// Every key of a number is above 0; 0 stands for "no candidate". NaN ranks as -inf.
__device__ __forceinline__ uint32_t key_of(float c) {
    c = c != c ? -__builtin_inff() : c + 0.0f;   // (-0 ranks as +0)
    const uint32_t u = __float_as_uint(c);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// maximum over the wave's 64 lanes, the same in every lane
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = umax(v, dpp<0xB1>(v));            // quad_perm [1,0,3,2]
    v = umax(v, dpp<0x4E>(v));            // quad_perm [2,3,0,1]
    v = umax(v, dpp<0x141>(v));           // row_half_mirror
    v = umax(v, dpp<0x140>(v));           // row_mirror: every lane has its row's maximum
    v = umax(v, dpp<0x142, 0xA>(v));      // row_bcast15 into rows 1 and 3
    v = umax(v, dpp<0x143, 0xC>(v));      // row_bcast31 into rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// sum over the wave's 64 lanes, the same in every lane and of a fixed order
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    return v;
}

template <int BF16>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
    else return reinterpret_cast<const float *>(p)[i];
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// softmax's maximum and denominator from each lane's values (-inf where there is none);
// total = 0 when no value is above -inf, and every score is then 0
template <int V>
__device__ __forceinline__ void softmax_of(const float (&x)[V], float &top, float &total) {
    uint32_t m = key_of(x[0]);
#pragma unroll
    for (int i = 1; i < V; ++i) m = umax(m, key_of(x[i]));
    top = of_key(wave_max(m));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += (double)expf(x[i] - top);
    total = top == -__builtin_inff() ? 0.0f : (float)wave_sum(sum);
}

// One wave per token. Lane l belongs to group l >> lane_shift and holds V consecutive experts
// of it, so lane order is expert order, and a reduction over a group is one over a power of
// two of adjacent lanes.
template <int V, int BF16, int SOFTMAX>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const int lanes = 1 << a.lane_shift;
    const int group = lane >> a.lane_shift;
    const int at = (lane & (lanes - 1)) * V;                     // first expert within the group
    const int n = group < a.groups ? min(a.per - at, V) : 0;     // (may be negative: none)
    const int e0 = group * a.per + at;
    const int64_t row = t * a.E;

    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < n ? load_logit<BF16>(a.logits, row + e0 + i) : -__builtin_inff();
    float top = 0.0f, total = 1.0f;
    if constexpr (SOFTMAX) softmax_of<V>(x, top, total);
    auto score = [&](float v) {
        if constexpr (SOFTMAX) return total > 0.0f ? expf(v - top) / total : 0.0f;
        else return sigmoid(v);
    };
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = 0;
        if (i < n) key[i] = key_of(score(x[i]) + (a.bias ? a.bias[e0 + i] : 0.0f));
    }

    if (a.groups > 1) {
        uint32_t m1 = 0, m2 = 0;   // the two largest keys of the group
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m2 = umax(m2, m1 < key[i] ? m1 : key[i]);
            m1 = umax(m1, key[i]);
        }
        for (int d = 1; d < lanes; d <<= 1) {
            const uint32_t o1 = __shfl_xor(m1, d, 64), o2 = __shfl_xor(m2, d, 64);
            m2 = umax(umax(m2, o2), m1 < o1 ? m1 : o1);
            m1 = umax(m1, o1);
        }
        uint32_t value = m1;
        if (a.group_top2 && m2) value = key_of(of_key(m1) + of_key(m2));
        bool kept = false;
        for (int r = 0; r < a.topk_groups; ++r) {
            const uint32_t best = wave_max(value);
            const int owner = __builtin_ctzll(__ballot(value == best)) >> a.lane_shift;
            if (group == owner) {
                kept = true;
                value = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = kept ? key[i] : 0;
    }

    int mine = 0;   // lane j: the token's j-th expert
    for (int j = 0; j < a.k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = umax(m, key[i]);
        const uint32_t best = wave_max(m);
        const int owner = __builtin_ctzll(__ballot(m == best));
        int pos = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) pos = key[i] == best ? i : pos;
        const bool own = lane == owner;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = own && i == pos ? 0u : key[i];
        const int e = __builtin_amdgcn_readlane(e0 + pos, owner);
        mine = lane == j ? e : mine;
    }

    float s = 0.0f;
    if (lane < a.k) s = score(load_logit<BF16>(a.logits, row + mine));
    float w = s;
    if (a.renormalize) {
        const float sum = wave_sum(s);
        w = sum != 0.0f ? s / sum : 0.0f;   // (a token none of whose experts has a score has weights 0)
    }
    if (lane < a.k) {
        a.weights[t * a.k + lane] = w * a.scale;
        a.experts[t * a.k + lane] = mine;
    }
}

struct RouteGradArgs {
    const float *dweights;
    const void *logits;
    const int32_t *experts;
    void *dlogits;
    int64_t T;
    int E, k;
    int renormalize;
    float scale;
};

// Gradient of the logits, one wave per token (the selection itself has none):
//     g_j = scale * dw_j;   ds_j = (g_j - sum_i g_i s_i / S) / S, S = sum of the selected s
//     (renormalised), or g_j
//     sigmoid: dx_j = ds_j s_j (1 - s_j), 0 for the experts that were not selected
//     softmax: dx_i = s_i (ds_i - sum_j ds_j s_j), ds_i = 0 for those
// The row of ds goes through LDS, from the k selected experts' lanes to the experts' lanes.
template <int V, int BF16, int SOFTMAX>
__global__ __launch_bounds__(64 * kWaves) void route_grad_kernel(RouteGradArgs a) {
    __shared__ float rows[kWaves][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.T) return;
    float *ds_row = rows[wave];
    const int e0 = lane * V, n = min(a.E - e0, V);
    const int64_t row = t * a.E;

    float x[V], top = 0.0f, total = 1.0f;
    if constexpr (SOFTMAX) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < n ? load_logit<BF16>(a.logits, row + e0 + i) : -__builtin_inff();
        softmax_of<V>(x, top, total);
    }
    auto score = [&](float v) {
        if constexpr (SOFTMAX) return total > 0.0f ? expf(v - top) / total : 0.0f;
        else return sigmoid(v);
    };
#pragma unroll
    for (int i = 0; i < V; ++i) ds_row[i * 64 + lane] = 0.0f;

    const int e = lane < a.k ? a.experts[t * a.k + lane] : -1;
    const bool there = e >= 0 && e < a.E;
    const float xe = there ? load_logit<BF16>(a.logits, row + e) : 0.0f;
    const float s = there ? score(xe) : 0.0f;
    float d = there ? a.dweights[t * a.k + lane] * a.scale : 0.0f;
    if (a.renormalize) {
        const float sum = wave_sum(s), dot = wave_sum(d * s);
        d = there && sum != 0.0f ? (d - dot / sum) / sum : 0.0f;
    }
    const float all = SOFTMAX ? wave_sum(d * s) : 0.0f;
    if constexpr (!SOFTMAX) d *= s * (1.0f - s);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (there) ds_row[e] = d;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i < n) {
            float v = ds_row[e0 + i];
            if constexpr (SOFTMAX) v = score(x[i]) * (v - all);
            if constexpr (BF16) reinterpret_cast<uint16_t *>(a.dlogits)[row + e0 + i] = (uint16_t)pack_bf16x2(v, 0.0f);
            else reinterpret_cast<float *>(a.dlogits)[row + e0 + i] = v;
        }
    }
}

template <int V>
void route_v(const RouteArgs &a, bool bf16, bool softmax, dim3 grid, hipStream_t st) {
    const dim3 block(64 * kWaves);
    if (bf16) {
        if (softmax) route_kernel<V, 1, 1><<<grid, block, 0, st>>>(a);
        else route_kernel<V, 1, 0><<<grid, block, 0, st>>>(a);
    } else {
        if (softmax) route_kernel<V, 0, 1><<<grid, block, 0, st>>>(a);
        else route_kernel<V, 0, 0><<<grid, block, 0, st>>>(a);
    }
}

template <int V>
void route_grad_v(const RouteGradArgs &a, bool bf16, bool softmax, dim3 grid, hipStream_t st) {
    const dim3 block(64 * kWaves);
    if (bf16) {
        if (softmax) route_grad_kernel<V, 1, 1><<<grid, block, 0, st>>>(a);
        else route_grad_kernel<V, 1, 0><<<grid, block, 0, st>>>(a);
    } else {
        if (softmax) route_grad_kernel<V, 0, 1><<<grid, block, 0, st>>>(a);
        else route_grad_kernel<V, 0, 0><<<grid, block, 0, st>>>(a);
    }
}

}  // namespace

hipError_t launch_moe_route(const void *logits, bool bf16, const float *bias, float *weights, int32_t *experts,
                            int64_t T, int E, int k, int groups, int topk_groups, bool softmax, bool group_top2,
                            bool renormalize, float scale, hipStream_t stream) {
    RouteArgs a{logits, bias, weights, experts, T, E, k, groups, topk_groups, E / groups, 6, group_top2, renormalize,
                scale};
    for (int g = 1; g < groups; g <<= 1) --a.lane_shift;
    const int v = ((a.per - 1) >> a.lane_shift) + 1;   // experts per lane
    const dim3 grid((unsigned)((T + kWaves - 1) / kWaves));
    if (v <= 1) route_v<1>(a, bf16, softmax, grid, stream);
    else if (v <= 2) route_v<2>(a, bf16, softmax, grid, stream);
    else if (v <= 4) route_v<4>(a, bf16, softmax, grid, stream);
    else if (v <= 8) route_v<8>(a, bf16, softmax, grid, stream);
    else if (v <= 16) route_v<16>(a, bf16, softmax, grid, stream);
    else if (v <= 32) route_v<32>(a, bf16, softmax, grid, stream);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const float *dweights, const void *logits, bool bf16, const int32_t *experts,
                                     void *dlogits, int64_t T, int E, int k, bool softmax, bool renormalize,
                                     float scale, hipStream_t stream) {
    const RouteGradArgs a{dweights, logits, experts, dlogits, T, E, k, renormalize, scale};
    const dim3 grid((unsigned)((T + kWaves - 1) / kWaves));
    if (E <= 64) route_grad_v<1>(a, bf16, softmax, grid, stream);
    else if (E <= 128) route_grad_v<2>(a, bf16, softmax, grid, stream);
    else if (E <= 256) route_grad_v<4>(a, bf16, softmax, grid, stream);
    else if (E <= 512) route_grad_v<8>(a, bf16, softmax, grid, stream);
    else if (E <= 1024) route_grad_v<16>(a, bf16, softmax, grid, stream);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace fp8q
